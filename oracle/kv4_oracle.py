"""Plain float64 CPU oracle of the 4-bit KV cache: the cache's byte layout, block tables and
slot maps, and attention with its error bound. TEST INFRASTRUCTURE ONLY, like the rest of this
package. The quantizer's oracle is ``quantize_rtn_asym`` on rows [token * head, head_dim]."""
from __future__ import annotations

import numpy as np

__all__ = ["kv4_row_place", "kv4_pack_cache", "kv4_block_tables", "kv4_attention"]


def kv4_row_place(dim, key, token):
    """Where byte n (codes 2n and 2n + 1) of a row is stored within it: K rows have their
    32-bit words 4 j + c at c (dim/32) + j; V rows their bytes 8 i + g at g (dim/16) + i, and
    for 128 dims the halves exchanged on tokens with bit 1 set."""
    place = []
    for n in range(dim // 2):
        if key:
            word, byte = n // 4, n % 4
            place.append(4 * ((word % 4) * (dim // 32) + word // 4) + byte)
        else:
            at = (n % 8) * (dim // 16) + n // 8
            place.append((at + 32) % 64 if dim == 128 and token & 2 else at)
    return np.array(place)


def kv4_pack_cache(cache, slots, k, v, block):
    """Enter rows into `cache` uint8 [blocks, heads, bytes]: k = (codes [T, H, D], S [T, H, G],
    Z [T, H, G]), v likewise; token t at slots[t] (negative: skipped)."""
    codes = k[0]
    dim, groups = codes.shape[-1], k[1].shape[-1]
    for t, slot in enumerate(slots):
        if slot < 0:
            continue
        n, at = divmod(int(slot), block)
        for h in range(codes.shape[1]):
            chunk = cache[n, h]
            for key, (q, s, z) in ((True, k), (False, v)):
                row = q[t, h, 0::2] | q[t, h, 1::2] << 4
                base = (0 if key else block * dim // 2) + at * dim // 2
                chunk[base + kv4_row_place(dim, key, at)] = row
                base = block * dim + (0 if key else 4 * block * groups) + 4 * groups * at
                sz = np.stack((s[t, h], z[t, h]), -1).astype(np.float16)
                chunk[base: base + 4 * groups] = sz.view(np.uint8).ravel()


def kv4_block_tables(ctx, new, free, tables, block, n_slots):
    """(tables, slots, q_starts, kv_lens, taken) by counting, one token at a time."""
    tables, at, slots, starts = tables.copy(), 0, [], [0]
    for b, (c, n) in enumerate(zip(ctx, new)):
        for pos in range(c, c + n):
            if pos % block == 0:
                tables[b, pos // block] = free[at]
                at += 1
            slots.append(int(tables[b, pos // block]) * block + pos % block)
        starts.append(starts[-1] + n)
    slots += [-1] * (n_slots - len(slots))
    return tables, np.array(slots), np.array(starts), np.array(ctx) + np.array(new), at


def kv4_attention(q, k, v, scale, causal=True, window=0, s_max=None,
                  exact_values=False):
    """One request: q [n, heads, D], k and v [kv, kv_heads, D], float64. Returns (out, lse,
    bound_out, bound_lse): the formula's values, and how far a kernel may be from them before
    its output is rounded.

    The bound. A kernel's score is an fp32 sum of D/8 steps at most, of 16 exact products
    x (16 + q_code) S scale with 16 + q_code <= 31, minus x-sum (16 + Z) S scale, or of the
    products with both 16-bit parts of S (q - Z): each step and each of about 8 further fp32
    operations errs by at most 2^-23 of the largest magnitude in it, at most 31 S scale sum|x|
    (`s_max`: the largest S of the request's keys). Binary16 parts are of S (q - Z) 2^-E with the
    largest S 2^-E of the row's groups at 2^11 at least; S 2^-E of another may be a subnormal,
    half a step of 2^-24 off, times 15: 2^-32 of the largest S. That makes every probability
    wrong by a relative
        e = ((D/8 + 8) 2^-23 31 + 2^-32) S scale sum|x|
    at most, and numerator and denominator by e each; with it 2^-11 for its rounding to binary16
    (half a step) and 2^-11 for that of its value (`exact_values`: none, as with few rows or fp16
    results), 2^-20 for exp2, log2 and the scale products, and (kv/16 + 64) 2^-23 for the two fp32
    sums over the keys. The error of out is
    that times sum_j p_j |v_j|. Where a rounded p is a binary16 subnormal it errs by half its
    step, 2^-25. With p_j = 2^(s_j + E_j - m + c), c >= 6, and m at most the largest s_j + E_j of
    the row, key *'s, the sum of p_j 2^-E_j is at least 2^(6 - E_*) l, and the error that key j
    brings into out at most 2^-31 |v_j| 2^(E_* - E_j) / l. |v_j| is at most 15 S_j, S_j the key's
    largest. Few rows have E = log2 S: 2^-31 15 S_*. For prompts S_j < 2^(E_j + 5), and keys of one
    tile share E unless the exponents of their S differ by more than 6, so S_* >= 2^(E_* - 2):
    2^-24 15 S_*; where S 2^-E meets p, an error of 15 2^-25 and S_* >= 2^(E_* - 6): 2^-25. Where
    a rounded value S 2^-E (q - Z) of a prompt, or its S 2^-E, is a subnormal it errs by 15 2^-25,
    with the key's largest S 2^-E at 2^-2 at least: 2^-23 15 S. Only keys that the row sees come into
    this. 15 S <= 2.2 max_d |v_j| (the range 15 S lies within twice the largest stored value, each
    end of it within S/2), but S = 1 for a group of zeros, taken to be where 32 values are. For a
    masked row all of it is 0."""
    n, heads, dim = q.shape
    kv, kv_heads = k.shape[0], k.shape[1]
    out = np.zeros((n, heads, dim))
    lse = np.full((n, heads), -np.inf)
    bound = np.zeros((n, heads, dim))
    bound_lse = np.zeros((n, heads))
    ratio = heads // kv_heads
    for i in range(n):
        last = kv - n + i if causal else kv - 1
        first = max(0, last - window + 1) if window else 0
        if last < 0 or kv == 0:
            continue
        for h in range(heads):
            kk, vv = k[first: last + 1, h // ratio], v[first: last + 1, h // ratio]
            s = kk @ q[i, h] * scale
            m = s.max()
            p = np.exp(s - m)
            l = p.sum()
            out[i, h] = p @ vv / l
            lse[i, h] = m + np.log(l)
            e = 0.0
            if s_max is not None:
                e = ((dim / 8 + 8) * 2.0**-23 * 31 + 2.0**-32) * s_max * abs(scale) * np.abs(q[i, h]).sum()
            rel = 2 * e + (2.0**-11 if exact_values else 2.0**-10) + 2.0**-20 + (kv / 16 + 64) * 2.0**-23
            zeros = (vv.reshape(len(vv), -1, min(32, dim)) == 0).all(-1).any()
            top = max(2.2 * np.abs(vv).max(), 15.0 if zeros else 0.0)  # 15 S of the keys seen
            low = ((last + 1 - first) * 2.0**-24 / l + 2.0**-23) * top
            bound[i, h] = rel * (p @ np.abs(vv) / l) + low
            bound_lse[i, h] = e + 2.0**-20 * (1 + abs(lse[i, h])) + (kv / 16 + 64) * 2.0**-23
    return out, lse, bound, bound_lse

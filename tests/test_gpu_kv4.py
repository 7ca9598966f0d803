"""The 4-bit KV cache on a GPU against the float64 oracle: block tables and slot maps (equal),
append and read (bit for bit, the cache's bytes included), and attention within the bound that
the oracle derives for it, for single tokens, drafts and prompts; rows that see nothing, stale
and uninitialised memory, bad pages, strides, graphs, streams and a run of the operators
together."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import oracle  # noqa: E402
import w4a16_dequant_matmul_b200 as wq  # noqa: E402

DEV = "cuda"
BF16, F16 = torch.bfloat16, torch.float16
RANGE, NONFINITE = 9, 7


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


def ok():
    assert wq.wq_get_status() == 0


# ------------------------------------------------------------------------- block tables

def tables_case(ctx, new, block, extra_slots=0, extra_width=1, seed=0):
    rng = np.random.default_rng(seed)
    held = [-(-c // block) for c in ctx]
    need = [-(-(c + n) // block) for c, n in zip(ctx, new)]
    pool = rng.permutation(sum(need) + 3)
    tab = np.full((len(ctx), max(need + [0]) + extra_width), -7)
    at = 0
    for b, n in enumerate(held):
        tab[b, :n] = pool[at: at + n]
        at += n
    return tab, pool[at:], sum(new) + extra_slots


@pytest.mark.parametrize("ctx,new,block,extra", [
    ([0], [1], 16, 0), ([0], [0], 16, 3), ([15], [1], 16, 0), ([16], [1], 16, 0), ([31, 0, 5], [1, 1, 1], 32, 2),
    ([0, 0, 0, 0], [0, 17, 0, 64], 64, 5), ([100], [1000], 128, 1), ([1000], [513], 256, 0)])
def test_block_tables_small(ctx, new, block, extra):
    tab, free, n = tables_case(ctx, new, block, extra)
    want = oracle.kv4_block_tables(ctx, new, free, tab, block, n)
    got = ints(tab)
    slots, starts, kv, taken = wq.wq_kv4_block_tables(ints(ctx), ints(new), ints(free), got, block, n)
    ok()
    for g, w in zip((got, slots, starts, kv, taken), want):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))


@pytest.mark.parametrize("requests", [511, 512, 513, 1500])
@pytest.mark.parametrize("most", [1, 40])
def test_block_tables_many(requests, most):
    rng = np.random.default_rng(requests + most)
    ctx, new = rng.integers(0, 300, requests), rng.integers(0, most + 1, requests)
    tab, free, n = tables_case(ctx.tolist(), new.tolist(), 16, 11, 2, seed=requests)
    want = oracle.kv4_block_tables(ctx.tolist(), new.tolist(), free, tab, 16, n)
    wide = torch.full((requests, tab.shape[1] + 5), -9, dtype=torch.int32, device=DEV)
    got = wide[:, : tab.shape[1]]  # rows with a stride of their own
    got.copy_(ints(tab))
    for _ in range(2):  # repeating the call changes nothing
        out = wq.wq_kv4_block_tables(ints(ctx), ints(new), ints(free), got, 16, n)
        for g, w in zip((got, *out), want):
            assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))
    assert bool((wide[:, tab.shape[1]:] == -9).all())
    ok()


def test_block_tables_errors():
    """Each shortage is reported in the status word, the tokens concerned get slot -1 and what
    fits is right."""
    tab = ints(np.full((2, 2), -1))
    slots, *_ = wq.wq_kv4_block_tables(ints([0, 0]), ints([20, 20]), ints([5, 6, 7]), tab, 16, 40)
    assert wq.wq_get_status() == RANGE  # the fourth block is missing
    s = slots.cpu().numpy()
    assert (s[:36] >= 0).all() and (s[36:] == -1).all() and tab.cpu().tolist() == [[5, 6], [7, -1]]
    slots, starts, kv, taken = wq.wq_kv4_block_tables(ints([0]), ints([40]), ints([5, 6, 7]), ints([[-1, -1]]), 16, 40)
    assert wq.wq_get_status() == RANGE and (slots[32:] == -1).all() and kv.item() == 40  # width 2
    slots, *_ = wq.wq_kv4_block_tables(ints([3]), ints([2]), ints([1]), ints([[-1]]), 16, 2)
    assert wq.wq_get_status() == RANGE and (slots == -1).all()  # the held block is missing
    slots, starts, kv, taken = wq.wq_kv4_block_tables(ints([-4, 0]), ints([2, 2]), ints([3]), ints([[-1], [-1]]), 16, 4)
    assert wq.wq_get_status() == RANGE and starts.tolist() == [0, 0, 2] and kv.tolist() == [0, 2]
    assert slots.tolist() == [48, 49, -1, -1]
    slots, *_ = wq.wq_kv4_block_tables(ints([0]), ints([5]), ints([2]), ints([[-1]]), 16, 3)
    assert wq.wq_get_status() == RANGE and slots.tolist() == [32, 33, 34]  # more tokens than slots
    slots, starts, kv, taken = wq.wq_kv4_block_tables(ints([]), ints([]), ints([]), torch.empty(0, 0, dtype=torch.int32, device=DEV), 16, 2)
    assert slots.tolist() == [-1, -1] and starts.tolist() == [0] and taken.item() == 0
    ok()


# ---------------------------------------------------------------------- append and read

def quantized(x, group):
    """Oracle codes, S, Z of x [T, H, D] (float64 values)."""
    T, H, D = x.shape
    q, s, z = oracle.quantize_rtn_asym(x.reshape(-1, D), group)
    return q.reshape(x.shape), s.reshape(T, H, -1), z.reshape(T, H, -1)


def rows(T, H, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, D, generator=g, dtype=torch.float64) * (1 + 5 * (torch.rand(H, D, generator=g) < 0.05))
    x[0] = 0.0                      # S' = 0 -> 1
    if T > 3:
        x[1] = x[1].abs() + 0.25    # one-signed
        x[2] = torch.arange(D) - D // 2  # ties
        x[3] *= 1e-6                # subnormal scales
    return x.to(dtype)


@pytest.mark.parametrize("dim,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("block,T,H", [(16, 37, 3), (64, 70, 1), (256, 5, 2)])
def test_append_and_read(dim, group, dtype, block, T, H):
    k, v = rows(T, H, dim, dtype, 1), rows(T, H, dim, dtype, 2)
    blocks = -(-T // block) + 2
    rng = np.random.default_rng(T)
    slots = rng.permutation(blocks * block)[:T]
    slots[T // 2] = -1
    slots[-1] = -5
    cache = wq.wq_kv4_alloc(blocks, H, dim, group, block)
    cache.fill_(0xA5)
    want = cache.cpu().numpy().copy()
    kq, vq = quantized(k.double().numpy(), group), quantized(v.double().numpy(), group)
    oracle.kv4_pack_cache(want, slots, kq, vq, block)
    wq.wq_kv4_append(k.to(DEV), v.to(DEV), ints(slots), cache, group=group)
    ok()
    assert np.array_equal(cache.cpu().numpy(), want), "cache bytes"
    live = (slots >= 0)[:, None, None]
    for out_dtype in (torch.float32, BF16, F16):
        got = wq.wq_kv4_read(cache, ints(slots), dim, group=group, out_dtype=out_dtype)
        ok()
        for x, (q, s, z) in zip(got, (kq, vq)):
            exact = (s[..., None] * (q.reshape(T, H, -1, group) - z[..., None])).reshape(T, H, dim) * live
            assert torch.equal(x.cpu(), torch.from_numpy(exact).float().to(out_dtype))


@pytest.mark.parametrize("dim,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_append_where_codes_are_clipped(dim, group, dtype):
    """A few groups whose end codes leave [0, 15] before the clipping (a range just above 15 S'
    with ties at both ends, or a subnormal S' rounded far down) among ordinary ones, first in a
    warp alone, then together."""
    T, H, block = 96, 3, 64
    x = rows(T, H, dim, dtype, 5).double()
    x[3] = 1.0                                     # the other subnormal row of rows()
    tie, low, far = (-7.5, 7.5), (-20 * 2.0 ** -24, 0.0), (-10 * 2.0 ** -24, 10 * 2.0 ** -24)
    for t, h, g, ends in [(20, 1, 0, tie), (40, 2, dim // group - 1, low), (60, 0, 0, far),
                          (61, 1, 0, tie), (61, 2, 0, low)]:
        x[t, h, g * group:(g + 1) * group] = 0.0
        x[t, h, g * group:g * group + 2] = torch.tensor(ends, dtype=torch.float64)
    x = x.to(dtype)
    q, s, z = quantized(x.double().numpy(), group)
    exact = x.double().numpy().reshape(T, H, -1, group) / s[..., None]
    level = np.rint(exact) + z[..., None]
    assert (level > 15).any(-1).sum() >= 3 and (level < 0).any(-1).sum() >= 2  # the plan holds
    v = x.flip(0).contiguous()
    vq = quantized(v.double().numpy(), group)
    blocks = -(-T // block)
    cache = wq.wq_kv4_alloc(blocks, H, dim, group, block)
    cache.fill_(0x5A)
    want = cache.cpu().numpy().copy()
    oracle.kv4_pack_cache(want, np.arange(T), (q, s, z), vq, block)
    wq.wq_kv4_append(x.to(DEV), v.to(DEV), ints(np.arange(T)), cache, group=group)
    ok()
    assert np.array_equal(cache.cpu().numpy(), want)


@pytest.mark.parametrize("dim,group,dtype", [(128, 128, BF16), (128, 32, F16), (64, 64, F16), (64, 32, BF16)])
def test_append_many_equals_append_in_pieces(dim, group, dtype):
    """A call large enough for several rounds a warp stores what small calls do, tokens in any
    order, some skipped, the last round ragged."""
    T, H, block = 12345, 5 if dim == 128 else 11, 64
    g = torch.Generator(device=DEV).manual_seed(dim + group)
    k, v = (torch.randn(2, T, H, dim, generator=g, device=DEV) * 3).to(dtype).unbind(0)
    slots = torch.randperm(T + 100, generator=g, device=DEV)[:T].int()
    slots[::97] = -1
    a = wq.wq_kv4_alloc(-(-(T + 100) // block), H, dim, group, block)
    a.zero_()
    b = a.clone()
    wq.wq_kv4_append(k, v, slots, a, group=group)
    for i in range(0, T, 500):
        wq.wq_kv4_append(k[i: i + 500], v[i: i + 500], slots[i: i + 500], b, group=group)
    ok()
    assert torch.equal(a, b)
    some = [1, 5000, T - 1]
    got, _ = wq.wq_kv4_read(a, slots[some], dim, group=group)
    q, s, z = quantized(k[some].double().cpu().numpy(), group)
    exact = (s[..., None] * (q.reshape(3, H, -1, group) - z[..., None])).reshape(3, H, dim)
    assert np.array_equal(got.double().cpu().numpy(), exact)


def test_append_strided():
    """K and V as slices of a fused projection's output, heads in another order in memory."""
    T, H, D = 19, 4, 64
    x = torch.randn(T, 3 * H * D, device=DEV).to(BF16)
    k = x[:, H * D: 2 * H * D].unflatten(-1, (H, D))
    v = torch.randn(H, T, D, device=DEV).to(BF16).transpose(0, 1)
    slots = ints(np.arange(T) + 3)
    a, b = wq.wq_kv4_alloc(2, H, D, 32, 16), wq.wq_kv4_alloc(2, H, D, 32, 16)
    a.zero_(), b.zero_()
    wq.wq_kv4_append(k, v, slots, a, group=32)
    wq.wq_kv4_append(k.contiguous(), v.contiguous(), slots, b, group=32)
    assert torch.equal(a, b) and bool(a.any())
    ok()


def test_append_reports_bad_input():
    cache = wq.wq_kv4_alloc(2, 1, 64, 32, 16)
    cache.zero_()
    k = torch.ones(3, 1, 64, device=DEV, dtype=BF16)
    bad = k.clone()
    bad[1, 0, 40] = float("nan")
    bad[2, 0, 3] = float("inf")
    wq.wq_kv4_append(bad, k, ints([0, 1, 2]), cache, group=32)
    assert wq.wq_get_status() == NONFINITE
    got, _ = wq.wq_kv4_read(cache, ints([0, 1, 2]), 64, group=32)
    one = 15 * float(np.float16(1 / 15))  # S' q of a row of ones
    assert bool((got[1, 0, :32] == one).all()) and not bool(got[1, 0, 32:].any()) and not bool(got[2, 0, :32].any())
    before = cache.clone()
    wq.wq_kv4_append(k, k, ints([32, -1, 1 << 30]), cache, group=32)  # 32 slots: 0 .. 31
    assert wq.wq_get_status() == RANGE and torch.equal(cache, before)
    got, _ = wq.wq_kv4_read(cache, ints([32, -1, 0]), 64, group=32)
    assert wq.wq_get_status() == RANGE and not bool(got[:2].any()) and bool(got[2].all())
    huge = torch.full((1, 1, 64), 1e30, device=DEV, dtype=BF16)  # S' passes binary16
    wq.wq_kv4_append(huge, huge, ints([5]), cache, group=32)
    assert wq.wq_get_status() == NONFINITE


def test_slots_past_32_bits_of_bytes():
    """A cache of more than 2^32 bytes: its last blocks are written and read."""
    blocks = (1 << 32) // (16 * 8 * 136) + 100
    cache = wq.wq_kv4_alloc(blocks, 8, 128, 128, 16)
    assert cache.numel() > 1 << 32
    T = 7
    k, v = rows(T, 8, 128, BF16, 3), rows(T, 8, 128, BF16, 4)
    slots = ints(np.arange(T) + (blocks - 1) * 16 + 4)
    wq.wq_kv4_append(k.to(DEV), v.to(DEV), slots, cache)
    got = wq.wq_kv4_read(cache, slots, 128)
    ok()
    for x, w in zip(got, (k, v)):
        q, s, z = quantized(w.double().numpy(), 128)
        assert np.array_equal(x.double().cpu().numpy(), s * (q - z))
    table = torch.full((1, 1), blocks - 1, dtype=torch.int32, device=DEV)
    q = torch.randn(1, 8, 128, device=DEV).to(BF16)
    small = cache[blocks - 1:].clone()
    a = wq.wq_kv4_attention(q, cache, table, ints([0, 1]), ints([9]), 1)
    b = wq.wq_kv4_attention(q, small, table * 0, ints([0, 1]), ints([9]), 1)
    ok()
    assert torch.equal(a, b)


# --------------------------------------------------------------------------- attention

class Case:
    """A cache with quantized random keys and values, everything else in it hostile: stale
    blocks and the tails of the last ones hold random bytes, their scales NaN and infinities."""

    def __init__(self, kv_lens, q_lens, heads, kv_heads, dim, group, block, dtype, seed=0, spread=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.kv_lens, self.q_lens, self.dim, self.group, self.dtype = kv_lens, q_lens, dim, group, dtype
        need = [-(-n // block) for n in kv_lens]
        blocks = sum(need) + 2
        self.cache = wq.wq_kv4_alloc(blocks, kv_heads, dim, group, block)
        self.cache.copy_(torch.randint(0, 256, self.cache.shape, generator=g, device=DEV, dtype=torch.uint8))
        half = block * dim
        self.cache[..., half:].view(torch.float16)[...] = float("nan")
        self.cache[..., half::8] = 0
        order, at = rng.permutation(blocks), 0
        tab = np.full((len(kv_lens), max(need + [1]) + 1), -1)
        self.k, self.v, self.smax = [], [], []
        for b, n in enumerate(need):
            tab[b, :n] = order[at: at + n]
            at += n
            m = kv_lens[b]
            slots = ints([tab[b, j // block] * block + j % block for j in range(m)])
            k = (torch.randn(m, kv_heads, dim, generator=g, device=DEV) * spread).to(dtype)
            v = (torch.randn(m, kv_heads, dim, generator=g, device=DEV) * (0.1 + torch.rand(m, kv_heads, 1, generator=g, device=DEV) * 3)).to(dtype)
            wq.wq_kv4_append(k, v, slots, self.cache, group=group)
            kk, vv = wq.wq_kv4_read(self.cache, slots, dim, group=group)
            self.k.append(kk.double().cpu().numpy())
            self.v.append(vv.double().cpu().numpy())
            x = k.float().unflatten(-1, (-1, group))
            span = (x.amax(-1).clamp(min=0) - x.amin(-1).clamp(max=0)) / 15 * (1 + 2.0**-11)
            self.smax.append(float(span.max()) if m else 0.0)
        self.tables, self.kv = ints(tab), ints(kv_lens)
        self.starts = ints(np.concatenate(([0], np.cumsum(q_lens))))
        T = sum(q_lens)
        self.q = torch.randn(T, heads, dim, generator=g, device=DEV).to(dtype)
        ok()

    def run(self, **kw):
        kw = {"causal": True, "window": 0, **kw}
        max_q = kw.pop("max_q", max(self.q_lens + [1]))
        return wq.wq_kv4_attention(self.q, self.cache, self.tables, self.starts, self.kv, max_q, group=self.group, return_lse=True, **kw)

    def check(self, out, lse, scale=None, causal=True, window=0):
        scale = self.dim ** -0.5 if scale is None else scale
        half_step = torch.finfo(self.dtype).eps / 2
        tiny = float(torch.finfo(self.dtype).smallest_normal) * half_step
        at = 0
        for b, n in enumerate(self.q_lens):
            q = self.q[at: at + n].double().cpu().numpy()
            want, wlse, bound, blse = oracle.kv4_attention(q, self.k[b], self.v[b], scale, causal, window, s_max=self.smax[b])
            got = out[at: at + n].double().cpu().numpy()
            gl = lse[at: at + n].double().cpu().numpy()
            limit = bound + (np.abs(want) + bound) * half_step + tiny
            assert np.isfinite(got).all()
            worst = np.max((np.abs(got - want) - limit).ravel(), initial=-1)
            assert worst <= 0, f"request {b}: {np.max(np.abs(got - want) / (limit + 1e-300)):.3g} of the bound"
            assert np.array_equal(np.isneginf(gl), np.isneginf(wlse))
            f = np.isfinite(wlse)
            assert (np.abs(gl[f] - wlse[f]) <= blse[f]).all(), f"lse of request {b}"
            at += n


SHAPES = [(128, 128), (128, 64), (128, 32), (64, 64), (64, 32)]


@pytest.mark.parametrize("dim,group", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_decode_one_token(dim, group, dtype):
    for kv in (1, 2, 15, 16, 17, 63, 64, 65, 300):
        c = Case([kv], [1], 8, 2, dim, group, 16, dtype, seed=kv)
        c.check(*c.run())
        ok()


@pytest.mark.parametrize("dim,group", SHAPES)
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 3), (7, 1), (8, 1), (9, 1), (16, 1), (33, 3), (40, 2)])
def test_decode_head_layouts(dim, group, heads, kv_heads):
    c = Case([77, 0, 130], [1, 1, 1], heads, kv_heads, dim, group, 32, BF16, seed=heads)
    c.check(*c.run())
    ok()


@pytest.mark.parametrize("block", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dim,group", [(128, 128), (64, 32)])
def test_decode_ragged_batch(block, dim, group):
    """Lengths of all kinds, an empty place among them; pages end inside a tile."""
    c = Case([0, 1, 257, 64, 1000, 31, 128, 513], [1] * 8, 8, 2, dim, group, block, BF16, seed=block)
    c.check(*c.run())
    ok()


@pytest.mark.parametrize("q_lens", [[1, 0, 2, 5], [3, 3, 3, 3], [8, 1, 30, 2]])
@pytest.mark.parametrize("dim,group,dtype", [(128, 128, BF16), (128, 32, F16), (64, 64, F16)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 7), (True, 100), (False, 0), (False, 33)])
def test_drafts(q_lens, dim, group, dtype, causal, window):
    """Several queries a request, the first of them before its keys where a request is short."""
    c = Case([200, 3, 1, 66], q_lens, 12, 4, dim, group, 16, dtype, seed=sum(q_lens))
    c.check(*c.run(causal=causal, window=window), causal=causal, window=window)
    ok()


@pytest.mark.parametrize("dim,group,dtype", [(128, 128, BF16), (128, 128, F16), (128, 64, BF16), (64, 64, BF16), (64, 32, F16)])
@pytest.mark.parametrize("q_lens,kv_lens", [([130], [130]), ([64, 1, 0, 200], [64, 300, 5, 333]), ([129], [700]), ([50, 33], [20, 33])])
@pytest.mark.parametrize("heads,kv_heads", [(4, 4), (8, 2), (7, 1)])
def test_prompts(dim, group, dtype, q_lens, kv_lens, heads, kv_heads):
    c = Case(kv_lens, q_lens, heads, kv_heads, dim, group, 32, dtype, seed=heads)
    c.check(*c.run())
    ok()


@pytest.mark.parametrize("causal,window", [(True, 1), (True, 65), (False, 0), (False, 50)])
@pytest.mark.parametrize("block", [16, 64, 128])
def test_prompt_masks(causal, window, block):
    c = Case([140, 300], [140, 90], 8, 2, 128, 128, block, BF16, seed=block)
    c.check(*c.run(causal=causal, window=window), causal=causal, window=window)
    ok()


def test_scales_and_sharp_softmax():
    """Scores of hundreds (the running maximum moves far and often), a scale of 0 (the mean of
    the values), a negative one."""
    for scale, spread in ((0.5, 4.0), (0.0, 1.0), (-0.1, 1.0)):
        for q_lens in ([1, 2], [40, 1]):
            c = Case([400, 90], q_lens, 8, 2, 128, 128, 16, BF16, seed=5, spread=spread)
            c.check(*c.run(scale=scale), scale=scale)
    ok()


def test_far_apart_value_scales():
    """Values whose scales lie 2^20 apart: a token of weight near 1 with tiny values beside
    ones of little weight with large values."""
    c = Case([130], [1], 4, 1, 64, 64, 16, F16, seed=9)
    v = torch.randn(130, 1, 64, device=DEV) * torch.exp2(torch.randint(-14, 7, (130, 1, 1), device=DEV).float())
    k = torch.randn(130, 1, 64, device=DEV)
    slots = c.tables[0].long()[torch.arange(130, device=DEV) // 16] * 16 + torch.arange(130, device=DEV) % 16
    wq.wq_kv4_append(k.half(), v.half(), slots.int(), c.cache, group=64)
    kk, vv = wq.wq_kv4_read(c.cache, slots.int(), 64, group=64)
    c.k, c.v = [kk.double().cpu().numpy()], [vv.double().cpu().numpy()]
    c.smax = [float((k.half().float().amax(-1).clamp(min=0) - k.half().float().amin(-1).clamp(max=0)).max()) / 15 * 1.001]
    c.check(*c.run())
    ok()


def test_long_context_split_over_the_grid():
    """One request whose keys are spread over every CTA, against torch in float64."""
    kv, heads, kv_heads, dim = 40000, 8, 1, 128
    cache = wq.wq_kv4_alloc(kv // 64 + 1, kv_heads, dim)
    k, v = torch.randn(2, kv, kv_heads, dim, device=DEV).to(BF16).unbind(0)
    slots = torch.arange(kv, device=DEV, dtype=torch.int32)
    wq.wq_kv4_append(k, v, slots, cache)
    kk, vv = wq.wq_kv4_read(cache, slots, dim)
    q = torch.randn(1, heads, dim, device=DEV).to(BF16)
    table = torch.arange(cache.shape[0], device=DEV, dtype=torch.int32)[None]
    out, lse = wq.wq_kv4_attention(q, cache, table, ints([0, 1]), ints([kv]), 1, return_lse=True)
    ok()
    s = torch.einsum("hd,kd->hk", q[0].double(), kk[:, 0].double()) * dim**-0.5
    p = torch.softmax(s, 1)
    want = p @ vv[:, 0].double()
    # rounding of p 2^-11, of out 2^-8, sums and scores as in the oracle's bound (kv/16 steps)
    size = p @ vv[:, 0].double().abs()
    limit = size * (2.0**-11 + 2.0**-14 + kv / 16 * 2.0**-23) + want.abs() * 2.0**-8
    assert bool(((out[0].double() - want).abs() <= limit).all())
    assert torch.allclose(lse[0].double(), torch.logsumexp(s, 1), rtol=0, atol=1e-4)
    again = wq.wq_kv4_attention(q, cache, table, ints([0, 1]), ints([kv]), 1)
    assert torch.equal(out, again), "deterministic"


def dense(cache, table, kv, dim, group, block):
    slots = table.long()[torch.arange(kv, device=DEV) // block] * block + torch.arange(kv, device=DEV) % block
    return (x.double() for x in wq.wq_kv4_read(cache, slots.int(), dim, group=group))


@pytest.mark.parametrize("dim,group,dtype", [(128, 128, BF16), (128, 128, F16), (128, 64, BF16), (128, 32, F16), (64, 64, BF16), (64, 32, F16)])
@pytest.mark.parametrize("new,kv,heads,kv_heads,window", [(700, 3001, 4, 2, 0), (333, 2000, 7, 1, 900), (1, 9000, 24, 1, 0), (300, 1500, 75, 75, 0)])
def test_long_prompts(dim, group, dtype, new, kv, heads, kv_heads, window):
    """Many tiles of keys (every ring goes round several times), split over CTAs and (75 heads)
    not, values whose scale grows a
    thousandfold along the keys, against torch in float64."""
    block = 32
    g = torch.Generator(device=DEV).manual_seed(kv)
    blocks = -(-kv // block)
    cache = wq.wq_kv4_alloc(blocks, kv_heads, dim, group, block)
    table = torch.randperm(blocks, generator=g, device=DEV).int()[None]
    slots = table[0].long()[torch.arange(kv, device=DEV) // block] * block + torch.arange(kv, device=DEV) % block
    k, v = torch.randn(2, kv, kv_heads, dim, generator=g, device=DEV).unbind(0)
    v = v * torch.exp2(torch.linspace(-6, 4, kv, device=DEV))[:, None, None]
    wq.wq_kv4_append(k.to(dtype), v.to(dtype), slots.int(), cache, group=group)
    q = torch.randn(new, heads, dim, generator=g, device=DEV).to(dtype)
    out, lse = wq.wq_kv4_attention(q, cache, table, ints([0, new]), ints([kv]), new, group=group, window=window, return_lse=True)
    ok()
    kk, vv = dense(cache, table[0], kv, dim, group, block)
    s_max = 8 / 15  # of keys within 4 standard deviations to both sides
    last = torch.arange(new, device=DEV)[:, None] + kv - new
    hidden = torch.arange(kv, device=DEV) > last
    if window:
        hidden |= torch.arange(kv, device=DEV) <= last - window
    for h in range(heads):
        x = q[:, h].double()
        s = (x @ kk[:, h * kv_heads // heads].T * dim**-0.5).masked_fill(hidden, -float("inf"))
        p = torch.softmax(s, 1)
        vh = vv[:, h * kv_heads // heads]
        want = p @ vh
        # the oracle's bound of a request, by rows
        e = ((dim / 8 + 8) * 2.0**-23 * 31 * s_max + 2.0**-21) * dim**-0.5 * x.abs().sum(1)
        rel = 2 * e + 2.0**-10 + 2.0**-20 + (kv / 16 + 64) * 2.0**-23
        limit = rel[:, None] * (p @ vh.abs()) + (kv * 2.0**-31 + 2.0**-29) * 2.2 * vh.abs().max()
        half_step = torch.finfo(dtype).eps / 2
        limit = limit + (want.abs() + limit) * half_step
        assert bool(((out[:, h].double() - want).abs() <= limit).all()), h
        wl = torch.logsumexp(s, 1)
        bound = e + 2.0**-20 * (1 + wl.abs()) + (kv / 16 + 64) * 2.0**-23
        assert bool(((lse[:, h].double() - wl).abs() <= bound).all()), h
    again = wq.wq_kv4_attention(q, cache, table, ints([0, new]), ints([kv]), new, group=group, window=window)
    assert torch.equal(out, again), "deterministic"


def test_bad_pages_and_lengths():
    """Table entries outside the cache and lengths beyond the table: reported, those keys left
    out, the rest right, other requests untouched."""
    for q_lens in ([1, 1, 1], [40, 1, 1]):
        c = Case([100, 90, 50], q_lens, 4, 2, 128, 128, 16, BF16, seed=3)
        good = c.run()
        ok()
        tab = c.tables.clone()
        tab[1, 2], tab[1, 4] = -1, 1 << 20
        keep = c.tables
        c.tables = tab
        out, lse = c.run()
        assert wq.wq_get_status() == RANGE
        n = q_lens[0]
        assert torch.equal(out[:n], good[0][:n]) and torch.equal(out[n + 1:], good[0][n + 1:])
        seen = np.r_[0:32, 48:64, 80:90]
        s = np.einsum("hd,khd->hk", c.q[n].double().cpu().numpy(), np.repeat(c.k[1][seen], 2, 1)) * 128**-0.5
        p = np.exp(s - s.max(1, keepdims=True))
        want = np.einsum("hk,khd->hd", p / p.sum(1, keepdims=True), np.repeat(c.v[1][seen], 2, 1))
        assert np.abs(out[n].double().cpu().numpy() - want).max() < 2.0**-7 * np.abs(want).max()
        c.tables = keep[:, :2].contiguous()  # 32 tokens
        out, lse = c.run()
        assert wq.wq_get_status() == RANGE and bool(torch.isfinite(out).all())


def test_rows_behind_the_last_are_left():
    for q_lens in ([1, 2], [60, 1]):
        c = Case([90, 33], q_lens, 4, 2, 64, 64, 16, F16, seed=1)
        T = sum(q_lens)
        q = torch.cat((c.q, torch.full((5, 4, 64), float("nan"), device=DEV, dtype=F16)))
        out = torch.full((T + 5, 4, 64), 7.0, device=DEV, dtype=F16)
        got, lse = wq.wq_kv4_attention(q, c.cache, c.tables, c.starts, c.kv, max(q_lens), group=64, out=out, return_lse=True)
        ok()
        assert got is out and bool((out[T:] == 7).all())
        c.check(out[:T], lse[:T])


def test_strided_queries_and_outputs():
    for q_lens in ([2, 1], [70, 3]):
        c = Case([90, 33], q_lens, 4, 2, 128, 128, 16, BF16, seed=2)
        T = sum(q_lens)
        wide = torch.zeros(T, 6, 136, device=DEV, dtype=BF16)
        wide[:, 1:5, :128] = c.q
        out = torch.zeros(4, T, 256, device=DEV, dtype=BF16)
        view = out.transpose(0, 1)[..., 128:]
        got = wq.wq_kv4_attention(wide[:, 1:5, :128], c.cache, c.tables, c.starts, c.kv, max(q_lens), out=view)
        ok()
        assert torch.equal(got, c.run()[0]) and not bool(out[..., :128].any())


def test_a_wrong_max_q_changes_no_result():
    c = Case([300, 90, 64], [80, 1, 20], 8, 2, 128, 128, 32, BF16, seed=4)
    for max_q in (0, 1, 80, 5000):
        c.check(*c.run(max_q=max_q))
    ok()


def test_one_request_with_a_wrong_max_q():
    for n in (1, 3, 90):
        c = Case([300], [n], 8, 2, 64, 32, 32, F16, seed=n)
        for max_q in (0, 1, 4000):
            c.check(*c.run(max_q=max_q))
    ok()


def test_a_row_that_is_not_finite_stays_alone():
    """NaN and infinity in one query row change no other row, of its tile or its request."""
    for q_lens in ([1, 4], [60, 3]):
        c = Case([200, 90], q_lens, 8, 2, 128, 128, 16, BF16, seed=7)
        good, glse = c.run()
        for bad in (float("nan"), float("inf")):
            keep = c.q.clone()
            c.q[0, 1] = bad
            out, lse = c.run()
            mask = torch.ones_like(glse, dtype=torch.bool)
            mask[0, 1] = False
            assert torch.equal(out[mask], good[mask]) and torch.equal(lse[mask], glse[mask])
            assert bool(torch.isnan(out[0, 1]).all())
            c.q = keep
    ok()


def test_many_requests():
    """More requests than threads of a CTA."""
    rng = np.random.default_rng(0)
    kv = rng.integers(0, 70, 700).tolist()
    c = Case(kv, [1] * 700, 2, 1, 64, 64, 16, BF16, seed=11)
    out, lse = c.run()
    ok()
    c.check(out, lse)


def test_graph_streams_and_workspaces():
    """Captured and replayed with other contents; two streams with a workspace each; one
    workspace for two graphs that run one after the other."""
    c = Case([500, 70, 128], [1, 1, 1], 8, 2, 128, 128, 16, BF16, seed=6)
    c.run()
    ws = torch.full((wq.wq_kv4_attention_workspace_bytes(),), 0xFF, dtype=torch.uint8, device=DEV)
    out1, out2 = torch.zeros_like(c.q), torch.zeros_like(c.q)
    q2 = c.q * 2
    graphs = []
    for q, out in ((c.q, out1), (q2, out2)):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            wq.wq_kv4_attention(q, c.cache, c.tables, c.starts, c.kv, 1, out=out, workspace=ws)
        graphs.append(g)
    want2 = wq.wq_kv4_attention(q2, c.cache, c.tables, c.starts, c.kv, 1)
    for _ in range(3):
        out1.zero_(), out2.zero_()
        for g in graphs:
            g.replay()
        assert torch.equal(out1, c.run()[0]) and torch.equal(out2, want2)
    # other lengths and contents in the same buffers
    c.kv.copy_(ints([200, 0, 17]))
    graphs[0].replay()
    c.kv_lens, c.k, c.v = [200, 0, 17], [x[:n] for x, n in zip(c.k, (200, 0, 17))], [x[:n] for x, n in zip(c.v, (200, 0, 17))]
    c.check(out1, c.run()[1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(c.run()[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs)
    ok()


def test_prompt_and_storage_in_a_graph():
    """A whole step captured (tables, append, attention of a prompt and a single token) and
    replayed with other lengths and contents."""
    heads, kv_heads, dim, block = 8, 2, 64, 16
    ctx, new = ints([0, 40]), ints([50, 1])
    tables = torch.full((2, 8), -1, dtype=torch.int32, device=DEV)
    tables[1, :3] = ints([20, 21, 22])
    free = ints(np.arange(12))
    cache = wq.wq_kv4_alloc(24, kv_heads, dim, dim, block)
    cache.zero_()
    x = torch.randn(64, 2, kv_heads, dim, device=DEV).to(F16)
    q = torch.randn(64, heads, dim, device=DEV).to(F16)
    out = torch.zeros_like(q)

    def step():
        slots, starts, kv, taken = wq.wq_kv4_block_tables(ctx, new, free, tables, block, 64)
        wq.wq_kv4_append(x[:, 0], x[:, 1], slots, cache)
        wq.wq_kv4_attention(q, cache, tables, starts, kv, 50, out=out)

    keep = tables.clone()
    step()
    eager = out.clone()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
    out.zero_(), cache.zero_(), tables.copy_(keep)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:51], eager[:51]) and not bool(out[51:].any())
    q.normal_(), x.normal_(), new.copy_(ints([3, 1])), out.zero_(), cache.zero_(), tables.copy_(keep)
    g.replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    out.zero_(), cache.zero_(), tables.copy_(keep)
    step()
    ok()
    assert torch.equal(replayed, out) and bool(out[:4].any()) and not bool(out[4:].any())


def test_a_serving_run():
    """The operators as they are used together: prompts are admitted, appended and attended,
    then tokens are decoded one by one, a prompt joining in between; each step's attention
    against the oracle on what the cache holds by then."""
    heads, kv_heads, dim, block, budget = 8, 2, 128, 16, 64
    cache = wq.wq_kv4_alloc(40, kv_heads, dim, dim, block)
    tables = torch.full((3, 12), -1, dtype=torch.int32, device=DEV)
    free = torch.from_numpy(np.random.default_rng(0).permutation(40)).int().to(DEV)
    ctx, held = np.zeros(3, int), [[np.zeros((0, kv_heads, dim))] * 2 for _ in range(3)]
    used = 0
    g = torch.Generator(device=DEV).manual_seed(0)
    for new in ([37, 0, 20], [1, 0, 1], [1, 50, 1], [1, 1, 1], [1, 1, 0], [1, 1, 1]):
        n = sum(new)
        slots, starts, kv, taken = wq.wq_kv4_block_tables(ints(ctx), ints(new), free[used:], tables, block, budget)
        q = torch.randn(budget, heads, dim, generator=g, device=DEV).to(BF16)
        k, v = torch.randn(2, budget, kv_heads, dim, generator=g, device=DEV).to(BF16).unbind(0)
        wq.wq_kv4_append(k, v, slots, cache)
        out, lse = wq.wq_kv4_attention(q, cache, tables, starts, kv, max(new), return_lse=True)
        ok()
        used += taken.item()
        kq, vq = quantized(k[:n].double().cpu().numpy(), dim), quantized(v[:n].double().cpu().numpy(), dim)
        kk, vv = (x[1] * (x[0] - x[2]) for x in (kq, vq))
        at = 0
        for b in range(3):
            held[b] = [np.concatenate((old, x[at: at + new[b]])) for old, x in zip(held[b], (kk, vv))]
            want, wl, bound, bl = oracle.kv4_attention(q[at: at + new[b]].double().cpu().numpy(), *held[b], dim**-0.5, s_max=1.0)
            got = out[at: at + new[b]].double().cpu().numpy()
            assert (np.abs(got - want) <= bound + (np.abs(want) + bound) * 2.0**-8).all()
            assert (np.abs(lse[at: at + new[b]].double().cpu().numpy() - wl) <= bl).all()
            at += new[b]
        ctx += np.array(new)
    assert kv.tolist() == ctx.tolist()


# ------------------------------------------------------- ranges of scores and of value scales

def refill(c, k, v):
    """Other keys and values [kv, kv_heads, dim] (float) for a Case of one request."""
    block = c.cache.shape[2] // (c.dim + 8 * c.dim // c.group)
    at = torch.arange(c.kv_lens[0], device=DEV)
    slots = (c.tables[0].long()[at // block] * block + at % block).int()
    k, v = k.to(c.dtype), v.to(c.dtype)
    wq.wq_kv4_append(k, v, slots, c.cache, group=c.group)
    kk, vv = wq.wq_kv4_read(c.cache, slots, c.dim, group=c.group)
    ok()
    c.k, c.v = [kk.double().cpu().numpy()], [vv.double().cpu().numpy()]
    x = k.double().unflatten(-1, (-1, c.group))
    span = (x.amax(-1).clamp(min=0) - x.amin(-1).clamp(max=0)) / 15
    c.smax = [float(torch.where(span < 2.0**-25, 1.0, span * (1 + 2.0**-11) + 2.0**-25).max())]


@pytest.mark.parametrize("dim,group", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_score_and_value_scale_jump_in_one_tile(dim, group, dtype):
    """The third tile of keys brings value scales 2^14 as large and scores far above all before:
    the sums of the rows are rescaled for both in one step."""
    kv, heads, kv_heads = 450, 8, 2
    c = Case([kv], [33], heads, kv_heads, dim, group, 32, dtype, seed=12)
    g = torch.Generator(device=DEV).manual_seed(12)
    k, v = torch.randn(2, kv, kv_heads, dim, generator=g, device=DEV).unbind(0)
    k[256:] *= 12
    v[:256] *= 2.0**-7
    v[256:] *= 2.0**7
    refill(c, k, v)
    c.check(*c.run())
    ok()


def test_calls_on_given_streams():
    """Calls with `stream=` from one current stream, on two others in turn, each with a workspace
    and results of its own: a long request split over the grid, so that every call has parts in
    its workspace, as results under the stream and after other allocations of the current one."""
    c = Case([6000, 77], [1, 2], 8, 2, 128, 128, 32, BF16, seed=13)
    want, wlse = c.run()
    streams = [torch.cuda.Stream() for _ in range(2)]
    slots = ints(np.arange(64))
    k, v = wq.wq_kv4_read(c.cache, slots, 128)
    x = torch.randn(64, 2, 128, device=DEV).to(BF16)
    other = [torch.zeros_like(c.cache) for _ in streams]
    free, ctx, new = ints(np.arange(10)), ints([0, 0]), ints([100, 40])
    tab = [torch.full((2, 8), -1, dtype=torch.int32, device=DEV) for _ in streams]
    wq.wq_kv4_append(x, x, slots, want_cache := torch.zeros_like(c.cache))
    wtab = tab[0].clone()
    wslots = wq.wq_kv4_block_tables(ctx, new, free, wtab, 16, 150)[0]
    torch.cuda.synchronize()
    outs = []
    for i in range(20):
        for s, t, o in zip(streams, tab, other):
            outs.append((*c.run(stream=s), *wq.wq_kv4_read(c.cache, slots, 128, stream=s),
                         wq.wq_kv4_block_tables(ctx, new, free, t, 16, 150, stream=s)[0]))
            wq.wq_kv4_append(x, x, slots, o, stream=s)
            torch.full((1 << 20,), -1.0, device=DEV)  # takes up what the current stream let go
    torch.cuda.synchronize()
    ok()
    for got in outs:
        for a, b in zip(got, (want, wlse, k, v, wslots)):
            assert torch.equal(a, b)
    assert all(torch.equal(t, wtab) for t in tab) and all(torch.equal(o, want_cache) for o in other)


@pytest.mark.parametrize("dim,group", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("spread", [3e-3, 2e-4, 1e-5, 6e3])
def test_small_and_large_keys(dim, group, dtype, spread):
    """Keys from where their scales are binary16 subnormals to where S (q - Z) nears the largest
    binary16 number, with a softmax scale that brings the scores back to a few units: as a
    prompt and, by a max_q of 0, on the kernel for few rows. Groups of a key lie up to 2^6
    apart."""
    kv, heads, kv_heads = 200, 4, 2
    c = Case([kv], [20], heads, kv_heads, dim, group, 16, dtype, seed=14)
    g = torch.Generator(device=DEV).manual_seed(14)
    k, v = torch.randn(2, kv, kv_heads, dim, generator=g, device=DEV).unbind(0)
    apart = torch.randint(0, 7, (kv, kv_heads, dim // group, 1), generator=g, device=DEV)
    k = (k.unflatten(-1, (-1, group)) * torch.exp2(-apart.float())).flatten(-2) * spread
    refill(c, k, v)
    scale = dim**-0.5 / spread
    for max_q in (20, 0):
        c.check(*c.run(scale=scale, max_q=max_q), scale=scale)
    ok()


@pytest.mark.parametrize("dim,group", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("where", ["later", "one_later", "behind", "zeros", "mixed", "near"])
def test_value_scales_that_a_row_does_not_see(dim, group, dtype, where):
    """Values 2^22 as large on keys that most rows of the tile do not see (later ones, one only,
    those behind the window) take no bits from the others; rows of zeros (S' = 1) and scales from
    all over the range, or within 2^6, among small values."""
    kv, heads, kv_heads, window = 230, 4, 2, 0
    c = Case([kv], [kv if where in ("later", "one_later") else 100], heads, kv_heads, dim, group, 16, dtype, seed=15)
    g = torch.Generator(device=DEV).manual_seed(15)
    k, v = torch.randn(2, kv, kv_heads, dim, generator=g, device=DEV).unbind(0)
    v *= 2.0**-10
    if where == "later":
        v[100:] *= 2.0**22
    elif where == "one_later":
        v[90] *= 2.0**22
        v[200, 1] *= 2.0**22
    elif where == "behind":
        window = 50
        v[:81] *= 2.0**22
    elif where == "zeros":
        v[::3] = 0
    elif where == "near":  # one exponent a tile, the key of most weight with the smallest values
        v *= torch.exp2(torch.randint(0, 6, (kv, kv_heads, 1), generator=g, device=DEV).float())
        k[5], v[5] = c.q[-1, ::2].float() * 2, v[5] * 2.0**-5
    else:
        v *= torch.exp2(torch.randint(-4, 21, (kv, kv_heads, 1), generator=g, device=DEV).float())
    refill(c, k, v)
    c.check(*c.run(window=window), window=window)
    ok()


def test_hidden_keys_of_a_long_prompt():
    """Rows of a prompt of many tiles, split over CTAs and not, hold while the values of later
    keys grow 2^22 times: each side is off by half a step of out, and by 2^-10 (p and v rounded,
    the smaller terms below 2^-11) of the largest value."""
    cut = 300
    for kv, heads in ((1500, 2), (700, 80)):
        c = Case([kv], [kv], heads, heads // 2, 128, 128, 32, BF16, seed=16)
        g = torch.Generator(device=DEV).manual_seed(16)
        k, v = torch.randn(2, kv, heads // 2, 128, generator=g, device=DEV).unbind(0)
        v *= 2.0**-10
        refill(c, k, v)
        a, la = c.run()
        v[cut:] *= 2.0**22
        refill(c, k, v)
        b, lb = c.run()
        ok()
        off = (a[:cut].double() - b[:cut].double()).abs()
        limit = 2 * (2.0**-10 + 2.0**-11) * float(v[:cut].abs().max())
        assert bool((off <= limit + 2.0**-7 * (a[:cut].double().abs() + limit)).all())
        assert torch.allclose(la[:cut], lb[:cut], rtol=0, atol=1e-4)


@pytest.mark.parametrize("q_lens", [[1, 1], [40, 40]])
@pytest.mark.parametrize("entry", [-1, -2, -(1 << 31), 1 << 20, (1 << 31) - 1, "blocks"])
def test_each_bad_entry_is_reported(q_lens, entry):
    """One needed table entry outside the cache, the first number past it among them."""
    c = Case([100, 90], q_lens, 8, 2, 128, 128, 16, BF16, seed=17)
    c.run()
    ok()
    c.tables[1, 3] = c.cache.shape[0] if entry == "blocks" else entry
    out, lse = c.run()
    assert wq.wq_get_status() == RANGE and bool(torch.isfinite(out).all())


@pytest.mark.parametrize("block", [16, 64, 128, 256])
@pytest.mark.parametrize("q_lens", [[1, 3], [40, 1], [300, 70]])
@pytest.mark.parametrize("causal,window", [(True, 1), (True, 37), (True, 200), (False, 50)])
def test_blocks_behind_the_window_may_be_gone(block, q_lens, causal, window):
    """A server gives back the blocks that no later row sees: their table entries are not read.
    An entry that is needed is still reported."""
    c = Case([700, 523], q_lens, 8, 2, 128, 64, block, F16, seed=block)
    c.check(*c.run(causal=causal, window=window), causal=causal, window=window)
    tab = c.tables.clone()
    for b, n in enumerate(q_lens):
        first = max(0, c.kv_lens[b] - (n - 1 if causal else 0) - window)
        tab[b, : first // block] = -1
        tab[b, : first // block: 2] = 1 << 20
    c.tables = tab
    c.check(*c.run(causal=causal, window=window), causal=causal, window=window)
    ok()
    first = max(0, c.kv_lens[1] - (q_lens[1] - 1 if causal else 0) - window)
    tab[1, first // block] = -1
    c.run(causal=causal, window=window)
    assert wq.wq_get_status() == RANGE


@pytest.mark.parametrize("starts", [[0, 300, 0, 300], [0, 250, 200, 300], [-5, 100, 200, 300], [0, 100, 200, 301],
                                    [300, 200, 100, 0], [0, 1 << 30, -(1 << 30), 300]])
def test_row_starts_that_do_not_ascend_are_reported(starts):
    """Whatever q_starts hold, rows inside Q are written or left, and the status says so."""
    c = Case([400, 350, 330], [100, 100, 100], 8, 2, 128, 128, 32, BF16, seed=18)
    c.run()
    ok()
    c.starts = ints(starts)
    for max_q in (100, 0):
        out, _ = c.run(max_q=max_q, out=torch.zeros_like(c.q))
        assert wq.wq_get_status() == RANGE and bool(torch.isfinite(out).all())
    one = wq.wq_kv4_attention(c.q, c.cache, c.tables[:1], ints([10, 5]), c.kv[:1], 100, out=torch.zeros_like(c.q))
    assert wq.wq_get_status() == RANGE and not bool(one.any())


def test_requests_may_leave_rows_between_them():
    """Starts that ascend with the first above 0 and the last below T are no error."""
    c = Case([400, 350], [100, 30], 8, 2, 128, 128, 32, BF16, seed=19)
    want, _ = c.run()
    q = torch.cat((c.q[:7] * 0, c.q, c.q[:9] * 0))
    out = torch.full_like(q, 3.0)
    wq.wq_kv4_attention(q, c.cache, c.tables, c.starts + 7, c.kv, 100, out=out)
    ok()
    assert torch.equal(out[7:-9], want) and bool((out[:7] == 3).all()) and bool((out[-9:] == 3).all())


def test_block_tables_of_wild_lengths():
    """Lengths near 2^31 of many requests: reported, what fits is right, and the call takes no
    longer for them."""
    B, n = 5000, (1 << 31) - 300
    tab = torch.full((B, 4), -1, dtype=torch.int32, device=DEV)
    args = (ints([0] * B), ints([n] * B), ints([5, 6, 7]), tab, 16, 100)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    slots, starts, kv, taken = wq.wq_kv4_block_tables(*args)
    end.record()
    assert wq.wq_get_status() == RANGE
    assert start.elapsed_time(end) < 100
    assert slots.tolist() == [16 * (5 + i // 16) + i % 16 for i in range(48)] + [-1] * 52
    assert tab[0].tolist() == [5, 6, 7, -1] and bool((tab[1:] == -1).all()) and taken.item() == 3
    assert starts[:3].tolist() == [0, n, (1 << 31) - 1] and bool((kv == n).all())


@pytest.mark.parametrize("dim,group", SHAPES)
@pytest.mark.parametrize("dtype,q_lens", [(BF16, [1, 2]), (F16, [1, 2]), (F16, [90, 1])])
def test_values_are_exact(dim, group, dtype, q_lens):
    """Few rows, and fp16 results: of the two operands of the second product only the
    probabilities are rounded."""
    c = Case([300, 77], q_lens, 8, 2, dim, group, 64, dtype, seed=20)
    out, lse = c.run()
    ok()
    half_step, at = torch.finfo(dtype).eps / 2, 0
    tiny = float(torch.finfo(dtype).smallest_normal) * half_step
    for b, n in enumerate(q_lens):
        q = c.q[at: at + n].double().cpu().numpy()
        want, _, bound, _ = oracle.kv4_attention(q, c.k[b], c.v[b], dim**-0.5, s_max=c.smax[b], exact_values=True)
        got = out[at: at + n].double().cpu().numpy()
        assert (np.abs(got - want) <= bound + (np.abs(want) + bound) * half_step + tiny).all()
        at += n


@pytest.mark.parametrize("dim,group", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("block", [128, 256])
def test_prompts_over_large_blocks(dim, group, dtype, block):
    """Blocks of one tile and of two, the last one ragged in either half."""
    c = Case([700, 380, 129], [60, 150, 129], 8, 2, dim, group, block, dtype, seed=block)
    c.check(*c.run())
    c.check(*c.run(causal=False, window=300), causal=False, window=300)
    ok()


@pytest.mark.parametrize("heads,kv_heads", [(300, 1), (130, 2), (256, 1)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_very_many_query_heads_a_kv_head(heads, kv_heads, dtype):
    """A token's rows pass a row tile, and several; as prompts and on the kernel for few rows."""
    c = Case([150, 40], [1, 2], heads, kv_heads, 64, 32, 16, dtype, seed=21)
    for max_q in (2, 0):
        c.check(*c.run(max_q=max_q))
    ok()


def test_prompts_among_many_requests():
    """More requests than threads of either kernel, a few of them prompts."""
    rng = np.random.default_rng(1)
    q_lens = np.ones(600, int)
    q_lens[[3, 511, 512, 599]] = 40, 70, 0, 33
    c = Case((q_lens + rng.integers(0, 50, 600)).tolist(), q_lens.tolist(), 8, 2, 64, 64, 16, BF16, seed=22)
    c.check(*c.run())
    ok()


def test_requests_without_rows_only():
    c = Case([30, 0, 7], [1, 0, 0], 8, 2, 64, 64, 16, BF16, seed=23)
    for max_q in (1, 100):
        out = torch.full_like(c.q, 5.0)
        wq.wq_kv4_attention(c.q, c.cache, c.tables, c.starts * 0, c.kv, max_q, out=out)
        ok()
        assert bool((out == 5).all())

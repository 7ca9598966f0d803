"""Model check of the barrier protocol of the prompt attention over the 4-bit KV cache
(kv4_prompt.cu): its roles played by Python generators under random schedules, the tensor core
a FIFO of issued MMAs that completes them in order at random times, a commit arriving once every
MMA issued before it has completed.

  producer   per tile j of keys: wait rk_empty (tile j - 1 read), write there[j % 4], copy K's
             codes and the scales -> rk_full; wait rv_empty, copy V's codes -> rv_full
  expand     4 warps; per tile: wait rk_full and k_empty[j % KB], read there, write exponent and
             vec [j % 4] and K's operand, arrive k_full, vec_full[j % 4] and rk_empty; wait
             rv_full and v_empty[j % VB], read there, write V's operand, arrive v_full, rv_empty
  MMA lane   S_0, S_1 of tile 0; per tile: wait v_full; per row tile i: wait p_full[i], issue
             O_i += P_i V, wait k_full of the next tile, issue the next S_i, commit s_full[i];
             commit v_empty and the next tile's k_empty; at last commit o_full
  softmax    two row tiles of SW warps; per tile: wait s_full[i] and vec_full[j % 4], read S_i,
             vec, exponent and there, rescale O_i, write P_i over S_i, arrive p_full[i]

The rings of four (there, exponent, vec) have no barrier that says they are free. Asserted: a
wait that passes sees the fill that it names; nothing is overwritten that a warp or a queued MMA
has still to read; the softmax touches O_i only when no product into it is queued; every schedule
ends. Planted mistakes (a missing wait) must be caught.
"""
import random

import pytest

from test_gemm_protocol import Bar

NW = 4  # expand warps


def run_prompt_protocol(tiles, KB, VB, SW, seed, skip=()):
    rnd = random.Random(seed)
    rk_full, rk_empty, rv_full, rv_empty = Bar(1), Bar(NW), Bar(1), Bar(NW)
    k_full, k_empty = [Bar(NW) for _ in range(KB)], [Bar(1) for _ in range(KB)]
    v_full, v_empty = [Bar(NW) for _ in range(VB)], [Bar(1) for _ in range(VB)]
    vec_full = [Bar(NW) for _ in range(4)]
    s_full, p_full, o_full = [Bar(1), Bar(1)], [Bar(SW), Bar(SW)], Bar(1)
    inflight, fifo = [], []  # copies not landed; issued MMAs and commits
    raw_k, raw_v = [None, 0], [None, 0]  # tile in the raw buffers, warps that have still to read it
    there = [[None, 0] for _ in range(4)]  # tile, reads to come
    vec = [[None, 0, 0] for _ in range(4)]  # tile, warps that wrote it, reads to come
    ops = {"k": [[None, 0, 0] for _ in range(KB)], "v": [[None, 0, 0] for _ in range(VB)]}
    S = [None, None]   # tile whose scores S_i holds (all of them, once completed)
    P = [[None, 0], [None, 0]]
    o_busy = [0, 0]    # products into O_i in the queue
    done = [0, 0]      # products into O_i completed

    def wait(bar, parity, use):
        while not bar.ready(parity):
            yield
        assert bar.phase == use + 1, ("a wait passed in another phase", use, bar.phase)

    def producer():
        for j in range(tiles):
            if j and "rk_empty" not in skip:
                yield from wait(rk_empty, (j - 1) & 1, j - 1)
            assert there[j & 3][1] == 0, ("there overwritten", j)
            there[j & 3][:] = [j, 2 * NW + 2 * SW]
            assert raw_k[1] == 0, ("raw K overwritten", j)
            raw_k[:] = [j, NW]
            rk_full.expect(j, 1)
            inflight.append(rk_full)
            yield
            if j and "rv_empty" not in skip:
                yield from wait(rv_empty, (j - 1) & 1, j - 1)
            assert raw_v[1] == 0, ("raw V overwritten", j)
            raw_v[:] = [j, NW]
            rv_full.expect(j, 1)
            inflight.append(rv_full)
            yield

    def write(op, buf, j):
        o = ops[op][buf]
        assert o[2] == 0, (op, "rewritten under a queued MMA", j)
        if o[0] != j:
            assert o[0] is None or o[1] == NW
            o[0], o[1] = j, 0
        o[1] += 1

    def expand():
        for j in range(tiles):
            kb, vb = j % KB, j % VB
            yield from wait(rk_full, j & 1, j)
            if j >= KB and "k_empty" not in skip:
                yield from wait(k_empty[kb], (j // KB - 1) & 1, j // KB - 1)
            assert raw_k[0] == j and there[j & 3][0] == j
            r = vec[j & 3]
            if r[0] != j:
                assert r[2] == 0, ("vec overwritten", j)
                r[:] = [j, 0, 2 * SW]
            yield
            there[j & 3][1] -= 1
            r[1] += 1
            write("k", kb, j)
            raw_k[1] -= 1
            yield
            k_full[kb].arrive()
            yield
            vec_full[j & 3].arrive()
            yield
            rk_empty.arrive()
            yield from wait(rv_full, j & 1, j)
            if j >= VB and "v_empty" not in skip:
                yield from wait(v_empty[vb], (j // VB - 1) & 1, j // VB - 1)
            assert raw_v[0] == j and there[j & 3][0] == j
            yield
            there[j & 3][1] -= 1
            write("v", vb, j)
            raw_v[1] -= 1
            yield
            v_full[vb].arrive()
            rv_empty.arrive()

    def issue(kind, i, j, buf):
        o = ops["k" if kind == "S" else "v"][buf]
        assert o[0] == j and o[1] == NW, (kind, "on an unfinished operand", j)
        o[2] += 1
        if kind == "O":
            o_busy[i] += 1
        fifo.append((kind, i, j, o))

    def mma():
        yield from wait(k_full[0], 0, 0)
        for i in range(2):
            issue("S", i, 0, 0)
            fifo.append(("commit", s_full[i]))
        fifo.append(("commit", k_empty[0]))
        yield
        for j in range(tiles):
            vb, kb = j % VB, (j + 1) % KB
            yield from wait(v_full[vb], (j // VB) & 1, j // VB)
            for i in range(2):
                if "p_full" not in skip:
                    yield from wait(p_full[i], j & 1, j)
                issue("O", i, j, vb)
                if j + 1 < tiles:
                    if i == 0:
                        yield from wait(k_full[kb], ((j + 1) // KB) & 1, (j + 1) // KB)
                    issue("S", i, j + 1, kb)
                    fifo.append(("commit", s_full[i]))
                yield
            fifo.append(("commit", v_empty[vb]))
            if j + 1 < tiles:
                fifo.append(("commit", k_empty[kb]))
        fifo.append(("commit", o_full))

    def softmax(i):
        for j in range(tiles):
            yield from wait(s_full[i], j & 1, j)
            yield from wait(vec_full[j & 3], (j >> 2) & 1, j >> 2)
            assert S[i] == j, ("scores of another tile", i, j, S[i])
            assert there[j & 3][0] == j and vec[j & 3][0] == j and vec[j & 3][1] == NW, ("ring", j)
            assert o_busy[i] == 0 and done[i] == j, ("O touched under a product", i, j)
            yield
            there[j & 3][1] -= 1
            vec[j & 3][2] -= 1
            if P[i][0] != j:
                P[i][:] = [j, 0]
            P[i][1] += 1
            yield
            p_full[i].arrive()
        yield from wait(o_full, 0, 0)
        assert done[i] == tiles and o_busy[i] == 0

    def complete():
        what = fifo.pop(0)
        if what[0] == "commit":
            what[1].arrive()
            return
        kind, i, j, o = what
        o[2] -= 1
        if kind == "S":
            assert j == 0 or (P[i] == [j - 1, SW] and done[i] == j), ("P overwritten", i, j)
            S[i] = j
        else:
            assert P[i] == [j, SW], ("product of unfinished probabilities", i, j)
            o_busy[i] -= 1
            done[i] += 1

    alive = [producer(), mma()] + [expand() for _ in range(NW)] + [softmax(i % 2) for i in range(2 * SW)]
    # some warps are much slower than others in a schedule
    weights = {id(g): rnd.choice((1, 1, 4, 20)) for g in alive}
    steps = 0
    while alive or inflight or fifo:
        steps += 1
        if steps > 300000:
            raise RuntimeError("deadlock")
        r = rnd.random()
        if inflight and (not alive or r < 0.2):
            inflight.pop(rnd.randrange(len(inflight))).land(1)
        elif fifo and (not alive or r < 0.4):
            complete()
        elif alive:
            g = rnd.choices(alive, [weights[id(x)] for x in alive])[0]
            try:
                next(g)
            except StopIteration:
                alive.remove(g)


@pytest.mark.parametrize("tiles", [1, 2, 3, 7, 14])
@pytest.mark.parametrize("KB,VB", [(2, 2), (1, 2), (1, 1)])
def test_prompt_protocol_random_schedules(tiles, KB, VB):
    for seed in range(12):
        run_prompt_protocol(tiles, KB, VB, SW=2, seed=seed * 7919 + tiles)


@pytest.mark.parametrize("wait,KB", [("rk_empty", 2), ("rv_empty", 2), ("k_empty", 1), ("v_empty", 2), ("p_full", 2)])
def test_prompt_model_catches_a_missing_wait(wait, KB):
    """(vec_full comes no later than the scores and orders memory only; with K two deep as V is,
    k_empty comes no later than v_empty of the tile before: neither can be missed here.)"""
    caught = 0
    for seed in range(40):
        try:
            run_prompt_protocol(9, KB, 2, SW=2, seed=seed, skip=(wait,))
        except (AssertionError, RuntimeError):
            caught += 1
    assert caught > 0

"""4-bit KV cache on the host: argument checks of the C entry points and of the binding (no
kernel runs; fake pointers are never dereferenced), the oracle's pins, and the cases'
arithmetic of the cache layout."""
import ctypes

import numpy as np
import pytest

import oracle
import w4a16_dequant_matmul_b200 as wq
from w4a16_dequant_matmul_b200 import _build

torch = pytest.importorskip("torch")

OK, NULL, SHAPE, ALIGN, DTYPE, UNSUP, NODEV = 0, 1, 2, 3, 4, 5, 10
F, ODD = 0x10000, 0x10008


@pytest.fixture(scope="module")
def lib():
    _build.build_library()
    return wq.lib()


def cache(data=F, blocks=8, heads=2, dim=128, group=128, block=64):
    return wq._KV4_CACHE.pack(data, blocks, heads, dim, group, block)


def test_cache_bytes():
    assert wq.wq_kv4_cache_bytes(1, 1, 128) == 64 * (128 + 8)
    assert wq.wq_kv4_cache_bytes(10, 3, 64, 32, 16) == 10 * 3 * 16 * (64 + 16)
    assert wq.wq_kv4_cache_bytes(40000, 8, 128, 128, 256) == 40000 * 8 * 256 * 136  # past 2^31
    for bad in (dict(head_dim=96), dict(head_dim=256), dict(group=16), dict(group=48),
                dict(block_size=8), dict(block_size=48), dict(block_size=512), dict(kv_heads=0),
                dict(num_blocks=-1), dict(num_blocks=1 << 26)):
        kw = {**dict(num_blocks=4, kv_heads=2, head_dim=128, group=128, block_size=64), **bad}
        assert wq.wq_kv4_cache_bytes(**kw) == 0, bad
    assert wq.wq_kv4_cache_bytes(4, 2, 64, 128) == 0  # group > head_dim
    with pytest.raises(wq.WQError):
        wq.wq_kv4_alloc(4, 2, 96, device="cpu")
    assert wq.wq_kv4_alloc(4, 2, 64, 32, 16, device="cpu").shape == (4, 2, 16 * 80)
    assert wq.wq_kv4_alloc(0, 2, 64, device="cpu").shape[0] == 0


def test_append_checks(lib):
    def f(K=F, V=F, dt=wq.WQ_BF16, T=4, kt=256, kh=128, vt=256, vh=128, slots=F, c=None):
        return lib.wq_kv4_append(K, V, dt, T, kt, kh, vt, vh, slots, c or cache(), None)

    assert f(T=-1) == SHAPE
    assert f(T=0, K=None, V=None, slots=None) == OK
    assert f(dt=wq.WQ_F32) == DTYPE
    assert f(K=None) == NULL and f(V=None) == NULL and f(slots=None) == NULL
    assert f(c=cache(data=0)) == NULL
    assert f(K=ODD) == ALIGN and f(V=ODD) == ALIGN and f(slots=F + 2) == ALIGN
    assert f(kt=257) == ALIGN and f(vh=4) == ALIGN and f(c=cache(data=ODD)) == ALIGN
    assert f(kt=-256) == SHAPE
    assert f(c=cache(dim=80)) == UNSUP and f(c=cache(block=40)) == UNSUP
    assert f(c=cache(dim=64, group=128)) == SHAPE and f(c=cache(heads=0)) == SHAPE
    assert lib.wq_kv4_append(F, F, wq.WQ_BF16, 4, 256, 128, 256, 128, F, None, None) == NULL


def test_read_checks(lib):
    def f(c=None, slots=F, T=4, K=F, V=F, dt=wq.WQ_F32):
        return lib.wq_kv4_read(c or cache(), slots, T, K, V, dt, None)

    assert f(T=-1) == SHAPE and f(T=0, K=None) == OK and f(dt=wq.WQ_U8) == DTYPE
    assert f(slots=None) == NULL and f(K=None) == NULL and f(V=None) == NULL
    assert f(K=ODD) == ALIGN and f(slots=F + 1) == ALIGN and f(c=cache(dim=32)) == UNSUP


def test_block_tables_checks(lib):
    def f(ctx=F, new=F, B=4, free=F, nf=8, bs=64, tab=F, w=4, ld=4, slots=F, ns=16, qs=F, kv=F,
          taken=F):
        return lib.wq_kv4_block_tables(ctx, new, B, free, nf, bs, tab, w, ld, slots, ns, qs, kv,
                                       taken, None)

    assert f(B=-1) == SHAPE and f(nf=-1) == SHAPE and f(w=-1) == SHAPE and f(ns=-1) == SHAPE
    assert f(ld=3) == SHAPE and f(ns=1 << 31) == SHAPE
    assert f(bs=8) == UNSUP and f(bs=100) == UNSUP
    for name in ("ctx", "new", "free", "tab", "slots", "qs", "kv", "taken"):
        assert f(**{name: None}) == NULL, name
        assert f(**{name: F + 2}) == ALIGN, name


def attention_args(**kw):
    d = dict(Q=F, T=4, qt=512, qh=128, c=None, tab=F, w=4, ld=4, qs=F, kv=F, B=2, out=2 * F, ot=512,
             oh=128, lse=F, ws=F, wsb=1 << 40, dt=wq.WQ_BF16, heads=4, mq=2, causal=1, win=0,
             scale=0.1)
    d.update(kw)
    c = wq._KV4_CACHE.unpack(d["c"] or cache())
    return wq._KV4_ATTENTION.pack(d["Q"], d["T"], d["qt"], d["qh"], *c, d["tab"], d["w"], d["ld"],
                                  d["qs"], d["kv"], d["B"], d["out"], d["ot"], d["oh"], d["lse"],
                                  d["ws"], d["wsb"], d["dt"], d["heads"], d["mq"], d["causal"],
                                  d["win"], d["scale"])


def test_attention_checks(lib):
    def f(**kw):
        return lib.wq_kv4_attention(attention_args(**kw), None)

    assert lib.wq_kv4_attention(None, None) == NULL
    assert f(T=0, Q=0) == OK and f(B=0, qs=0) == OK
    for bad in (dict(T=-1), dict(B=-1), dict(heads=0), dict(heads=3), dict(mq=-1), dict(win=-1),
                dict(win=(1 << 30) + 1), dict(w=-1), dict(ld=3), dict(scale=float("inf")),
                dict(scale=float("nan")), dict(qt=-8), dict(T=1 << 30), dict(B=65537)):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(Q=0), dict(qs=0), dict(kv=0), dict(out=0), dict(ws=0), dict(tab=0),
                dict(c=cache(data=0))):
        assert f(**bad) == NULL, bad
    for bad in (dict(Q=ODD), dict(out=ODD), dict(ws=ODD), dict(lse=F + 2), dict(qs=F + 1),
                dict(qt=516), dict(qh=4), dict(ot=4), dict(oh=1)):
        assert f(**bad) == ALIGN, bad
    assert f(dt=wq.WQ_F32) == DTYPE
    assert f(c=cache(dim=72)) == UNSUP and f(out=F) == UNSUP  # in place


@pytest.mark.skipif(torch.cuda.is_available(), reason="host without a GPU only")
def test_valid_calls_without_device_report_nodevice(lib):
    assert lib.wq_kv4_append(F, F, wq.WQ_BF16, 4, 256, 128, 256, 128, F, cache(), None) == NODEV
    assert lib.wq_kv4_read(cache(), F, 4, F, F, wq.WQ_F32, None) == NODEV
    assert lib.wq_kv4_attention(attention_args(), None) == NODEV
    assert lib.wq_kv4_block_tables(F, F, 2, F, 4, 64, F, 4, 4, F, 8, F, F, F, None) == NODEV


def test_binding_refuses():
    ints = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    c = wq.wq_kv4_alloc(4, 2, 64, 32, 16, device="cpu")
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        wq.wq_kv4_append(x, x, torch.zeros(3, dtype=torch.int64), c, group=32)
    with pytest.raises(ValueError):
        wq.wq_kv4_append(x, x, ints(4), c, group=32)
    with pytest.raises(ValueError):
        wq.wq_kv4_append(x, x.half(), ints(3), c, group=32)
    with pytest.raises(ValueError):
        wq.wq_kv4_append(x[:, :1], x[:, :1], ints(3), c, group=32)
    with pytest.raises(TypeError):
        wq.wq_kv4_append(x.float(), x.float(), ints(3), c, group=32)
    with pytest.raises(ValueError):
        wq.wq_kv4_append(x.transpose(1, 2).contiguous().transpose(1, 2), x, ints(3), c, group=32)
    with pytest.raises(ValueError):  # the bytes are not those of group 64, block 16 .. 256
        wq.wq_kv4_read(c[:, :, :-16], ints(3), 64, group=32)
    with pytest.raises(ValueError):
        wq.wq_kv4_attention(x, c, ints(2, 4), ints(2), ints(2), 1, group=32)
    with pytest.raises(ValueError):
        wq.wq_kv4_attention(x, c, ints(1, 4), ints(3), ints(2), 1, group=32)
    with pytest.raises(ValueError):
        wq.wq_kv4_block_tables(ints(2), ints(3), ints(4), ints(2, 4), 16, 8)


def test_binding_makes_the_tensors_device_current(monkeypatch):
    """A call on tensors of another device than the current one is made with theirs current, and
    the current one is back afterwards (host-side stand-ins: no GPU is touched)."""
    current, seen = [0], []

    class Dev:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            self.prev, current[0] = current[0], self.d

        def __exit__(self, *exc):
            current[0] = self.prev

    k = wq._kv4()
    stub = type("Stub", (), dict(vars(k)))()
    stub.device, stub.current_device = Dev, lambda: current[0]
    stub.raw_stream = lambda d: 77
    stub.empty = lambda shape, strides, dtype, device: torch.empty(shape, dtype=dtype)

    def call(name):
        def f(*args):
            seen.append((name, current[0], args[-1]))
            return 0
        return f

    for name in ("block_tables", "append", "read", "attention"):
        setattr(stub, name, call(name))
    stub.workspace_bytes = {1: 16}
    monkeypatch.setattr(wq, "_KV4", stub)

    class OnOne(torch.Tensor):
        """A host tensor that says it is on device 1."""
        def get_device(self):
            return 1

        device = property(lambda self: 1)

    one = lambda t: t.as_subclass(OnOne)  # noqa: E731
    ints = lambda *s: one(torch.zeros(s, dtype=torch.int32))  # noqa: E731
    c = one(wq.wq_kv4_alloc(4, 2, 64, 32, 16, device="cpu"))
    x = one(torch.zeros(3, 2, 64, dtype=torch.bfloat16))
    wq.wq_kv4_append(x, x, ints(3), c, group=32)
    wq.wq_kv4_read(c, ints(3), 64, group=32)
    wq.wq_kv4_block_tables(ints(2), ints(2), ints(4), ints(2, 4), 16, 8)
    wq.wq_kv4_attention(x, c, ints(1, 4), ints(2), ints(1), 3, group=32)
    assert seen == [(n, 1, 77) for n in ("append", "read", "block_tables", "attention")]
    assert current == [0]


@pytest.mark.parametrize("dim", [64, 128])
def test_layout_is_a_permutation(dim):
    for key in (True, False):
        for token in range(4):
            p = oracle.kv4_row_place(dim, key, token)
            assert sorted(p) == list(range(dim // 2))


def test_oracle_attention_pins():
    """Closed forms: equal scores give the mean of the values seen, one key its own value, and
    keys in ratio 2 : 1 of weight their weighted mean; no key gives 0 and -inf."""
    rng = np.random.default_rng(0)
    v = rng.normal(size=(6, 1, 4))
    q = np.zeros((3, 2, 4))
    out, lse, _, _ = oracle.kv4_attention(q, rng.normal(size=(6, 1, 4)), v, 1.0)
    for i in range(3):
        assert np.allclose(out[i, 0], v[: 4 + i, 0].mean(0)) and np.isclose(lse[i, 1], np.log(4 + i))
    out, _, _, _ = oracle.kv4_attention(q, v, v, 1.0, window=1)
    assert np.allclose(out[:, 0], v[3:, 0])
    k = np.zeros((2, 1, 4))
    k[0, 0, 0] = np.log(2)
    x = np.zeros((1, 1, 4))
    x[0, 0, 0] = 1
    out, lse, _, _ = oracle.kv4_attention(x, k, v[:2], 1.0)
    assert np.allclose(out[0, 0], (2 * v[0, 0] + v[1, 0]) / 3) and np.isclose(lse[0, 0], np.log(3))
    out, lse, _, _ = oracle.kv4_attention(q, v[:2], v[:2], 1.0)
    assert not out[0].any() and np.all(np.isneginf(lse[0])) and np.allclose(out[1, 0], v[0, 0])
    out, _, _, _ = oracle.kv4_attention(q, v, v, 1.0, causal=False, window=2)
    assert np.allclose(out[0, 0], v[4:, 0].mean(0))


def test_oracle_block_tables_pin():
    tab = np.full((3, 3), -1)
    tab[0, 0] = 7
    t, slots, starts, kv, taken = oracle.kv4_block_tables([15, 0, 0], [3, 0, 17], [2, 9, 4], tab, 16, 22)
    assert t.tolist() == [[7, 2, -1], [-1, -1, -1], [9, 4, -1]]
    assert slots.tolist() == [7 * 16 + 15, 32, 33] + [9 * 16 + i for i in range(16)] + [64, -1, -1]
    assert starts.tolist() == [0, 3, 3, 20] and kv.tolist() == [18, 0, 17] and taken == 3


def test_binding_allocates_on_the_given_stream(monkeypatch):
    """With `stream`, that stream is the current one while a call allocates its results and its
    workspace (torch hands memory of one stream to that stream's later work only), and the call
    runs on it; without, or where it is current already, nothing changes. Host-side stand-ins."""
    current, seen = [70], []

    class Stream:
        def __init__(self, handle, index):
            self.cuda_stream, self.device = handle, torch.device("cuda", index)

    class Current:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            self.prev, current[0] = current[0], self.s.cuda_stream

        def __exit__(self, *exc):
            current[0] = self.prev

    def empty(shape, strides, dtype, device):
        seen.append(("alloc", current[0]))
        return torch.empty(shape, dtype=dtype)

    k = wq._kv4()
    stub = type("Stub", (), dict(vars(k)))()
    stub.current_device, stub.raw_stream = lambda: 0, lambda d: current[0]
    stub.empty, stub.workspace_bytes = empty, {0: 16}
    for name in ("block_tables", "append", "read", "attention"):
        setattr(stub, name, lambda *args, name=name: seen.append((name, args[-1])) or 0)
    stub.on_stream = Current
    monkeypatch.setattr(wq, "_KV4", stub)

    class OnZero(torch.Tensor):
        """A host tensor that says it is on device 0."""
        def get_device(self):
            return 0

        device = property(lambda self: 0)

    zero = lambda t: t.as_subclass(OnZero)  # noqa: E731
    ints = lambda *s: zero(torch.zeros(s, dtype=torch.int32))  # noqa: E731
    c = zero(wq.wq_kv4_alloc(4, 2, 64, 32, 16, device="cpu"))
    x = zero(torch.zeros(3, 2, 64, dtype=torch.bfloat16))

    def calls(stream):
        seen.clear()
        wq.wq_kv4_append(x, x, ints(3), c, group=32, stream=stream)
        wq.wq_kv4_read(c, ints(3), 64, group=32, stream=stream)
        wq.wq_kv4_block_tables(ints(2), ints(2), ints(4), ints(2, 4), 16, 8, stream=stream)
        wq.wq_kv4_attention(x, c, ints(1, 4), ints(2), ints(1), 3, group=32, return_lse=True,
                            stream=stream)
        assert current == [70]
        return list(seen)

    for stream, handle in ((None, 70), (Stream(70, 0), 70), (Stream(88, 0), 88)):
        alloc = ("alloc", handle)
        assert calls(stream) == [("append", handle), alloc, alloc, ("read", handle), alloc,
                                 ("block_tables", handle), alloc, alloc, alloc,
                                 ("attention", handle)]
    with pytest.raises(ValueError):  # a stream of another device
        calls(Stream(88, 1))


def test_attention_grid_of_very_many_heads_and_requests(lib):
    """kv_heads x B past the largest grid is refused where the prompt kernel would run."""
    def f(kv_heads, B, mq):
        c = cache(blocks=1, heads=kv_heads)
        return lib.wq_kv4_attention(attention_args(c=c, heads=kv_heads, B=B, mq=mq), None)

    assert f(65535, 65536, 17) == SHAPE and f(32768, 65536, 17) == SHAPE
    assert f(65535, 65536, 16) not in (OK, SHAPE) and f(32767, 65536, 17) not in (OK, SHAPE)

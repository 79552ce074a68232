"""Refusals of the operators around append and decode, before any device work (C ABI and binding)."""

import ctypes
import os

import pytest
import torch

from kv_cache_quantization_append_gb300 import lib

OK, INVALID, UNSUPPORTED, ALIGN, CAPACITY, CUDA, NOT_INIT = range(7)
P = ctypes.c_void_p
FAKE = 0x7F0000000000          # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def kvq():
    if not os.path.exists(lib.LIB_PATH):
        from kv_cache_quantization_append_gb300 import build

        build.build()
    return lib.load()


def _cache(**kw):
    """A handle with a valid configuration and fake addresses: host checks only."""
    c = lib.kvq_cache()
    c.cfg = lib.make_config(2, 8, 24, 4, 1024, **kw)
    c.dev, c.block_table, c.max_pages_per_seq, c.n_pages = FAKE, FAKE, 16, 64
    c.magic = 0x4B565131
    return c


def test_rope_handle(kvq):
    r = lib.kvq_rope()
    init = lambda *a: kvq.kv_rope_init(ctypes.byref(r), *a)  # noqa: E731
    good = (128, 0, 10000.0, 0, 1.0, 0.0, 0.0, 0.0, 1.0)
    assert init(*good) == OK and r.magic != 0
    # pair 0 turns one radian a position: 2^64 / 2 pi
    assert abs(r.turns[0] / 2 ** 64 - 0.15915494309189535) < 1e-16
    r.magic = 0
    for i, bad, code in ((0, 130, UNSUPPORTED), (0, 3, UNSUPPORTED), (0, -2, UNSUPPORTED), (1, 2, UNSUPPORTED), (3, 5, UNSUPPORTED),
                         (2, 1.0, INVALID), (2, float("nan"), INVALID), (2, float("inf"), INVALID), (8, 0.0, INVALID),
                         (8, float("nan"), INVALID)):
        a = list(good)
        a[i] = bad
        assert init(*a) == code, (i, bad)
    assert init(128, 0, 1e4, 1, 0.0, 0.0, 0.0, 0.0, 1.0) == INVALID
    assert init(2, 0, 1e4, 2, 2.0, 0.0, 0.0, 0.0, 1.0) == UNSUPPORTED
    assert init(64, 0, 1e4, 3, 2.0, 0.0, 1.0, 4.0, 1.0) == INVALID
    assert init(64, 0, 1e4, 4, 2.0, 4096.0, 4.0, 4.0, 1.0) == INVALID
    assert init(64, 0, 1e4, 4, 2.0, 4096.0, 0.0, 4.0, 1.0) == INVALID
    assert kvq.kv_rope_init(None, *good) == INVALID
    assert r.magic == 0


def test_rope_turns_against_60_digits(kvq):
    """Turns per position of every pair: pow, the division and the quotient in double round by a few 2^-53 of at most 0.16
    turns, and the 64-bit fraction is cut at 2^-64: within 2^-54 in all."""
    from decimal import Decimal, getcontext

    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    for rot, theta, kind, factor in ((128, 1e4, 0, 1.0), (128, 5e5, 0, 1.0), (96, 1e6, 1, 8.0), (64, 1e4, 2, 8.0), (90, 1e7, 0, 1.0)):
        base = Decimal(theta)
        if kind == 2:
            base *= Decimal(factor) ** (Decimal(rot) / (rot - 2))
        r = lib.kv_rope_init(rot, theta=theta, scaling=kind, factor=factor)
        for i in range(rot // 2):
            f = base ** (Decimal(-2 * i) / rot) / two_pi / (Decimal(factor) if kind == 1 else 1)
            assert abs(Decimal(r.turns[i]) / 2 ** 64 - f % 1) < Decimal(2) ** -54, (rot, theta, kind, i)


def test_norm_rope(kvq):
    r = lib.kv_rope_init(128)
    d = P(FAKE)
    names = ("rope", "qkv", "stride", "pos", "wq", "wk", "eps", "q", "k", "v", "B", "T", "hq", "hkv", "dt", "stream")
    good = dict(zip(names, (ctypes.byref(r), d, 12 * 128, d, None, None, 1e-6, d, d, d, 2, 3, 8, 2, 1, None)))

    def call(**kw):
        return kvq.kv_qk_norm_rope(*({**good, **kw}[n] for n in names))

    for n in ("rope", "qkv", "pos", "q", "k"):
        assert call(**{n: None}) == INVALID, n
    assert call(rope=ctypes.byref(lib.kvq_rope())) == NOT_INIT
    for n in ("B", "T", "hq", "hkv"):
        assert call(**{n: 0}) == INVALID, n
    assert call(B=1 << 20, T=1 << 20) == INVALID
    assert call(stride=12 * 128 - 8) == INVALID and call(stride=12 * 128 + 4) == ALIGN
    assert call(dt=2) == UNSUPPORTED
    assert call(eps=-1.0) == INVALID and call(eps=float("nan")) == INVALID and call(eps=float("inf")) == INVALID
    for n in ("qkv", "pos", "wq", "wk", "q", "k", "v"):
        assert call(**{n: P(FAKE + 8)}) == ALIGN, n


def test_uninitialised_cache(kvq):
    c = lib.kvq_cache()
    c.cfg = lib.make_config(2, 8, 24, 1, 1024)
    r, d = ctypes.byref(c), P(FAKE)
    for cache, code in ((r, NOT_INIT), (None, INVALID)):
        assert kvq.kv_tree_attention(cache, 0, d, d, d, d, d, d, 1, 4, d, 1 << 30, None) == code
        assert kvq.kv_tree_commit(cache, 0, d, d, d, d, d, 1, 4, 4, None) == code
        assert kvq.kv_attention_weights(cache, 0, d, d, 1.0, d, 1, 1, d, 1 << 30, None) == code
        assert kvq.kv_evict(cache, 0, d, d, d, P(FAKE + 16), 1, 64, 64, None) == code
        assert kvq.kv_tree_scratch_bytes(cache, 0, 1, 4) == 0
        assert kvq.kv_weights_scratch_bytes(cache, 0, 1, 4) == 0


@pytest.mark.parametrize("i", [1, 2, 3, 4, 5, 6, 9])
def test_tree_null_and_misaligned(kvq, i):
    c, d = _cache(), P(FAKE)
    good = [ctypes.byref(c), 0, d, d, d, d, d, d, 2, 4, d, 1 << 40, None]
    at = i + 1
    a = list(good)
    a[at] = None
    if at < 8 or at == 10:
        assert kvq.kv_tree_attention(*a) == INVALID
        a[at] = P(FAKE + 4)
        assert kvq.kv_tree_attention(*a) == ALIGN


def test_tree_ranges(kvq):
    c, d = _cache(), P(FAKE)
    call = lambda layer=0, B=2, n=4, sb=1 << 40: kvq.kv_tree_attention(  # noqa: E731
        ctypes.byref(c), layer, d, d, d, d, d, d, B, n, d, sb, None)
    assert call(layer=2) == INVALID and call(layer=-2) == INVALID
    assert call(B=0) == INVALID and call(B=5) == INVALID
    assert call(n=0) == INVALID and call(n=65) == INVALID
    assert call(sb=255) == CAPACITY
    assert kvq.kv_tree_scratch_bytes(ctypes.byref(c), 0, 2, 65) == 0
    assert kvq.kv_tree_scratch_bytes(ctypes.byref(c), -1, 4, 64) >= 256


def test_commit_ranges(kvq):
    c, d = _cache(), P(FAKE)

    def call(layer=0, k=d, v=d, path=d, n=d, pos=d, B=2, N=4, mp=4):
        return kvq.kv_tree_commit(ctypes.byref(c), layer, k, v, path, n, pos, B, N, mp, None)

    for name in ("k", "v", "path", "n", "pos"):
        assert call(**{name: None}) == INVALID, name
        assert call(**{name: P(FAKE + 4)}) == ALIGN, name
    assert call(layer=2) == INVALID and call(B=5) == INVALID and call(B=0) == INVALID
    assert call(N=65) == INVALID and call(N=0) == INVALID
    assert call(mp=0) == INVALID and call(mp=5) == INVALID


def test_weights_ranges(kvq):
    c, d = _cache(), P(FAKE)

    def call(layer=0, q=d, w=d, decay=1.0, ln=d, B=2, n=4, s=d, sb=1 << 40):
        return kvq.kv_attention_weights(ctypes.byref(c), layer, q, w, decay, ln, B, n, s, sb, None)

    for name in ("q", "w", "ln", "s"):
        assert call(**{name: None}) == INVALID, name
        assert call(**{name: P(FAKE + 4)}) == ALIGN, name
    assert call(decay=-0.1) == INVALID and call(decay=1.5) == INVALID and call(decay=float("nan")) == INVALID
    assert call(layer=3) == INVALID and call(B=5) == INVALID and call(n=0) == INVALID and call(n=65) == INVALID
    assert call(sb=16) == CAPACITY


def test_weights_scratch_does_not_grow_with_the_layers(kvq):
    c = _cache()
    sizes = []
    for layers in (1, 28):
        c.cfg = lib.make_config(layers, 8, 32, 8, 131072)
        c.max_pages_per_seq, c.n_pages = 2048, 8 * 2048
        sizes.append([kvq.kv_weights_scratch_bytes(ctypes.byref(c), -1, 8, n) for n in (1, 2, 3)])
    one, all_ = sizes
    assert one[0] >= 8 * 8 * 4 * 131072 * 4 and one[1] >= 8 * 8 * 8 * 131072 * 4      # a layer's logits
    for i in range(2):
        assert all_[i] <= (256 << 20) + (32 << 20)
    assert all_[2] < 64 << 20                               # 12 rows: logits are not stored


def test_evict_ranges(kvq):
    c, d = _cache(), P(FAKE)

    def call(layer=0, w=d, ln=d, kept=d, new=P(FAKE + 64), B=2, budget=256, recent=128):
        return kvq.kv_evict(ctypes.byref(c), layer, w, ln, kept, new, B, budget, recent, None)

    for name in ("w", "ln", "kept", "new"):
        assert call(**{name: None}) == INVALID, name
        assert call(**{name: P(FAKE + 4)}) == ALIGN, name
    assert call(new=d) == INVALID                              # the lengths are still read while new ones are written
    assert call(recent=127) == INVALID and call(recent=-1) == INVALID and call(recent=257) == INVALID
    assert call(budget=0) == INVALID and call(budget=1025) == INVALID
    assert call(layer=5) == INVALID and call(B=5) == INVALID


def test_binding_shapes():
    c = _cache()
    bf, i32 = torch.bfloat16, torch.int32
    z = torch.zeros
    s = z(16, dtype=torch.uint8)
    kv, q, ln = z(2, 8, 4, 128, dtype=bf), z(2, 24, 4, 128, dtype=bf), z(2, dtype=i32)
    par = z(2, 4, dtype=i32)
    for args in ((kv, kv, q[:, :8], q, ln, par), (kv, kv, q, q.float(), ln, par), (kv, kv, q, q, ln.long(), par),
                 (kv, kv, q, q, ln, par[:, :3]), (kv, kv[:, :, :3], q, q, ln, par), (kv, kv, q, q[:1], ln, par)):
        with pytest.raises(lib.KVQError):
            lib.kv_tree_attention(c, 0, *args, s)
    for args in ((kv, kv, par[:1], ln, ln), (kv, kv, par.long(), ln, ln), (kv, kv, par, ln[:1], ln), (kv, kv, par, ln, ln.long())):
        with pytest.raises(lib.KVQError):
            lib.kv_tree_commit(c, 0, *args)
    w = z(2, 8, 1024)
    for args in ((q, w[:, :, :1000], 1.0, ln), (q, w.double(), 1.0, ln), (q.float(), w, 1.0, ln), (q, w, 1.0, ln.long()),
                 (q[0], w, 1.0, ln), (q, w, 1.0, ln[:1])):
        with pytest.raises(lib.KVQError):
            lib.kv_attention_weights(c, 0, *args, s)
    kept = z(2, 8, 256, dtype=i32)
    for args in ((w, ln, kept[..., :255], ln.clone(), 256, 128), (w, ln, kept.long(), ln.clone(), 256, 128),
                 (w, ln.long(), kept, ln.clone(), 256, 128), (w[:1], ln, kept, ln.clone(), 256, 128),
                 (w, ln, kept, ln[:1], 256, 128), (w, ln[None], kept, ln.clone(), 256, 128)):
        with pytest.raises(lib.KVQError):
            lib.kv_evict(c, 0, *args)
    r = lib.kv_rope_init(128)
    x = z(2, 3, 12 * 128, dtype=bf)
    pos = z(2, 3, dtype=i32)
    qo, ko = z(2, 8, 3, 128, dtype=bf), z(2, 2, 3, 128, dtype=bf)
    wt = z(128, dtype=bf)
    for args in ((x[0], pos, qo, ko, ko), (x.half(), pos, qo, ko, ko), (x, pos.long(), qo, ko, ko), (x, pos[:1], qo, ko, ko),
                 (x, pos, qo[:1], ko, ko), (x, pos, qo, ko, ko[:, :1]), (x[:, :, :-128], pos, qo, ko, ko),
                 (x, pos, qo.float(), ko, ko), (x, pos, qo, ko, ko, wt[:64]), (x, pos, qo, ko, ko, wt.float()),
                 (x.transpose(0, 1), pos, qo, ko, ko), (x[:, :, ::2], pos, qo, ko, ko), (x, pos, qo[:, :, 0], ko[:, :, 0], None),
                 (x, pos, qo, ko, ko)):             # the last: host tensors
        with pytest.raises(lib.KVQError):
            lib.kv_qk_norm_rope(r, *args)


class _Elsewhere:
    """A tensor that says it is on another GPU than the cache (device 0)."""

    def __init__(self, t):
        self._t = t
        self.is_cuda = True

    def get_device(self):
        return 1

    def __getattr__(self, name):
        return getattr(self._t, name)


def test_tensors_of_another_device_are_refused():
    """Each tensor argument in turn is on another device than the cache's, the ones before it on the cache's own."""

    class Here(_Elsewhere):
        def get_device(self):
            return 0

    c = _cache()
    bf, i32, z = torch.bfloat16, torch.int32, torch.zeros
    kv, q, ln, par = z(2, 8, 4, 128, dtype=bf), z(2, 24, 4, 128, dtype=bf), z(2, dtype=i32), z(2, 4, dtype=i32)
    q1, o1, s, w = z(2, 24, 128, dtype=bf), z(2, 24, 128), z(16, dtype=torch.uint8), z(2, 8, 1024)
    calls = {
        lib.kv_tree_attention: (kv, kv, q, q, ln, par, s),
        lib.kv_tree_commit: (kv, kv, par, ln, ln),
        lib.kv_attention_weights: (q, w, 1.0, ln, s),
        lib.kv_evict: (w, ln, z(2, 8, 256, dtype=i32), ln, 256, 128),
        lib.kv_quant_append: (kv, kv, ln),
        lib.kv_decode_attention: (q1, o1, ln, s),
        lib.kv_decode_attention_noalloc: (q1, o1, ln),
        lib.kv_prefill_attention: (kv, kv, q, q.float(), ln, s),
        lib.kv_calibrate: (kv[0], kv[0], s),
    }
    for call, args in calls.items():
        tensors = [i for i, a in enumerate(args) if isinstance(a, torch.Tensor)]
        for n in tensors:
            given = [a if i not in tensors else _Elsewhere(a) if i == n else Here(a) for i, a in enumerate(args)]
            with pytest.raises(lib.KVQError, match="tensor on device 1"):
                call(c, 0, *given)


def test_evict_lengths_that_overlap(kvq):
    c, d = _cache(), P(FAKE)
    call = lambda ln, new, B: kvq.kv_evict(ctypes.byref(c), 0, d, P(ln), d, P(new), B, 256, 128, None)  # noqa: E731
    c.cfg = lib.make_config(2, 8, 24, 40, 1024)
    c.n_pages = 640
    for B, apart in ((40, 144), (40, 16), (5, 16)):
        assert call(FAKE, FAKE + apart, B) == INVALID and call(FAKE + apart, FAKE, B) == INVALID
    assert call(FAKE, FAKE + 160, 40) != INVALID and call(FAKE + 16, FAKE, 4) != INVALID   # (no device here)

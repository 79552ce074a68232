"""Caches of 8-bit codes with one scale per block of 32 tokens (KVQ_Q8B32): append, decode and prefill against the definition."""

import numpy as np
import pytest
import torch

from kv_cache_quantization_append_gb300 import lib

from . import block_reference as br
from . import harness

pytestmark = pytest.mark.gpu

# Outputs are float.  Queries, weights and raw operands have 22 bits (2^-22 each), codes are exact; a logit of up to 40
# (base 2) adds at most 32 truncated partial sums (2^-23): 40 (2^-22 + 32 * 2^-23) = 1.7e-4 at the very worst for a
# weight's relative error, a few times less on average over signs; outputs are averages of values up to the largest.
TOL = 2e-4


def _t(x, in_dtype):
    return torch.as_tensor(x).to(torch.bfloat16 if in_dtype == "bf16" else torch.float32).contiguous()


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def _vectors(rng, shape, in_dtype, scale=1.0):
    x = rng.standard_normal(shape + (128,)).astype(np.float32) * scale
    x[..., 7] *= 5
    return _t(x, in_dtype)


def _append(gpu, ref, layer, rng, T, pos, in_dtype, scale=1.0):
    cfg = gpu.cfg
    lead = (cfg.n_layers,) if layer == -1 else ()
    k, v = (_vectors(rng, lead + (len(pos), cfg.n_kv_heads, T), in_dtype, scale) for _ in range(2))
    gpu.append(layer, k.cuda(), v.cuda(), _i32(pos))
    ref.append(layer, harness.to_np(k), harness.to_np(v), pos)
    return k, v


def _units(cfg):
    return [(lay, b, h) for lay in range(cfg.n_layers) for b in range(cfg.max_batch) for h in range(cfg.n_kv_heads)]


def _check_decode(gpu, ref, rng, lens, in_dtype, layer=0, tol=TOL, qscale=1.0):
    cfg = gpu.cfg
    lead = (cfg.n_layers,) if layer == -1 else ()
    q = _t(rng.standard_normal(lead + (len(lens), cfg.n_q_heads, 128)).astype(np.float32) * qscale, in_dtype)
    out = gpu.decode(layer, q.cuda(), _i32(lens)).double().cpu().numpy()
    assert gpu.status() == 0
    qn = harness.to_np(q)
    for i, lay in enumerate(range(cfg.n_layers) if layer == -1 else [layer]):
        got = out[i] if layer == -1 else out
        want = ref.decode(lay, qn[i] if layer == -1 else qn, lens)
        for b in range(len(lens)):
            harness.assert_attention_close(got[b], want[b], tol)


@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [32, 64, 100, 1024])
@pytest.mark.parametrize("steps", [[1] * 70, [31, 1, 1, 33, 5, 64], [200], [7, 150, 3, 90], [32, 32, 1]])
def test_append_bytes(in_dtype, window, steps):
    """Any division of the tokens into calls leaves the definition's bytes; sequences at different places, one left alone."""
    rng = np.random.default_rng(sum(steps) + window)
    table = rng.permutation(4 * 8 + 3)[:4 * 8].reshape(4, 8)
    gpu, ref = br.make(1, 2, 2, 4, 512, window=window, in_dtype=in_dtype, n_pages=35, table=table)
    at = np.array([0, 13, 0, 77])
    _append(gpu, ref, 0, rng, 13, [-1, 0, -1, -1], in_dtype)
    _append(gpu, ref, 0, rng, 77, [-1, -1, -1, 0], in_dtype)
    for T in steps:
        pos = [int(at[0]), int(at[1]), -1, int(at[3])]
        _append(gpu, ref, 0, rng, T, pos, in_dtype)
        at[[0, 1, 3]] += T
    assert gpu.status() == 0
    br.check_state(gpu, ref, _units(gpu.cfg), table)


def test_append_layers_and_refused_sequences():
    rng = np.random.default_rng(3)
    gpu, ref = br.make(3, 4, 8, 3, 160, window=64)
    _append(gpu, ref, -1, rng, 100, [0, 0, 0], "bf16")
    _append(gpu, ref, -1, rng, 50, [100, 120, 100], "bf16")          # the second would end past capacity
    assert gpu.status() == lib.DEV_POS_RANGE
    br.check_state(gpu, ref, _units(gpu.cfg))
    _check_decode(gpu, ref, rng, [150, 100, 150], "bf16", -1)
    with pytest.raises(lib.KVQError):                                # keys of another dtype
        gpu.append(0, torch.zeros(1, 4, 1, 128, device="cuda"), torch.zeros(1, 4, 1, 128, device="cuda"), _i32([0]))


def test_bad_pages_are_flagged_and_skipped():
    rng = np.random.default_rng(4)
    table = np.arange(8).reshape(2, 4).copy()
    table[0, 1], table[1, 2] = -1, 100
    gpu, ref = br.make(1, 2, 4, 2, 256, window=32, n_pages=8, table=table)
    _append(gpu, ref, 0, rng, 200, [0, -1], "bf16")
    assert gpu.status() == lib.DEV_BAD_PAGE
    good = br.stored(gpu, 0, 0, 0, 2, table)
    c, d = ref.blocks(0, 0, 0, 0, 2)
    assert np.array_equal(good[0][0], c) and np.array_equal(good[0][1], d)
    out = gpu.decode(0, _t(rng.standard_normal((2, 4, 128)).astype(np.float32), "bf16").cuda(), _i32([200, 0]))
    assert gpu.status() == lib.DEV_BAD_PAGE and torch.isfinite(out).all() and (out[1] == 0).all()
    k, v, q = (_vectors(rng, (2, h, 5), "bf16").cuda() for h in (2, 2, 4))
    out = gpu.prefill(0, k, v, q, _i32([200, -1]))
    assert gpu.status() == lib.DEV_BAD_PAGE and torch.isfinite(out).all() and (out[1] == 0).all()


@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("g", [1, 2, 3, 4])
@pytest.mark.parametrize("window", [32, 128, 100])
def test_decode(in_dtype, g, window):
    rng = np.random.default_rng(10 * g + window)
    lens = [0, 1, 31, 32, 33, window - 1, window, window + 1, window + 32, 300, 511, 512]
    gpu, ref = br.make(1, 2, 2 * g, len(lens), 512, window=window, in_dtype=in_dtype)
    for b, n in enumerate(lens):
        if n:
            pos = [-1] * len(lens)
            pos[b] = 0
            _append(gpu, ref, 0, rng, n, pos, in_dtype)
    _check_decode(gpu, ref, rng, lens, in_dtype)


def test_decode_long_and_layers():
    rng = np.random.default_rng(77)
    gpu, ref = br.make(2, 2, 6, 2, 9000, window=128)
    _append(gpu, ref, -1, rng, 8999, [0, -1], "bf16")
    _append(gpu, ref, -1, rng, 4321, [-1, 0], "bf16")
    _check_decode(gpu, ref, rng, [8999, 4321], "bf16", -1)
    _check_decode(gpu, ref, rng, [8999, 4321], "bf16", 1)


def test_sinkhorn():
    rng = np.random.default_rng(5)
    gpu, ref = br.make(1, 2, 4, 1, 400, window=64, sinkhorn=True)
    spread = np.exp(rng.uniform(-2, 2, 128)).astype(np.float32)
    k, v = (_t(rng.standard_normal((2, 256, 128)).astype(np.float32) * spread, "bf16") for _ in range(2))
    gpu.calibrate(0, k.cuda(), v.cuda())
    ref.sigma = [s.astype(np.float32) for s in _sigma(gpu)]
    kk, vv = (_t(rng.standard_normal((1, 2, 390, 128)).astype(np.float32) * spread, "bf16") for _ in range(2))
    gpu.append(0, kk.cuda(), vv.cuda(), _i32([0]))
    ref.append(0, harness.to_np(kk), harness.to_np(vv), [0])
    br.check_state(gpu, ref, _units(gpu.cfg))
    _check_decode(gpu, ref, rng, [390], "bf16")
    k, v, q = (_vectors(rng, (1, h, 10), "bf16") for h in (2, 2, 4))
    _check_prefill(gpu, ref, rng, k, v, q, [390])


def _sigma(gpu):
    """The balancing scales: the two fp16 [n_layers][n_kv_heads][128] that lie before the identity table and the rings."""
    cfg = gpu.cfg
    a = lambda x: -(-x // 256) * 256  # noqa: E731
    maxpps = -(-cfg.max_seq_len // 64)
    n_pages = cfg.n_pages or cfg.max_batch * maxpps
    ring = a(cfg.n_layers * cfg.max_batch * cfg.n_kv_heads * cfg.window * 512)
    sig = cfg.n_layers * cfg.n_kv_heads * 256
    end = lib.kv_cache_bytes(cfg) - a(cfg.n_layers * n_pages * cfg.n_kv_heads * 16416) - 2 * ring - a(cfg.max_batch * maxpps * 4)
    shape = (cfg.n_layers, cfg.n_kv_heads, 128)
    return [gpu.buffer[o:o + sig].cpu().numpy().view(np.float16).reshape(shape) for o in (end - 2 * a(sig), end - a(sig))]


def _check_prefill(gpu, ref, rng, k, v, q, pos, tol=TOL, layer=0):
    """The chunk's outputs are those of its tokens' single steps; the cache is left as they leave it."""
    T = q.shape[-2]
    out = gpu.prefill(layer, k.cuda(), v.cuda(), q.cuda(), _i32(pos)).double().cpu().numpy()
    assert gpu.status() == 0
    ref.append(layer, harness.to_np(k), harness.to_np(v), pos)
    qn = harness.to_np(q)
    for b, p in enumerate(pos):
        if p < 0:
            assert (out[b] == 0).all()
            continue
        # (a look at every token near the ends and at some between)
        ts = sorted(set(list(range(min(T, 3))) + list(range(max(0, T - 2), T)) + list(rng.integers(0, T, 4))))
        want = np.stack([[ref.attend(layer, b, j, qn[b, j, t], p + t + 1) for t in ts] for j in range(q.shape[1])])
        harness.assert_attention_close(out[b][:, ts], want, tol)


@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("g,window", [(1, 32), (2, 128), (3, 100), (4, 64)])
@pytest.mark.parametrize("first,T", [(0, 1), (0, 300), (5, 1), (31, 1), (100, 33), (333, 65), (400, 130)])
def test_prefill(in_dtype, g, window, first, T):
    rng = np.random.default_rng(first + T + g)
    gpu, ref = br.make(1, 2, 2 * g, 3, 600, window=window, in_dtype=in_dtype)
    pos = [first, -1, max(0, first - 3)]
    for b in (0, 2):
        if pos[b]:
            at = [-1] * 3
            at[b] = 0
            _append(gpu, ref, 0, rng, pos[b], at, in_dtype)
    k, v, q = (_vectors(rng, (3, h, T), in_dtype) for h in (2, 2, 2 * g))
    _check_prefill(gpu, ref, rng, k, v, q, pos)
    br.check_state(gpu, ref, [(0, 0, 0), (0, 0, 1), (0, 2, 1)])


def test_prefill_many_tiles_and_layers():
    rng = np.random.default_rng(9)
    gpu, ref = br.make(2, 1, 4, 1, 6200, window=128)
    _append(gpu, ref, -1, rng, 6000, [0], "bf16")
    k, v = (_vectors(rng, (2, 1, 1, 100), "bf16") for _ in range(2))
    q = _vectors(rng, (2, 1, 4, 100), "bf16")
    out = gpu.prefill(-1, k.cuda(), v.cuda(), q.cuda(), _i32([6000])).double().cpu().numpy()
    ref.append(-1, harness.to_np(k), harness.to_np(v), [6000])
    for lay in range(2):
        for t in (0, 57, 99):
            want = np.stack([ref.attend(lay, 0, j, harness.to_np(q)[lay, 0, j, t], 6001 + t) for j in range(4)])
            harness.assert_attention_close(out[lay, 0, :, t], want, TOL)


@pytest.mark.parametrize("kscale,vscale,qscale", [(1, 1e-7, 1), (1, 1e6, 1), (1e-5, 1, 1e5), (1e5, 1, 1e-5), (1, 1e-30, 1), (1e4, 1e20, 1e-4)])
def test_values_of_any_size(kscale, vscale, qscale):
    """Float inputs far from 1: products keep their bits (TOL of the largest output)."""
    rng = np.random.default_rng(21)
    gpu, ref = br.make(1, 2, 4, 1, 400, window=64, in_dtype="f32")
    k, v = (_vectors(rng, (1, 2, 333), "f32", s) for s in (kscale, vscale))
    gpu.append(0, k.cuda(), v.cuda(), _i32([0]))
    ref.append(0, harness.to_np(k), harness.to_np(v), [0])
    br.check_state(gpu, ref, _units(gpu.cfg))
    _check_decode(gpu, ref, rng, [333], "f32", qscale=qscale)
    k, v, q = (_vectors(rng, (1, h, 40), "f32", s) for h, s in ((2, kscale), (2, vscale), (4, qscale)))
    _check_prefill(gpu, ref, rng, k, v, q, [333])


def test_blocks_of_very_different_scales_and_zeros():
    """Blocks whose values grow and shrink by many powers of two, blocks of zeros, one whose scale underflows."""
    rng = np.random.default_rng(22)
    gpu, ref = br.make(1, 1, 4, 1, 1024, window=32, in_dtype="f32")
    grow = np.repeat(np.array([1e-3, 1, 1e-6, 30, 0, 1e-4, 5e3, 2e-2, 0, 1.0]), 96)[:, None].astype(np.float32)
    k = _t(rng.standard_normal((1, 1, 960, 128)).astype(np.float32) * np.minimum(grow, 1), "f32")
    v = _t(rng.standard_normal((1, 1, 960, 128)).astype(np.float32) * grow, "f32")
    k[0, 0, 96:128] = 0
    k[0, 0, 96, 0] = 1e-43
    gpu.append(0, k.cuda(), v.cuda(), _i32([0]))
    ref.append(0, harness.to_np(k), harness.to_np(v), [0])
    br.check_state(gpu, ref, [(0, 0, 0)])
    for n in (960, 700, 330, 200, 90):
        # (the ring holds the newest tokens of the last call)
        gpu.append(0, k[:, :, :n].contiguous().cuda(), v[:, :, :n].contiguous().cuda(), _i32([0]))
        _check_decode(gpu, ref, rng, [n], "f32")
    for p in (300, 640, 930):
        kk, vv, q = (_t(rng.standard_normal((1, h, 30, 128)).astype(np.float32), "f32") for h in (1, 1, 4))
        gpu.append(0, k[:, :, :p].contiguous().cuda(), v[:, :, :p].contiguous().cuda(), _i32([0]))
        ref.append(0, harness.to_np(k[:, :, :p]), harness.to_np(v[:, :, :p]), [0])
        _check_prefill(gpu, ref, rng, kk, vv, q, [p])


def test_peaked_attention_and_a_sink():
    """An early position far above thousands of equal ones: their many small weights still add up."""
    rng = np.random.default_rng(23)
    gpu, ref = br.make(1, 1, 4, 1, 7000, window=64, in_dtype="f32")
    q = rng.standard_normal(128).astype(np.float32)
    k = rng.standard_normal((1, 1, 6800, 128)).astype(np.float32) * 0.02
    k[0, 0, 3] = q * (11.8 * np.sqrt(128) / (q @ q))
    v = rng.standard_normal((1, 1, 6800, 128)).astype(np.float32) * 0.1 + 1
    v[0, 0, 3] = -1
    k, v = _t(k, "f32"), _t(v, "f32")
    gpu.append(0, k.cuda(), v.cuda(), _i32([0]))
    ref.append(0, harness.to_np(k), harness.to_np(v), [0])
    qq = np.broadcast_to(q, (1, 4, 128)).copy()
    out = gpu.decode(0, _t(qq, "f32").cuda(), _i32([6800])).double().cpu().numpy()
    harness.assert_attention_close(out[0], ref.decode(0, qq, [6800])[0], TOL)
    kk, vv = (_t(rng.standard_normal((1, 1, 3, 128)).astype(np.float32) * 0.02, "f32") for _ in range(2))
    _check_prefill(gpu, ref, rng, kk, vv, _t(np.broadcast_to(q, (1, 4, 3, 128)).copy(), "f32"), [6800])


def test_one_query_that_is_not_finite():
    """It spoils its own output only (what that is, decode leaves open)."""
    rng = np.random.default_rng(24)
    gpu, ref = br.make(1, 2, 8, 1, 400, window=64)
    _append(gpu, ref, 0, rng, 300, [0], "bf16")
    q = _vectors(rng, (1, 8), "bf16")
    good = gpu.decode(0, q.cuda(), _i32([300]))
    q[0, 5, 3] = float("inf")
    out = gpu.decode(0, q.cuda(), _i32([300]))
    keep = [j for j in range(8) if j != 5]
    assert torch.equal(good[0, keep], out[0, keep])
    k, v, q = (_vectors(rng, (1, h, 20), "bf16") for h in (2, 2, 8))
    state = gpu.buffer.clone()
    good = gpu.prefill(0, k.cuda(), v.cuda(), q.cuda(), _i32([300]))
    gpu.buffer.copy_(state)
    q[0, 2, 7, 100] = float("nan")
    out = gpu.prefill(0, k.cuda(), v.cuda(), q.cuda(), _i32([300]))
    same = (out == good).all(-1)[0]
    assert not same[2, 7] and same.sum() == same.numel() - 1


def test_decode_step_by_step_is_prefill_is_captured():
    """Single steps, one chunk, and a captured step replayed at moving positions agree; two layers, two sequences."""
    rng = np.random.default_rng(25)
    lens = [90, 250]
    a, ref = br.make(2, 2, 6, 2, 400, window=64)
    b, _ = br.make(2, 2, 6, 2, 400, window=64)
    c, _ = br.make(2, 2, 6, 2, 400, window=64)
    for i, n in enumerate(lens):
        pos = [-1, -1]
        pos[i] = 0
        k, v = _append(a, ref, -1, rng, n, pos, "bf16")
        for other in (b, c):
            other.append(-1, k.cuda(), v.cuda(), _i32(pos))
    T = 70
    k, v = (_vectors(rng, (2, 2, 2, T), "bf16").cuda() for _ in range(2))
    q = _vectors(rng, (2, 2, 6, T), "bf16").cuda()
    chunk = b.prefill(-1, k, v, q, _i32(lens))
    pos, ln = _i32(lens), _i32(lens) + 1
    ks, vs, qs = (x[..., 0, :].unsqueeze(-2).contiguous() for x in (k, v, q))
    qs = qs.squeeze(-2).contiguous()
    out = torch.empty(2, 2, 6, 128, device="cuda")

    def step():
        c.append(-1, ks, vs, pos)
        c.decode(-1, qs, ln, out=out)
        pos.add_(1)
        ln.add_(1)

    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    pos0 = _i32(lens)
    a.decode(-1, qs, pos0)                         # (a call outside capture before the first inside)
    with torch.cuda.graph(graph, stream=side):
        step()
    pos.copy_(_i32(lens))
    ln.copy_(_i32(lens) + 1)
    for t in range(T):
        kt, vt, qt = (x[..., t, :].contiguous() for x in (k, v, q))
        a.append(-1, kt.unsqueeze(-2), vt.unsqueeze(-2), _i32([n + t for n in lens]))
        want = a.decode(-1, qt, _i32([n + t + 1 for n in lens]))
        ks.copy_(kt.unsqueeze(-2))
        vs.copy_(vt.unsqueeze(-2))
        qs.copy_(qt)
        graph.replay()
        assert torch.equal(out, want)
        got = chunk[..., t, :]
        assert (got - want).abs().max() <= 2 * TOL * want.abs().max()
    assert a.status() == 0 and b.status() == 0 and c.status() == 0
    ref.append(-1, harness.to_np(k), harness.to_np(v), lens)
    for x in (a, b, c):
        br.check_state(x, ref, _units(x.cfg))


def test_noalloc_and_named_streams():
    rng = np.random.default_rng(26)
    gpu, ref = br.make(1, 2, 4, 2, 700, window=128)
    _append(gpu, ref, 0, rng, 650, [0, 0], "bf16")
    q = _vectors(rng, (2, 4), "bf16").cuda()
    ln = _i32([650, 123])
    want = gpu.decode(0, q, ln)
    out = torch.empty_like(want)
    lib.kv_decode_attention_noalloc(gpu.handle, 0, q, out, ln)
    assert torch.equal(out, want)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = gpu.decode(0, q, ln, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_the_largest_batch():
    """1024 sequences: decode, a chunk of two tokens each, some left alone."""
    rng = np.random.default_rng(27)
    gpu, ref = br.make(1, 1, 2, 1024, 96, window=32)
    lens = rng.integers(0, 90, 1024)
    k, v = (_vectors(rng, (1024, 1, 90), "bf16") for _ in range(2))
    for n in sorted(set(lens.tolist()) - {0}):
        pos = np.where(lens == n, 0, -1)
        gpu.append(0, k[:, :, :n].contiguous().cuda(), v[:, :, :n].contiguous().cuda(), _i32(pos))
        ref.append(0, harness.to_np(k[:, :, :n]), harness.to_np(v[:, :, :n]), pos.tolist())
    _check_decode(gpu, ref, rng, lens, "bf16")
    k, v, q = (_vectors(rng, (1024, h, 2), "bf16") for h in (1, 1, 2))
    pos = np.where(np.arange(1024) % 5 == 3, -1, lens)
    _check_prefill(gpu, ref, rng, k, v, q, pos.tolist())
    br.check_state(gpu, ref, [(0, b, 0) for b in range(0, 1024, 31)])


@pytest.mark.parametrize("lens,T", [([3000, 0, 17, 900, 2047, 64, 333, -1], 250), ([5000, 10, 20, 30], 33), ([700] * 30, 20)])
def test_prefill_divided_over_all_blocks(lens, T):
    """Sequences of very different lengths over several layers: row tiles that many blocks work on, and many in one block."""
    rng = np.random.default_rng(28)
    gpu, ref = br.make(3, 2, 6, len(lens), max(lens) + T, window=96)
    for b, n in enumerate(lens):
        if n > 0:
            at = [-1] * len(lens)
            at[b] = 0
            _append(gpu, ref, -1, rng, n, at, "bf16")
    k, v = (_vectors(rng, (3, len(lens), 2, T), "bf16") for _ in range(2))
    q = _vectors(rng, (3, len(lens), 6, T), "bf16")
    out = gpu.prefill(-1, k.cuda(), v.cuda(), q.cuda(), _i32(lens)).double().cpu().numpy()
    assert gpu.status() == 0
    ref.append(-1, harness.to_np(k), harness.to_np(v), lens)
    qn = harness.to_np(q)
    for b, n in enumerate(lens):
        if n < 0:
            assert (out[:, b] == 0).all()
            continue
        for lay in range(3):
            for t in {0, T - 1, int(rng.integers(0, T))}:
                want = np.stack([ref.attend(lay, b, j, qn[lay, b, j, t], n + t + 1) for j in range(6)])
                harness.assert_attention_close(out[lay, b, :, t], want, TOL)


def test_pages_past_4_gib():
    """The last pages of a pool of 5 GB, keys and values of two layers."""
    rng = np.random.default_rng(29)
    n_pages = 20500
    table = n_pages - 1 - np.arange(2 * 8).reshape(2, 8)
    gpu, ref = br.make(2, 8, 8, 2, 512, window=64, n_pages=n_pages, table=table)
    _append(gpu, ref, -1, rng, 400, [0, 0], "bf16")  # (decode reads the newest tokens from the ring: lengths are what was appended)
    br.check_state(gpu, ref, [(lay, b, h) for lay in range(2) for b in range(2) for h in (0, 7)], table)
    _check_decode(gpu, ref, rng, [400, 400], "bf16", 1)
    k, v, q = (_vectors(rng, (2, 8, 45), "bf16") for _ in range(3))
    _check_prefill(gpu, ref, rng, k, v, q, [400, 400], layer=1)
    br.check_state(gpu, ref, [(1, b, h) for b in range(2) for h in (0, 7)], table)


def test_a_captured_chunk_at_other_positions():
    """A chunk captured once and replayed while positions and inputs change gives what calls give."""
    rng = np.random.default_rng(30)
    a, _ = br.make(2, 2, 8, 3, 1500, window=64)
    b, _ = br.make(2, 2, 8, 3, 1500, window=64)
    T = 90
    k, v, q = (torch.zeros(2, 3, h, T, 128, dtype=torch.bfloat16, device="cuda") for h in (2, 2, 8))
    pos, out = _i32([0, 0, 0]), torch.zeros(2, 3, 8, T, 128, device="cuda")
    for x in (a, b):                                    # (also the calls outside capture before the first inside)
        x.prefill(-1, k, v, q, pos, out=out)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        b.prefill(-1, k, v, q, pos, out=out)
    at = np.array([0, 5, 0])
    for step in range(12):
        p = at.copy()
        if step % 3 == 1:
            p[1] = -1
        for x, h in ((k, 2), (v, 2), (q, 8)):
            x.copy_(_vectors(rng, (2, 3, h, T), "bf16"))
        pos.copy_(_i32(p))
        graph.replay()
        want = a.prefill(-1, k, v, q, _i32(p))
        assert torch.equal(out, want)
        at[p >= 0] += T
    assert a.status() == 0 and b.status() == 0


@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
def test_prefill_of_many_row_tiles(in_dtype):
    """More row tiles than blocks divide: each is one block's, whichever is free; two calls give the same bytes."""
    rng = np.random.default_rng(31)
    gpu, ref = br.make(3, 4, 16, 4, 1200, window=64, in_dtype=in_dtype)
    pos, T = [0, -1, 300, 77], 700
    for b in (2, 3):
        at = [-1] * 4
        at[b] = 0
        _append(gpu, ref, -1, rng, pos[b], at, in_dtype)
    k, v = (_vectors(rng, (3, 4, 4, T), in_dtype) for _ in range(2))
    q = _vectors(rng, (3, 4, 16, T), in_dtype)
    state = gpu.buffer.clone()
    first = gpu.prefill(-1, k.cuda(), v.cuda(), q.cuda(), _i32(pos))
    gpu.buffer.copy_(state)
    out = gpu.prefill(-1, k.cuda(), v.cuda(), q.cuda(), _i32(pos))
    assert torch.equal(first, out) and gpu.status() == 0 and (out[:, 1] == 0).all()
    out = out.double().cpu().numpy()
    ref.append(-1, harness.to_np(k), harness.to_np(v), pos)
    qn = harness.to_np(q)
    for b in (0, 2, 3):
        for lay in range(3):
            ts = sorted({0, T - 1, *(int(t) for t in rng.integers(0, T, 3))})
            want = np.stack([[ref.attend(lay, b, j, qn[lay, b, j, t], pos[b] + t + 1) for t in ts] for j in range(16)])
            harness.assert_attention_close(out[lay, b][:, ts], want, TOL)
    br.check_state(gpu, ref, [(lay, b, h) for lay in (0, 2) for b in (0, 2, 3) for h in (0, 3)])


@pytest.mark.parametrize("T", [1, 20, 150])
def test_the_ring_is_read_in_full(T):
    """Tokens of earlier calls are what the ring holds, floats, in a bf16 cache too (as decode reads them)."""
    rng = np.random.default_rng(32)
    gpu, ref = br.make(1, 2, 4, 2, 400, window=64)
    pos = [127, 127]
    _append(gpu, ref, 0, rng, 127, [0, 0], "bf16")
    n = 2 * 2 * 64 * 128 * 4
    v0 = lib.kv_cache_bytes(gpu.cfg) - -(-2 * 7 * 2 * 16416 // 256) * 256 - n
    p = np.arange(96, 127)                       # of a block that is not yet coded
    for side, o in enumerate((v0 - n, v0)):
        ring = gpu.buffer[o:o + n].view(torch.float32).view(2, 2, 64, 128)
        x = rng.standard_normal((2, 2, len(p), 128)).astype(np.float32)
        ring[:, :, torch.as_tensor(p % 64).cuda()] = torch.as_tensor(x).cuda()
        ref.raw[side][0, :, :, p] = np.moveaxis(x, 2, 0)
    _check_decode(gpu, ref, rng, pos, "bf16")
    k, v, q = (_vectors(rng, (2, h, T), "bf16") for h in (2, 2, 4))
    # (bounded by float's error: bf16's would be 4e-3)
    _check_prefill(gpu, ref, rng, k, v, q, pos)
    br.check_state(gpu, ref, _units(gpu.cfg))


def test_many_row_tiles_captured():
    """The count of row tiles taken begins anew with each replay, at other positions too."""
    rng = np.random.default_rng(33)
    a, _ = br.make(4, 4, 16, 2, 1200, window=64)
    b, _ = br.make(4, 4, 16, 2, 1200, window=64)
    T = 500
    k, v, q = (torch.zeros(4, 2, h, T, 128, dtype=torch.bfloat16, device="cuda") for h in (4, 4, 16))
    pos, out = _i32([0, 0]), torch.zeros(4, 2, 16, T, 128, device="cuda")
    for x in (a, b):
        x.prefill(-1, k, v, q, pos, out=out)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        b.prefill(-1, k, v, q, pos, out=out)
    for p in ([0, 0], [500, -1], [650, 500], [0, 0]):
        for x, h in ((k, 4), (v, 4), (q, 16)):
            x.copy_(_vectors(rng, (4, 2, h, T), "bf16"))
        pos.copy_(_i32(p))
        graph.replay()
        assert torch.equal(out, a.prefill(-1, k, v, q, _i32(p)))
    assert a.status() == 0 and b.status() == 0

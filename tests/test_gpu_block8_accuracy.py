"""Prefill over KVQ_Q8B32 caches, row by row: what a query does not attend to, or hardly, costs its output no bits.

The error of a row (one query of one head) is measured against S = sum_j p_j rms(v_j), p its weights: RMS over the 128
channels, which a rotation keeps.  Bound, with A = max_j |q| |k_j| log2(e) / sqrt(128) over the attended j:

  a logit is off by A (2 * 2^-22 (operands of 22 bits) + 24 * 2^-23 (up to 24 truncated sums, each below A)) and by 2^-18
  (exponents of up to 64, rounded twice in float): dl; a weight by ln 2 dl, an average of values by twice that;
  the products with the values: their weights and values have 22 bits, 24 truncated sums: 2 * 2^-22 + 24 * 2^-23, and as
  much again for float sums over tiles and the rotation back;
  weights below the largest's 2^-29 are rounded to multiples of 2^-28 of the largest, n of them: n 2^-28.
"""

import numpy as np
import pytest
import torch

from . import block_reference as br
from . import harness
from .test_gpu_block8 import _i32

pytestmark = pytest.mark.gpu

LOG2E = 1.4426950408889634
SUMS = 2 * 2.0 ** -22 + 24 * 2.0 ** -23


def _rows(ref, b, j, q, p, t):
    """(output, S, A, n) in 64 bits of one query (head j, token t of a chunk at p)."""
    h = j // (ref.cfg.n_q_heads // ref.cfg.n_kv_heads)
    L = p + t + 1
    m = max(0, L - ref.cfg.window)
    k, v = (np.concatenate([ref.records(s, 0, b, h, m), ref.raw[s][0, b, h, m:L].astype(np.float64)]) for s in range(2))
    q = q.astype(np.float64)
    lg = k @ q / np.sqrt(128.0)
    w = np.exp(lg - lg.max())
    w /= w.sum()
    A = np.linalg.norm(q) * np.linalg.norm(k, axis=1).max() * LOG2E / np.sqrt(128.0)
    return w @ v, w @ np.sqrt((v * v).mean(1)), A, L


def _check(out, ref, b, q, p, ts, typical=None):
    """Every head's row of the tokens ts."""
    errs = []
    for j in range(q.shape[1]):
        for t in ts:
            want, S, A, n = _rows(ref, b, j, q[b, j, t], p, t)
            err = np.sqrt(((out[b, j, t] - want) ** 2).mean())
            tol = 2 * np.log(2) * (A * SUMS + 2.0 ** -18) + 2 * SUMS + n * 2.0 ** -28
            assert err <= tol * S + 1e-37, (j, t, err / S, tol)
            errs.append(err / S)
    if typical is not None:
        assert np.median(errs) <= typical, np.median(errs)
    return errs


def _to(x, in_dtype):
    return torch.as_tensor(np.asarray(x, np.float32)).to(torch.bfloat16 if in_dtype == "bf16" else torch.float32).contiguous()


def _prefill(gpu, ref, k, v, q, p):
    out = gpu.prefill(0, k.cuda(), v.cuda(), q.cuda(), _i32([p])).double().cpu().numpy()
    assert gpu.status() == 0
    ref.append(0, harness.to_np(k), harness.to_np(v), [p])
    return out


def _normal(rng, h, T):
    return rng.standard_normal((1, h, T, 128))


@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("p,T,window", [(0, 300, 128), (1000, 90, 64), (517, 1, 100), (3000, 40, 128)])
def test_both_planes_of_every_product(in_dtype, p, T, window):
    """Peaked attention (logits of 9 and more): weights feel the last bits of queries and keys.  Logits of about 9 are off by
    24 * 2^-23 * 9 = 2.6e-5 at most, a third of it on average, and half of that cancels between weight and sum: 2e-5 is
    kept by the median row, where queries, weights or float values without their lower parts (2^-12 each) give 1e-4."""
    rng = np.random.default_rng(p + T)
    gpu, ref = br.make(1, 2, 8, 1, p + T, window=window, in_dtype=in_dtype)
    if p:
        k, v = (_to(_normal(rng, 2, p), in_dtype) for _ in range(2))
        gpu.append(0, k.cuda(), v.cuda(), _i32([0]))
        ref.append(0, harness.to_np(k), harness.to_np(v), [0])
    k, v, q = _to(_normal(rng, 2, T), in_dtype), _to(_normal(rng, 2, T), in_dtype), _to(3 * _normal(rng, 8, T), in_dtype)
    out = _prefill(gpu, ref, k, v, q, p)
    _check(out, ref, 0, harness.to_np(q), p, sorted({0, T // 3, T // 2, T - 1}), typical=2e-5)


@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["values", "keys", "both"])
@pytest.mark.parametrize("size", [2.0 ** 16, 2.0 ** 40, 2.0 ** -30])
@pytest.mark.parametrize("p", [0, 77])
def test_later_tokens_take_no_bits(in_dtype, what, size, p):
    """A later token of the chunk, masked for the queries before it, is far larger or smaller than they."""
    rng = np.random.default_rng(41)
    T = 60
    gpu, ref = br.make(1, 1, 4, 1, 300, window=64, in_dtype=in_dtype)
    if p:
        k, v = (_to(_normal(rng, 1, p), in_dtype) for _ in range(2))
        gpu.append(0, k.cuda(), v.cuda(), _i32([0]))
        ref.append(0, harness.to_np(k), harness.to_np(v), [0])
    k, v, q = (_normal(rng, h, T) for h in (1, 1, 4))
    for t in (20, 41):
        if what != "keys":
            v[:, :, t] *= size
        if what != "values" and size < 2.0 ** 30:
            k[:, :, t] *= size
    k, v, q = (_to(x, in_dtype) for x in (k, v, q))
    out = _prefill(gpu, ref, k, v, q, p)
    ts = [t for t in range(T) if what == "values" or t < 20]     # (logits of 2^16 behind it: the bound says nothing)
    _check(out, ref, 0, harness.to_np(q), p, ts)


@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e3, 1e5, 1e8])
@pytest.mark.parametrize("where", ["window", "chunk", "block", "first"])
def test_large_values_of_next_to_no_weight(in_dtype, size, where):
    """Tokens with values `size` times larger, whose logits are so low that even so they count for 1e-3 of the output; a sink
    and thousands of equal weights 12 powers of two below it, whose values are the small ones."""
    rng = np.random.default_rng(42)
    p, T, W = 5000, 30, 64
    gpu, ref = br.make(1, 1, 4, 1, p + T, window=W, in_dtype=in_dtype)
    d = rng.standard_normal(128)
    d /= np.linalg.norm(d)
    unit = np.sqrt(128.0) / LOG2E                       # a key of x unit d has a logit of x (base 2) under the query d
    k, v = 0.02 * rng.standard_normal((p + T, 128)), 1 + 0.1 * rng.standard_normal((p + T, 128))
    k[10] += 12 * unit * d
    v[10] *= -1
    at = {"window": range(p - 40, p - 20), "chunk": range(p + 3, p + 9), "block": range(2048, 2080), "first": range(64, 96)}[where]
    low = np.log2(size * 1e3)
    for i in at:
        k[i] = 0.02 * rng.standard_normal(128) - low * unit * d
        v[i] = size * rng.standard_normal(128)
    q = np.broadcast_to(d, (1, 4, T, 128)) * (1 + 0.01 * rng.standard_normal((1, 4, T, 1)))
    k, v, q = (_to(x, in_dtype) for x in (k[None, None], v[None, None], q))
    old, new = (x[:, :, :p].contiguous() for x in (k, v)), [x[:, :, p:].contiguous() for x in (k, v)]
    old = list(old)
    gpu.append(0, old[0].cuda(), old[1].cuda(), _i32([0]))
    ref.append(0, harness.to_np(old[0]), harness.to_np(old[1]), [0])
    out = _prefill(gpu, ref, new[0], new[1], q, p)
    _check(out, ref, 0, harness.to_np(q), p, [0, 5, 15, T - 1])


@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
def test_values_that_grow_and_shrink(in_dtype):
    """Every token's values (and some blocks') have a size of their own, over 2^60: each row is what its weights make of it."""
    rng = np.random.default_rng(43)
    p, T, W = 700, 140, 96
    gpu, ref = br.make(1, 1, 4, 1, p + T, window=W, in_dtype=in_dtype)
    k = rng.standard_normal((p + T, 128))
    size = 2.0 ** rng.integers(-30, 31, p + T)
    size[:p // 32 * 32] = np.repeat(2.0 ** rng.integers(-30, 31, p // 32), 32)
    size[64:128] = 0
    v = rng.standard_normal((p + T, 128)) * size[:, None]
    k, v, q = (_to(x, in_dtype) for x in (k[None, None], v[None, None], _normal(rng, 4, T)))
    gpu.append(0, k[:, :, :p].contiguous().cuda(), v[:, :, :p].contiguous().cuda(), _i32([0]))
    ref.append(0, harness.to_np(k[:, :, :p]), harness.to_np(v[:, :, :p]), [0])
    out = _prefill(gpu, ref, k[:, :, p:].contiguous(), v[:, :, p:].contiguous(), q, p)
    _check(out, ref, 0, harness.to_np(q), p, [0, 1, 30, 31, 64, 100, T - 1])


def test_values_of_zero_and_then_not():
    """Rows whose first positions all have values of zero, and one that attends to nothing else."""
    rng = np.random.default_rng(44)
    gpu, ref = br.make(1, 1, 4, 1, 600, window=32, in_dtype="f32")
    k, v = rng.standard_normal((1, 1, 500, 128)), rng.standard_normal((1, 1, 500, 128))
    v[:, :, :320] = 0
    k, v, q = (_to(x, "f32") for x in (k, v, _normal(rng, 4, 500)))
    out = _prefill(gpu, ref, k, v, q, 0)
    assert (out[:, :, :320] == 0).all()
    _check(out, ref, 0, harness.to_np(q), 0, [320, 321, 352, 383, 384, 499])


@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["nan value", "inf value", "nan key", "-inf key"])
@pytest.mark.parametrize("p", [0, 77])
def test_what_is_not_finite_spoils_who_attends_to_it(in_dtype, what, p):
    """A token of the chunk that is not finite makes NaN of its own query and the later ones, and nothing of the earlier ones."""
    rng = np.random.default_rng(45)
    T, at = 60, 21
    k, v, q = (_to(_normal(rng, h, T), in_dtype).cuda() for h in (2, 2, 8))
    old = [_to(_normal(rng, 2, max(p, 1)), in_dtype).cuda() for _ in range(2)]
    outs = []
    for sick in (False, True):
        gpu, _ = br.make(1, 2, 8, 1, 300, window=64, in_dtype=in_dtype)
        if p:
            gpu.append(0, old[0], old[1], _i32([0]))
        kk, vv = k.clone(), v.clone()
        if sick:
            (vv if "value" in what else kk)[0, 1, at, 5] = float(what.split()[0])
        outs.append(gpu.prefill(0, kk, vv, q, _i32([p])))
    good, out = outs
    assert torch.isfinite(good).all()
    assert torch.equal(out[:, :4], good[:, :4]) and torch.equal(out[:, 4:, :at], good[:, 4:, :at])
    assert torch.isnan(out[:, 4:, at:]).all()


@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
def test_an_earlier_token_that_is_not_finite(in_dtype):
    """... and one of an earlier call, of the queries whose window has left it: its block is what the append made of it."""
    rng = np.random.default_rng(46)
    W, p, T, at = 32, 90, 30, 65
    k, v, q = (_to(_normal(rng, h, T), in_dtype).cuda() for h in (1, 1, 4))
    old = [_to(_normal(rng, 1, p), in_dtype).cuda() for _ in range(2)]
    outs = []
    for sick in (False, True):
        gpu, _ = br.make(1, 1, 4, 1, 300, window=W, in_dtype=in_dtype)
        gpu.append(0, old[0], old[1], _i32([0]))
        if sick:
            _slots(gpu)[1][0, 0, 0, at % W, 9] = float("nan")     # (only the ring's copy)
        outs.append(gpu.prefill(0, k, v, q, _i32([p])))
    good, out = outs
    last = at + W - 1 - p                                          # the last query that attends to it raw
    assert torch.isnan(out[:, :, :last + 1]).all() and torch.isfinite(out[:, :, last + 1:]).all()
    assert torch.isfinite(good).all()


@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L,window", [(20, 32), (300, 100), (4000, 128)])
def test_decode_row_by_row(in_dtype, L, window):
    """Single tokens are held to the same bounds (the raw products are float sums of 128 and less: within them)."""
    rng = np.random.default_rng(L)
    gpu, ref = br.make(1, 2, 8, 2, L, window=window, in_dtype=in_dtype)
    k, v = (_to(rng.standard_normal((2, 2, L, 128)), in_dtype) for _ in range(2))
    gpu.append(0, k.cuda(), v.cuda(), _i32([0, 0]))
    ref.append(0, harness.to_np(k), harness.to_np(v), [0, 0])
    q = _to(3 * rng.standard_normal((2, 8, 128)), in_dtype)
    out = gpu.decode(0, q.cuda(), _i32([L, L])).double().cpu().numpy()[:, :, None]
    for b in range(2):
        _check(out, ref, b, harness.to_np(q)[:, :, None], L - 1, [0], typical=2e-5)


def _slots(gpu):
    """The rings of keys and values, [layers][batch][heads][window][128] each."""
    cfg = gpu.cfg
    a = lambda x: -(-x // 256) * 256  # noqa: E731
    n = cfg.n_layers * cfg.max_batch * cfg.n_kv_heads * cfg.window * 512
    n_pages = cfg.n_pages or cfg.max_batch * -(-cfg.max_seq_len // 64)
    v0 = br.lib.kv_cache_bytes(cfg) - a(cfg.n_layers * n_pages * cfg.n_kv_heads * 16416) - a(n)
    shape = (cfg.n_layers, cfg.max_batch, cfg.n_kv_heads, cfg.window, 128)
    return [gpu.buffer[o:o + n].view(torch.float32).view(shape) for o in (v0 - a(n), v0)]

"""Tree attention against its 64-bit definition where operands of fewer bits would show: outputs of bf16 caches that are
the definition rounded once."""

import numpy as np
import pytest
import torch

from kv_cache_quantization_append_gb300 import lib

from . import harness
from . import ops_reference as ref
from .test_gpu_tree import TOL, _drafts, _fill

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def _tree(gpu, k, v, q, lens, parents):
    out = gpu.tree_decode(0, k.cuda(), v.cuda(), q.cuda(), _i32(lens), _i32(parents))
    torch.cuda.synchronize()
    assert gpu.status() == 0
    return out.double().cpu().numpy()


def _half_step(in_dtype, want):
    return 2.0 ** -8 * np.abs(want) if in_dtype == "bf16" else 0.0


@pytest.mark.parametrize("k_format", ["q4g32", "q8g32", "tq3_qjl"])
@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_q,N,L,window", [(3, 5, 700, 128), (3, 16, 700, 0), (4, 32, 500, 64), (3, 64, 300, 128)])
def test_outputs_are_the_definition_rounded_once(k_format, in_dtype, n_q, N, L, window):
    """Peaked attention (queries of four times a unit head's size), whose logits of up to 60 magnify what queries and keys
    lose.  Each output element is off by its own half step and, beside that, by what a float cache's may be: operands of 22
    bits (of a bf16 cache's raw vectors 16: |q| |k| / sqrt(128) = 45, so six standard deviations of the logit's error are
    6 * 4 * 2^-18 / sqrt(3) = 5e-5, the values' and weights' 2^-17 each) and the truncating accumulations of 2e-4."""
    rng = np.random.default_rng(N + L)
    gpu, ora, _ = harness.make_pair(1, 1, n_q, 1, 720, window=window, k_format=k_format, in_dtype=in_dtype)
    _fill(gpu, ora, [L], L, rng, in_dtype)
    k, v, q = _drafts(rng, gpu.cfg, 1, N, in_dtype)
    q = q * 4
    parents = ref.random_tree(rng, N)[None]
    got = _tree(gpu, k, v, q, [L], parents)
    want = ref.tree_attention(ora, 0, harness.to_np(k), harness.to_np(v), harness.to_np(q), np.array([L]), parents)
    err = np.abs(got - want) - _half_step(in_dtype, want)
    assert err.max() <= TOL["f32"] * np.abs(want).max(), err.max() / np.abs(want).max()


@pytest.mark.parametrize("in_dtype,scale", [("bf16", 2.0 ** -24), ("bf16", 2.0 ** 12), ("f32", 2.0 ** -110),
                                            ("f32", 2.0 ** -24), ("f32", 2.0 ** -10), ("f32", 2.0 ** 12)])
def test_raw_values_of_any_size(in_dtype, scale):
    """Values in the ring and the drafts far below and above one: the output scales with them."""
    rng = np.random.default_rng(3)
    gpu, ora, _ = harness.make_pair(1, 2, 4, 1, 200, in_dtype=in_dtype)
    dt = torch.bfloat16 if in_dtype == "bf16" else torch.float32
    _fill(gpu, ora, [100], 100, rng, in_dtype)
    kk, vv = (torch.as_tensor((rng.standard_normal((1, 2, 100, 128)) * s).astype(np.float32)).to(dt) for s in (1, scale))
    gpu.append(0, kk.cuda(), vv.cuda(), _i32([0]))
    ora.append(0, harness.to_np(kk), harness.to_np(vv), np.zeros(1, int))
    k, v, q = _drafts(rng, gpu.cfg, 1, 9, in_dtype)
    v = v * scale
    parents = ref.random_tree(rng, 9)[None]
    got = _tree(gpu, k, v, q, [100], parents)
    want = ref.tree_attention(ora, 0, harness.to_np(k), harness.to_np(v), harness.to_np(q), np.array([100]), parents)
    err = np.abs(got - want) - _half_step(in_dtype, want)
    assert err.max() <= TOL["f32"] * np.abs(want).max(), err.max() / np.abs(want).max()


@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gap", [12.0, 16.7, 17.3, 20.0])
def test_positions_behind_a_sink_keep_their_weight(in_dtype, gap):
    """The first position's logit is ``gap`` above all others, its value small: the output is the sum of thousands of weights
    of e^-gap.  160 sequences share the pages, so that a CTA meets the sink and many tiles behind it.  A weight's absolute
    error is at most 2^-32 of the sink's (below half of e^-gap 2^-2 for each gap here), 6400 of them 1.5e-6 of it; outputs are
    at least 0.02, so 1e-4 of the largest, within the float bound; bf16 adds its half step."""
    rng = np.random.default_rng(2)
    B, L = 160, 6400
    pages = np.tile(np.arange(L // 64, dtype=np.int32), (B, 1))
    gpu, _, _ = harness.make_pair(1, 2, 2, B, L, window=0, k_format="q8g32", in_dtype=in_dtype, n_pages=L // 64, block_table=pages)
    ora = harness.make_pair(1, 2, 2, 1, L, window=0, k_format="q8g32", in_dtype=in_dtype)[1]
    dt = torch.bfloat16 if in_dtype == "bf16" else torch.float32
    u = rng.standard_normal(128)
    u /= np.linalg.norm(u)
    k, v = rng.standard_normal((1, 2, L, 128)) * 0.05, 1 + 0.3 * rng.standard_normal((1, 2, L, 128))
    k[:, :, 0] += u * gap
    v[:, :, 0] = -0.05
    k, v = (torch.as_tensor(x.astype(np.float32)).to(dt) for x in (k, v))
    wide = lambda t: t.expand(B, *t.shape[1:]).contiguous()  # noqa: E731
    pos = np.full(B, -1)
    pos[0] = 0
    gpu.append(0, wide(k).cuda(), wide(v).cuda(), _i32(pos))
    ora.append(0, harness.to_np(k), harness.to_np(v), np.zeros(1, int))
    q = torch.as_tensor(np.tile(u * 128 ** 0.5, (1, 2, 1, 1)).astype(np.float32)).to(dt)
    dk = torch.as_tensor((rng.standard_normal((1, 2, 1, 128)) * 0.05).astype(np.float32)).to(dt)
    dv = torch.ones(1, 2, 1, 128, dtype=dt)
    got = _tree(gpu, wide(dk), wide(dv), wide(q), [L] * B, [[-1]] * B)
    want = ref.tree_attention(ora, 0, *(harness.to_np(t) for t in (dk, dv, q)), np.array([L]), np.array([[-1]]))
    err = np.abs(got - want) - _half_step(in_dtype, want)
    assert err.max() <= TOL["f32"] * np.abs(want).max(), err.max() / np.abs(want).max()


@pytest.mark.parametrize("k_format", ["q4g32", "q8g32", "tq3_qjl"])
@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
def test_queries_of_absent_nodes_touch_no_other_row(k_format, in_dtype):
    """What the queries of nodes that are not there hold -- finite values whose rotated channels pass fp16's range here and
    there, infinities, NaN -- leaves the rows beside them as they are, over tiles that every node reads in full."""
    rng = np.random.default_rng(9)
    B, L = 120, 900
    pages = np.tile(np.arange(15, dtype=np.int32), (B, 1))
    gpu, ora, _ = harness.make_pair(1, 2, 4, B, 960, window=64, k_format=k_format, in_dtype=in_dtype, n_pages=15, block_table=pages)
    dt = torch.bfloat16 if in_dtype == "bf16" else torch.float32
    k, v = (torch.as_tensor(rng.standard_normal((B, 2, L, 128)).astype(np.float32)).to(dt) for _ in range(2))
    pos = np.full(B, -1)
    pos[0] = 0
    gpu.append(0, k.cuda(), v.cuda(), _i32(pos))           # (the other sequences read the first one's pages, rings of their own)
    pos[:] = L - 64
    gpu.append(0, k[:1, :, L - 64:].expand(B, 2, 64, 128).contiguous().cuda(), v[:1, :, L - 64:].expand(B, 2, 64, 128).contiguous().cuda(), _i32(pos))
    k, v, q = _drafts(rng, gpu.cfg, B, 7, in_dtype)
    parents = [[-1, 0, -2, 1, -2, 0, 4]] * B               # 2 and 4 are not there, nor is 4's child
    gone = [2, 4, 6]
    q[:, :, gone] = 0
    base = _tree(gpu, k, v, q, [L] * B, parents)
    assert np.isfinite(base).all() and (base[:, :, gone] == 0).all()
    for b in range(B):                                     # from 2^14 to 2^20, then infinities and NaN
        q[b, :, gone] = torch.as_tensor(rng.standard_normal((4, 3, 128)).astype(np.float32) * 2.0 ** (14 + 6 * b / (B - 4))).to(dt)
    q[-3, :, gone], q[-2, :, gone], q[-1, :, gone] = float("inf"), float("-inf"), float("nan")
    got = _tree(gpu, k, v, q, [L] * B, parents)
    assert [b for b in range(B) if not np.array_equal(got[b], base[b])] == []


@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [float("inf"), 3e38])
def test_a_query_out_of_range_spoils_its_own_row_only(in_dtype, value):
    """Nodes whose query holds infinities, or values so large that products with keys above one overflow, in two channels: by
    the keys' signs their logits are infinities of both signs and NaN.  Every other row is what it is without them."""
    rng = np.random.default_rng(19)
    gpu, ora, _ = harness.make_pair(1, 2, 4, 2, 500, in_dtype=in_dtype)
    lens = [400, 90]
    _fill(gpu, ora, lens, 400, rng, in_dtype)
    k, v, q = _drafts(rng, gpu.cfg, 2, 9, in_dtype)
    k[:, :, 0, 3] = 0
    parents = np.stack([ref.random_tree(rng, 9, chain=True)] * 2)
    base = _tree(gpu, k, v, q, lens, parents)
    q[:, :, 2, 3:5], q[:, 1:3, 5, 3:5] = value, -value
    got = _tree(gpu, k, v, q, lens, parents)
    bad = np.zeros((2, 4, 9), bool)
    bad[:, :, 2] = bad[:, 1:3, 5] = True
    assert not np.isfinite(got[bad]).all(-1).any()
    assert np.array_equal(got[~bad], base[~bad])


@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_values_that_are_not_finite_reach_who_attends_to_them(in_dtype, value):
    """An infinity or NaN in a draft's value or key: outputs of the node and its descendants are not finite, those of the
    other branches are what they are without it.  The same in a ring slot that only shallow nodes read raw."""
    rng = np.random.default_rng(29)
    gpu, ora, _ = harness.make_pair(1, 2, 6, 2, 500, window=8, in_dtype=in_dtype)
    lens = np.array([400, 90])
    _fill(gpu, ora, lens, 400, rng, in_dtype)
    k, v, q = _drafts(rng, gpu.cfg, 2, 9, in_dtype)
    parents = np.array([[-1, 0, 0, 1, 1, 2, 3, -1, 7]] * 2)
    base = _tree(gpu, k, v, q, lens, parents)
    hit = np.array([i for i in range(9) if 1 in ref.chain_of(parents[0], i)])
    rest = np.setdiff1d(np.arange(9), hit)
    v2, k2 = v.clone(), k.clone()
    v2[:, :, 1, 77] = value
    k2[:, :, 1, 5] = value
    for kk, vv in ((k, v2), (k2, v)):
        got = _tree(gpu, kk, vv, q, lens, parents)
        assert np.array_equal(got[:, :, rest], base[:, :, rest])
        assert not np.isfinite(got[:, :, hit]).all(-1).any()
    # the oldest raw position, L - 7: read raw by nodes at depth 0, through its record by deeper ones
    at = harness.layout.regions(gpu.cfg, gpu.buffer.numel())["off_ringv"]
    ring = gpu.buffer[at:at + 2 * 2 * 8 * 128 * 4].view(torch.float32).view(2, 2, 8, 128)
    for b, L in enumerate(lens):
        ring[b, :, (int(L) - 7) % 8, 100] = value
    got = _tree(gpu, k, v, q, lens, parents)
    shallow = [0, 7]
    deep = np.setdiff1d(np.arange(9), shallow)
    assert np.array_equal(got[:, :, deep], base[:, :, deep]) and not np.isfinite(got[:, :, shallow]).all(-1).any()


@pytest.mark.parametrize("window", [0, 8, 128])
def test_where_a_chain_is_what_single_tokens_see(window):
    """Nodes that the window covers (depth < window) equal their own single-token steps; deeper ones read their path raw where
    those read records, which shows."""
    rng = np.random.default_rng(5)
    gpu, ora, _ = harness.make_pair(1, 1, 2, 1, 400, window=window, in_dtype="f32")
    _fill(gpu, ora, [90], 90, rng, "f32")
    k, v, q = _drafts(rng, gpu.cfg, 1, 14, "f32")
    got = _tree(gpu, k, v, q, [90], ref.random_tree(rng, 14, chain=True)[None])
    for i in range(14):
        ora.append(0, harness.to_np(k[:, :, i:i + 1]), harness.to_np(v[:, :, i:i + 1]), np.array([90 + i]))
        step = ora.decode(0, harness.to_np(q[:, :, i]), np.array([91 + i]))
        err = np.abs(got[:, :, i] - step).max() / np.abs(step).max()
        assert err <= TOL["f32"] if i < window else err > 10 * TOL["f32"], (i, err)


@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
def test_long_contexts_sum_as_short_ones(in_dtype):
    """512 tiles in one CTA (320 units that share their pages), values of one sign: the tensor cores cut off every sum's low
    bits, so that 512 tiles of 24 sums in one accumulator would lose 512 * 24 * 2^-24 = 7e-4 of the last sum, half of it on the
    way up to it.  Sums of 16 tiles lose 2.3e-5 at most, and are joined with rounding to nearest."""
    rng = np.random.default_rng(31)
    B, L = 160, 65536
    pages = np.tile(np.arange(L // 64, dtype=np.int32), (B, 1))
    gpu, _, _ = harness.make_pair(1, 2, 2, B, L, window=0, in_dtype=in_dtype, n_pages=L // 64, block_table=pages)
    ora = harness.make_pair(1, 2, 2, 1, L, window=0, in_dtype=in_dtype)[1]
    dt = torch.bfloat16 if in_dtype == "bf16" else torch.float32
    for at in range(0, L, 8192):
        k = torch.as_tensor(rng.standard_normal((1, 2, 8192, 128)).astype(np.float32)).to(dt)
        v = torch.as_tensor((1 + 0.3 * rng.standard_normal((1, 2, 8192, 128))).astype(np.float32)).to(dt)
        one = lib.kvq_cache.from_buffer_copy(gpu.handle)       # (the first sequence's pages are everyone's)
        lib.kv_quant_append(one, 0, k.cuda(), v.cuda(), _i32([at]))
        ora.append(0, harness.to_np(k), harness.to_np(v), np.array([at]))
    k, v, q = _drafts(rng, gpu.cfg, 1, 1, in_dtype)
    wide = lambda t: t.expand(B, *t.shape[1:]).contiguous()  # noqa: E731
    got = _tree(gpu, wide(k), wide(v), wide(q), [L] * B, [[-1]] * B)
    want = ref.tree_attention(ora, 0, *(harness.to_np(t) for t in (k, v, q)), np.array([L]), np.array([[-1]]))
    err = np.abs(got - want) - _half_step(in_dtype, want)
    assert err.max() <= 0.25 * TOL["f32"] * np.abs(want).max(), err.max() / np.abs(want).max()

"""Attention weights of cached positions and eviction by them, against the 64-bit definitions."""

import os
import subprocess
import sys

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


def _check_weights(gpu, ora, q, lens, decay, rng, layer=0):
    B, S = len(lens), gpu.cfg.max_seq_len
    before = rng.random((B, gpu.cfg.n_kv_heads, S)).astype(np.float32)
    if decay == 0:
        before[:] = np.nan                          # written without being read
    w = torch.as_tensor(before).cuda()
    gpu.attention_weights(layer, q.cuda(), _i32(lens), w, decay)
    torch.cuda.synchronize()
    assert gpu.status() == 0
    want = ref.attention_weights(ora, layer, harness.to_np(q), lens, before, np.float32(decay))
    got = w.double().cpu().numpy()
    for b, L in enumerate(lens):
        # logits from operands of 22 bits: |q| |k| / sqrt(128) is at most about 40 here, so 2 * 40 * 2^-20 = 8e-5 relative;
        # the sums and the old weight add a few 2^-24 of the result
        err = np.abs(got[b, :, :L] - want[b, :, :L])
        assert (err <= 1e-4 * want[b, :, :L] + 1e-12).all(), (b, (err / (want[b, :, :L] + 1e-12)).max())
        assert np.array_equal(got[b, :, L:], before[b, :, L:].astype(np.float64), equal_nan=True)
    return w


@pytest.mark.parametrize("k_format", ["q4g32", "q8g32", "tq3_qjl"])
@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_q,n_kv,T,window,decay", [(2, 2, 1, 128, 1.0), (6, 2, 5, 128, 0.0), (8, 2, 17, 64, 0.5), (4, 1, 64, 0, 1.0),
                                                     (3, 3, 33, 4, 0.0)])
def test_weights_match_definition(k_format, in_dtype, n_q, n_kv, T, window, decay):
    rng = np.random.default_rng(T * 5 + n_q)
    lens = np.array([300, 0, 1, 129, 64, 190])
    gpu, ora, _ = harness.make_pair(1, n_kv, n_q, 6, 320, window=window, k_format=k_format, in_dtype=in_dtype)
    _fill(gpu, ora, lens, 300, rng, in_dtype)
    _, _, q = _drafts(rng, gpu.cfg, 6, T, in_dtype)
    _check_weights(gpu, ora, q, lens, decay, rng)


@pytest.mark.parametrize("L", [31, 63, 65, 127, 128, 129, 192, 193, 700])
def test_weights_lengths_and_unit_sum(L):
    rng = np.random.default_rng(L)
    gpu, ora, _ = harness.make_pair(1, 1, 3, 1, 720, window=60)
    _fill(gpu, ora, [L], L, rng, "bf16")
    _, _, q = _drafts(rng, gpu.cfg, 1, 2, "bf16")
    w = _check_weights(gpu, ora, q, np.array([L]), 0.0, rng)
    assert abs(w[0, 0, :L].double().sum().item() - 6) < 6e-4   # every query's softmax sums to one


def test_weights_sinkhorn_paged_all_layers():
    rng = np.random.default_rng(31)
    bt = rng.permutation(3 * 5 + 4)[:15].reshape(3, 5).astype(np.int32)
    gpu, ora, _ = harness.make_pair(2, 2, 8, 3, 300, sinkhorn=True, n_pages=19, block_table=bt)
    for layer in range(2):
        c = torch.as_tensor(rng.standard_normal((2, 2, 256, 128)).astype(np.float32) * 2).bfloat16()
        gpu.calibrate(layer, c[0].cuda(), c[1].cuda())
        ora.calibrate(layer, harness.to_np(c[0]), harness.to_np(c[1]))
    lens = np.array([290, 64, 200])
    _fill(gpu, ora, lens, 290, rng, "bf16", layers=2)
    _, _, q = _drafts(rng, gpu.cfg, 3, 3, "bf16", layers=2)
    w = torch.ones(2, 3, 2, 300, device="cuda")
    gpu.attention_weights(-1, q.cuda(), _i32(lens), w, 0.25)
    for layer in range(2):
        want = ref.attention_weights(ora, layer, harness.to_np(q[layer]), lens, np.ones((3, 2, 300)), 0.25)
        assert np.abs(w[layer].double().cpu().numpy() - want).max() < 1e-4 * want.max()


@pytest.mark.parametrize("k_format", ["q4g32", "q8g32", "tq3_qjl"])
@pytest.mark.parametrize("g,T", [(3, 6), (3, 22), (2, 64), (3, 43), (4, 40)])
def test_weights_row_counts_around_the_blocks(k_format, g, T):
    """18, 66, 128, 129 and 160 rows a KV head: blocks of 16 or 32 rows full or not, one launch or two."""
    rng = np.random.default_rng(50 * g + T)
    gpu, ora, _ = harness.make_pair(1, 1, g, 2, 460, window=40, k_format=k_format)
    lens = np.array([450, 333])
    _fill(gpu, ora, lens, 450, rng, "bf16")
    _, _, q = _drafts(rng, gpu.cfg, 2, T, "bf16")
    _check_weights(gpu, ora, q, lens, 0.5, rng)


def test_first_call_of_a_process_may_be_of_any_size():
    """Shared-memory limits are set per kernel and device: a call's own must not depend on a larger one before it."""
    code = """
import torch
import kv_cache_quantization_append_gb300 as kvq
for n_q, n in ((24, 8), (8, 1), (16, 4), (32, 8), (32, 32)):
    c = kvq.QuantKVCache(kvq.make_config(1, 8, n_q, 1, 400))
    k = torch.randn(1, 8, 300, 128, device="cuda").bfloat16()
    ln = torch.tensor([300], dtype=torch.int32, device="cuda")
    c.append(0, k, k, torch.zeros_like(ln))
    w = torch.zeros(1, 8, 400, device="cuda")
    q = torch.randn(1, n_q, n, 128, device="cuda").bfloat16()
    c.attention_weights(0, q, ln, w)
    assert abs(w.sum().item() / (n_q * n) - 1) < 1e-3, (n_q, n, w.sum().item())
    c.tree_decode(0, k[:, :, :n].contiguous(), k[:, :, :n].contiguous(), q, ln, torch.arange(-1, n - 1, dtype=torch.int32, device="cuda")[None])
    torch.cuda.synchronize()
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_weights_deterministic_and_captured():
    rng = np.random.default_rng(33)
    gpu, ora, _ = harness.make_pair(1, 8, 24, 2, 3000)
    lens = np.array([2900, 700])
    _fill(gpu, ora, lens, 2900, rng, "bf16")
    _, _, q = _drafts(rng, gpu.cfg, 2, 8, "bf16")
    q, ln = q.cuda(), _i32(lens)
    first = gpu.attention_weights(0, q, ln, torch.zeros(2, 8, 3000, device="cuda"), 1.0)
    for _ in range(3):
        assert torch.equal(gpu.attention_weights(0, q, ln, torch.zeros(2, 8, 3000, device="cuda"), 1.0), first)
    w = torch.zeros(2, 8, 3000, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu.attention_weights(0, q, ln, w, 1.0)
    ln.copy_(_i32([5, 2000]))
    graph.replay()
    graph.replay()
    one = gpu.attention_weights(0, q, ln, torch.zeros(2, 8, 3000, device="cuda"), 1.0)
    # the second sequence is read past what was appended: whatever the pages hold (NaN among it), both calls see the same
    torch.testing.assert_close(w, 2 * one, rtol=0, atol=0, equal_nan=True)


# ---------------------------------------------------------------------------- eviction
def _weights_like(rng, shape, kind):
    w = rng.random(shape).astype(np.float32)
    if kind == "ties":
        w = np.floor(w * 4) / 4
    elif kind == "equal":
        w[:] = 0.5
    elif kind == "odd":                             # signs, zeros of both signs, infinities and NaN
        w = (w - 0.5) * 1e3
        w[rng.random(shape) < 0.2] = 0.0
        w[rng.random(shape) < 0.2] = -0.0
        w[rng.random(shape) < 0.05] = np.inf
        w[rng.random(shape) < 0.05] = -np.inf
        w[rng.random(shape) < 0.1] = np.nan
    return w


@pytest.mark.parametrize("k_format", ["q4g32", "q8g32", "tq3_qjl"])
@pytest.mark.parametrize("budget,recent,window,kind", [(130, 128, 128, "plain"), (257, 200, 64, "ties"), (100, 100, 4, "equal"),
                                                       (311, 0, 0, "odd"), (33, 1, 0, "equal"), (1, 0, 0, "plain"),
                                                       (289, 64, 60, "odd")])
def test_evict_matches_definition(k_format, budget, recent, window, kind):
    rng = np.random.default_rng(budget)
    bt = rng.permutation(4 * 5 + 2)[:20].reshape(4, 5).astype(np.int32)
    gpu, ora, _ = harness.make_pair(2, 2, 2, 4, 320, window=window, k_format=k_format, n_pages=22, block_table=bt)
    lens = np.array([320, 260, 0, 97])
    _fill(gpu, ora, lens, 320, rng, "bf16", layers=2)
    w = _weights_like(rng, (2, 4, 2, 320), kind)
    wd = torch.as_tensor(w).cuda()
    before = gpu.buffer.clone()
    kept, new = gpu.evict(-1, wd, _i32(lens), budget, recent)
    torch.cuda.synchronize()
    assert gpu.status() == 0
    want = ref.evict(ora, w, lens, budget, recent)
    assert np.array_equal(kept.cpu().numpy(), want)
    assert np.array_equal(new.cpu().numpy(), np.minimum(lens, budget))
    assert np.array_equal(wd.cpu().numpy(), w, equal_nan=True)
    for layer in range(2):
        for b in range(4):
            for h in range(2):
                n = int(min(lens[b], budget))
                if n:
                    harness.compare_codes(gpu, ora, layer, b, h, max(n, int(lens[b])), bt)  # moved, and left as they were
                    harness.compare_ring(gpu, ora, layer, b, h, n)
    assert torch.equal(gpu.buffer[:1024], before[:1024])   # signs and codebook


def test_evict_long_context_one_layer_at_a_time():
    """More positions than a CTA's threads, skewed weights; per-layer calls equal the all-layer call."""
    rng = np.random.default_rng(41)
    gpu, ora, _ = harness.make_pair(2, 1, 1, 2, 5000)
    lens = np.array([4999, 3333])
    _fill(gpu, ora, lens, 4999, rng, "bf16", layers=2)
    w = np.exp(8 * rng.random((2, 2, 1, 5000))).astype(np.float32)
    wd = torch.as_tensor(w).cuda()
    for layer in range(2):
        kept, _ = gpu.evict(layer, wd[layer], _i32(lens), 2049, 130)
        got = kept.cpu().numpy()
        for b in range(2):
            assert np.array_equal(got[b, 0], ref.kept_positions(w[layer, b, 0], int(lens[b]), 2049, 130))
    ref.evict(ora, w, lens, 2049, 130)
    assert np.array_equal(wd.cpu().numpy(), w)
    for layer in range(2):
        for b in range(2):
            harness.compare_codes(gpu, ora, layer, b, 0, 2049)
            harness.compare_ring(gpu, ora, layer, b, 0, 2049)


def test_evict_flags_a_length_out_of_range():
    gpu, _, _ = harness.make_pair(1, 1, 1, 2, 100, window=0)
    before = gpu.buffer.clone()
    kept, new = gpu.evict(0, torch.zeros(2, 1, 100, device="cuda"), _i32([101, -1]), 10, 2)
    assert gpu.status() == lib.DEV_SEQLEN_RANGE
    assert (kept == -1).all() and (new == 0).all() and torch.equal(gpu.buffer, before)


def test_evict_bad_page():
    """A page out of range: its records count as zeros, slots in it are not written, other pages are."""
    rng = np.random.default_rng(43)
    bt = np.arange(4, dtype=np.int32)[None]
    gpu, ora, _ = harness.make_pair(1, 1, 1, 1, 256, window=0, n_pages=4, block_table=bt)
    _fill(gpu, ora, [256], 256, rng, "bf16")
    before = gpu.buffer.clone()
    w = np.zeros((1, 1, 256), np.float32)
    w[0, 0, 64:192] = 1
    gpu.block_table[0, 1] = -7
    gpu.evict(0, torch.as_tensor(w).cuda(), _i32([256]), 128, 0)
    assert gpu.status() == lib.DEV_BAD_PAGE
    got = harness.layout.read_unit(gpu.buffer, gpu.cfg, 0, 0, 0, 64, bt)
    assert (got["k_scale"] == 0).all() and (got["v_code"] == 0).all()
    page = 2 * 5120
    off = gpu.buffer.numel() - 4 * page
    assert torch.equal(gpu.buffer[off + page:], before[off + page:])


# ---------------------------------------------------------------------------- the loop they serve
@pytest.mark.parametrize("k_format", ["q4g32", "tq3_qjl"])
def test_decode_loop_with_drafts_and_eviction(k_format):
    """Rows of a projection -> rotated q, k, v -> prompt append -> weights -> eviction -> drafts -> commit -> decode, each step
    against the definitions on the oracle's cache."""
    rng = np.random.default_rng(51)
    B, hq, hkv, S, T = 2, 6, 2, 512, 400
    gpu, ora, _ = harness.make_pair(1, hkv, hq, B, S, window=64, k_format=k_format)
    rope = lib.kv_rope_init(128, theta=500000.0)
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")

    def project(n, positions):
        x = torch.as_tensor(rng.standard_normal((B, n, (hq + 2 * hkv) * 128)).astype(np.float32)).bfloat16().cuda()
        q = torch.empty(B, hq, n, 128, dtype=torch.bfloat16, device="cuda")
        k, v = (torch.empty(B, hkv, n, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        lib.kv_qk_norm_rope(rope, x, _i32(positions), q, k, v, w, w)
        return q, k, v

    q, k, v = project(T, np.arange(T)[None].repeat(B, 0))
    gpu.append(0, k, v, _i32([0] * B))
    ora.append(0, harness.to_np(k), harness.to_np(v), np.zeros(B, int))
    lens = np.array([T] * B)
    weights = torch.zeros(B, hkv, S, device="cuda")
    gpu.attention_weights(0, q[:, :, -16:].contiguous(), _i32(lens), weights, 0.0)
    host = weights.cpu().numpy()
    want = ref.attention_weights(ora, 0, harness.to_np(q[:, :, -16:]), lens, np.zeros((B, hkv, S)), 0.0)
    assert np.abs(host - want).max() <= 1e-4 * want.max()
    _, new = gpu.evict(0, weights, _i32(lens), 150, 64)
    ref.evict(ora, host[None], lens, 150, 64)
    true_pos = T                                      # rotary positions go on; cache slots start after the cut
    lens = np.array([150] * B)
    assert np.array_equal(new.cpu().numpy(), lens)
    for _ in range(3):
        parents = np.stack([ref.random_tree(rng, 8) for _ in range(B)])
        depth = np.array([[len(ref.chain_of(p, i)) - 1 for i in range(8)] for p in parents])
        q, k, v = project(8, true_pos + depth)
        out = gpu.tree_decode(0, k, v, q, _i32(lens), _i32(parents))
        want = ref.tree_attention(ora, 0, harness.to_np(k), harness.to_np(v), harness.to_np(q), lens, parents)
        harness.assert_attention_close(out.double().cpu().numpy(), want, TOL["bf16"])
        paths = [max((ref.chain_of(p, i) for i in range(8)), key=len) for p in parents]
        n = np.array([len(p) for p in paths])
        path = np.array([p + [0] * (8 - len(p)) for p in paths])
        gpu.commit(0, k, v, _i32(path), _i32(n), _i32(lens))
        for b in range(B):
            one = np.full(B, -1)
            one[b] = lens[b]
            ora.append(0, harness.to_np(k)[:, :, paths[b]], harness.to_np(v)[:, :, paths[b]], one)
        lens = lens + n
        true_pos += int(n.max())
        q, k, v = project(1, np.full((B, 1), true_pos))
        gpu.append(0, k, v, _i32(lens))
        ora.append(0, harness.to_np(k), harness.to_np(v), lens)
        lens = lens + 1
        got = gpu.decode(0, q[:, :, 0].contiguous(), _i32(lens))
        harness.assert_attention_close(got.cpu().numpy(), ora.decode(0, harness.to_np(q[:, :, 0]), lens))
        true_pos += 1
    for b in range(B):
        for h in range(hkv):
            harness.compare_codes(gpu, ora, 0, b, h, int(lens[b]))
    assert gpu.status() == 0

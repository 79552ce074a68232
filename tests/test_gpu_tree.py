"""Trees of drafted tokens over the cache: attention against the 64-bit definition, and the accepted path's append."""

import numpy as np
import pytest
import torch

from kv_cache_quantization_append_gb300 import lib

from . import harness
from . import ops_reference as ref

pytestmark = pytest.mark.gpu

# Attention outputs: the framework's 2e-3 of the largest value for bf16 caches (operands rounded once to fp16), plus the
# output's own half step 2^-8; float caches: operands of 22 bits and at most 2^9 truncating accumulations of 2^-23 in a row
# (6e-5), times three
TOL = {"bf16": 2e-3 + 2.0 ** -8, "f32": 2e-4}


def _fill(gpu, ora, lens, T, rng, in_dtype, layers=1, scale=1.0):
    """Append T tokens of every sequence (the first lens[b] count) to both caches."""
    cfg = gpu.cfg
    dt = torch.bfloat16 if in_dtype == "bf16" else torch.float32
    for layer in range(layers):
        k = torch.as_tensor(rng.standard_normal((cfg.max_batch, cfg.n_kv_heads, T, 128)).astype(np.float32) * scale).to(dt)
        v = torch.as_tensor(rng.standard_normal((cfg.max_batch, cfg.n_kv_heads, T, 128)).astype(np.float32)).to(dt)
        k[..., 7] *= 5
        for b in range(cfg.max_batch):
            L = int(lens[b])
            if not L:
                continue
            pos = torch.full((cfg.max_batch,), -1, dtype=torch.int32)
            pos[b] = 0
            gpu.append(layer, k[:, :, :L].contiguous().cuda(), v[:, :, :L].contiguous().cuda(), pos.cuda())
            ora.append(layer, harness.to_np(k[:, :, :L]), harness.to_np(v[:, :, :L]), pos.numpy())


def _drafts(rng, cfg, B, N, in_dtype, layers=None):
    dt = torch.bfloat16 if in_dtype == "bf16" else torch.float32
    lead = () if layers is None else (layers,)
    mk = lambda h: torch.as_tensor(rng.standard_normal(lead + (B, h, N, 128)).astype(np.float32)).to(dt)  # noqa: E731
    return mk(cfg.n_kv_heads), mk(cfg.n_kv_heads), mk(cfg.n_q_heads)


def _check(gpu, ora, k, v, q, lens, parents, in_dtype, layer=0):
    out = gpu.tree_decode(layer, k.cuda(), v.cuda(), q.cuda(), torch.as_tensor(lens, dtype=torch.int32).cuda(),
                          torch.as_tensor(parents, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert gpu.status() == 0
    want = ref.tree_attention(ora, layer, harness.to_np(k), harness.to_np(v), harness.to_np(q), lens, parents)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    for b in range(len(lens)):
        harness.assert_attention_close(got[b], want[b], TOL[in_dtype])
        for i in range(parents.shape[1]):
            if not ref.chain_of(parents[b], i):
                assert (got[b, :, i] == 0).all()
    return out


@pytest.mark.parametrize("k_format", ["q4g32", "q8g32", "tq3_qjl"])
@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_q,n_kv,N,window", [(2, 2, 1, 128), (6, 2, 5, 128), (8, 2, 17, 64), (4, 1, 64, 0), (3, 3, 33, 4)])
def test_matches_definition(k_format, in_dtype, n_q, n_kv, N, window):
    rng = np.random.default_rng(N * 7 + n_q)
    lens = np.array([300, 0, 1, 129, 64])
    gpu, ora, _ = harness.make_pair(1, n_kv, n_q, 5, 320, window=window, k_format=k_format, in_dtype=in_dtype)
    _fill(gpu, ora, lens, 300, rng, in_dtype)
    k, v, q = _drafts(rng, gpu.cfg, 5, N, in_dtype)
    parents = np.stack([ref.random_tree(rng, N) for _ in range(5)])
    _check(gpu, ora, k, v, q, lens, parents, in_dtype)


@pytest.mark.parametrize("L", [31, 32, 33, 63, 65, 127, 128, 130, 191, 192, 193, 256, 700])
def test_lengths_around_tiles_and_pages(L):
    rng = np.random.default_rng(L)
    gpu, ora, _ = harness.make_pair(1, 1, 3, 1, 720, window=60)
    _fill(gpu, ora, [L], L, rng, "bf16")
    k, v, q = _drafts(rng, gpu.cfg, 1, 9, "bf16")
    _check(gpu, ora, k, v, q, np.array([L]), ref.random_tree(rng, 9)[None], "bf16")


@pytest.mark.parametrize("k_format", ["q4g32", "q8g32", "tq3_qjl"])
@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("g,N", [(1, 64), (3, 22), (3, 32), (2, 50), (4, 33), (3, 64)])
def test_row_counts_around_the_blocks(k_format, in_dtype, g, N):
    """64, 66, 96, 100, 132 and 192 rows a KV head: one block or two, full or not."""
    rng = np.random.default_rng(100 * g + N)
    gpu, ora, _ = harness.make_pair(1, 1, g, 2, 460, window=40, k_format=k_format, in_dtype=in_dtype)
    lens = np.array([450, 333])
    _fill(gpu, ora, lens, 450, rng, in_dtype)
    k, v, q = _drafts(rng, gpu.cfg, 2, N, in_dtype)
    _check(gpu, ora, k, v, q, lens, np.stack([ref.random_tree(rng, N) for _ in range(2)]), in_dtype)


def test_chain_equals_single_token_steps():
    """A chain of drafts over a window that covers it: exactly what append + decode of each token computes."""
    rng = np.random.default_rng(5)
    gpu, ora, _ = harness.make_pair(1, 2, 8, 2, 400, window=128, in_dtype="f32")
    lens = np.array([260, 90])
    _fill(gpu, ora, lens, 260, rng, "f32")
    N = 12
    k, v, q = _drafts(rng, gpu.cfg, 2, N, "f32")
    parents = np.stack([ref.random_tree(rng, N, chain=True)] * 2)
    out = _check(gpu, ora, k, v, q, lens, parents, "f32").double().cpu().numpy()
    for i in range(N):
        ora.append(0, harness.to_np(k[:, :, i:i + 1]), harness.to_np(v[:, :, i:i + 1]), lens + i)
        step = ora.decode(0, harness.to_np(q[:, :, i]), lens + i + 1)
        harness.assert_attention_close(out[:, :, i], step, TOL["f32"])


def test_absent_nodes_and_their_children():
    rng = np.random.default_rng(9)
    gpu, ora, _ = harness.make_pair(1, 2, 4, 3, 200)
    lens = np.array([150, 20, 0])
    _fill(gpu, ora, lens, 150, rng, "bf16")
    k, v, q = _drafts(rng, gpu.cfg, 3, 6, "bf16")
    parents = np.array([[-1, 0, -2, 2, 3, 1], [-2] * 6, [-1, -5, 0, 1, 2, -2]], np.int32)
    _check(gpu, ora, k, v, q, lens, parents, "bf16")
    k[:, :, 2] = float("nan")      # a node that is not there may hold anything
    k[1], v[1], q[1] = float("inf"), float("nan"), float("nan")
    out = gpu.tree_decode(0, k.cuda(), v.cuda(), q.cuda(), torch.as_tensor(lens, dtype=torch.int32).cuda(),
                          torch.as_tensor(parents).cuda())
    assert torch.isfinite(out[:2]).all()


def test_sinkhorn_paged_all_layers():
    """Balanced records, a shuffled block table, every layer in one call."""
    rng = np.random.default_rng(11)
    bt = rng.permutation(3 * 5 + 4)[:15].reshape(3, 5).astype(np.int32)
    gpu, ora, _ = harness.make_pair(2, 2, 8, 3, 300, sinkhorn=True, n_pages=19, block_table=bt)
    for layer in range(2):
        c = rng.standard_normal((2, 2, 256, 128)).astype(np.float32) * np.exp(rng.uniform(-1, 1, (2, 2, 1, 128))).astype(np.float32)
        ck = torch.as_tensor(c).bfloat16()
        gpu.calibrate(layer, ck[0].cuda(), ck[1].cuda())
        ora.calibrate(layer, harness.to_np(ck[0]), harness.to_np(ck[1]))
    lens = np.array([290, 64, 200])
    _fill(gpu, ora, lens, 290, rng, "bf16", layers=2)
    k, v, q = _drafts(rng, gpu.cfg, 3, 16, "bf16", layers=2)
    parents = np.stack([ref.random_tree(rng, 16) for _ in range(3)])
    out = gpu.tree_decode(-1, k.cuda(), v.cuda(), q.cuda(), torch.as_tensor(lens, dtype=torch.int32).cuda(),
                          torch.as_tensor(parents).cuda())
    for layer in range(2):
        want = ref.tree_attention(ora, layer, *(harness.to_np(t[layer]) for t in (k, v, q)), lens, parents)
        harness.assert_attention_close(out[layer].double().cpu().numpy(), want, TOL["bf16"])
        one = gpu.tree_decode(layer, k[layer].cuda(), v[layer].cuda(), q[layer].cuda(),
                              torch.as_tensor(lens, dtype=torch.int32).cuda(), torch.as_tensor(parents).cuda())
        harness.assert_attention_close(one.double().cpu().numpy(), want, TOL["bf16"])


def test_large_logits_and_a_dominant_draft():
    rng = np.random.default_rng(13)
    gpu, ora, _ = harness.make_pair(1, 1, 4, 1, 520, in_dtype="f32")
    _fill(gpu, ora, [500], 500, rng, "f32", scale=30.0)
    k, v, q = _drafts(rng, gpu.cfg, 1, 7, "f32")
    k[:, :, 3] = 40 * q[:, :1, 3]
    _check(gpu, ora, k, v, q * 4, np.array([500]), ref.random_tree(rng, 7, chain=True)[None], "f32")


def test_flags():
    """A parent that is not an earlier node and a length out of range are flagged; the other sequence is unharmed."""
    rng = np.random.default_rng(15)
    gpu, ora, _ = harness.make_pair(1, 1, 2, 3, 100)
    lens = np.array([90, 90, 90])
    _fill(gpu, ora, lens, 90, rng, "bf16")
    k, v, q = _drafts(rng, gpu.cfg, 3, 3, "bf16")
    good = np.array([[-1, 0, 1]] * 3, np.int32)
    want = ref.tree_attention(ora, 0, harness.to_np(k), harness.to_np(v), harness.to_np(q), np.array([90, 0, 90]), good)
    bad = good.copy()
    bad[2, 1] = 2
    out = gpu.tree_decode(0, k.cuda(), v.cuda(), q.cuda(), torch.tensor([90, 101, 90], dtype=torch.int32).cuda(),
                          torch.as_tensor(bad).cuda()).double().cpu().numpy()
    assert gpu.status() == lib.DEV_BAD_NODE | lib.DEV_SEQLEN_RANGE
    harness.assert_attention_close(out[:2], want[:2], TOL["bf16"])
    harness.assert_attention_close(out[2, :, 0], want[2, :, 0], TOL["bf16"])
    assert (out[2, :, 1:] == 0).all()


def test_bad_page_is_skipped():
    rng = np.random.default_rng(16)
    bt = np.array([[0, 1, 2]], np.int32)
    gpu, ora, _ = harness.make_pair(1, 1, 2, 1, 192, window=0, n_pages=3, block_table=bt)
    _fill(gpu, ora, [192], 192, rng, "bf16")
    k, v, q = _drafts(rng, gpu.cfg, 1, 2, "bf16")
    gpu.block_table[0, 2] = 99
    par = torch.tensor([[-1, 0]], dtype=torch.int32).cuda()
    got = gpu.tree_decode(0, k.cuda(), v.cuda(), q.cuda(), torch.tensor([192], dtype=torch.int32).cuda(), par)
    assert gpu.status() == lib.DEV_BAD_PAGE
    want = ref.tree_attention(ora, 0, harness.to_np(k), harness.to_np(v), harness.to_np(q), np.array([128]), np.array([[-1, 0]]))
    harness.assert_attention_close(got.double().cpu().numpy(), want, TOL["bf16"])


def test_deterministic_captured_and_on_another_stream():
    rng = np.random.default_rng(17)
    gpu, ora, _ = harness.make_pair(1, 8, 24, 2, 3000)
    lens = np.array([2900, 700])
    _fill(gpu, ora, lens, 2900, rng, "bf16")
    k, v, q = (t.cuda() for t in _drafts(rng, gpu.cfg, 2, 16, "bf16"))
    par = torch.as_tensor(np.stack([ref.random_tree(rng, 16) for _ in range(2)])).cuda()
    ln = torch.as_tensor(lens, dtype=torch.int32).cuda()
    first = gpu.tree_decode(0, k, v, q, ln, par).clone()
    for _ in range(3):
        assert torch.equal(gpu.tree_decode(0, k, v, q, ln, par), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = gpu.tree_decode(0, k, v, q, ln, par)
    side.synchronize()
    assert torch.equal(out, first)
    # two captured calls that share the cache's scratch, replayed in order on changed inputs
    out1, out2 = torch.zeros_like(q), torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu.tree_decode(0, k, v, q, ln, par, out=out1)
        gpu.tree_decode(0, v, k, q, ln, par, out=out2)
    q.neg_()
    ln.copy_(torch.tensor([2000, 1], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out1, gpu.tree_decode(0, k, v, q, ln, par))
    assert torch.equal(out2, gpu.tree_decode(0, v, k, q, ln, par))


# ---------------------------------------------------------------------------- commit
@pytest.mark.parametrize("k_format", ["q4g32", "q8g32", "tq3_qjl"])
@pytest.mark.parametrize("in_dtype,window", [("bf16", 128), ("bf16", 4), ("f32", 0)])
def test_commit_writes_what_appends_write(k_format, in_dtype, window):
    rng = np.random.default_rng(21)
    B, N, P = 5, 12, 6
    a, ora, _ = harness.make_pair(2, 2, 4, B, 200, window=window, k_format=k_format, in_dtype=in_dtype)
    b, _, _ = harness.make_pair(2, 2, 4, B, 200, window=window, k_format=k_format, in_dtype=in_dtype)
    a.buffer.zero_()
    b.buffer.zero_()
    for c in (a, b):
        c.handle = lib.kv_cache_init(c.cfg, c.buffer, None, harness.synth.qjl_projection(4242) if k_format == "tq3_qjl" else None)
    k, v, _ = _drafts(rng, a.cfg, B, N, in_dtype, layers=2)
    path = np.stack([np.sort(rng.permutation(N)[:P]) for _ in range(B)]).astype(np.int32)
    path[4, :] = 3                                  # one node again and again is a path too
    n = np.array([6, 0, 1, 3, 5], np.int32)
    pos = np.array([0, 10, 63, 126, -1], np.int32)
    pos[4] = 190
    a.commit(-1, k.cuda(), v.cuda(), torch.as_tensor(path).cuda(), torch.as_tensor(n).cuda(), torch.as_tensor(pos).cuda())
    for s in range(B):
        for t in range(n[s]):
            one = torch.full((B,), -1, dtype=torch.int32)
            one[s] = pos[s] + t
            i = int(path[s, t])
            b.append(-1, k[:, :, :, i:i + 1].contiguous().cuda(), v[:, :, :, i:i + 1].contiguous().cuda(), one.cuda())
    torch.cuda.synchronize()
    assert a.status() == 0
    assert torch.equal(a.buffer, b.buffer)


def test_commit_flags_and_leaves_alone():
    rng = np.random.default_rng(22)
    gpu, _, _ = harness.make_pair(1, 1, 1, 5, 100)
    k, v, _ = _drafts(rng, gpu.cfg, 5, 4, "bf16")
    before = gpu.buffer.clone()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    args = (0, k.cuda(), v.cuda(), i32([[0, 1]] * 5))
    gpu.commit(*args, i32([0, -3, 2, 2, 0]), i32([1, 1, -1, -9, 99]))
    assert gpu.status() == 0 and torch.equal(gpu.buffer, before)
    gpu.commit(*args, i32([3, 0, 0, 0, 0]), i32([0] * 5))
    assert gpu.status() == lib.DEV_BAD_NODE and torch.equal(gpu.buffer, before)
    gpu.commit(*args, i32([2, 0, 0, 0, 0]), i32([99] + [0] * 4))
    assert gpu.status() == lib.DEV_POS_RANGE and torch.equal(gpu.buffer, before)
    gpu.commit(0, k.cuda(), v.cuda(), i32([[4, -1]] * 5), i32([2, 0, 0, 0, 0]), i32([0] * 5))
    assert gpu.status() == lib.DEV_BAD_NODE and torch.equal(gpu.buffer, before)

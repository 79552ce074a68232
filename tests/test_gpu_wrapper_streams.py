"""QuantKVCache's own workspaces: calls on two streams at once, graphs replayed at once, buffers shared by sizes."""

import numpy as np
import pytest
import torch

from . import harness
from . import ops_reference as ref
from .test_gpu_tree import _drafts, _fill

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


@pytest.fixture(scope="module")
def made():
    rng = np.random.default_rng(71)
    gpu, ora, _ = harness.make_pair(1, 4, 8, 3, 2000)
    lens = np.array([2000, 700, 1300])
    _fill(gpu, ora, lens, 2000, rng, "bf16")
    drafts = [tuple(t.cuda() for t in _drafts(rng, gpu.cfg, 3, 24, "bf16")) for _ in range(2)]
    parents = _i32([ref.random_tree(rng, 24) for _ in range(3)])
    return gpu, drafts, _i32(lens), parents


def _calls(gpu, d, ln, parents, w, stream=None):
    k, v, q = d
    return (gpu.tree_decode(0, k, v, q, ln, parents, stream=stream),
            gpu.attention_weights(0, q, ln, w, 0.0, stream=stream),
            gpu.decode(0, q[:, :, 0].contiguous(), ln, stream=stream))


def _weights():
    return torch.full((3, 4, 2000), -1.0, device="cuda")


@pytest.mark.parametrize("named", [False, True])
def test_two_streams_at_once(made, named):
    """Each stream's calls give what they give alone, whether the stream is the current one or named."""
    gpu, drafts, ln, parents = made
    want = [[t.clone() for t in _calls(gpu, d, ln, parents, _weights())] for d in drafts]
    streams = [torch.cuda.Stream() for _ in range(2)]
    spare = [[_weights() for _ in range(8)] for _ in range(2)]
    heads = [d[2][:, :, 0].contiguous() for d in drafts]
    outs = [[(torch.empty_like(d[2]), torch.empty(3, 8, 128, device="cuda")) for _ in range(8)] for d in drafts]
    torch.cuda.synchronize()
    for i in range(8):
        for n, s in enumerate(streams):
            k, v, q = drafts[n]
            with torch.cuda.stream(None if named else s):
                gpu.tree_decode(0, k, v, q, ln, parents, out=outs[n][i][0], stream=s if named else None)
                gpu.attention_weights(0, q, ln, spare[n][i], 0.0, stream=s if named else None)
                gpu.decode(0, heads[n], ln, out=outs[n][i][1], stream=s if named else None)
    torch.cuda.synchronize()
    assert gpu.status() == 0
    for n in range(2):
        for i in range(8):
            for a, b in zip((outs[n][i][0], spare[n][i], outs[n][i][1]), want[n]):
                assert torch.equal(a, b)


def test_graphs_replayed_at_once_and_after_the_buffers_grew(made):
    gpu, drafts, ln, parents = made
    want = [[t.clone() for t in _calls(gpu, d, ln, parents, _weights())] for d in drafts]
    graphs, outs = [], []
    for d in drafts:
        w = _weights()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_calls(gpu, d, ln, parents, w))
        graphs.append(g)
    big = [torch.cat([t, t], 2) for t in drafts[0]]                  # a larger call, and whoever takes memory now
    chain = _i32([ref.random_tree(np.random.default_rng(1), 48, chain=True)] * 3)
    gpu.tree_decode(0, *big, ln, chain)
    gpu.attention_weights(0, big[2], ln, _weights(), 0.0)
    junk = [torch.full((1 << 22,), 7.0, device="cuda") for _ in range(8)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        gpu.tree_decode(0, *big, ln, chain)
    torch.cuda.synchronize()
    for got, expected in zip(outs, want):
        for a, b in zip(got, expected):
            assert torch.equal(a, b)
    assert all((j == 7).all() for j in junk) and gpu.status() == 0


def test_one_buffer_for_all_sizes(made):
    """Batches and trees of every size leave one buffer per operation and stream, of the largest's size."""
    gpu, drafts, ln, parents = made
    k, v, q = drafts[0]
    gpu._work.clear()
    for b in (1, 2, 3, 1):
        for n in (1, 24, 7):
            args = [t[:b, :, :n].contiguous() for t in (k, v, q)]
            got = gpu.tree_decode(0, *args, ln[:b].contiguous(), parents[:b, :n].contiguous())
            w = gpu.attention_weights(0, args[2], ln[:b].contiguous(), _weights()[:b], 0.0)
            if (b, n) == (3, 24):
                torch.cuda.synchronize()
    assert torch.isfinite(got.float()).all() and torch.isfinite(w).all()
    assert sorted(op for op, _ in gpu._work) == ["tree", "weights"]
    from kv_cache_quantization_append_gb300 import lib

    assert gpu._work[next(k for k in gpu._work if k[0] == "tree")].numel() == max(
        lib.kv_tree_scratch_bytes(gpu.handle, 0, b, n) for b in (1, 2, 3) for n in (1, 24, 7))


def test_the_library_refuses_a_call_while_another_device_is_current(made):
    """The C entry points of trees, commits, weights and eviction look at the current device themselves."""
    import ctypes

    from kv_cache_quantization_append_gb300 import lib

    gpu = made[0]
    other = lib.kvq_cache.from_buffer_copy(gpu.handle)
    other.device = gpu.handle.device + 1
    buf = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    p, r, c = buf.data_ptr(), ctypes.byref(other), lib.load()
    before = gpu.buffer.clone()
    assert c.kv_tree_commit(r, 0, p, p, p, p, p, 1, 4, 4, None) == 1
    assert c.kv_evict(r, 0, p, p, p, p + 64, 1, 200, 128, None) == 1
    assert c.kv_quant_append(r, 0, p, p, p, 1, 1, None) == 1
    for call in (lambda n: c.kv_tree_attention(r, 0, p, p, p, p, p, p, 1, 4, p, n, None),
                 lambda n: c.kv_attention_weights(r, 0, p, p, 1.0, p, 1, 1, p, n, None)):
        assert call(1 << 60) == 1
    torch.cuda.synchronize()
    assert torch.equal(before, gpu.buffer) and not buf.any()


def test_calibration_keeps_no_workspace():
    """Calibration happens once: its copies (here 16 MB) go back to the allocator."""
    gpu, _, _ = harness.make_pair(1, 2, 2, 1, 64, window=0, sinkhorn=True)
    x = torch.randn(2, 4096, 128, device="cuda").bfloat16()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    gpu.calibrate(0, x, x, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == before

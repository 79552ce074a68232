"""Trees, attention weights and eviction where sizes and uses are unusual: wide windows, many or empty sequences, full
sequences, caches past 4 GB, two streams at once, captured calls."""

import numpy as np
import pytest
import torch

from kv_cache_quantization_append_gb300 import QuantKVCache, lib

from . import harness
from . import ops_reference as ref
from .test_gpu_evict import _check_weights, _i32
from .test_gpu_tree import _check, _drafts, _fill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k_format,window", [("q4g32", 300), ("q8g32", 1024), ("tq3_qjl", 132)])
def test_windows_of_several_tiles(k_format, window, in_dtype):
    """Raw positions over several tiles, sequences shorter and longer than the window, and eviction's turn of the ring."""
    rng = np.random.default_rng(window)
    S = window + 260
    gpu, ora, _ = harness.make_pair(1, 1, 2, 3, S, window=window, k_format=k_format, in_dtype=in_dtype)
    lens = np.array([S, window - 1, window + 130])
    _fill(gpu, ora, lens, S, rng, in_dtype)
    k, v, q = _drafts(rng, gpu.cfg, 3, 20, in_dtype)
    _check(gpu, ora, k, v, q, lens, np.stack([ref.random_tree(rng, 20) for _ in range(3)]), in_dtype)
    w = _check_weights(gpu, ora, q, lens, 0.5, rng)
    host = w.cpu().numpy()[None]
    kept, _ = gpu.evict(0, w, _i32(lens), window + 60, window)
    assert np.array_equal(kept.cpu().numpy(), ref.evict(ora, host, lens, window + 60, window)[0])
    assert np.array_equal(w.cpu().numpy(), host[0])
    assert gpu.status() == 0
    lens = np.minimum(lens, window + 60)
    for b in range(3):
        harness.compare_codes(gpu, ora, 0, b, 0, int(lens[b]))
        harness.compare_ring(gpu, ora, 0, b, 0, int(lens[b]))
    _check(gpu, ora, k, v, q, lens, np.stack([ref.random_tree(rng, 20) for _ in range(3)]), in_dtype)


def test_many_sequences_and_none_with_tokens():
    rng = np.random.default_rng(3)
    B = 71
    gpu, ora, _ = harness.make_pair(1, 1, 2, B, 70, window=8)
    lens = rng.integers(0, 71, B)
    lens[[0, 5, 70]] = 0, 70, 0
    _fill(gpu, ora, lens, 70, rng, "bf16")
    k, v, q = _drafts(rng, gpu.cfg, B, 3, "bf16")
    parents = np.stack([ref.random_tree(rng, 3) for _ in range(B)])
    _check(gpu, ora, k, v, q, lens, parents, "bf16")
    _check_weights(gpu, ora, q, lens, 1.0, rng)
    none = np.zeros(B, np.int64)
    _check(gpu, ora, k, v, q, none, parents, "bf16")
    _check_weights(gpu, ora, q, none, 1.0, rng)
    _, _, q = _drafts(rng, gpu.cfg, B, 9, "bf16")           # rows whose logits are not stored
    _check_weights(gpu, ora, q, none, 0.0, rng)


@pytest.mark.parametrize("k_format", ["q4g32", "tq3_qjl"])
def test_full_sequences(k_format):
    """seq_lens == max_seq_len: drafts attend to all of it (their own positions need no room)."""
    rng = np.random.default_rng(13)
    gpu, ora, _ = harness.make_pair(1, 2, 2, 2, 257, window=16, k_format=k_format)
    lens = np.array([257, 256])
    _fill(gpu, ora, lens, 257, rng, "bf16")
    k, v, q = _drafts(rng, gpu.cfg, 2, 64, "bf16")
    _check(gpu, ora, k, v, q, lens, np.stack([ref.random_tree(rng, 64, chain=True) for _ in range(2)]), "bf16")
    _check_weights(gpu, ora, q, lens, 0.0, rng)


@pytest.mark.parametrize("T", [2, 12])
def test_weights_bad_page_takes_none(T):
    """A block-table entry out of range: flagged, its positions take no weight (they keep decay times theirs), the other
    sequence's are what they are without it."""
    rng = np.random.default_rng(23)
    bt = np.arange(8, dtype=np.int32).reshape(2, 4)
    gpu, ora, _ = harness.make_pair(1, 1, 1, 2, 256, window=0, n_pages=8, block_table=bt)
    _fill(gpu, ora, [256, 200], 256, rng, "bf16")
    _, _, q = _drafts(rng, gpu.cfg, 2, T, "bf16")
    ln = _i32([256, 200])
    good = gpu.attention_weights(0, q.cuda(), ln, torch.zeros(2, 1, 256, device="cuda"), 0.0)
    gpu.block_table[0, 1] = 8
    got = gpu.attention_weights(0, q.cuda(), ln, torch.ones(2, 1, 256, device="cuda"), 0.5)
    assert gpu.status() == lib.DEV_BAD_PAGE
    # the second sequence: decay times one, plus what it takes, in one rounded fma
    assert torch.equal(got[1, 0, :200], (good[1, 0, :200].double() + 0.5).float())
    assert torch.equal(got[0, 0, 64:128], torch.full((64,), 0.5, device="cuda"))
    rest = torch.cat([got[0, 0, :64], got[0, 0, 128:]]) - 0.5
    assert abs(rest.sum().item() - T) < 1e-4


def test_caches_past_four_gigabytes():
    """The last layer of a 6 GB cache gives what a small cache of the same tokens gives, to the bit."""
    rng = np.random.default_rng(61)
    big = QuantKVCache(lib.make_config(73, 8, 8, 2, 32768), "cuda")
    small = QuantKVCache(lib.make_config(1, 8, 8, 2, 320), "cuda")
    assert big.buffer.numel() > 5 << 30                    # (the last layer begins past 2^32)
    k = torch.as_tensor(rng.standard_normal((2, 8, 310, 128)).astype(np.float32)).bfloat16().cuda()
    v = torch.as_tensor(rng.standard_normal((2, 8, 310, 128)).astype(np.float32)).bfloat16().cuda()
    q = torch.as_tensor(rng.standard_normal((2, 8, 7, 128)).astype(np.float32)).bfloat16().cuda()
    path = _i32([[0, 2, 3], [1, 4, 5]])
    results = []
    for cache, layer in ((big, 72), (small, 0)):
        cache.append(layer, k[:, :, :300].contiguous(), v[:, :, :300].contiguous(), _i32([0, 0]))
        ln = _i32([300, 300])
        dk, dv = k[:, :, 303:].contiguous(), v[:, :, 303:].contiguous()
        out = [cache.tree_decode(layer, dk, dv, q, ln, _i32([[-1, 0, 1, 2, 0, 0, 1]] * 2))]
        cache.commit(layer, dk, dv, path, _i32([3, 2]), ln)
        ln = _i32([303, 302])
        for T in (1, 7):
            w = torch.zeros(2, 8, cache.cfg.max_seq_len, device="cuda")
            cache.attention_weights(layer, q[:, :, :T].contiguous(), ln, w, 0.0)
            out.append(w[..., :303].clone())
        out += list(cache.evict(layer, w, ln, 200, 130))
        out.append(cache.decode(layer, q[:, :, 0].contiguous(), _i32([200, 200])))
        assert cache.status() == 0
        results.append(out)
    for a, b in zip(*results):
        assert torch.equal(a, b)


@pytest.mark.parametrize("L,budget,recent,offset", [(100001, 30001, 200, 0), (54000, 53000, 130, 3), (4100, 4099, 128, 0)])
def test_evict_more_weights_than_shared_memory_holds(L, budget, recent, offset):
    """Many equal weights over long sequences; a weights tensor whose units lie on odd addresses."""
    rng = np.random.default_rng(L)
    gpu = QuantKVCache(lib.make_config(1, 2, 2, 1, L + offset), "cuda")
    k = torch.as_tensor(rng.standard_normal((1, 2, L, 128)).astype(np.float32)).bfloat16().cuda()
    gpu.append(0, k, k, _i32([0]))
    w = np.floor(rng.random((1, 2, L + offset)) ** 4 * 50).astype(np.float32)
    wd = torch.as_tensor(w).cuda()
    before = [harness.layout.read_unit(gpu.buffer, gpu.cfg, 0, 0, h, L) for h in range(2)]
    kept, new = gpu.evict(0, wd, _i32([L]), budget, recent)
    assert gpu.status() == 0 and new.item() == budget
    for h in range(2):
        src = ref.kept_positions(w[0, h], L, budget, recent)
        assert np.array_equal(kept[0, h].cpu().numpy(), src)
        want = w[0, h].copy()
        want[:budget] = w[0, h, src]
        assert np.array_equal(wd[0, h].cpu().numpy(), want)
        after = harness.layout.read_unit(gpu.buffer, gpu.cfg, 0, 0, h, budget)
        for name in after:
            assert np.array_equal(after[name], before[h][name][src]), name


def test_two_streams_at_once():
    """Calls with scratch of their own on two streams of one cache, many in flight: each gives what it gives alone."""
    rng = np.random.default_rng(71)
    gpu, ora, _ = harness.make_pair(1, 4, 8, 3, 2000)
    lens = np.array([2000, 700, 1300])
    _fill(gpu, ora, lens, 2000, rng, "bf16")
    k, v, q = (t.cuda() for t in _drafts(rng, gpu.cfg, 3, 24, "bf16"))
    ln, parents = _i32(lens), _i32([ref.random_tree(rng, 24) for _ in range(3)])
    tree = gpu.tree_decode(0, k, v, q, ln, parents)
    weights = gpu.attention_weights(0, q, ln, torch.zeros(3, 4, 2000, device="cuda"), 0.0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs, ws, scratch = [], [], []
    for s in streams:
        scratch.append([torch.empty(f(gpu.handle, 0, 3, 24), dtype=torch.uint8, device="cuda")
                        for f in (lib.kv_tree_scratch_bytes, lib.kv_weights_scratch_bytes)])
        outs.append([torch.empty_like(q) for _ in range(6)])
        ws.append([torch.empty(3, 4, 2000, device="cuda").fill_(-1) for _ in range(6)])
    torch.cuda.synchronize()
    for i in range(6):
        for n, s in enumerate(streams):
            lib.kv_tree_attention(gpu.handle, 0, k, v, q, outs[n][i], ln, parents, scratch[n][0], stream=s)
            lib.kv_attention_weights(gpu.handle, 0, q, ws[n][i], 0.0, ln, scratch[n][1], stream=s)
    torch.cuda.synchronize()
    assert gpu.status() == 0
    for n in range(2):
        for i in range(6):
            assert torch.equal(outs[n][i], tree)
            for b in range(3):
                assert torch.equal(ws[n][i][b, :, :lens[b]], weights[b, :, :lens[b]])


@pytest.mark.parametrize("k_format", ["q4g32", "q8g32", "tq3_qjl"])
@pytest.mark.parametrize("T", [1, 3])
def test_weights_many_calls_none_gives_up(k_format, T):
    """A wait between the warps of a CTA that missed its phase would run out of time, be flagged and leave weights out: over
    many calls, with the caches of the GPU turned over in between, none does and all agree."""
    rng = np.random.default_rng(91)
    gpu, ora, _ = harness.make_pair(1, 8, 32, 4, 9000, k_format=k_format)
    k = torch.as_tensor(rng.standard_normal((4, 8, 9000, 128)).astype(np.float32)).bfloat16().cuda()
    gpu.append(0, k, k, _i32([0] * 4))
    _, _, q = _drafts(rng, gpu.cfg, 4, T, "bf16")
    q, ln = q.cuda(), _i32([9000, 8000, 5000, 8700])
    first = gpu.attention_weights(0, q, ln, torch.zeros(4, 8, 9000, device="cuda"), 0.0)
    other = torch.empty(160 << 20, dtype=torch.uint8, device="cuda")
    bad = torch.zeros((), dtype=torch.bool, device="cuda")
    w = torch.zeros_like(first)
    for i in range(400):
        if i % 2:
            other.zero_()
        gpu.attention_weights(0, q, ln, w, 0.0)
        bad |= (w != first).any()
    assert not bad.item() and gpu.status() == 0


def test_captured_serving_step():
    """Tree, commit, weights and eviction in one graph, replayed on other lengths: what the calls give one by one."""
    rng = np.random.default_rng(81)
    a, _, _ = harness.make_pair(2, 2, 4, 2, 400, window=64)
    b, _, _ = harness.make_pair(2, 2, 4, 2, 400, window=64)
    k = torch.as_tensor(rng.standard_normal((2, 2, 2, 400, 128)).astype(np.float32)).bfloat16().cuda()
    for c in (a, b):
        c.buffer.zero_()
        c.handle = lib.kv_cache_init(c.cfg, c.buffer)
        c.append(-1, k, k, _i32([0, 0]))
    dk, dv, q = (t.cuda() for t in _drafts(rng, a.cfg, 2, 6, "bf16", layers=2))
    state = {}
    for name, c in (("a", a), ("b", b)):
        state[name] = dict(ln=_i32([300, 100]), parents=_i32([[-1, 0, 1, 2, 0, 0], [-1, 0, 0, 0, 1, 1]]),
                           path=_i32([[0, 1, 2], [0, 2, 2]]), n=_i32([3, 1]), out=torch.empty_like(q),
                           w=torch.zeros(2, 2, 2, 400, device="cuda"), after=_i32([303, 101]),
                           kept=_i32(np.zeros((2, 2, 2, 200))), new=_i32([0, 0]))

    def step(c, s):
        c.tree_decode(-1, dk, dv, q, s["ln"], s["parents"], out=s["out"])
        c.commit(-1, dk, dv, s["path"], s["n"], s["ln"])
        c.attention_weights(-1, q, s["after"], s["w"], 0.0)
        c.evict(-1, s["w"], s["after"], 200, 64, kept=s["kept"], new_lens=s["new"])

    warm, _, _ = harness.make_pair(2, 2, 4, 2, 400, window=64)      # shared-memory limits are set outside a capture
    warm.append(-1, k, k, _i32([0, 0]))
    step(warm, dict(state["a"], w=state["a"]["w"].clone(), out=torch.empty_like(q)))
    a.tree_decode(-1, dk, dv, q, state["a"]["ln"], state["a"]["parents"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a, state["a"])
    for lens, n in (([300, 100], [3, 1]), ([203, 350], [2, 3])):
        for s in state.values():
            s["ln"].copy_(_i32(lens))
            s["n"].copy_(_i32(n))
            s["after"].copy_(_i32(np.add(lens, n)))
            s["w"].zero_()
        graph.replay()
        step(b, state["b"])
        torch.cuda.synchronize()
        for key in ("out", "w", "kept", "new"):
            assert torch.equal(state["a"][key], state["b"][key]), key
        assert torch.equal(a.buffer, b.buffer)
    assert a.status() == 0 and b.status() == 0


def test_weights_of_more_layers_than_the_scratch_holds():
    """Stored logits of 160 MiB a layer, of which the 256 MiB hold one: a call of every layer gives, to the bit, what the layers' own
    calls give (layers taken together are cut into other ranges, whose sums join in another order)."""
    T = 2
    rng = np.random.default_rng(101)
    L, B, H, g, S = 3, 5, 8, 4, 131072
    gpu = QuantKVCache(lib.make_config(L, H, H * g, B, S), "cuda")
    lens = [5000, 0, 1025, 130, 2048]
    k = torch.as_tensor(rng.standard_normal((L, B, H, 5000, 128)).astype(np.float32)).bfloat16().cuda()
    gpu.append(-1, k, k, _i32([0] * B))
    q = torch.as_tensor(rng.standard_normal((L, B, H * g, T, 128)).astype(np.float32)).bfloat16().cuda()
    old = torch.rand(L, B, H, S, device="cuda")
    w = gpu.attention_weights(-1, q, _i32(lens), old.clone(), 0.5)
    for layer in range(L):
        one = gpu.attention_weights(layer, q[layer].contiguous(), _i32(lens), old[layer].clone(), 0.5)
        assert torch.equal(w[layer], one)
        for b, n in enumerate(lens):
            assert torch.equal(one[b, :, n:], old[layer, b, :, n:])
            if n:
                got = (one[b, :, :n].double() - 0.5 * old[layer, b, :, :n].double()).sum(-1)
                assert (got - g * T).abs().max() < 1e-3
    assert gpu.status() == 0

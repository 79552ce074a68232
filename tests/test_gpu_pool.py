"""Pages of a cache: reserve, fork, release and compact against the definition, and as a serving loop uses them."""

import ctypes

import numpy as np
import pytest
import torch

from kv_cache_quantization_append_gb300 import QuantKVCache, lib, synth

from . import block_reference as br
from . import harness
from .pool_reference import Pool

pytestmark = pytest.mark.gpu
PAGE_BYTES = {"q4g32": 10240, "tq3_qjl": 9472, "q8g32": 13824, "q8b32": 16416}


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


class Both:
    """A cache with a pool and its definition; every page's contents are random bytes of their own."""

    def __init__(self, n_seqs, max_seq_len, n_pages, fmt="q4g32", layers=2, heads=2, window=64, seed=0):
        mpp = -(-max_seq_len // 64)
        self.cfg = lib.make_config(layers, heads, heads, n_seqs, max_seq_len, window=window, n_pages=n_pages, k_format=lib.K_FORMATS[fmt])
        self.bt = torch.full((n_seqs, mpp), 7, dtype=torch.int32, device="cuda")
        self.gpu = QuantKVCache(self.cfg, "cuda", self.bt, synth.qjl_projection(1))
        self.gpu.pool_init()
        self.ref = Pool(n_seqs, mpp, n_pages, max_seq_len)
        total = lib.kv_cache_bytes(self.cfg)
        size = layers * n_pages * heads * PAGE_BYTES[fmt]
        off = total - -(-size // 256) * 256
        self.pages = self.gpu.buffer[off:off + size].view(layers, n_pages, -1)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.pages.copy_(torch.randint(0, 256, self.pages.shape, generator=g, device="cuda", dtype=torch.uint8))
        self.first = self.pages.clone()
        ring = layers * n_seqs * heads * window * 512
        self.rings = [self.gpu.buffer[o:o + ring].view(torch.float32).view(layers, n_seqs, heads, window, 128)
                      for o in (off - 2 * (-(-ring // 256) * 256), off - -(-ring // 256) * 256)]
        for r in self.rings:
            r.copy_(torch.randn(r.shape, generator=g, device="cuda"))

    def check(self):
        assert np.array_equal(self.bt.cpu().numpy(), self.ref.table)
        assert np.array_equal(self.gpu.page_refs.cpu().numpy(), self.ref.refs)
        assert torch.equal(self.pages, self.first[:, torch.as_tensor(self.ref.holds).cuda()])
        assert self.gpu.status() == self.ref.flags
        self.ref.flags = 0
        # the workspace behind the counts is as a call expects it
        n = -(-4 * self.ref.n_pages // 256) * 256
        w = self.gpu.pool[n + 256:].view(torch.int32)
        assert (w[:self.ref.n_pages] == 0).all() and (w[n // 4:n // 4 + self.ref.n_pages] == -1).all()

    def reserve(self, pos, n):
        counts = [n] * len(pos) if isinstance(n, int) else n
        got = self.gpu.reserve(_i32(pos), n if isinstance(n, int) else _i32(n))
        want = self.ref.reserve(pos, counts)
        assert got.tolist() == want
        self.check()
        return want

    def fork(self, parents, lens):
        before = [r.clone() for r in self.rings]
        got = self.gpu.fork(_i32(parents), _i32(lens))
        want = self.ref.fork(parents, lens)
        assert got.tolist() == want
        for r, old in zip(self.rings, before):
            for b in range(r.shape[1]):
                q = parents[b] if b < len(parents) and 0 <= parents[b] < len(parents) else b
                n = min(lens[q], r.shape[3]) if q != b else 0
                assert torch.equal(r[:, b, :, :n], old[:, q, :, :n]) and torch.equal(r[:, b, :, n:], old[:, b, :, n:])
        self.check()
        return want

    def release(self, keep):
        self.gpu.release(_i32(keep))
        self.ref.release(keep)
        self.check()

    def compact(self):
        assert self.gpu.compact().item() == self.ref.compact()
        self.check()


def test_init():
    x = Both(3, 300, 9)
    x.check()
    assert x.bt.shape == (3, 5) and (x.bt == -1).all()


@pytest.mark.parametrize("fmt", list(PAGE_BYTES))
def test_a_life(fmt):
    x = Both(6, 640, 40, fmt)
    x.reserve([0, -1, 0], [130, 10, 64])
    x.reserve([130, -1, 64], 1)                    # one within its page, one at a page's first token
    x.reserve([129, -1, 1], 63)                    # nothing new
    n = x.fork([0, 0, 2, 0, 2, -1], [131, 0, 65, 7, 0, 0])
    assert n == [131, 131, 65, 131, 65, 0]
    x.reserve(n, 1)                                # shared tails become each one's own, the last keeps the page
    x.release([131, 0, 65, 132, 0, 0])
    x.compact()
    x.reserve([132, 0, 66, 132], [500, 0, 1, 3])
    x.release([0] * 6)
    assert (x.gpu.page_refs == 0).all()
    x.compact()


def test_shared_with_sequences_outside_the_call():
    """A page that a sequence outside the call shares is copied for every writer; within the call the last keeps it."""
    x = Both(5, 200, 30)
    x.reserve([0], 100)
    x.fork([0, 0, 0, 0, 0], [100, 0, 0, 0, 0])
    x.reserve([100, 100], 1)
    x.reserve([-1, -1, 100, 100, 100], 1)
    assert sorted(x.gpu.page_refs.tolist())[-1] == 5 and (x.gpu.page_refs == 1).sum() == 5
    x.reserve([0, 0, 0, 0, 0], 100)                # whole sequences of their own
    assert x.gpu.page_refs.max() == 1


def test_forks_that_change_places():
    x = Both(8, 500, 60)
    lens = [10, 64, 65, 200, 400, 1, 0, 128]
    for b, n in enumerate(lens):
        pos = [-1] * 8
        pos[b] = 0
        x.reserve(pos, max(n, 1))
    lens = x.fork([1, 2, 3, 4, 5, 6, 7, 0], lens)
    lens = x.fork([1, 0, 2, 2, 2, -1, 6, 5], lens)
    x.fork([3, 3, 3], lens[:3])                    # a parent that is no sequence of the call
    x.compact()


def test_not_enough_pages():
    x = Both(5, 640, 12)
    x.reserve([0, 0], [300, 64])                   # 6 of 12
    x.reserve([300, 64, 0, 0], [64, 200, 64, 64])  # the second takes what is left, from the third on none
    x.reserve([0] * 5, [64, 64, 64, 0, 64])        # nothing is needed before the third; a count of 0 behind it is refused too
    x.release([0, -1, -1])
    x.reserve([-1, -1, 0, 0, 0], 64)
    x.reserve([600, 10, 0], [41, 1, 1])            # past capacity
    y = Both(4, 128, 5)
    y.reserve([0], 100)
    y.fork([0, 0, 0, 0], [100] * 4)
    y.reserve([100] * 4, 1)                        # three copies, exactly what is free
    y.release([-1, 0, -1, -1])
    y.fork([0, 0, 2, 2], [100] * 4)
    y.reserve([100] * 4, 1)
    z = Both(4, 128, 3)
    z.reserve([0], 100)
    z.fork([0, 0, 0, 0], [100] * 4)
    z.reserve([100] * 4, 1)                        # one copy fits: the shared page is no one else's to write
    z.release([-1, 0])
    z.reserve([100, -1, 100, 100], 1)


@pytest.mark.parametrize("n_pages,n_seqs,max_len", [(33, 4, 700), (1500, 40, 6400), (5000, 1024, 700)])
def test_any_order_of_calls(n_pages, n_seqs, max_len):
    rng = np.random.default_rng(n_pages)
    x = Both(n_seqs, max_len, n_pages, layers=1, heads=1, window=32)
    lens = [0] * n_seqs
    for step in range(25):
        op = rng.integers(0, 8)
        if op < 4:
            n = [int(v) for v in rng.choice([0, 1, 5, 64, 200], n_seqs)]
            pos = [p if rng.random() < 0.7 else -1 for p in lens]
            for b, p in enumerate(x.reserve(pos, n)):
                lens[b] = max(lens[b], p + n[b]) if p >= 0 else lens[b]
        elif op < 6:
            parents = [int(v) if rng.random() < 0.5 else -1 for v in rng.integers(0, n_seqs, n_seqs)]
            lens = x.fork(parents, lens)
        elif op == 6:
            keep = [int(rng.integers(0, n + 1)) if rng.random() < 0.4 else -1 for n in lens]
            x.release(keep)
            lens = [n if k < 0 else min(n, k) for n, k in zip(lens, keep)]
        else:
            x.compact()


@pytest.mark.parametrize("n_seqs,window,layers,heads", [(1, 128, 1, 1), (2, 1024, 1, 2), (7, 100, 3, 2), (200, 32, 2, 1), (1024, 32, 1, 1), (3, 0, 2, 2)])
def test_rings_of_any_shape(n_seqs, window, layers, heads):
    rng = np.random.default_rng(n_seqs)
    x = Both(n_seqs, 2000, 50, layers=layers, heads=heads, window=window)
    lens = [int(v) for v in rng.integers(0, 2000, n_seqs)]
    lens[0] = 1
    x.fork([int(v) for v in rng.integers(-1, n_seqs, n_seqs)], lens)


def test_bad_arguments_on_the_device():
    x = Both(4, 200, 10)
    x.reserve([0, 0], 70)
    assert x.gpu.fork(_i32([0, 5, -3, 0]), _i32([70, 70, 3, 9])).tolist() == [70, 70, 3, 70]
    assert x.ref.fork([0, 5, -3, 0], [70, 70, 3, 9]) == [70, 70, 3, 70]
    x.check()
    assert x.gpu.fork(_i32([0, 0]), _i32([-1, 300])).tolist() == [0, 0]
    assert x.gpu.status() == lib.DEV_SEQLEN_RANGE
    x.ref.fork([0, 0], [0, 0])
    x.check()


def test_reserve_over_its_own_positions_and_captured():
    """granted may be pos; a captured round (fork, reserve, release) replayed gives what calls give; another stream."""
    x, y = Both(4, 640, 40, "q8b32"), Both(4, 640, 40, "q8b32")
    for z in (x, y):
        z.reserve([0], 150)
    pos, parents, lens, keep = _i32([150, 150, 150, -1]), _i32([0, 0, 0, -1]), _i32([150, 0, 0, 0]), _i32([150, 0, 0, 0])
    new, granted = torch.empty_like(lens), torch.empty_like(lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    x.gpu.fork(_i32([-1] * 4), _i32([150, 0, 0, 0]))     # (a call outside capture before the first inside)
    with torch.cuda.graph(graph, stream=side):
        x.gpu.fork(parents, lens, new_lens=new)
        x.gpu.reserve(pos, 3, granted=granted)
        x.gpu.compact()
    for _ in range(3):
        graph.replay()
        y.fork([0, 0, 0, -1], [150, 0, 0, 0])
        y.reserve([150, 150, 150, -1], 3)
        y.compact()
        torch.cuda.synchronize()
        assert torch.equal(x.bt, y.bt) and torch.equal(x.gpu.page_refs, y.gpu.page_refs) and torch.equal(x.pages, y.pages)
        assert granted.tolist() == [150, 150, 150, -1] and new.tolist() == [150, 150, 150, 0]
    assert x.gpu.reserve(pos, 1, granted=pos) is pos and pos.tolist() == [150, 150, 150, -1]
    torch.cuda.synchronize()
    y.gpu.release(keep, stream=side)
    side.synchronize()
    y.ref.release([150, 0, 0, 0])
    y.check()


def test_refusals_with_a_device():
    x = Both(2, 200, 6)
    gpu = x.gpu
    own_table = QuantKVCache(x.cfg, "cuda")
    with pytest.raises(lib.KVQError):
        own_table.pool_init()
    fresh = QuantKVCache(x.cfg, "cuda", torch.zeros(2, 4, dtype=torch.int32, device="cuda"))
    for call in (lambda: fresh.reserve(_i32([0]), 1), lambda: fresh.compact(), lambda: fresh.page_refs):
        with pytest.raises(lib.KVQError, match="pool_init"):
            call()
    with pytest.raises(lib.KVQError):
        gpu.reserve(torch.zeros(1, dtype=torch.int64, device="cuda"), 1)
    with pytest.raises(lib.KVQError):
        gpu.reserve(_i32([0, 0, 0]), 1)                       # more sequences than the cache has
    with pytest.raises(lib.KVQError):
        gpu.reserve(_i32([0]), 0)
    with pytest.raises(lib.KVQError):
        gpu.reserve(_i32([0, 0]), _i32([1]))
    with pytest.raises(lib.KVQError):
        gpu.fork(_i32([0, 0]), _i32([0]))
    ln = _i32([0, 0])
    with pytest.raises(lib.KVQError):
        gpu.fork(_i32([0, 0]), ln, new_lens=ln)
    with pytest.raises(lib.KVQError):
        gpu.release(torch.zeros(2, 1, dtype=torch.int32, device="cuda").t()[0].float())
    with pytest.raises(lib.KVQError):
        lib.kv_pool_compact(gpu.handle, gpu.pool[:64], _i32([0]))
    other = lib.kvq_cache.from_buffer_copy(gpu.handle)
    other.device += 1
    c, r, p = lib.load(), ctypes.byref(other), gpu.pool.data_ptr()
    q = ln.data_ptr()
    for rc in (c.kv_pool_init(r, p, 1 << 40, None), c.kv_pool_reserve(r, p, 1 << 40, q, None, q, 1, 1, None),
               c.kv_pool_release(r, p, 1 << 40, q, 1, None), c.kv_pool_compact(r, p, 1 << 40, q, None)):
        assert rc == 1
    x.check()


@pytest.mark.parametrize("k_format", ["q4g32", "q8g32", "tq3_qjl", "q8b32"])
def test_sampling_from_shared_prompts(k_format):
    """Two prompts, five samples that share their pages and go on by themselves: every one decodes as a cache does in which
    it was appended alone.  Samples end, others take their places, the pool is closed up in between."""
    rng = np.random.default_rng(31)
    S, L, H, W = 5, 2, 2, 64
    proj = synth.qjl_projection(4242)
    cfg = lib.make_config(L, H, 4, S, 640, window=W, n_pages=34, k_format=lib.K_FORMATS[k_format])
    table = torch.zeros(S, 10, dtype=torch.int32, device="cuda")
    gpu = QuantKVCache(cfg, "cuda", table, proj)
    gpu.pool_init()
    plain = QuantKVCache(lib.make_config(L, H, 4, S, 640, window=W, k_format=lib.K_FORMATS[k_format]), "cuda", None, proj)
    history = [None] * S                                  # every sequence's tokens so far

    def vec(T, h=H):
        return torch.as_tensor(rng.standard_normal((L, S, h, T, 128)).astype(np.float32)).bfloat16().cuda()

    def append(T, pos):
        k, v = vec(T), vec(T)
        granted = gpu.reserve(_i32(pos), T)
        assert granted.tolist() == list(pos)
        gpu.append(-1, k, v, granted)
        for b, p in enumerate(pos):
            if p >= 0:
                new = (k[:, b], v[:, b])
                history[b] = new if p == 0 else tuple(torch.cat((o[:, :, :p], n), 2) for o, n in zip(history[b], new))

    def check(lens):
        q = vec(1, 4).squeeze(3).contiguous()
        for b, n in enumerate(lens):
            if n:
                k, v = (torch.zeros(L, S, H, n, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
                k[:, b], v[:, b] = history[b]
                pos = [-1] * S
                pos[b] = 0
                plain.append(-1, k, v, _i32(pos))
        assert torch.equal(gpu.decode(-1, q, _i32(lens)), plain.decode(-1, q, _i32(lens)))
        assert gpu.status() == 0 and plain.status() == 0

    append(150, [0, -1, -1, -1, -1])
    append(200, [-1, -1, -1, 0, -1])
    lens = [150, 0, 0, 200, 0]
    check(lens)
    parents = [0, 0, 0, 3, 3]
    for turn in range(3):
        lens = gpu.fork(_i32(parents), _i32(lens)).tolist()
        history[:] = [history[q] if q >= 0 else history[b] for b, q in enumerate(parents)]
        check(lens)
        for T in (1, 30, 1, 45):
            append(T, lens)
            lens = [n + T for n in lens]
            check(lens)
        gpu.release(_i32([-1, 0, -1, -1, 0]))
        lens[1] = lens[4] = 0
        gpu.compact()
        check(lens)
        parents = [0, 2, 0, -1, 3]                        # (a sample ends its place and takes another's)
    refs = gpu.page_refs.cpu().numpy()
    t = table.cpu().numpy()
    assert np.array_equal(np.bincount(t[t >= 0], minlength=34), refs)


def test_prefill_onto_a_fork_and_eviction_of_a_shared_one():
    """A chunk appended to forks of one prompt (8-bit blocks), and a shared sequence made its own before it is cut."""
    rng = np.random.default_rng(33)
    table = torch.zeros(3, 10, dtype=torch.int32, device="cuda")
    cfg = lib.make_config(1, 2, 4, 3, 640, window=64, n_pages=30, k_format=lib.KVQ_Q8B32)
    gpu, ref = QuantKVCache(cfg, "cuda", table), br.Reference(cfg)
    gpu.pool_init()
    k, v = (torch.as_tensor(rng.standard_normal((3, 2, 111, 128)).astype(np.float32)).bfloat16() for _ in range(2))
    pos = gpu.reserve(_i32([0, -1, -1]), 111)
    gpu.append(0, k.cuda(), v.cuda(), pos)
    ref.append(0, harness.to_np(k), harness.to_np(v), [0, -1, -1])
    lens = gpu.fork(_i32([0, 0, 0]), _i32([111, 0, 0]))
    ref.fork([0, 0, 0])
    k, v, q = (torch.as_tensor(rng.standard_normal((3, h, 90, 128)).astype(np.float32)).bfloat16() for h in (2, 2, 4))
    out = gpu.prefill(0, k.cuda(), v.cuda(), q.cuda(), gpu.reserve(lens, 90)).cpu().numpy()
    ref.append(0, harness.to_np(k), harness.to_np(v), [111] * 3)
    for b in range(3):
        for t in (0, 40, 89):
            want = np.stack([ref.attend(0, b, j, harness.to_np(q)[b, j, t], 112 + t) for j in range(4)])
            harness.assert_attention_close(out[b, :, t], want, 2e-4)
    br.check_state(gpu, ref, [(0, b, h) for b in range(3) for h in range(2)], table.cpu().numpy())
    assert gpu.status() == 0

    x = Both(2, 640, 20)
    x.reserve([0], 600)
    x.fork([0, 0], [600, 0])
    x.reserve([-1, 0], 600)
    w = torch.rand(2, 2, 2, 640, device="cuda")
    before = x.pages.clone()
    _, new = x.gpu.evict(-1, w, _i32([0, 600]), 200, 64)
    x.gpu.release(torch.where(new < 600, new, -1).int() * _i32([0, 1]) + _i32([-1, 0]))
    x.ref.release([-1, 200])
    assert np.array_equal(x.bt.cpu().numpy(), x.ref.table)
    kept = x.bt[0].long()
    assert torch.equal(x.pages[:, kept], before[:, kept]) and (x.bt[1] >= 0).sum() == 4


def test_pages_and_rings_past_4_gib():
    """Pages copied, moved and rings forked at the far ends of arrays of 5 GB."""
    n_pages, n_seqs = 33000, 600
    cfg = lib.make_config(2, 8, 8, n_seqs, 640, window=1024, n_pages=n_pages)
    bt = torch.zeros(n_seqs, 10, dtype=torch.int32, device="cuda")
    gpu = QuantKVCache(cfg, "cuda", bt)
    gpu.pool_init()
    page, ring = 8 * 10240, 2 * n_seqs * 8 * 1024 * 512
    size = -(-2 * n_pages * page // 256) * 256
    off = lib.kv_cache_bytes(cfg) - size
    pages = gpu.buffer[off:off + 2 * n_pages * page].view(2, n_pages, page)
    assert ring % 256 == 0 and ring > 1 << 32 and n_pages * page * 2 > 1 << 32
    rings = [gpu.buffer[o:o + ring].view(torch.float32).view(2, n_seqs, 8, 1024, 128) for o in (off - 2 * ring, off - ring)]
    for r in rings:
        r[:, 3] = torch.randn_like(r[:, 3])
        r[:, 599] = 0
    pages[:, 32990] = torch.randint(0, 256, (2, page), dtype=torch.uint8, device="cuda")
    # sequence 3 has the far page, all the others below 32995 are counted as in use
    bt[3, 0] = 32990
    gpu.page_refs[:32995] = 1
    parents = torch.full((n_seqs,), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros_like(parents)
    parents[599], lens[3] = 3, 50
    new = gpu.fork(parents, lens)
    assert new[599] == 50 and bt[599, 0] == 32990 and gpu.page_refs[32990] == 2
    for r in rings:
        assert torch.equal(r[:, 599, :, :50], r[:, 3, :, :50]) and (r[:, 599, :, 50:] == 0).all()
    pos = torch.full_like(parents, -1)
    pos[599] = 50
    assert torch.equal(gpu.reserve(pos, 4), pos)
    assert bt[599, 0] == 32995 and gpu.page_refs[32990] == 1 and gpu.page_refs[32995] == 1
    assert torch.equal(pages[:, 32995], pages[:, 32990])
    # all but two pages given up, two far ones move to the front
    gpu.page_refs[:32990] = 0
    gpu.page_refs[32991:32995] = 0
    assert gpu.compact().item() == 2 and bt[3, 0] == 0 and bt[599, 0] == 1 and gpu.page_refs.sum() == 2
    assert torch.equal(pages[:, 0], pages[:, 32990]) and torch.equal(pages[:, 1], pages[:, 32990])
    assert gpu.status() == 0

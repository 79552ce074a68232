"""What the pool's calls and 8-bit block caches refuse before any device work, and the blocks' stored order (CPU)."""

import ctypes
import os

import numpy as np
import pytest
import torch

from kv_cache_quantization_append_gb300 import QuantKVCache, lib

from . import block_reference as br

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
    c = lib.kvq_cache()
    c.cfg = lib.make_config(2, 8, 24, 4, 1024, **kw)
    c.dev, c.block_table, c.max_pages_per_seq, c.n_pages = FAKE, FAKE + (1 << 40), 16, 64
    c.magic = 0x4B565131
    return c


def test_config(kvq):
    make = lambda **kw: lib.kv_cache_bytes(lib.make_config(2, 8, 24, 4, 1024, **kw))  # noqa: E731
    both = dict(k_format=lib.KVQ_Q8B32, v_format=lib.KVQ_Q8B32)
    assert make(**both) == make(k_format=lib.KVQ_Q8B32) > 0
    for window in (0, 4, 28):
        assert make(window=window, **both) == 0
    assert make(window=32, **both) > 0 and make(sinkhorn=True, **both) > 0
    assert make(k_format=lib.KVQ_Q8B32, v_format=lib.KVQ_Q4G32) == 0
    assert make(k_format=lib.KVQ_Q4G32, v_format=lib.KVQ_Q8B32) == 0
    # pages of 64 tokens: 256 B a token and 16 B a block
    assert make(n_pages=165, **both) - make(n_pages=164, **both) == 2 * 8 * 64 * 256 + 2 * 8 * 2 * 16


def test_operators_not_offered_for_block_caches(kvq):
    c = _cache(k_format=lib.KVQ_Q8B32)
    r, d = ctypes.byref(c), P(FAKE)
    assert kvq.kv_tree_scratch_bytes(r, 0, 1, 4) == 0 and kvq.kv_weights_scratch_bytes(r, 0, 1, 1) == 0
    assert kvq.kv_tree_attention(r, 0, d, d, d, d, d, d, 1, 4, d, 1 << 40, None) == UNSUPPORTED
    assert kvq.kv_tree_commit(r, 0, d, d, d, d, d, 1, 4, 4, None) == UNSUPPORTED
    assert kvq.kv_attention_weights(r, 0, d, d, 1.0, d, 1, 1, d, 1 << 40, None) == UNSUPPORTED
    assert kvq.kv_evict(r, 0, d, d, d, d, 1, 512, 128, None) == UNSUPPORTED


def test_pool(kvq):
    c = _cache()
    r, d, odd, big = ctypes.byref(c), P(FAKE), P(FAKE + 4), 1 << 30
    far = P(FAKE + 4096)
    n = kvq.kv_pool_bytes(r)
    assert n >= 64 * 4 and kvq.kv_pool_bytes(None) == 0 and kvq.kv_pool_bytes(ctypes.byref(lib.kvq_cache())) == 0
    calls = {
        "init": (kvq.kv_pool_init, [r, d, big, None], []),
        "reserve": (kvq.kv_pool_reserve, [r, d, big, d, None, far, 2, 1, None], [3, 5]),
        "fork": (kvq.kv_pool_fork, [r, d, big, d, d, far, 2, None], [3, 4, 5]),
        "release": (kvq.kv_pool_release, [r, d, big, d, 2, None], [3]),
        "compact": (kvq.kv_pool_compact, [r, d, big, d, None], [3]),
    }
    for name, (fn, good, pointers) in calls.items():
        def call(**at):
            args = list(good)
            for i, v in at.items():
                args[int(i[1:])] = v
            return fn(*args)

        assert call(_0=None) == INVALID and call(_0=ctypes.byref(lib.kvq_cache())) == NOT_INIT, name
        assert call(_1=None) == INVALID and call(_1=odd) == ALIGN and call(_2=n - 1) == CAPACITY, name
        for i in pointers:
            assert call(**{f"_{i}": None}) == INVALID and call(**{f"_{i}": odd}) == ALIGN, (name, i)
    for name, i in (("reserve", 6), ("fork", 6), ("release", 4)):
        fn, good, _ = calls[name]
        for b in (0, 5):
            args = list(good)
            args[i] = b
            assert fn(*args) == INVALID, (name, b)
    assert kvq.kv_pool_reserve(r, d, big, d, None, far, 2, 0, None) == INVALID
    assert kvq.kv_pool_reserve(r, d, big, d, odd, far, 2, 0, None) == ALIGN
    assert kvq.kv_pool_reserve(r, d, big, d, far, far, 2, 0, None) == INVALID          # granted over counts
    c.cfg.max_batch, c.n_pages = 8, 128
    assert kvq.kv_pool_reserve(r, d, big, P(FAKE + 16), None, P(FAKE), 8, 1, None) == INVALID   # half over pos
    assert kvq.kv_pool_fork(r, d, big, far, d, d, 2, None) == INVALID and kvq.kv_pool_fork(r, d, big, d, far, d, 2, None) == INVALID


def test_pool_needs_the_callers_table(kvq):
    """The table within the buffer is the identity that decode goes by without reading it: no pool writes it."""
    c = _cache()
    for off in range(256, 1 << 16, 256):                      # it lies within the header, at a 256-byte boundary
        c.block_table = FAKE + off
        if kvq.kv_pool_init(ctypes.byref(c), P(FAKE), 1 << 30, None) == UNSUPPORTED:
            break
    else:
        raise AssertionError("the identity table was taken")


def test_wrapper_without_a_pool():
    q = QuantKVCache.__new__(QuantKVCache)
    q.pool = q.handle = None
    for call in (lambda: q.reserve(None, 1), lambda: q.fork(None, torch.zeros(1)), lambda: q.release(None), lambda: q.page_refs):
        with pytest.raises(lib.KVQError, match="pool_init"):
            call()


def test_stored_order_is_one_to_one():
    k, v = br.offsets()
    assert sorted(k.ravel()) == list(range(4096)) and sorted(v.ravel()) == list(range(4096, 8192))


def test_block_codec():
    """The codes' definition: nearest of 255 levels of the largest magnitude, ties to even, zero blocks, tiny scales."""
    rng = np.random.default_rng(0)
    y = rng.standard_normal((5, 32, 128)).astype(np.float32)
    y[1] = 0
    y[2] *= 1e-42
    y[3, 0, 0] = 127.0
    y[3, 1:] = np.float32(2.5)
    c, d = br.encode(y)
    assert np.abs(c).max() <= 127 and (c[1] == 0).all() and d[1] == 0
    assert d[3] == 1.0 and (c[3, 1:] == 2).all()
    back = c[0] * d[0].astype(np.float64)
    assert np.abs(back - y[0]).max() <= d[0] * (0.5 + 2.0 ** -16) and np.abs(c[0]).max() == 127

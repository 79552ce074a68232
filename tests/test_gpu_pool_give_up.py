"""A fork whose waits run out (a limit of 1 ns): flagged, the table and counts as documented, no ring but the changing ones touched."""

import time

import pytest
import torch

from kv_cache_quantization_append_gb300 import lib

from .test_gpu_pool import Both, _i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,layers,heads,window", [("q4g32", 8, 8, 128), ("q8b32", 2, 2, 64)])
def test_a_fork_that_gives_up(fmt, layers, heads, window):
    x = Both(6, 640, 60, fmt, layers=layers, heads=heads, window=window)
    lens = [200, 70, 300, 1, 128, 0]
    x.reserve([0] * 6, lens)
    parents = [1, 0, -1, 2, 2, 2]
    before = [r.clone() for r in x.rings]
    lib.kv_set_wait_limit_ns(1)
    try:
        t0 = time.time()
        new = x.gpu.fork(_i32(parents), _i32(lens))
        flags = x.gpu.status()
        assert time.time() - t0 < 5
    finally:
        lib.kv_set_wait_limit_ns(10 ** 9)
    assert flags == lib.DEV_TIMEOUT
    assert new.tolist() == x.ref.fork(parents, lens)
    x.check()
    for r, old in zip(x.rings, before):
        assert torch.equal(r[:, 2], old[:, 2])
        for b, q in enumerate(parents):
            if q >= 0:                                     # each vector is the old one or the parent's
                assert ((r[:, b] == old[:, b]) | (r[:, b] == old[:, q])).all()
    # forked again from the one that stayed, all is whole; so is what is released and taken anew
    lens = x.fork([2, 2, -1, 2, -1, -1], new.tolist())
    x.release([-1, -1, -1, -1, 0, 0])
    lens[4] = lens[5] = 0
    x.reserve(lens, 1)
    x.fork([-1, -1, -1, -1, 0, 3], lens)

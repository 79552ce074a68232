"""Waits within the blocks of a prefill over KVQ_Q8B32 caches that run out (a limit of 1 ns, which no wait for a copy or a
product meets): the call comes back soon, is flagged, leaves NaN and an appended chunk, and nothing that the next call sees."""

import time

import numpy as np
import pytest
import torch

from kv_cache_quantization_append_gb300 import lib

from . import block_reference as br
from . import harness
from .test_gpu_block8 import _append, _i32, _units, _vectors

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,T,hkv,layers", [([3000, -1, 17], 40, 2, 1),          # cut over all blocks
                                               ([0, -1, 300, 0], 500, 4, 2),        # row tiles taken whole
                                               ([5], 1, 1, 1)])
def test_a_prefill_that_gives_up(in_dtype, lens, T, hkv, layers):
    rng = np.random.default_rng(T)
    B = len(lens)
    gpu, ref = br.make(layers, hkv, 4 * hkv, B, max(lens) + T, window=64, in_dtype=in_dtype)
    for b, n in enumerate(lens):
        if n > 0:
            _append(gpu, ref, -1, rng, n, [n and (0 if i == b else -1) for i in range(B)], in_dtype)
    k, v = (_vectors(rng, (layers, B, hkv, T), in_dtype) for _ in range(2))
    q = _vectors(rng, (layers, B, 4 * hkv, T), in_dtype).cuda()
    state = gpu.buffer.clone()

    def call(limit):
        gpu.buffer.copy_(state)
        out = torch.full(q.shape, 7.0, device="cuda")
        lib.kv_set_wait_limit_ns(limit)
        t0 = time.time()
        try:
            gpu.prefill(-1, k.cuda(), v.cuda(), q, _i32(lens), out=out)
            flags = gpu.status()
        finally:
            lib.kv_set_wait_limit_ns(10 ** 9)
        return out, flags, time.time() - t0

    good, flags, _ = call(10 ** 9)
    assert flags == 0
    ref.append(-1, harness.to_np(k), harness.to_np(v), lens)
    out, flags, took = call(1)
    assert flags == lib.DEV_TIMEOUT and took < 5
    here = torch.as_tensor(np.asarray(lens) >= 0).cuda()
    assert torch.isnan(out[:, here]).all() and (out[:, ~here] == 0).all()
    br.check_state(gpu, ref, _units(gpu.cfg))
    again, flags, _ = call(10 ** 9)
    assert flags == 0 and torch.equal(again, good)

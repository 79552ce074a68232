"""Waits within the tree's and the weights' blocks that run out (a limit of 1 ns, which no wait for a copy or a product
meets): the call comes back soon, is flagged, and leaves nothing behind that the next call could see."""

import time

import numpy as np
import pytest
import torch

from kv_cache_quantization_append_gb300 import lib

from . import harness
from . import ops_reference as ref
from .test_gpu_tree import _drafts

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


@pytest.mark.parametrize("k_format", ["q4g32", "q8g32", "tq3_qjl"])
@pytest.mark.parametrize("in_dtype,g,N", [("bf16", 1, 3), ("bf16", 3, 30), ("f32", 2, 1), ("f32", 4, 20)])
def test_a_wait_that_runs_out(k_format, in_dtype, g, N):
    rng = np.random.default_rng(N)
    gpu, _, _ = harness.make_pair(1, 4, 4 * g, 3, 3000, k_format=k_format, in_dtype=in_dtype)
    dt = torch.bfloat16 if in_dtype == "bf16" else torch.float32
    k = torch.as_tensor(rng.standard_normal((3, 4, 3000, 128)).astype(np.float32)).to(dt).cuda()
    gpu.append(0, k, k, _i32([0] * 3))
    dk, dv, q = (t.cuda() for t in _drafts(rng, gpu.cfg, 3, N, in_dtype))
    lens = [3000, 17, 1400]
    ln = _i32(lens)
    parents = np.stack([ref.random_tree(rng, N) for _ in range(3)])
    parents[1, N // 2:] = -2
    here = torch.as_tensor(np.array([[bool(ref.chain_of(p, i)) for i in range(N)] for p in parents])).cuda()
    parents = _i32(parents)
    old = torch.as_tensor(rng.random((3, 4, 3000)).astype(np.float32)).cuda()

    def calls():
        w = old.clone()
        out = gpu.tree_decode(0, dk, dv, q, ln, parents).transpose(1, 2)      # [B][N][Hq][128]
        flags = gpu.status()
        gpu.attention_weights(0, q, ln, w, 0.5)
        return out, w, flags, gpu.status()

    good = calls()
    assert good[2:] == (0, 0)
    lib.kv_set_wait_limit_ns(1)
    try:
        t0 = time.time()
        out, w, *flags = calls()
        assert time.time() - t0 < 5
    finally:
        lib.kv_set_wait_limit_ns(10 ** 9)
    assert flags == [lib.DEV_TIMEOUT] * 2
    assert torch.isnan(out[here]).all() and (out[~here] == 0).all()
    assert ((w == old) | (w == old * 0.5)).all()
    again = calls()
    assert again[2:] == (0, 0)
    assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])

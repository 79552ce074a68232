"""A CUDA call that failed is reported by the entry point that made it, and by no later one."""

import ctypes

import pytest
import torch

from kv_cache_quantization_append_gb300 import lib

from . import harness

pytestmark = pytest.mark.gpu


def test_a_failed_query_does_not_fail_the_next_call():
    gpu, _, _ = harness.make_pair(1, 1, 1, 1, 64, window=0)
    other = lib.kvq_cache.from_buffer_copy(gpu.handle)
    other.device = 63                                       # (no such device: the query of its size fails)
    x = torch.zeros(1, 1, 3 * 128, dtype=torch.bfloat16, device="cuda")
    q, k, v = (torch.empty(1, 1, 1, 128, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    path = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    rope = lib.kv_rope_init(128)
    calls = (lambda: lib.kv_qk_norm_rope(rope, x, path, q, k, v),
             lambda: lib.kv_tree_commit(gpu.handle, 0, k, v, path, pos + 1, pos),
             lambda: lib.kv_quant_append(gpu.handle, 0, k, v, pos),
             lambda: lib.kv_prefill_attention(gpu.handle, 0, k, v, q, torch.empty(1, 1, 1, 128, device="cuda"), pos,
                                              torch.empty(1 << 16, dtype=torch.uint8, device="cuda")))
    for call in calls:
        call()
        lib.load().kv_tree_scratch_bytes(ctypes.byref(other), 0, 1, 1)
        call()
    torch.cuda.synchronize()
    assert gpu.status() == 0


def test_a_single_row_of_any_width():
    """One row of projections with a few values behind its heads: there is no second row that its width could misalign."""
    rope = lib.kv_rope_init(128)
    wide = torch.randn(1, 1, 3 * 128 + 3, device="cuda")
    outs = []
    for x in (wide, wide[:, :, :3 * 128].contiguous()):
        q, k, v = (torch.empty(1, 1, 1, 128, device="cuda") for _ in range(3))
        lib.kv_qk_norm_rope(rope, x, torch.full((1, 1), 5, dtype=torch.int32, device="cuda"), q, k, v)
        outs.append(torch.cat([q, k, v]))
    assert torch.equal(*outs)

"""Tree attention against its 64-bit definition where operands of fewer bits would show: outputs of bf16 caches that are
the definition rounded once."""

import numpy as np
import pytest
import torch

from . import harness
from . import ops_reference as ref
from .test_gpu_tree import TOL, _drafts, _fill

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def _tree(gpu, k, v, q, lens, parents):
    out = gpu.tree_decode(0, k.cuda(), v.cuda(), q.cuda(), _i32(lens), _i32(parents))
    torch.cuda.synchronize()
    assert gpu.status() == 0
    return out.double().cpu().numpy()


def _half_step(in_dtype, want):
    return 2.0 ** -8 * np.abs(want) if in_dtype == "bf16" else 0.0


@pytest.mark.parametrize("k_format", ["q4g32", "q8g32", "tq3_qjl"])
@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_q,N,L,window", [(3, 5, 700, 128), (3, 16, 700, 0), (4, 32, 500, 64), (3, 64, 300, 128)])
def test_outputs_are_the_definition_rounded_once(k_format, in_dtype, n_q, N, L, window):
    """Peaked attention (queries of four times a unit head's size), whose logits of up to 60 magnify what queries and keys
    lose.  Each output element is off by its own half step and, beside that, by what a float cache's may be: operands of 22
    bits (of a bf16 cache's raw vectors 16: |q| |k| / sqrt(128) = 45, so six standard deviations of the logit's error are
    6 * 4 * 2^-18 / sqrt(3) = 5e-5, the values' and weights' 2^-17 each) and the truncating accumulations of 2e-4."""
    rng = np.random.default_rng(N + L)
    gpu, ora, _ = harness.make_pair(1, 1, n_q, 1, 720, window=window, k_format=k_format, in_dtype=in_dtype)
    _fill(gpu, ora, [L], L, rng, in_dtype)
    k, v, q = _drafts(rng, gpu.cfg, 1, N, in_dtype)
    q = q * 4
    parents = ref.random_tree(rng, N)[None]
    got = _tree(gpu, k, v, q, [L], parents)
    want = ref.tree_attention(ora, 0, harness.to_np(k), harness.to_np(v), harness.to_np(q), np.array([L]), parents)
    err = np.abs(got - want) - _half_step(in_dtype, want)
    assert err.max() <= TOL["f32"] * np.abs(want).max(), err.max() / np.abs(want).max()


@pytest.mark.parametrize("in_dtype,scale", [("bf16", 2.0 ** -24), ("bf16", 2.0 ** 12), ("f32", 2.0 ** -110),
                                            ("f32", 2.0 ** -24), ("f32", 2.0 ** -10), ("f32", 2.0 ** 12)])
def test_raw_values_of_any_size(in_dtype, scale):
    """Values in the ring and the drafts far below and above one: the output scales with them."""
    rng = np.random.default_rng(3)
    gpu, ora, _ = harness.make_pair(1, 2, 4, 1, 200, in_dtype=in_dtype)
    dt = torch.bfloat16 if in_dtype == "bf16" else torch.float32
    _fill(gpu, ora, [100], 100, rng, in_dtype)
    kk, vv = (torch.as_tensor((rng.standard_normal((1, 2, 100, 128)) * s).astype(np.float32)).to(dt) for s in (1, scale))
    gpu.append(0, kk.cuda(), vv.cuda(), _i32([0]))
    ora.append(0, harness.to_np(kk), harness.to_np(vv), np.zeros(1, int))
    k, v, q = _drafts(rng, gpu.cfg, 1, 9, in_dtype)
    v = v * scale
    parents = ref.random_tree(rng, 9)[None]
    got = _tree(gpu, k, v, q, [100], parents)
    want = ref.tree_attention(ora, 0, harness.to_np(k), harness.to_np(v), harness.to_np(q), np.array([100]), parents)
    err = np.abs(got - want) - _half_step(in_dtype, want)
    assert err.max() <= TOL["f32"] * np.abs(want).max(), err.max() / np.abs(want).max()

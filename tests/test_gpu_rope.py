"""kv_qk_norm_rope against its 64-bit definition: layouts, partial and scaled rotations, far positions, odd sizes."""

import numpy as np
import pytest
import torch

from kv_cache_quantization_append_gb300 import lib

from . import ops_reference as ref

pytestmark = pytest.mark.gpu

SCALINGS = {0: (500000.0, 1.0, 0.0, 0.0, 0.0, 1.0), 1: (10000.0, 4.0, 0.0, 0.0, 0.0, 1.0), 2: (10000.0, 8.0, 0.0, 0.0, 0.0, 1.0),
            3: (500000.0, 8.0, 8192.0, 1.0, 4.0, 1.0), 4: (10000.0, 16.0, 4096.0, 1.0, 32.0, 1.277)}


def _tol(dtype, want):
    """fp32 arithmetic: the angle's 2^-24 of up to pi and the sines' 2^-22, the norm's sum of 128 (2^-21), three products:
    2^-19 of the pair's magnitude covers them (the head's largest value bounds that); bf16 adds half a step, 2^-8."""
    scale = np.abs(want).max(-1, keepdims=True)
    return scale * 2.0 ** -19 + (np.abs(want) * 2.0 ** -8 if dtype == torch.bfloat16 else 0.0) + 1e-30


def _run(B, T, hq, hkv, dtype, layout, rot, scaling, norm, first, pad=0, seed=0, with_v=True):
    g = torch.Generator().manual_seed(seed)
    row = (hq + (2 if with_v else 1) * hkv) * 128
    x = torch.randn(B, T, row + pad, generator=g).to(dtype)
    pos = (first + torch.arange(T)[None] + 7 * torch.arange(B)[:, None]).int()
    wq, wk = ((1 + 0.2 * torch.randn(128, generator=g)).to(dtype) if norm else None for _ in range(2))
    th, fac, n0, lo, hi, att = SCALINGS[scaling]
    rope = lib.kv_rope_init(rot, layout, th, scaling, fac, n0, lo, hi, att)
    q = torch.full((B, hq, T, 128), 7.0, dtype=dtype, device="cuda")
    k, v = (torch.full((B, hkv, T, 128), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    xd = x.cuda()[:, :, :row]
    lib.kv_qk_norm_rope(rope, xd, pos.cuda(), q, k, v if with_v else None, dev(wq), dev(wk), 1e-6)
    torch.cuda.synchronize()
    xs = x[:, :, :row].double().numpy().reshape(B, T, -1, 128).transpose(0, 2, 1, 3)
    f = ref.frequencies(rot, th, scaling, fac, n0, lo, hi) if rot else np.zeros(0)
    num = lambda w: None if w is None else w.double().numpy()  # noqa: E731
    want_q = ref.norm_rope(xs[:, :hq], pos.numpy(), num(wq), 1e-6, rot, layout, f, np.float32(att))
    want_k = ref.norm_rope(xs[:, hq:hq + hkv], pos.numpy(), num(wk), 1e-6, rot, layout, f, np.float32(att))
    for got, want in ((q, want_q), (k, want_k)):
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= _tol(dtype, want)).all(), (err / _tol(dtype, want)).max()
    if with_v:
        assert np.array_equal(v.double().cpu().numpy(), xs[:, hq + hkv:])
    else:
        assert (v == 7).all()


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rot", [0, 2, 6, 16, 48, 64, 90, 128])
def test_partial_rotations(layout, dtype, rot):
    _run(2, 5, 6, 2, dtype, layout, rot, 0, rot % 4 == 0, 100)


@pytest.mark.parametrize("scaling", [1, 2, 3, 4])
@pytest.mark.parametrize("first", [0, 131000, 2 ** 31 - 64])
def test_scalings_at_near_and_far_positions(scaling, first):
    _run(2, 9, 3, 1, torch.float32, 0, 128, scaling, True, first)
    _run(1, 3, 4, 2, torch.bfloat16, 1, 64, scaling, False, first)


@pytest.mark.parametrize("B,T,hq,hkv", [(1, 1, 1, 1), (8, 1, 32, 8), (3, 257, 5, 5), (1, 2500, 24, 8)])
def test_shapes(B, T, hq, hkv):
    _run(B, T, hq, hkv, torch.bfloat16, 0, 128, 3, True, 11)


def test_row_stride_and_no_values():
    _run(2, 3, 4, 2, torch.bfloat16, 0, 128, 0, True, 5, pad=24)
    _run(1, 4, 4, 2, torch.float32, 1, 32, 0, True, 5, pad=4)
    _run(2, 3, 4, 2, torch.bfloat16, 0, 64, 0, True, 5, with_v=False)


def test_decode_form_and_padded_rows():
    """Without the T axis; a negative position leaves its row's outputs as they were."""
    x = torch.randn(3, 1, 8 * 128, device="cuda").bfloat16()
    rope = lib.kv_rope_init(128, theta=500000.0)
    pos = torch.tensor([[5], [-1], [9]], dtype=torch.int32, device="cuda")
    q = torch.full((3, 4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.full((3, 2, 128), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lib.kv_qk_norm_rope(rope, x, pos, q, k, v)
    full = [torch.empty(3, h, 1, 128, dtype=torch.bfloat16, device="cuda") for h in (4, 2, 2)]
    lib.kv_qk_norm_rope(rope, x, pos.clamp_min(0), *full)
    for a, b in zip((q, k, v), full):
        assert torch.equal(a[0], b[0, :, 0]) and torch.equal(a[2], b[2, :, 0])
        assert (a[1] == 3).all()


def test_infinities_stay_in_their_head():
    """A head with an infinity or NaN does not touch the others."""
    x = torch.randn(1, 2, 6 * 128, device="cuda")
    rope = lib.kv_rope_init(128)
    pos = torch.arange(2, dtype=torch.int32, device="cuda")[None]
    w = torch.ones(128, device="cuda")
    out = [torch.empty(1, h, 2, 128, device="cuda") for h in (4, 1, 1)]
    lib.kv_qk_norm_rope(rope, x, pos, *out, w, w)
    y = x.clone()
    y[0, 0, 130] = float("inf")
    y[0, 1, 3] = float("nan")
    out2 = [torch.empty_like(t) for t in out]
    lib.kv_qk_norm_rope(rope, y, pos, *out2, w, w)
    same = torch.ones(1, 4, 2, dtype=torch.bool)
    same[0, 1, 0] = same[0, 0, 1] = False
    assert torch.equal(out[0][same.cuda()], out2[0][same.cuda()]) and torch.equal(out[1], out2[1])
    assert out2[0][0, 0, 1].isnan().any() and out2[0][0, 1, 0].isnan().any()


def test_captured_and_replayed():
    """Captured into a graph and replayed on new inputs in the same buffers."""
    x = torch.randn(2, 3, 8 * 128, device="cuda").bfloat16()
    pos = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    rope = lib.kv_rope_init(64, lib.ROPE_INTERLEAVED)
    out = [torch.zeros(2, h, 3, 128, dtype=torch.bfloat16, device="cuda") for h in (4, 2, 2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.kv_qk_norm_rope(rope, x, pos, *out)
    x.normal_()
    pos.copy_(torch.arange(6, dtype=torch.int32).view(2, 3))
    graph.replay()
    want = [torch.zeros_like(t) for t in out]
    lib.kv_qk_norm_rope(rope, x, pos, *want)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_refuses_tensors_off_the_current_device(monkeypatch):
    rope = lib.kv_rope_init(128)
    x = torch.zeros(1, 1, 3 * 128, device="cuda")
    q, k, v = (torch.zeros(1, 1, 1, 128, device="cuda") for _ in range(3))
    pos = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    lib.kv_qk_norm_rope(rope, x, pos, q, k, v)
    with pytest.raises(lib.KVQError):
        lib.kv_qk_norm_rope(rope, x, pos.cpu(), q, k, v)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: x.get_device() + 1)
    with pytest.raises(lib.KVQError):
        lib.kv_qk_norm_rope(rope, x, pos, q, k, v)

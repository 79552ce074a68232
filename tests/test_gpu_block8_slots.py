"""Prefill over KVQ_Q8B32 caches of many slots of which few are active: every row of an active slot is computed."""

import numpy as np
import pytest
import torch

from . import block_reference as br
from . import harness
from .test_gpu_block8 import TOL, _i32, _vectors

pytestmark = pytest.mark.gpu


def _case(rng, hkv, g, T, p, in_dtype, window):
    """A prompt, a chunk behind it and some of the chunk's outputs by the definition: [tokens looked at], [Hq][tokens][128]."""
    ref = br.Reference(br.lib.make_config(1, hkv, hkv * g, 1, 1200, window=window, k_format=br.lib.KVQ_Q8B32))
    prompt = [_vectors(rng, (hkv, max(p, 1)), in_dtype) for _ in range(2)]
    k, v, q = (_vectors(rng, (h, T), in_dtype) for h in (hkv, hkv, hkv * g))
    if p:
        ref.append(0, *(harness.to_np(x)[None] for x in prompt), [0])
    ref.append(0, harness.to_np(k)[None], harness.to_np(v)[None], [p])
    ts = sorted({0, T // 2, T - 1})
    qn = harness.to_np(q)
    want = np.stack([[ref.attend(0, 0, j, qn[j, t], p + t + 1) for t in ts] for j in range(hkv * g)])
    return [x.cuda() for x in prompt], [x.cuda() for x in (k, v, q)], ts, want


def _run(gpu, rows, B, pos, where):
    """The chunk at the slots `where` (the others hold other vectors and are absent); what the call makes of a buffer of NaN."""
    k, v, q = (torch.full((B,) + tuple(x.shape), 3.0, dtype=x.dtype, device="cuda") for x in rows)
    for x, row in zip((k, v, q), rows):
        x[where] = row
    at = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    at[where] = pos
    out = torch.full(q.shape, float("nan"), device="cuda")
    gpu.prefill(0, k, v, q, at, out=out)
    return out


@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,hkv,g", [(9, 1, 4), (16, 8, 4), (16, 4, 3), (32, 2, 4), (32, 8, 1), (64, 8, 2), (64, 1, 4)])
def test_one_active_slot(in_dtype, B, hkv, g):
    """Any slot: the same outputs, the definition's; zeros elsewhere."""
    rng = np.random.default_rng(B + hkv + g)
    window = 64
    for p in (0, 50, 1000):
        for T in (1, 20, 37, 64, 100):
            prompt, rows, ts, want = _case(rng, hkv, g, T, p, in_dtype, window)
            gpu, _ = br.make(1, hkv, hkv * g, B, 1200, window=window, in_dtype=in_dtype)
            if p:
                gpu.append(0, *(x.expand(B, -1, -1, -1).contiguous() for x in prompt), _i32([0] * B))
            first = None
            for s in range(B):
                out = _run(gpu, rows, B, p, [s])
                if first is None:
                    first = out[s].clone()
                    harness.assert_attention_close(first[:, ts].double().cpu().numpy(), want, TOL)
                assert torch.equal(out[s], first), (p, T, s)
                out[s] = 0
                assert (out == 0).all(), (p, T, s)
            assert gpu.status() == 0


@pytest.mark.parametrize("where", [[0, 63], [15, 16, 47], [7, 8, 9, 40], list(range(0, 64, 5)), list(range(32, 64))])
@pytest.mark.parametrize("hkv,g,T,p", [(8, 4, 20, 0), (1, 4, 130, 0), (2, 1, 37, 70), (4, 2, 1, 0), (8, 2, 300, 5)])
def test_some_active_slots(hkv, g, T, p, where):
    rng = np.random.default_rng(T + p + len(where))
    prompt, rows, ts, want = _case(rng, hkv, g, T, p, "bf16", 32)
    gpu, _ = br.make(1, hkv, hkv * g, 64, 1200, window=32)
    if p:
        gpu.append(0, *(x.expand(64, -1, -1, -1).contiguous() for x in prompt), _i32([0] * 64))
    out = _run(gpu, rows, 64, p, where)
    for s in where:
        harness.assert_attention_close(out[s][:, ts].double().cpu().numpy(), want, TOL)
    assert torch.isfinite(out).all()
    out[where] = 0
    assert (out == 0).all() and gpu.status() == 0


def test_the_last_of_1024_slots():
    rng = np.random.default_rng(5)
    prompt, rows, ts, want = _case(rng, 1, 4, 40, 0, "bf16", 32)
    gpu, _ = br.make(1, 1, 4, 1024, 128, window=32)
    for s in (0, 511, 1023):
        out = _run(gpu, rows, 1024, 0, [s])
        harness.assert_attention_close(out[s][:, ts].double().cpu().numpy(), want, TOL)
        out[s] = 0
        assert (out == 0).all()

"""Weights and eviction over several cuts, with what a loop has to do between them; the README's loop, as it stands."""

import os

import numpy as np
import pytest
import torch

from kv_cache_quantization_append_gb300 import lib

from . import harness
from . import ops_reference as ref
from .test_gpu_tree import _drafts, _fill

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def _close(got, want):
    # as in the other tests of the weights: logits to 8e-5, sums to a few 2^-24
    assert (np.abs(got - want) <= 1e-4 * want + 1e-12).all(), (np.abs(got - want) / (want + 1e-12)).max()


@pytest.mark.parametrize("k_format", ["q4g32", "q8g32", "tq3_qjl"])
def test_weights_decay_over_two_cuts(k_format):
    """Evict, commit drafts, accumulate with a decay, evict again: positions, weights and records follow the definition, and
    tokens in slots that the first cut freed carry nothing of the positions that were there."""
    rng = np.random.default_rng(61)
    B, hq, hkv, S, budget, recent = 2, 4, 2, 400, 180, 40
    gpu, ora, _ = harness.make_pair(1, hkv, hq, B, S, window=32, k_format=k_format)
    lens = np.array([390, 260])
    _fill(gpu, ora, lens, 390, rng, "bf16")
    w = torch.zeros(B, hkv, S, device="cuda")
    host = np.zeros((B, hkv, S))
    for turn in range(3):
        for _ in range(4 if turn else 1):
            k, v, q = _drafts(rng, gpu.cfg, B, 9, "bf16")
            parents = [ref.random_tree(rng, 9) for _ in range(B)]
            paths = [max((ref.chain_of(p, i) for i in range(9)), key=len) for p in parents]
            n = np.array([len(p) for p in paths])
            gpu.commit(0, k.cuda(), v.cuda(), _i32([p + [0] * (9 - len(p)) for p in paths]), _i32(n), _i32(lens))
            for b in range(B):
                one = np.full(B, -1)
                one[b] = lens[b]
                ora.append(0, harness.to_np(k)[:, :, paths[b]], harness.to_np(v)[:, :, paths[b]], one)
            lens = lens + n
            T = int(n.min())                                   # the newest T tokens' queries, in order
            newest = torch.stack([q[b][:, paths[b][len(paths[b]) - T:]] for b in range(B)])
            gpu.attention_weights(0, newest.cuda(), _i32(lens), w, 0.75)
            host = ref.attention_weights(ora, 0, harness.to_np(newest), lens, host, 0.75)
            for b in range(B):
                _close(w[b, :, :lens[b]].double().cpu().numpy(), host[b, :, :lens[b]])
        before = w.cpu().numpy()[None].copy()                  # (ranks of what the kernel summed)
        kept, new = gpu.evict(0, w, _i32(lens), budget, recent)
        want = ref.evict(ora, before, lens, budget, recent)[0]
        assert np.array_equal(kept.cpu().numpy(), want)
        host64 = host.copy()
        for b in range(B):
            for h in range(hkv):
                src = want[b, h][want[b, h] >= 0]
                host64[b, h, :len(src)] = host[b, h, src]
        host, lens = host64, np.minimum(lens, budget)
        assert np.array_equal(new.cpu().numpy(), lens)
        w[..., budget:] = 0
        host[..., budget:] = 0
        for b in range(B):
            for h in range(hkv):
                harness.compare_codes(gpu, ora, 0, b, h, int(lens[b]))
                harness.compare_ring(gpu, ora, 0, b, h, int(lens[b]))
    assert gpu.status() == 0


def test_the_readme_loop():
    """The block that shows the operators around append and decode, run as it is at the sizes it names: the lengths, weights
    and kept positions that it ends with are those of the definition after the commit."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md")) as f:
        code = next(b.split("```")[0] for b in f.read().split("```python")[1:] if "tree_decode" in b)
    rng = np.random.default_rng(67)
    B, N, hq, hkv, S = 2, 6, 24, 8, 8448
    gpu, ora, _ = harness.make_pair(1, hkv, hq, B, S)
    lens = np.array([8300, 200])
    _fill(gpu, ora, lens, 8300, rng, "bf16")
    dt = dict(dtype=torch.bfloat16, device="cuda")
    paths, n = np.array([[0, 2, 5, 0, 0, 0], [0, 1, 0, 0, 0, 0]]), np.array([3, 2])
    q, k, v = (torch.empty(B, h, N, 128, **dt) for h in (hq, hkv, hkv))
    env = dict(torch=torch, lib=lib, cache=gpu, rows=torch.randn(B, N, (hq + 2 * hkv) * 128, **dt), q=q, k=k, v=v, wq=torch.ones(128, **dt),
               wk=torch.ones(128, **dt), positions=_i32(lens[:, None] + np.array([0, 1, 1, 2, 1, 2])),
               parents=_i32([[-1, 0, 0, 1, 0, 2]] * B), path=_i32(paths), n_accept=_i32(n), lens=_i32(lens),
               weights=torch.zeros(B, hkv, S, device="cuda"))
    exec(code, env)
    torch.cuda.synchronize()
    assert gpu.status() == 0
    for b in range(B):
        one = np.full(B, -1)
        one[b] = lens[b]
        ora.append(0, harness.to_np(k)[:, :, paths[b, :n[b]]], harness.to_np(v)[:, :, paths[b, :n[b]]], one)
    lens = lens + n
    newest = np.stack([harness.to_np(q)[b][:, paths[b, n[b] - 1:n[b]]] for b in range(B)])
    want = ref.attention_weights(ora, 0, newest, lens, np.zeros((B, hkv, S)), 0.0)
    assert env["lens"].tolist() == [8192, 202]
    got, kept = env["weights"].double().cpu().numpy(), env["kept"].cpu().numpy()
    assert np.array_equal(kept[1, :, :202], np.tile(np.arange(202), (hkv, 1))) and (kept[1, :, 202:] == -1).all()
    _close(got[1, :, :202], want[1, :, :202])
    for h in range(hkv):
        src = kept[0, h]
        assert (np.diff(src) > 0).all() and np.array_equal(src[-256:], np.arange(lens[0] - 256, lens[0]))
        _close(got[0, h, :8192], want[0, h, src])
        gone = np.setdiff1d(np.arange(lens[0]), src)
        assert want[0, h, gone].max() <= want[0, h, src[:-256]].min() * (1 + 2e-4)
    assert (got[:, :, 8192:] == 0).all()

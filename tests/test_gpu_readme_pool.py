"""The README's sampling loop, run as it stands, with pages for everyone and with too few."""

import os

import numpy as np
import pytest
import torch

from kv_cache_quantization_append_gb300 import QuantKVCache, lib

from . import block_reference as br
from . import harness
from .test_gpu_block8 import TOL, _i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_pages", [40, 5])
def test_the_sampling_loop(n_pages):
    """Two prompts of 127 tokens, three samples of the first.  With 5 pages, of which the prompts take 4, only the first sample gets
    the copy that its next token needs: the others are decoded as they were."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md")) as f:
        code = next(b.split("```")[0] for b in f.read().split("```python")[1:] if "cache.fork" in b)
    rng = np.random.default_rng(71)
    B, L, H, Hq, T = 4, 2, 2, 4, 127
    cfg = lib.make_config(L, H, Hq, B, 320, window=64, n_pages=n_pages, k_format=lib.KVQ_Q8B32)
    ref = br.Reference(cfg)

    def vec(h, t):
        return torch.as_tensor(rng.standard_normal((L, B, h, t, 128)).astype(np.float32)).bfloat16()

    k, v, q, k1, v1, q1 = vec(H, T), vec(H, T), vec(Hq, T), vec(H, 1), vec(H, 1), vec(Hq, 1).squeeze(3).contiguous()
    env = dict(torch=torch, QuantKVCache=QuantKVCache, cfg=cfg, max_batch=B, max_pages=5, T=T, pos=_i32([0, -1, 0, -1]),
               lens=_i32([0] * B), parents=_i32([0, 0, 2, 0]), keep_lens=_i32([0, -1, -1, -1]),
               **{n: x.cuda() for n, x in dict(k=k, v=v, q=q, k1=k1, v1=v1, q1=q1).items()})
    exec(code, env)
    cache = env["cache"]
    # tokens 127 are within the second page: shared by 0, 1, 3 (the last keeps it) and 2's own; the copies need two pages
    got = [127, 127, 127, 127] if n_pages == 40 else [127, -1, -1, -1]
    assert env["granted"].tolist() == got
    assert cache.status() == (0 if n_pages == 40 else lib.DEV_NO_PAGES)
    lens = [128 if g >= 0 else 127 for g in got]
    assert env["lens"].tolist() == lens
    ref.append(-1, harness.to_np(k), harness.to_np(v), [0, -1, 0, -1])
    ref.fork([0, 0, 2, 0])
    ref.append(-1, harness.to_np(k1), harness.to_np(v1), got)
    out = env["out"].double().cpu().numpy()
    for lay in range(L):
        want = ref.decode(lay, harness.to_np(q1)[lay], lens)
        for b in range(B):
            harness.assert_attention_close(out[lay, b], want[b], TOL)
    refs = cache.page_refs.cpu().numpy()
    t = env["table"].cpu().numpy()
    assert (t[0] == -1).all() and np.array_equal(np.bincount(t[t >= 0], minlength=n_pages), refs)
    assert env["n_used"].item() == (refs > 0).sum()

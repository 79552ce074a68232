"""Quantized KV cache for GB300: append (rotate, balance, 4-bit / 3-bit+QJL pack) and decode
attention over the compressed cache, as hand-written sm_103a CUDA behind a C ABI (include/kvq.h).

``lib`` is the thin ctypes binding (same names as the C entry points).  ``QuantKVCache`` only
owns the torch allocations a caller needs (cache buffer, block table, scratch) and forwards to it.
"""

from __future__ import annotations

import torch

from . import lib
from .lib import (KVQ_IN_BF16, KVQ_IN_F32, KVQ_Q4G32, KVQ_Q8G32, KVQ_TQ3_QJL, kv_cache_bytes,  # noqa: F401
                  kv_cache_init,
                  kv_calibrate, kv_calibrate_scratch_bytes, kv_decode_attention,
                  kv_decode_scratch_bytes, kv_qk_norm_rope, kv_quant_append, kv_rope_init, kv_status, kv_strerror,
                  make_config)


class QuantKVCache:
    """Device buffers of one cache, allocated with torch; all work runs in libkvq's kernels.

    Calls may run on several streams at once: what an operation needs besides its arguments is kept per operation and
    stream, one buffer that grows to the largest call so far.  A captured call takes memory of its graph's own, so that
    graphs may be replayed at the same time as each other and as calls.
    """

    def __init__(self, cfg: lib.kvq_config, device="cuda", block_table: torch.Tensor | None = None,
                 qjl_proj=None):
        self.cfg = cfg
        nbytes = kv_cache_bytes(cfg)
        if nbytes == 0:
            raise lib.KVQError("unsupported cache configuration")
        self.buffer = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.block_table = block_table
        self.handle = kv_cache_init(cfg, self.buffer, block_table, qjl_proj)
        self._work = {}    # (operation, stream) -> its buffer
        self._needs = {}   # (operation, sizes) -> bytes

    def _workspace(self, op: str, size, sizes: tuple, stream=None) -> torch.Tensor:
        """Uninitialised bytes for one call of ``op`` on ``stream``, at least size(handle, *sizes) (the layer first)."""
        key = (op, sizes[0] == -1) + sizes[1:]
        need = self._needs.get(key)
        if need is None:
            need = max(1, size(self.handle, *sizes))  # (no size: the call itself will be refused)
            self._needs[key] = need
        if stream is None:
            if torch.cuda.is_current_stream_capturing():
                return torch.empty(need, dtype=torch.uint8, device=self.buffer.device)
            raw = torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
        else:
            with torch.cuda.stream(stream):
                if torch.cuda.is_current_stream_capturing():
                    return torch.empty(need, dtype=torch.uint8, device=self.buffer.device)
            raw = stream.cuda_stream
        t = self._work.get((op, raw))
        if t is None or t.numel() < need:
            # allocated on the stream it is used on, so that the buffer it replaces is not handed out before its calls end
            with torch.cuda.stream(stream):
                t = torch.empty(need, dtype=torch.uint8, device=self.buffer.device)
            self._work[op, raw] = t
        return t

    def scratch(self, layer: int, batch: int, stream=None) -> torch.Tensor:
        """Decode scratch (uninitialised) for calls on ``stream`` (the current one), kept and reused by them."""
        return self._workspace("decode", kv_decode_scratch_bytes, (layer, batch), stream)

    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor, stream=None):
        kv_quant_append(self.handle, layer, k, v, pos, stream)

    def calibrate(self, layer: int, k_calib: torch.Tensor, v_calib: torch.Tensor, stream=None):
        need = kv_calibrate_scratch_bytes(self.handle, layer, k_calib.shape[-2])
        with torch.cuda.stream(stream):  # (given back to the stream that used it)
            work = torch.empty(need, dtype=torch.uint8, device=self.buffer.device)
        kv_calibrate(self.handle, layer, k_calib, v_calib, work, stream)

    def decode(self, layer: int, q: torch.Tensor, seq_lens: torch.Tensor, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
        if out is None:
            out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
        kv_decode_attention(self.handle, layer, q, out, seq_lens, self.scratch(layer, q.shape[-3], stream), stream)
        return out

    def prefill(self, layer: int, k: torch.Tensor, v: torch.Tensor, q: torch.Tensor, pos: torch.Tensor,
                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Append the chunk (k, v at pos) and return its queries' attention [L?][B][Hq][T][128]."""
        if out is None:
            out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
        t = self._workspace("prefill", lib.kv_prefill_scratch_bytes, (layer, q.shape[-4]), stream)
        lib.kv_prefill_attention(self.handle, layer, k, v, q, out, pos, t, stream)
        return out

    def tree_decode(self, layer: int, k: torch.Tensor, v: torch.Tensor, q: torch.Tensor, seq_lens: torch.Tensor,
                    parents: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Attention of a tree of drafted tokens (k, v, q; parents [B][N]) over the cache: [L?][B][Hq][N][128]."""
        if out is None:
            out = torch.empty_like(q)
        scratch = self._workspace("tree", lib.kv_tree_scratch_bytes, (layer, q.shape[-4], q.shape[-2]), stream)
        lib.kv_tree_attention(self.handle, layer, k, v, q, out, seq_lens, parents, scratch, stream)
        return out

    def commit(self, layer: int, k: torch.Tensor, v: torch.Tensor, path: torch.Tensor, n_accept: torch.Tensor,
               pos: torch.Tensor, stream=None):
        """Append the accepted path of each sequence's tree at pos (see lib.kv_tree_commit)."""
        lib.kv_tree_commit(self.handle, layer, k, v, path, n_accept, pos, stream)

    def attention_weights(self, layer: int, q: torch.Tensor, seq_lens: torch.Tensor, weights: torch.Tensor,
                          decay: float = 1.0, stream=None) -> torch.Tensor:
        """Add the attention weight that cached positions receive from the newest cached tokens' queries to ``weights``.

        q: [L?][B][Hq][T][128] of the T newest tokens of seq_lens, in order of position; ``weights`` holds zeros where a
        position has taken no weight yet.
        """
        scratch = self._workspace("weights", lib.kv_weights_scratch_bytes, (layer, q.shape[-4], q.shape[-2]), stream)
        lib.kv_attention_weights(self.handle, layer, q, weights, decay, seq_lens, scratch, stream)
        return weights

    def evict(self, layer: int, weights: torch.Tensor, seq_lens: torch.Tensor, budget: int, recent: int,
              kept: torch.Tensor | None = None, new_lens: torch.Tensor | None = None, stream=None):
        """Cut every sequence to ``budget`` positions by weight; returns (kept, new_lens).

        ``weights`` is compacted; set weights[..., budget:] to zero before tokens appended there take weight.
        """
        if kept is None:
            kept = torch.empty(tuple(weights.shape[:-1]) + (budget,), dtype=torch.int32, device=weights.device)
        if new_lens is None:
            new_lens = torch.empty_like(seq_lens)
        lib.kv_evict(self.handle, layer, weights, seq_lens, kept, new_lens, budget, recent, stream)
        return kept, new_lens

    def status(self) -> int:
        return kv_status(self.handle)

"""Definition of a KVQ_Q8B32 cache: raw vectors of every position, codes of finished blocks in float32 single operations,
attention in float64."""

from __future__ import annotations

import numpy as np
import torch

from kv_cache_quantization_append_gb300 import QuantKVCache, lib
from oracle import codec

from . import layout

B32, D = 32, 128


def encode(y: np.ndarray):
    """Blocks [...][32][128] of rotated (balanced) float32 vectors: codes int and the float scale."""
    amax = np.abs(y).max(axis=(-1, -2))
    d = (amax / np.float32(127.0)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        q = (y / d[..., None, None]).astype(np.float32)
        c = np.clip(np.rint(q), -127, 127)
    return np.where(d[..., None, None] > 0, c, 0).astype(np.int32), d


def offsets():
    """Byte offsets within a half-page of the codes of (token, channel), keys and values, as the header states them."""
    t, c = np.meshgrid(np.arange(B32), np.arange(D), indexing="ij")
    k = 512 * (4 * (t // 16) + c // 32) + 16 * (4 * (t % 8) + (c % 8) // 2) + 8 * (c // 16 % 2) + 4 * (c // 8 % 2) + 2 * (t // 8 % 2) + c % 2
    v = 4096 + 512 * (c // 16) + 16 * (4 * (c % 8) + (t % 8) // 2) + 8 * (t // 16) + 4 * (t // 8 % 2) + 2 * (c // 8 % 2) + t % 2
    return k, v


def make(n_layers, n_kv, n_q, max_batch, max_seq_len, window=128, sinkhorn=False, in_dtype="bf16", seed=0, n_pages=0, table=None):
    cfg = lib.make_config(n_layers, n_kv, n_q, max_batch, max_seq_len, window=window, n_pages=n_pages, k_format=lib.KVQ_Q8B32,
                          sinkhorn=sinkhorn, in_dtype=lib.KVQ_IN_BF16 if in_dtype == "bf16" else lib.KVQ_IN_F32, seed=seed)
    bt = None if table is None else torch.as_tensor(np.asarray(table), dtype=torch.int32).cuda().contiguous()
    return QuantKVCache(cfg, "cuda", bt), Reference(cfg)


class Reference:
    """raw[side][layer, b, h, position] of what has been appended; nothing else is state."""

    def __init__(self, cfg):
        self.cfg = cfg
        shape = (cfg.n_layers, cfg.max_batch, cfg.n_kv_heads, cfg.max_seq_len, D)
        self.raw = [np.zeros(shape, np.float32) for _ in range(2)]
        self.lens = np.zeros(cfg.max_batch, int)
        self.signs = codec.wht_signs(cfg.seed)
        self.sigma = [np.ones((cfg.n_layers, cfg.n_kv_heads, D), np.float32) for _ in range(2)]

    def append(self, layer, k, v, pos):
        T = k.shape[-2]
        layers = range(self.cfg.n_layers) if layer == -1 else [layer]
        for b, p in enumerate(pos):
            if p < 0 or p + T > self.cfg.max_seq_len:
                continue
            for i, lay in enumerate(layers):
                for side, x in enumerate((k, v)):
                    self.raw[side][lay, b, :, p:p + T] = x[i][b] if layer == -1 else x[b]
            self.lens[b] = p + T

    def fork(self, parents):
        raw, lens = [x.copy() for x in self.raw], self.lens.copy()
        for b, q in enumerate(parents):
            if 0 <= q < len(parents):
                for side in range(2):
                    self.raw[side][:, b] = raw[side][:, q]
                self.lens[b] = lens[q]

    def blocks(self, side, layer, b, h, n):
        """Codes [n][32][128] and scales [n] of the first n blocks."""
        x = self.raw[side][layer, b, h, :n * B32]
        y = codec.rotate(x, self.signs)
        s = self.sigma[side][layer, h]
        if self.cfg.sinkhorn:
            y = (y / s).astype(np.float32)
        return encode(y.reshape(n, B32, D))

    def records(self, side, layer, b, h, n):
        """What the records of the first n positions stand for, in the heads' space, float64 (finished blocks only)."""
        nb = -(-n // B32)
        if not nb:
            return np.zeros((0, D))
        c, d = self.blocks(side, layer, b, h, nb)
        y = (c.astype(np.float64) * d.astype(np.float64)[:, None, None]).reshape(-1, D)[:n]
        return codec.unrotate64(y * self.sigma[side][layer, h].astype(np.float64), self.signs)

    def attend(self, layer, b, j, q, L):
        """One query (head j) over L positions: the newest ``window`` raw, the others through records."""
        if L == 0:
            return np.zeros(D)
        h = j // (self.cfg.n_q_heads // self.cfg.n_kv_heads)
        m = max(0, L - self.cfg.window)
        k, v = (np.concatenate([self.records(side, layer, b, h, m), self.raw[side][layer, b, h, m:L].astype(np.float64)]) for side in range(2))
        lg = k @ q.astype(np.float64) / np.sqrt(128.0)
        p = np.exp(lg - lg.max())
        return p @ v / p.sum()

    def decode(self, layer, q, lens):
        return np.stack([np.stack([self.attend(layer, b, j, q[b, j], int(lens[b])) for j in range(q.shape[1])]) for b in range(q.shape[0])])


def stored(gpu, layer, b, h, n, table=None):
    """(codes, scale) of keys and of values of a unit's first n blocks, read from the buffer: two of ([n][32][128], [n])."""
    cfg, H = gpu.cfg, layout.H
    maxpps = -(-cfg.max_seq_len // 64)
    n_pages = cfg.n_pages or cfg.max_batch * maxpps
    if table is None:
        table = np.arange(cfg.max_batch * maxpps).reshape(cfg.max_batch, maxpps)
    total = lib.kv_cache_bytes(cfg)
    size = cfg.n_layers * n_pages * cfg.n_kv_heads * 2 * 8208
    off = total - -(-size // 256) * 256
    pages = gpu.buffer[off:off + size].view(cfg.n_layers, n_pages, cfg.n_kv_heads, 2, 8208)
    assert H == B32
    blk = np.arange(n)
    half = pages[layer, torch.as_tensor(table[b][blk // 2].astype(np.int64)).cuda(), h, torch.as_tensor(blk % 2).cuda()].cpu().numpy()
    d = half[:, 8192:8200].copy().view(np.float32)
    return [(half[:, o].astype(np.int32) - 128, d[:, i]) for i, o in enumerate(offsets())]


def ring(gpu, layer, b, h):
    cfg = gpu.cfg
    maxpps = -(-cfg.max_seq_len // 64)
    n_pages = cfg.n_pages or cfg.max_batch * maxpps
    a = lambda x: -(-x // 256) * 256  # noqa: E731
    n = cfg.n_layers * cfg.max_batch * cfg.n_kv_heads * cfg.window * D * 4
    v0 = lib.kv_cache_bytes(cfg) - a(cfg.n_layers * n_pages * cfg.n_kv_heads * 2 * 8208) - a(n)
    shape = (cfg.n_layers, cfg.max_batch, cfg.n_kv_heads, cfg.window, D)
    return [gpu.buffer[o:o + n].view(torch.float32).view(shape)[layer, b, h].cpu().numpy() for o in (v0 - a(n), v0)]


def check_state(gpu, ref, units, table=None):
    """Every finished block's bytes and every ring slot in use, of (layer, b, h) units, are the definition's."""
    W = gpu.cfg.window
    for layer, b, h in units:
        L = int(ref.lens[b])
        n = L // B32
        if n:
            got = stored(gpu, layer, b, h, n, table)
            for side in range(2):
                c, d = ref.blocks(side, layer, b, h, n)
                assert np.array_equal(got[side][1].view(np.uint32), d.view(np.uint32)), (layer, b, h, side)
                bad = np.argwhere(got[side][0] != c)
                assert not len(bad), (layer, b, h, side, bad[:4].tolist())
        at = np.arange(max(0, L - W), L)
        for side, r in enumerate(ring(gpu, layer, b, h)):
            assert np.array_equal(r[at % W], ref.raw[side][layer, b, h, at]), (layer, b, h, side)

"""Plain 64-bit definitions of the operators around append and decode, over an OracleCache (test helper)."""

from __future__ import annotations

import math

import numpy as np

from oracle import attention, codec

D = 128
NOT_THERE = -2


def random_tree(rng, n, chain=False):
    """Parents of a random tree of n nodes (-1: under the context)."""
    if chain:
        return np.arange(n, dtype=np.int32) - 1
    return np.array([rng.integers(-1, i) if i else -1 for i in range(n)], np.int32)


def chain_of(parents, i):
    """Node i and its ancestors, root first; empty where one of them is not there."""
    out = []
    while i >= 0:
        out.append(i)
        p = int(parents[i])
        if p < -1 or p >= i:
            return []
        i = p
    return out[::-1]


def record_logits(ora, layer, b, h, q, n):
    """q . k / sqrt(128) of queries [R][128] with the records of positions 0..n-1 (rotated space)."""
    qt = codec.rotate64(q, ora.signs)
    if ora.cfg.k_format == attention.TQ3_QJL:
        kk = {name: a[layer, b, h, :n] for name, a in ora.k.items()}
        lg = np.stack([codec.tq3_qjl_dot64(x, kk["code"], kk["bits"], kk["norm"], kk["gamma"], ora.proj) for x in qt])
    else:
        if ora.cfg.k_format == attention.Q8G32:
            kd = codec.q8g32_decode(ora.k["code"][layer, b, h, :n], ora.k["scale"][layer, b, h, :n])
        else:
            kd = codec.q4g32_decode(ora.k["code"][layer, b, h, :n], ora.k["scale"][layer, b, h, :n],
                                    ora.k["zero"][layer, b, h, :n])
        kd = kd.astype(np.float64)
        if ora.cfg.sinkhorn:
            kd = kd * ora.sigma_k[layer, h].astype(np.float64)
        lg = qt @ kd.T
    return lg / math.sqrt(D)


def record_values(ora, layer, b, h, n):
    """Values of the records of positions 0..n-1, in the heads' own space."""
    vd = codec.q4g32_decode(ora.v["code"][layer, b, h, :n], ora.v["scale"][layer, b, h, :n],
                            ora.v["zero"][layer, b, h, :n]).astype(np.float64)
    if ora.cfg.sinkhorn:
        vd = vd * ora.sigma_v[layer, h].astype(np.float64)
    return codec.unrotate64(vd, ora.signs)


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


def tree_attention(ora, layer, k, v, q, lens, parents):
    """k, v [B][H][N][128], q [B][Hq][N][128], lens [B], parents [B][N] -> [B][Hq][N][128]."""
    B, Hq, N, _ = q.shape
    g, W = ora.cfg.gqa, ora.cfg.window
    out = np.zeros(q.shape)
    for b in range(B):
        L = int(lens[b])
        for h in range(ora.cfg.n_kv_heads):
            qs = q[b, h * g:(h + 1) * g].astype(np.float64)
            vals = record_values(ora, layer, b, h, L) if L else np.zeros((0, D))
            lg = record_logits(ora, layer, b, h, qs.reshape(-1, D), L).reshape(g, N, L) if L else np.zeros((g, N, 0))
            for i in range(N):
                path = chain_of(parents[b], i)
                if not path:
                    continue
                P = L + len(path) - 1
                nrec = max(0, min(L, P - W + 1)) if W else L
                slots = np.arange(nrec, L) % max(W, 1)
                kr = np.concatenate([ora.ring_k[layer, b, h, slots], k[b, h, path]]).astype(np.float64)
                vr = np.concatenate([ora.ring_v[layer, b, h, slots], v[b, h, path]]).astype(np.float64)
                x = np.concatenate([lg[:, i, :nrec], qs[:, i] @ kr.T / math.sqrt(D)], 1)
                out[b, h * g:(h + 1) * g, i] = softmax(x) @ np.concatenate([vals[:nrec], vr])
    return out


def attention_weights(ora, layer, q, lens, before, decay):
    """q [B][Hq][T][128], before [B][H][S] -> the weights after the call, float64."""
    B, Hq, T, _ = q.shape
    g, W = ora.cfg.gqa, ora.cfg.window
    out = before.astype(np.float64).copy()
    for b in range(B):
        L = int(lens[b])
        for h in range(ora.cfg.n_kv_heads):
            if not L:
                continue
            qs = q[b, h * g:(h + 1) * g].astype(np.float64).reshape(-1, D)
            lg = record_logits(ora, layer, b, h, qs, L)
            n = max(0, L - W)
            if W:
                lg[:, n:] = qs @ ora.ring_k[layer, b, h, np.arange(n, L) % W].astype(np.float64).T / math.sqrt(D)
            got = np.zeros(L)
            for r in range(g * T):
                P = L - T + r % T
                if P >= 0:
                    got[:P + 1] += softmax(lg[r, :P + 1])
            out[b, h, :L] = got + (decay * out[b, h, :L] if decay else 0.0)
    return out


def kept_positions(w, L, budget, recent):
    """Positions that one unit keeps, ascending."""
    if L <= budget:
        return np.arange(L)
    old = L - recent
    x = w[:old].astype(np.float64)
    # last key first: by weight descending (NaN last), then by position
    order = np.lexsort((np.arange(old), -np.where(np.isnan(x), -np.inf, x), np.isnan(x)))
    return np.concatenate([np.sort(order[:budget - recent]), np.arange(old, L)])


def evict(ora, weights, lens, budget, recent):
    """Cuts the oracle cache in place; weights [L][B][H][S] (float32, compacted in place).  Returns kept [L][B][H][budget]."""
    cfg = ora.cfg
    kept = np.full(weights.shape[:3] + (budget,), -1, np.int32)
    for layer in range(weights.shape[0]):
        for b in range(weights.shape[1]):
            L = int(lens[b])
            for h in range(cfg.n_kv_heads):
                src = kept_positions(weights[layer, b, h], L, budget, recent)
                n = len(src)
                kept[layer, b, h, :n] = src
                if L <= budget:
                    continue
                for store in (ora.k, ora.v):
                    for a in store.values():
                        a[layer, b, h, :n] = a[layer, b, h, src].copy()
                weights[layer, b, h, :n] = weights[layer, b, h, src].copy()
                W = cfg.window
                if W:
                    new = np.arange(n - W, n)
                    old = new + (L - n)
                    for ring in (ora.ring_k, ora.ring_v):
                        ring[layer, b, h, new % W] = ring[layer, b, h, old % W].copy()
    return kept


def frequencies(rot, theta, scaling, factor, n0, low, high):
    """Radians per position of each pair (scalings 0..4 as in include/kvq.h), by scalar arithmetic."""
    if scaling == 2:
        theta = theta * factor ** (rot / (rot - 2))
    out = []
    for i in range(rot // 2):
        f = theta ** (-2 * i / rot)
        if scaling == 1:
            f /= factor
        elif scaling in (3, 4):
            if scaling == 3:
                keep = (n0 * f / (2 * math.pi) - low) / (high - low)
            else:
                dim = lambda r: rot * math.log(n0 / (r * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
                a, b = max(math.floor(dim(high)), 0), min(math.ceil(dim(low)), rot - 1)
                keep = 1 - min(1.0, max(0.0, (i - a) / max(b - a, 0.001)))
            keep = min(1.0, max(0.0, keep))
            f = keep * f + (1 - keep) * f / factor
        out.append(f)
    return np.array(out)


def norm_rope(x, pos, w, eps, rot, interleaved, freq, attn):
    """x [B][H][T][128] float64, pos [B][T] -> normalised (where w is given) and rotated."""
    y = x.copy()
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * w
    ang = pos[:, None, :, None].astype(np.float64) * freq
    c, s = attn * np.cos(ang), attn * np.sin(ang)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    ya, yb = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = ya * c - yb * s, yb * c + ya * s
    return y

"""The operators around append and decode, as measured cases: rows of a fused projection to normalised, rotated
queries and keys (kv_qk_norm_rope), attention of a tree of drafted tokens over the quantised cache
(kv_tree_attention), the accepted path's append (kv_tree_commit), the attention weight that cached positions
receive (kv_attention_weights) and eviction by it (kv_evict).

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU from a seed, ``run`` does one pass: in
plain torch operations where ``own`` is false, through the package where it is true.  The cache's contents are
packed here, from the buffer layout that include/kvq.h documents: the same bytes for both.
"""

import math

import numpy as np
import torch

own = False

D = 128
PAGE, HALF = 64, 32
DEV = "cuda"
FMT = {"q4": 1, "tq3": 3, "q8": 4}               # KVQ_Q4G32, KVQ_TQ3_QJL, KVQ_Q8G32
K_MAIN = {"q4": 64, "tq3": 64, "q8": 128}        # key bytes per token
K_META = {"q4": 16, "tq3": 4, "q8": 8}           # bytes of key scales or norms per token
QJL = math.sqrt(math.pi / 2) / 128
C_WHT = float(np.float32(1 / math.sqrt(128)))
SQRT_D = math.sqrt(128.0)


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of eight sequences far into their contexts, half of each head rotated: latency counts
        dict(name="rope step b8", op="rope", batch=8, tokens=1, hq=32, hkv=8, dtype="bf16", layout="interleaved",
             rot=64, scaling="dims", norm=True, start=120000),
        # a prompt of 8192 tokens: bandwidth counts
        dict(name="rope prompt 8192", op="rope", batch=1, tokens=8192, hq=32, hkv=8, dtype="bf16", layout="half",
             rot=128, scaling="turns", norm=True, start=0),
        # a short chat with a handful of drafts: latency
        dict(name="tree 5 at 700", op="tree", batch=1, seq=700, spread=0.0, hq=24, hkv=8, nodes=5, fmt="q4",
             window=128),
        # one long context, a usual tree
        dict(name="tree 16 at 32K", op="tree", batch=1, seq=32768, spread=0.0, hq=24, hkv=8, nodes=16, fmt="q4",
             window=128),
        # eight long ragged contexts with 3-bit keys
        dict(name="tree 32 at 8x32K tq3", op="tree", batch=8, seq=32768, spread=0.6, hq=32, hkv=8, nodes=32,
             fmt="tq3", window=128),
        # a wide tree over 8-bit keys, odd lengths
        dict(name="tree 64 at 4x9001 q8", op="tree", batch=4, seq=9001, spread=0.5, hq=24, hkv=8, nodes=64, fmt="q8",
             window=128),
        # the accepted paths of one layer, and of a whole model in one call
        dict(name="commit layer", op="commit", layers=1, batch=8, seq=512, hq=32, hkv=8, nodes=32, path=6, fmt="q4",
             window=128),
        dict(name="commit 28 layers", op="commit", layers=28, batch=4, seq=320, hq=24, hkv=8, nodes=16, path=5,
             fmt="q8", window=128),
        # weights of a decode step's queries, accumulated; of a prompt's last 32 queries, written
        dict(name="weights step 8x16K", op="weights", batch=8, seq=16384, spread=0.5, hq=32, hkv=8, queries=1,
             fmt="q4", window=128, decay=1.0),
        dict(name="weights 32 at 32K q8", op="weights", batch=1, seq=32768, spread=0.0, hq=24, hkv=8, queries=32,
             fmt="q8", window=128, decay=0.0),
        # eight layers of a long prompt cut to a quarter
        dict(name="evict 32K to 8K", op="evict", layers=8, batch=1, seq=32768, spread=0.0, hq=24, hkv=8, budget=8192,
             recent=256, fmt="q4", window=128),
        # one layer of a ragged batch, its last sequences already within the budget
        dict(name="evict 8K to 2K ragged", op="evict", layers=1, batch=4, seq=8192, spread=0.95, hq=32, hkv=8,
             budget=2048, recent=128, fmt="q4", window=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "tree", "tree", "commit", "weights", "evict"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4])
    window = rng.choice([0, 4, 64, 100, 128])
    if op == "rope":
        rot = rng.choice([128, 128, 64, 32, 96, 2 * rng.randint(2, 64)])
        return dict(op=op, batch=rng.randint(1, 8), tokens=_log(rng, 1, 900), hq=hq, hkv=hkv,
                    dtype=rng.choice(["bf16", "f32"]), layout=rng.choice(["half", "interleaved"]), rot=rot,
                    scaling=rng.choice(["none", "linear", "ntk", "turns", "dims"]), norm=rng.random() < 0.6,
                    start=_log(rng, 1, 200000) - 1)
    if op == "tree":
        return dict(op=op, batch=rng.randint(1, 6), seq=_log(rng, 1, 30000), spread=rng.choice([0.0, 0.5, 0.99]), hq=hq,
                    hkv=hkv, nodes=_log(rng, 1, 64), fmt=rng.choice(["q4", "q8", "tq3"]), window=window)
    if op == "commit":
        nodes = _log(rng, 1, 64)
        return dict(op=op, layers=_log(rng, 1, 12), batch=rng.randint(1, 8), seq=_log(rng, 80, 400), hq=hq, hkv=hkv,
                    nodes=nodes, path=min(nodes, rng.randint(1, 9)), fmt=rng.choice(["q4", "q8"]), window=window)
    if op == "weights":
        return dict(op=op, batch=rng.randint(1, 6), seq=_log(rng, 1, 16000), spread=rng.choice([0.0, 0.5, 0.99]), hq=hq,
                    hkv=hkv, queries=_log(rng, 1, 64), fmt=rng.choice(["q4", "q8", "tq3"]), window=window,
                    decay=rng.choice([0.0, 0.9, 1.0]))
    seq = _log(rng, 300, 12000)
    budget = rng.randint(140, seq)
    return dict(op=op, layers=rng.randint(1, 4), batch=rng.randint(1, 4), seq=seq, spread=rng.choice([0.0, 0.5, 0.99]),
                hq=hq, hkv=hkv, budget=budget, recent=rng.randint(max(window, 1), budget),
                fmt=rng.choice(["q4", "q8", "tq3"]), window=window)


def _lens(c):
    """Cached tokens of each sequence: ``seq`` down to (1 - spread) of it."""
    return [max(1, int(round(c["seq"] * (1 - c["spread"] * b / max(1, c["batch"] - 1))))) for b in range(c["batch"])]


def _rec(fmt):
    return K_MAIN[fmt] + K_META[fmt] + 64 + 16


def work(c):
    """Bytes: each input read once, each output written once.  Operations: the products of the formulas."""
    if c["op"] == "rope":
        e = 2 if c["dtype"] == "bf16" else 4
        vals = c["batch"] * c["tokens"] * (c["hq"] + 2 * c["hkv"]) * D
        return {"bytes": 2 * vals * e + 4 * c["batch"] * c["tokens"], "flops": 8 * vals}
    W, hkv, hq, fmt = c["window"], c["hkv"], c["hq"], c["fmt"]
    if c["op"] == "commit":
        vec = c["layers"] * c["batch"] * hkv * max(1, c["path"] // 2)
        return {"bytes": vec * (2 * D * 2 + _rec(fmt) + (2 * D * 4 if W else 0)), "flops": vec * 2 * (7 * D + 8 * D)}
    lens = _lens(c)
    quant = sum(max(0, n - W) for n in lens)
    raw = sum(lens) - quant
    if c["op"] == "tree":
        n = c["nodes"]
        return {"bytes": hkv * (quant * _rec(fmt) + raw * 2 * D * 4) + c["batch"] * n * D * 2 * (2 * hq + 2 * hkv),
                "flops": 4 * D * hq * n * (sum(lens) + c["batch"] * n / 2)}
    if c["op"] == "weights":
        t = c["queries"]
        k = K_MAIN[fmt] + K_META[fmt]
        return {"bytes": hkv * (quant * k + raw * D * 4 + sum(lens) * (8 if c["decay"] else 4)) + c["batch"] * t * hq * D * 2,
                "flops": 2 * D * hq * t * sum(lens)}
    cut = [n for n in lens if n > c["budget"]]
    moved = c["layers"] * hkv * len(cut) * c["budget"]
    return {"bytes": c["layers"] * hkv * 4 * sum(lens) + moved * (2 * _rec(fmt) + 12), "flops": 2 * c["layers"] * hkv * sum(lens)}


# ---------------------------------------------------------------------------- the cache's layout and codecs
def _signs():
    """SplitMix64 of seed 0: sign j is -1 where bit 0 of output j + 1 is set."""
    m = (1 << 64) - 1

    def out(j):
        z = ((j + 1) * 0x9E3779B97F4A7C15) & m
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & m
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & m
        return z ^ (z >> 31)

    return torch.tensor([-1.0 if out(j) & 1 else 1.0 for j in range(D)], device=DEV)


def _centroids():
    """The 8-level quantiser of least mean square error of N(0, 1/128), to fp16."""
    phi = lambda x: math.exp(-x * x / 2) / math.sqrt(2 * math.pi)  # noqa: E731
    cdf = lambda x: math.erfc(-x / math.sqrt(2)) / 2  # noqa: E731
    c = [-2 + 4 * k / 7 for k in range(8)]
    for _ in range(3000):
        e = [-40.0] + [(c[k] + c[k + 1]) / 2 for k in range(7)] + [40.0]
        c = [(phi(e[k]) - phi(e[k + 1])) / (cdf(e[k + 1]) - cdf(e[k])) for k in range(8)]
    return torch.tensor(c, dtype=torch.float64).div(SQRT_D).half().to(DEV)


def _stage(x, h):
    v = x.reshape(*x.shape[:-1], D // (2 * h), 2, h)
    a, b = v[..., 0, :], v[..., 1, :]
    return torch.stack((a + b, a - b), -2).reshape(x.shape)


def _rotate(x, signs):
    """c H (s . x): butterflies of 1, 2, ..., 64, each sum rounded once, then one product by c."""
    y = _stage(_stage(_stage(x * signs, 1), 2), 4)
    return _stage(_stage(_stage(_stage(y, 8), 16), 32), 64) * C_WHT


def _unrotate(y, signs):
    y = _stage(_stage(_stage(y, 1), 2), 4)
    return _stage(_stage(_stage(_stage(y, 8), 16), 32), 64) * C_WHT * signs


def _q4(y):
    g = y.reshape(*y.shape[:-1], 4, 32)
    mn, mx = g.amin(-1), g.amax(-1)
    scale = ((mx - mn) / torch.full_like(mn, 15.0)).half()
    zero = mn.half()
    s = scale.float()[..., None]
    code = torch.where(s > 0, ((g - zero.float()[..., None]) / s).round().clamp(0, 15), torch.zeros_like(g))
    return code.reshape(y.shape).to(torch.uint8), scale, zero


def _q8(y):
    g = y.reshape(*y.shape[:-1], 4, 32)
    d = (g.abs().amax(-1) / torch.full_like(g[..., 0], 127.0)).half()
    s = d.float()[..., None]
    code = torch.where(s > 0, (g / s).round().clamp(-127, 127), torch.zeros_like(g))
    return (code.reshape(y.shape) + 128).to(torch.uint8), d


def _bytes_of(*halves):
    return torch.cat([h.contiguous().view(torch.uint8) for h in halves], -1)


def _pairs(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _encode(k, v, fmt, signs, cent, proj):
    """Records of key and value vectors [...][128] as bytes in channel order: keys, key scales, values, value scales."""
    y = _rotate(k, signs)
    if fmt == "q4":
        c, s, z = _q4(y)
        key = [_pairs(c), _bytes_of(s, z)]
    elif fmt == "q8":
        c, s = _q8(y)
        key = [c, _bytes_of(s)]
    else:
        n = y.norm(dim=-1)
        u = y / n.clamp_min(1e-30)[..., None]
        cf = cent.float()
        code = torch.bucketize(u, (cf[:-1] + cf[1:]) / 2, right=True)
        r = u - cf[code]
        bit = (r @ proj.t() >= 0).to(torch.uint8)
        code = code.to(torch.uint8)
        key = [_pairs3(code, bit), _bytes_of(n.half()[..., None], r.norm(dim=-1).half()[..., None])]
    c, s, z = _q4(_rotate(v, signs))
    return torch.cat(key + [_pairs(c), _bytes_of(s, z)], -1)


def _pairs3(code, bit):
    return code[..., 0::2] | (code[..., 1::2] << 3) | (bit[..., 0::2] << 6) | (bit[..., 1::2] << 7)


def _address(fmt):
    """Byte offsets within a half-page of 32 tokens of each token's record bytes (in _encode's order): [32][record]."""
    t = np.arange(HALF)[:, None]
    j = np.arange(64)[None, :]
    if fmt == "q4":
        k = 64 * t + 16 * ((j % 16) // 4) + 4 * (j // 16) + j % 4
    elif fmt == "tq3":
        k = 64 * t + j
    else:
        c = np.arange(128)[None, :]
        kk, w = c >> 4, c & 15
        m = 2 * ((w & 7) >> 1) + (kk >> 2)
        k = 128 * t + 16 * (m ^ (t & 1)) + 4 * (kk & 3) + (w & 1) + 2 * (w >> 3)
    o_v = K_MAIN[fmt] * HALF
    p, r = t // 2, (j % 16) // 2
    v = o_v + 128 * p + 16 * ((r + 2 * (p & 3)) & 7) + 4 * (j // 16) + t % 2 + 2 * (j % 2)
    o_m = o_v + 64 * HALF
    e = np.arange(K_META[fmt])[None, :]
    km = o_m + (e // 2) * 64 + 2 * t + e % 2 if fmt == "tq3" else o_m + K_META[fmt] * t + e
    o_s = o_m + K_META[fmt] * HALF
    e = np.arange(16)[None, :]
    vm = o_s + (e // 2) * 64 + 2 * t + e % 2
    return torch.as_tensor(np.concatenate([k, km, v, vm], 1), dtype=torch.int64, device=DEV)


def _half_bytes(fmt):
    return HALF * _rec(fmt)


def _records(s, n):
    """Records of the first n positions (rounded up to pages) of every sequence: [layers][batch][heads][positions][record]."""
    pages, bt, addr = s["pages"], s["bt"], s["addr"]
    lp = -(-n // PAGE)
    b = bt.shape[0]
    got = pages[:, bt[:, :lp].long()]                                         # [L][B][lp][H][page]
    got = got.reshape(pages.shape[0], b, lp, pages.shape[2], 2, -1)[..., addr]  # [L][B][lp][H][2][32][rec]
    return got.permute(0, 1, 3, 2, 4, 5, 6).reshape(pages.shape[0], b, pages.shape[2], lp * PAGE, -1)


def _store(s, rec, pos, keep):
    """Writes records [L][B][H][T][rec] at positions pos [L or 1][B][H or 1][T] where keep (same shape) is true."""
    pages, bt, addr = s["pages"], s["bt"], s["addr"]
    L, n_pages, H, size = pages.shape
    B, T = rec.shape[1], rec.shape[3]
    keep = keep.expand(L, B, H, T)
    pos = pos.expand(L, B, H, T)
    lay, b, h, t = torch.nonzero(keep, as_tuple=True)
    p = pos[lay, b, h, t]
    phys = bt[b, p // PAGE].long()
    base = ((lay * n_pages + phys) * H + h) * size + ((p % PAGE) // HALF) * (size // 2)
    pages.view(-1)[base[:, None] + addr[p % HALF]] = rec[lay, b, h, t]


def _nibbles(b):
    return torch.stack((b & 15, b >> 4), -1).reshape(*b.shape[:-1], D)


def _half_values(b):
    return b.contiguous().view(torch.float16)


def _affine(code, meta, kind):
    sz = _half_values(meta).to(kind)
    c = code.to(kind).reshape(*code.shape[:-1], 4, 32)
    return (sz[..., 4:, None] + sz[..., :4, None] * c).reshape(code.shape)


def _split(rec, fmt):
    a, m = K_MAIN[fmt], K_META[fmt]
    return rec[..., :a], rec[..., a:a + m], rec[..., a + m:a + m + 64], rec[..., a + m + 64:]


def _values(rec, fmt, kind):
    _, _, v, vm = _split(rec, fmt)
    return _affine(_nibbles(v), vm, kind)


def _key_logits(q, rec, s, fmt, kind):
    """q~ . k of rotated queries [..][R][128] with the records' keys [..][S][128], in the formats' own terms."""
    k, km, _, _ = _split(rec, fmt)
    if fmt == "q4":
        return q @ _affine(_nibbles(k), km, kind).transpose(-1, -2)
    if fmt == "q8":
        d = _half_values(km).to(kind)
        c = (k.to(kind) - 128).reshape(*k.shape[:-1], 4, 32)
        return q @ (d[..., None] * c).reshape(k.shape).transpose(-1, -2)
    code = torch.stack((k & 7, (k >> 3) & 7), -1).reshape(*k.shape[:-1], D)
    bit = torch.stack(((k >> 6) & 1, k >> 7), -1).reshape(*k.shape[:-1], D)
    ng = _half_values(km).to(kind)
    dot = q @ s["cent"].to(kind)[code.long()].transpose(-1, -2)
    sgn = (q @ s["proj"].to(kind).t()) @ (2 * bit.to(kind) - 1).transpose(-1, -2)
    return ng[..., None, :, 0] * (dot + QJL * ng[..., None, :, 1] * sgn)


# ---------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _heads(g, *shape):
    """Gaussian key or value vectors with three louder channels, as attention heads have."""
    x = torch.randn(*shape, D, generator=g, device=DEV)
    x[..., [5, 70, 101]] *= 6
    return x


def _cache(c, g, layers, max_len, store=True):
    """A paged cache of ``batch`` sequences in a shuffled pool of pages, filled for max_len positions."""
    B, H, W, fmt = c["batch"], c["hkv"], c["window"], c["fmt"]
    mpp = -(-max_len // PAGE)
    n_pages = B * mpp + 3
    s = {"signs": _signs(), "cent": _centroids(), "addr": _address(fmt), "proj": torch.randn(D, D, generator=g, device=DEV)}
    s["bt"] = torch.randperm(n_pages, generator=g, device=DEV)[:B * mpp].reshape(B, mpp).int().contiguous()
    size = 2 * _half_bytes(fmt)
    shape, ring = (layers, n_pages, H, size), (layers, B, H, W, D)
    if own:
        from kv_cache_quantization_append_gb300 import QuantKVCache, lib

        cfg = lib.make_config(layers, H, c["hq"], B, max_len, window=W, n_pages=n_pages, k_format=FMT[fmt])
        s["cache"] = cache = QuantKVCache(cfg, DEV, s["bt"], s["proj"].cpu().numpy())
        nb = layers * n_pages * H * size
        end = cache.buffer.numel() // 256 * 256
        off = lib.kv_cache_bytes(cfg) - (-(-nb // 256) * 256)
        rb = -(-(layers * B * H * W * D * 4) // 256) * 256
        assert off > 0 and off + nb <= end
        s["pages"] = cache.buffer[off:off + nb].view(shape)
        nf = layers * B * H * W * D * 4
        s["ring_v"] = cache.buffer[off - rb:off - rb + nf].view(torch.float32).view(ring)
        s["ring_k"] = cache.buffer[off - 2 * rb:off - 2 * rb + nf].view(torch.float32).view(ring)
        s["pages"].zero_()
    else:
        s["pages"] = torch.zeros(shape, dtype=torch.uint8, device=DEV)
        s["ring_k"], s["ring_v"] = (torch.empty(ring, device=DEV) for _ in range(2))
    s["ring_k"].copy_(_heads(g, *ring[:-1]))
    s["ring_v"].copy_(_heads(g, *ring[:-1]))
    for lay in range(layers):
        for lo in range(0, mpp, 128):
            n = min(128, mpp - lo)
            k, v = _heads(g, B, H, n * PAGE), _heads(g, B, H, n * PAGE)
            rec = _encode(k, v, fmt, s["signs"], s["cent"], s["proj"])     # [B][H][n * 64][rec]
            half = torch.empty(B, H, n, 2, size // 2, dtype=torch.uint8, device=DEV)
            half[..., s["addr"]] = rec.reshape(B, H, n, 2, HALF, -1)
            s["pages"][lay][s["bt"][:, lo:lo + n].long()] = half.permute(0, 2, 1, 3, 4).reshape(B, n, H, size)
    return s


def _scaling(c):
    """(theta, scaling, factor, original length, low, high, attention factor) of a case's positions."""
    return {"none": (500000.0, 0, 1.0, 0.0, 0.0, 0.0, 1.0), "linear": (10000.0, 1, 4.0, 0.0, 0.0, 0.0, 1.0),
            "ntk": (10000.0, 2, 8.0, 0.0, 0.0, 0.0, 1.0), "turns": (500000.0, 3, 8.0, 8192.0, 1.0, 4.0, 1.0),
            "dims": (10000.0, 4, 16.0, 4096.0, 1.0, 32.0, 0.1 * math.log(16.0) + 1)}[c["scaling"]]


def _tree(c, g):
    """Parents [batch][nodes]: -1 under the cached context, -2 a node that is not there (a shorter draft in the batch)."""
    B, n = c["batch"], c["nodes"]
    u = torch.rand(B, n, generator=g, device=DEV)
    par = (u * (torch.arange(n, device=DEV) + 1)).floor().int() - 1
    gone = torch.arange(n, device=DEV)[None, :] >= n - (torch.arange(B, device=DEV)[:, None] % 3) * (n // 8)
    return torch.where(gone, torch.full_like(par, -2), par).contiguous()


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    B, hq, hkv = c["batch"], c["hq"], c["hkv"]
    if c["op"] == "rope":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        T = c["tokens"]
        s = {"c": c, "x": torch.randn(B, T, (hq + 2 * hkv) * D, generator=g, device=DEV).to(dt)}
        first = c["start"] + torch.randint(0, 64, (B, 1), generator=g, device=DEV)
        s["pos"] = (first + torch.arange(T, device=DEV)).int().contiguous()
        s["wq"], s["wk"] = ((1 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(dt) if c["norm"] else None for _ in range(2))
        if own:
            from kv_cache_quantization_append_gb300 import lib

            th, kind, fac, n0, lo, hi, att = _scaling(c)
            s["rope"] = lib.kv_rope_init(c["rot"], layout=int(c["layout"] == "interleaved"), theta=th, scaling=kind,
                                         factor=fac, original_len=n0, low=lo, high=hi, attn_factor=att)
            s["q"] = torch.empty(B, hq, T, D, dtype=dt, device=DEV)
            s["k"], s["v"] = (torch.empty(B, hkv, T, D, dtype=dt, device=DEV) for _ in range(2))
        return s
    lens = torch.tensor(_lens(c) if "spread" in c else [c["seq"]] * B, dtype=torch.int32, device=DEV)
    bf = torch.bfloat16
    if c["op"] == "commit":
        s = _cache(c, g, c["layers"], c["seq"])
        s["k"], s["v"] = (_heads(g, c["layers"], B, hkv, c["nodes"]).to(bf) for _ in range(2))
        s["path"] = torch.rand(B, c["nodes"], generator=g, device=DEV).argsort(1)[:, :c["path"]].sort(1).values.int().contiguous()
        s["accepted"] = torch.randint(0, c["path"] + 1, (B,), generator=g, device=DEV).int()
        s["accepted"][0] = c["path"]
        s["pos"] = torch.randint(0, c["seq"] - c["path"] + 1, (B,), generator=g, device=DEV).int()
        s["c"] = c
        return s
    layers = c.get("layers", 1)
    s = _cache(c, g, layers, c["seq"])
    s["c"], s["lens"] = c, lens
    if c["op"] == "tree":
        n = c["nodes"]
        s["q"] = torch.randn(B, hq, n, D, generator=g, device=DEV).to(bf)
        s["k"], s["v"] = (_heads(g, B, hkv, n).to(bf) for _ in range(2))
        s["parents"] = _tree(c, g)
        s["out"] = torch.empty(B, hq, n, D, dtype=bf, device=DEV)
    elif c["op"] == "weights":
        s["q"] = torch.randn(B, hq, c["queries"], D, generator=g, device=DEV).to(bf)
        s["weights"] = torch.rand(B, hkv, c["seq"], generator=g, device=DEV) * 0.005   # what a few steps left
        s["before"] = s["weights"].clone()
    else:
        # accumulated weights are skewed: a few positions hold most of the mass, many are equal at zero
        u = torch.rand(layers, B, hkv, c["seq"], generator=g, device=DEV)
        s["weights"] = torch.where(u < 0.1, torch.zeros_like(u), (u * 8).exp() / 3000)
        s["kept"] = torch.empty(layers, B, hkv, c["budget"], dtype=torch.int32, device=DEV)
        s["new_lens"] = torch.empty(B, dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------------------- one pass
def run(s):
    return {"rope": _run_rope, "tree": _run_tree, "commit": _run_commit, "weights": _run_weights,
            "evict": _run_evict}[s["c"]["op"]](s)


def _frequencies(c):
    """Radians per position of each pair, in 64 bits."""
    th, kind, fac, n0, lo, hi, _ = _scaling(c)
    rot = c["rot"]
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    if kind == 2:
        th = th * fac ** (rot / (rot - 2))
    f = torch.exp(-math.log(th) * 2 * i / rot)
    if kind == 1:
        return f / fac
    if kind == 3:
        keep = ((n0 * f / (2 * math.pi) - lo) / (hi - lo)).clamp(0, 1)
    elif kind == 4:
        at = lambda turns: rot * math.log(n0 / (turns * 2 * math.pi)) / (2 * math.log(th))  # noqa: E731
        first, last = max(math.floor(at(hi)), 0), min(math.ceil(at(lo)), rot - 1)
        keep = 1 - ((i - first) / max(last - first, 0.001)).clamp(0, 1)
    else:
        return f
    return f * keep + f / fac * (1 - keep)


def _run_rope(s):
    c = s["c"]
    B, T, hq, hkv, rot = c["batch"], c["tokens"], c["hq"], c["hkv"], c["rot"]
    if own:
        from kv_cache_quantization_append_gb300 import lib

        lib.kv_qk_norm_rope(s["rope"], s["x"], s["pos"], s["q"], s["k"], s["v"], q_weight=s["wq"], k_weight=s["wk"], eps=1e-6)
        return {"q": s["q"], "k": s["k"], "v": s["v"]}
    x = s["x"].float().view(B, T, hq + 2 * hkv, D).transpose(1, 2)
    ang = s["pos"].double()[:, None, :, None] * _frequencies(c)
    att = _scaling(c)[-1]
    cos, sin = (ang.cos() * att).float(), (ang.sin() * att).float()

    def head(y, w):
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
        r = y[..., :rot]
        if c["layout"] == "half":
            a, b = r[..., :rot // 2], r[..., rot // 2:]
            r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        else:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        return torch.cat((r, y[..., rot:]), -1).to(s["x"].dtype)

    return {"q": head(x[:, :hq], s["wq"]), "k": head(x[:, hq:hq + hkv], s["wk"]), "v": x[:, hq + hkv:].to(s["x"].dtype)}


def _ring_positions(lens, W):
    """Position that each ring slot holds of sequences of these lengths (negative: none)."""
    last = lens.long()[:, None] - 1
    slot = torch.arange(W, device=DEV)[None, :]
    return last - (last - slot) % max(W, 1)


def _ancestors(parents):
    """Ancestor-or-self of every node, and its depth (-1: not there): squarings of the parent relation."""
    n = parents.shape[1]
    here = parents >= -1
    rel = torch.zeros(parents.shape[0], n, n + 1, device=DEV)
    rel.scatter_(2, parents.clamp_min(-1).long()[..., None] % (n + 1), here.float()[..., None])
    a = rel[..., :n] + torch.eye(n, device=DEV)
    a = ((a @ a) > 0).float()
    a = ((a @ a) > 0).float()
    a = ((a @ a) > 0).float()
    a = ((a @ a) > 0).float()
    a = ((a @ a) > 0).float()
    a = ((a @ a) > 0) & here[:, :, None]
    return a, a.sum(-1) - 1


def _softmax(x):
    m = x.amax(-1, keepdim=True)
    p = (x - torch.where(m == -math.inf, torch.zeros_like(m), m)).exp()
    return p / p.sum(-1, keepdim=True).clamp_min(1e-300 if x.dtype == torch.float64 else 1e-38)


def _tree_masks(c, lens, parents, n_rec):
    """Which records, ring slots and drafts each node attends to: [batch][nodes][...]."""
    W = c["window"]
    anc, depth = _ancestors(parents)
    here = (parents >= -1)[:, :, None]
    at = (lens.long()[:, None] + depth)[:, :, None]
    j = torch.arange(n_rec, device=DEV)
    rec = here & (j < lens.long()[:, None, None]) & (j <= at - W if W else torch.ones_like(here))
    rp = _ring_positions(lens, W)[:, None, :]
    return rec, here & (rp >= 0) & (rp > at - W), anc


def _run_tree(s):
    c = s["c"]
    if own:
        return s["cache"].tree_decode(0, s["k"], s["v"], s["q"], s["lens"], s["parents"], out=s["out"])
    B, hq, hkv, n, W, fmt = c["batch"], c["hq"], c["hkv"], c["nodes"], c["window"], c["fmt"]
    g = hq // hkv
    rec = _records(s, c["seq"])[0]                                            # [B][H][S][rec]
    q = s["q"].float().view(B, hkv, g * n, D)
    k, v = s["k"].float(), s["v"].float()
    lg = torch.cat((_key_logits(_rotate(q, s["signs"]), rec, s, fmt, torch.float32),
                    q @ s["ring_k"][0].transpose(-1, -2), q @ k.transpose(-1, -2)), -1) / SQRT_D
    m = torch.cat(_tree_masks(c, s["lens"], s["parents"], rec.shape[2]), -1)
    m = m[:, None, None].expand(B, hkv, g, n, m.shape[-1]).reshape(lg.shape)
    p = _softmax(lg.masked_fill(~m, -math.inf))
    S = rec.shape[2]
    o = _unrotate(p[..., :S] @ _values(rec, fmt, torch.float32), s["signs"])
    o = o + p[..., S:S + W] @ s["ring_v"][0] + p[..., S + W:] @ v
    return o.reshape(B, hq, n, D).to(s["q"].dtype)


def _run_commit(s):
    c = s["c"]
    if own:
        s["cache"].commit(-1, s["k"], s["v"], s["path"], s["accepted"], s["pos"])
        return {"pages": s["pages"], "ring_k": s["ring_k"], "ring_v": s["ring_v"]}
    L, B, H, W, T = c["layers"], c["batch"], c["hkv"], c["window"], c["path"]
    at = s["path"].long()[None, :, None, :, None].expand(L, B, H, T, D)
    k, v = s["k"].float().gather(3, at), s["v"].float().gather(3, at)
    t = torch.arange(T, device=DEV)[None, None, None, :]
    acc = s["accepted"].long()[None, :, None, None]
    pos = s["pos"].long()[None, :, None, None] + t
    keep = (t < acc).expand(1, B, 1, T)
    _store(s, _encode(k, v, c["fmt"], s["signs"], s["cent"], s["proj"]), pos, keep)
    if W:
        b, j = torch.nonzero((keep & (t >= acc - W))[0, :, 0], as_tuple=True)
        slot = pos[0, b, 0, j] % W
        s["ring_k"][:, b, :, slot] = k[:, b, :, j]
        s["ring_v"][:, b, :, slot] = v[:, b, :, j]
    return {"pages": s["pages"], "ring_k": s["ring_k"], "ring_v": s["ring_v"]}


def _weights_masks(c, lens, n_rec):
    W, T = c["window"], c["queries"]
    ln = lens.long()[:, None, None]
    at = ln - T + torch.arange(T, device=DEV)[None, :, None]
    j = torch.arange(n_rec, device=DEV)
    rp = _ring_positions(lens, W)[:, None, :]
    return (j < ln - W) & (j <= at), (rp >= 0) & (rp <= at)


def _run_weights(s):
    c = s["c"]
    if own:
        s["cache"].attention_weights(0, s["q"], s["lens"], s["weights"], decay=c["decay"])
        return s["weights"]
    B, hq, hkv, T, W, fmt = c["batch"], c["hq"], c["hkv"], c["queries"], c["window"], c["fmt"]
    g = hq // hkv
    rec = _records(s, c["seq"])[0]
    S = rec.shape[2]
    q = s["q"].float().view(B, hkv, g * T, D)
    lg = torch.cat((_key_logits(_rotate(q, s["signs"]), rec, s, fmt, torch.float32),
                    q @ s["ring_k"][0].transpose(-1, -2)), -1) / SQRT_D
    m = torch.cat(_weights_masks(c, s["lens"], S), -1)[:, None, None].expand(B, hkv, g, T, S + W).reshape(lg.shape)
    p = _softmax(lg.masked_fill(~m, -math.inf)).sum(2)                        # [B][H][S + W]
    got = p[..., :c["seq"]].clone()
    rp = _ring_positions(s["lens"], W)
    got = torch.cat((got, torch.zeros_like(got[..., :1])), -1)
    got.scatter_add_(2, torch.where(rp < 0, torch.full_like(rp, c["seq"]), rp)[:, None].expand(B, hkv, W), p[..., S:])
    got = got[..., :c["seq"]]
    inside = torch.arange(c["seq"], device=DEV) < s["lens"][:, None, None]
    old = s["weights"]
    old.copy_(torch.where(inside, got + (c["decay"] * old if c["decay"] else 0.0), old))
    return old


def _run_evict(s):
    c = s["c"]
    if own:
        s["cache"].evict(-1, s["weights"], s["lens"], c["budget"], c["recent"], kept=s["kept"], new_lens=s["new_lens"])
        return {"kept": s["kept"], "new_lens": s["new_lens"], "weights": s["weights"], "pages": s["pages"],
                "ring_k": s["ring_k"], "ring_v": s["ring_v"]}
    n, W, S = c["budget"], c["window"], c["seq"]
    ln = s["lens"].long()[None, :, None, None]
    j = torch.arange(S, device=DEV)
    w = s["weights"].double()
    key = torch.where(w != w, torch.full_like(w, -1e300), w.clamp(-1e300, 1e300))
    key = torch.where(j >= ln - c["recent"], torch.full_like(w, math.inf), key)
    key = torch.where(j >= ln, torch.full_like(w, -math.inf), key)
    best = key.sort(dim=-1, descending=True, stable=True).indices[..., :n]
    best = torch.where(best < ln, best, torch.full_like(best, S)).sort(-1).values
    kept = torch.where(best < S, best, torch.full_like(best, -1))
    src = kept.clamp_min(0)
    new = s["lens"].clamp_max(n)
    cut = (s["lens"] > n)[None, :, None, None]
    rec = _records(s, S)
    moved = rec.gather(3, src[..., None].expand(*src.shape, rec.shape[-1]))
    _store(s, moved, torch.arange(n, device=DEV)[None, None, None, :], cut.expand(src.shape))
    s["weights"][..., :n] = torch.where(cut, s["weights"].gather(-1, src), s["weights"][..., :n])
    if W:
        p = _ring_positions(new, W)
        slot = ((p + (s["lens"] - new).long()[:, None]) % W)[None, :, None, :, None].expand(s["ring_k"].shape)
        s["ring_k"].copy_(torch.where(cut[..., None], s["ring_k"].gather(3, slot), s["ring_k"]))
        s["ring_v"].copy_(torch.where(cut[..., None], s["ring_v"].gather(3, slot), s["ring_v"]))
    return {"kept": kept.int(), "new_lens": new, "weights": s["weights"], "pages": s["pages"], "ring_k": s["ring_k"],
            "ring_v": s["ring_v"]}


# ---------------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    """The definitions in 64 bits: rotations as complex factors; keys and values taken back to the heads' own space and
    every sequence by itself.  Moved bytes and indices have no value here."""
    c = dict(case)
    if c["op"] == "commit":
        return None
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    if c["op"] == "rope":
        return _exact_rope(s, c)
    if c["op"] == "evict":
        return _exact_evict(s, c)
    return _exact_attention(s, c)


def _exact_rope(s, c):
    B, T, hq, hkv, rot = c["batch"], c["tokens"], c["hq"], c["hkv"], c["rot"]
    th, kind, fac, n0, lo, hi, att = _scaling(c)
    if kind == 2:
        th *= fac ** (rot / (rot - 2))
    f = []
    for i in range(rot // 2):
        w = th ** (-2 * i / rot)
        if kind == 1:
            w /= fac
        elif kind == 3:
            r = n0 * w / (2 * math.pi)
            part = min(1.0, max(0.0, (r - lo) / (hi - lo)))
            w = part * w + (1 - part) * w / fac
        elif kind == 4:
            a = max(math.floor(rot * math.log(n0 / (2 * math.pi * hi)) / (2 * math.log(th))), 0)
            b = min(math.ceil(rot * math.log(n0 / (2 * math.pi * lo)) / (2 * math.log(th))), rot - 1)
            part = min(1.0, max(0.0, (i - a) / max(b - a, 0.001)))
            w = (1 - part) * w + part * w / fac
        f.append(w)
    ang = s["pos"].double()[..., None] * torch.tensor(f, dtype=torch.float64, device=DEV)
    turn = torch.polar(torch.full_like(ang, att), ang)[:, :, None]             # [B][T][1][rot / 2]
    x = s["x"].double().view(B, T, -1, D)
    out = {"v": x[:, :, hq + hkv:].transpose(1, 2).contiguous()}
    for name, y, w in (("q", x[:, :, :hq], s["wq"]), ("k", x[:, :, hq:hq + hkv], s["wk"])):
        if w is not None:
            y = y / (y.square().sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
        y = y.clone()
        if c["layout"] == "half":
            z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * turn
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        else:
            z = torch.view_as_complex(y[..., :rot].reshape(B, T, -1, rot // 2, 2).contiguous()) * turn
            y[..., :rot] = torch.view_as_real(z).flatten(-2)
        out[name] = y.transpose(1, 2).contiguous()
    return out


def _exact_attention(s, c):
    B, hq, hkv, W, fmt = c["batch"], c["hq"], c["hkv"], c["window"], c["fmt"]
    g, f64 = hq // hkv, torch.float64
    had = torch.tensor([[(-1.0) ** bin(i & j).count("1") for j in range(D)] for i in range(D)], dtype=f64, device=DEV) * C_WHT
    back = had * s["signs"].double()[None, :]                                 # y @ back = s . (c H y)
    tree = c["op"] == "tree"
    out = torch.zeros_like(s["q"], dtype=f64) if tree else s["before"].double()
    for b in range(B):
        n = int(s["lens"][b])
        lay, page = s["pages"][0], s["bt"][b].long()
        half = lay[page].transpose(0, 1).reshape(hkv, -1, _half_bytes(fmt))
        rec = half[:, :, s["addr"]].reshape(hkv, -1, _rec(fmt))[:, :n]
        kb, km, vb, vm = _split(rec, fmt)
        val = _affine(_nibbles(vb), vm, f64) @ back
        q = s["q"][b].double().view(hkv, -1, D)
        if fmt == "tq3":
            code = torch.stack((kb & 7, (kb >> 3) & 7), -1).reshape(hkv, n, D).long()
            sgn = torch.stack((kb >> 6 & 1, kb >> 7), -1).reshape(hkv, n, D).double() * 2 - 1
            ng = _half_values(km).double()
            est = s["cent"].double()[code] + QJL * ng[..., 1:] * (sgn @ s["proj"].double())
            key = (ng[..., :1] * est) @ back
        elif fmt == "q8":
            key = ((kb.double() - 128).view(hkv, n, 4, 32) * _half_values(km).double()[..., None]).view(hkv, n, D) @ back
        else:
            key = _affine(_nibbles(kb), km, f64) @ back
        lq = (q @ key.transpose(1, 2)).view(hkv, -1, n) / SQRT_D
        pos = torch.arange(n, device=DEV)
        if W:
            rk, rv = s["ring_k"][0, b].double(), s["ring_v"][0, b].double()
            held = [p for p in range(max(0, n - W), n)]
            slots = torch.tensor([p % W for p in held], device=DEV)
            lr = q @ rk[:, slots].transpose(1, 2) / SQRT_D
        if not tree:
            T = c["queries"]
            at = (n - T + torch.arange(T, device=DEV)).repeat(g)[:, None]
            if W:
                lq[:, :, max(0, n - W):] = lr
            lq = lq.masked_fill(pos[None, :] > at, -math.inf)
            p = torch.softmax(lq, -1).nan_to_num(0.0).sum(1)
            out[b, :, :n] = p + c["decay"] * out[b, :, :n] if c["decay"] else p
            continue
        N = c["nodes"]
        par = s["parents"][b].tolist()
        kd, vd = s["k"][b].double(), s["v"][b].double()
        ld = q @ kd.transpose(1, 2) / SQRT_D
        lq, ld = lq.view(hkv, g, N, n), ld.view(hkv, g, N, N)
        if W:
            lr = lr.view(hkv, g, N, -1)
        for i in range(N):
            if par[i] < -1:
                continue
            chain, a = [], i
            while a >= 0:
                chain.append(a)
                a = par[a]
            first_raw = max(0, min(n, n + len(chain) - 1 - W + 1)) if W else n
            row = lq[:, :, i, :first_raw]
            vals = [val[:, :first_raw]]
            parts = [row]
            if W and first_raw < n:
                skip = first_raw - max(0, n - W)
                parts.append(lr[:, :, i, skip:])
                vals.append(rv[:, slots[skip:]])
            parts.append(ld[:, :, i, chain])
            vals.append(vd[:, chain])
            p = torch.softmax(torch.cat(parts, -1), -1)
            out[b].view(hkv, g, N, D)[:, :, i] = p @ torch.cat(vals, 1)
    return out


def _exact_evict(s, c):
    w = s["weights"].double().cpu().numpy()
    res = w.copy()
    for b, n in enumerate(_lens(c)):
        if n <= c["budget"]:
            continue
        old = n - c["recent"]
        for lay in range(w.shape[0]):
            for h in range(w.shape[2]):
                x = w[lay, b, h]
                best = np.lexsort((np.arange(old), -x[:old]))[:c["budget"] - c["recent"]]
                res[lay, b, h, :c["budget"]] = np.concatenate((x[np.sort(best)], x[old:n]))
    return {"weights": torch.as_tensor(res), "kept": None, "new_lens": None, "pages": None, "ring_k": None, "ring_v": None}

"""The cache held in 8 bits with a scale for each block of tokens and head (format KVQ_Q8B32: decode and chunked prefill,
which appends), and the operators on a cache's pages (kv_pool_fork, kv_pool_reserve, kv_pool_release, kv_pool_compact), as
measured cases.

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU from a seed, ``run`` does one pass: in
plain torch operations where ``own`` is false, through the package where it is true.  The cache's contents are
packed here, from the buffer layout that include/kvq.h documents: the same bytes for both.  Every pass leaves a state
that the same pass can be made of again.
"""

import math

import numpy as np
import torch

own = False

D = 128
PAGE, HALF = 64, 32
DEV = "cuda"
FMT = {"q4": (1, 1, 2 * 5120), "tq3": (3, 1, 2 * 4736), "q8": (4, 1, 2 * 6912), "q8b": (5, 5, 2 * 8208)}  # K, V, page bytes
HALF_BYTES = 8208                                # q8b: 4096 key codes, 4096 value codes, two float scales, 8 unused
C_WHT = float(np.float32(1 / math.sqrt(128)))
SQRT_D = math.sqrt(128.0)


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one layer's decode step early in a chat: latency counts
        dict(name="decode 1 at 700", op="decode", layers=1, batch=1, seq=700, spread=0.0, hq=24, hkv=8, window=128),
        # one layer's step of eight long ragged contexts
        dict(name="decode 8x16K ragged", op="decode", layers=1, batch=8, seq=16384, spread=0.5, hq=32, hkv=8, window=128),
        # every layer of a model in one call over a long context: bandwidth counts
        dict(name="decode 28 layers 32K", op="decode", layers=28, batch=1, seq=32768, spread=0.0, hq=24, hkv=8, window=128),
        # one layer of a whole prompt
        dict(name="prefill prompt 2048", op="prefill", batch=1, tokens=2048, start=0, hq=32, hkv=8, window=128, dtype="bf16"),
        # one layer of a later chunk of a long document, at an odd position within its block
        dict(name="prefill 1024 at 15001", op="prefill", batch=1, tokens=1024, start=15001, hq=24, hkv=8, window=128,
             dtype="bf16"),
        # short follow-up turns of three conversations, float inputs
        dict(name="prefill 3x37 at 1000", op="prefill", batch=3, tokens=37, start=1000, hq=8, hkv=2, window=64, dtype="f32"),
        # a step of beam search: every beam takes over one of the beams, all layers
        dict(name="beams 16, 28 layers", op="beams", layers=28, batch=16, seq=1500, spread=0.0, hkv=8, window=128, fmt="q4"),
        dict(name="beams 4, one layer", op="beams", layers=1, batch=4, seq=333, spread=0.0, hkv=8, window=128, fmt="q8"),
        # four prompts sampled eight times each: shared pages, and the page of the next token made each one's own
        dict(name="sample 4x8, 28 layers", op="sample", layers=28, prompts=4, samples=8, seq=1000, spread=0.4, hkv=8, window=128,
             fmt="q8b"),
        # pages for 64 prompts out of a large pool in use, and back
        dict(name="admit 64 prompts", op="admit", batch=64, tokens=900, held=4000, fmt="q4", hkv=8),
        # two waves of requests that end, the pool closed up after each
        dict(name="compact 8 layers", op="compact", layers=8, batch=8, tokens=2000, hkv=8, fmt="q8b"),
        dict(name="compact small ragged", op="compact", layers=1, batch=6, tokens=700, hkv=2, fmt="tq3"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "beams", "sample", "admit", "compact"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4])
    window = rng.choice([32, 64, 100, 128, 256])
    fmt = rng.choice(["q4", "q8", "tq3", "q8b"])
    if op == "decode":
        return dict(op=op, layers=_log(rng, 1, 4), batch=rng.randint(1, 8), seq=_log(rng, 1, 24000),
                    spread=rng.choice([0.0, 0.5, 0.99]), hq=hq, hkv=hkv, window=window)
    if op == "prefill":
        start = rng.choice([0, _log(rng, 1, 12000)])
        return dict(op=op, batch=rng.randint(1, 3), tokens=_log(rng, 1, 280 if start else 1500), start=start, hq=hq, hkv=hkv,
                    window=window, dtype=rng.choice(["bf16", "f32"]))
    if op == "beams":
        return dict(op=op, layers=_log(rng, 1, 8), batch=_log(rng, 2, 24), seq=_log(rng, 1, 900), spread=rng.choice([0.0, 0.9]),
                    hkv=hkv, window=rng.choice([0, window]) if fmt != "q8b" else window, fmt=fmt)
    if op == "sample":
        return dict(op=op, layers=_log(rng, 1, 12), prompts=rng.randint(1, 4), samples=rng.randint(2, 9), seq=_log(rng, 1, 1200),
                    spread=rng.choice([0.0, 0.9]), hkv=hkv, window=rng.choice([0, window]) if fmt != "q8b" else window, fmt=fmt)
    if op == "admit":
        return dict(op=op, batch=_log(rng, 1, 200), tokens=_log(rng, 1, 3000), held=_log(rng, 1, 9000), fmt=fmt, hkv=hkv)
    return dict(op=op, layers=_log(rng, 1, 6), batch=2 * rng.randint(1, 6), tokens=_log(rng, 1, 1800), hkv=hkv, fmt=fmt)


def _lens(c, n):
    """Cached tokens of n sequences: ``seq`` down to (1 - spread) of it."""
    return [max(1, int(round(c["seq"] * (1 - c["spread"] * b / max(1, n - 1))))) for b in range(n)]


def _compact_tokens(c, b):
    """Tokens of request b of the wave that begins: every third one a little shorter."""
    return max(1, c["tokens"] - 90 * (b % 3))


def work(c):
    """Bytes: each input read once, each output written once.  Operations: the products of the formulas."""
    if c["op"] == "decode":
        W, hkv, hq, lens = c["window"], c["hkv"], c["hq"], _lens(c, c["batch"])
        quant = sum(-(-max(0, n - W) // HALF) for n in lens)
        raw = sum(min(n, W) for n in lens)
        return {"bytes": c["layers"] * (hkv * (quant * HALF_BYTES + raw * 2 * D * 4) + c["batch"] * hq * D * 6),
                "flops": c["layers"] * 4 * D * hq * sum(lens)}
    if c["op"] == "prefill":
        B, T, p, W, hkv, hq = c["batch"], c["tokens"], c["start"], c["window"], c["hkv"], c["hq"]
        e = 2 if c["dtype"] == "bf16" else 4
        seen = T * p + T * (T + 1) // 2
        blocks = -(-max(0, p + T - W) // HALF)
        return {"bytes": B * (T * D * (e * (hq + 2 * hkv) + 4 * hq) + hkv * (blocks * HALF_BYTES + (min(p, W) + min(T, W)) * 8 * D)),
                "flops": B * 4 * D * hq * seen}
    page = FMT[c["fmt"]][2] * c["hkv"]
    if c["op"] == "beams":
        lens = _lens(c, c["batch"])
        ring = c["layers"] * c["hkv"] * 8 * D
        # (about half of the beams are parents: read once, each beam written once)
        return {"bytes": sum(1.5 * min(n, c["window"]) * ring + 12 * -(-n // PAGE) for n in lens), "flops": 0}
    if c["op"] == "sample":
        lens = _lens(c, c["prompts"])
        ring = c["layers"] * c["hkv"] * 8 * D
        n = c["samples"]
        return {"bytes": sum(n * min(x, c["window"]) * ring + (n * c["layers"] * page if x % PAGE else 0) + 12 * n * -(-x // PAGE)
                             for x in lens), "flops": 0}
    if c["op"] == "admit":
        return {"bytes": 16 * c["batch"] * -(-c["tokens"] // PAGE) + 4 * c["held"], "flops": 0}
    h = c["batch"] // 2
    gone = sum(-(-_compact_tokens(c, b) // PAGE) for b in range(h))
    stay = sum(-(-_compact_tokens(c, b) // PAGE) for b in range(h, 2 * h))
    return {"bytes": 2 * 2 * min(gone, stay) * c["layers"] * page + 40 * (gone + stay), "flops": 0}


# ---------------------------------------------------------------------------- the format's layout and codec
def _signs():
    """SplitMix64 of seed 0: sign j is -1 where bit 0 of output j + 1 is set."""
    m = (1 << 64) - 1

    def out(j):
        z = ((j + 1) * 0x9E3779B97F4A7C15) & m
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & m
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & m
        return z ^ (z >> 31)

    return torch.tensor([-1.0 if out(j) & 1 else 1.0 for j in range(D)], device=DEV)


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


def _address():
    """Byte offsets within a half-page of the codes of (token, channel): keys, values [32][128]."""
    t, ch = np.meshgrid(np.arange(HALF), np.arange(D), indexing="ij")
    k = (t // 16 * 4 + ch // 32) * 512 + (t % 8 * 4 + ch % 8 // 2) * 16 + ch // 16 % 2 * 8 + ch // 8 % 2 * 4 + t // 8 % 2 * 2 + ch % 2
    v = 4096 + ch // 16 * 512 + (ch % 8 * 4 + t % 8 // 2) * 16 + t // 16 * 8 + t // 8 % 2 * 4 + ch // 8 % 2 * 2 + t % 2
    return [torch.as_tensor(a, dtype=torch.int64, device=DEV) for a in (k, v)]


def _code(y):
    """Blocks [...][32][128] of rotated vectors: codes + 128 and the block's scale."""
    amax = y.abs().amax((-1, -2))
    d = amax / torch.full_like(amax, 127.0)
    s = d[..., None, None]
    return torch.where(s > 0, (y / s).round().clamp(-127, 127) + 128, torch.full_like(y, 128.0)).to(torch.uint8), d


def _blocks(k, v, s):
    """Half-pages [...][HALF_BYTES] of raw blocks k, v [...][32][128]."""
    half = torch.zeros(*k.shape[:-2], HALF_BYTES, dtype=torch.uint8, device=DEV)
    (ck, dk), (cv, dv) = _code(_rotate(k, s["signs"])), _code(_rotate(v, s["signs"]))
    half[..., s["addr"][0]] = ck
    half[..., s["addr"][1]] = cv
    half[..., 8192:8200] = torch.stack((dk, dv), -1).contiguous().view(torch.uint8)
    return half


def _values(s, n, kind):
    """Rotated keys and values of the first n positions, rounded up to pages: two of [layers][batch][heads][positions][128]."""
    pages, bt = s["pages"], s["bt"]
    lp = -(-n // PAGE)
    B = bt.shape[0]
    got = pages[:, bt[:, :lp].long()].reshape(pages.shape[0], B, lp, pages.shape[2], 2, HALF_BYTES)
    d = got[..., 8192:8200].contiguous().view(torch.float32).to(kind)

    def side(i):
        x = (got[..., s["addr"][i]].to(kind) - 128) * d[..., i, None, None]     # [L][B][lp][H][2][32][128]
        return x.permute(0, 1, 3, 2, 4, 5, 6).reshape(pages.shape[0], B, pages.shape[2], lp * PAGE, D)

    return side(0), side(1)


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


def _buffers(c, layers, B, mpp, n_pages, hq, dtype, bt):
    """Pages, rings, block table and reference counts of a cache, its own buffer's where it is the package's."""
    kf, vf, size = FMT[c.get("fmt", "q8b")]
    H, W = c["hkv"], c.get("window", 32)
    shape, ring = (layers, n_pages, H, size), (layers, B, H, W, D)
    s = {"c": c, "bt": bt}
    if own:
        from kv_cache_quantization_append_gb300 import QuantKVCache, lib

        cfg = lib.make_config(layers, H, hq, B, mpp * PAGE, window=W, n_pages=n_pages, k_format=kf, v_format=vf,
                              in_dtype=lib.KVQ_IN_BF16 if dtype == "bf16" else lib.KVQ_IN_F32)
        s["cache"] = cache = QuantKVCache(cfg, DEV, bt, np.zeros((D, D), np.float32))
        nb, nf = layers * n_pages * H * size, layers * B * H * W * D * 4
        off = lib.kv_cache_bytes(cfg) - -(-nb // 256) * 256
        rb = -(-nf // 256) * 256
        s["pages"] = cache.buffer[off:off + nb].view(shape)
        s["ring_v"] = cache.buffer[off - rb:off - rb + nf].view(torch.float32).view(ring)
        s["ring_k"] = cache.buffer[off - 2 * rb:off - 2 * rb + nf].view(torch.float32).view(ring)
        if c["op"] not in ("decode", "prefill"):
            table = bt.clone()
            cache.pool_init()                                              # (clears the table)
            bt.copy_(table)
            s["refs"] = cache.page_refs
        s["pages"].zero_()
    else:
        s["pages"] = torch.zeros(shape, dtype=torch.uint8, device=DEV)
        s["ring_k"], s["ring_v"] = (torch.empty(ring, device=DEV) for _ in range(2))
        s["refs"] = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    return s


def _attention_state(c, g, layers, max_len, filled, dtype):
    """A paged 8-bit cache in a shuffled pool of pages, the first ``filled`` positions coded, a ring of raw vectors."""
    B, H = c["batch"], c["hkv"]
    mpp = -(-max_len // PAGE)
    n_pages = B * mpp + 3
    bt = torch.randperm(n_pages, generator=g, device=DEV)[:B * mpp].reshape(B, mpp).int().contiguous()
    s = _buffers(c, layers, B, mpp, n_pages, c["hq"], dtype, bt)
    s["signs"], s["addr"] = _signs(), _address()
    s["ring_k"].copy_(_heads(g, *s["ring_k"].shape[:-1]))
    s["ring_v"].copy_(_heads(g, *s["ring_v"].shape[:-1]))
    for lay in range(layers):
        for lo in range(0, -(-filled // PAGE), 256):
            n = min(256, -(-filled // PAGE) - lo)
            half = _blocks(_heads(g, B, n, H, 2, HALF), _heads(g, B, n, H, 2, HALF), s)
            s["pages"][lay][bt[:, lo:lo + n].long()] = half.reshape(B, n, H, 2 * HALF_BYTES)
    return s


def _fill(s, g):
    """Any bytes in the pages, any vectors in the rings."""
    s["pages"].copy_(torch.randint(0, 256, s["pages"].shape, generator=g, device=DEV, dtype=torch.uint8))
    s["ring_k"].copy_(torch.randn(s["ring_k"].shape, generator=g, device=DEV))
    s["ring_v"].copy_(torch.randn(s["ring_v"].shape, generator=g, device=DEV))


def _count(s):
    """Reference counts of the block table as it stands."""
    at = s["bt"].long().flatten()
    s["refs"].copy_(torch.zeros_like(s["refs"]).scatter_add_(0, at.clamp_min(0), (at >= 0).int()))


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    if c["op"] == "decode":
        s = _attention_state(c, g, c["layers"], c["seq"], c["seq"], "bf16")
        s["lens"] = _int(_lens(c, c["batch"]))
        s["q"] = torch.randn(c["layers"], c["batch"], c["hq"], D, generator=g, device=DEV).to(torch.bfloat16)
        s["out"] = torch.empty(s["q"].shape, device=DEV)
        return s
    if c["op"] == "prefill":
        B, T, p, W = c["batch"], c["tokens"], c["start"], c["window"]
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        s = _attention_state(c, g, 1, p + T, p // HALF * HALF, c["dtype"])
        s["q"] = torch.randn(B, c["hq"], T, D, generator=g, device=DEV).to(dt)
        s["k"], s["v"] = (_heads(g, B, c["hkv"], T).to(dt) for _ in range(2))
        s["pos"] = _int([p] * B)
        s["out"] = torch.empty(s["q"].shape, device=DEV)
        # the ring as a pass leaves it: the same for every pass
        last = torch.arange(max(0, T - W), T, device=DEV)
        s["ring_k"][0, :, :, (p + last) % W] = s["k"][:, :, last].float()
        s["ring_v"][0, :, :, (p + last) % W] = s["v"][:, :, last].float()
        return s
    if c["op"] in ("beams", "sample"):
        groups, each = (c["batch"], 1) if c["op"] == "beams" else (c["prompts"], c["samples"])
        B, lens = groups * each, _lens(c, groups)
        mpp = -(-(max(lens) + 1) // PAGE)
        n_pages = groups * mpp + B + 2
        bt = torch.full((B, mpp), -1, dtype=torch.int32, device=DEV)
        page = torch.randperm(n_pages, generator=g, device=DEV)[:groups * mpp].reshape(groups, mpp).int()
        held = torch.arange(mpp, device=DEV)[None, :] < -(-_int(lens)[:, None] // PAGE)
        bt[::each] = torch.where(held, page, torch.full_like(page, -1))
        s = _buffers(c, c["layers"], B, mpp, n_pages, c["hkv"], "bf16", bt)
        _fill(s, g)
        _count(s)
        s["lens"] = torch.zeros(B, dtype=torch.int32, device=DEV)
        s["lens"][::each] = _int(lens)
        if c["op"] == "beams":
            # most beams go on under one of the best few
            s["parents"] = (torch.rand(B, generator=g, device=DEV) ** 2 * B).int().clamp_max(B - 1)
        else:
            s["parents"] = (torch.arange(B, device=DEV) // each * each).int()
        s["new_lens"], s["granted"] = torch.empty_like(s["lens"]), torch.empty_like(s["lens"])
        return s
    if c["op"] == "admit":
        # `held` pages of older sequences, scattered; the prompts' sequences hold nothing yet
        B, mpp = c["batch"], max(-(-c["tokens"] // PAGE), -(-c["held"] // 256))
        old = -(-c["held"] // mpp)
        n_pages = c["held"] + B * mpp + B * mpp // 4 + 8
        bt = torch.full((B + old, mpp), -1, dtype=torch.int32, device=DEV)
        page = torch.randperm(n_pages, generator=g, device=DEV)[:c["held"]].int()
        bt[B:].view(-1)[:c["held"]] = page
        c["window"] = 32
        s = _buffers(c, 1, B + old, mpp, n_pages, c["hkv"], "bf16", bt)
        _count(s)
        s["pos"], s["keep"] = _int([0] * B), _int([0] * B)
        s["granted"] = torch.empty_like(s["pos"])
        return s
    # compact: two halves of the sequences; the first holds the lower pages
    B, mpp = c["batch"], -(-c["tokens"] // PAGE)
    tokens = [_compact_tokens(c, b) for b in range(B)]
    held = torch.arange(mpp, device=DEV)[None, :] < _int([-(-n // PAGE) for n in tokens])[:, None]
    bt = torch.where(held, (held.flatten().cumsum(0) - 1).view(B, mpp), torch.full((B, mpp), -1, device=DEV)).int().contiguous()
    n_pages = B * mpp + 5
    c["window"] = 32
    s = _buffers(c, c["layers"], B, mpp, n_pages, c["hkv"], "bf16", bt)
    _fill(s, g)
    _count(s)
    first = torch.arange(B, device=DEV) < B // 2
    s["waves"] = [(torch.where(w, 0, -1).int(), torch.where(w, 0, -1).int(), _int(tokens)) for w in (first, ~first)]
    s["granted"] = torch.empty(B, dtype=torch.int32, device=DEV)
    s["n_used"] = torch.empty(1, dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------------------- one pass
def run(s):
    return {"decode": _run_decode, "prefill": _run_prefill, "beams": _run_fork, "sample": _run_fork, "admit": _run_admit,
            "compact": _run_compact}[s["c"]["op"]](s)


def _softmax(x):
    m = x.amax(-1, keepdim=True)
    p = (x - torch.where(m == -math.inf, torch.zeros_like(m), m)).exp()
    return p / p.sum(-1, keepdim=True).clamp_min(1e-38)


def _ring_positions(lens, W):
    """Position that each ring slot holds of sequences of these lengths (negative: none)."""
    last = lens.long()[:, None] - 1
    return last - (last - torch.arange(W, device=DEV)[None, :]) % W


def _run_decode(s):
    c = s["c"]
    if own:
        return s["cache"].decode(-1, s["q"], s["lens"], out=s["out"])
    L, B, hq, hkv, W = c["layers"], c["batch"], c["hq"], c["hkv"], c["window"]
    k, v = _values(s, c["seq"], torch.float32)
    S = k.shape[3]
    q = s["q"].float().view(L, B, hkv, hq // hkv, D)
    lg = torch.cat((_rotate(q, s["signs"]) @ k.transpose(-1, -2), q @ s["ring_k"].transpose(-1, -2)), -1) / SQRT_D
    ln = s["lens"].long()[:, None]
    seen = torch.cat((torch.arange(S, device=DEV)[None, :] < ln - W, _ring_positions(s["lens"], W) >= 0), -1)
    p = _softmax(lg.masked_fill(~seen[None, :, None, None], -math.inf))
    o = _unrotate(p[..., :S] @ v, s["signs"]) + p[..., S:] @ s["ring_v"]
    return o.reshape(L, B, hq, D)


def _around(s, x, ring):
    """Raw vectors of positions base .. start + T - 1 (the ring's, then the chunk's), base a block's first position."""
    c = s["c"]
    p, W = c["start"], c["window"]
    base = max(0, p - W) // HALF * HALF
    old = torch.arange(base, p, device=DEV)
    return torch.cat((ring[0][:, :, old % W], x.float()), 2), base


def _run_prefill(s):
    c = s["c"]
    if own:
        s["cache"].prefill(0, s["k"], s["v"], s["q"], s["pos"], out=s["out"])
        return {"out": s["out"], "pages": s["pages"], "ring_k": s["ring_k"], "ring_v": s["ring_v"]}
    B, T, p, W, hq, hkv = c["batch"], c["tokens"], c["start"], c["window"], c["hq"], c["hkv"]
    (rk, base), (rv, _) = _around(s, s["k"], s["ring_k"]), _around(s, s["v"], s["ring_v"])
    # the blocks that the chunk finishes
    b0, b1 = p // HALF, (p + T) // HALF
    if b1 > b0:
        sl = slice(b0 * HALF - base, b1 * HALF - base)
        half = _blocks(rk[:, :, sl].reshape(B, hkv, b1 - b0, HALF, D), rv[:, :, sl].reshape(B, hkv, b1 - b0, HALF, D), s)
        at = torch.arange(b0, b1, device=DEV)
        size = s["pages"].shape[-1]
        two = s["pages"][0].view(-1, hkv, 2, size // 2)
        two[s["bt"][:, at // 2].long(), :, at % 2] = half.permute(0, 2, 1, 3)
    n = max(0, p + T - W)
    k, v = _values(s, max(n, 1), torch.float32)
    k, v = k[0], v[0]
    S = k.shape[2]
    q = s["q"].float().view(B, hkv, hq // hkv * T, D)
    lg = torch.cat((_rotate(q, s["signs"]) @ k.transpose(-1, -2), q @ rk.transpose(-1, -2)), -1) / SQRT_D
    at = p + torch.arange(T, device=DEV)[:, None]
    j, r = torch.arange(S, device=DEV)[None, :], base + torch.arange(rk.shape[2], device=DEV)[None, :]
    seen = torch.cat((j <= at - W, (r <= at) & (r > at - W)), -1).repeat(hq // hkv, 1)
    w = _softmax(lg.masked_fill(~seen, -math.inf))
    o = _unrotate(w[..., :S] @ v, s["signs"]) + w[..., S:] @ rv
    last = torch.arange(max(0, T - W), T, device=DEV)
    s["ring_k"][0, :, :, (p + last) % W] = s["k"][:, :, last].float()
    s["ring_v"][0, :, :, (p + last) % W] = s["v"][:, :, last].float()
    return {"out": o.view(B, hq, T, D), "pages": s["pages"], "ring_k": s["ring_k"], "ring_v": s["ring_v"]}


def _fork(s):
    """Every sequence takes over its parent's pages and ring as they were; new lengths."""
    bt, W, par = s["bt"], s["c"]["window"], s["parents"].long()
    old, lens = bt.clone(), s["lens"]
    new_lens = lens[par]
    col = torch.arange(bt.shape[1], device=DEV)[None, :]
    stays = (par == torch.arange(par.shape[0], device=DEV))[:, None]
    bt.copy_(torch.where(stays | (col < -(-new_lens[:, None] // PAGE)), old[par], torch.full_like(old, -1)))
    _count(s)
    if W:
        moved = (torch.arange(W, device=DEV)[None, :] < new_lens[:, None])[None, :, None, :, None]
        s["ring_k"].copy_(torch.where(moved, s["ring_k"][:, par], s["ring_k"]))
        s["ring_v"].copy_(torch.where(moved, s["ring_v"][:, par], s["ring_v"]))
    return new_lens


def _reserve(s, pos, tokens):
    """Pages for positions pos .. pos + tokens - 1, in order of sequence and page, the lowest free ones first; pages that
    others share are copied, but for the last writer where all that share a page write it."""
    bt, refs = s["bt"], s["refs"]
    B = pos.shape[0]
    rows = bt[:B]
    p = pos.long()[:, None]
    n = tokens if isinstance(tokens, int) else tokens.long()[:, None]
    col = torch.arange(bt.shape[1], device=DEV)[None, :]
    hit = (p >= 0) & (col >= p // PAGE) & (col <= (p + n - 1) // PAGE)
    at = rows.long().clamp_min(0)
    shared = hit & (rows >= 0) & (refs[at] > 1)
    item = torch.arange(rows.numel(), device=DEV).view(rows.shape)
    writers = torch.zeros_like(refs).scatter_add_(0, at.flatten(), shared.flatten().int())
    last = torch.full(refs.shape, -1, dtype=torch.int64, device=DEV).scatter_reduce_(
        0, at.flatten(), torch.where(shared, item, torch.full_like(item, -1)).flatten(), "amax")
    copied = shared & ~((writers[at] == refs[at]) & (last[at] == item))
    need = copied | (hit & (rows < 0))
    rank = need.flatten().cumsum(0).view(rows.shape)
    free = torch.argsort((refs != 0).int(), stable=True)
    fits = rank[:, -1:] <= (refs == 0).sum()
    take = need & fits
    page = free[(rank - 1).clamp(0, free.numel() - 1)]
    copied = copied & fits
    src, dst = at[copied], page[copied]
    if src.numel():
        s["pages"][:, dst] = s["pages"][:, src]
    rows.copy_(torch.where(take, page.int(), rows))
    _count(s)
    return torch.where((p >= 0) & fits, p, torch.full_like(p, -1))[:, 0].int()


def _release(s, keep):
    rows = s["bt"][:keep.shape[0]]
    col = torch.arange(rows.shape[1], device=DEV)[None, :]
    gone = (keep[:, None] >= 0) & (col >= -(-keep[:, None] // PAGE))
    rows.copy_(torch.where(gone, torch.full_like(rows, -1), rows))
    _count(s)


def _compact(s):
    refs, bt = s["refs"], s["bt"]
    used = refs > 0
    U = used.sum()
    page = torch.arange(refs.shape[0], device=DEV)
    dst, src = torch.nonzero(~used & (page < U))[:, 0], torch.nonzero(used & (page >= U))[:, 0]
    s["pages"][:, dst] = s["pages"][:, src]
    page[src] = dst
    bt.copy_(torch.where(bt >= 0, page[bt.long().clamp_min(0)].int(), bt))
    _count(s)
    return U.int().view(1)


def _run_fork(s):
    sample = s["c"]["op"] == "sample"
    if own:
        s["cache"].fork(s["parents"], s["lens"], new_lens=s["new_lens"])
        new_lens = s["new_lens"]
        granted = s["cache"].reserve(new_lens, 1, granted=s["granted"]) if sample else None
    else:
        new_lens = _fork(s)
        granted = _reserve(s, new_lens, 1) if sample else None
    return {"table": s["bt"], "refs": s["refs"], "lens": new_lens, "granted": granted, "ring_k": s["ring_k"], "ring_v": s["ring_v"],
            "pages": s["pages"] if sample else None}


def _run_admit(s):
    c = s["c"]
    if own:
        granted = s["cache"].reserve(s["pos"], c["tokens"], granted=s["granted"])
        table = s["bt"][:c["batch"]].clone()
        s["cache"].release(s["keep"])
    else:
        granted = _reserve(s, s["pos"], c["tokens"])
        table = s["bt"][:c["batch"]].clone()
        _release(s, s["keep"])
    return {"granted": granted, "table": table, "after": s["bt"], "refs": s["refs"]}


def _wave(s, k):
    """Half of the requests end, the pool is closed up, new ones take pages; how many pages were in use."""
    keep, pos, tokens = s["waves"][k]
    if own:
        s["cache"].release(keep)
        s["cache"].compact(n_used=s["n_used"])
        used = s["n_used"].clone()
        s["cache"].reserve(pos, tokens, granted=s["granted"])
        return used
    _release(s, keep)
    used = _compact(s)
    s["granted"] = _reserve(s, pos, tokens)
    return used


def _run_compact(s):
    used = (_wave(s, 0), _wave(s, 1))
    return {"used": used, "granted": s["granted"], "table": s["bt"], "refs": s["refs"], "pages": s["pages"]}


# ---------------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    """Attention in 64 bits, each sequence and head by itself, keys and values taken back to the heads' own space; the codes
    are those of the format, which defines them in single operations of 32 bits.  Moved bytes have no value here."""
    c = dict(case)
    if c["op"] not in ("decode", "prefill"):
        return None
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    f64 = torch.float64
    had = torch.tensor([[(-1.0) ** bin(i & j).count("1") for j in range(D)] for i in range(D)], dtype=f64, device=DEV) / SQRT_D
    back = had * s["signs"].double()[None, :]                                  # y @ back = s . (H y) / sqrt(128)
    hkv, g, W = c["hkv"], c["hq"] // c["hkv"], c["window"]
    if c["op"] == "decode":
        out = torch.zeros(s["q"].shape, dtype=f64, device=DEV)
        for lay in range(c["layers"]):
            for b, n in enumerate(_lens(c, c["batch"])):
                m = max(0, n - W)
                slots = torch.arange(m, n, device=DEV) % W
                for h in range(hkv):
                    k, v = _stored(s, lay, b, h, m, back)
                    k = torch.cat((k, s["ring_k"][lay, b, h, slots].double()))
                    v = torch.cat((v, s["ring_v"][lay, b, h, slots].double()))
                    q = s["q"][lay, b, h * g:(h + 1) * g].double()
                    out[lay, b, h * g:(h + 1) * g] = torch.softmax(q @ k.T / SQRT_D, -1) @ v
        return out
    B, T, p = c["batch"], c["tokens"], c["start"]
    out = torch.zeros(s["q"].shape, dtype=f64, device=DEV)
    n = p + T
    at = p + torch.arange(T, device=DEV)[:, None]
    j = torch.arange(n, device=DEV)[None, :]
    raw_seen, rec_seen = (j <= at) & (j > at - W), j <= at - W
    for b in range(B):
        for h in range(hkv):
            q = s["q"][b, h * g:(h + 1) * g].double()
            rec, raw = [], []
            for side, (x, ring) in enumerate(((s["k"], s["ring_k"]), (s["v"], s["ring_v"]))):
                r = torch.zeros(n, D, device=DEV)                              # raw vectors of every position that is read raw or coded
                lo = max(0, p - W)
                r[lo:p] = ring[0, b, h, torch.arange(lo, p, device=DEV) % W]
                r[p:] = x[b, h].float()
                y = torch.zeros(n, D, dtype=f64, device=DEV)
                b0, b1 = p // HALF * HALF, n // HALF * HALF
                y[:b0] = _stored(s, 0, b, h, b0, back)[side]
                if b1 > b0:
                    y[b0:b1] = _dequantised(r[b0:b1] * s["signs"]) @ back
                rec.append(y)
                raw.append(r.double())
            for i in range(g):
                lr = (q[i] @ raw[0].T / SQRT_D).masked_fill(~raw_seen, -math.inf)
                lq = (q[i] @ rec[0].T / SQRT_D).masked_fill(~rec_seen, -math.inf)
                w = torch.softmax(torch.cat((lr, lq), -1), -1)
                out[b, h * g + i] = w[:, :n] @ raw[1] + w[:, n:] @ rec[1]
    return {"out": out, "pages": None, "ring_k": None, "ring_v": None}


def _stored(s, lay, b, h, n, back):
    """Keys and values of positions 0 .. n - 1 in the heads' space, from the pages' bytes."""
    lp = -(-n // PAGE)
    half = s["pages"][lay][s["bt"][b, :lp].long(), h].reshape(2 * lp, HALF_BYTES)
    d = half[:, 8192:8200].contiguous().view(torch.float32).double()
    return [(((half[:, s["addr"][i]].double() - 128) * d[:, i, None, None]).reshape(-1, D)[:n]) @ back for i in range(2)]


def _dequantised(x):
    """What the codes of whole blocks of sign-flipped vectors stand for, rotated: pairs (i, i + h) become their sum and difference."""
    y = x.clone()
    h = 1
    while h < D:
        lo = torch.tensor([i for i in range(D) if not i & h], device=DEV)
        a, b = y[:, lo], y[:, lo + h]
        y[:, lo], y[:, lo + h] = a + b, a - b
        h *= 2
    y = (y * C_WHT).view(-1, HALF * D)
    d = y.abs().amax(1, keepdim=True) / torch.full((1,), 127.0, device=DEV)
    code = torch.where(d > 0, torch.round(y / d).clamp(-127, 127), torch.zeros_like(y))
    return (code.double() * d.double()).view(-1, D)

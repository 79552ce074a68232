"""ctypes binding of libkvq (the C ABI in include/kvq.h): argument marshalling only.

Every function here has the name of the C entry point it calls and does nothing but check tensor
properties, take ``data_ptr()`` and the current CUDA stream, and translate status codes into
exceptions.  All computation happens in the library's CUDA kernels; there is no fallback path.
"""

from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_lib", "libkvq.so")

KVQ_Q4G32 = 1
KVQ_TQ3_QJL = 3
KVQ_Q8G32 = 4
KVQ_Q8B32 = 5
# the key formats by the names the workloads and the oracle use
K_FORMATS = {"q4g32": KVQ_Q4G32, "tq3_qjl": KVQ_TQ3_QJL, "q8g32": KVQ_Q8G32, "q8b32": KVQ_Q8B32}
KVQ_IN_F32 = 0
KVQ_IN_BF16 = 1

DEV_BAD_PAGE = 1
DEV_POS_RANGE = 2
DEV_SEQLEN_RANGE = 4
DEV_TIMEOUT = 8
DEV_BAD_NODE = 16
DEV_NO_PAGES = 32
DEV_BAD_PARENT = 64

MAX_TREE = 64
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_PLAIN, ROPE_LINEAR, ROPE_NTK, ROPE_TURNS, ROPE_DIMS = range(5)

EXPORTS = ("kv_cache_bytes", "kv_cache_init", "kv_calibrate_scratch_bytes", "kv_calibrate",
           "kv_quant_append", "kv_decode_scratch_bytes", "kv_decode_attention",
           "kv_decode_attention_noalloc", "kv_prefill_scratch_bytes", "kv_prefill_attention",
           "kv_tbq_block_bytes", "kv_tbq_encode", "kv_tbq_decode", "kv_split_record_bytes",
           "kv_split_outliers", "kv_split_encode", "kv_split_decode", "kv_status", "kv_set_wait_limit_ns",
           "kv_strerror", "kv_rope_init", "kv_qk_norm_rope", "kv_tree_scratch_bytes", "kv_tree_attention",
           "kv_tree_commit", "kv_weights_scratch_bytes", "kv_attention_weights", "kv_evict",
           "kv_pool_bytes", "kv_pool_init", "kv_pool_reserve", "kv_pool_fork", "kv_pool_release", "kv_pool_compact")
NOALLOC_SCRATCH_MAX = 32 * 1024 * 1024


class kvq_config(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("n_q_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("max_batch", ctypes.c_int32), ("max_seq_len", ctypes.c_int32),
                ("window", ctypes.c_int32), ("page_tokens", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("k_format", ctypes.c_int32),
                ("v_format", ctypes.c_int32), ("sinkhorn", ctypes.c_int32),
                ("group", ctypes.c_int32), ("in_dtype", ctypes.c_int32),
                ("seed", ctypes.c_uint64)]


class kvq_cache(ctypes.Structure):
    _fields_ = [("cfg", kvq_config), ("dev", ctypes.c_void_p), ("bytes", ctypes.c_uint64),
                ("block_table", ctypes.c_void_p), ("max_pages_per_seq", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("device", ctypes.c_int32), ("magic", ctypes.c_uint32)]


class kvq_rope(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("attn_factor", ctypes.c_float),
                ("magic", ctypes.c_uint32), ("turns", ctypes.c_uint64 * 64)]


class KVQError(RuntimeError):
    pass


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libkvq.so; raises if it has not been built (there is no CPU fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise KVQError(f"libkvq.so not built ({path}); run __graft_entry__.build() first")
    lib = ctypes.CDLL(path)
    P, I32, SZ, U32P = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.POINTER(ctypes.c_uint32)
    cfgp, cachep = ctypes.POINTER(kvq_config), ctypes.POINTER(kvq_cache)
    ropep, I64, F32, F64 = ctypes.POINTER(kvq_rope), ctypes.c_int64, ctypes.c_float, ctypes.c_double
    sig = {
        "kv_cache_bytes": (SZ, [cfgp]),
        "kv_cache_init": (ctypes.c_int, [cachep, cfgp, P, SZ, P, P, P]),
        "kv_calibrate_scratch_bytes": (SZ, [cachep, I32, I32]),
        "kv_calibrate": (ctypes.c_int, [cachep, I32, P, P, I32, P, SZ, P]),
        "kv_quant_append": (ctypes.c_int, [cachep, I32, P, P, P, I32, I32, P]),
        "kv_decode_scratch_bytes": (SZ, [cachep, I32, I32]),
        "kv_decode_attention": (ctypes.c_int, [cachep, I32, P, P, P, I32, P, SZ, P]),
        "kv_decode_attention_noalloc": (ctypes.c_int, [cachep, I32, P, P, P, I32, P]),
        "kv_prefill_scratch_bytes": (SZ, [cachep, I32, I32]),
        "kv_prefill_attention": (ctypes.c_int, [cachep, I32, P, P, P, P, P, I32, I32, P, SZ, P]),
        "kv_tbq_block_bytes": (SZ, [I32]),
        "kv_tbq_encode": (ctypes.c_int, [I32, ctypes.c_uint64, P, I32, ctypes.c_int64, P, P]),
        "kv_tbq_decode": (ctypes.c_int, [I32, ctypes.c_uint64, P, ctypes.c_int64, P, P]),
        "kv_split_record_bytes": (SZ, [I32]),
        "kv_split_outliers": (ctypes.c_int, [P, I32, I32, I32, P, P]),
        "kv_split_encode": (ctypes.c_int, [I32, ctypes.c_uint64, P, I32, P, I32, ctypes.c_int64, P, P]),
        "kv_split_decode": (ctypes.c_int, [I32, ctypes.c_uint64, P, I32, P, ctypes.c_int64, P, P]),
        "kv_status": (ctypes.c_int, [cachep, U32P, P]),
        "kv_set_wait_limit_ns": (ctypes.c_int, [ctypes.c_uint64]),
        "kv_strerror": (ctypes.c_char_p, [ctypes.c_int]),
        "kv_rope_init": (ctypes.c_int, [ropep, I32, I32, F64, I32, F64, F64, F64, F64, F64]),
        "kv_qk_norm_rope": (ctypes.c_int, [ropep, P, I64, P, P, P, F32, P, P, P, I32, I32, I32, I32, I32, P]),
        "kv_tree_scratch_bytes": (SZ, [cachep, I32, I32, I32]),
        "kv_tree_attention": (ctypes.c_int, [cachep, I32, P, P, P, P, P, P, I32, I32, P, SZ, P]),
        "kv_tree_commit": (ctypes.c_int, [cachep, I32, P, P, P, P, P, I32, I32, I32, P]),
        "kv_weights_scratch_bytes": (SZ, [cachep, I32, I32, I32]),
        "kv_attention_weights": (ctypes.c_int, [cachep, I32, P, P, F32, P, I32, I32, P, SZ, P]),
        "kv_evict": (ctypes.c_int, [cachep, I32, P, P, P, P, I32, I32, I32, P]),
        "kv_pool_bytes": (SZ, [cachep]),
        "kv_pool_init": (ctypes.c_int, [cachep, P, SZ, P]),
        "kv_pool_reserve": (ctypes.c_int, [cachep, P, SZ, P, P, P, I32, I32, P]),
        "kv_pool_fork": (ctypes.c_int, [cachep, P, SZ, P, P, P, I32, P]),
        "kv_pool_release": (ctypes.c_int, [cachep, P, SZ, P, I32, P]),
        "kv_pool_compact": (ctypes.c_int, [cachep, P, SZ, P, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(rc: int):
    if rc != 0:
        raise KVQError(f"libkvq: {load().kv_strerror(rc).decode()} (code {rc})")


def _stream(stream=None) -> int:
    """The cudaStream_t of ``stream``, or of the current stream of the current device."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _ptr(t: torch.Tensor | None, device: int | None = None) -> int:
    """The address of a tensor on the device (on the cache's, where that is given: the library could not tell)."""
    if t is None:
        return 0
    if not t.is_cuda:
        raise KVQError("device tensor expected")
    if device is not None and t.get_device() != device:
        raise KVQError(f"tensor on device {t.get_device()}, the cache is on device {device} (code 1)")
    if not t.is_contiguous():
        raise KVQError("contiguous tensor expected")
    return t.data_ptr()


def _check_in_dtype(cache: kvq_cache, *tensors: torch.Tensor):
    """k, v, q and calibration blocks must have the cache's input dtype (cfg.in_dtype)."""
    want = torch.bfloat16 if cache.cfg.in_dtype == KVQ_IN_BF16 else torch.float32
    for t in tensors:
        if t.dtype != want:
            raise KVQError(f"input dtype {t.dtype} does not match the cache's in_dtype ({want})")


def _layers_in_call(cache: kvq_cache, layer: int) -> int:
    return cache.cfg.n_layers if layer == -1 else 1


def _check_shape(name: str, t: torch.Tensor, want: tuple):
    """The library reads and writes whole rows of these shapes from the bare pointer; a tensor of
    another size would be read or written past its end, which the C ABI cannot see."""
    if t.shape != want:
        raise KVQError(f"{name} has shape {tuple(t.shape)}, expected {tuple(want)}")


def _check_decode_shapes(cache: kvq_cache, layer: int, q: torch.Tensor, out: torch.Tensor,
                         seq_lens: torch.Tensor) -> int:
    """q and out [L?][B][Hq][128] (the layer axis present iff layer == -1), seq_lens [B]; returns B."""
    if q.dim() not in (3, 4) or q.dim() != (4 if layer == -1 else 3):
        raise KVQError(f"q must be {'[L][B][Hq][128]' if layer == -1 else '[B][Hq][128]'}, got {tuple(q.shape)}")
    B = q.shape[-3]
    lead = (_layers_in_call(cache, layer),) if layer == -1 else ()
    _check_shape("q", q, lead + (B, cache.cfg.n_q_heads, 128))
    _check_shape("out", out, tuple(q.shape))
    _check_shape("seq_lens", seq_lens, (B,))
    return B


def _check_append_shapes(cache: kvq_cache, layer: int, k: torch.Tensor, v: torch.Tensor,
                         pos: torch.Tensor) -> tuple:
    """k and v [L?][B][Hkv][T][128] (the layer axis present iff layer == -1), pos [B]; returns (B, T)."""
    if k.dim() != (5 if layer == -1 else 4):
        raise KVQError(f"k must be {'[L][B][Hkv][T][128]' if layer == -1 else '[B][Hkv][T][128]'}, "
                       f"got {tuple(k.shape)}")
    B, T = k.shape[-4], k.shape[-2]
    lead = (_layers_in_call(cache, layer),) if layer == -1 else ()
    _check_shape("k", k, lead + (B, cache.cfg.n_kv_heads, T, 128))
    _check_shape("v", v, tuple(k.shape))
    _check_shape("pos", pos, (B,))
    return B, T


def make_config(n_layers, n_kv_heads, n_q_heads, max_batch, max_seq_len, window=128, n_pages=0,
                k_format=KVQ_Q4G32, v_format=None, sinkhorn=False, in_dtype=KVQ_IN_BF16,
                seed=0) -> kvq_config:
    """A cache's configuration; v_format None is what goes with the keys' format (Q8B32 values with Q8B32 keys, else Q4G32)."""
    if v_format is None:
        v_format = KVQ_Q8B32 if k_format == KVQ_Q8B32 else KVQ_Q4G32
    return kvq_config(n_layers, n_kv_heads, n_q_heads, 128, max_batch, max_seq_len, window, 64,
                      n_pages, k_format, v_format, int(bool(sinkhorn)), 32, in_dtype, seed)


def kv_cache_bytes(cfg: kvq_config) -> int:
    return int(load().kv_cache_bytes(ctypes.byref(cfg)))


def kv_cache_init(cfg: kvq_config, dev_mem: torch.Tensor, block_table: torch.Tensor | None = None,
                  qjl_proj: np.ndarray | None = None, stream=None) -> kvq_cache:
    cache = kvq_cache()
    proj = None
    if qjl_proj is not None:
        proj = np.ascontiguousarray(qjl_proj, dtype=np.float32)
    pp = ctypes.c_void_p(proj.ctypes.data) if proj is not None else ctypes.c_void_p(0)
    _check(load().kv_cache_init(ctypes.byref(cache), ctypes.byref(cfg), _ptr(dev_mem),
                                dev_mem.numel() * dev_mem.element_size(), _ptr(block_table), pp,
                                _stream(stream)))
    return cache


def kv_calibrate_scratch_bytes(cache: kvq_cache, layer: int, n_tokens: int) -> int:
    return int(load().kv_calibrate_scratch_bytes(ctypes.byref(cache), layer, n_tokens))


def kv_calibrate(cache: kvq_cache, layer: int, k_calib: torch.Tensor, v_calib: torch.Tensor,
                 scratch: torch.Tensor, stream=None):
    _check_in_dtype(cache, k_calib, v_calib)
    n_tokens = k_calib.shape[-2]
    lead = (_layers_in_call(cache, layer),) if layer == -1 else ()
    _check_shape("k_calib", k_calib, lead + (cache.cfg.n_kv_heads, n_tokens, 128))
    _check_shape("v_calib", v_calib, tuple(k_calib.shape))
    dev = cache.device
    _check(load().kv_calibrate(ctypes.byref(cache), layer, _ptr(k_calib, dev), _ptr(v_calib, dev), n_tokens,
                               _ptr(scratch, dev), scratch.numel() * scratch.element_size(),
                               _stream(stream)))


def kv_quant_append(cache: kvq_cache, layer: int, k: torch.Tensor, v: torch.Tensor,
                    pos: torch.Tensor, stream=None):
    """k, v: [L?][B][Hkv][T][128]; pos: int32 [B] on the device."""
    if pos.dtype != torch.int32:
        raise KVQError("pos must be int32")
    _check_in_dtype(cache, k, v)
    B, T = _check_append_shapes(cache, layer, k, v, pos)
    dev = cache.device
    _check(load().kv_quant_append(ctypes.byref(cache), layer, _ptr(k, dev), _ptr(v, dev), _ptr(pos, dev), B, T,
                                  _stream(stream)))


def kv_decode_scratch_bytes(cache: kvq_cache, layer: int, batch: int) -> int:
    return int(load().kv_decode_scratch_bytes(ctypes.byref(cache), layer, batch))


def kv_decode_attention(cache: kvq_cache, layer: int, q: torch.Tensor, out: torch.Tensor,
                        seq_lens: torch.Tensor, scratch: torch.Tensor, stream=None):
    """q: [L?][B][Hq][128]; out: float32 like q; seq_lens: int32 [B]; scratch: device bytes (any
    contents), at least kv_decode_scratch_bytes."""
    if seq_lens.dtype != torch.int32 or out.dtype != torch.float32:
        raise KVQError("seq_lens must be int32 and out float32")
    _check_in_dtype(cache, q)
    B = _check_decode_shapes(cache, layer, q, out, seq_lens)
    dev = cache.device
    _check(load().kv_decode_attention(ctypes.byref(cache), layer, _ptr(q, dev), _ptr(out, dev), _ptr(seq_lens, dev),
                                      B, _ptr(scratch, dev), scratch.numel() * scratch.element_size(),
                                      _stream(stream)))


def kv_decode_attention_noalloc(cache: kvq_cache, layer: int, q: torch.Tensor, out: torch.Tensor,
                                seq_lens: torch.Tensor, stream=None):
    """Decode without a caller scratch buffer: the library's own fixed device array is used (for
    callers that cannot allocate).  Same shapes as kv_decode_attention."""
    if seq_lens.dtype != torch.int32 or out.dtype != torch.float32:
        raise KVQError("seq_lens must be int32 and out float32")
    _check_in_dtype(cache, q)
    B = _check_decode_shapes(cache, layer, q, out, seq_lens)
    dev = cache.device
    _check(load().kv_decode_attention_noalloc(ctypes.byref(cache), layer, _ptr(q, dev), _ptr(out, dev),
                                              _ptr(seq_lens, dev), B, _stream(stream)))


def kv_prefill_scratch_bytes(cache: kvq_cache, layer: int, batch: int) -> int:
    return int(load().kv_prefill_scratch_bytes(ctypes.byref(cache), layer, batch))


def kv_prefill_attention(cache: kvq_cache, layer: int, k: torch.Tensor, v: torch.Tensor, q: torch.Tensor,
                         out: torch.Tensor, pos: torch.Tensor, scratch: torch.Tensor, stream=None):
    """Append a chunk and attend its queries.  k, v: [L?][B][Hkv][T][128]; q: [L?][B][Hq][T][128];
    out: float32 like q; pos: int32 [B]; scratch: device bytes, at least kv_prefill_scratch_bytes."""
    if pos.dtype != torch.int32 or out.dtype != torch.float32:
        raise KVQError("pos must be int32 and out float32")
    _check_in_dtype(cache, k, v, q)
    B, T = _check_append_shapes(cache, layer, k, v, pos)
    lead = (_layers_in_call(cache, layer),) if layer == -1 else ()
    _check_shape("q", q, lead + (B, cache.cfg.n_q_heads, T, 128))
    _check_shape("out", out, tuple(q.shape))
    dev = cache.device
    _check(load().kv_prefill_attention(ctypes.byref(cache), layer, _ptr(k, dev), _ptr(v, dev), _ptr(q, dev),
                                       _ptr(out, dev), _ptr(pos, dev), B, T, _ptr(scratch, dev),
                                       scratch.numel() * scratch.element_size(), _stream(stream)))


def kv_rope_init(rot_dim: int, layout: int = ROPE_HALF, theta: float = 10000.0, scaling: int = ROPE_PLAIN,
                 factor: float = 1.0, original_len: float = 0.0, low: float = 0.0, high: float = 0.0,
                 attn_factor: float = 1.0) -> kvq_rope:
    """The rotary positions' handle (host data; see include/kvq.h for the scalings)."""
    rope = kvq_rope()
    _check(load().kv_rope_init(ctypes.byref(rope), rot_dim, layout, theta, scaling, factor, original_len, low, high,
                               attn_factor))
    return rope


def kv_qk_norm_rope(rope: kvq_rope, qkv: torch.Tensor, positions: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                    v: torch.Tensor | None, q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                    eps: float = 1e-6, stream=None):
    """qkv: [B][T][>= (Hq + 2 Hkv) * 128] (rows of one stride; Hkv once less where v is None); positions: int32 [B][T];
    q: [B][Hq][T][128], k, v: [B][Hkv][T][128] (written; without the T axis where T is 1, as kv_decode_attention takes
    q); weights [128], all of qkv's dtype."""
    dt = _in_dtype_of(qkv)
    if qkv.dim() != 3 or positions.dtype != torch.int32:
        raise KVQError("qkv must be [B][T][row] and positions int32")
    B, T, row = qkv.shape
    sb, st, s1 = qkv.stride()
    if row > 1 and s1 != 1 or T > 1 and B > 1 and sb != T * st:
        raise KVQError("qkv's rows must be contiguous and of one stride")
    if q.dim() != 4 and not (T == 1 and q.dim() == 3) or k.dim() != q.dim():
        raise KVQError(f"q and k must be [B][heads][T][128], got {tuple(q.shape)} and {tuple(k.shape)}")
    hq, hkv = q.shape[1], k.shape[1]
    tail = (T, 128) if q.dim() == 4 else (128,)
    _check_shape("q", q, (B, hq) + tail)
    _check_shape("k", k, (B, hkv) + tail)
    _check_shape("positions", positions, (B, T))
    if v is not None:
        _check_shape("v", v, tuple(k.shape))
    need = (hq + (1 if v is None else 2) * hkv) * 128
    st = st if T > 1 else sb if B > 1 else need  # (a single row has no stride)
    if row < need:
        raise KVQError(f"qkv rows hold {row} values, fewer than their heads")
    for w in (q_weight, k_weight):
        if w is not None:
            _check_shape("weight", w, (128,))
    if not qkv.is_cuda:
        raise KVQError("device tensor expected")
    device, dtype = torch.cuda.current_device(), qkv.dtype  # (there is no cache whose device the library would check)
    if qkv.get_device() != device or positions.get_device() != device:
        raise KVQError("tensors must be on the current device")
    for x in (q, k, v, q_weight, k_weight):
        if x is not None:
            if x.dtype != dtype:
                raise KVQError(f"dtype {x.dtype} does not match qkv's ({dtype})")
            if x.get_device() != device:
                raise KVQError("tensors must be on the current device")
    cuda_stream = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(device)
    _check(load().kv_qk_norm_rope(ctypes.byref(rope), qkv.data_ptr(), st, _ptr(positions), _ptr(q_weight), _ptr(k_weight),
                                  eps, _ptr(q), _ptr(k), _ptr(v), B, T, hq, hkv, dt, cuda_stream))


def kv_tree_scratch_bytes(cache: kvq_cache, layer: int, batch: int, n_nodes: int) -> int:
    return int(load().kv_tree_scratch_bytes(ctypes.byref(cache), layer, batch, n_nodes))


def kv_tree_attention(cache: kvq_cache, layer: int, k: torch.Tensor, v: torch.Tensor, q: torch.Tensor,
                      out: torch.Tensor, seq_lens: torch.Tensor, parents: torch.Tensor, scratch: torch.Tensor,
                      stream=None):
    """k, v: [L?][B][Hkv][N][128]; q: [L?][B][Hq][N][128]; out like q, in the cache's input dtype; seq_lens: int32 [B];
    parents: int32 [B][N]; scratch: device bytes, at least kv_tree_scratch_bytes."""
    if seq_lens.dtype != torch.int32 or parents.dtype != torch.int32:
        raise KVQError("seq_lens and parents must be int32")
    _check_in_dtype(cache, k, v, q, out)
    B, N = _check_append_shapes(cache, layer, k, v, seq_lens)
    lead = (_layers_in_call(cache, layer),) if layer == -1 else ()
    _check_shape("q", q, lead + (B, cache.cfg.n_q_heads, N, 128))
    _check_shape("out", out, tuple(q.shape))
    _check_shape("parents", parents, (B, N))
    dev = cache.device
    _check(load().kv_tree_attention(ctypes.byref(cache), layer, _ptr(k, dev), _ptr(v, dev), _ptr(q, dev),
                                    _ptr(out, dev), _ptr(seq_lens, dev), _ptr(parents, dev), B, N, _ptr(scratch, dev),
                                    scratch.numel() * scratch.element_size(), _stream(stream)))


def kv_tree_commit(cache: kvq_cache, layer: int, k: torch.Tensor, v: torch.Tensor, path: torch.Tensor,
                   n_accept: torch.Tensor, pos: torch.Tensor, stream=None):
    """k, v: [L?][B][Hkv][N][128] (the tree's); path: int32 [B][P] node indices; n_accept, pos: int32 [B]."""
    if path.dtype != torch.int32 or n_accept.dtype != torch.int32 or pos.dtype != torch.int32:
        raise KVQError("path, n_accept and pos must be int32")
    _check_in_dtype(cache, k, v)
    B, N = _check_append_shapes(cache, layer, k, v, pos)
    if path.dim() != 2 or path.shape[0] != B:
        raise KVQError(f"path must be [{B}][max_path], got {tuple(path.shape)}")
    _check_shape("n_accept", n_accept, (B,))
    dev = cache.device
    _check(load().kv_tree_commit(ctypes.byref(cache), layer, _ptr(k, dev), _ptr(v, dev), _ptr(path, dev),
                                 _ptr(n_accept, dev), _ptr(pos, dev), B, N, path.shape[1], _stream(stream)))


def kv_weights_scratch_bytes(cache: kvq_cache, layer: int, batch: int, n_queries: int) -> int:
    return int(load().kv_weights_scratch_bytes(ctypes.byref(cache), layer, batch, n_queries))


def _check_weights(cache: kvq_cache, layer: int, batch: int, weights: torch.Tensor):
    lead = (_layers_in_call(cache, layer),) if layer == -1 else ()
    if weights.dtype != torch.float32:
        raise KVQError("weights must be float32")
    _check_shape("weights", weights, lead + (batch, cache.cfg.n_kv_heads, cache.cfg.max_seq_len))


def kv_attention_weights(cache: kvq_cache, layer: int, q: torch.Tensor, weights: torch.Tensor, decay: float,
                         seq_lens: torch.Tensor, scratch: torch.Tensor, stream=None):
    """q: [L?][B][Hq][T][128], the newest T tokens' queries; weights: float32 [L?][B][Hkv][max_seq_len] (updated);
    seq_lens: int32 [B]; scratch: device bytes, at least kv_weights_scratch_bytes."""
    if seq_lens.dtype != torch.int32:
        raise KVQError("seq_lens must be int32")
    _check_in_dtype(cache, q)
    if q.dim() != (5 if layer == -1 else 4):
        raise KVQError(f"q must be {'[L][B][Hq][T][128]' if layer == -1 else '[B][Hq][T][128]'}, got {tuple(q.shape)}")
    B, T = q.shape[-4], q.shape[-2]
    lead = (_layers_in_call(cache, layer),) if layer == -1 else ()
    _check_shape("q", q, lead + (B, cache.cfg.n_q_heads, T, 128))
    _check_shape("seq_lens", seq_lens, (B,))
    _check_weights(cache, layer, B, weights)
    dev = cache.device
    _check(load().kv_attention_weights(ctypes.byref(cache), layer, _ptr(q, dev), _ptr(weights, dev), decay,
                                       _ptr(seq_lens, dev), B, T, _ptr(scratch, dev),
                                       scratch.numel() * scratch.element_size(), _stream(stream)))


def kv_evict(cache: kvq_cache, layer: int, weights: torch.Tensor, seq_lens: torch.Tensor, kept: torch.Tensor,
             new_lens: torch.Tensor, budget: int, recent: int, stream=None):
    """weights: float32 [L?][B][Hkv][max_seq_len] (compacted); seq_lens: int32 [B]; kept: int32 [L?][B][Hkv][budget] and
    new_lens: int32 [B] (written)."""
    if seq_lens.dtype != torch.int32 or kept.dtype != torch.int32 or new_lens.dtype != torch.int32:
        raise KVQError("seq_lens, kept and new_lens must be int32")
    B = seq_lens.shape[0] if seq_lens.dim() == 1 else -1
    _check_shape("seq_lens", seq_lens, (B,))
    _check_shape("new_lens", new_lens, (B,))
    _check_weights(cache, layer, B, weights)
    _check_shape("kept", kept, tuple(weights.shape[:-1]) + (budget,))
    dev = cache.device
    _check(load().kv_evict(ctypes.byref(cache), layer, _ptr(weights, dev), _ptr(seq_lens, dev), _ptr(kept, dev),
                           _ptr(new_lens, dev), B, budget, recent, _stream(stream)))


def kv_pool_bytes(cache: kvq_cache) -> int:
    return int(load().kv_pool_bytes(ctypes.byref(cache)))


def _pool(cache: kvq_cache, pool: torch.Tensor, *ints: torch.Tensor) -> list:
    """The cache, the pool's address and size and the addresses of the call's int32 [batch] tensors, after checks of all."""
    dev = cache.device
    args = [ctypes.byref(cache), _ptr(pool, dev), pool.numel() * pool.element_size()]
    shape = (ints[0].numel(),) if ints else ()
    for t in ints:
        # (one test where all is well: these calls are a few microseconds long)
        if t.dtype is not torch.int32 or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
            if t.dtype is not torch.int32:
                raise KVQError("the pool's arguments are int32 tensors")
            _check_shape("argument", t, shape)
            _ptr(t, dev)
        args.append(t.data_ptr())
    return args


def kv_pool_init(cache: kvq_cache, pool: torch.Tensor, stream=None):
    """pool: device bytes, at least kv_pool_bytes; the cache's block table (all of it) becomes -1."""
    _check(load().kv_pool_init(*_pool(cache, pool), _stream(stream)))


def kv_pool_reserve(cache: kvq_cache, pool: torch.Tensor, pos: torch.Tensor, n_tokens, granted: torch.Tensor, stream=None):
    """pos, granted (written; may be pos): int32 [B]; n_tokens: one number, or int32 [B] on the device."""
    if isinstance(n_tokens, torch.Tensor):
        c, at, size, p, out, counts = _pool(cache, pool, pos, granted, n_tokens)
        n_tokens = 0
    else:
        c, at, size, p, out = _pool(cache, pool, pos, granted)
        counts = 0
    _check(load().kv_pool_reserve(c, at, size, p, counts, out, pos.numel(), n_tokens, _stream(stream)))


def kv_pool_fork(cache: kvq_cache, pool: torch.Tensor, parents: torch.Tensor, seq_lens: torch.Tensor,
                 new_lens: torch.Tensor, stream=None):
    """parents, seq_lens, new_lens (written): int32 [B]."""
    _check(load().kv_pool_fork(*_pool(cache, pool, parents, seq_lens, new_lens), parents.numel(), _stream(stream)))


def kv_pool_release(cache: kvq_cache, pool: torch.Tensor, keep_lens: torch.Tensor, stream=None):
    """keep_lens: int32 [B]."""
    _check(load().kv_pool_release(*_pool(cache, pool, keep_lens), keep_lens.numel(), _stream(stream)))


def kv_pool_compact(cache: kvq_cache, pool: torch.Tensor, n_used: torch.Tensor, stream=None):
    """n_used: int32 [1] (written)."""
    args = _pool(cache, pool, n_used)
    if n_used.numel() != 1:
        raise KVQError("n_used must be int32 [1]")
    _check(load().kv_pool_compact(*args, _stream(stream)))


def _in_dtype_of(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return KVQ_IN_BF16
    if t.dtype == torch.float32:
        return KVQ_IN_F32
    raise KVQError(f"float32 or bfloat16 input expected, got {t.dtype}")


def kv_tbq_block_bytes(bits: int) -> int:
    return int(load().kv_tbq_block_bytes(bits))


def kv_tbq_encode(bits: int, seed: int, x: torch.Tensor, blocks: torch.Tensor, stream=None):
    """x: [..., 256] float32/bf16 (n_blocks = numel / 256); blocks: uint8 [n_blocks][98 or 130]."""
    nb = x.numel() // 256
    if x.shape[-1] != 256 or blocks.dtype != torch.uint8 or blocks.numel() != nb * kv_tbq_block_bytes(bits):
        raise KVQError("x must be [..., 256] and blocks uint8 of n_blocks * kv_tbq_block_bytes(bits) bytes")
    _check(load().kv_tbq_encode(bits, seed, _ptr(x), _in_dtype_of(x), nb, _ptr(blocks), _stream(stream)))


def kv_tbq_decode(bits: int, seed: int, blocks: torch.Tensor, out: torch.Tensor, stream=None):
    """blocks: uint8 [n_blocks][98 or 130]; out: float32 [..., 256] with n_blocks * 256 values."""
    nb = out.numel() // 256
    if out.dtype != torch.float32 or out.shape[-1] != 256 or blocks.numel() != nb * kv_tbq_block_bytes(bits):
        raise KVQError("out must be float32 [..., 256] and blocks n_blocks * kv_tbq_block_bytes(bits) bytes")
    _check(load().kv_tbq_decode(bits, seed, _ptr(blocks), nb, _ptr(out), _stream(stream)))


def kv_split_record_bytes(hi_bits: int) -> int:
    return int(load().kv_split_record_bytes(hi_bits))


def kv_split_outliers(calib: torch.Tensor, outliers: torch.Tensor, stream=None):
    """calib: [n_sets][n_tokens][128] float32/bf16; outliers: int16 [n_sets][64] (written)."""
    if calib.dim() != 3 or calib.shape[-1] != 128 or outliers.dtype != torch.int16:
        raise KVQError("calib must be [n_sets][n_tokens][128] and outliers int16")
    _check_shape("outliers", outliers, (calib.shape[0], 64))
    _check(load().kv_split_outliers(_ptr(calib), _in_dtype_of(calib), calib.shape[0], calib.shape[1],
                                    _ptr(outliers), _stream(stream)))


def kv_split_encode(hi_bits: int, seed: int, outliers: torch.Tensor, x: torch.Tensor, records: torch.Tensor,
                    stream=None):
    """x: [n_sets][...][128]; records: uint8 [n_vectors][44 or 60]; outliers: int16 [n_sets][64]."""
    n_sets = outliers.shape[0]
    nv = x.numel() // 128
    if x.shape[0] != n_sets or x.shape[-1] != 128 or records.numel() != nv * kv_split_record_bytes(hi_bits):
        raise KVQError("x must be [n_sets][...][128] and records n_vectors * kv_split_record_bytes bytes")
    _check(load().kv_split_encode(hi_bits, seed, _ptr(outliers), n_sets, _ptr(x), _in_dtype_of(x), nv,
                                  _ptr(records), _stream(stream)))


def kv_split_decode(hi_bits: int, seed: int, outliers: torch.Tensor, records: torch.Tensor, out: torch.Tensor,
                    stream=None):
    n_sets = outliers.shape[0]
    nv = out.numel() // 128
    if out.dtype != torch.float32 or out.shape[0] != n_sets or records.numel() != nv * kv_split_record_bytes(hi_bits):
        raise KVQError("out must be float32 [n_sets][...][128] and records n_vectors * kv_split_record_bytes bytes")
    _check(load().kv_split_decode(hi_bits, seed, _ptr(outliers), n_sets, _ptr(records), nv, _ptr(out),
                                  _stream(stream)))


def kv_status(cache: kvq_cache, stream=None) -> int:
    v = ctypes.c_uint32(0)
    _check(load().kv_status(ctypes.byref(cache), ctypes.byref(v), _stream(stream)))
    return int(v.value)


def kv_set_wait_limit_ns(ns: int) -> None:
    """Stall limit (ns, 1..1e10) of waits within later decode, tree, weights and fork calls and prefills over 8-bit blocks; the default
    is 1e9 (see include/kvq.h)."""
    _check(load().kv_set_wait_limit_ns(int(ns)))


def kv_strerror(code: int) -> str:
    return load().kv_strerror(code).decode()

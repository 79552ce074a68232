// Queries and keys out of a fused projection: per-head RMS norm, rotary position and the cache's layouts,
// in one pass over the rows.
//
// Per head vector x of 128 channels: y = x / sqrt(mean(x^2) + eps) * w (where a norm weight is given), then
// every pair (y_a, y_b) of the first rot_dim channels turns by the angle pos f_i:
//   (y_a cos - y_b sin, y_b cos + y_a sin), pairs (i, i + rot_dim / 2) or (2i, 2i + 1);
// everything in fp32, rounded once to the output type.
//
// Angles: f_i / (2 pi) is kept as a 64-bit binary fraction of a turn, so pos * f_i modulo one turn is the
// wrapping 64-bit product, exact at any position and without fp64 instructions.  The fraction comes from a
// double: the angle is good to pos * 2^-54 turns (at position 2^20 6e-11 of a turn), where an fp32 product at
// position 100,000 is off by 0.01 rad.  It goes to fp32 (2^-24 relative, under 2e-7 rad) and through sincospi.
//
// Bound by memory: every value is read once and written once.  Eight lanes hold a head, each two 16-byte
// blocks of 8 channels chosen so that both members of a pair sit in one lane (blocks l and l + rot_dim / 16
// for halves, 2 l and 2 l + 1 for adjacent pairs): no exchange but the three steps of the norm's sum.
// rot_dim not a multiple of 16 with halves reads the partner channels again (from L1).  The sines of a
// token are computed once per CTA for all its heads.
// Measured, bf16: 8192 tokens of 48 heads (201 MB) 39.9 us, 5.05 TB/s, 74 % of the copy rate (keeping the next
// head's loads under way took registers, with them CTAs, and 57 us); 8 tokens 3.1 us on the device (one of many
// in a graph), one trip through memory, and 10.4 a call, the host's.
#include <cmath>

#include "kvq_internal.cuh"

namespace kvq {

namespace {

constexpr int THREADS = 256;
constexpr int GROUPS = THREADS / 8;  // heads in flight per CTA
constexpr int TPC_MAX = 4;           // tokens per CTA

struct RopeArgs {
  const void* x;
  int64_t row_stride;  // elements
  const int32_t* pos;
  const void* wq;
  const void* wk;
  void* q;
  void* k;
  void* v;
  int T, Hq, Hkv, jobs, rows, rot;  // jobs: head vectors per row
  float eps, attn;
  uint64_t turns[D / 2];
};

enum { IN_LANE, ADJACENT, REREAD };

// place of a pair's sine and cosine in shared memory: eight lanes, each with eight consecutive pairs, read without conflicts
__device__ __forceinline__ int cs_at(int pair) { return (pair & 7) * 8 + (pair >> 3); }

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
// two running sums of squares
__device__ __forceinline__ void fma2_acc(float& s0, float& s1, float x0, float x1) {
  float a0 = x0, a1 = x1;
  fma2(a0, a1, x0, x1, s0, s1);
  s0 = a0;
  s1 = a1;
}
__device__ __forceinline__ void store8v(__nv_bfloat16* p, const float (&v)[8]) {
  uint4 u;
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  u.x = *reinterpret_cast<uint32_t*>(&h[0]);
  u.y = *reinterpret_cast<uint32_t*>(&h[1]);
  u.z = *reinterpret_cast<uint32_t*>(&h[2]);
  u.w = *reinterpret_cast<uint32_t*>(&h[3]);
  *reinterpret_cast<uint4*>(p) = u;
}
__device__ __forceinline__ void store8v(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(float x) { return x; }

template <typename T, int MODE>
__global__ void __launch_bounds__(THREADS) norm_rope_kernel(const __grid_constant__ RopeArgs a, int tpc) {
  __shared__ float2 cs[TPC_MAX][D / 2];
  __shared__ int2 tok_sh[TPC_MAX];  // sequence and token of each row; token < 0: a padded row
  const int tid = threadIdx.x;
  const int row0 = blockIdx.x * tpc, nrow = min(tpc, a.rows - row0);
  const int half = a.rot >> 1;
  for (int i = tid; i < nrow * (D / 2); i += THREADS) {
    const int r = i / (D / 2), c = i % (D / 2), p = a.pos[row0 + r];
    if (c == 0) {
      const int b = (row0 + r) / a.T;
      tok_sh[r] = make_int2(b, p < 0 ? -1 : row0 + r - b * a.T);
    }
    if (c < half) {
      const long long turn = (long long)((uint64_t)(uint32_t)p * a.turns[c]);  // modulo one turn, signed
      float s, co;
      sincospif(__ll2float_rn(turn) * 1.0842021724855044e-19f, &s, &co);     // 2^-63: half turns
      cs[r][cs_at(c)] = make_float2(co * a.attn, s * a.attn);
    }
  }
  __syncthreads();
  const int l = tid & 7;
  const int nb = a.rot >> 4;  // IN_LANE: blocks of 8 channels in each half
  const int b0 = MODE == IN_LANE ? (l < nb ? l : 2 * l) : 2 * l;
  const int b1 = MODE == IN_LANE && l < nb ? l + nb : b0 + 1;
  const unsigned grp_mask = 0xffu << (tid & 24);
  const T* row = static_cast<const T*>(a.x) + (int64_t)row0 * a.row_stride;
  int r = 0, hd = tid >> 3;  // this group's row and head vector
  while (true) {
    while (hd >= a.jobs) {
      hd -= a.jobs;
      row += a.row_stride;
      ++r;
    }
    if (r >= nrow) break;
    const T* src = row + hd * D;
    float x[16];
    load8(src + 8 * b0, *reinterpret_cast<float(*)[8]>(x));
    load8(src + 8 * b1, *reinterpret_cast<float(*)[8]>(x + 8));
    const int kind = hd < a.Hq ? 0 : hd < a.Hq + a.Hkv ? 1 : 2;
    const int2 tok = tok_sh[r];
    const int heads = kind == 0 ? a.Hq : a.Hkv, hh = hd - (kind == 0 ? 0 : kind == 1 ? a.Hq : a.Hq + a.Hkv);
    T* dst = static_cast<T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) + (((int64_t)tok.x * heads + hh) * a.T + max(tok.y, 0)) * D;
    if (kind < 2) {
      const T* w = static_cast<const T*>(kind == 0 ? a.wq : a.wk);
      const bool norm = w != nullptr;
      float inv = 1.f;
      if (norm) {
        // (the eight lanes of a head take part together; heads of one warp may differ in kind)
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < 16; i += 2) fma2_acc(s0, s1, x[i], x[i + 1]);
        float ss = s0 + s1;
        ss += __shfl_xor_sync(grp_mask, ss, 1);
        ss += __shfl_xor_sync(grp_mask, ss, 2);
        ss += __shfl_xor_sync(grp_mask, ss, 4);
        inv = rsqrtf(ss * (1.f / D) + a.eps);
        float w0[8], w1[8];
        load8(w + 8 * b0, w0);
        load8(w + 8 * b1, w1);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          mul2(w0[i], w0[i + 1], inv, inv);
          mul2(w1[i], w1[i + 1], inv, inv);
          mul2(x[i], x[i + 1], w0[i], w0[i + 1]);
          mul2(x[8 + i], x[9 + i], w1[i], w1[i + 1]);
        }
      }
      const float2* c = cs[r];
      if (MODE == IN_LANE) {
        if (l < nb) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 f = c[i * 8 + l];
            const float u = x[i], v = x[8 + i];
            x[i] = u * f.x - v * f.y;
            x[8 + i] = v * f.x + u * f.y;
          }
        }
      } else if (MODE == ADJACENT) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (8 * l + i < half) {
            const float2 f = c[i * 8 + l];
            const float u = x[2 * i], v = x[2 * i + 1];
            x[2 * i] = u * f.x - v * f.y;
            x[2 * i + 1] = v * f.x + u * f.y;
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int ch = 8 * (e < 8 ? b0 : b1) + (e & 7);
          if (ch < a.rot) {
            const bool first = ch < half;
            const int mate = first ? ch + half : ch - half;
            float m = to_f(src[mate]);
            if (norm) m *= inv * to_f(w[mate]);
            const float2 f = c[cs_at(first ? ch : mate)];
            x[e] = first ? x[e] * f.x - m * f.y : x[e] * f.x + m * f.y;
          }
        }
      }
    }
    if (tok.y >= 0) {
      store8v(dst + 8 * b0, *reinterpret_cast<float(*)[8]>(x));
      store8v(dst + 8 * b1, *reinterpret_cast<float(*)[8]>(x + 8));
    }
    hd += GROUPS;
  }
}

template <typename T>
cudaError_t launch(const RopeArgs& a, int mode, cudaStream_t s) {
  // A token a CTA while there are hardly more of them than run at once (8 an SM); more tokens go four to a CTA, which share
  // the sines' set-up.  On the device, 48 heads: 8 tokens 3.1 us, four to a CTA 5.8; 1216 6.8 and 7.2; 1300 7.0 and 8.3; 1800
  // 9.2 and 8.4; 2431 11.6 and 9.8.
  const int tpc = a.rows > 10 * 152 ? TPC_MAX : 1;
  const unsigned grid = (unsigned)((a.rows + tpc - 1) / tpc);
  if (mode == IN_LANE) norm_rope_kernel<T, IN_LANE><<<grid, THREADS, 0, s>>>(a, tpc);
  else if (mode == ADJACENT) norm_rope_kernel<T, ADJACENT><<<grid, THREADS, 0, s>>>(a, tpc);
  else norm_rope_kernel<T, REREAD><<<grid, THREADS, 0, s>>>(a, tpc);
  return cudaGetLastError();
}

constexpr uint32_t ROPE_MAGIC = 0x4b565152u;  // "KVQR"
constexpr double TWO_PI = 6.283185307179586476925286766559;

// Rotations per position of pair i, scaled for contexts longer than the trained one.
bool pair_turns(int rot, double theta, int scaling, double factor, double n0, double low, double high, double* out) {
  if (scaling == KVQ_ROPE_NTK) theta *= std::pow(factor, (double)rot / (rot - 2));
  const auto at = [&](double turns) { return rot * std::log(n0 / (turns * TWO_PI)) / (2 * std::log(theta)); };
  double first = 0, last = 0;
  if (scaling == KVQ_ROPE_DIMS) {
    first = std::fmax(std::floor(at(high)), 0.0);
    last = std::fmin(std::ceil(at(low)), (double)rot - 1);
  }
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / rot);
    if (scaling == KVQ_ROPE_LINEAR) f /= factor;
    if (scaling == KVQ_ROPE_TURNS || scaling == KVQ_ROPE_DIMS) {
      double keep;
      if (scaling == KVQ_ROPE_TURNS) keep = (n0 * f / TWO_PI - low) / (high - low);
      else keep = 1.0 - std::fmin(1.0, std::fmax(0.0, (i - first) / std::fmax(last - first, 0.001)));
      keep = std::fmin(1.0, std::fmax(0.0, keep));
      f = f * keep + f / factor * (1.0 - keep);
    }
    out[i] = f / TWO_PI;
    if (!std::isfinite(out[i])) return false;
  }
  return true;
}

}  // namespace

}  // namespace kvq

using namespace kvq;

extern "C" {

int kv_rope_init(kvq_rope* rope, int32_t rot_dim, int32_t layout, double theta, int32_t scaling, double factor,
                 double original_len, double low, double high, double attn_factor) {
  if (!rope) return KVQ_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim > D || rot_dim % 2 != 0) return KVQ_ERR_UNSUPPORTED;
  if (layout != KVQ_ROPE_HALF && layout != KVQ_ROPE_INTERLEAVED) return KVQ_ERR_UNSUPPORTED;
  if (scaling < KVQ_ROPE_PLAIN || scaling > KVQ_ROPE_DIMS) return KVQ_ERR_UNSUPPORTED;
  if (!(theta > 1.0) || !std::isfinite(theta) || !(attn_factor > 0.0) || !std::isfinite(attn_factor))
    return KVQ_ERR_INVALID_ARG;
  if (scaling != KVQ_ROPE_PLAIN && (!(factor > 0.0) || !std::isfinite(factor))) return KVQ_ERR_INVALID_ARG;
  if (scaling == KVQ_ROPE_NTK && rot_dim == 2) return KVQ_ERR_UNSUPPORTED;
  if (scaling >= KVQ_ROPE_TURNS &&
      (!(original_len > 0.0) || !(low > 0.0) || !(high > low) || !std::isfinite(high) || !std::isfinite(original_len)))
    return KVQ_ERR_INVALID_ARG;
  double t[D / 2] = {};
  if (!pair_turns(rot_dim, theta, scaling, factor, original_len, low, high, t)) return KVQ_ERR_INVALID_ARG;
  kvq_rope r = {};
  r.rot_dim = rot_dim;
  r.layout = layout;
  r.attn_factor = (float)attn_factor;
  // whole turns fall away (positions are whole numbers); 2^64 fractions of the rest, the low bits of a
  // double being exact there
  for (int i = 0; i < rot_dim / 2; ++i) r.turns[i] = (uint64_t)std::floor((t[i] - std::floor(t[i])) * 18446744073709551616.0);
  r.magic = ROPE_MAGIC;
  *rope = r;
  return KVQ_OK;
}

int kv_qk_norm_rope(const kvq_rope* rope, const void* qkv, int64_t row_stride, const int32_t* positions,
                    const void* q_weight, const void* k_weight, float eps, void* q, void* k, void* v, int32_t batch,
                    int32_t n_tokens, int32_t n_q_heads, int32_t n_kv_heads, int32_t in_dtype, void* stream) {
  if (!rope || !qkv || !positions || !q || !k) return KVQ_ERR_INVALID_ARG;
  if (rope->magic != ROPE_MAGIC) return KVQ_ERR_NOT_INIT;
  if (in_dtype != KVQ_IN_F32 && in_dtype != KVQ_IN_BF16) return KVQ_ERR_UNSUPPORTED;
  if (batch < 1 || n_tokens < 1 || n_q_heads < 1 || n_kv_heads < 1 || n_q_heads > 65536 || n_kv_heads > 65536)
    return KVQ_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return KVQ_ERR_INVALID_ARG;
  const int64_t jobs = (int64_t)n_q_heads + n_kv_heads + (v ? n_kv_heads : 0);
  if (row_stride < jobs * D || (int64_t)batch * n_tokens > 0x7fffffff - TPC_MAX) return KVQ_ERR_INVALID_ARG;
  const auto mis = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; };
  const int esize = in_dtype == KVQ_IN_BF16 ? 2 : 4;
  if (mis(qkv) || mis(positions) || mis(q_weight) || mis(k_weight) || mis(q) || mis(k) || mis(v) ||
      (row_stride * esize) % 16 != 0)
    return KVQ_ERR_ALIGN;
  RopeArgs a = {};
  a.x = qkv;
  a.row_stride = row_stride;
  a.pos = positions;
  a.wq = q_weight;
  a.wk = k_weight;
  a.q = q;
  a.k = k;
  a.v = v;
  a.T = n_tokens;
  a.Hq = n_q_heads;
  a.Hkv = n_kv_heads;
  a.jobs = (int)jobs;
  a.rows = batch * n_tokens;
  a.rot = rope->rot_dim;
  a.eps = eps;
  a.attn = rope->attn_factor;
  for (int i = 0; i < D / 2; ++i) a.turns[i] = rope->turns[i];
  const int mode = rope->layout == KVQ_ROPE_INTERLEAVED ? ADJACENT : a.rot % 16 == 0 ? IN_LANE : REREAD;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = in_dtype == KVQ_IN_BF16 ? launch<__nv_bfloat16>(a, mode, s) : launch<float>(a, mode, s);
  return call_status(e);
}

}  // extern "C"

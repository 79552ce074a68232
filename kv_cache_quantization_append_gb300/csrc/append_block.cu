// Append to a KVQ_Q8B32 cache: 8-bit codes of keys and values with one float scale for each block of 32 tokens of a
// (layer, sequence, kv-head).
//
//   y = c H (s . x) [/ sigma],  d = max over the block's 32 x 128 values of |y| / 127,  code = clamp(rint(y / d), -127, 127)
//
// The rotation spreads a vector's outlier channels over all of them ([KV] TLDR, [TQ] "key idea" row), which is what makes
// one scale enough.  A block's scale is known when its last token is: the block is coded then, once, from the call's own
// vectors and the ring's raw ones of earlier calls, so no code is ever scaled anew and a bulk append writes the bytes
// of per-token ones ([QC] v3.2 note).  Until then its tokens are read raw: the window (at least 32) covers them.
//
// One CTA per block that the call touches and per keys or values.  Four lanes hold a token, 32 channels each (the
// butterfly's stages 1 .. 16 stay in a lane, 32 and 64 are one shuffle a value); each warp's eight tokens are those that
// share 16-byte chunks of the stored order, so codes reach their places by few shuffles and whole 16-byte stores.  Every
// floating-point step is one IEEE operation in the order that the codec defines.
//
// Bound by latency: input or ring, rotation, the block's largest, codes.  2048 tokens of 8 heads (21 MB in and out, 3 us at the
// copy rate) take 12.6 us, 3 x 37 tokens of 2 heads 6.5; before a prefill its start overlaps the ring's copy.
#include "kvq_internal.cuh"

namespace kvq {

namespace {

constexpr int WARPS = 4;
constexpr float RINT_MAGIC = 12582912.0f;             // 1.5 * 2^23: x + this rounds x to an integer
constexpr float FAST_LIMIT = 0.5f - 6.103515625e-5f;  // 0.5 - 2^-14

__device__ __forceinline__ float max3nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t gather_low_bytes(uint32_t b0, uint32_t b1, uint32_t b2, uint32_t b3) {
  return __byte_perm(__byte_perm(b0, b1, 0x0040u), __byte_perm(b2, b3, 0x4000u), 0x7610u);
}

// 32 channels (from 32 G) of a raw vector
__device__ __forceinline__ void load32(const void* src, size_t off, bool bf16, float (&x)[32]) {
  if (bf16) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(src) + off);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 u = __ldcs(p + c);
      const uint32_t uu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[8 * c + 2 * e] = __uint_as_float(uu[e] << 16);
        x[8 * c + 2 * e + 1] = __uint_as_float(uu[e] & 0xffff0000u);
      }
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(src) + off);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float4 f = __ldcs(p + c);
      x[4 * c] = f.x;
      x[4 * c + 1] = f.y;
      x[4 * c + 2] = f.z;
      x[4 * c + 3] = f.w;
    }
  }
}
__device__ __forceinline__ void store32(float* dst, const float (&x)[32]) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    reinterpret_cast<float4*>(dst)[c] = make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
}

// codes + 128 of the lane's 32 values, four channels a word.  y / d is formed as y RN(1 / d), which is within 3.1e-5 of the
// IEEE quotient for magnitudes up to 127.5; where that lies within 2^-14 of a half-integer, or is larger (a scale that
// underflowed), the lane takes the IEEE quotients instead: every code is clamp(rint(RN(y / d)), -127, 127).
__device__ __forceinline__ void code32(const float (&x)[32], float d, uint32_t (&u8)[8]) {
  if (!(d > 0.0f)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) u8[j] = 0x80808080u;
    return;
  }
  const float inv = __frcp_rn(d);
  float off = 0.f, top = 0.f;  // (NaN if a quotient is)
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t tb[4];
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      float q0 = x[4 * j + e], q1 = x[4 * j + e + 1];
      mul2(q0, q1, inv, inv);
      top = max3nan(top, fabsf(q0), fabsf(q1));
      float t0 = q0, t1 = q1;
      add2(t0, t1, RINT_MAGIC, RINT_MAGIC);
      float n0 = RINT_MAGIC, n1 = RINT_MAGIC;
      sub2(n0, n1, t0, t1);
      add2(q0, q1, n0, n1);
      off = max3nan(off, fabsf(q0), fabsf(q1));
      tb[e] = __float_as_uint(t0);
      tb[e + 1] = __float_as_uint(t1);
    }
    // the low byte of t's bits is its code in two's complement; bit 7 flipped gives code + 128
    u8[j] = gather_low_bytes(tb[0], tb[1], tb[2], tb[3]) ^ 0x80808080u;
  }
  if (!(off <= FAST_LIMIT) || !(top < 127.5f)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t word = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = min(max(__float2int_rn(__fdiv_rn(x[4 * j + e], d)), -127), 127);
        word |= (uint32_t)(c + 128) << (8 * e);
      }
      u8[j] = word;
    }
  }
}

// Token (within its block) of lane group v of warp w.  Keys: the low and high eight of a 16-token tile pair up in a
// stored word, so a warp has four of each; values: the eight tokens of its 16-byte chunks, in their order there.
__device__ __forceinline__ int key_token(int w, int v) { return 16 * (w >> 1) + 4 * (w & 1) + (v & 3) + 8 * (v >> 2); }
__device__ __forceinline__ int value_token(int w, int v) { return 2 * w + (v & 1) + 8 * (v >> 1); }

__device__ __forceinline__ void store_keys(uint8_t* half, const uint32_t (&u8)[8], int w, int v, int G) {
  // word q = 2 ks + half of chunk i: channels 2i, 2i + 1 of its eight, of tokens r and r + 8.  u8[2q] holds i = 0, 1,
  // u8[2q + 1] i = 2, 3: the lane of token r stores the first two chunks, that of r + 8 the others
  const bool hi = v >> 2;
  uint32_t a[4], b[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t mine = hi ? u8[2 * q + 1] : u8[2 * q];
    const uint32_t part = __shfl_xor_sync(FULL, hi ? u8[2 * q] : u8[2 * q + 1], 16);
    const uint32_t lo8 = hi ? part : mine, hi8 = hi ? mine : part;
    a[q] = __byte_perm(lo8, hi8, 0x5410u);
    b[q] = __byte_perm(lo8, hi8, 0x7632u);
  }
  const int r = 4 * (w & 1) + (v & 3);
  uint4* dst = reinterpret_cast<uint4*>(half + (4 * (w >> 1) + G) * 512 + r * 64 + (hi ? 32 : 0));
  dst[0] = make_uint4(a[0], a[1], a[2], a[3]);
  dst[1] = make_uint4(b[0], b[1], b[2], b[3]);
}

__device__ __forceinline__ void store_values(uint8_t* half, const uint32_t (&u8)[8], int w, int v, int G) {
  // x[r]: channels r, r + 8, r + 16, r + 24 of the lane's 32
  uint32_t x[8];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const uint32_t a0 = __byte_perm(u8[p], u8[p + 2], 0x5140u), a1 = __byte_perm(u8[p], u8[p + 2], 0x7362u);
    const uint32_t b0 = __byte_perm(u8[p + 4], u8[p + 6], 0x5140u), b1 = __byte_perm(u8[p + 4], u8[p + 6], 0x7362u);
    x[4 * p] = __byte_perm(a0, b0, 0x5410u);
    x[4 * p + 1] = __byte_perm(a0, b0, 0x7632u);
    x[4 * p + 2] = __byte_perm(a1, b1, 0x5410u);
    x[4 * p + 3] = __byte_perm(a1, b1, 0x7632u);
  }
  // 8 x 8 transpose over the warp's tokens: afterwards lane v has x[t] = token t's channels of r = v
#pragma unroll
  for (int m = 1; m < 8; m <<= 1) {
    const bool up = v & m;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j & m) continue;
      const uint32_t got = __shfl_xor_sync(FULL, up ? x[j] : x[j + m], 4 * m);
      if (up) x[j] = got;
      else x[j + m] = got;
    }
  }
  uint32_t a[4], b[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {  // tokens 2q, 2q + 1 of the warp's eight
    a[q] = __byte_perm(x[2 * q], x[2 * q + 1], 0x5140u);
    b[q] = __byte_perm(x[2 * q], x[2 * q + 1], 0x7362u);
  }
  uint8_t* dst = half + 4096 + 2 * G * 512 + (4 * v + w) * 16;
  *reinterpret_cast<uint4*>(dst) = make_uint4(a[0], a[1], a[2], a[3]);
  *reinterpret_cast<uint4*>(dst + 512) = make_uint4(b[0], b[1], b[2], b[3]);
}

__global__ void __launch_bounds__(WARPS * 32) append_block_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ float most[WARPS];
  // a dependent decode launch may start its set-up now; it waits for this grid before reading
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, v = lane >> 2, G = lane & 3;
  const int H = a.Hkv, T = a.T, W = a.W;
  const unsigned per_seq = (unsigned)(T - 1) / HALF + 2;  // blocks that a sequence's call can touch
  unsigned rest = blockIdx.x;
  const int bi = (int)(rest % per_seq);
  rest /= per_seq;
  const int kv = (int)(rest & 1u);
  rest >>= 1;
  const int h = (int)(rest % H);
  rest /= H;
  const int b = (int)(rest % a.batch), ll = (int)(rest / a.batch);
  const int layer = a.layer0 + ll;

  const int p0 = a.pos[b];
  const bool in = p0 >= 0 && (long long)p0 + T <= a.max_seq_len;
  const int end = p0 + T, first = p0 / HALF * HALF, base = first + bi * HALF;
  const bool whole = base + HALF <= end;
  const int tok = kv ? value_token(w, v) : key_token(w, v), pos = base + tok;
  const bool bf16 = a.in_bf16;
  const void* src = kv ? a.v : a.k;
  const size_t unit = ((size_t)ll * a.batch + b) * H + h;
  float* ring = (kv ? a.p.ringv : a.p.ringk) + (((size_t)layer * a.max_batch + b) * H + h) * W * D;

  const bool mine = in && pos >= p0 && pos < end;
  float x[32];
  if (mine) load32(src, (unit * T + (pos - p0)) * D + 32 * G, bf16, x);
  // Before a prefill this is a dependent launch of the copy of the ring: what it writes waits for that.  (All threads do, so
  // that this grid never ends before the other.)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (p0 >= 0 && !in && threadIdx.x == 0 && bi == 0 && kv == 0 && h == 0) atomicOr(a.p.status, KVQ_DEV_POS_RANGE);
  if (!in || base >= end) return;  // (or the sequence is not part of the call)
  if (!mine && whole) load32(ring, (size_t)(pos % W) * D + 32 * G, false, x);
  // The newest W tokens of the call go to the ring raw.  Those whose slots hold tokens that the first block still has to
  // read are left to the CTA of that block, after it has read them.
  const int held = p0 - first;
  const bool raw = mine && pos >= end - W && !((pos - first) % W < held && pos - first >= W);
  if (raw) store32(ring + (size_t)(pos % W) * D + 32 * G, x);

  const int phys = a.block_table[(size_t)b * a.L.max_pages_per_seq + base / PAGE];
  const bool bad = phys < 0 || phys >= a.L.n_pages;
  if (bad && threadIdx.x == 0) atomicOr(a.p.status, KVQ_DEV_BAD_PAGE);
  if (!whole) return;  // (its old tokens stay in the ring: the call ends within 32 of them)
  if (!bad) {
    rotate32(x, G, a.p.signs, a.sinkhorn ? (kv ? a.p.sigv : a.p.sigk) + ((size_t)layer * H + h) * D : nullptr);
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 32; ++j) m = fmaxf(m, fabsf(x[j]));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
    if (lane == 0) most[w] = m;
  }
  __syncthreads();
  if (bi == 0 && held > 0) {
    // tokens first + W + j, first + 2 W + j, ... of j < held: the newest of each that the call appends
    for (int j = w * 8 + v; j < held; j += WARPS * 8) {
      const int p = first + j + (end - 1 - first - j) / W * W;
      if (p < p0 || p < first + W) continue;
      float y[32];
      load32(src, (unit * T + (p - p0)) * D + 32 * G, bf16, y);
      store32(ring + (size_t)(p % W) * D + 32 * G, y);
    }
  }
  if (bad) return;
  const float d = __fdiv_rn(fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3])), 127.0f);
  uint8_t* half = a.p.pages + (((size_t)layer * a.L.n_pages + phys) * H + h) * (size_t)a.L.page_bytes +
                  (size_t)(base % PAGE / HALF) * a.L.half_bytes;
  if (threadIdx.x == 0) *reinterpret_cast<float*>(half + (kv ? a.L.off_vmeta : a.L.off_kmeta)) = d;
  uint32_t u8[8];
  code32(x, d, u8);
  if (kv) store_values(half, u8, w, v, G);
  else store_keys(half, u8, w, v, G);
}

}  // namespace

cudaError_t launch_append_blocks(const AppendArgs& a, bool dependent, cudaStream_t s) {
  const long long ctas = (long long)((a.T - 1) / HALF + 2) * 2 * a.Hkv * a.batch * a.n_layers_call;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(WARPS * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, append_block_kernel, a);
}

}  // namespace kvq

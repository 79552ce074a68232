// What the kernels that go through a cache's records in tiles of 128 positions share: the list of tiles, a thread's
// part of a tile, operand layouts in shared memory, launches.
#pragma once

#include "tc.cuh"

namespace kvq {
namespace records {

using namespace tc;

constexpr int TILE = 128;  // positions per tile = MMA M

// warp 0: the sequences' lengths (0 where out of range) and the exclusive prefix of their tiles, [batch + 1]
template <typename Tiles>
__device__ __forceinline__ void tile_prefix(const MultiArgs& a, int* lens, int* pre, bool flag, Tiles tiles) {
  const int lane = threadIdx.x & 31, per = (a.batch + 31) / 32;
  const int b0 = min(a.batch, lane * per), b1 = min(a.batch, b0 + per);
  int s = 0;
  for (int b = b0; b < b1; ++b) {
    int L = a.seq_lens[b];
    if (L < 0 || L > a.max_seq_len) {
      if (flag) atomicOr(a.p.status, KVQ_DEV_SEQLEN_RANGE);
      L = 0;
    }
    lens[b] = L;
    s += tiles(L);
  }
  int incl = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(FULL, incl, o);
    if (lane >= o) incl += y;
  }
  int run = incl - s;
  for (int b = b0; b < b1; ++b) {
    pre[b] = run;
    run += tiles(lens[b]);
  }
  if (lane == 31) pre[a.batch] = incl;
}
// n / d of numbers that usually fit 32 bits
__device__ __forceinline__ long long quick_div(long long n, long long d) {
  return ((unsigned long long)n | (unsigned long long)d) < 0x80000000ull ? (long long)((unsigned)n / (unsigned)d) : n / d;
}

// byte offset of (row, k) in a K-major operand of R rows
__host__ __device__ constexpr uint32_t km_off(int row, int k, int R) {
  return (uint32_t)((k >> 3) * (R >> 3) * 128 + (row >> 3) * 128 + (row & 7) * 16 + (k & 7) * 2);
}
// byte offset of (n, k) in an N-major (or M-major) operand of R n, and of (m, k) where they are 128
__host__ __device__ constexpr uint32_t mn_off(int n, int k, int R) {
  return (uint32_t)((k >> 3) * (R >> 3) * 128 + (n >> 3) * 128 + (k & 7) * 16 + (n & 7) * 2);
}
__host__ __device__ constexpr uint32_t mm_off(int m, int k) { return mn_off(m, k, D); }

// Four channels (4 lane .. + 3) of a vector held by a warp, as the 8 bytes that belong at 8 (lane & 1) of their
// 16-byte group: in order, or in the order in which nibbles() leaves eight codes
template <bool NIBBLE_ORDER>
__device__ __forceinline__ uint2 pack4(uint32_t a, uint32_t b, int lane) {  // pairs (0, 1) and (2, 3)
  if (!NIBBLE_ORDER) return make_uint2(a, b);
  const bool odd = lane & 1;
  const uint32_t r = __shfl_xor_sync(FULL, odd ? a : b, 1);
  // even: (c0 c4)(c1 c5), odd: (c2 c6)(c3 c7)
  return odd ? make_uint2(__byte_perm(r, b, 0x5410), __byte_perm(r, b, 0x7632))
             : make_uint2(__byte_perm(a, r, 0x5410), __byte_perm(a, r, 0x7632));
}
__device__ __forceinline__ float2 load2_in(const void* base, int off, bool bf16) {
  if (!bf16) return *reinterpret_cast<const float2*>(static_cast<const float*>(base) + off);
  const uint32_t u = *reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(base) + off);
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ float lo_part(float v) { return v - __half2float(__float2half_rn(v)); }
// store the four channels' hi parts to a plane and their lo parts to the next
template <bool NIBBLE_ORDER>
__device__ __forceinline__ void put4(uint8_t* dst, uint32_t plane, const float (&y)[4], int lane) {
  uint32_t h[2], l[2];
  split2(y[0], y[1], h[0], l[0]);
  split2(y[2], y[3], h[1], l[1]);
  *reinterpret_cast<uint2*>(dst) = pack4<NIBBLE_ORDER>(h[0], h[1], lane);
  *reinterpret_cast<uint2*>(dst + plane) = pack4<NIBBLE_ORDER>(l[0], l[1], lane);
}

// ------------------------------------------------------------------ a tile's records
// A thread's part of a tile, of P threads to a position (2 or 4): keys of position t = tid & 127 (part hf of its record),
// values of the position pair vp, rows 2 vr and 2 vr + 1, all groups of 32 channels (P = 2) or groups 2 vg and 2 vg + 1.
struct Lane {
  int t, hf, vp, vr, vg;
};
template <int P = 2>
__device__ __forceinline__ Lane lane_of(int tid) {
  // values: 8 consecutive lanes write 8 distinct 16-byte slots of their core matrices (the odd rows' lanes take the odd
  // position of the pair first)
  if (P == 4) return {tid & 127, (tid >> 7) & 3, (tid & 3) | ((tid >> 3) & 60), (tid >> 2) & 3, (tid >> 4) & 1};
  return {tid & 127, (tid >> 7) & 1, (tid & 3) | ((tid >> 2) & 4) | ((tid >> 2) & 56), (tid >> 2) & 3, 0};
}

// The records of a tile in shared memory: four half-pages' keys (main, metadata), then their values.
template <int KF>
struct Rec {
  static constexpr int K_MAIN = KF == KVQ_Q8G32 ? 128 * HALF : 64 * HALF, V_MAIN = 64 * HALF;
  static constexpr int K_META = (KF == KVQ_Q8G32 ? 8 : KF == KVQ_TQ3_QJL ? 4 : 16) * HALF, V_META = 16 * HALF;
  static constexpr int KH = K_MAIN + K_META, VH = V_MAIN + V_META;  // of one half-page
  static constexpr int V0 = 4 * KH, BYTES = 4 * (KH + VH);
};

// physical page of position j of a sequence (-1: out of range)
__device__ __forceinline__ int checked(int phys, int n_pages) { return phys < n_pages ? phys : -1; }

__device__ __forceinline__ uint32_t dup_lo(uint32_t x) { return __byte_perm(x, x, 0x1010); }
__device__ __forceinline__ uint32_t dup_hi(uint32_t x) { return __byte_perm(x, x, 0x3232); }

// the 32 bytes at `at` as two words, the order in which they are read alternating over the lanes (fewer bank conflicts)
__device__ __forceinline__ void lds32(const uint8_t* at, bool swap, uint4& a, uint4& b) {
  const uint4 x = *reinterpret_cast<const uint4*>(at + (swap ? 16 : 0)), y = *reinterpret_cast<const uint4*>(at + (swap ? 0 : 16));
  a = make_uint4(swap ? y.x : x.x, swap ? y.y : x.y, swap ? y.z : x.z, swap ? y.w : x.w);
  b = make_uint4(swap ? x.x : y.x, swap ? x.y : y.y, swap ? x.z : y.z, swap ? x.w : y.w);
}

// ------------------------------------------------------------------ launches
// Launches kernel K, as a programmatic dependent of the kernel before it in the stream or after it
template <auto K, typename... A>
cudaError_t go(dim3 grid, unsigned threads, size_t smem, bool dependent, cudaStream_t s, A... args) {
  if (smem > 32 * 1024) {  // (static shared memory, up to 8 KB of it here, counts towards the 48 KB that need no leave)
    const cudaError_t e = allow_shared_memory<K>();
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, K, args...);
}

}  // namespace records
}  // namespace kvq

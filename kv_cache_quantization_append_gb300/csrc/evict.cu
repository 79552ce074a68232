// Eviction: cut sequences of the cache to a budget of positions, keeping the newest `recent` and, of the
// older ones, those with the largest accumulated attention weight; per (layer, sequence, kv-head), in place.
//
// Records move as they are (a token's codes and scales do not depend on its slot, only their place in the
// half-page does), so nothing is quantised again; kept positions stay in order.  Four launches:
//  1. select_kernel, one CTA per unit: radix select of the (budget - recent)-th largest weight over the older
//     positions -- 8 bits of the weights' order-preserving integer image at a time, counted in shared memory --
//     then one ordered pass that lists the kept positions (weight above the threshold, or equal to it and among
//     the lowest such indices) and compacts the weights.  Counting and ranking are integer sums: the result
//     does not depend on timing.
//  2. gather_kernel, one CTA per (unit, 32 kept positions): the half-page image of the kept records, in scratch.
//  3. scatter_kernel: the images to their pages.  (In place: a half-page's old records may still be wanted by
//     another CTA while its new ones are known, so all are read before any is written.)
//  4. ring_kernel: the window ring holds the newest tokens at slot position % window; positions shift by the
//     number of tokens cut, so its rows turn.
#include "kvq_internal.cuh"

namespace kvq {

namespace {

constexpr int SEL_THREADS = 1024;
constexpr int GATHER_THREADS = 128;

__device__ __forceinline__ int checked_len(const EvictArgs& a, int b, bool flag) {
  const int L = a.seq_lens[b];
  if (L < 0 || L > a.max_seq_len) {
    if (flag) atomicOr(a.p.status, KVQ_DEV_SEQLEN_RANGE);
    return 0;
  }
  return L;
}

// order-preserving integer image of a weight; NaN below everything, both zeros alike
__device__ __forceinline__ uint32_t order_of(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// exclusive prefix of v over the block, and its total
__device__ __forceinline__ int block_exclusive(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(FULL, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[w] = incl;
  __syncthreads();
  int ws = warp_sums[lane];
  int wi = ws;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(FULL, wi, o);
    if (lane >= o) wi += y;
  }
  total = __shfl_sync(FULL, wi, 31);
  return __shfl_sync(FULL, wi - ws, w) + incl - v;
}

__global__ void __launch_bounds__(SEL_THREADS) select_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int warp_sums[32];
  __shared__ int pick_sh[2];
  const int tid = threadIdx.x;
  const int unit = blockIdx.x;  // ((ll * batch) + b) * Hkv + h
  const int h = unit % a.Hkv, b = (unit / a.Hkv) % a.batch;
  const int L = checked_len(a, b, tid == 0 && h == 0 && unit < a.batch * a.Hkv);
  int32_t* kept = a.kept + (size_t)unit * a.budget;
  if (unit < a.batch * a.Hkv && h == 0 && tid == 0) a.new_lens[b] = min(L, a.budget);
  if (L <= a.budget) {
    for (int j = tid; j < a.budget; j += SEL_THREADS) kept[j] = j < L ? j : -1;
    return;
  }
  float* w = a.weights + (size_t)unit * a.max_seq_len;
  const int old = L - a.recent, want = a.budget - a.recent;  // old > want >= 0
  // threshold: the want-th largest image, and how many equal to it are kept
  uint32_t thr = 0u, mask = 0u;
  int need = want;
  if (want > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int j = tid; j < old; j += SEL_THREADS) {
        const uint32_t u = order_of(w[j]);
        if ((u & mask) == thr) atomicAdd(&hist[(u >> shift) & 255u], 1);
      }
      __syncthreads();
      // digit d with count(> d) < need <= count(>= d), from the top
      if (tid < 32) {
        int c[8], s = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += c[i] = hist[255 - (8 * tid + i)];
        int incl = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(FULL, incl, o);
          if (tid >= o) incl += y;
        }
        int above = incl - s;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (above < need && need <= above + c[i]) {
            pick_sh[0] = 255 - (8 * tid + i);
            pick_sh[1] = above;
          }
          above += c[i];
        }
      }
      __syncthreads();
      thr |= (uint32_t)pick_sh[0] << shift;
      mask |= 255u << shift;
      need -= pick_sh[1];
      __syncthreads();
    }
  }
  // ordered pass: a chunk's weights are all read before any is written, and no write passes the chunk's end
  int n_kept = 0, n_equal = 0;
  for (int j0 = 0; j0 < L; j0 += SEL_THREADS) {
    const int j = j0 + tid;
    const float wj = j < L ? w[j] : 0.f;
    const uint32_t u = order_of(wj);
    const bool cand = want > 0 && j < old;
    int total;
    const int eq = cand && u == thr ? 1 : 0;
    const int eq_before = n_equal + block_exclusive(eq, warp_sums, total);
    n_equal += total;
    const int keep = j < L && (j >= old || (cand && (u > thr || (eq && eq_before < need)))) ? 1 : 0;
    const int at = n_kept + block_exclusive(keep, warp_sums, total);
    n_kept += total;
    if (keep) {
      kept[at] = j;
      w[at] = wj;
    }
    __syncthreads();
  }
}

// 16-byte row r (0..7) of pair p's 128 bytes of values sits at 16 ((r + 2 (p & 3)) & 7)
__device__ __forceinline__ int v_row(int p, int r) { return 128 * p + 16 * ((r + 2 * (p & 3)) & 7); }

template <int KF>
__global__ void __launch_bounds__(GATHER_THREADS) gather_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ int src_sh[HALF];              // source position of each slot (its own where nothing is moved there)
  __shared__ const uint8_t* base_sh[HALF];  // the half-page that holds it
  const int tid = threadIdx.x, hb = blockIdx.x, unit = blockIdx.y + blockIdx.z * 32768;
  if (unit >= a.n_units) return;
  const int h = unit % a.Hkv, b = (unit / a.Hkv) % a.batch, layer = a.layer0 + unit / (a.Hkv * a.batch);
  const int L = checked_len(a, b, false);
  if (L <= a.budget) return;
  const size_t page_stride = (size_t)a.Hkv * a.L.page_bytes;
  const uint8_t* pages = a.p.pages + ((size_t)layer * a.L.n_pages * a.Hkv + h) * (size_t)a.L.page_bytes;
  if (tid < HALF) {
    const int j = hb * HALF + tid;
    const int s = j < a.budget ? a.kept[(size_t)unit * a.budget + j] : j;
    // slots past the budget in its last half-page keep their bytes; they are in the same page as kept ones
    const int phys = a.block_table[(size_t)b * a.max_pages_per_seq + s / PAGE];
    const bool bad = phys < 0 || phys >= a.L.n_pages;
    if (bad) atomicOr(a.p.status, KVQ_DEV_BAD_PAGE);
    src_sh[tid] = s;
    base_sh[tid] = bad ? nullptr : pages + (size_t)phys * page_stride + (size_t)((s % PAGE) / HALF) * a.L.half_bytes;
  }
  __syncthreads();
  uint8_t* img = a.images + ((size_t)unit * a.n_halves + hb) * (size_t)a.L.half_bytes;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  // keys: 16-byte chunks of each record (Q8G32: chunk m at 16 (m ^ (token & 1)))
  constexpr int CH = KF == KVQ_Q8G32 ? 8 : 4;
#pragma unroll
  for (int i = tid; i < HALF * CH; i += GATHER_THREADS) {
    const int t = i / CH, m = i % CH, st = src_sh[t] % HALF;
    const uint8_t* sb = base_sh[t];
    const int sm = KF == KVQ_Q8G32 ? m ^ (st & 1) : m, dm = KF == KVQ_Q8G32 ? m ^ (t & 1) : m;
    *reinterpret_cast<uint4*>(img + (t * CH + dm) * 16) =
        sb ? *reinterpret_cast<const uint4*>(sb + (st * CH + sm) * 16) : zero;
  }
  // values: 16-byte row r of pair p holds both tokens' bytes interleaved
  {
    const int p = tid >> 3, r = tid & 7;
    const int s0 = src_sh[2 * p] % HALF, s1 = src_sh[2 * p + 1] % HALF;
    const uint8_t *b0 = base_sh[2 * p], *b1 = base_sh[2 * p + 1];
    const uint4 x = b0 ? *reinterpret_cast<const uint4*>(b0 + a.L.off_vmain + v_row(s0 >> 1, r)) : zero;
    const uint4 y = b1 ? *reinterpret_cast<const uint4*>(b1 + a.L.off_vmain + v_row(s1 >> 1, r)) : zero;
    // bytes (slot, slot + 2) of the sources -> bytes (0, 2) and (1, 3)
    const uint32_t sel = (s0 & 1 ? 0x0301u : 0x0200u), sel1 = (s1 & 1 ? 0x0705u : 0x0604u);
    const uint32_t pick = (sel & 0xfu) | ((sel1 & 0xfu) << 4) | (sel & 0xf00u) | ((sel1 & 0xf00u) << 4);
    *reinterpret_cast<uint4*>(img + a.L.off_vmain + v_row(p, r)) =
        make_uint4(__byte_perm(x.x, y.x, pick), __byte_perm(x.y, y.y, pick), __byte_perm(x.z, y.z, pick),
                   __byte_perm(x.w, y.w, pick));
  }
  // key metadata
  if (KF == KVQ_TQ3_QJL) {
    if (tid < 2 * HALF) {
      const int t = tid % HALF, f = tid / HALF;
      const uint8_t* sb = base_sh[t];
      reinterpret_cast<uint16_t*>(img + a.L.off_kmeta)[tid] =
          sb ? reinterpret_cast<const uint16_t*>(sb + a.L.off_kmeta)[f * HALF + src_sh[t] % HALF] : (uint16_t)0;
    }
  } else if (tid < HALF) {
    const uint8_t* sb = base_sh[tid];
    const int st = src_sh[tid] % HALF;
    if (KF == KVQ_Q4G32)
      reinterpret_cast<uint4*>(img + a.L.off_kmeta)[tid] =
          sb ? reinterpret_cast<const uint4*>(sb + a.L.off_kmeta)[st] : zero;
    else
      reinterpret_cast<uint2*>(img + a.L.off_kmeta)[tid] =
          sb ? reinterpret_cast<const uint2*>(sb + a.L.off_kmeta)[st] : make_uint2(0u, 0u);
  }
  // value metadata: eight rows (4 scales, 4 zeros) of 32 halves
#pragma unroll
  for (int i = tid; i < 8 * HALF; i += GATHER_THREADS) {
    const int t = i % HALF, f = i / HALF;
    const uint8_t* sb = base_sh[t];
    reinterpret_cast<uint16_t*>(img + a.L.off_vmeta)[i] =
        sb ? reinterpret_cast<const uint16_t*>(sb + a.L.off_vmeta)[f * HALF + src_sh[t] % HALF] : (uint16_t)0;
  }
}

__global__ void __launch_bounds__(GATHER_THREADS) scatter_kernel(const __grid_constant__ EvictArgs a) {
  const int hb = blockIdx.x, unit = blockIdx.y + blockIdx.z * 32768;
  if (unit >= a.n_units) return;
  const int h = unit % a.Hkv, b = (unit / a.Hkv) % a.batch, layer = a.layer0 + unit / (a.Hkv * a.batch);
  if (checked_len(a, b, false) <= a.budget) return;
  const int phys = a.block_table[(size_t)b * a.max_pages_per_seq + hb * HALF / PAGE];
  if (phys < 0 || phys >= a.L.n_pages) return;
  const uint4* img = reinterpret_cast<const uint4*>(a.images + ((size_t)unit * a.n_halves + hb) * (size_t)a.L.half_bytes);
  uint4* dst = reinterpret_cast<uint4*>(a.p.pages + (((size_t)layer * a.L.n_pages + phys) * a.Hkv + h) * (size_t)a.L.page_bytes +
                                        (size_t)(hb & 1) * a.L.half_bytes);
  for (int i = threadIdx.x; i < a.L.half_bytes / 16; i += GATHER_THREADS) dst[i] = img[i];
}

// one CTA per (unit, K|V, 8 channels): the new slot of position p' = p - cut is p' % W
__global__ void __launch_bounds__(256) ring_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ float4 col[MAX_WINDOW][2];
  const int unit = blockIdx.y + blockIdx.z * 32768, c = blockIdx.x & 15, kv = blockIdx.x >> 4;
  if (unit >= a.n_units) return;
  const int h = unit % a.Hkv, b = (unit / a.Hkv) % a.batch, layer = a.layer0 + unit / (a.Hkv * a.batch);
  const int L = checked_len(a, b, false);
  const int cut = L - a.budget, turn = cut > 0 ? cut % a.W : 0;
  if (cut <= 0 || turn == 0) return;
  float4* ring = reinterpret_cast<float4*>((kv ? a.p.ringv : a.p.ringk) +
                                           (((size_t)layer * a.max_batch + b) * a.Hkv + h) * (size_t)a.W * D + 8 * c);
  for (int i = threadIdx.x; i < 2 * a.W; i += 256) col[i >> 1][i & 1] = ring[(size_t)(i >> 1) * (D / 4) + (i & 1)];
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.W; i += 256) {
    int s = (i >> 1) + turn;
    if (s >= a.W) s -= a.W;
    ring[(size_t)(i >> 1) * (D / 4) + (i & 1)] = col[s][i & 1];
  }
}

}  // namespace

size_t evict_scratch_bytes(int n_units, int budget, int half_bytes) {
  return (size_t)n_units * ((budget + HALF - 1) / HALF) * (size_t)half_bytes;
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  select_kernel<<<a.n_units, SEL_THREADS, 0, s>>>(a);
  const unsigned y = a.n_units < 32768 ? a.n_units : 32768, z = (a.n_units + 32767) / 32768;
  const dim3 grid(a.n_halves, y, z);
  if (a.k_format == KVQ_TQ3_QJL) gather_kernel<KVQ_TQ3_QJL><<<grid, GATHER_THREADS, 0, s>>>(a);
  else if (a.k_format == KVQ_Q8G32) gather_kernel<KVQ_Q8G32><<<grid, GATHER_THREADS, 0, s>>>(a);
  else gather_kernel<KVQ_Q4G32><<<grid, GATHER_THREADS, 0, s>>>(a);
  scatter_kernel<<<grid, GATHER_THREADS, 0, s>>>(a);
  if (a.W > 0) ring_kernel<<<dim3(32, y, z), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq

// Eviction: cut sequences of the cache to a budget of positions, keeping the newest `recent` and, of the
// older ones, those with the largest accumulated attention weight; per (layer, sequence, kv-head), in place.
//
// Records move as they are (a token's codes and scales do not depend on its slot, only their place in the
// half-page does), so nothing is quantised again; kept positions stay in order.  Two launches:
//  1. select_kernel, one CTA per unit: radix select of the (budget - recent)-th largest weight over the older
//     positions -- 11, 11 and 10 bits of the weights' order-preserving integer image, counted in shared memory,
//     where the weights lie meanwhile (up to 48K of them; longer sequences are read again for each step) --
//     then one ordered pass that lists the kept positions (weight above the threshold, or equal to it and among
//     the lowest such indices) and compacts the weights.  Counting and ranking are integer sums: the result
//     does not depend on timing.  Further CTAs turn the window ring meanwhile: its slot is position % window,
//     and positions shift by the number of tokens cut.
//  2. move_kernel, a cluster of CTAs per unit: windows of half-pages in ascending order, each gathered into
//     shared memory by all CTAs of the cluster before any of it is written.  A slot's position is never below the
//     slot, so a window's sources lie at or behind its own start, where no earlier window has written: one cluster
//     barrier per window makes the move safe in place, and the next window is gathered while the last is written.
//     Bound by memory: each kept record is read once and written once.
#include "kvq_internal.cuh"

namespace kvq {

namespace {

constexpr int SEL_THREADS = 1024;
constexpr int SEL_CACHE = 48 * 1024;   // weights that shared memory holds
constexpr int BINS = 2048;
constexpr int MOVE_THREADS = 256;
constexpr int CLUSTER = 8;
constexpr int HPW = 4;                 // half-pages of a CTA per window
static_assert(MOVE_THREADS == 8 * HALF && HPW * HALF <= MOVE_THREADS, "a thread's share of a window");

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
  const uint32_t u = __float_as_uint(w + 0.f);
  return w != w ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// exclusive prefix of v over the block (32 warps), and its total
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t* warp_sums, uint32_t& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(FULL, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sums[w] = incl;
  __syncthreads();
  const uint32_t ws = warp_sums[lane];
  uint32_t wi = ws;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(FULL, wi, o);
    if (lane >= o) wi += y;
  }
  total = __shfl_sync(FULL, wi, 31);
  const uint32_t before = __shfl_sync(FULL, wi - ws, w);
  __syncthreads();
  return before + incl - v;
}

// The ring of one unit's keys or values: rows turn by the tokens cut, as many channels at a time as `room` floats hold.
__device__ void turn_ring(const EvictArgs& a, int unit, int kv, float4* buf, int room) {
  const int h = unit % a.Hkv, b = (unit / a.Hkv) % a.batch, layer = a.layer0 + unit / (a.Hkv * a.batch);
  const int cut = checked_len(a, b, false) - a.budget, turn = cut > 0 ? cut % a.W : 0;
  if (turn == 0) return;
  float4* ring = reinterpret_cast<float4*>((kv ? a.p.ringv : a.p.ringk) +
                                           (((size_t)layer * a.max_batch + b) * a.Hkv + h) * (size_t)a.W * D);
  int cols = D / 4;  // float4 columns at a time: a power of two
  while (cols * a.W * 4 > room) cols >>= 1;
  for (int c0 = 0; c0 < D / 4; c0 += cols) {
    for (int i = threadIdx.x; i < cols * a.W; i += SEL_THREADS) buf[i] = ring[(size_t)(i / cols) * (D / 4) + c0 + i % cols];
    __syncthreads();
    for (int i = threadIdx.x; i < cols * a.W; i += SEL_THREADS) {
      int s = i / cols + turn;
      if (s >= a.W) s -= a.W;
      ring[(size_t)(i / cols) * (D / 4) + c0 + i % cols] = buf[s * cols + i % cols];
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(SEL_THREADS) select_kernel(const __grid_constant__ EvictArgs a, int room) {
  extern __shared__ __align__(16) float cache[];  // `room` floats
  __shared__ int hist[BINS];
  __shared__ uint32_t warp_sums[32];
  __shared__ int pick_sh[2];
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x;
  if ((int)blockIdx.x >= a.n_units) {
    turn_ring(a, (blockIdx.x - a.n_units) >> 1, (blockIdx.x - a.n_units) & 1, reinterpret_cast<float4*>(cache), room);
    return;
  }
  const int unit = blockIdx.x;  // ((ll * batch) + b) * Hkv + h
  const int h = unit % a.Hkv, b = (unit / a.Hkv) % a.batch;
  const bool first = h == 0 && unit < a.batch * a.Hkv;
  const int L = checked_len(a, b, first && tid == 0);
  int32_t* kept = a.kept + (size_t)unit * a.budget;
  if (first && tid == 0) a.new_lens[b] = min(L, a.budget);
  if (L <= a.budget) {
    for (int j = tid; j < a.budget; j += SEL_THREADS) kept[j] = j < L ? j : -1;
    return;
  }
  float* w = a.weights + (size_t)unit * a.max_seq_len;
  const int old = L - a.recent, want = a.budget - a.recent;  // old > want >= 0
  const bool cached = L <= room;
  if (cached) {
    const int L4 = (reinterpret_cast<uintptr_t>(w) & 15) == 0 ? L / 4 : 0;
#pragma unroll 4
    for (int j = tid; j < L4; j += SEL_THREADS) reinterpret_cast<float4*>(cache)[j] = reinterpret_cast<const float4*>(w)[j];
    for (int j = 4 * L4 + tid; j < L; j += SEL_THREADS) cache[j] = w[j];
  }
  const float* src = cached ? cache : w;
  // threshold: the want-th largest image, and how many equal to it are kept
  uint32_t thr = 0u, mask = 0u;
  int need = want;
  if (want > 0) {
#pragma unroll 1
    for (int step = 0; step < 3; ++step) {
      const int shift = step == 0 ? 21 : step == 1 ? 10 : 0, bins = step == 2 ? 1024 : 2048;
      for (int i = tid; i < BINS; i += SEL_THREADS) hist[i] = 0;
      __syncthreads();
#pragma unroll 4
      for (int j = tid; j < old; j += SEL_THREADS) {
        const uint32_t u = order_of(src[j]);
        if ((u & mask) == thr) atomicAdd(&hist[(u >> shift) & (bins - 1)], 1);
      }
      __syncthreads();
      // digit d with count(> d) < need <= count(>= d), from the top: two bins a thread
      const int hi = BINS - 1 - 2 * tid;
      const int c0 = hist[hi], c1 = hist[hi - 1];
      uint32_t total;
      const int above = (int)block_exclusive((uint32_t)(c0 + c1), warp_sums, total);
      if (above < need && need <= above + c0 + c1) {
        const bool second = need > above + c0;
        pick_sh[0] = second ? hi - 1 : hi;
        pick_sh[1] = above + (second ? c0 : 0);
      }
      __syncthreads();
      thr |= (uint32_t)pick_sh[0] << shift;
      mask |= (uint32_t)(bins - 1) << shift;
      need -= pick_sh[1];
      __syncthreads();
    }
  }
  __syncthreads();
  // ordered pass, eight consecutive positions a thread.  (Read again from global memory, a chunk's weights are all read
  // before any is written, and no write passes the chunk's end.)
  uint32_t n_above = 0, n_equal = 0;  // kept for their weight or age, and equal to the threshold, before the chunk
  constexpr int PER = 8;
  for (int j0 = 0; j0 < L; j0 += SEL_THREADS * PER) {
    float wj[PER];
    uint32_t keep = 0, equal = 0;
    const int jt = j0 + tid * PER;
    if (cached && jt + PER <= L) {
      const float4 x = *reinterpret_cast<const float4*>(cache + jt), y = *reinterpret_cast<const float4*>(cache + jt + 4);
      wj[0] = x.x, wj[1] = x.y, wj[2] = x.z, wj[3] = x.w, wj[4] = y.x, wj[5] = y.y, wj[6] = y.z, wj[7] = y.w;
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) wj[i] = jt + i < L ? src[jt + i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int j = jt + i;
      const uint32_t u = order_of(wj[i]);
      const bool cand = want > 0 && j < old;
      keep |= (uint32_t)((j < L && j >= old) || (cand && u > thr)) << i;
      equal |= (uint32_t)(cand && u == thr) << i;
    }
    uint32_t total;
    const uint32_t before = block_exclusive((uint32_t)__popc(keep) | (uint32_t)__popc(equal) << 16, warp_sums, total);
    uint32_t na = n_above + (before & 0xffffu), ne = n_equal + (before >> 16);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const bool e = (equal >> i) & 1, k = (keep >> i) & 1;
      if (k || (e && ne < (uint32_t)need)) {
        const uint32_t at = na + min(ne, (uint32_t)need);
        kept[at] = j0 + tid * PER + i;
        w[at] = wj[i];
      }
      na += k;
      ne += e;
    }
    n_above += total & 0xffffu;
    n_equal += total >> 16;
  }
}

// 16-byte row r (0..7) of pair p's 128 bytes of values sits at 16 ((r + 2 (p & 3)) & 7)
__device__ __forceinline__ int v_row(int p, int r) { return 128 * p + 16 * ((r + 2 * (p & 3)) & 7); }

template <int KF>
__global__ void __cluster_dims__(CLUSTER, 1, 1) __launch_bounds__(MOVE_THREADS) move_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(16) uint8_t images[];  // [2][HPW][half_bytes]
  __shared__ int src_sh[2][HPW * HALF];              // source token (within its half-page) of each slot
  __shared__ const uint8_t* base_sh[2][HPW * HALF];  // the half-page that holds it (null: on a bad page)
  const int tid = threadIdx.x, rank = blockIdx.x % CLUSTER, unit = blockIdx.x / CLUSTER;
  const int h = unit % a.Hkv, b = (unit / a.Hkv) % a.batch, layer = a.layer0 + unit / (a.Hkv * a.batch);
  const int L = checked_len(a, b, false);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (L <= a.budget) return;  // (the whole cluster)
  const size_t page_stride = (size_t)a.Hkv * a.L.page_bytes;
  uint8_t* pages = a.p.pages + ((size_t)layer * a.L.n_pages * a.Hkv + h) * (size_t)a.L.page_bytes;
  const int32_t* bt = a.block_table + (size_t)b * a.max_pages_per_seq;
  const int32_t* kept = a.kept + (size_t)unit * a.budget;
  const int hb = a.L.half_bytes, windows = (a.n_halves + CLUSTER * HPW - 1) / (CLUSTER * HPW);
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);

  // Of window w this CTA has half-pages half_of(w) .. + HPW - 1.  The kept position of a thread's slot is requested two
  // windows ahead, its page a window ahead.
  const auto half_of = [&](int w) { return (w * CLUSTER + rank) * HPW; };
  const auto kept_of = [&](int w) {
    const int j = half_of(w) * HALF + tid;
    if (tid >= HPW * HALF || half_of(w) + tid / HALF >= a.n_halves) return -1;
    // slots past the budget in its last half-page keep their bytes; they are in the same page as kept ones
    return j < a.budget ? kept[j] : j;
  };
  const auto resolve = [&](int w, int s) {
    if (s < 0) return;
    const int phys = bt[s / PAGE];
    const bool bad = phys < 0 || phys >= a.L.n_pages;
    if (bad) atomicOr(a.p.status, KVQ_DEV_BAD_PAGE);
    src_sh[w & 1][tid] = s % HALF;
    base_sh[w & 1][tid] = bad ? nullptr : pages + (size_t)phys * page_stride + (size_t)((s % PAGE) / HALF) * hb;
  };
  // gathers window w into images[w & 1]: everything is requested before anything is stored
  const auto gather = [&](int w) {
    const int n = min(HPW, a.n_halves - half_of(w));
    const int* src = src_sh[w & 1];
    const uint8_t* const* base = base_sh[w & 1];
    uint8_t* img0 = images + (size_t)(w & 1) * HPW * hb;
    constexpr int CH = KF == KVQ_Q8G32 ? 8 : 4;                  // 16-byte chunks of a key record
    constexpr int NK = HPW * HALF * CH / MOVE_THREADS, NV = HPW * HALF * 4 / MOVE_THREADS, NM = HPW * HALF * 8 / MOVE_THREADS;
    uint4 k[NK], x[NV], y[NV], km = zero;
    uint16_t vm[NM];
#pragma unroll
    for (int q = 0; q < NK; ++q) {  // keys (Q8G32: chunk m at 16 (m ^ (token & 1)))
      const int i = q * MOVE_THREADS + tid, t = i / CH, m = i % CH;
      k[q] = zero;
      if (t < n * HALF && base[t])
        k[q] = *reinterpret_cast<const uint4*>(base[t] + (src[t] * CH + (KF == KVQ_Q8G32 ? m ^ (src[t] & 1) : m)) * 16);
    }
#pragma unroll
    for (int q = 0; q < NV; ++q) {  // values: 16-byte row r of a pair holds both tokens' bytes interleaved
      const int i = q * MOVE_THREADS + tid, pr = i >> 3, r = i & 7;
      x[q] = y[q] = zero;
      if (pr < n * (HALF / 2)) {
        if (base[2 * pr]) x[q] = *reinterpret_cast<const uint4*>(base[2 * pr] + a.L.off_vmain + v_row(src[2 * pr] >> 1, r));
        if (base[2 * pr + 1]) y[q] = *reinterpret_cast<const uint4*>(base[2 * pr + 1] + a.L.off_vmain + v_row(src[2 * pr + 1] >> 1, r));
      }
    }
    // key metadata: Q4 16 bytes, Q8 8 bytes a token, TQ3 two halves
    if (KF == KVQ_TQ3_QJL) {
      const int t = tid / (2 * HALF) * HALF + tid % HALF, f = tid / HALF % 2;
      if (t < n * HALF && base[t]) km.x = reinterpret_cast<const uint16_t*>(base[t] + a.L.off_kmeta)[f * HALF + src[t]];
    } else if (tid < n * HALF && base[tid]) {
      if (KF == KVQ_Q4G32) {
        km = reinterpret_cast<const uint4*>(base[tid] + a.L.off_kmeta)[src[tid]];
      } else {
        const uint2 v = reinterpret_cast<const uint2*>(base[tid] + a.L.off_kmeta)[src[tid]];
        km.x = v.x, km.y = v.y;
      }
    }
#pragma unroll
    for (int q = 0; q < NM; ++q) {  // value metadata: half-page q's eight rows (4 scales, 4 zeros) of 32 halves
      const int f = tid / HALF, t = q * HALF + tid % HALF;
      vm[q] = t < n * HALF && base[t] ? reinterpret_cast<const uint16_t*>(base[t] + a.L.off_vmeta)[f * HALF + src[t]] : (uint16_t)0;
    }
#pragma unroll
    for (int q = 0; q < NK; ++q) {
      const int i = q * MOVE_THREADS + tid, t = i / CH, m = i % CH, td = t % HALF;
      if (t < n * HALF)
        *reinterpret_cast<uint4*>(img0 + t / HALF * hb + (td * CH + (KF == KVQ_Q8G32 ? m ^ (td & 1) : m)) * 16) = k[q];
    }
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      const int i = q * MOVE_THREADS + tid, pr = i >> 3, r = i & 7;
      if (pr < n * (HALF / 2)) {
        // bytes (slot, slot + 2) of the sources -> bytes (0, 2) and (1, 3)
        const uint32_t pick = (src[2 * pr] & 1 ? 0x0301u : 0x0200u) | (src[2 * pr + 1] & 1 ? 0x7050u : 0x6040u);
        *reinterpret_cast<uint4*>(img0 + pr / (HALF / 2) * hb + a.L.off_vmain + v_row(pr % (HALF / 2), r)) =
            make_uint4(__byte_perm(x[q].x, y[q].x, pick), __byte_perm(x[q].y, y[q].y, pick), __byte_perm(x[q].z, y[q].z, pick),
                       __byte_perm(x[q].w, y[q].w, pick));
      }
    }
    if (KF == KVQ_TQ3_QJL) {
      const int half = tid / (2 * HALF);
      if (half < n) reinterpret_cast<uint16_t*>(img0 + half * hb + a.L.off_kmeta)[tid % (2 * HALF)] = (uint16_t)km.x;
    } else if (tid < n * HALF) {
      uint8_t* dst = img0 + tid / HALF * hb + a.L.off_kmeta;
      if (KF == KVQ_Q4G32) reinterpret_cast<uint4*>(dst)[tid % HALF] = km;
      else reinterpret_cast<uint2*>(dst)[tid % HALF] = make_uint2(km.x, km.y);
    }
#pragma unroll
    for (int q = 0; q < NM; ++q)
      if (q < n) reinterpret_cast<uint16_t*>(img0 + q * hb + a.L.off_vmeta)[tid] = vm[q];
  };

  resolve(0, kept_of(0));
  int s_next = kept_of(1);
  __syncthreads();
  gather(0);
  for (int w = 0; w < windows; ++w) {
    // (the values just gathered are in shared memory, so their sources have been read)
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (w + 1 < windows) {
      resolve(w + 1, s_next);
      s_next = kept_of(w + 2);
      __syncthreads();
      gather(w + 1);
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    const int half0 = half_of(w), n = min(HPW, a.n_halves - half0), chunks = hb / 16;
    const uint4* img = reinterpret_cast<const uint4*>(images + (size_t)(w & 1) * HPW * hb);
#pragma unroll 2
    for (int i = tid; i < n * chunks; i += MOVE_THREADS) {
      const int half = i / chunks, g = half0 + half, phys = bt[g * HALF / PAGE];
      if (phys >= 0 && phys < a.L.n_pages)
        reinterpret_cast<uint4*>(pages + (size_t)phys * page_stride + (size_t)(g & 1) * hb)[i % chunks] = img[i];
    }
    __syncthreads();  // (the images are free for the window after next)
  }
}

template <int KF>
cudaError_t launch_move(const EvictArgs& a, cudaStream_t s) {
  const size_t smem = 2 * HPW * (size_t)a.L.half_bytes;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(move_kernel<KF>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.n_units * CLUSTER);
  cfg.blockDim = dim3(MOVE_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, move_kernel<KF>, a);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  // the weights of the longest sequence, or of SEL_CACHE positions; at least eight channels of the largest ring
  const int want = a.max_seq_len < SEL_CACHE ? a.max_seq_len : SEL_CACHE, least = 8 * MAX_WINDOW;
  const int room = ((want > least ? want : least) + 3) / 4 * 4;
  cudaError_t e = cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SEL_CACHE * 4);
  if (e != cudaSuccess) return e;
  select_kernel<<<a.n_units + (a.W > 0 ? 2 * a.n_units : 0), SEL_THREADS, (size_t)room * 4, s>>>(a, room);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return a.k_format == KVQ_TQ3_QJL ? launch_move<KVQ_TQ3_QJL>(a, s)
         : a.k_format == KVQ_Q8G32 ? launch_move<KVQ_Q8G32>(a, s)
                                   : launch_move<KVQ_Q4G32>(a, s);
}

}  // namespace kvq

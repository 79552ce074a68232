// Eviction: cut sequences of the cache to a budget of positions, keeping the newest `recent` and, of the
// older ones, those with the largest accumulated attention weight; per (layer, sequence, kv-head), in place.
//
// Records move as they are (a token's codes and scales do not depend on its slot, only their place in the
// half-page does), so nothing is quantised again; kept positions stay in order.  One launch, a cluster of eight
// CTAs per unit:
//  1. radix select of the (budget - recent)-th largest weight over the older positions -- 11, 11 and 10 bits of
//     the weights' order-preserving integer image, counted by each CTA over its share (which it keeps in shared
//     memory where it fits, and reads again for each step where it does not) and added up over the cluster -- then
//     one ordered pass that lists the kept positions (weight above the threshold, or equal to it and among the
//     lowest such indices) and compacts the weights.  Counting and ranking are integer sums: the result does not
//     depend on timing.
//  2. the move: windows of half-pages in ascending order, each gathered into shared memory by all CTAs of the
//     cluster before any of it is written.  A slot's position is never below the slot, so a window's sources lie at
//     or behind its own start, where no earlier window has written: one cluster barrier per window makes the move
//     safe in place, and the next window is gathered while the last is written.
//  3. the window ring turns: its slot is position % window, and positions shift by the number of tokens cut.
// Each kept record is read once and written once, but a quarter of the positions lies in nearly every sector of values
// and metadata, so the reads come to half as much again as what is kept.  Measured: 32K positions to 8K over 8 layers of 8
// heads Q4 68 us (2.7 TB/s of the bytes that cannot be avoided), 4 sequences of up to 8K to 2K 22.6 us.  Bound by latency:
// the steps of the select (six cluster barriers, then one per 8192 positions) and one gather at a time per CTA of the move.
#include "records.cuh"

namespace kvq {

namespace {

using namespace records;

constexpr int BINS = 2048;
constexpr int THREADS = 256;
constexpr int CLUSTER = 8;
constexpr int SHARE = 4 * THREADS;  // a CTA's weights of a window of the ordered pass
constexpr int SEL_WINDOW = CLUSTER * SHARE;
constexpr int HPW = 4;                 // half-pages of a CTA per window
static_assert(THREADS == 8 * HALF && HPW * HALF <= THREADS, "a thread's share of a window");

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

// exclusive prefix of v over the block, and its total
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t* warp_sums, uint32_t& total) {
  constexpr int WARPS = THREADS / 32;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(FULL, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sums[w] = incl;
  __syncthreads();
  uint32_t before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) {
    const uint32_t s = warp_sums[i];
    before += i < w ? s : 0;
    total += s;
  }
  __syncthreads();
  return before + incl - v;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the address of `p` (shared memory) in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t in_cta(const void* p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ int cluster_load(uint32_t at) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_store(uint32_t at, int v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// CTA `rank`'s channels of the ring of one unit's keys or values: rows turn by `turn`, as many channels at a time as
// `room` bytes hold (at least one float4 column: 16 KB at the widest window)
__device__ void turn_ring(const EvictArgs& a, float* ring_f, int turn, int rank, float4* buf, int room) {
  constexpr int MINE = D / 4 / CLUSTER;  // float4 columns
  float4* ring = reinterpret_cast<float4*>(ring_f) + rank * MINE;
  int cols = MINE;  // at a time: a power of two
  while (cols * a.W * 16 > room) cols >>= 1;
  for (int c0 = 0; c0 < MINE; c0 += cols) {
#pragma unroll 4
    for (int i = threadIdx.x; i < cols * a.W; i += THREADS) buf[i] = ring[(size_t)(i / cols) * (D / 4) + c0 + i % cols];
    __syncthreads();
#pragma unroll 4
    for (int i = threadIdx.x; i < cols * a.W; i += THREADS) {
      int s = i / cols + turn;
      if (s >= a.W) s -= a.W;
      ring[(size_t)(i / cols) * (D / 4) + c0 + i % cols] = buf[s * cols + i % cols];
    }
    __syncthreads();
  }
}

// Lists the kept positions of one unit and compacts its weights, by a cluster.  Of window n CTA `rank` has positions
// n SEL_WINDOW + rank SHARE .. + SHARE - 1.  area: `room` bytes, the same place in every CTA.
__device__ void select_kept(const EvictArgs& a, float* w, int32_t* kept, int L, int rank, uint8_t* area, int room) {
  int* hist = reinterpret_cast<int*>(area);           // this CTA's counts
  int* sums = hist + BINS;                            // the cluster's
  float* cache = reinterpret_cast<float*>(sums + BINS);
  __shared__ uint32_t warp_sums[THREADS / 32];
  __shared__ int pick_sh[2], counts[2][CLUSTER];
  const int tid = threadIdx.x;
  const int old = L - a.recent, want = a.budget - a.recent;  // old > want >= 0
  const int windows = (L + SEL_WINDOW - 1) / SEL_WINDOW;
  const bool cached = windows * SHARE * 4 <= room - 2 * BINS * 4;
  // of this CTA's i-th weight
  const auto position = [&](int i) { return i / SHARE * SEL_WINDOW + rank * SHARE + i % SHARE; };
  const bool wide = (reinterpret_cast<uintptr_t>(w) & 15) == 0;
  // four weights from position j on (zeros past the end)
  const auto load4 = [&](int j) {
    if (wide && j + 4 <= L) return *reinterpret_cast<const float4*>(w + j);
    return make_float4(j < L ? w[j] : 0.f, j + 1 < L ? w[j + 1] : 0.f, j + 2 < L ? w[j + 2] : 0.f, j + 3 < L ? w[j + 3] : 0.f);
  };
  if (cached) {
#pragma unroll 4
    for (int n = 0; n < windows; ++n) reinterpret_cast<float4*>(cache)[n * THREADS + tid] = load4(position(n * SHARE + 4 * tid));
  }
  // threshold: the want-th largest image, and how many equal to it are kept
  uint32_t thr = 0u, mask = 0u;
  int need = want;
  if (want > 0) {
#pragma unroll 1
    for (int step = 0; step < 3; ++step) {
      const int shift = step == 0 ? 21 : step == 1 ? 10 : 0, bins = step == 2 ? 1024 : 2048;
#pragma unroll
      for (int i = tid; i < BINS; i += THREADS) hist[i] = 0;
      __syncthreads();
#pragma unroll 2
      for (int n = 0; n < windows; ++n) {
        const int j = position(n * SHARE + 4 * tid);
        const float4 x = cached ? reinterpret_cast<const float4*>(cache)[n * THREADS + tid] : load4(j);
        const float f[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t u = order_of(f[i]);
          if (j + i < old && (u & mask) == thr) atomicAdd(&hist[(u >> shift) & (bins - 1)], 1);
        }
      }
      cluster_sync();
      {  // an eighth of the bins each, and their sums to everyone
        constexpr int MINE = BINS / CLUSTER;
        static_assert(MINE == THREADS, "a bin a thread");
        const int bin = rank * MINE + tid;
        int s = 0;
#pragma unroll
        for (int r = 0; r < CLUSTER; ++r) s += cluster_load(in_cta(hist + bin, r));
#pragma unroll
        for (int r = 0; r < CLUSTER; ++r) cluster_store(in_cta(sums + bin, r), s);
      }
      cluster_sync();
      // digit d with count(> d) < need <= count(>= d), from the top: eight bins a thread
      constexpr int PER = BINS / THREADS;
      const int top = BINS - 1 - PER * tid;
      int c[PER], all = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) all += c[i] = sums[top - i];
      uint32_t total;
      int above = (int)block_exclusive((uint32_t)all, warp_sums, total);
      if (above < need && need <= above + all) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          if (above < need && need <= above + c[i]) {
            pick_sh[0] = top - i;
            pick_sh[1] = above;
          }
          above += c[i];
        }
      }
      __syncthreads();
      thr |= (uint32_t)pick_sh[0] << shift;
      mask |= (uint32_t)(bins - 1) << shift;
      need -= pick_sh[1];
      __syncthreads();
    }
  } else {
    cluster_sync();  // (shared memory of a CTA that has not begun is nobody's to write)
  }
  // Ordered pass, four consecutive positions a thread.  A window's weights are all read before any is written, and no
  // write passes the window's end.
  int n_above = 0, n_equal = 0;  // kept for their weight or age, and equal to the threshold, before the window
#pragma unroll 1
  for (int n = 0; n < windows; ++n) {
    const int j = position(n * SHARE + 4 * tid);
    const float4 x = cached ? reinterpret_cast<const float4*>(cache)[n * THREADS + tid] : load4(j);
    const float f[4] = {x.x, x.y, x.z, x.w};
    uint32_t keep = 0, equal = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = order_of(f[i]);
      const bool cand = want > 0 && j + i < old;
      keep |= (uint32_t)((j + i < L && j + i >= old) || (cand && u > thr)) << i;
      equal |= (uint32_t)(cand && u == thr) << i;
    }
    uint32_t total;
    const uint32_t before = block_exclusive((uint32_t)__popc(keep) | (uint32_t)__popc(equal) << 16, warp_sums, total);
    if (tid < CLUSTER) cluster_store(in_cta(&counts[n & 1][rank], tid), (int)total);
    cluster_sync();
    int na = n_above + (int)(before & 0xffffu), ne = n_equal + (int)(before >> 16);
#pragma unroll
    for (int r = 0; r < CLUSTER; ++r) {
      const uint32_t c = (uint32_t)counts[n & 1][r];
      if (r < rank) {
        na += (int)(c & 0xffffu);
        ne += (int)(c >> 16);
      }
      n_above += (int)(c & 0xffffu);
      n_equal += (int)(c >> 16);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool e = (equal >> i) & 1, k = (keep >> i) & 1;
      if (k || (e && ne < need)) {
        const int at = na + min(ne, need);
        kept[at] = j + i;
        w[at] = f[i];
      }
      na += k;
      ne += e;
    }
  }
}

// 16-byte row r (0..7) of pair p's 128 bytes of values sits at 16 ((r + 2 (p & 3)) & 7)
__device__ __forceinline__ int v_row(int p, int r) { return 128 * p + 16 * ((r + 2 * (p & 3)) & 7); }

template <int KF>
__global__ void __cluster_dims__(CLUSTER, 1, 1) __launch_bounds__(THREADS) evict_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(16) uint8_t images[];  // [2][HPW][half_bytes]
  __shared__ int src_sh[2][HPW * HALF];              // source token (within its half-page) of each slot
  __shared__ const uint8_t* base_sh[2][HPW * HALF];  // the half-page that holds it (null: on a bad page)
  const int tid = threadIdx.x, rank = blockIdx.x % CLUSTER, unit = blockIdx.x / CLUSTER;  // ((ll * batch) + b) * Hkv + h
  const int h = unit % a.Hkv, b = (unit / a.Hkv) % a.batch, layer = a.layer0 + unit / (a.Hkv * a.batch);
  const bool first = h == 0 && unit < a.batch * a.Hkv && rank == 0 && tid == 0;
  const int L = checked_len(a, b, first);
  int32_t* kept = a.kept + (size_t)unit * a.budget;
  if (first) a.new_lens[b] = min(L, a.budget);
  if (L <= a.budget) {  // (the whole cluster)
    for (int j = rank * THREADS + tid; j < a.budget; j += CLUSTER * THREADS) kept[j] = j < L ? j : -1;
    return;
  }
  select_kept(a, a.weights + (size_t)unit * a.max_seq_len, kept, L, rank, images, 2 * HPW * a.L.half_bytes);
  cluster_sync();  // the list is complete
  const size_t page_stride = (size_t)a.Hkv * a.L.page_bytes;
  uint8_t* pages = a.p.pages + ((size_t)layer * a.L.n_pages * a.Hkv + h) * (size_t)a.L.page_bytes;
  const int32_t* bt = a.block_table + (size_t)b * a.max_pages_per_seq;
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
    constexpr int NK = HPW * HALF * CH / THREADS, NV = HPW * HALF * 4 / THREADS, NM = HPW * HALF * 8 / THREADS;
    uint4 k[NK], x[NV], y[NV], km = zero;
    uint16_t vm[NM];
#pragma unroll
    for (int q = 0; q < NK; ++q) {  // keys (Q8G32: chunk m at 16 (m ^ (token & 1)))
      const int i = q * THREADS + tid, t = i / CH, m = i % CH;
      k[q] = zero;
      if (t < n * HALF && base[t])
        k[q] = *reinterpret_cast<const uint4*>(base[t] + (src[t] * CH + (KF == KVQ_Q8G32 ? m ^ (src[t] & 1) : m)) * 16);
    }
#pragma unroll
    for (int q = 0; q < NV; ++q) {  // values: 16-byte row r of a pair holds both tokens' bytes interleaved
      const int i = q * THREADS + tid, pr = i >> 3, r = i & 7;
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
      const int i = q * THREADS + tid, t = i / CH, m = i % CH, td = t % HALF;
      if (t < n * HALF)
        *reinterpret_cast<uint4*>(img0 + t / HALF * hb + (td * CH + (KF == KVQ_Q8G32 ? m ^ (td & 1) : m)) * 16) = k[q];
    }
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      const int i = q * THREADS + tid, pr = i >> 3, r = i & 7;
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
    for (int i = tid; i < n * chunks; i += THREADS) {
      const int half = i / chunks, g = half0 + half, phys = bt[g * HALF / PAGE];
      if (phys >= 0 && phys < a.L.n_pages)
        reinterpret_cast<uint4*>(pages + (size_t)phys * page_stride + (size_t)(g & 1) * hb)[i % chunks] = img[i];
    }
    __syncthreads();  // (the images are free for the window after next)
  }
  if (a.W > 0 && (L - a.budget) % a.W != 0) {
    const size_t at = (((size_t)layer * a.max_batch + b) * a.Hkv + h) * (size_t)a.W * D;
    turn_ring(a, a.p.ringk + at, (L - a.budget) % a.W, rank, reinterpret_cast<float4*>(images), 2 * HPW * hb);
    turn_ring(a, a.p.ringv + at, (L - a.budget) % a.W, rank, reinterpret_cast<float4*>(images), 2 * HPW * hb);
  }
}

template <int KF>
cudaError_t launch_format(const EvictArgs& a, cudaStream_t s) {
  return go<evict_kernel<KF>>(dim3((unsigned)a.n_units * CLUSTER), THREADS, 2 * HPW * (size_t)a.L.half_bytes, false, s, a);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  return a.k_format == KVQ_TQ3_QJL ? launch_format<KVQ_TQ3_QJL>(a, s)
         : a.k_format == KVQ_Q8G32 ? launch_format<KVQ_Q8G32>(a, s)
                                   : launch_format<KVQ_Q4G32>(a, s);
}

}  // namespace kvq

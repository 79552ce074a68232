// Pages of a cache taken, shared, copied, given back and moved together, all on the device (kv_pool_*).
//
// State: refs[n_pages], how many entries of the block table name each page, and the table.  A free page is one with refs
// 0; the lowest is taken first.  Planning (which entry gets which page) is one CTA's work: prefix sums over the call's
// entries, then over refs.  What weighs is moved by a second, wide launch, a programmatic dependent of the plan, from the
// plan's list of (from, to) pages: a page of one layer is contiguous, n_kv_heads * page_bytes.
#include "kvq_internal.cuh"

namespace kvq {

namespace {

constexpr int PLAN = 1024;          // threads of a planning CTA
constexpr int COPY_THREADS = 256;
constexpr int COPY_VECS = 4;        // 16-byte vectors under way per thread
constexpr int COLS = 32;            // table columns of a fork's table CTA

// Inclusive prefix sum over the CTA's PLAN threads; total gets the sum.  sums: 33 ints.
__device__ __forceinline__ int block_scan(int v, int* sums, int& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(FULL, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();  // (the sums of the scan before have been read)
  if (lane == 31) sums[w] = incl;
  __syncthreads();
  if (w == 0) {
    int s = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(FULL, s, o);
      if (lane >= o) s += y;
    }
    sums[lane] = s;
  }
  __syncthreads();
  total = sums[31];
  return incl + (w > 0 ? sums[w - 1] : 0);
}

// The free pages in ascending order into pick[0 ..], until there are `want` of them; how many there are (up to the end
// of the stretch that holds the last wanted one).
__device__ int list_free(const PoolArgs& a, int want, int* sums) {
  int found = 0;
  for (int p0 = 0; p0 < a.L.n_pages && found < want; p0 += PLAN) {
    const int p = p0 + threadIdx.x;
    const bool is = p < a.L.n_pages && __ldcg(a.refs + p) == 0;
    int total;
    const int at = found + block_scan(is, sums, total) - 1;
    if (is) a.pick[at] = p;
    found += total;
  }
  return found;
}

struct Item {
  int b, lp, page;  // page -1: none
};

__global__ void __launch_bounds__(PLAN) reserve_kernel(const __grid_constant__ PoolArgs a) {
  __shared__ int sums[33];
  __shared__ int start[PLAN + 1], first[PLAN], needs[PLAN];
  __shared__ int n_copies;
  const int t = threadIdx.x, n_pages = a.L.n_pages, mpp = a.L.max_pages_per_seq;
  asm volatile("griddepcontrol.launch_dependents;");
  // the pages that each sequence's positions touch
  int p = -1, pages = 0;
  if (t < a.batch) {
    p = a.pos[t];
    const int n = a.counts ? max(a.counts[t], 0) : a.n_tokens;
    if (p >= 0 && (long long)p + n > a.max_seq_len) {
      atomicOr(a.p.status, KVQ_DEV_POS_RANGE);
      p = -1;
    }
    if (p >= 0 && n > 0) pages = (p + n - 1) / PAGE - p / PAGE + 1;
    first[t] = p / PAGE;
  }
  needs[t] = 0;
  if (t == 0) n_copies = 0;
  int items;
  const int incl = block_scan(pages, sums, items);
  start[t] = incl - pages;
  if (t == PLAN - 1) start[PLAN] = incl;
  __syncthreads();
  auto item = [&](int i) {
    int lo = 0, hi = a.batch - 1;
    while (lo < hi) {  // the last sequence that starts at or before i (those without pages start where the next does)
      const int mid = (lo + hi + 1) >> 1;
      if (start[mid] <= i) lo = mid;
      else hi = mid - 1;
    }
    Item it;
    it.b = lo;
    it.lp = first[lo] + i - start[lo];
    const int e = __ldcg(a.table + (size_t)lo * mpp + it.lp);
    it.page = e >= 0 && e < n_pages ? e : -1;
    return it;
  };
  // pages that several entries name: how many of the call's would write each, and the last of them
  for (int i = t; i < items; i += PLAN) {
    const Item it = item(i);
    if (it.page >= 0 && __ldcg(a.refs + it.page) > 1) {
      atomicAdd(a.writers + it.page, 1);
      atomicMax(a.last + it.page, i);
    }
  }
  __syncthreads();
  // 0: has its page, 1: needs one, 2: needs a copy
  auto need = [&](const Item& it, int i) {
    if (it.page < 0) return 1;
    const int r = __ldcg(a.refs + it.page);
    if (r <= 1) return 0;
    return __ldcg(a.writers + it.page) == r && __ldcg(a.last + it.page) == i ? 0 : 2;
  };
  for (int i = t; i < items; i += PLAN) {
    const Item it = item(i);
    if (need(it, i)) atomicAdd(&needs[it.b], 1);
  }
  __syncthreads();
  int wanted;
  const int upto = block_scan(needs[t], sums, wanted);
  const int found = list_free(a, wanted, sums);
  const bool fits = upto <= found;
  __syncthreads();
  needs[t] = fits;
  if (t < a.batch) {
    if (!fits && p >= 0) atomicOr(a.p.status, KVQ_DEV_NO_PAGES);
    a.out[t] = fits ? (p >= 0 ? p : -1) : -1;
  }
  __syncthreads();
  int taken = 0;
  for (int i0 = 0; i0 < items; i0 += PLAN) {
    const int i = i0 + t;
    Item it = {0, 0, -1};
    int kind = 0;
    if (i < items) {
      it = item(i);
      kind = need(it, i);
    }
    int total;
    const int at = taken + block_scan(kind != 0, sums, total) - 1;
    taken += total;
    if (kind != 0 && needs[it.b]) {
      const int page = __ldcg(a.pick + at);
      a.table[(size_t)it.b * mpp + it.lp] = page;
      a.refs[page] = 1;
      if (kind == 2) a.copies[atomicAdd(&n_copies, 1)] = make_int2(it.page, page);
    }
  }
  __syncthreads();
  // the counts of shared pages, and their marks as they were
  for (int c = t; c < n_copies; c += PLAN) {
    const int from = __ldcg(a.copies + c).x;
    atomicSub(a.refs + from, 1);
    a.writers[from] = 0;
    a.last[from] = -1;
  }
  for (int i = t; i < items; i += PLAN) {
    const Item it = item(i);
    if (it.page >= 0 && __ldcg(a.writers + it.page) != 0) {
      a.writers[it.page] = 0;
      a.last[it.page] = -1;
    }
  }
  if (t == 0) *a.n_copies = n_copies;
}

// Pages in use: U of them.  Those from U on and the free ones below U, each in order, are the moves' two ends.
__global__ void __launch_bounds__(PLAN) compact_kernel(const __grid_constant__ PoolArgs a) {
  __shared__ int sums[33];
  const int t = threadIdx.x, n_pages = a.L.n_pages;
  asm volatile("griddepcontrol.launch_dependents;");
  int mine = 0;
  for (int p = t; p < n_pages; p += PLAN) mine += __ldcg(a.refs + p) > 0;
  int used;
  block_scan(mine, sums, used);
  int free_ends = 0, moves = 0;
  for (int p0 = 0; p0 < n_pages; p0 += PLAN) {
    const int p = p0 + t;
    const bool in_use = p < n_pages && __ldcg(a.refs + p) > 0;
    const bool hole = p < used && !in_use, mover = in_use && p >= used;
    int total;
    // (a stretch of PLAN pages may hold both ends: counted in the two halves of one sum)
    const int at = block_scan((int)hole | ((int)mover << 16), sums, total);
    if (hole) a.copies[free_ends + (at & 0xffff) - 1].y = p;
    if (mover) a.copies[moves + (at >> 16) - 1].x = p;
    free_ends += total & 0xffff;
    moves += total >> 16;
  }
  __syncthreads();
  for (int c = t; c < moves; c += PLAN) {
    const int2 m = __ldcg(a.copies + c);
    a.pick[m.x] = m.y;
    a.refs[m.y] = __ldcg(a.refs + m.x);
    a.refs[m.x] = 0;
  }
  if (t == 0) {
    *a.n_copies = moves;
    *a.out = used;
  }
}

// The plan's copies, every layer of each page; TABLE: entries that name a moved page follow it.
template <bool TABLE>
__global__ void __launch_bounds__(COPY_THREADS) copy_kernel(const __grid_constant__ PoolArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = __ldcg(a.n_copies);
  if (n == 0) return;
  if (TABLE) {
    const int used = __ldcg(a.out);
    const long long entries = (long long)a.max_batch * a.L.max_pages_per_seq;
    for (long long i = (long long)blockIdx.x * COPY_THREADS + threadIdx.x; i < entries; i += (long long)gridDim.x * COPY_THREADS) {
      const int e = a.table[i];
      if (e >= used && e < a.L.n_pages) a.table[i] = __ldcg(a.pick + e);
    }
  }
  const size_t bytes = (size_t)a.Hkv * a.L.page_bytes;  // of one layer's page
  const int vecs = (int)(bytes / 16);
  const int parts = (vecs + COPY_THREADS * COPY_VECS - 1) / (COPY_THREADS * COPY_VECS);
  const long long work = (long long)n * a.n_layers * parts;
  for (long long w = blockIdx.x; w < work; w += gridDim.x) {
    const int part = (int)(w % parts);
    const long long r = w / parts;
    const int layer = (int)(r % a.n_layers);
    const int2 c = __ldcg(a.copies + r / a.n_layers);
    const uint4* src = reinterpret_cast<const uint4*>(a.p.pages + ((size_t)layer * a.L.n_pages + c.x) * bytes);
    uint4* dst = reinterpret_cast<uint4*>(a.p.pages + ((size_t)layer * a.L.n_pages + c.y) * bytes);
    const int v0 = part * COPY_THREADS * COPY_VECS + threadIdx.x;
    uint4 x[COPY_VECS];
#pragma unroll
    for (int i = 0; i < COPY_VECS; ++i)
      if (v0 + i * COPY_THREADS < vecs) x[i] = __ldcs(src + v0 + i * COPY_THREADS);
#pragma unroll
    for (int i = 0; i < COPY_VECS; ++i)
      if (v0 + i * COPY_THREADS < vecs) dst[v0 + i * COPY_THREADS] = x[i];
  }
}

// what a fork's CTAs go by: each sequence's parent (itself where it stays as it is) and the parent's length
__device__ __forceinline__ int parent_of(const PoolArgs& a, int b, bool flag) {
  const int q = a.pos[b];
  if (q >= 0 && q < a.batch) return q;
  if (q != -1 && flag) atomicOr(a.p.status, KVQ_DEV_BAD_PARENT);
  return b;
}
__device__ __forceinline__ int length_of(const PoolArgs& a, int b, bool flag) {
  const int n = a.counts[b];
  if (n >= 0 && n <= a.max_seq_len) return n;
  if (flag) atomicOr(a.p.status, KVQ_DEV_SEQLEN_RANGE);
  return 0;
}

// Blocks below table_ctas: COLS columns of the table each, all sequences of the call (entries of a page are in one
// column: its counts are one block's).  The others: `slice` bytes of the rings of one (layer, head, keys or values),
// every parent's read before any child's is written.
__global__ void __launch_bounds__(COPY_THREADS) fork_kernel(const __grid_constant__ PoolArgs a, int table_ctas, int slice) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int t = threadIdx.x, B = a.batch;
  if ((int)blockIdx.x < table_ctas) {
    int* old = reinterpret_cast<int*>(smem);  // [B][COLS]
    const int mpp = a.L.max_pages_per_seq, c = blockIdx.x * COLS + (t & (COLS - 1));
    const bool here = c < mpp;
    for (int b = t / COLS; b < B; b += COPY_THREADS / COLS) old[b * COLS + (t & (COLS - 1))] = here ? a.table[(size_t)b * mpp + c] : -1;
    if (blockIdx.x == 0)
      for (int b = t; b < B; b += COPY_THREADS) a.out[b] = length_of(a, parent_of(a, b, true), true);
    __syncthreads();
    for (int b = t / COLS; b < B; b += COPY_THREADS / COLS) {
      const int q = parent_of(a, b, false);
      if (q == b || !here) continue;
      const int was = old[b * COLS + (t & (COLS - 1))];
      const int now = c < (length_of(a, q, false) + PAGE - 1) / PAGE ? old[q * COLS + (t & (COLS - 1))] : -1;
      if (was == now) continue;
      if (was >= 0 && was < a.L.n_pages) atomicSub(a.refs + was, 1);
      if (now >= 0 && now < a.L.n_pages) atomicAdd(a.refs + now, 1);
      a.table[(size_t)b * mpp + c] = now;
    }
    return;
  }
  const size_t ring = (size_t)a.W * D * sizeof(float);  // of one (layer, sequence, head)
  const int parts = (int)((ring + slice - 1) / slice);
  unsigned r = blockIdx.x - table_ctas;
  const int part = (int)(r % parts);
  r /= parts;
  const int h = (int)(r % a.Hkv);
  r /= a.Hkv;
  const int kv = (int)(r & 1), layer = (int)(r >> 1);
  const size_t off = (size_t)part * slice;
  uint8_t* base = reinterpret_cast<uint8_t*>(kv ? a.p.ringv : a.p.ringk) + ((size_t)layer * a.max_batch * a.Hkv + h) * ring + off;
  const size_t step = (size_t)a.Hkv * ring;  // from one sequence to the next
  int* parent = reinterpret_cast<int*>(smem);
  int* bytes = parent + B;  // of the parent's slice that hold tokens
  int* wanted = bytes + B;
  uint8_t* held = smem + ((size_t)3 * B * 4 + 15) / 16 * 16;
  for (int b = t; b < B; b += COPY_THREADS) {
    const int q = parent_of(a, b, false);
    parent[b] = q;
    const long long n = (long long)min(length_of(a, q, false), a.W) * D * 4 - (long long)off;
    bytes[b] = (int)max(0LL, min((long long)min((size_t)slice, ring - off), n));
    wanted[b] = 0;
  }
  __syncthreads();
  for (int b = t; b < B; b += COPY_THREADS)
    if (parent[b] != b) wanted[parent[b]] = bytes[b];
  __syncthreads();
  const int vecs = slice / 16;
  for (int i = t; i < B * vecs; i += COPY_THREADS) {
    const int b = i / vecs, v = i % vecs;
    if (16 * v < wanted[b]) *reinterpret_cast<uint4*>(held + (size_t)i * 16) = __ldcs(reinterpret_cast<const uint4*>(base + b * step) + v);
  }
  __syncthreads();
  for (int i = t; i < B * vecs; i += COPY_THREADS) {
    const int b = i / vecs, v = i % vecs;
    if (parent[b] != b && 16 * v < bytes[b])
      reinterpret_cast<uint4*>(base + b * step)[v] = *reinterpret_cast<const uint4*>(held + ((size_t)parent[b] * vecs + v) * 16);
  }
}

__global__ void __launch_bounds__(COPY_THREADS) release_kernel(const __grid_constant__ PoolArgs a) {
  const int mpp = a.L.max_pages_per_seq;
  const long long n = (long long)a.batch * mpp;
  for (long long i = (long long)blockIdx.x * COPY_THREADS + threadIdx.x; i < n; i += (long long)gridDim.x * COPY_THREADS) {
    const int b = (int)(i / mpp), lp = (int)(i % mpp);
    const int keep = a.pos[b];
    if (keep < 0 || (long long)lp * PAGE < keep) continue;
    const int e = a.table[i];
    if (e < 0) continue;
    if (e < a.L.n_pages) atomicSub(a.refs + e, 1);
    a.table[i] = -1;
  }
}

__global__ void __launch_bounds__(COPY_THREADS) init_kernel(const __grid_constant__ PoolArgs a) {
  const long long entries = (long long)a.max_batch * a.L.max_pages_per_seq;
  const long long n = max(entries, (long long)a.L.n_pages);
  for (long long i = (long long)blockIdx.x * COPY_THREADS + threadIdx.x; i < n; i += (long long)gridDim.x * COPY_THREADS) {
    if (i < entries) a.table[i] = -1;
    if (i < a.L.n_pages) {
      a.refs[i] = 0;
      a.writers[i] = 0;
      a.last[i] = -1;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.n_copies = 0;
}

unsigned blocks_for(long long threads) {
  const long long b = (threads + COPY_THREADS - 1) / COPY_THREADS;
  return (unsigned)(b < 1 ? 1 : b > 2048 ? 2048 : b);
}

template <bool TABLE>
cudaError_t launch_copies(const PoolArgs& a, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(8 * sms));
  cfg.blockDim = dim3(COPY_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, copy_kernel<TABLE>, a);
}

}  // namespace

size_t pool_layout(void* pool, int n_pages, PoolArgs* a) {
  const size_t n = align256((size_t)n_pages * sizeof(int32_t));
  uint8_t* b = static_cast<uint8_t*>(pool);
  if (b) {
    a->refs = reinterpret_cast<int32_t*>(b);
    a->n_copies = reinterpret_cast<int32_t*>(b + n);
    a->writers = reinterpret_cast<int32_t*>(b + n + 256);
    a->last = reinterpret_cast<int32_t*>(b + 2 * n + 256);
    a->pick = reinterpret_cast<int32_t*>(b + 3 * n + 256);
    a->copies = reinterpret_cast<int2*>(b + 4 * n + 256);
  }
  return 6 * n + 256;
}

cudaError_t launch_pool_init(const PoolArgs& a, cudaStream_t s) {
  const long long entries = (long long)a.max_batch * a.L.max_pages_per_seq;
  init_kernel<<<blocks_for(entries > a.L.n_pages ? entries : a.L.n_pages), COPY_THREADS, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_pool_reserve(const PoolArgs& a, cudaStream_t s) {
  static_assert(MAX_BATCH <= PLAN, "a thread for each sequence");
  reserve_kernel<<<1, PLAN, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_copies<false>(a, s);
}

cudaError_t launch_pool_compact(const PoolArgs& a, cudaStream_t s) {
  compact_kernel<<<1, PLAN, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_copies<true>(a, s);
}

cudaError_t launch_pool_fork(const PoolArgs& a, cudaStream_t s) {
  const int table_ctas = (a.L.max_pages_per_seq + COLS - 1) / COLS;
  const size_t ring = (size_t)a.W * D * sizeof(float);
  // slices of every sequence's ring side by side: about 32 KB of them a block, so that several blocks share an SM, but
  // whole 128-byte lines
  int slice = 32 * 1024 / a.batch / 128 * 128;
  slice = slice < 128 ? 128 : slice > 4096 ? 4096 : slice;
  const long long ring_ctas = (long long)2 * a.n_layers * a.Hkv * (long long)((ring + slice - 1) / slice);
  if (table_ctas + ring_ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  const size_t table_smem = (size_t)a.batch * COLS * 4, ring_smem = ((size_t)3 * a.batch * 4 + 15) / 16 * 16 + (size_t)a.batch * slice;
  const size_t smem = table_smem > ring_smem ? table_smem : ring_smem;
  const cudaError_t e = allow_shared_memory<fork_kernel>();
  if (e != cudaSuccess) return e;
  fork_kernel<<<(unsigned)(table_ctas + ring_ctas), COPY_THREADS, smem, s>>>(a, table_ctas, slice);
  return cudaGetLastError();
}

cudaError_t launch_pool_release(const PoolArgs& a, cudaStream_t s) {
  release_kernel<<<blocks_for((long long)a.batch * a.L.max_pages_per_seq), COPY_THREADS, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq

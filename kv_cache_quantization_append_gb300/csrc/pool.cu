// Pages of a cache taken, shared, copied, given back and moved together, all on the device (kv_pool_*).
//
// State: refs[n_pages], how many entries of the block table name each page, and the table.  A free page is one with refs
// 0; the lowest is taken first.  Planning (which entry gets which page) is one CTA's work: prefix sums over the call's
// entries, then over refs.  It is a chain of barriers and of trips to L2, so a call of few sequences takes a quarter of
// the threads.  What weighs is moved by a second, wide launch, a programmatic dependent of the plan, from the plan's list
// of (from, to) pages: a page of one layer is contiguous, n_kv_heads * page_bytes.
//
// Measured: 64 sequences take and give back 15 pages each in 18 us on the device; 123 pages of 8 layers (131 KB each) move in 38 us, the copy
// rate; a plan without copies 5 us, 1.5 of them the second launch's end.
#include "tc.cuh"

namespace kvq {

namespace {

constexpr int PLAN = 1024, PLAN_FEW = 256;  // threads of a planning CTA
constexpr int COPY_THREADS = 512;
constexpr int COPY_VECS = 4;        // 16-byte vectors under way per thread
constexpr int THREADS = 256;
constexpr int COLS = 32;            // table columns of a fork's table CTA
constexpr int FORK_SMEM = 96 * 1024, FORK_STAGES = 3, FORK_STAGE = FORK_SMEM / FORK_STAGES, MAX_SLICE = 16 * 1024, FORK_LISTS = 5;

// Inclusive prefix sum over the CTA's N threads; total gets the sum.  sums: 32 ints.
template <int N>
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
  // every warp adds up the warps' sums for itself
  int s = lane < N / 32 ? sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < N / 32; o <<= 1) {
    const int y = __shfl_up_sync(FULL, s, o);
    if (lane >= o) s += y;
  }
  total = __shfl_sync(FULL, s, N / 32 - 1);
  const int before = __shfl_sync(FULL, s, w > 0 ? w - 1 : 0);
  return incl + (w > 0 ? before : 0);
}

// The free pages in ascending order into pick[0 ..], until there are `want` of them; how many there are (up to the end
// of the stretch that holds the last wanted one).
template <int N>
__device__ int list_free(const PoolArgs& a, int want, int* sums) {
  int found = 0;
  for (int p0 = 0; p0 < a.L.n_pages && found < want; p0 += 4 * N) {
    const int p = p0 + 4 * threadIdx.x;
    int4 r = make_int4(1, 1, 1, 1);  // (refs has room for whole vectors: what follows it is 256 bytes aligned)
    if (p < a.L.n_pages) r = __ldcg(reinterpret_cast<const int4*>(a.refs + p));
    const bool is[4] = {r.x == 0, r.y == 0 && p + 1 < a.L.n_pages, r.z == 0 && p + 2 < a.L.n_pages, r.w == 0 && p + 3 < a.L.n_pages};
    int total;
    int at = found + block_scan<N>(is[0] + is[1] + is[2] + is[3], sums, total) - (is[0] + is[1] + is[2] + is[3]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (is[k]) a.pick[at++] = p + k;
    found += total;
  }
  return found;
}

struct Item {
  int b, lp, page;  // page -1: none
};

template <int N>
__global__ void __launch_bounds__(N) reserve_kernel(const __grid_constant__ PoolArgs a) {
  __shared__ int sums[32];
  __shared__ int start[N], first[N], needs[N];
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
  start[t] = block_scan<N>(pages, sums, items) - pages;
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
  // entries without a page; pages that several entries name: how many of the call's would write each, and the last of them
  bool shares = false;
  Item own = {0, 0, 0};  // of i = t
  for (int i = t; i < items; i += N) {
    const Item it = item(i);
    if (i == t) own = it;
    if (it.page < 0) {
      atomicAdd(&needs[it.b], 1);
    } else if (__ldcg(a.refs + it.page) > 1) {
      shares = true;
      atomicAdd(a.writers + it.page, 1);
      atomicMax(a.last + it.page, i);
    }
  }
  shares = __syncthreads_or(shares);
  // 0: has its page, 1: needs one, 2: needs a copy
  auto need = [&](const Item& it, int i) {
    if (it.page < 0) return 1;
    if (!shares) return 0;
    const int r = __ldcg(a.refs + it.page);
    if (r <= 1) return 0;
    return __ldcg(a.writers + it.page) == r && __ldcg(a.last + it.page) == i ? 0 : 2;
  };
  if (shares) {
    for (int i = t; i < items; i += N) {
      const Item it = item(i);
      if (need(it, i) == 2) atomicAdd(&needs[it.b], 1);
    }
    __syncthreads();
  }
  int wanted;
  const int upto = block_scan<N>(needs[t], sums, wanted);
  const int found = list_free<N>(a, wanted, sums);
  const bool fits = upto <= found;
  __syncthreads();
  needs[t] = fits;
  if (t < a.batch) {
    if (!fits && p >= 0) atomicOr(a.p.status, KVQ_DEV_NO_PAGES);
    a.out[t] = fits ? p : -1;
  }
  __syncthreads();
  if (wanted > 0) {
    int taken = 0;
    for (int i0 = 0; i0 < items; i0 += N) {
      const int i = i0 + t;
      Item it = {0, 0, -1};
      int kind = 0;
      if (i < items) {
        it = i == t ? own : item(i);
        kind = need(it, i);
      }
      int total;
      const int at = taken + block_scan<N>(kind != 0, sums, total) - 1;
      taken += total;
      if (kind != 0 && needs[it.b]) {
        const int page = __ldcg(a.pick + at);
        a.table[(size_t)it.b * mpp + it.lp] = page;
        a.refs[page] = 1;
        if (kind == 2) a.copies[atomicAdd(&n_copies, 1)] = make_int2(it.page, page);
      }
    }
    __syncthreads();
  }
  if (shares) {
    // the counts of shared pages, and their marks as they were
    for (int c = t; c < n_copies; c += N) {
      const int from = __ldcg(a.copies + c).x;
      atomicSub(a.refs + from, 1);
      a.writers[from] = 0;
      a.last[from] = -1;
    }
    for (int i = t; i < items; i += N) {
      const Item it = item(i);
      if (it.page >= 0 && __ldcg(a.writers + it.page) != 0) {
        a.writers[it.page] = 0;
        a.last[it.page] = -1;
      }
    }
  }
  if (t == 0) *a.n_copies = n_copies;
}

// Pages in use: U of them.  Those from U on and the free ones below U, each in order, are the moves' two ends.
template <int N>
__global__ void __launch_bounds__(N) compact_kernel(const __grid_constant__ PoolArgs a) {
  __shared__ int sums[32];
  const int t = threadIdx.x, n_pages = a.L.n_pages;
  asm volatile("griddepcontrol.launch_dependents;");
  int mine = 0;
  for (int p = t; p < n_pages; p += N) mine += __ldcg(a.refs + p) > 0;
  int used;
  block_scan<N>(mine, sums, used);
  int free_ends = 0, moves = 0;
  for (int p0 = 0; p0 < n_pages; p0 += N) {
    const int p = p0 + t;
    const bool in_use = p < n_pages && __ldcg(a.refs + p) > 0;
    const bool hole = p < used && !in_use, mover = in_use && p >= used;
    int total;
    // (a stretch of pages may hold both ends: counted in the two halves of one sum)
    const int at = block_scan<N>((int)hole | ((int)mover << 16), sums, total);
    if (hole) a.copies[free_ends + (at & 0xffff) - 1].y = p;
    if (mover) a.copies[moves + (at >> 16) - 1].x = p;
    free_ends += total & 0xffff;
    moves += total >> 16;
  }
  __syncthreads();
  for (int c = t; c < moves; c += N) {
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

// What a fork does to the block table: COLS columns of it, all sequences of the call (entries that name a page are in one
// column: its counts are one block's)
__device__ void fork_table(const PoolArgs& a, int* old) {
  const int t = threadIdx.x, B = a.batch, mpp = a.L.max_pages_per_seq, col = t & (COLS - 1), c = blockIdx.x * COLS + col;
  const bool here = c < mpp;
  for (int b = t / COLS; b < B; b += THREADS / COLS) old[b * COLS + col] = here ? a.table[(size_t)b * mpp + c] : -1;
  if (blockIdx.x == 0)
    for (int b = t; b < B; b += THREADS) a.out[b] = length_of(a, parent_of(a, b, true), true);
  __syncthreads();
  for (int b = t / COLS; b < B; b += THREADS / COLS) {
    const int q = parent_of(a, b, false);
    if (q == b || !here) continue;
    const int was = old[b * COLS + col];
    const int now = c < (length_of(a, q, false) + PAGE - 1) / PAGE ? old[q * COLS + col] : -1;
    if (was == now) continue;
    if (was >= 0 && was < a.L.n_pages) atomicSub(a.refs + was, 1);
    if (now >= 0 && now < a.L.n_pages) atomicAdd(a.refs + now, 1);
    a.table[(size_t)b * mpp + c] = now;
  }
}

// The rings.  A task is a slice of one (layer, head, keys or values): every parent's slice comes into shared memory by a
// bulk copy (each parent's once, however many children it has), and once all of them are there each child's goes out by
// another; so beams change places without a second copy of anything.  A CTA goes through its tasks FORK_STAGES deep; one
// warp issues.  Bounded by memory: reads of the parents, writes of the children.  32 children of 4 parents, 28 layers of 8 heads:
// 0.94 GB in 154 us, 6.1 TB/s (through registers, a slice at a time: 215 us); 16 beams that change places 114 us.
__device__ void fork_rings(const PoolArgs& a, uint8_t* smem, int cta, int ctas) {
  __shared__ __align__(8) uint64_t full[FORK_STAGES];
  __shared__ int gone, n_parents, n_children, longest;
  const int t = threadIdx.x, B = a.batch;
  int* slot = reinterpret_cast<int*>(smem);  // of a sequence that is a parent: its place in a stage; -1: it is none
  int* from = slot + B;                      // parents, in the order of their places
  int* held = from + B;                      // bytes of a parent's ring that hold tokens
  int* to = held + B;                        // children
  int* of = to + B;                          // a child's parent's place
  uint8_t* stages = smem + ((size_t)FORK_LISTS * B * 4 + 127) / 128 * 128;
  if (t == 0) {
    for (int i = 0; i < FORK_STAGES; ++i) tc::bar_init(&full[i], 1);
    gone = n_parents = n_children = longest = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  for (int b = t; b < B; b += THREADS) slot[b] = -1;
  __syncthreads();
  for (int b = t; b < B; b += THREADS) {
    const int q = parent_of(a, b, false), n = min(length_of(a, q, false), a.W);
    if (q != b && n > 0) {
      slot[q] = 0;
      const int i = atomicAdd(&n_children, 1);  // (their order does not matter)
      to[i] = b;
      of[i] = q;
      atomicMax(&longest, n);
    }
  }
  __syncthreads();
  for (int b = t; b < B; b += THREADS)
    if (slot[b] == 0) {
      const int s = atomicAdd(&n_parents, 1);
      from[s] = b;
      held[s] = min(length_of(a, b, false), a.W) * D * 4;
      slot[b] = s;
    }
  __syncthreads();
  for (int i = t; i < n_children; i += THREADS) of[i] = slot[of[i]];
  __syncthreads();
  if (t >= 32 || n_children == 0) return;
  const int lane = t, np = n_parents, nc = n_children;
  const int used = longest * D * 4;                                     // bytes of the longest ring that hold tokens
  const int slice = min(min(max(FORK_STAGE / np / 128 * 128, 128), MAX_SLICE), used);
  const int stage_bytes = max(FORK_STAGE, np * slice), n_stages = max(1, min(FORK_STAGES, a.fork_smem / stage_bytes));
  const size_t ring = (size_t)a.W * D * 4, step = (size_t)a.Hkv * ring;  // of one (layer, sequence, head); between sequences
  const int parts = (used + slice - 1) / slice;
  const long long tasks = (long long)2 * a.n_layers * a.Hkv * parts;
  auto bytes_of = [&](int s, int off) { return max(0, min(slice, held[s] - off)); };  // of the slice of parent s's ring
  auto place = [&](long long task, int& off) {
    const int part = (int)(task % parts);
    const long long r = task / parts;
    const int h = (int)(r % a.Hkv);
    const long long kl = r / a.Hkv;
    off = part * slice;
    return reinterpret_cast<uint8_t*>((kl & 1) ? a.p.ringv : a.p.ringk) + ((size_t)(kl >> 1) * a.max_batch * a.Hkv + h) * ring + off;
  };
  auto load = [&](long long task, int st) {
    int off, sum = 0;
    const uint8_t* base = place(task, off);
    for (int i = lane; i < np; i += 32) sum += bytes_of(i, off);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
    if (lane == 0) tc::bar_expect(&full[st], sum);
    __syncwarp();
    for (int i = lane; i < np; i += 32) {
      const int n = bytes_of(i, off);
      if (n > 0) tc::bulk_g2s(stages + (size_t)st * stage_bytes + (size_t)i * slice, base + from[i] * step, n, &full[st]);
    }
  };
  // stage i % n_stages holds the CTA's i-th task
  long long next = cta;
  int loaded = 0;
  for (; loaded < n_stages && next < tasks; ++loaded, next += ctas) load(next, loaded);
  int done = 0;
  for (long long task = cta; task < tasks; task += ctas, ++done) {
    const int st = done % n_stages;
    tc::bar_wait(&full[st], (done / n_stages) & 1, &gone, a.p.status, a.wait_ns);
    if (__any_sync(FULL, *const_cast<volatile int*>(&gone))) break;
    int off;
    uint8_t* base = place(task, off);
    for (int i = lane; i < nc; i += 32) {
      const int n = bytes_of(of[i], off);
      if (n > 0) tc::bulk_s2g(base + to[i] * step, stages + (size_t)st * stage_bytes + (size_t)of[i] * slice, n);
    }
    tc::bulk_commit();
    if (next < tasks) {
      tc::bulk_read_wait();  // the stage's stores have read it
      __syncwarp();
      load(next, st);
      next += ctas;
      ++loaded;
    }
  }
  // what is under way lands before the CTA leaves
  for (; done < loaded; ++done) tc::bar_land(&full[done % n_stages], (done / n_stages) & 1);
  tc::bulk_wait();
}

__global__ void __launch_bounds__(THREADS) fork_kernel(const __grid_constant__ PoolArgs a, int table_ctas) {
  extern __shared__ __align__(128) uint8_t smem[];
  if ((int)blockIdx.x < table_ctas) fork_table(a, reinterpret_cast<int*>(smem));
  else fork_rings(a, smem, blockIdx.x - table_ctas, gridDim.x - table_ctas);
}

__global__ void __launch_bounds__(THREADS) release_kernel(const __grid_constant__ PoolArgs a) {
  const int mpp = a.L.max_pages_per_seq;
  const long long n = (long long)a.batch * mpp;
  for (long long i = (long long)blockIdx.x * THREADS + threadIdx.x; i < n; i += (long long)gridDim.x * THREADS) {
    const int b = (int)(i / mpp), lp = (int)(i % mpp);
    const int keep = a.pos[b];
    if (keep < 0 || (long long)lp * PAGE < keep) continue;
    const int e = a.table[i];
    if (e < 0) continue;
    if (e < a.L.n_pages) atomicSub(a.refs + e, 1);
    a.table[i] = -1;
  }
}

__global__ void __launch_bounds__(THREADS) init_kernel(const __grid_constant__ PoolArgs a) {
  const long long entries = (long long)a.max_batch * a.L.max_pages_per_seq;
  const long long n = max(entries, (long long)a.L.n_pages);
  for (long long i = (long long)blockIdx.x * THREADS + threadIdx.x; i < n; i += (long long)gridDim.x * THREADS) {
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
  const long long b = (threads + THREADS - 1) / THREADS;
  return (unsigned)(b < 1 ? 1 : b > 2048 ? 2048 : b);
}

template <bool TABLE>
cudaError_t launch_copies(const PoolArgs& a, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(3 * sms));
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
  init_kernel<<<blocks_for(entries > a.L.n_pages ? entries : a.L.n_pages), THREADS, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_pool_reserve(const PoolArgs& a, cudaStream_t s) {
  static_assert(MAX_BATCH <= PLAN, "a thread for each sequence");
  // Threads of the plan: for up to 512 entries a quarter of them (a step of 6 sequences 7.6 -> 5.3 us); two entries a thread
  // and more are slower with few (64 sequences of 15 pages 13.7 -> 12 us with all).
  const long long entries = (long long)a.batch * (a.counts ? a.L.max_pages_per_seq : a.n_tokens / PAGE + 2);
  if (a.batch <= PLAN_FEW && entries <= 2 * PLAN_FEW) reserve_kernel<PLAN_FEW><<<1, PLAN_FEW, 0, s>>>(a);
  else reserve_kernel<PLAN><<<1, PLAN, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_copies<false>(a, s);
}

cudaError_t launch_pool_compact(const PoolArgs& a, cudaStream_t s) {
  if (a.L.n_pages <= 4 * PLAN_FEW) compact_kernel<PLAN_FEW><<<1, PLAN_FEW, 0, s>>>(a);
  else compact_kernel<PLAN><<<1, PLAN, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_copies<true>(a, s);
}

cudaError_t launch_pool_fork(const PoolArgs& a0, cudaStream_t s) {
  PoolArgs a = a0;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = allow_shared_memory<fork_kernel>();
  if (e != cudaSuccess) return e;
  const int table_ctas = (a.L.max_pages_per_seq + COLS - 1) / COLS;
  // stages for slices of at least 128 bytes of as many parents as there may be; two blocks share an SM.  As many ring blocks
  // as there are slices of MAX_SLICE at least (more parents make shorter ones), two an SM at most.
  a.fork_smem = a.batch * 128 > FORK_SMEM ? a.batch * 128 : FORK_SMEM;
  const long long ring = (long long)a.W * D * 4;
  const long long slices = (long long)2 * a.n_layers * a.Hkv * ((ring + 2047) / 2048);
  const int ring_ctas = (int)(slices < 2LL * sms ? slices : 2LL * sms);
  const size_t table_smem = (size_t)a.batch * COLS * 4, ring_smem = ((size_t)FORK_LISTS * a.batch * 4 + 127) / 128 * 128 + a.fork_smem;
  const size_t smem = table_smem > ring_smem ? table_smem : ring_smem;
  fork_kernel<<<(unsigned)(table_ctas + ring_ctas), THREADS, smem, s>>>(a, table_ctas);
  return cudaGetLastError();
}

cudaError_t launch_pool_release(const PoolArgs& a, cudaStream_t s) {
  release_kernel<<<blocks_for((long long)a.batch * a.L.max_pages_per_seq), THREADS, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq

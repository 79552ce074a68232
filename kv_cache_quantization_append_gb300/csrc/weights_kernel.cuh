// Attention weights of cached positions: the kernels of one key format (included by one translation unit per format).
//
// For the rows of a unit (query heads of its newest n tokens, row = token * g + head; at most 128 a launch) every
// position's logit is wanted twice: for the rows' normalisers, and for the positions' weights, the sum over rows of
// 2^(logit - normaliser):
//  1. weights_kernel<.., SUM = false>: per row the maximum and sum over this CTA's range of tiles (stream-K, as in tree
//     attention: 8 or 16 warps convert keys and finish logits, one more copies records and issues products;
//     the next tile's keys are converted while a tile's first products run, the next block's products run while a
//     block's logits are finished).
//     With at most 8 rows it also stores the logits: 4 bytes a row and position against at least 68 of key record.
//  2. With stored logits weights_add_kernel, an elementwise pass that joins the ranges' maxima and sums in a fixed order
//     first; else normaliser_kernel, which joins them once per row, and weights_kernel<.., SUM = true>, which takes the
//     logits again.
//
// The weights accumulate in fp32, so logits are taken to fp32's accuracy: the keys' codes go to the tensor cores as they
// are, exact in fp16 (S^T = codes [128 positions x 128] Q~^T, the queries as fp16 hi and lo), one accumulator per group of
// 32 channels (TQ3: centroids and signs), and the thread that owns the position applies its scales and zeros in fp32:
//   logit = sum_G scale_G S_G + zero_G (sum of q~ over G);  TQ3: n (S_c + w S_sign).
// Raw keys (the window) are fp16 hi and lo against the queries as they are: hi hi in all accumulators but one, hi lo + lo hi
// in that.
// Each warp keeps its own reference per row, which moves only when a logit passes it by 2^60: no exchange between warps
// until the range ends.
//
// Measured (a call): 4 rows of each of 8 KV heads over 8 sequences of up to 16K Q4 49 us (1.5 TB/s, 9 of them the adding
// pass), bound by the workers' chain per tile -- code conversion, barrier, product, barrier, 4 rows of logits; 96 rows over
// 32K Q8 93 us, two passes of about 42, of which 8 us each are the queries' preparation and code seen for the first time.
// Before the issuing warp's values were taken from one lane (111 us) leaving out half of the products, three quarters of the
// accumulators' reads and the sums over lanes together saved 12 %: what bounds it is not one pipe but the sequence of short
// steps between barriers.
#pragma once

#include "records.cuh"

namespace kvq {
namespace weights {

using namespace tc;
using namespace records;

constexpr float NO_REF = -1e30f;
constexpr int STORE_ROWS = 8;
constexpr int MAX_ROWS = 128;   // of a launch
// Rows of TQ3 keys whose queries (1 KB a row with their projections) leave room for two CTAs an SM.  More take one CTA an
// SM with four threads to a position (96 rows over 32K: 125 us, with two threads 203); the other formats have room for two
// at 128 rows, and one with four threads was no faster (96 rows over 32K Q8: 113 us against 111).
constexpr int NARROW_ROWS = 64;
constexpr int ADD_THREADS = 256;
// Places in the list of tiles: a raw tile counts as four of records (it comes with queries of its own), and belongs to the
// range that holds its first place.  Measured with 2 to 6 places: 16 queries over 4 x 1000 Q4 35, 36, 38, 49, 54 us; a step over
// 8 x 16K 51, 50, 49, 49, 50; 32 queries at 32K Q8 101, 95, 92, 91, 90; five other sizes the same within 8 %.
constexpr int RAW_PLACES = 4;

struct Plan {
  MultiArgs a;
  int row0, rows;     // this launch's rows of every unit
  int P, nb;          // threads to a position, blocks of N = 8 P rows
  int n_units, G;
  long long s_pad;    // positions a row of stored logits has room for
  float decay;
  // [2 n_units + G][rows][2]: range c's maxima and sums of unit u's records (+ 0), raw keys (+ 1) at 2 u + c
  float* parts;     
  float* logits;      // [n_units][rows][s_pad], or null
  float* norms;       // [n_units][rows] normalisers, where logits are taken again
};

__host__ __device__ inline int quant_tiles(int L, int W) { return (L > W ? L - W + TILE - 1 : 0) / TILE; }
__device__ __forceinline__ int seq_tiles(int L, int W) {
  return quant_tiles(L, W) + ((L < W ? L : W) + TILE - 1) / TILE * RAW_PLACES;
}

template <int KF>
struct Cfg {
  static constexpr bool TQ = KF == KVQ_TQ3_QJL;
  static constexpr int KD = TQ ? 256 : 128;   // width of a query
  static constexpr int ACC = TQ ? 2 : 4;      // accumulators: centroids and signs, or groups of 32 channels
  static constexpr int K_COLS = KD / 2;       // tensor-memory columns of a tile's keys
  static constexpr int STAGES = KF == KVQ_Q8G32 ? 2 : 3;  // tiles of records in shared memory
};
// place of channel c among the keys' K elements: groups of 32 channels stay together
template <int KF>
__host__ __device__ constexpr int place(int c) {
  if (KF == KVQ_Q4G32) return (c & ~7) + nibble_place(c & 7);
  if (KF == KVQ_TQ3_QJL) return c;
  // Q8 record chunk 2 i + h, word w, byte: channel 16 (4 h + w) + 2 i + (byte & 1) + 8 (byte >> 1)
  const int w = (c >> 4) & 3, h = c >> 6, i = (c & 7) >> 1, byte = (c & 1) + 2 * ((c >> 3) & 1);
  return 8 * (8 * h + 4 * (w >> 1) + i) + 4 * (w & 1) + byte;
}

template <int KF>
struct Smem {
  using C = Cfg<KF>;
  static __host__ __device__ constexpr uint32_t plane(int rows) { return rows * C::KD * 2; }  // of nb * N rows
  static __host__ __device__ constexpr uint32_t rec(int rows) { return 2 * plane(rows); }
  static constexpr uint32_t REC = 4 * Rec<KF>::KH;
  // (TQ3: a plane of the projection first takes the records' place)
  // [4 P warps][rows / P]
  static __host__ __device__ constexpr uint32_t wm(int rows) { return rec(rows) + (C::TQ ? 32768 : C::STAGES * REC); }
  static __host__ __device__ constexpr uint32_t wl(int rows) { return wm(rows) + 16 * rows; }
  static __host__ __device__ constexpr uint32_t qs(int rows) { return wl(rows) + 16 * rows; }              // [rows][4]
  static __host__ __device__ constexpr uint32_t pre(int rows) { return qs(rows) + 16 * rows; }
};

// the codes of the thread's position, exact, to its tensor-memory lane (TQ3: centroids, then signs as +-1)
template <int KF, int P>
__device__ __forceinline__ void put_codes(uint32_t col, const Lane& ln, const uint8_t* rec, const uint4& cent) {
  using R = Rec<KF>;
  const uint8_t* hb = rec + (ln.t >> 5) * R::KH;
  const int tt = ln.t & 31;
  if (KF == KVQ_Q8G32) {
    const __half2 off = u2h(0x64806480u);  // 1024 + 128
#pragma unroll
    for (int c = 0; c < 8 / P; ++c) {
      const int m = 8 / P * ln.hf + c;  // chunk 2 i + h
      const uint4 q = *reinterpret_cast<const uint4*>(hb + tt * 128 + 16 * (m ^ (tt & 1)));
      const uint32_t wd[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = h2u(__hsub2(u2h(prmt(wd[2 * half + (i >> 1)], 0x64646464u, i & 1 ? 0x4342 : 0x4140)), off));
        tm_st4(col + 4 * (8 * (m & 1) + 4 * half + (m >> 1)), make_uint4(o[0], o[1], o[2], o[3]));
      }
    }
    return;
  }
  constexpr int CHUNKS = 4 / P;  // 16-byte chunks of the record
  uint4 k[CHUNKS];
  if constexpr (CHUNKS == 2) lds32(hb + tt * 64 + 32 * ln.hf, tt & 2, k[0], k[1]);
  else k[0] = *reinterpret_cast<const uint4*>(hb + tt * 64 + 16 * ln.hf);
  if (KF == KVQ_Q4G32) {
#pragma unroll
    for (int G = 0; G < 4; ++G) {
      uint4 o[CHUNKS];
#pragma unroll
      for (int i = 0; i < CHUNKS; ++i) {
        __half2 c[4];
        nibbles(G == 0 ? k[i].x : G == 1 ? k[i].y : G == 2 ? k[i].z : k[i].w, c);
        o[i] = make_uint4(h2u(c[0]), h2u(c[1]), h2u(c[2]), h2u(c[3]));
      }
      if constexpr (CHUNKS == 2) tm_st8(col + 16 * G + 8 * ln.hf, o[0], o[1]);
      else tm_st4(col + 16 * G + 4 * ln.hf, o[0]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4 * CHUNKS; i += 2) {
    uint4 o[2], s[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint4& q = k[i >> 2];
      const uint32_t word = ((i + x) & 3) == 0 ? q.x : ((i + x) & 3) == 1 ? q.y : ((i + x) & 3) == 2 ? q.z : q.w;
      const uint32_t sel = (word & 0x07070707u) | ((word << 1) & 0x70707070u);
      const uint32_t l0 = prmt(cent.x, cent.y, sel), h0 = prmt(cent.z, cent.w, sel);
      const uint32_t l1 = prmt(cent.x, cent.y, sel >> 16), h1 = prmt(cent.z, cent.w, sel >> 16);
      o[x] = make_uint4(__byte_perm(l0, h0, 0x5140), __byte_perm(l0, h0, 0x7362), __byte_perm(l1, h1, 0x5140),
                        __byte_perm(l1, h1, 0x7362));
      const uint32_t lo = word << 1;
      uint32_t m[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        m[j] = 0xBC00BC00u ^ (prmt(lo, word, (uint32_t)((8 + j) << 4) | (uint32_t)((12 + j) << 12)) & 0x80008000u);
      s[x] = make_uint4(m[0], m[1], m[2], m[3]);
    }
    tm_st8(col + 16 * CHUNKS * ln.hf + 4 * i, o[0], o[1]);
    tm_st8(col + 64 + 16 * CHUNKS * ln.hf + 4 * i, s[0], s[1]);
  }
}

// normaliser (base-2 logarithm of the sum) of one row of unit u by a warp: the parts of every range in a fixed order; NaN
// where one of them gave up
__device__ __forceinline__ float normaliser(const Plan& p, int u, int row, long long first, int nq, int tiles, long long G,
                                            long long total, int lane) {
  const auto owner = [&](long long x) { return (int)quick_div((x + 1) * G - 1, total); };
  const int c0 = owner(first), c1 = nq > 0 ? owner(first + nq - 1) : c0 - 1;
  float m = NO_REF, l = 0.f;
  bool lost = false;
  const auto add = [&](int kind, int c) {
    const float2 x = *reinterpret_cast<const float2*>(p.parts + ((size_t)(2 * u + kind + c) * p.rows + row) * 2);
    lost = lost || x.x != x.x;
    const float mn = fmaxf(m, x.x);
    l = l * ex2(m - mn) + x.y * ex2(x.x - mn);
    m = mn;
  };
  for (int c = c0 + lane; c <= c1; c += 32) add(0, c);
  if (lane == 31) {
    int last = -1;
    for (int x = nq; x < tiles; x += RAW_PLACES) {
      const int c = owner(first + x);
      if (c != last) add(1, c);
      last = c;
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float m2 = __shfl_xor_sync(FULL, m, o), l2 = __shfl_xor_sync(FULL, l, o), mn = fmaxf(m, m2);
    // (the lower lane's term first, on both sides)
    const float a = l * ex2(m - mn), b = l2 * ex2(m2 - mn);
    l = lane & o ? b + a : a + b;
    m = mn;
  }
  if (__any_sync(FULL, lost)) return NAN;
  return l > 0.f ? m + log2f(l) : INFINITY;
}

// CH: a thread's rows of a block at a time: 8, or 2 where there are no more than 4 (they then keep their sums in registers)
template <int KF, bool SUM, int CH, int P>
__global__ void __launch_bounds__(128 * P + 32, 4 / P) weights_kernel(const __grid_constant__ Plan p) {
  using C = Cfg<KF>;
  using SM = Smem<KF>;
  constexpr bool TQ = C::TQ, Q4 = KF == KVQ_Q4G32;
  constexpr int WORKERS = 128 * P, WARPS = WORKERS / 32;  // and the warp that issues the products
  // rows of a block: the accumulators of two blocks fit beside the keys
  constexpr int N = 8 * P;                              
  constexpr int ACC = C::ACC;
  constexpr bool FEW = CH == 2;
  // tensor memory: K (128 columns: two tiles' codes; raw keys' hi and lo; TQ3 centroids and signs) | S, two buffers of ACC
  // accumulators of N columns
  constexpr uint32_t C_S = 128, TM_COLS = C_S + 2 * ACC * N <= 256 ? 256 : 512;
  static_assert(C_S + 2 * ACC * N <= TM_COLS && TM_COLS * (4 / P) <= 512, "tensor memory");
  static_assert(!TQ || C::STAGES * SM::REC <= 32768, "the records lie in the projection's place");
  constexpr uint32_t ID_S = idesc(TILE, N, false, false);
  extern __shared__ __align__(1024) uint8_t smem[];
  // kr_bar: a tile's keys have landed; k_bar: they are in place (one arrival a worker warp; two barriers by turns, as the
  // workers place a second tile's before the ninth warp has to have seen the first's); s_bar: a block's logits have been
  // read; qk_bar: a block's products are done
  __shared__ __align__(8) uint64_t kr_bar[C::STAGES], k_bar[2], s_bar[2], qk_bar[2], proj_bar, end_bar;
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh;
  __shared__ float part_sum[2][P - 1][TILE];  // of the groups of columns after the first, by turns of the tiles
  const MultiArgs& a = p.a;
  const int tid = threadIdx.x, warp = __shfl_sync(FULL, tid >> 5, 0), lane = tid & 31, NR = p.nb * N;
  const uint32_t q_plane = SM::plane(NR);
  float* qs = reinterpret_cast<float*>(smem + SM::qs(NR));
  int* pre = reinterpret_cast<int*>(smem + SM::pre(NR));
  int* lens = pre + a.batch + 1;

  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) bar_init(&kr_bar[i], 1);
    for (int i = 0; i < 2; ++i) {
      bar_init(&k_bar[i], WARPS);
      bar_init(&s_bar[i], WARPS);
      bar_init(&qk_bar[i], 1);
    }
    bar_init(&proj_bar, 1);
    bar_init(&end_bar, 1);
    abort_sh = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) tile_prefix(a, lens, pre, blockIdx.x == 0, [&](int L) { return seq_tiles(L, a.W); });
  if (warp == 1) tm_alloc(&tmem_sh, TM_COLS);
  fence_before();
  asm volatile("griddepcontrol.launch_dependents;");
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(FULL, tmem_sh, 0), sbase = smem_u32(smem);
  const long long per_layer = (long long)pre[a.batch] * a.Hkv, total = per_layer * a.n_layers_call;
  const long long G = min((long long)p.G, total);
  long long t = blockIdx.x < G ? quick_div(total * blockIdx.x, G) : 0;
  const long long t_end = blockIdx.x < G ? quick_div(total * (blockIdx.x + 1), G) : 0;

  const Lane ln = lane_of<P>(tid);
  const size_t page_stride = (size_t)a.Hkv * a.L.page_bytes;
  const float4 sg = *reinterpret_cast<const float4*>(a.p.signs + 4 * lane);
  uint4 cent = make_uint4(0u, 0u, 0u, 0u);
  if (TQ) {
    const uint4 c = *reinterpret_cast<const uint4*>(a.p.cb->cent);
    cent = make_uint4(__byte_perm(c.x, c.y, 0x6420), __byte_perm(c.z, c.w, 0x6420), __byte_perm(c.x, c.y, 0x7531),
                      __byte_perm(c.z, c.w, 0x7531));
  }
  uint32_t k_n = 0, kr_n = 0, proj_n = 0, job = 0;  // tiles of keys, copies, projections and blocks so far: their phases
  const auto wait_nth = [&](uint64_t* bar, uint32_t n) { bar_wait(bar, n & 1, &abort_sh, a.p.status, a.wait_ns); };
  const auto k_done = [&] {
    tm_wait_st();
    fence_before();
    __syncwarp();
    if (lane == 0) bar_arrive(&k_bar[k_n & 1]);
    ++k_n;
  };
  const auto k_wait = [&] {
    wait_nth(&k_bar[k_n & 1], k_n >> 1);
    ++k_n;
  };
  const int col0 = (warp >> 2) * (FEW ? 2 : N / P);
  const uint32_t lane_addr = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
  float* wm = reinterpret_cast<float*>(smem + SM::wm(NR)) + warp * (NR / P);  // this warp's references and sums
  float* wl = reinterpret_cast<float*>(smem + SM::wl(NR)) + warp * (NR / P);
  float* lse = reinterpret_cast<float*>(smem + SM::wm(NR));                   // SUM: the rows' normalisers
  bool ok = true;

  // the part that begins at place t: its unit (sequence and head) and this CTA's tiles of it; t goes on behind it
  struct Part {
    int ll, b, h, u, it0, it1, nq;
    bool raw;
  };
  const auto part_at = [&](long long& t) {
    Part w;
    w.ll = a.n_layers_call > 1 ? (int)quick_div(t, per_layer) : 0;
    const long long in_layer = t - w.ll * per_layer;
    int lo = 0, hi = a.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((long long)pre[mid] * a.Hkv <= in_layer) lo = mid;
      else hi = mid - 1;
    }
    w.b = lo;
    const int tiles = pre[lo + 1] - pre[lo];
    const long long r = in_layer - (long long)pre[lo] * a.Hkv;
    w.h = (int)quick_div(r, tiles);
    const int place0 = (int)(r - (long long)w.h * tiles);
    w.u = (w.ll * a.batch + lo) * a.Hkv + w.h;
    w.nq = quant_tiles(lens[lo], a.W);
    w.raw = place0 >= w.nq;
    const int place1 = (int)min((long long)(w.raw ? tiles : w.nq), place0 + (t_end - t));
    t += place1 - place0;
    w.it0 = w.raw ? w.nq + (place0 - w.nq + RAW_PLACES - 1) / RAW_PLACES : place0;
    w.it1 = w.raw ? w.nq + (place1 - w.nq + RAW_PLACES - 1) / RAW_PLACES : place1;
    return w;
  };
  const auto part_sums = [&](const Part& w) { return p.parts + (size_t)(2 * w.u + w.raw + blockIdx.x) * p.rows * 2; };
  const auto gave_up = [&] { return *(volatile int*)&abort_sh != 0; };
  long long t_part = t;

  while (t < t_end && ok) {
    t_part = t;
    const Part w = part_at(t);
    const int ll = w.ll, b = w.b, h = w.h, layer = a.layer0 + ll, u = w.u, nq = w.nq, it0 = w.it0, it1 = w.it1;
    const int L = lens[b], qend = max(0, L - a.W);
    const bool raw = w.raw;
    if (it0 == it1) continue;
    const int* bt = a.block_table + (size_t)b * a.max_pages_per_seq;

    if (warp == WARPS) {
      // (taken from one lane, as the warp's number and the tensor memory's address: its lanes branch together by construction,
      // and the products' operands are computed once for the warp)
      const int it0 = __shfl_sync(FULL, w.it0, 0), it1 = __shfl_sync(FULL, w.it1, 0);
      const bool raw = __shfl_sync(FULL, (int)w.raw, 0) != 0;
      // ================================================================ the products and the copies
      const uint8_t* unit_pages = a.p.pages + ((size_t)layer * a.L.n_pages * a.Hkv + h) * (size_t)a.L.page_bytes;
      using R = Rec<KF>;
      const auto page_of = [&](int it) {
        const int j = it * TILE + lane * HALF;
        return lane < 4 && it < it1 && j < qend ? __ldg(bt + j / PAGE) : -1;
      };
      const auto copy = [&](int entry) {  // (checked here, not where it is read: nothing waits for it there)
        const int phys = checked(entry, a.L.n_pages), stage = kr_n % C::STAGES;
        ++kr_n;
        const int n = __popc(__ballot_sync(FULL, phys >= 0));
        if (lane == 0) bar_expect(&kr_bar[stage], n * R::KH);
        __syncwarp();
        if (phys >= 0) {
          const uint8_t* src = unit_pages + (size_t)phys * page_stride + (lane & 1) * (size_t)(R::KH + R::VH);
          uint8_t* dst = smem + SM::rec(NR) + stage * SM::REC + lane * R::KH;
          bulk_g2s(dst, src, R::K_MAIN, &kr_bar[stage]);
          bulk_g2s(dst + R::K_MAIN, src + R::K_MAIN + R::V_MAIN, R::K_META, &kr_bar[stage]);
        }
        __syncwarp();
      };
      if (TQ && !raw) {
        // S q~ of all rows to columns 0 .. NR - 1: the projection comes as its hi plane, then its lo plane
        for (int part = 0; part < 2; ++part) {
          k_wait();
          fence_after();
#pragma unroll 1
          for (int rb = 0; rb < p.nb; ++rb) {
            uint64_t sa = sdesc(sbase + SM::rec(NR), 2048, 128), qa = sdesc(sbase + rb * N * C::KD * 2, N * 16, 128);
#pragma unroll 1
            for (int ks = 0; ks < D / 16; ++ks, sa += 256, qa += 2 * N) {
              mma_ss(tmem + rb * N, sa, qa, ID_S, part > 0 || ks > 0);
              if (part == 0) mma_ss(tmem + rb * N, sa, qa + (q_plane >> 4), ID_S, 1);
            }
          }
          mma_commit(&proj_bar);
        }
        wait_nth(&proj_bar, proj_n + 1);  // (the records come to the projection's place)
        proj_n += 2;
      }
      int phys = -1;  // this lane's page of the tile to be copied next, read before it is needed
      if (!raw) {
        int first[C::STAGES];
#pragma unroll
        for (int i = 0; i < C::STAGES; ++i) first[i] = page_of(it0 + i);
        phys = page_of(it0 + C::STAGES);
#pragma unroll
        for (int i = 0; i < C::STAGES; ++i)
          if (it0 + i < it1) copy(first[i]);
      } else {
        // raw keys go through registers a few at a time: the part's are brought to L2 while its queries are prepared
        const int j1 = min(L, qend + (it1 - nq) * TILE);
        const size_t ring = (((size_t)layer * a.max_batch + b) * a.Hkv + h) * a.W;
        for (int j = qend + (it0 - nq) * TILE + lane; j < j1; j += 32) prefetch(a.p.ringk + (ring + (unsigned)j % (unsigned)a.W) * D, D * 4);
      }
      for (int it = it0; it < it1; ++it) {
        k_wait();
        if (__any_sync(FULL, gave_up())) break;  // (the whole warp)
        if (!raw && it + C::STAGES < it1) {  // the workers have read this tile's keys
          copy(phys);
          phys = page_of(it + C::STAGES + 1);
        }
        for (int rb = 0; rb < p.nb; ++rb, ++job) {
          const int sb = job & 1;
          if (job >= 2) wait_nth(&s_bar[sb], (job - 2) >> 1);
          if (__any_sync(FULL, gave_up())) break;
          fence_after();
          uint64_t qa = sdesc(sbase + rb * N * C::KD * 2, N * 16, 128);
          const uint64_t qb = q_plane >> 4;
          uint32_t ka = tmem + (!TQ && !raw ? ((it - it0) & 1) * C::K_COLS : 0);
          const uint32_t d = tmem + C_S + sb * (ACC * N);
          if (raw) {
            // the tensor cores cut off each sum's low bits: hi hi over all accumulators but the last, which has the small
            // rest
            constexpr int LAST = (ACC - 1) * N;
#pragma unroll 1
            for (int ks = 0, i = -1; ks < D / 16; ++ks, ka += 8, qa += 2 * N) {
              const int to = ks * (ACC - 1) / (D / 16);
              mma_ts(d + to * N, ka, qa, ID_S, to == i);
              mma_ts(d + LAST, ka, qa + qb, ID_S, ks > 0);
              mma_ts(d + LAST, ka + 64, qa, ID_S, 1);
              i = to;
            }
          } else {
            constexpr int STEPS = C::KD / 16 / ACC;  // k-steps per accumulator
#pragma unroll 2
            for (int ks = 0; ks < C::KD / 16; ++ks, ka += 8, qa += 2 * N) {
              mma_ts(d + ks / STEPS * N, ka, qa, ID_S, ks % STEPS > 0);
              mma_ts(d + ks / STEPS * N, ka, qa + qb, ID_S, 1);
            }
          }
          mma_commit(&qk_bar[sb]);
        }
      }
      ok = !__any_sync(FULL, gave_up());
      continue;
    }

    // ================================================================ the workers
    const auto page_of = [&](int it) {  // of this thread's position, read a tile ahead
      const int j = it * TILE + (ln.t & 64);
      return it < it1 && !raw && j < qend ? __ldg(bt + j / PAGE) : -1;
    };
    int page = page_of(it0);
    // ---- queries in base-2 units as hi and lo images, for records rotated and balanced; sums over groups for the zeros
    float f[4];  // of this lane's channels
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = raw ? LOGIT_SCALE : C_WHT * LOGIT_SCALE;
      if (a.sinkhorn && !raw) f[e] *= __half2float(a.p.sigk[((size_t)layer * a.Hkv + h) * D + 4 * lane + e]);
    }
    const auto query = [&](int lr) {
      const int row = p.row0 + lr;
      return lr < p.rows ? load4_in(a.q, ((((size_t)ll * a.batch + b) * a.Hkv * a.g + (size_t)h * a.g + row % a.g) * a.n + row / a.g) * D + 4 * lane,
                                    a.in_bf16)
                         : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    float4 next[2] = {query(warp), query(warp + WARPS)};
#pragma unroll 1
    for (int r0 = warp; r0 < NR; r0 += 2 * WARPS) {  // two rows at a time, the next two under way
      float y[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        y[i][0] = next[i].x, y[i][1] = next[i].y, y[i][2] = next[i].z, y[i][3] = next[i].w;
        next[i] = query(r0 + (2 + i) * WARPS);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int lr = r0 + i * WARPS;  // (NR is a multiple of 2 WARPS: both rows are there)
        if (!raw) {
          y[i][0] *= sg.x, y[i][1] *= sg.y, y[i][2] *= sg.z, y[i][3] *= sg.w;
          hadamard_warp(y[i][0], y[i][1], y[i][2], y[i][3], lane);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) y[i][e] *= f[e];
        uint8_t* img = smem + (lr / N) * (N * C::KD * 2);
        if (KF == KVQ_Q8G32) {
#pragma unroll
          for (int e = 0; e < 4; e += 2) {  // channels c and c + 1 are neighbours
            uint32_t hi2, lo2;
            split2(y[i][e], y[i][e + 1], hi2, lo2);
            uint8_t* dst = img + km_off(lr % N, place<KF>(4 * lane + e), N);
            *reinterpret_cast<uint32_t*>(dst) = hi2;
            *reinterpret_cast<uint32_t*>(dst + q_plane) = lo2;
          }
        } else {
          put4<Q4>(img + km_off(lr % N, 4 * lane & ~7, N) + 8 * (lane & 1), q_plane, y[i], lane);
        }
        if (Q4) {
          float s = (y[i][0] + y[i][1]) + (y[i][2] + y[i][3]);
          s += __shfl_xor_sync(FULL, s, 1);
          s += __shfl_xor_sync(FULL, s, 2);
          s += __shfl_xor_sync(FULL, s, 4);
          if ((lane & 7) == 0) qs[4 * lr + (lane >> 3)] = raw ? 0.f : s;
        }
      }
    }
    if (SUM) {
      asm volatile("griddepcontrol.wait;" ::: "memory");  // the normalisers (what came before does not need them)
      for (int lr = tid; lr < NR; lr += WORKERS) lse[lr] = lr < p.rows ? p.norms[(size_t)u * p.rows + lr] : INFINITY;
    } else {
      for (int c = lane; c < NR / P; c += 32) {
        wm[c] = NO_REF;
        wl[c] = 0.f;
      }
    }
    if (TQ && !raw) {
      const int i = tid & 127;
#pragma unroll 1
      for (int part = 0; part < 2; ++part) {
        if (part) wait_nth(&proj_bar, proj_n);
#pragma unroll 1
        for (int kg = tid >> 7; kg < D / 8; kg += P) {
          float s[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) s[e] = __ldg(a.p.qjl_t + (8 * kg + e) * D + i);
          uint4 o, l;
          split2(s[0], s[1], o.x, l.x);
          split2(s[2], s[3], o.y, l.y);
          split2(s[4], s[5], o.z, l.z);
          split2(s[6], s[7], o.w, l.w);
          *reinterpret_cast<uint4*>(smem + SM::rec(NR) + km_off(i, 8 * kg, D)) = part ? l : o;
        }
        fence_async_smem();
        k_done();
      }
      wait_nth(&proj_bar, proj_n + 1);
      proj_n += 2;
      fence_after();
#pragma unroll 1
      for (int c = (warp >> 2) * (NR / P); c < ((warp >> 2) + 1) * (NR / P); c += 8) {
        float x[8];
        tm_ld(lane_addr + c, x);
        tm_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          uint8_t* dst = smem + ((c + e) / N) * (N * C::KD * 2) + km_off((c + e) % N, D + i, N);
          const __half hi16 = __float2half_rn(x[e]);
          *reinterpret_cast<__half*>(dst) = hi16;
          *reinterpret_cast<__half*>(dst + q_plane) = __float2half_rn(x[e] - __half2float(hi16));
        }
      }
      fence_before();
    }
    fence_async_smem();
    part_sync(1, WORKERS);

    // keys of tile `it` to tensor memory; scales and zeros (TQ3: norm, weight) of this thread's position as they are
    uint4 meta = make_uint4(0u, 0u, 0u, 0u);
    bool bad = false;
    const auto put = [&](int it) {
      const int j = (raw ? qend - nq * TILE : 0) + it * TILE + ln.t;
      if (!raw) {
        bad = checked(page, a.L.n_pages) < 0;
        if (bad && j < qend && (tid & 63) == 0) atomicOr(a.p.status, KVQ_DEV_BAD_PAGE);
        page = page_of(it + 1);
        const int stage = kr_n % C::STAGES;
        wait_nth(&kr_bar[stage], kr_n / C::STAGES);
        ++kr_n;
        const uint8_t* rec = smem + SM::rec(NR) + stage * SM::REC;
        put_codes<KF, P>(lane_addr + (TQ ? 0 : ((it - it0) & 1) * C::K_COLS), ln, rec, cent);
        const uint8_t* m = rec + (ln.t >> 5) * Rec<KF>::KH + Rec<KF>::K_MAIN;
        const int tt = ln.t & 31;
        if (TQ) {
          meta.x = reinterpret_cast<const unsigned short*>(m)[tt];
          meta.y = reinterpret_cast<const unsigned short*>(m)[HALF + tt];
        } else if (Q4) {
          meta = *reinterpret_cast<const uint4*>(m + 16 * tt);
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(m + 8 * tt);
          meta.x = v.x, meta.y = v.y;
        }
      } else {
        const float* row = a.p.ringk + ((((size_t)layer * a.max_batch + b) * a.Hkv + h) * a.W + (j < L ? (unsigned)j % (unsigned)a.W : 0u)) * D;
#pragma unroll 4
        for (int i = 0; i < 16 / P; ++i) {
          const int kg = 16 / P * ln.hf + i;
          float f[8];
          if (KF == KVQ_Q8G32) {
            const int c = 64 * (kg >> 3) + 32 * ((kg >> 2) & 1) + 2 * (kg & 3);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const float2 v = *reinterpret_cast<const float2*>(row + c + 8 * y);
              f[2 * y] = v.x, f[2 * y + 1] = v.y;
            }
          } else {
            const float4 v0 = *reinterpret_cast<const float4*>(row + 8 * kg), v1 = *reinterpret_cast<const float4*>(row + 8 * kg + 4);
            const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
            for (int y = 0; y < 8; ++y) f[y] = v[Q4 ? nibble_channel(y) : y];
          }
          uint4 o, l;
          split2(f[0], f[1], o.x, l.x);
          split2(f[2], f[3], o.y, l.y);
          split2(f[4], f[5], o.z, l.z);
          split2(f[6], f[7], o.w, l.w);
          tm_st4(lane_addr + 4 * kg, o);
          tm_st4(lane_addr + 64 + 4 * kg, l);
        }
      }
      k_done();
    };
    // FEW: the warp's references, the thread's sums, its rows' sums for the zeros
    float rm[2] = {NO_REF, NO_REF}, rl[2] = {};
    float4 few_qs[2] = {};
    if (FEW && Q4) {
      few_qs[0] = *reinterpret_cast<const float4*>(qs + 4 * col0);
      few_qs[1] = *reinterpret_cast<const float4*>(qs + 4 * col0 + 4);
    }
    float* const logits = p.logits ? p.logits + (size_t)u * p.rows * p.s_pad : nullptr;  // of this unit
    put(it0);
    for (int it = it0; it < it1; ++it) {
      const int j = (raw ? qend - nq * TILE : 0) + it * TILE + ln.t;  // this thread's position
      const bool mine = j < (raw ? L : qend), valid = mine && !bad;   // (a page out of range takes no weight)
      float s0[4] = {}, z0[4] = {};
      if (TQ) {
        s0[0] = __half2float(__ushort_as_half((unsigned short)meta.x));
        s0[1] = s0[0] * QJL_CONST * __half2float(__ushort_as_half((unsigned short)meta.y));
      } else {
        const float2 a0 = __half22float2(u2h(meta.x)), a1 = __half22float2(u2h(meta.y));
        s0[0] = a0.x, s0[1] = a0.y, s0[2] = a1.x, s0[3] = a1.y;
        if (Q4) {
          const float2 b0 = __half22float2(u2h(meta.z)), b1 = __half22float2(u2h(meta.w));
          z0[0] = b0.x, z0[1] = b0.y, z0[2] = b1.x, z0[3] = b1.y;
        }
      }
      // the next tile's keys, while this one's products run (TQ3's and raw ones have no second place)
      if (!TQ && !raw && it + 1 < it1) put(it + 1);
      // rows from this one on attend to the position (token of the row >= j - L + n)
      const int cut = valid ? a.g * max(0, j - L + a.n) - p.row0 : 1 << 30;
      const bool some_cut = __any_sync(FULL, cut > 0);
      float acc = 0.f;
#pragma unroll 1
      for (int rb = 0; rb < p.nb; ++rb, ++job) {
        const int sb = job & 1;
        const uint32_t s_addr = lane_addr + C_S + sb * (ACC * N);
        wait_nth(&qk_bar[sb], job >> 1);
        fence_after();
#pragma unroll 1
        for (int c = col0; c < col0 + (FEW ? CH : N / P) && rb * N + c < p.rows; c += CH) {
          const int row = rb * N + c;
          // ---- CH rows' logits
          float s[CH], part[ACC][CH];
#pragma unroll
          for (int i = 0; i < ACC; ++i) tm_ld(s_addr + i * N + c, part[i]);
          tm_wait_ld();
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            if (raw) {
              s[i] = part[0][i];
#pragma unroll
              for (int y = 1; y < ACC; ++y) s[i] += part[y][i];
            } else if (TQ) {
              s[i] = fmaf(part[1][i], s0[1], part[0][i] * s0[0]);
            } else {
              s[i] = part[0][i] * s0[0];
#pragma unroll
              for (int y = 1; y < ACC; ++y) s[i] = fmaf(part[y % ACC][i], s0[y], s[i]);
              if (Q4) {
                const float4 q = FEW ? few_qs[i & 1] : *reinterpret_cast<const float4*>(qs + 4 * (row + i));
                s[i] = fmaf(q.x, z0[0], fmaf(q.y, z0[1], fmaf(q.z, z0[2], fmaf(q.w, z0[3], s[i]))));
              }
            }
          }
          if (some_cut) {
#pragma unroll
            for (int i = 0; i < CH; ++i)
              if (row + i < cut) s[i] = -INFINITY;
          }
          if constexpr (SUM) {
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < CH; i += 4) {
              const float4 m = *reinterpret_cast<const float4*>(lse + row + i);
              sum[0] += ex2(s[i] - m.x) + ex2(s[i + 1] - m.y);
              sum[1] += ex2(s[i + 2] - m.z) + ex2(s[i + 3] - m.w);
            }
            acc += sum[0] + sum[1];
            continue;
          }
          if (logits != nullptr && mine) {
            float* at = logits + row * p.s_pad + j;
#pragma unroll
            for (int i = 0; i < CH; ++i, at += p.s_pad)
              if (row + i < p.rows) *at = s[i];
          }
          const int at = rb * (N / P) + c - col0;
          float m[CH];
          if constexpr (FEW) {
#pragma unroll
            for (int i = 0; i < CH; ++i) m[i] = rm[i];
          } else {
#pragma unroll
            for (int i = 0; i < CH; i += 4) {
              const float4 v = *reinterpret_cast<const float4*>(wm + at + i);
              m[i] = v.x, m[i + 1] = v.y, m[i + 2] = v.z, m[i + 3] = v.w;
            }
          }
          float e[CH], top = -INFINITY;
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            e[i] = s[i] - m[i];
            top = fmaxf(top, e[i]);
          }
          if (__any_sync(FULL, top > 60.f)) {  // (the first tile, hardly ever another)
#pragma unroll
            for (int i = 0; i < CH; ++i) {
              const int v = __float_as_int(s[i]);
              const int most = __reduce_max_sync(FULL, v ^ ((v >> 31) & 0x7fffffff));
              const float ft = __int_as_float(most ^ ((most >> 31) & 0x7fffffff));
              if (ft > m[i] + 60.f) {
                if constexpr (FEW) rl[i] *= ex2(m[i] - ft);
                else if (lane == 0) wl[at + i] *= ex2(m[i] - ft);
                m[i] = ft;
              }
              e[i] = s[i] - m[i];
            }
            if constexpr (FEW) {
#pragma unroll
              for (int i = 0; i < CH; ++i) rm[i] = m[i];
            } else {
              __syncwarp();
              if (lane == 0) {
#pragma unroll
                for (int i = 0; i < CH; ++i) wm[at + i] = m[i];
              }
              __syncwarp();
            }
          }
#pragma unroll
          for (int i = 0; i < CH; ++i) e[i] = ex2(e[i]);
          if constexpr (FEW) {
#pragma unroll
            for (int i = 0; i < CH; ++i) rl[i] += e[i];
          } else {
            // sums over the lanes, halving the rows a lane holds: row lane >> 2 ends in the lanes
            const bool u16 = lane & 16, u8 = lane & 8, u4 = lane & 4;
            float f[4], g[2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              f[i] = u16 ? e[4 + i] : e[i];
              f[i] += __shfl_xor_sync(FULL, u16 ? e[i] : e[4 + i], 16);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              g[i] = u8 ? f[2 + i] : f[i];
              g[i] += __shfl_xor_sync(FULL, u8 ? f[i] : f[2 + i], 8);
            }
            float v = u4 ? g[1] : g[0];
            v += __shfl_xor_sync(FULL, u4 ? g[0] : g[1], 4);
            v += __shfl_xor_sync(FULL, v, 2);
            v += __shfl_xor_sync(FULL, v, 1);
            if ((lane & 3) == 0) wl[at + (lane >> 2)] += v;
            __syncwarp();
          }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&s_bar[sb]);
      }
      if ((TQ || raw) && it + 1 < it1) put(it + 1);
      if (SUM) {
        float(*sums)[TILE] = part_sum[(it - it0) & 1];
        if (warp >= 4) sums[(warp >> 2) - 1][ln.t] = acc;
        if (part_or(1, WORKERS, gave_up())) break;  // (all workers or none)
        if (warp < 4 && mine) {
          float* w = a.weights + (size_t)u * a.max_seq_len + j;
          float v = acc;
#pragma unroll
          for (int i = 0; i < P - 1; ++i) v += sums[i][ln.t];
          *w = p.decay != 0.f ? fmaf(p.decay, *w, v) : v;
        }
      }
    }
    if (FEW && !SUM) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v = rl[i];
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
        if (lane == 0) {
          wm[i] = rm[i];
          wl[i] = v;
        }
      }
    }
    // (with the flag up every wait returns at once: all workers come here, and leave together or not at all)
    if (part_or(1, WORKERS, gave_up())) {
      ok = false;
      break;
    }
    if (!SUM) {
      // ---- the range's maxima and sums: the four warps that hold a row's columns, joined in order
      float* out = part_sums(w);
      for (int lr = tid; lr < p.rows; lr += WORKERS) {
        const int c = lr % N, wg = FEW ? c / 2 : c / (N / P), at = FEW ? c % 2 : lr / N * (N / P) + c % (N / P);
        const float* m0 = reinterpret_cast<const float*>(smem + SM::wm(NR)) + 4 * wg * (NR / P) + at;
        const float* l0 = reinterpret_cast<const float*>(smem + SM::wl(NR)) + 4 * wg * (NR / P) + at;
        float m = NO_REF, l = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float mi = m0[i * (NR / P)], mn = fmaxf(m, mi);
          l = l * ex2(m - mn) + l0[i * (NR / P)] * ex2(mi - mn);
          m = mn;
        }
        out[2 * lr] = m;
        out[2 * lr + 1] = l;
      }
    }
    part_sync(1, WORKERS);  // the next part's queries and sums may come
  }
  // A CTA that gave up leaves maxima that are NaN for its part and those it did not come to: their units take no weight from
  // the call.  What it still has under way lands before it leaves; the waits are bounded.
  if (!SUM && warp < WARPS && !ok) {
    for (t = t_part; t < t_end;) {
      const Part w = part_at(t);
      float* out = part_sums(w);
      if (w.it0 < w.it1)
        for (int lr = tid; lr < p.rows; lr += WORKERS) out[2 * lr] = NAN;
    }
  }
  __syncthreads();  // (nobody waits any more)
  if (warp == WARPS && gave_up()) {
    for (uint32_t i = kr_n < C::STAGES ? 0 : kr_n - C::STAGES; i < kr_n; ++i) bar_land(&kr_bar[i % C::STAGES], i / C::STAGES & 1);
    mma_commit(&end_bar);
    bar_land(&end_bar, 0);
  }
  // (a CTA without tiles too: no kernel ends before the one it follows)
  if (SUM) asm volatile("griddepcontrol.wait;" ::: "memory");
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    tm_free(tmem, TM_COLS);
  }
}

// the rows' normalisers, a warp each
static __global__ void __launch_bounds__(ADD_THREADS) normaliser_kernel(const __grid_constant__ Plan p) {
  extern __shared__ int pre[];
  const MultiArgs& a = p.a;
  int* lens = pre + a.batch + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;");
  if (warp == 0) tile_prefix(a, lens, pre, false, [&](int L) { return seq_tiles(L, a.W); });
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long i = (long long)blockIdx.x * (ADD_THREADS / 32) + warp;
  if (i >= (long long)p.n_units * p.rows) return;
  const int u = (int)(i / p.rows), row = (int)(i % p.rows), h = u % a.Hkv, b = (u / a.Hkv) % a.batch, ll = u / (a.Hkv * a.batch);
  const int L = lens[b], tiles = pre[b + 1] - pre[b];
  if (L <= 0) return;
  const long long per_layer = (long long)pre[a.batch] * a.Hkv, total = per_layer * a.n_layers_call;
  const float v = normaliser(p, u, row, ll * per_layer + (long long)pre[b] * a.Hkv + (long long)h * tiles, quant_tiles(L, a.W), tiles,
                             min((long long)p.G, total), total, lane);
  if (lane == 0) p.norms[i] = v == v ? v : INFINITY;  // (no weight from a row that was given up)
}

// Weights from stored logits: pieces of 1024 positions of the units, in one list (of the positions there are, whatever the
// capacity), dealt out to the CTAs in turn.
constexpr int PIECE = 4 * ADD_THREADS;
static __global__ void __launch_bounds__(ADD_THREADS) weights_add_kernel(const __grid_constant__ Plan p) {
  __shared__ float lse[STORE_ROWS];
  extern __shared__ int pre[];
  const MultiArgs& a = p.a;
  int* lens = pre + a.batch + 1;
  int* pieces = lens + a.batch;                // prefix of the sequences' pieces
  int* again = pieces + a.batch + 1;           // the lengths once more (by another warp)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 0) tile_prefix(a, lens, pre, false, [&](int L) { return seq_tiles(L, a.W); });
  if (warp == 1) tile_prefix(a, again, pieces, false, [&](int L) { return (L + PIECE - 1) / PIECE; });
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long per_layer = (long long)pre[a.batch] * a.Hkv, total = per_layer * a.n_layers_call;
  const long long layer_pieces = (long long)pieces[a.batch] * a.Hkv;
  for (long long i = blockIdx.x; i < layer_pieces * a.n_layers_call; i += gridDim.x) {
    const int ll = a.n_layers_call > 1 ? (int)quick_div(i, layer_pieces) : 0;
    const long long in_layer = i - ll * layer_pieces;
    int lo = 0, hi = a.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((long long)pieces[mid] * a.Hkv <= in_layer) lo = mid;
      else hi = mid - 1;
    }
    const int b = lo, L = lens[b], n = pieces[b + 1] - pieces[b], tiles = pre[b + 1] - pre[b];
    const long long r = in_layer - (long long)pieces[b] * a.Hkv;
    const int h = (int)quick_div(r, n), j0 = (int)(r - (long long)h * n) * PIECE + tid * 4;
    const int u = (ll * a.batch + b) * a.Hkv + h;
    float4 x[STORE_ROWS];
    const float* src = p.logits + (size_t)u * p.rows * p.s_pad + j0;
#pragma unroll
    for (int r = 0; r < STORE_ROWS; ++r)
      if (r < p.rows && j0 < L) x[r] = *reinterpret_cast<const float4*>(src + r * p.s_pad);
    if (warp < p.rows) {
      const float v = normaliser(p, u, warp, ll * per_layer + (long long)pre[b] * a.Hkv + (long long)h * tiles, quant_tiles(L, a.W),
                                 tiles, min((long long)p.G, total), total, lane);
      if (lane == 0) lse[warp] = v;
    }
    __syncthreads();
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < STORE_ROWS; ++r)
      if (r < p.rows && lse[r] == lse[r]) {  // (a row that was given up has logits that were never written)
        s[0] += ex2(x[r].x - lse[r]);
        s[1] += ex2(x[r].y - lse[r]);
        s[2] += ex2(x[r].z - lse[r]);
        s[3] += ex2(x[r].w - lse[r]);
      }
    float* w = a.weights + (size_t)u * a.max_seq_len + j0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (j0 + i < L) w[i] = p.decay != 0.f ? fmaf(p.decay, w[i], s[i]) : s[i];
    __syncthreads();  // (the normalisers have been read)
  }
}

// layers of one set of launches: stored logits take up to LOGITS_ROOM (or one layer's), the layers after them their place
constexpr size_t LOGITS_ROOM = (size_t)256 << 20;
inline int layers_at_once(const MultiArgs& a) {
  const int rows = a.n * a.g;
  if (rows > STORE_ROWS) return a.n_layers_call;
  const size_t layer = (size_t)a.batch * a.Hkv * rows * (((size_t)a.max_seq_len + 3) / 4 * 4) * sizeof(float);
  const size_t n = layer >= LOGITS_ROOM ? 1 : LOGITS_ROOM / layer;
  return n < (size_t)a.n_layers_call ? (int)n : a.n_layers_call;
}
// layers l0 .. of a call, as a call of their own
inline MultiArgs layers_of(const MultiArgs& a, int l0, int n) {
  MultiArgs s = a;
  const size_t units = (size_t)l0 * a.batch * a.Hkv;
  s.layer0 += l0;
  s.n_layers_call = n;
  s.q = static_cast<const uint8_t*>(a.q) + units * a.g * a.n * D * (a.in_bf16 ? 2 : 4);
  s.weights = a.weights + units * a.max_seq_len;
  return s;
}

// rows of one launch, and the plan of the launches that begin at row0; returns the scratch bytes
template <int KF>
size_t make_plan(const MultiArgs& a, int sms, int row0, Plan* p) {
  const int all = a.n * a.g;
  p->a = a;
  p->row0 = row0;
  p->rows = all - row0 < MAX_ROWS ? all - row0 : MAX_ROWS;
  p->P = KF == KVQ_TQ3_QJL && p->rows > NARROW_ROWS ? 4 : 2;
  p->nb = (p->rows + 8 * p->P - 1) / (8 * p->P);
  p->n_units = a.n_layers_call * a.batch * a.Hkv;
  p->G = sms * (4 / p->P);
  p->s_pad = ((long long)a.max_seq_len + 3) / 4 * 4;
  p->decay = row0 == 0 ? a.decay : 1.f;
  const bool store = all <= STORE_ROWS;
  const size_t parts = align256((size_t)(2 * p->n_units + p->G) * p->rows * 2 * sizeof(float));
  p->parts = reinterpret_cast<float*>(a.scratch);
  p->logits = store && a.scratch ? reinterpret_cast<float*>(a.scratch + parts) : nullptr;
  p->norms = !store && a.scratch ? reinterpret_cast<float*>(a.scratch + parts) : nullptr;
  return parts + (size_t)p->n_units * p->rows * (store ? p->s_pad : 1) * sizeof(float);
}

inline cudaError_t launch_norms(const Plan& p, size_t pre, cudaStream_t s) {
  const long long rows = (long long)p.n_units * p.rows;
  return go<normaliser_kernel>(dim3((unsigned)((rows + ADD_THREADS / 32 - 1) / (ADD_THREADS / 32))), ADD_THREADS, pre, true, s, p);
}

template <int KF>
cudaError_t launch_rows(const Plan& p, cudaStream_t s) {
  const size_t pre = (size_t)(2 * p.a.batch + 1) * 4, smem = Smem<KF>::pre(p.nb * 8 * p.P) + pre;
  const dim3 grid((unsigned)p.G);
  const unsigned threads = 128 * p.P + 32;
  cudaError_t e;
  if constexpr (KF == KVQ_TQ3_QJL) {
    if (p.P == 4) {
      e = go<weights_kernel<KF, false, 8, 4>>(grid, threads, smem, false, s, p);
      if (e == cudaSuccess) e = launch_norms(p, pre, s);
      return e != cudaSuccess ? e : go<weights_kernel<KF, true, 8, 4>>(grid, threads, smem, true, s, p);
    }
  }
  e = p.rows <= 4 ? go<weights_kernel<KF, false, 2, 2>>(grid, threads, smem, false, s, p)
                  : go<weights_kernel<KF, false, 8, 2>>(grid, threads, smem, false, s, p);
  if (e != cudaSuccess) return e;
  if (p.logits == nullptr) {
    e = launch_norms(p, pre, s);
    return e != cudaSuccess ? e : go<weights_kernel<KF, true, 8, 2>>(grid, threads, smem, true, s, p);
  }
  // eight CTAs an SM at most: no more than are there at once
  const long long most = (long long)p.n_units * ((p.a.max_seq_len + PIECE - 1) / PIECE), there = (long long)p.G * 4;
  return go<weights_add_kernel>(dim3((unsigned)(most < there ? most : there)), ADD_THREADS, (size_t)(4 * p.a.batch + 2) * 4, true, s, p);
}

template <int KF>
size_t scratch_bytes(const MultiArgs& a, int sms) {
  Plan p;
  return make_plan<KF>(layers_of(a, 0, layers_at_once(a)), sms, 0, &p);
}

template <int KF>
cudaError_t launch(const MultiArgs& a, int sms, cudaStream_t s) {
  const int most = layers_at_once(a);
  for (int l0 = 0; l0 < a.n_layers_call; l0 += most) {
    const MultiArgs part = layers_of(a, l0, a.n_layers_call - l0 < most ? a.n_layers_call - l0 : most);
    for (int row0 = 0; row0 < a.n * a.g;) {
      Plan p;
      make_plan<KF>(part, sms, row0, &p);
      const cudaError_t e = launch_rows<KF>(p, s);
      if (e != cudaSuccess) return e;
      row0 += p.rows;
    }
  }
  return cudaSuccess;
}

}  // namespace weights
}  // namespace kvq

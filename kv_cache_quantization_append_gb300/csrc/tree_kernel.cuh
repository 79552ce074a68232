// Tree attention: the kernels of one key format (included by one translation unit per format).
//
// A unit's rows (query heads of its nodes, node-major: row = node * g + head) are the N side of the products and
// its positions the M side, so that the tensor cores do work for the rows there are (16 a CTA with two threads to a
// position, up to 96 with four, more rows in further CTAs) and a position's scales and norms belong to one thread:
//   S^T [128 positions x N rows]  = K~ [128 x 128] Q~^T         (tcgen05.mma, K~ in tensor memory, Q~ in shared)
//   O^T [128 channels x N rows] += V~^T [128 x 128] P^T         (both in shared memory)
// where K~ and V~ are the dequantised records and Q~ the queries in the records' space (rotated, balanced), or the
// window's and the drafts' raw vectors and the queries as they are.  The softmax runs in base 2 down a thread's own
// columns against a reference per row that moves only when a logit passes it by 15 (weights stay below 2^15): no
// exchange between threads but one vote per tile.
//
// Two launches:
//  1. tree_kernel: the tiles of all units in one list, cut into equal ranges, one per CTA (stream-K).  The worker warps
//     (8, or 16 in one CTA an SM) dequantise K~, then V~ while the tensor cores run the logits, then take the softmax,
//     then go on to the next K~ while the tensor cores run P V; one more warp issues the products (issuing them costs a
//     warp about as long as they take, which the others would all wait for) and the copies of the next tile's records,
//     whose keys and values have one place each in shared memory (held in registers until used they spilled).  Two CTAs
//     an SM fill each other's waits.  A range's part of a unit's records, and of its raw positions, ends as one partial
//     record (reference, sum, O).
//  2. tree_merge_kernel (a programmatic dependent): joins a row's records in a fixed order, undoes the balancing and
//     the rotation.
// Rotating the queries and following the parents is done again by every CTA that needs them: a kernel in front that did
// it once cost 6 us of latency.
//
// Measured (a call, both launches): 48 rows of each of 8 KV heads over 32K positions Q4 60 us (108 TFLOP/s, 0.72 TB/s);
// 128 rows over 8 sequences of up to 32K TQ3 516 us (187 TFLOP/s); 192 rows over 4 sequences of up to 9001 Q8 119 us (180
// TFLOP/s); 15 rows over 700 positions 22.5 us.  Bound in the long cases by the chain of one tile, one under way in a CTA.  By
// clocks read in a private copy, TQ3 and 64 rows, a tile takes 6200 cycles: keys' records 500, key conversion 1250, the end of
// the last P V 400, value conversion 1750 (the logits are issued meanwhile, 54 cycles a product), logits 350, softmax 1500, and
// hand-overs.  The short case is one pass' latency through both launches: lengths, table, records, product, softmax, product,
// join.
//
// Operands: each of K~, V~, Q~ and P is a pair of 16-bit values, hi and lo, and every product hi hi + hi lo + lo hi, so that
// an output is the definition's up to its own rounding (1e-7 to 4e-6 of the largest beyond a bf16 output's half step).  fp16
// pairs hold 22 bits of records; once-rounded fp16 operands took 48, 250, 96 and 18.5 us for the cases above, but their
// errors, up to 1.3e-3 of the largest output where attention is peaked, came on top of the output's rounding.  Raw vectors
// of a bf16 cache are bf16 pairs, which hold 16 bits of any magnitude (its queries one, exactly); a float cache's are fp16
// pairs, the values scaled.  TQ3 keys are [c, +-w], 256 wide against [q~, S q~]: the centroids c are exact, the residual's
// weight w = sqrt(pi/2)/128 gamma is a pair, and the thread that owns the position multiplies by the norm n.
#pragma once

#include "records.cuh"

namespace kvq {
namespace tree {

using namespace tc;
using namespace records;

// Rows of a block (a CTA's): up to 16 take two threads to a position and two CTAs an SM (15 rows over 32K Q4 46 us, as a
// block of one CTA an SM 56; over 4000 positions 27 and 23), more take four threads and one CTA.  What a block holds in
// shared memory ends at 96 rows (192 rows over 4 x 9001 Q8 118 us, in blocks of 64 140), for TQ3 keys, whose queries come
// with their projections, at 64 (128 rows over 8 x 32K 515 us, in blocks of 32 948).
constexpr int FEW_ROWS = 16, MAX_ROWS = 96, TQ_ROWS = 64;
// Places in the list of tiles: a raw tile counts as three of records (its rows come as fp32 or bf16 and are not requested
// a tile ahead), and belongs to the range that holds its first place.  Measured with 1 to 5 places: 5 nodes at 32K Q4 58, 52,
// 46, 59, 52 us; 16 nodes 72, 66, 60, 56, 56; 16 nodes over 2 x 2000 TQ3 43, 31, 43, 43, 45; six other sizes the same within
// 6 %.
constexpr int RAW_PLACES = 3;
constexpr int MERGE_WARPS = 8;
constexpr float NO_REF = -1e30f;  // reference of a row that has met no position yet
// A reference is put so that the row's largest weight so far is 2^START, and put again when one passes 2^MOST.  Pairs of fp16
// end at 2^-24: with the first tile's largest at 1 the positions behind an early sink 17 above them lost a third of their
// weight in sums of 6400 positions (2.4e-3 of the output); at 2^7 what is lost is below 2^-32 of the sink's weight each.
constexpr float START = 7.f, MOST = 15.f;
// Tiles whose P V share an accumulator.  The tensor cores cut off each sum's low bits, 24 sums a tile: 512 tiles in one lost
// 3e-4 of the output, 16 lose 2.3e-5 at most and are then added to the part's record with rounding to nearest (1 % of the
// time).
constexpr int DRAIN = 16;

// what the launches share: sizes from the host, pointers into the caller's scratch
struct Plan {
  MultiArgs a;
  int rb, N, n_units, G;  // row blocks of N rows per unit, units (with row blocks), CTAs
  // [2 n_units + G][2 N + 128 N]: range c's part of unit u's records (+ 0) or raw positions (+ 1) at 2 u + c
  float* records;       
};

__host__ __device__ inline int raw_count(int L, int W, int n) { return (W > 0 ? (L < W - 1 ? L : W - 1) : 0) + n; }
// positions below this may be read through their records by some node (the deepest is at L + n - 1)
__host__ __device__ inline int quant_end(int L, int W, int n) {
  if (W <= 0) return L;
  const int e = L - W + n;
  return e < 0 ? 0 : e > L ? L : e;
}
__device__ __forceinline__ int seq_tiles(const MultiArgs& a, int L) {
  return (quant_end(L, a.W, a.n) + TILE - 1) / TILE + (raw_count(L, a.W, a.n) + TILE - 1) / TILE * RAW_PLACES;
}
template <int KF>
struct Cfg {
  static constexpr bool TQ = KF == KVQ_TQ3_QJL;
  static constexpr int KD = TQ ? 256 : 128;         // width of a query image: [q~] or [q~, S q~]
  static constexpr uint32_t PLANE = TILE * D * 2;   // 32 KB: values are two of them, hi and lo
  // columns of keys in tensor memory: KD / 2 (hi), then lo (TQ3: of the weights and of raw keys only, which share them)
  static constexpr uint32_t K_COLS = KD / 2 + 64;
};

// hi and lo of a pair as fp16, or as bf16 (16 bits of any magnitude)
__device__ __forceinline__ void split2(bool bf16, float a, float b, uint32_t& hi, uint32_t& lo) {
  if (!bf16) return tc::split2(a, b, hi, lo);
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  const float2 hf = __bfloat1622float2(h);
  const __nv_bfloat162 l = __floats2bfloat162_rn(a - hf.x, b - hf.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// channels 4 lane .. + 3 of row r of a query image, in the order in which put_k leaves the keys' channels
template <int KF>
__device__ __forceinline__ void put_q(uint8_t* img, int r, int N, uint32_t plane, const float (&y)[4], bool bf16, int lane) {
  uint32_t h[2], l[2];
  split2(bf16, y[0], y[1], h[0], l[0]);
  split2(bf16, y[2], y[3], h[1], l[1]);
  if (KF != KVQ_Q8G32) {
    uint8_t* dst = img + km_off(r, 4 * lane & ~7, N) + 8 * (lane & 1);
    *reinterpret_cast<uint2*>(dst) = pack4<KF == KVQ_Q4G32>(h[0], h[1], lane);
    *reinterpret_cast<uint2*>(dst + plane) = pack4<KF == KVQ_Q4G32>(l[0], l[1], lane);
    return;
  }
  const int kk = lane >> 2, i0 = 2 * (lane & 1), at = 4 * (kk & 3) + (lane & 2);  // channels 16 kk + 4 (lane & 3) + e
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    uint8_t* dst = img + km_off(r, 16 * (2 * (i0 + p) + (kk >> 2)) + at, N);
    *reinterpret_cast<uint32_t*>(dst) = h[p];
    *reinterpret_cast<uint32_t*>(dst + plane) = l[p];
  }
}

// ------------------------------------------------------------------ dequantising
// eight codes of a word times scale plus zero, and their lo parts
__device__ __forceinline__ void dequant8(uint32_t word, uint32_t s2, uint32_t z2, uint4& o, uint4& l) {
  __half2 c[4];
  nibbles(word, c);
  const float s = __low2float(u2h(s2)), z = __low2float(u2h(z2));
  const float2 f0 = __half22float2(c[0]), f1 = __half22float2(c[1]), f2 = __half22float2(c[2]), f3 = __half22float2(c[3]);
  tc::split2(z + s * f0.x, z + s * f0.y, o.x, l.x);
  tc::split2(z + s * f1.x, z + s * f1.y, o.y, l.y);
  tc::split2(z + s * f2.x, z + s * f2.y, o.z, l.z);
  tc::split2(z + s * f3.x, z + s * f3.y, o.w, l.w);
}

// keys of the thread's part of its position to the position's tensor-memory lane: columns 0..63 (TQ3: centroids), then
// TQ3's signed weights, then the lo parts
template <int KF, int P>
__device__ __forceinline__ void put_k(uint32_t col, const Lane& ln, const uint8_t* rec, const uint4& cent) {
  using R = Rec<KF>;
  const uint8_t* hb = rec + (ln.t >> 5) * R::KH;
  const int tt = ln.t & 31;
  constexpr int CHUNKS = (KF == KVQ_Q8G32 ? 8 : 4) / P;  // 16-byte chunks of the record
  uint4 k[CHUNKS];
  if (KF == KVQ_Q8G32) {
    // in the order of the record: 16-byte chunk m = 2 i + h, its word w the channels 16 (4 h + w) + 2 i + {0, 1, 8, 9};
    // chunk m lies at m ^ (t & 1)
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) k[c] = *reinterpret_cast<const uint4*>(hb + tt * 128 + 16 * (CHUNKS * ln.hf + (c ^ (tt & 1))));
  } else if constexpr (CHUNKS == 2) {
    lds32(hb + tt * 64 + 32 * ln.hf, tt & 2, k[0], k[1]);
  } else {
    k[0] = *reinterpret_cast<const uint4*>(hb + tt * 64 + 16 * ln.hf);
  }
  if (KF == KVQ_Q4G32) {
    const uint4 km = *reinterpret_cast<const uint4*>(hb + R::K_MAIN + tt * 16);
    const uint32_t sc[2] = {km.x, km.y}, zr[2] = {km.z, km.w};
#pragma unroll
    for (int G = 0; G < 4; ++G) {
      const uint32_t s2 = G & 1 ? dup_hi(sc[G >> 1]) : dup_lo(sc[G >> 1]), z2 = G & 1 ? dup_hi(zr[G >> 1]) : dup_lo(zr[G >> 1]);
      uint4 o[CHUNKS], l[CHUNKS];
#pragma unroll
      for (int i = 0; i < CHUNKS; ++i) dequant8(G == 0 ? k[i].x : G == 1 ? k[i].y : G == 2 ? k[i].z : k[i].w, s2, z2, o[i], l[i]);
      const uint32_t at = col + 16 * G + 4 * CHUNKS * ln.hf;
      if constexpr (CHUNKS == 2) {
        tm_st8(at, o[0], o[1]);
        tm_st8(at + 64, l[0], l[1]);
      } else {
        tm_st4(at, o[0]);
        tm_st4(at + 64, l[0]);
      }
    }
  } else if (KF == KVQ_Q8G32) {
    const __half2 off = u2h(0x64806480u);  // 1024 + 128
    const uint2 sc = *reinterpret_cast<const uint2*>(hb + R::K_MAIN + tt * 8);
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const uint32_t wd[4] = {k[c].x, k[c].y, k[c].z, k[c].w}, s = c & 1 ? sc.y : sc.x;
      uint32_t o[8], l[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t s2 = i & 2 ? dup_hi(s) : dup_lo(s);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const __half2 v = __hsub2(u2h(prmt(wd[i], 0x64646464u, x ? 0x4342 : 0x4140)), off);
          const float d = __low2float(u2h(s2));
          const float2 f = __half22float2(v);
          tc::split2(d * f.x, d * f.y, o[2 * i + x], l[2 * i + x]);
        }
      }
      const uint32_t at = col + 8 * (CHUNKS * ln.hf + c);
      tm_st8(at, make_uint4(o[0], o[1], o[2], o[3]), make_uint4(o[4], o[5], o[6], o[7]));
      tm_st8(at + 64, make_uint4(l[0], l[1], l[2], l[3]), make_uint4(l[4], l[5], l[6], l[7]));
    }
  } else {
    const float wf = QJL_CONST * __half2float(reinterpret_cast<const __half*>(hb + R::K_MAIN)[HALF + tt]);
    uint32_t wh, wl;
    tc::split2(wf, wf, wh, wl);
    wh ^= 0x80008000u;  // -w
    wl ^= 0x80008000u;
#pragma unroll
    for (int i = 0; i < 4 * CHUNKS; i += 2) {
      uint4 o[2], s[2], l[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint4& q = k[i >> 2];
        const uint32_t word = ((i + x) & 3) == 0 ? q.x : ((i + x) & 3) == 1 ? q.y : ((i + x) & 3) == 2 ? q.z : q.w;
        // the eight centroids' bytes in two register pairs (low bytes: cent.x, .y; high bytes: cent.z, .w), picked by
        // byte permutes with the codes as selectors
        const uint32_t sel = (word & 0x07070707u) | ((word << 1) & 0x70707070u);
        const uint32_t l0 = prmt(cent.x, cent.y, sel), h0 = prmt(cent.z, cent.w, sel);
        const uint32_t l1 = prmt(cent.x, cent.y, sel >> 16), h1 = prmt(cent.z, cent.w, sel >> 16);
        o[x] = make_uint4(__byte_perm(l0, h0, 0x5140), __byte_perm(l0, h0, 0x7362), __byte_perm(l1, h1, 0x5140),
                          __byte_perm(l1, h1, 0x7362));
        // bit 6: sign of projection 2j, bit 7: of 2j + 1 (set: +w): a permute that spreads a byte's top bit
        const uint32_t lo = word << 1;
        uint32_t m[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] = prmt(lo, word, (uint32_t)((8 + j) << 4) | (uint32_t)((12 + j) << 12)) & 0x80008000u;
        s[x] = make_uint4(wh ^ m[0], wh ^ m[1], wh ^ m[2], wh ^ m[3]);
        l[x] = make_uint4(wl ^ m[0], wl ^ m[1], wl ^ m[2], wl ^ m[3]);
      }
      const uint32_t at = col + 16 * CHUNKS * ln.hf + 4 * i;
      tm_st8(at, o[0], o[1]);
      tm_st8(at + 64, s[0], s[1]);
      tm_st8(at + 128, l[0], l[1]);
    }
  }
}

// values of the thread's two positions, eight channels of each of its groups; positions from `left` on (of the pair) are
// zero
template <int KF, int P>
__device__ __forceinline__ void put_v(uint8_t* vb, const Lane& ln, const uint8_t* rec, int left) {
  using R = Rec<KF>;
  constexpr uint32_t PLANE = Cfg<KF>::PLANE;
  constexpr int GROUPS = 8 / P;
  const uint8_t* hb = rec + R::V0 + (ln.vp >> 4) * R::VH;
  const int pp = ln.vp & 15;
  const uint32_t keep = left >= 2 ? 0xffffffffu : left == 1 ? 0x0000ffffu : 0u;  // (records there may hold anything)
  // rows 2 vr and 2 vr + 1 stay neighbours in the rotated order of a pair's rows
  const uint8_t* at = hb + 128 * pp + 32 * ((ln.vr + pp) & 3);
  uint32_t w0[GROUPS], w1[GROUPS];
  if constexpr (GROUPS == 4) {
    uint4 a, b;
    lds32(at, ln.vr & 1, a, b);
    w0[0] = a.x, w0[1] = a.y, w0[2] = a.z, w0[3] = a.w;
    w1[0] = b.x, w1[1] = b.y, w1[2] = b.z, w1[3] = b.w;
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(at + 8 * ln.vg), b = *reinterpret_cast<const uint2*>(at + 16 + 8 * ln.vg);
    w0[0] = a.x, w0[1] = a.y;
    w1[0] = b.x, w1[1] = b.y;
  }
  const uint32_t* meta = reinterpret_cast<const uint32_t*>(hb + R::V_MAIN) + 32 * ln.vg + pp;
  uint8_t* base = vb + mm_off(64 * ln.vg + 8 * ln.vr, 2 * ln.vp);
#pragma unroll
  for (int G = 0; G < GROUPS; ++G) {
    const uint32_t vs = meta[16 * G] & keep, vz = meta[64 + 16 * G] & keep;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool e = (i ^ ln.vr) & 1;  // which position of the pair
      const uint32_t pick = e ? 0x7531u : 0x6420u, dup = e ? 0x3232u : 0x1010u;
      uint8_t* dst = base + (e ? 16 : 0) + 512 * G;
      uint4 o, l;
      dequant8(prmt(w0[G], w1[G], pick), prmt(vs, vs, dup), prmt(vz, vz, dup), o, l);
      *reinterpret_cast<uint4*>(dst) = o;
      *reinterpret_cast<uint4*>(dst + PLANE) = l;
    }
  }
}

// the sums of 2 N columns with lane ^ BIT's: each keeps the N of its half
template <int N, int BIT>
__device__ __forceinline__ void halve(float* l, int lane) {
  const bool up = lane & BIT;
#pragma unroll
  for (int c = 0; c < N; ++c) {
    const float mine = up ? l[N + c] : l[c], other = up ? l[c] : l[N + c];
    l[c] = mine + __shfl_xor_sync(FULL, other, BIT);
  }
}

// ------------------------------------------------------------------ 1. the tiles
// dynamic shared memory: V planes | query image | P planes | records | prefix of the sequences' tiles, lengths
template <int KF>
struct Smem {
  using C = Cfg<KF>;
  static constexpr uint32_t V = 0, Q = 2 * C::PLANE;
  static __host__ __device__ constexpr uint32_t P(int N) { return Q + N * C::KD * 4; }
  static __host__ __device__ constexpr uint32_t R(int N) { return P(N) + N * TILE * 4; }
  static __host__ __device__ constexpr uint32_t total(int N) { return R(N) + Rec<KF>::BYTES; }
};

// P threads to a position: 2 (two CTAs an SM), or 4 for more than FEW_ROWS rows, which then share the dequantised keys and
// values (one CTA an SM); F32: the raw vectors and queries of a float cache
template <int KF, int NC, bool F32, int P>
__global__ void __launch_bounds__(128 * P + 32, P == 4 ? 1 : 2) tree_kernel(const __grid_constant__ Plan p) {
  using C = Cfg<KF>;
  using SM = Smem<KF>;
  constexpr int WORKERS = 128 * P, WARPS = WORKERS / 32;  // and the warp that issues the products
  constexpr int N = P * NC;  // rows, NC of them to a thread, CH at a time
  constexpr int CH = 8;
  constexpr bool TQ = C::TQ;
  // tensor memory: K | S | O
  constexpr uint32_t C_S = C::K_COLS, C_O = C_S + N, COLS = C_O + N;
  constexpr uint32_t TM_COLS = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  constexpr uint32_t ID_S = idesc(TILE, N, false, false), ID_O = idesc(D, N, true, true);
  constexpr uint32_t RAW_TYPE = F32 ? 0 : BF16_OPERANDS;  // of raw parts
  constexpr uint64_t LO_Q = (N * C::KD * 2) >> 4, LO_V = C::PLANE >> 4, LO_P = (N * TILE * 2) >> 4;
  extern __shared__ __align__(1024) uint8_t smem[];
  // kr_bar, vr_bar: a tile's records have landed; k_bar, v_bar: its keys, values are in place (one arrival a worker
  // warp); p_bar: its weights are; qk_bar, pv_bar: its products are done
  __shared__ __align__(8) uint64_t kr_bar, vr_bar, k_bar, v_bar, p_bar, qk_bar, pv_bar, end_bar;
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh, leave_sh[2];  // leave_sh: what the workers act on, by turns of the tiles
  __shared__ __align__(16) float mref[N], fac[N];
  __shared__ float mrec[N];  // the references of the part's record so far
  __shared__ float wmax[4][N];
  __shared__ unsigned long long nodes[KVQ_MAX_TREE];  // ancestors-or-self of each node (0: not there)
  // columns (rows of the unit) that are there and at depth at most i; that have node i among their ancestors-or-self
  // (by the threads' groups of columns)
  __shared__ uint32_t shallow[P][KVQ_MAX_TREE], below[P][KVQ_MAX_TREE];
  __shared__ int par[KVQ_MAX_TREE];
  __shared__ bool sick_sh[P][TILE];  // a raw position's values (by the threads that share it) were not all finite
  __shared__ int vtop;  // float caches: largest raw value of the part, as an integer
  const MultiArgs& a = p.a;
  const int tid = threadIdx.x, warp = __shfl_sync(FULL, tid >> 5, 0), lane = tid & 31;
  int* pre = reinterpret_cast<int*>(smem + SM::total(N));
  int* lens = pre + a.batch + 1;

  if (tid == 0) {
    bar_init(&kr_bar, 1);
    bar_init(&vr_bar, 1);
    bar_init(&k_bar, WARPS);
    bar_init(&v_bar, WARPS);
    bar_init(&p_bar, 1);
    bar_init(&end_bar, 1);
    bar_init(&qk_bar, 1);
    bar_init(&pv_bar, 1);
    abort_sh = leave_sh[0] = leave_sh[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) tile_prefix(a, lens, pre, blockIdx.x == 0, [&](int L) { return seq_tiles(a, L); });
  if (warp == 1) tm_alloc(&tmem_sh, TM_COLS);
  fence_before();
  asm volatile("griddepcontrol.launch_dependents;");
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(FULL, tmem_sh, 0), sbase = smem_u32(smem);

  // this CTA's range of the list of tiles
  const long long per_layer = (long long)pre[a.batch] * a.Hkv * p.rb, total = per_layer * a.n_layers_call;
  // (no range is empty: the merge reads every range that has records of a unit)
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
  uint32_t kr_phase = 0, vr_phase = 0, k_phase = 0, v_phase = 0, p_phase = 0, qk_phase = 0, pv_phase = 0;
  uint32_t kr_n = 0, vr_n = 0;  // copies that the ninth warp has begun
  bool pv_pending = false;
  const auto wait = [&](uint64_t* bar, uint32_t& phase) {
    bar_wait(bar, phase, &abort_sh, a.p.status, a.wait_ns);
    phase ^= 1;
  };
  const auto wait_pv = [&] {
    if (pv_pending) {
      wait(&pv_bar, pv_phase);
      pv_pending = false;
    }
  };
  // this warp's part of the keys is in tensor memory
  const auto k_done = [&] {
    tm_wait_st();
    fence_before();
    __syncwarp();
    if (lane == 0) bar_arrive(&k_bar);
  };
  // this thread's columns (rows of the unit)
  const int grp = (warp >> 2) % P, col0 = grp * NC;                                    
  const uint32_t lane_addr = tmem + ((uint32_t)(32 * (warp & 3)) << 16);  // its lane: position ln.t, channel ln.t
  bool ok = true;

  // the part that begins at place t: its unit (sequence, head and row block) and this CTA's tiles of it; t goes on behind it
  struct Part {
    int ll, b, h, rbi, u, it0, it1, nq, qend;
    bool raw;
  };
  const auto part_at = [&](long long& t) {
    Part w;
    w.ll = a.n_layers_call > 1 ? (int)quick_div(t, per_layer) : 0;
    const long long in_layer = t - w.ll * per_layer;
    int lo = 0, hi = a.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((long long)pre[mid] * a.Hkv * p.rb <= in_layer) lo = mid;
      else hi = mid - 1;
    }
    w.b = lo;
    const int tiles = pre[lo + 1] - pre[lo];
    const long long r = in_layer - (long long)pre[lo] * a.Hkv * p.rb;
    const int hr = (int)quick_div(r, tiles), place0 = (int)(r - (long long)hr * tiles);
    w.h = hr / p.rb;
    w.rbi = hr - w.h * p.rb;
    w.u = ((w.ll * a.batch + lo) * a.Hkv + w.h) * p.rb + w.rbi;
    w.qend = quant_end(lens[lo], a.W, a.n);
    w.nq = (w.qend + TILE - 1) / TILE;
    // tiles of records come first, then those of raw positions; a part is of one kind
    w.raw = place0 >= w.nq;
    const int place1 = (int)min((long long)(w.raw ? tiles : w.nq), place0 + (t_end - t));
    t += place1 - place0;
    w.it0 = w.raw ? w.nq + (place0 - w.nq + RAW_PLACES - 1) / RAW_PLACES : place0;
    w.it1 = w.raw ? w.nq + (place1 - w.nq + RAW_PLACES - 1) / RAW_PLACES : place1;
    return w;
  };
  const auto record_of = [&](const Part& w) { return p.records + (size_t)(2 * w.u + w.raw + blockIdx.x) * (2 * N + D * N); };
  const auto gave_up = [&] { return *(volatile int*)&abort_sh != 0; };
  long long t_part = t;

  while (t < t_end && ok) {
    t_part = t;
    const Part w = part_at(t);
    const int ll = w.ll, b = w.b, h = w.h, rbi = w.rbi, layer = a.layer0 + ll, it0 = w.it0, it1 = w.it1, nq = w.nq, qend = w.qend;
    const int L = lens[b];
    const bool raw = w.raw;
    if (it0 == it1) continue;  // (the later places of a raw tile that an earlier range has)

    const int* bt = a.block_table + (size_t)b * a.max_pages_per_seq;
    if (warp == WARPS) {
      // (taken from one lane, as the warp's number and the tensor memory's address: its lanes branch together by construction,
      // and the products' operands are computed once for the warp)
      const int it0 = __shfl_sync(FULL, w.it0, 0), it1 = __shfl_sync(FULL, w.it1, 0);
      const bool raw = __shfl_sync(FULL, (int)w.raw, 0) != 0;
      // ================================================================ the products and the copies
      const uint8_t* unit_pages = a.p.pages + ((size_t)layer * a.L.n_pages * a.Hkv + h) * (size_t)a.L.page_bytes;
      using R = Rec<KF>;
      // the keys (or values) of tile `it`: lane i < 4 its half-page i (those past the end and on bad pages are left out:
      // their positions are masked); phys: that half-page's page
      const auto page_of = [&](int it) {
        const int j = it * TILE + lane * HALF;
        return lane < 4 && it < it1 && j < qend ? checked(__ldg(bt + j / PAGE), a.L.n_pages) : -1;
      };
      const auto copy = [&](int phys, bool keys) {
        ++(keys ? kr_n : vr_n);
        const uint32_t bytes = keys ? R::KH : R::VH;
        const int n = __popc(__ballot_sync(FULL, phys >= 0));
        uint64_t* bar = keys ? &kr_bar : &vr_bar;
        if (lane == 0) bar_expect(bar, n * bytes);
        __syncwarp();
        if (phys >= 0) {
          const uint8_t* src = unit_pages + (size_t)phys * page_stride + (lane & 1) * (size_t)(R::KH + R::VH);
          uint8_t* dst = smem + SM::R(N) + (keys ? lane * R::KH : R::V0 + lane * R::VH);
          if (keys) {
            bulk_g2s(dst, src, R::K_MAIN, bar);
            bulk_g2s(dst + R::K_MAIN, src + R::K_MAIN + R::V_MAIN, R::K_META, bar);
          } else {
            bulk_g2s(dst, src + R::K_MAIN, R::V_MAIN, bar);
            bulk_g2s(dst + R::V_MAIN, src + R::K_MAIN + R::V_MAIN + R::K_META, R::V_META, bar);
          }
        }
        __syncwarp();
      };
      int phys = -1;
      if (raw) {
        // raw rows go through registers a few at a time: the part's are brought to L2 while its queries are prepared
        const int nraw = raw_count(L, a.W, a.n), nring = nraw - a.n, x1 = min(nraw, (it1 - nq) * TILE);
        const size_t ring = (((size_t)layer * a.max_batch + b) * a.Hkv + h) * a.W, drafts = (((size_t)ll * a.batch + b) * a.Hkv + h) * a.n;
        constexpr uint32_t ROW = D * (F32 ? 4 : 2);
        for (int x = (it0 - nq) * TILE + lane; x < x1; x += 32) {
          if (x < nring) {
            const size_t at = (ring + (unsigned)(L - nring + x) % (unsigned)a.W) * D;
            prefetch(a.p.ringk + at, D * 4);
            prefetch(a.p.ringv + at, D * 4);
          } else {
            const size_t at = (drafts + x - nring) * ROW;
            prefetch(static_cast<const uint8_t*>(a.k) + at, ROW);
            prefetch(static_cast<const uint8_t*>(a.v) + at, ROW);
          }
        }
      } else {
        phys = page_of(it0);
        copy(phys, true);
        copy(phys, false);
      }
      if (TQ && !raw) {
        // S q~ of every row: the projection lies in the values' place
        wait(&k_bar, k_phase);
        fence_after();
        uint64_t sa = sdesc(sbase + SM::V, 2048, 128), qa = sdesc(sbase + SM::Q, N * 16, 128);
#pragma unroll 1
        for (int ks = 0; ks < D / 16; ++ks, sa += 256, qa += 2 * N) {
          mma_ss(tmem + C_S, sa, qa, ID_S, ks > 0);
          mma_ss(tmem + C_S, sa + LO_V, qa, ID_S, 1);
          mma_ss(tmem + C_S, sa, qa + LO_Q, ID_S, 1);
        }
        mma_commit(&qk_bar);
      }
      for (int it = it0; it < it1; ++it) {
        // logits: a k-step of 16 channels is 8 columns of K and 32 N bytes of the queries
        if (!raw) phys = page_of(it + 1);
        wait(&k_bar, k_phase);
        if (__any_sync(FULL, gave_up())) break;  // (the whole warp)
        fence_after();
        {
          uint64_t qa = sdesc(sbase + SM::Q, N * 16, 128);
          uint32_t ka = tmem;
          const uint32_t id = raw ? ID_S | RAW_TYPE : ID_S;
#pragma unroll 4
          for (int ks = 0; ks < D / 16; ++ks, ka += 8, qa += 2 * N) {
            mma_ts(tmem + C_S, ka, qa, id, ks > 0);
            if (F32 || !raw) mma_ts(tmem + C_S, ka, qa + LO_Q, id, 1);  // (bf16 queries have no lo part)
            if (!TQ || raw) mma_ts(tmem + C_S, ka + C::KD / 2, qa, id, 1);
          }
          if (TQ && !raw) {  // the signed weights against S q~
#pragma unroll 4
            for (int ks = 0; ks < D / 16; ++ks, ka += 8, qa += 2 * N) {
              mma_ts(tmem + C_S, ka, qa, ID_S, 1);
              mma_ts(tmem + C_S, ka, qa + LO_Q, ID_S, 1);
              mma_ts(tmem + C_S, ka + 64, qa, ID_S, 1);
            }
          }
          mma_commit(&qk_bar);
        }
        if (!raw && it + 1 < it1) copy(phys, true);  // the workers have read this tile's keys
        wait(&v_bar, v_phase);
        if (__any_sync(FULL, gave_up())) break;  // (the whole warp)
        if (!raw && it + 1 < it1) copy(phys, false);
        // O += V^T P: a k-step of 16 positions is 4096 bytes of V and 32 N of P
        wait(&p_bar, p_phase);
        if (__any_sync(FULL, gave_up())) break;  // (the whole warp)
        fence_after();
        uint64_t va = sdesc(sbase + SM::V, 2048, 128), pa = sdesc(sbase + SM::P(N), N * 16, 128);
        const uint32_t id = raw ? ID_O | RAW_TYPE : ID_O;
#pragma unroll 4
        for (int ks = 0; ks < TILE / 16; ++ks, va += 256, pa += 2 * N) {
          mma_ss(tmem + C_O, va, pa, id, (it - it0) % DRAIN > 0 || ks > 0);
          mma_ss(tmem + C_O, va + LO_V, pa, id, 1);
          mma_ss(tmem + C_O, va, pa + LO_P, id, 1);
        }
        mma_commit(&pv_bar);
      }
      ok = !__any_sync(FULL, gave_up());
      continue;
    }

    // ================================================================ the workers
    const int nraw = raw_count(L, a.W, a.n), nring = nraw - a.n, rows = a.n * a.g;
    const int full_end = a.W > 0 ? L - a.W + 1 : L;  // positions below are read through records by every node
    // pages of this thread's position and pair of tile `it` (read a tile ahead)
    const auto page_of = [&](int it, bool second) {
      const int j = it * TILE + (second ? PAGE : 0);
      return it < it1 && !raw && j < qend ? __ldg(bt + j / PAGE) : -1;
    };
    // ---- its queries (to the values' place), the parents and the first pages are requested together
    constexpr int ESZ = F32 ? 4 : 2, Q_CHUNKS = D * ESZ / 16;
    const size_t q_unit = ((size_t)(ll * a.batch + b) * a.Hkv + h) * a.g * a.n;
#pragma unroll 1
    for (int i = tid; i < N * Q_CHUNKS; i += WORKERS) {
      const int row = rbi * N + i / Q_CHUNKS;
      if (row < rows)
        cp16(smem + SM::V + 16 * i, static_cast<const uint8_t*>(a.q) + ((q_unit + (size_t)(row % a.g) * a.n + row / a.g) * Q_CHUNKS + i % Q_CHUNKS) * 16);
    }
    const bool masked = raw || it1 * TILE > full_end;  // some position is not for every node
    if (masked && tid < a.n) par[tid] = a.parents[(size_t)b * a.n + tid];
    int page = page_of(it0, ln.t & 64), vpage = page_of(it0, ln.vp & 32);
    if (tid < N) mref[tid] = NO_REF;
    if (F32 && tid == 0) vtop = 0;
    cp_wait();
    part_sync(1, WORKERS);
    // ---- queries in base-2 units, for records rotated and balanced (a bf16 cache's for raw positions as they are: the
    // logits are scaled instead)
    constexpr float raw_q = F32 ? LOGIT_SCALE : 1.f, raw_logit = F32 ? 1.f : LOGIT_SCALE;
    {
      float f[4];  // of this lane's channels
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[e] = raw ? raw_q : C_WHT * LOGIT_SCALE;
        if (a.sinkhorn && !raw) f[e] *= __half2float(a.p.sigk[((size_t)layer * a.Hkv + h) * D + 4 * lane + e]);
      }
#pragma unroll 1
      for (int r1 = warp; r1 < N; r1 += 2 * WARPS) {  // two rows at a time
        float y[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = r1 + i * WARPS;
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          if (row < N && rbi * N + row < rows) x = load4_in(smem + SM::V, (size_t)row * D + 4 * lane, !F32);
          y[i][0] = x.x, y[i][1] = x.y, y[i][2] = x.z, y[i][3] = x.w;
          if (!raw) {
            y[i][0] *= sg.x, y[i][1] *= sg.y, y[i][2] *= sg.z, y[i][3] *= sg.w;
          }
        }
        if (!raw) {
          hadamard_warp(y[0][0], y[0][1], y[0][2], y[0][3], lane);
          hadamard_warp(y[1][0], y[1][1], y[1][2], y[1][3], lane);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int e = 0; e < 4; ++e) y[i][e] *= f[e];
          if (r1 + i * WARPS < N) put_q<KF>(smem + SM::Q, r1 + i * WARPS, N, N * C::KD * 2, y[i], !F32 && raw, lane);
        }
      }
    }
    if (masked) {
      // ---- the nodes' ancestors, and what they are to this block's columns
      if (tid < a.n) {
        unsigned long long m = 0;
        for (int j = tid; j >= 0;) {
          m |= 1ull << j;
          const int q = par[j];
          if (q < -1 || q >= j) {
            if (q >= j) atomicOr(a.p.status, KVQ_DEV_BAD_NODE);
            m = 0;
            break;
          }
          j = q;
        }
        nodes[tid] = m;
      }
      part_sync(1, WORKERS);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int row = rbi * N + i * NC + lane;
        const unsigned long long anc = lane < NC && row < rows ? nodes[row / a.g] : 0ull;
        const int depth = anc ? __popcll(anc) - 1 : KVQ_MAX_TREE;
#pragma unroll 1
        for (int x = warp; x < KVQ_MAX_TREE; x += WARPS) {
          const uint32_t s = __ballot_sync(FULL, depth <= x), d = __ballot_sync(FULL, (anc >> x) & 1);
          if (lane == 0) {
            shallow[i][x] = s;
            below[i][x] = d;
          }
        }
      }
    }
    if (TQ && !raw) part_sync(1, WORKERS);  // the queries have left the values' place
    if (TQ && !raw) {
      // S q~ of every row by the tensor cores: the projection as an operand in the values' place
      const int i = tid & 127;
#pragma unroll 1
      for (int kg = tid >> 7; kg < D / 8; kg += P) {
        float s[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = __ldg(a.p.qjl_t + (8 * kg + e) * D + i);
        uint4 o, l;
        tc::split2(s[0], s[1], o.x, l.x);
        tc::split2(s[2], s[3], o.y, l.y);
        tc::split2(s[4], s[5], o.z, l.z);
        tc::split2(s[6], s[7], o.w, l.w);
        *reinterpret_cast<uint4*>(smem + SM::V + km_off(i, 8 * kg, D)) = o;
        *reinterpret_cast<uint4*>(smem + SM::V + C::PLANE + km_off(i, 8 * kg, D)) = l;
      }
      fence_async_smem();
      k_done();
      wait(&qk_bar, qk_phase);
      fence_after();
#pragma unroll 1
      for (int c = 0; c < NC; c += CH) {
        float x[CH];
        tm_ld(lane_addr + C_S + col0 + c, x);
        tm_wait_ld();
#pragma unroll
        for (int e = 0; e < CH; ++e) {
          uint8_t* dst = smem + SM::Q + km_off(col0 + c + e, D + i, N);
          *reinterpret_cast<__half*>(dst) = __float2half_rn(x[e]);
          *reinterpret_cast<__half*>(dst + N * C::KD * 2) = __float2half_rn(lo_part(x[e]));
        }
      }
    }
    // raw vector of place x in the list of ring positions and drafts (null: none; nodes that are not there may hold anything)
    const auto raw_row = [&](int x, int kv) -> const void* {
      if (x < nring)
        return (kv ? a.p.ringv : a.p.ringk) +
               ((((size_t)layer * a.max_batch + b) * a.Hkv + h) * a.W + (unsigned)(L - nring + x) % (unsigned)a.W) * D;
      if (x < nraw && nodes[x - nring])
        return static_cast<const uint8_t*>(kv ? a.v : a.k) + ((((size_t)ll * a.batch + b) * a.Hkv + h) * a.n + x - nring) * D * ESZ;
      return nullptr;
    };
    // A float cache's raw values go into fp16 pairs scaled by a power of two that brings the part's largest to 2^14..2^15:
    // its output keeps 22 bits whatever their size (below 2^-14 fp16 would lose them).  bf16 pairs need no scale.
    float v_scale = 1.f, v_unscale = 1.f;
    if (F32 && raw) {
      float top = 0.f;
#pragma unroll 1
      for (int x = (it0 - nq) * TILE + ln.t; x < min(nraw, (it1 - nq) * TILE); x += TILE) {
        const float4* row = static_cast<const float4*>(raw_row(x, 1));
        if (row == nullptr) continue;
#pragma unroll
        for (int i = 0; i < 32 / P; ++i) {
          const float4 f = row[32 / P * ln.hf + i];
          const float v[4] = {fabsf(f.x), fabsf(f.y), fabsf(f.z), fabsf(f.w)};
#pragma unroll
          for (int y = 0; y < 4; ++y) top = v[y] < INFINITY ? fmaxf(top, v[y]) : top;
        }
      }
      const int most = __reduce_max_sync(FULL, __float_as_int(top));  // (not negative: ordered as integers)
      if (lane == 0) atomicMax(&vtop, most);
      part_sync(1, WORKERS);
      // exponents of 2^-98 and less are taken as 2^-98
      const int e = max(vtop >> 23, 127 - 98);
      v_scale = __int_as_float((127 + 14 - (e - 127)) << 23);
      v_unscale = __int_as_float((127 - 14 + (e - 127)) << 23);
    }
    // adds the accumulated O (of products that are done) to the part's record, whose first it may be
    float* const rec = record_of(w);
    const int ch = (ln.t & ~7) + nibble_channel(ln.t & 7);  // tensor-memory lane = place of the channel
    const auto drain = [&](bool first) {
      if (!first) {
        if (tid < N) fac[tid] = ex2(mrec[tid] - mref[tid]);
        part_sync(1, WORKERS);
      }
      if (tid < N) mrec[tid] = mref[tid];
      fence_after();
#pragma unroll 1
      for (int c = 0; c < NC; c += CH) {
        float o[CH];
        tm_ld(lane_addr + C_O + col0 + c, o);
        tm_wait_ld();
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          float* at = rec + 2 * N + (col0 + c + i) * D + ch;
          const float v = F32 ? o[i] * v_unscale : o[i];
          *at = first ? v : fmaf(*at, fac[col0 + c + i], v);
        }
      }
    };
    fence_async_smem();
    part_sync(1, WORKERS);  // the columns' masks and references
    float l[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) l[c] = 0.f;

    for (int it = it0; it < it1; ++it) {
      const int x = (it - nq) * TILE + ln.t;  // raw tiles: this thread's position in the list of ring positions and drafts
      // the eight channels of a group in nibble order, values times `scale`
      float sick = 0.f;  // not zero once one of them was an infinity or NaN, which then counts as zero here
      const auto raw_group = [&](const void* row, int kg, bool key, float scale, uint4& o, uint4& l) {
        float4 f0 = make_float4(0.f, 0.f, 0.f, 0.f), f1 = f0;
        if (row) {
          const bool bf = !F32 && x >= nring;
          if (KF == KVQ_Q8G32 && key) {  // words 2 (kg & 1) and + 1 of chunk kg >> 1
            const int c = 64 * ((kg >> 1) & 1) + 32 * (kg & 1) + 2 * (kg >> 2);
            const float2 p0 = load2_in(row, c, bf), p1 = load2_in(row, c + 8, bf), p2 = load2_in(row, c + 16, bf), p3 = load2_in(row, c + 24, bf);
            f0 = make_float4(p0.x, p0.y, p1.x, p1.y);
            f1 = make_float4(p2.x, p2.y, p3.x, p3.y);
          } else {
            f0 = load4_in(row, 8 * kg, bf);
            f1 = load4_in(row, 8 * kg + 4, bf);
          }
        }
        if (!key) {
          float* const f[8] = {&f0.x, &f0.y, &f0.z, &f0.w, &f1.x, &f1.y, &f1.z, &f1.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) sick = fmaf(*f[i], 0.f, sick);
          if (sick != 0.f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) *f[i] = fabsf(*f[i]) < INFINITY ? *f[i] : 0.f;
          }
        }
        if (F32 && !key) {
          f0.x *= scale, f0.y *= scale, f0.z *= scale, f0.w *= scale;
          f1.x *= scale, f1.y *= scale, f1.z *= scale, f1.w *= scale;
        }
        if (!key || KF == KVQ_Q4G32) {  // 0 4 1 5 2 6 3 7
          split2(!F32, f0.x, f1.x, o.x, l.x);
          split2(!F32, f0.y, f1.y, o.y, l.y);
          split2(!F32, f0.z, f1.z, o.z, l.z);
          split2(!F32, f0.w, f1.w, o.w, l.w);
        } else {
          split2(!F32, f0.x, f0.y, o.x, l.x);
          split2(!F32, f0.z, f0.w, o.y, l.y);
          split2(!F32, f1.x, f1.y, o.z, l.z);
          split2(!F32, f1.z, f1.w, o.w, l.w);
        }
      };
      // ---- keys (the previous tile's logits are done: its softmax has read them)
      float nn = raw ? raw_logit : 1.f;  // TQ3: norm of this thread's position
      bool valid = true;
      const uint8_t* rec_sh = smem + SM::R(N);
      if (!raw) {
        valid = checked(page, a.L.n_pages) >= 0;
        if (!valid && it * TILE + (ln.t & 64) < qend && (tid & 63) == 0) atomicOr(a.p.status, KVQ_DEV_BAD_PAGE);
        page = page_of(it + 1, ln.t & 64);
        wait(&kr_bar, kr_phase);
        put_k<KF, P>(lane_addr, ln, rec_sh, cent);
        if (TQ) nn = __half2float(reinterpret_cast<const __half*>(rec_sh + (ln.t >> 5) * Rec<KF>::KH + Rec<KF>::K_MAIN)[ln.t & 31]);
      } else {
        const void* row = raw_row(x, 0);
#pragma unroll 4
        for (int i = 0; i < 16 / P; ++i) {
          const int kg = 16 / P * ln.hf + i;
          uint4 o, l;
          raw_group(row, kg, true, 1.f, o, l);
          tm_st4(lane_addr + 4 * kg, o);
          tm_st4(lane_addr + C::KD / 2 + 4 * kg, l);
        }
      }
      k_done();
      // ---- values, while the logits run (the previous tile's P V must be done with their place)
      wait_pv();
      if (it > it0 && (it - it0) % DRAIN == 0) drain(it - it0 == DRAIN);
      if (!raw) {
        wait(&vr_bar, vr_phase);
        put_v<KF, P>(smem + SM::V, ln, rec_sh, checked(vpage, a.L.n_pages) >= 0 ? qend - it * TILE - 2 * ln.vp : 0);
        vpage = page_of(it + 1, ln.vp & 32);
      } else {
        const void* row = raw_row(x, 1);
#pragma unroll 4
        for (int i = 0; i < 16 / P; ++i) {
          const int kg = 16 / P * ln.hf + i;
          uint4 o, l;
          raw_group(row, kg, false, v_scale, o, l);
          *reinterpret_cast<uint4*>(smem + SM::V + mm_off(8 * kg, ln.t)) = o;
          *reinterpret_cast<uint4*>(smem + SM::V + C::PLANE + mm_off(8 * kg, ln.t)) = l;
        }
      }
      __syncwarp();
      if (lane == 0) bar_arrive(&v_bar);
      // Zero times such a value would be NaN for the rows that do not attend to it; those that do get a weight of NaN instead.
      bool spoilt = false;
      if (raw) {
        sick_sh[ln.hf][ln.t] = sick != 0.f;
        if (part_or(1, WORKERS, sick != 0.f)) {
#pragma unroll
          for (int i = 0; i < P; ++i) spoilt = spoilt || sick_sh[i][ln.t];
        }
      }
      // ---- which of the thread's columns attend to its position: by records a node at depth d reads j <= L + d - W,
      // raw ones the rest, drafts its ancestors and itself
      uint32_t bits = 0xffffffffu;
      if (raw || (it + 1) * TILE > full_end || !valid) {
        const int j = raw ? L - nring + x : it * TILE + ln.t, d = j - L + a.W - 1;  // the deepest node that reads j raw
        bits = 0u;
        if (!raw) {
          if (valid && j < full_end) bits = 0xffffffffu;
          else if (valid && j < L) bits = shallow[grp][KVQ_MAX_TREE - 1] & ~(a.W > 0 ? shallow[grp][min(d, KVQ_MAX_TREE - 1)] : 0u);
        } else if (x < nring) {
          bits = d >= 0 ? shallow[grp][min(d, KVQ_MAX_TREE - 1)] : 0u;
        } else if (x < nraw) {
          bits = below[grp][x - nring];
        }
      }
      constexpr uint32_t ALL = NC == 32 ? 0xffffffffu : (1u << (NC & 31)) - 1;
      const bool all = __all_sync(FULL, (bits & ALL) == ALL && !spoilt);
      // ---- softmax down the thread's columns
      wait(&qk_bar, qk_phase);
      fence_after();
      // CH columns' logits from tensor memory: requested, then waited for and finished less `ref`
      float xs[CH];
      const auto request = [&](int c) { tm_ld(lane_addr + C_S + col0 + c, xs); };
      const auto logits = [&](int c, float (&x)[CH], const float (&ref)[CH]) {
        tm_wait_ld();
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          x[i] = fmaf(xs[i], nn, -ref[i]);
        }
        if (!all) {
#pragma unroll
          for (int i = 0; i < CH; ++i)
            x[i] = !((bits >> (c + i)) & 1) ? -INFINITY : spoilt ? NAN : x[i];
        }
      };
      uint32_t summed = 0;  // by groups of CH columns, warp-uniform: the weights are in the sums
      for (int raises = it == it0 ? 0 : -1;; ++raises) {
        if (raises >= 0) {
          // ---- raise the references of the rows that passed theirs (all of them at first) to the tile's maxima, and
          // rescale what has been summed; then the weights are taken (again)
#pragma unroll 1
          for (int c = 0; c < NC; c += CH) {
            float x[CH];
            const float zero[CH] = {};
            request(c);
            logits(c, x, zero);
#pragma unroll
            for (int i = 0; i < CH; ++i) {
              const int v = __float_as_int(x[i]);
              const int m = __reduce_max_sync(FULL, v ^ ((v >> 31) & 0x7fffffff));
              if (lane == 0) wmax[warp & 3][col0 + c + i] = __int_as_float(m ^ ((m >> 31) & 0x7fffffff));
            }
          }
          part_sync(1, WORKERS);
          if (tid < N) {
            const float top = fmaxf(fmaxf(wmax[0][tid], wmax[1][tid]), fmaxf(wmax[2][tid], wmax[3][tid]));
            const float m0 = mref[tid], m1 = top > m0 + MOST ? top - START : m0;
            fac[tid] = ex2(m0 - m1);
            mref[tid] = m1;
          }
          part_sync(1, WORKERS);
          if (it > it0) {  // (O where it has just been drained is overwritten)
#pragma unroll
            for (int c = 0; c < NC; ++c) l[c] *= fac[col0 + c];
#pragma unroll 1
            for (int c = 0; c < NC; c += 4) {
              float o[4];
              tm_ld(lane_addr + C_O + col0 + c, o);
              tm_wait_ld();
#pragma unroll
              for (int i = 0; i < 4; ++i) o[i] *= fac[col0 + c + i];
              tm_st4(lane_addr + C_O + col0 + c,
                     make_uint4(__float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]), __float_as_uint(o[3])));
            }
            tm_wait_st();
          }
        }
        bool over = false;
        request(0);
#pragma unroll
        for (int c = 0; c < NC; c += CH) {
          float x[CH], ref[CH];
#pragma unroll
          for (int i = 0; i < CH; i += 4) {
            const float4 m = *reinterpret_cast<const float4*>(mref + col0 + c + i);
            ref[i] = m.x, ref[i + 1] = m.y, ref[i + 2] = m.z, ref[i + 3] = m.w;
          }
          logits(c, x, ref);
          if (c + CH < NC) request(c + CH);
          uint32_t ph[CH / 2], pl[CH / 2];
          float top = 0.f;
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            x[i] = ex2(x[i]);
            top = fmaxf(top, x[i]);
          }
#pragma unroll
          for (int i = 0; i < CH / 2; ++i) split2(!F32 && raw, x[2 * i], x[2 * i + 1], ph[i], pl[i]);
          uint8_t* dst = smem + SM::P(N) + mn_off(col0 + c, ln.t, N);
          *reinterpret_cast<uint4*>(dst) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
          *reinterpret_cast<uint4*>(dst + N * TILE * 2) = make_uint4(pl[0], pl[1], pl[2], pl[3]);
          // A weight over 2^MOST (infinity among them) waits for a higher reference, and the columns taken with it wait too.
          // What is over it once the references have moved belongs to rows that are not finite: their columns' own affair.
          const bool high = __any_sync(FULL, top > 32768.f);
          over = over || high;
          if ((!high || raises >= 0) && !((summed >> (c / CH)) & 1)) {
            summed |= 1u << (c / CH);
#pragma unroll
            for (int i = 0; i < CH; ++i) l[c + i] += x[i];
          }
        }
        fence_async_smem();
        fence_before();
        if (tid == 0) leave_sh[it & 1] = gave_up();
        // (one raise puts every weight at or below 2^MOST; only an infinity or NaN is still over it then)
        if (!part_or(1, WORKERS, over) || raises >= 0) break;
      }
      if (leave_sh[it & 1]) {  // (read once, before the barrier above: all workers leave together or none does)
        ok = false;
        break;
      }
      if (tid == 0) bar_arrive(&p_bar);
      pv_pending = true;
    }
    if (!ok) break;
    // ---- the range's part of the unit: reference, sum and O of every row
    wait_pv();
    drain(it1 - it0 <= DRAIN);
    // sums over the lanes; after three exchanges the lanes of one lane & 7 have NC / 8 columns, by its bits in reverse
    halve<NC / 2, 1>(l, lane);
    halve<NC / 4, 2>(l, lane);
    halve<NC / 8, 4>(l, lane);
    const int lc = ((lane & 1) * 4 + (lane & 2) + ((lane >> 2) & 1)) * (NC / 8);
#pragma unroll
    for (int c = 0; c < NC / 8; ++c) {
      float s = l[c];
      s += __shfl_xor_sync(FULL, s, 8);
      s += __shfl_xor_sync(FULL, s, 16);
      if (lane < 8) wmax[warp & 3][col0 + lc + c] = s;
    }
    fence_before();
    if (part_or(1, WORKERS, gave_up())) {
      ok = false;
      break;
    }
    if (tid < N) {
      rec[tid] = mref[tid];
      rec[N + tid] = wmax[0][tid] + wmax[1][tid] + wmax[2][tid] + wmax[3][tid];
    }
  }
  // A CTA that gave up leaves sums that are NaN in the records of its part and of those it did not come to (the merge reads
  // them), and what it still has under way, copies and products, lands before it leaves; the waits are bounded.
  if (warp < WARPS && !ok) {
    for (t = t_part; t < t_end;) {
      const Part w = part_at(t);
      float* rec = record_of(w);
      if (w.it0 < w.it1 && tid < N) {
        rec[tid] = NO_REF;
        rec[N + tid] = NAN;
      }
    }
  }
  __syncthreads();  // (nobody waits any more)
  if (warp == WARPS && gave_up()) {
    if (kr_n) bar_land(&kr_bar, (kr_n - 1) & 1);
    if (vr_n) bar_land(&vr_bar, (vr_n - 1) & 1);
    mma_commit(&end_bar);
    bar_land(&end_bar, 0);
  }
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    tm_free(tmem, TM_COLS);
  }
}

// ------------------------------------------------------------------ 2. merge
// WIDE: a CTA per row, its warps on slices of the row's records; else a warp per row
template <bool WIDE>
__global__ void __launch_bounds__(MERGE_WARPS * 32) tree_merge_kernel(const __grid_constant__ Plan p) {
  __shared__ float part[WIDE ? MERGE_WARPS : 1][2 * D + 2];
  extern __shared__ int pre[];
  const MultiArgs& a = p.a;
  int* lens = pre + a.batch + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) tile_prefix(a, lens, pre, false, [&](int L) { return seq_tiles(a, L); });
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int rows = a.n * a.g;
  const long long idx = WIDE ? blockIdx.x : (long long)blockIdx.x * MERGE_WARPS + warp;
  if (idx >= (long long)(p.n_units / p.rb) * rows) return;
  const int row = (int)(idx % rows), unit = (int)(idx / rows);
  const int h = unit % a.Hkv, b = (unit / a.Hkv) % a.batch, ll = unit / (a.Hkv * a.batch);
  const int u = unit * p.rb + row / p.N, col = row % p.N, node = row / a.g;
  const long long per_layer = (long long)pre[a.batch] * a.Hkv * p.rb, total = per_layer * a.n_layers_call;
  const int tiles = pre[b + 1] - pre[b], nq = (quant_end(lens[b], a.W, a.n) + TILE - 1) / TILE;
  const long long first = ll * per_layer + (long long)pre[b] * a.Hkv * p.rb + (long long)(h * p.rb + row / p.N) * tiles;
  const long long G = min((long long)p.G, total);
  const size_t rec_floats = 2 * p.N + (size_t)D * p.N;
  // the row's parts: first those of the records (o[0]), then those of the raw positions (o[1]), each kind in the order of
  // the ranges; range c holds tile x for c = floor(((x + 1) G - 1) / total)
  float M = NO_REF, l = 0.f, o[2][4] = {};
  const auto owner = [&](long long x) { return (int)quick_div((x + 1) * G - 1, total); };
  const auto add = [&](int kind, int c) {
    const float* rec = p.records + (size_t)(2 * u + kind + c) * rec_floats;
    const float m = rec[col], s = rec[p.N + col];
    const float4 x = *reinterpret_cast<const float4*>(rec + 2 * p.N + (size_t)col * D + 4 * lane);
    const float mn = fmaxf(M, m), f0 = ex2(M - mn), f1 = ex2(m - mn);
    M = mn;
    l = l * f0 + s * f1;
    if (kind) {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[0][e] *= f0;
    }
    o[kind][0] = o[kind][0] * f0 + x.x * f1;
    o[kind][1] = o[kind][1] * f0 + x.y * f1;
    o[kind][2] = o[kind][2] * f0 + x.z * f1;
    o[kind][3] = o[kind][3] * f0 + x.w * f1;
  };
  if (nq > 0) {
    const int c0 = owner(first), c1 = owner(first + nq - 1);
#pragma unroll 4
    for (int c = c0 + (WIDE ? warp : 0); c <= c1; c += WIDE ? MERGE_WARPS : 1) add(0, c);
  }
  if (!WIDE || warp == MERGE_WARPS - 1) {
    int last = -1;
    for (int x = nq; x < tiles; x += RAW_PLACES) {
      const int c = owner(first + x);
      if (c != last) add(1, c);
      last = c;
    }
  }
  if (WIDE) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      part[warp][4 * lane + e] = o[0][e];
      part[warp][D + 4 * lane + e] = o[1][e];
    }
    if (lane == 0) {
      part[warp][2 * D] = M;
      part[warp][2 * D + 1] = l;
    }
    __syncthreads();
    if (warp != 0) return;
    for (int k = 1; k < MERGE_WARPS; ++k) {  // (a warp without parts has weight zero)
      const float m = part[k][2 * D], mn = fmaxf(M, m), f0 = ex2(M - mn), f1 = ex2(m - mn);
      M = mn;
      l = l * f0 + part[k][2 * D + 1] * f1;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[0][e] = o[0][e] * f0 + part[k][4 * lane + e] * f1;
        o[1][e] = o[1][e] * f0 + part[k][D + 4 * lane + e] * f1;
      }
    }
  }
  // is the node there? (its chain of parents, two of them to a lane)
  const int* par = a.parents + (size_t)b * a.n;
  const int par_lo = lane < a.n ? par[lane] : -2, par_hi = lane + 32 < a.n ? par[lane + 32] : -2;
  bool there = true;
  for (int j = node; j >= 0;) {
    const int x = __shfl_sync(FULL, par_lo, j & 31), y = __shfl_sync(FULL, par_hi, j & 31);
    const int q = j < 32 ? x : y;
    there = there && q >= -1 && q < j;
    j = there ? q : -1;
  }
  const float inv = there && l != 0.f ? 1.f / l : 0.f;  // (a sum of NaN, where a range gave up too, makes NaN of the row)
  const __half* sig = a.p.sigv + ((size_t)(a.layer0 + ll) * a.Hkv + h) * D + 4 * lane;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    o[0][e] = there ? o[0][e] * inv : 0.f;
    o[1][e] = there ? o[1][e] * inv : 0.f;
    if (a.sinkhorn) o[0][e] *= __half2float(sig[e]);
  }
  hadamard_warp(o[0][0], o[0][1], o[0][2], o[0][3], lane);
  const float4 sg = *reinterpret_cast<const float4*>(a.p.signs + 4 * lane);
  const float y[4] = {o[0][0] * C_WHT * sg.x + o[1][0], o[0][1] * C_WHT * sg.y + o[1][1], o[0][2] * C_WHT * sg.z + o[1][2],
                      o[0][3] * C_WHT * sg.w + o[1][3]};
  const size_t at = ((((size_t)ll * a.batch + b) * a.Hkv * a.g + (size_t)h * a.g + row % a.g) * a.n + node) * D + 4 * lane;
  if (a.in_bf16) {
    const __nv_bfloat162 y0 = __floats2bfloat162_rn(y[0], y[1]), y1 = __floats2bfloat162_rn(y[2], y[3]);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(y[0], y[1], y[2], y[3]);
  }
}

// ------------------------------------------------------------------ host
// sizes of a call, and its records in scratch (which may be null: sizes only); returns the scratch bytes
template <int KF>
size_t make_plan(const MultiArgs& a, int sms, Plan* p) {
  const int rows = a.n * a.g;
  p->a = a;
  const bool few = rows <= FEW_ROWS;
  const int most = few ? FEW_ROWS : KF == KVQ_TQ3_QJL ? TQ_ROWS : MAX_ROWS, step = few ? 16 : 32;
  p->rb = (rows + most - 1) / most;
  p->N = ((rows + p->rb - 1) / p->rb + step - 1) / step * step;
  p->n_units = a.n_layers_call * a.batch * a.Hkv * p->rb;
  p->G = sms * (few ? 2 : 1);
  p->records = reinterpret_cast<float*>(a.scratch);
  return (size_t)(2 * p->n_units + p->G) * (2 * p->N + D * p->N) * 4;
}

template <int KF, bool F32>
cudaError_t launch(const MultiArgs& a, int sms, cudaStream_t s) {
  Plan p;
  make_plan<KF>(a, sms, &p);
  const long long out_rows = (long long)(p.n_units / p.rb) * a.n * a.g;
  if (out_rows > 0x7fffffffLL) return cudaErrorInvalidValue;
  const size_t pre = (size_t)(2 * a.batch + 1) * 4, smem = Smem<KF>::total(p.N) + pre;
  const dim3 grid((unsigned)p.G);
  cudaError_t e = cudaErrorInvalidValue;
  if (p.N == 16) e = go<tree_kernel<KF, 8, F32, 2>>(grid, 288, smem, false, s, p);
  if (p.N == 32) e = go<tree_kernel<KF, 8, F32, 4>>(grid, 544, smem, false, s, p);
  if (p.N == 64) e = go<tree_kernel<KF, 16, F32, 4>>(grid, 544, smem, false, s, p);
  if constexpr (KF != KVQ_TQ3_QJL) {
    if (p.N == 96) e = go<tree_kernel<KF, 24, F32, 4>>(grid, 544, smem, false, s, p);
  }
  if (e != cudaSuccess) return e;
  // Many records a row (few units over all CTAs): a CTA per row, else a warp per row.  16 nodes at 32K (8 units over 152 CTAs)
  // 60 us, by warps 67; 64 nodes over 4 x 9001 (64 units) by warps 118, by CTAs 140.
  if (p.G > 8 * p.n_units) return go<tree_merge_kernel<true>>(dim3((unsigned)out_rows), MERGE_WARPS * 32, pre, true, s, p);
  return go<tree_merge_kernel<false>>(dim3((unsigned)((out_rows + MERGE_WARPS - 1) / MERGE_WARPS)), MERGE_WARPS * 32, pre, true, s, p);
}

}  // namespace tree
}  // namespace kvq

// Attention of a prefill chunk over a KVQ_Q8B32 cache: query t of sequence b attends to positions [0, pos[b] + t], the
// newest `window` raw, the rest through the records (what its own single-token step would read), after the chunk's append.
//
//   o = sum_j w_j v_j / sum_j w_j,  w_j = 2^(l_j - m),  l_j = log2(e) / sqrt(128) q.k_j
//   recorded j:  q.k_j = d_k (q~ . c_j), v_j = d_v H c'_j ...: the codes c are the operands, the two scales of a block of 32
//   positions never meet them: logits are multiplied by d_k, weights by d_v before they go to P V
//
// The products run on the 5th-generation tensor cores (tcgen05.mma, kind::f16, fp32 accumulators in tensor memory).  Codes
// are exact in one fp16 plane, so a product takes two passes (hi and lo of the queries, or of the weights: 22 bits) where
// formats whose dequantised values need two planes take three.
//  * Work: a row tile is 128 (query, head) rows of one (layer, sequence, kv-head); its positions go in tiles of 64 recorded
//    ones (a page), then of raw ones.  The call's tiles form one list that is cut into equal ranges, one per CTA (one CTA
//    an SM), whatever the chunk's and the contexts' lengths: a row tile that a cut divides leaves partial results, which a
//    second launch joins in order.  Without the cut 1024 tokens of 24 heads are 192 row tiles on 152 SMs, and three short
//    turns keep 6 of them busy.
//  * A tile's stored order is the operands' order up to a permutation of channels (keys) or positions (values), which
//    queries and weights follow: 16 stored bytes become two 16-byte operand rows by byte permutes, nothing is transposed.
//  * Raw tiles are taken as they are, not rotated: queries are also kept unrotated (in shared memory), and the output
//    accumulator, a row per thread in registers, is rotated back once, before the first raw tile.
//  * Warps: two groups of four soften alternate tiles (a row a thread: lanes of tensor memory), each with a reference, a sum
//    and an output accumulator of its own, joined at the end; four warps turn bytes into operands; one issues the logits'
//    products, one those of the values.  Every tile's P V starts from zero and is added to the registers: the tensor
//    cores' truncating sums stay within a tile.
//  * Queries, raw keys and raw values are scaled by powers of two, each vector by its own, and weights against the largest
//    scale of values so far: fp16 parts keep their bits at any magnitude.
//  * Every wait is bounded; one that runs out flags the status word and the CTA leaves as a whole.
#include <cfloat>
#include <cstddef>

#include "tc.cuh"

namespace kvq {

namespace {

using namespace tc;

constexpr int ROWS = 128;            // rows of a row tile = MMA M = lanes of tensor memory
constexpr int NT = 64;               // recorded positions of a tile = a page
constexpr int NS = 4;                // operand stages
constexpr int N_SOFT = 8;            // softmax warps, two groups
constexpr int DQ0 = 8, N_DQ = 4;     // operand warps
constexpr int S_WARP = 12, PV_WARP = 13, NEXT_WARP = 14;
constexpr int THREADS = 512;
constexpr int SOFT_REGS = 184, OTHER_REGS = 72;  // 256 x (184 + 72) = 512 x 128, what the block is launched with
constexpr uint32_t TMEM_COLS = 512, C_QHI = 0, C_QLO = 64, C_S = 128, C_O = 256;  // Q hi | lo | two S or P | two O
constexpr uint32_t V_OFF = 16384, STAGE = 32768;        // a stage: keys, values; planes of 64 x 128 (or two of 32 x 128) fp16
constexpr uint32_t LO_PLANE = 8192;                     // raw tiles of float caches: from hi to lo
constexpr uint32_t Q_STRIDE = 2 * D * 2 + 16;           // query staging row: hi, lo, pad
constexpr uint32_t QR_LEAD = ROWS * 16 + 16;            // unrotated queries: from one 8 channels to the next
constexpr uint32_t QR_PLANE = 16 * QR_LEAD;
constexpr uint32_t QR_OFF = NS * STAGE, SMEM = QR_OFF + 2 * QR_PLANE;
constexpr uint32_t O_STRIDE = (D + 4) * 4;
static_assert(ROWS * Q_STRIDE <= NS * STAGE && 2 * ROWS * O_STRIDE <= SMEM, "what borrows the stages");
constexpr int MAX_RAW = ((MAX_WINDOW + ROWS) / 64 + 1) * 64;  // raw positions of a row tile, in whole tiles
constexpr float BOOST = 9.f;         // log2 of the largest weight over its reference when that is set
constexpr float RAISE_AT = 4.f;      // ... and how much further it may grow before the reference follows
constexpr long long K0 = 192;        // a row tile's fixed cost, in positions
constexpr long long MIN_SHARE = 512; // positions that a CTA takes at least
constexpr unsigned long long WAIT_NS = 1000000000ull;
constexpr int REC = ROWS * D + 2 * ROWS;  // floats of a partial result: O, m, l

// place of channel c (position c of a tile) along K, in the order in which 16-byte chunks hold codes; what is at a place
__host__ __device__ constexpr int place_of(int c) {
  return (c & ~31) | (((c >> 1) & 3) << 3) | (((c >> 4) & 1) << 2) | (((c >> 3) & 1) << 1) | (c & 1);
}
__host__ __device__ constexpr int at_place(int k) {
  return (k & ~31) | (((k >> 2) & 1) << 4) | (((k >> 1) & 1) << 3) | (((k >> 3) & 3) << 1) | (k & 1);
}
// (row, k) of a K-major operand whose groups of 8 k are `lead` bytes apart
__device__ __forceinline__ uint32_t km(int row, int k, uint32_t lead) {
  return (uint32_t)(k >> 3) * lead + (uint32_t)((row >> 3) * 128 + (row & 7) * 16 + (k & 7) * 2);
}

// ------------------------------------------------------------------ the list of tiles
struct Unit {
  int b, x, hl;           // sequence, row tile, (layer, kv-head)
  long long start, cost;  // on the cost line
};

// Costs in positions: row tile x of a sequence at p0 counts p0 + (x + 1) qpt + K0, about the positions it visits.  The line
// goes through sequences, row tiles, (layer, kv-head) pairs; cut c is at total * c / n.
struct Work {
  int B, T, qpt, nx, HL, n;
  const int* p0;           // per sequence; -1: not part of the call
  const long long* pre;    // cost before each sequence, [B + 1]
  __device__ __forceinline__ long long cost(int b, int x) const { return p0[b] + (long long)(x + 1) * qpt + K0; }
  __device__ __forceinline__ long long upto(int b, int x) const {
    return (x * (p0[b] + K0) + (long long)qpt * x * (x + 1) / 2) * HL;
  }
  __device__ __forceinline__ long long total() const { return pre[B]; }
  __device__ __forceinline__ long long cut(int c) const { return total() / n * c + total() % n * c / n; }
  __device__ Unit find(long long y) const {
    Unit u;
    int lo = 0, hi = B - 1;
    while (lo < hi) {  // the last sequence that starts at or before y (those without work start where the next does)
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= y) lo = mid;
      else hi = mid - 1;
    }
    u.b = lo;
    const long long r = y - pre[lo];
    int xl = 0, xh = nx - 1;
    while (xl < xh) {
      const int mid = (xl + xh + 1) >> 1;
      if (upto(lo, mid) <= r) xl = mid;
      else xh = mid - 1;
    }
    u.x = xl;
    u.cost = cost(lo, xl);
    const long long r2 = r - upto(lo, xl);
    u.hl = (int)(r2 / u.cost);
    u.start = y - r2 % u.cost;
    return u;
  }
};
// warp 0: positions and prefix of the sequences' costs into shared memory
__device__ void plan(const PrefillArgs& a, Work& w, int* p0, long long* pre, int ctas) {
  w.B = a.batch;
  w.T = a.T;
  w.qpt = ROWS / a.g;
  w.nx = (a.T + w.qpt - 1) / w.qpt;
  w.HL = a.Hkv * a.n_layers_call;
  w.p0 = p0;
  w.pre = pre;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, per = (a.batch + 31) / 32;
    const int b0 = min(a.batch, lane * per), b1 = min(a.batch, b0 + per);
    long long s = 0;
    for (int b = b0; b < b1; ++b) {
      const int p = a.pos[b];
      p0[b] = p >= 0 && (long long)p + a.T <= a.max_seq_len ? p : -1;
      if (p0[b] >= 0) s += w.upto(b, w.nx);
    }
    long long incl = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(FULL, incl, o);
      if (lane >= o) incl += y;
    }
    long long run = incl - s;
    for (int b = b0; b < b1; ++b) {
      pre[b] = run;
      if (p0[b] >= 0) run += w.upto(b, w.nx);
    }
    if (lane == 31) pre[a.batch] = incl;
  }
  __syncthreads();
  w.n = (int)max(1LL, min((long long)ctas, w.total() / MIN_SHARE));
}

// A row tile: its queries' positions, the recorded positions [0, qend) that any of them reads, the raw ones from rlo
struct Tiles {
  int t0, nq, Pmin, Pmax, qend, nqt, rlo, n;
  Tiles() = default;
  __device__ Tiles(const Work& w, const Unit& u, int W, int raw_nt) {
    t0 = u.x * w.qpt;
    nq = min(w.qpt, w.T - t0);
    Pmin = w.p0[u.b] + t0;
    Pmax = Pmin + nq - 1;
    qend = max(0, Pmax - W + 1);
    nqt = (qend + NT - 1) / NT;
    rlo = max(0, Pmin - W + 1);
    n = nqt + (Pmax - rlo) / raw_nt + 1;
  }
  // tiles before offset `off` of the row tile's stretch of the cost line
  __device__ __forceinline__ int before(long long off) const {
    return off <= K0 ? 0 : (int)min((long long)n, (off - K0 + NT - 1) / NT);
  }
};

// A CTA's stretch of one row tile: tiles ta .. tb - 1 of it, whole or to be joined with others
struct Stretch {
  int b, hl, unit, layer, h;  // unit: (layer of the call, sequence, kv-head)
  int p0, ta, tb, rec;        // rec: -1: the row tile as a whole
  Tiles tl;
  long long next;             // where on the cost line the CTA goes on
};

// ------------------------------------------------------------------ PTX helpers (besides tc.cuh's)
__device__ __forceinline__ void tm_ld32(uint32_t taddr, float (&f)[32]) {
  uint32_t r[32];
#define KVQ_R8(o, i) o(r[i + 0]), o(r[i + 1]), o(r[i + 2]), o(r[i + 3]), o(r[i + 4]), o(r[i + 5]), o(r[i + 6]), o(r[i + 7])
#define KVQ_OUT(x) "=r"(x)
#define KVQ_IN(x) "r"(x)
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : KVQ_R8(KVQ_OUT, 0), KVQ_R8(KVQ_OUT, 8), KVQ_R8(KVQ_OUT, 16), KVQ_R8(KVQ_OUT, 24)
      : "r"(taddr));
  tm_wait_ld();
#pragma unroll
  for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tm_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      KVQ_R8(KVQ_IN, 0), KVQ_R8(KVQ_IN, 8), KVQ_R8(KVQ_IN, 16), KVQ_R8(KVQ_IN, 24)
      : "memory");
}
// four columns at each of taddr, + 8, + 16, + 24
__device__ __forceinline__ void tm_ld4x4(uint32_t taddr, float (&f)[16]) {
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    uint32_t r[4];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr + 8 * n));
#pragma unroll
    for (int e = 0; e < 4; ++e) f[4 * n + e] = __uint_as_float(r[e]);
  }
  tm_wait_ld();
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// A warp's bounded wait.  false: this CTA gives up (a wait elsewhere ran out, or this one: flagged).
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* gone, unsigned* status) {
  bool ok = bar_try(bar, parity);
  if (!ok) {
    const unsigned long long t0 = gtimer();
    while (!(ok = bar_sleep(bar, parity))) {
      if (*gone) break;
      if (gtimer() - t0 > WAIT_NS) {
        atomicOr(status, KVQ_DEV_TIMEOUT);
        *gone = 1;
        break;
      }
    }
  }
  return __all_sync(FULL, ok);
}
__device__ __forceinline__ float warp_max(float m) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
  return m;
}

template <bool BF16>
struct Kernel {
  static constexpr int RNT = BF16 ? 64 : 32;  // raw positions of a tile: one plane of a bf16 cache's, hi and lo of a float one's
  static constexpr uint32_t ID_S = idesc(ROWS, NT, false, false), ID_SR = idesc(ROWS, RNT, false, false);
  static constexpr uint32_t ID_O = idesc(ROWS, D, false, false), ID_OR = idesc(ROWS, D, false, true);

  // shared by the CTA, besides the stages
  struct Shared {
    uint64_t kfull[NS], kempty[NS], vfull[NS], vempty[NS], sfull[2], pfull[2], pvdone[2], done[2];
    uint32_t tmem;
    int gone;
    float qscale[ROWS], qraw[ROWS];        // powers of two that the queries were divided by
    float m[2][ROWS], l[2][ROWS];          // both groups' references and sums, at the end
    float2 scale[8][2];                    // (keys', values') of a tile's two blocks
    float rawk[MAX_RAW], rawv[MAX_RAW];    // the raw vectors' powers of two
    alignas(16) float signs[D];            // (read four at a time)
    int p0[MAX_BATCH];
    long long pre[MAX_BATCH + 1];
    Stretch at[2];                         // this stretch and the next
  };

  static_assert(offsetof(Shared, signs) % 16 == 0 && alignof(Shared) % 16 == 0, "read as float4");

  const PrefillArgs& a;
  Shared& sh;
  uint8_t* smem;
  Work& work;
  float* recs;
  int warp, lane;
  uint32_t tmem;
  int gt = 0;  // tiles so far

  __device__ Kernel(const PrefillArgs& args, Shared& s, uint8_t* sm, Work& w, float* r) : a(args), sh(s), smem(sm), work(w), recs(r) {
    warp = threadIdx.x >> 5;
    lane = threadIdx.x & 31;
  }
  __device__ __forceinline__ bool held(uint64_t* bar, uint32_t parity) { return wait(bar, parity, &sh.gone, a.p.status); }
  __device__ __forceinline__ void sync_all() { part_sync(1, THREADS); }

  // the first stretch with tiles from y on (lo: where the CTA began)
  __device__ void locate(long long y, long long lo, long long hi, Stretch& st) const {
    st.tb = -1;
    while (y < hi) {
      const Unit u = work.find(y);
      const Tiles tl(work, u, a.W, RNT);
      st.ta = tl.before(y - u.start);
      st.tb = hi >= u.start + u.cost ? tl.n : tl.before(hi - u.start);
      st.rec = st.ta == 0 && st.tb == tl.n ? -1 : 2 * (int)blockIdx.x + (y == lo ? 0 : 1);
      st.b = u.b;
      st.hl = u.hl;
      st.h = u.hl % a.Hkv;
      st.layer = a.layer0 + u.hl / a.Hkv;
      st.unit = ((u.hl / a.Hkv) * a.batch + u.b) * a.Hkv + st.h;
      st.p0 = work.p0[u.b];
      st.tl = tl;
      y = st.next = u.start + u.cost;
      if (st.ta < st.tb) return;
      st.tb = -1;
    }
  }

  // ---------------------------------------------------------------- queries
  // rows warp, warp + 16, ...: unrotated (scaled) hi and lo to their operand, rotated ones to the staging rows
  __device__ void queries(const Stretch& u) {
    const Tiles& tl = u.tl;
    const int g = a.g, h = u.h;
    const size_t head0 = (size_t)u.unit * g;
    const float4 sg = *reinterpret_cast<const float4*>(a.p.signs + 4 * lane);
    float4 sk = make_float4(1.f, 1.f, 1.f, 1.f);
    if (a.sinkhorn) {
      const __half* sig = a.p.sigk + ((size_t)u.layer * a.Hkv + h) * D + 4 * lane;
      sk = make_float4(__half2float(sig[0]), __half2float(sig[1]), __half2float(sig[2]), __half2float(sig[3]));
    }
    const int nrows = tl.nq * g;
#pragma unroll 1
    for (int row = warp; row < ROWS; row += THREADS / 32) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < nrows) x = load4_in(a.q, ((head0 + row % g) * a.T + tl.t0 + row / g) * D + 4 * lane, a.in_bf16);
      {
        const float z[4] = {x.x * LOGIT_SCALE, x.y * LOGIT_SCALE, x.z * LOGIT_SCALE, x.w * LOGIT_SCALE};
        float inv;
        const float s2 = pow2_of(warp_max(fmaxf(fmaxf(fabsf(z[0]), fabsf(z[1])), fmaxf(fabsf(z[2]), fabsf(z[3])))), inv);
        if (lane == 0) sh.qraw[row] = s2;
        uint2 hv, lv;
        split2(z[0] * inv, z[1] * inv, hv.x, lv.x);
        split2(z[2] * inv, z[3] * inv, hv.y, lv.y);
        uint8_t* at = smem + QR_OFF + km(row, 4 * lane, QR_LEAD);
        *reinterpret_cast<uint2*>(at) = hv;
        *reinterpret_cast<uint2*>(at + QR_PLANE) = lv;
      }
      float y0 = x.x * sg.x, y1 = x.y * sg.y, y2 = x.z * sg.z, y3 = x.w * sg.w;
      hadamard_warp(y0, y1, y2, y3, lane);
      const float sc = C_WHT * LOGIT_SCALE;
      y0 *= sc * sk.x;
      y1 *= sc * sk.y;
      y2 *= sc * sk.z;
      y3 *= sc * sk.w;
      float inv;
      const float s2 = pow2_of(warp_max(fmaxf(fmaxf(fabsf(y0), fabsf(y1)), fmaxf(fabsf(y2), fabsf(y3)))), inv);
      if (lane == 0) sh.qscale[row] = s2;
      uint32_t h0, l0, h1, l1;
      split2(y0 * inv, y1 * inv, h0, l0);
      split2(y2 * inv, y3 * inv, h1, l1);
      uint8_t* st = smem + (size_t)row * Q_STRIDE;
      const int pa = 2 * place_of(4 * lane), pb = 2 * place_of(4 * lane + 2);
      *reinterpret_cast<uint32_t*>(st + pa) = h0;
      *reinterpret_cast<uint32_t*>(st + pb) = h1;
      *reinterpret_cast<uint32_t*>(st + 2 * D + pa) = l0;
      *reinterpret_cast<uint32_t*>(st + 2 * D + pb) = l1;
    }
    fence_async_smem();
  }
  // this thread's staging row to its lane of tensor memory (softmax warps: the first group hi, the second lo)
  __device__ void queries_to_tmem() {
    const int part = warp >> 2, row = 32 * (warp & 3) + lane;
    const uint32_t addr = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (part ? C_QLO : C_QHI);
    const uint8_t* st = smem + (size_t)row * Q_STRIDE + part * 2 * D;
#pragma unroll
    for (int c0 = 0; c0 < 64; c0 += 32) {
      uint32_t r[32];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 v = *reinterpret_cast<const uint4*>(st + 4 * c0 + 16 * i);
        r[4 * i] = v.x;
        r[4 * i + 1] = v.y;
        r[4 * i + 2] = v.z;
        r[4 * i + 3] = v.w;
      }
      tm_st32(addr + c0, r);
    }
    tm_wait_st();
  }

  // ---------------------------------------------------------------- the products' issue
  __device__ void issue_logits(const Stretch& u) {
    const Tiles& tl = u.tl;
    const uint32_t base = smem_u32(smem);
    for (int it = u.ta; it < u.tb; ++it, ++gt) {
      const int s = gt % NS, bb = gt & 1;
      // the stage's keys; the buffer is free once the values' products of two tiles before have read its weights
      if (!held(&sh.kfull[s], (gt / NS) & 1)) return;
      if (gt >= 2 && !held(&sh.pvdone[bb], ((gt - 2) >> 1) & 1)) return;
      fence_after();
      const uint32_t dS = tmem + C_S + NT * bb;
      if (it < tl.nqt) {
        uint64_t k = sdesc(base + s * STAGE, 1024, 128);
        uint32_t q = tmem + C_QHI;
#pragma unroll 1
        for (int ks = 0; ks < D / 16; ++ks, k += 128, q += 8) {
          mma_ts(dS, q, k, ID_S, ks > 0);
          mma_ts(dS, q + (C_QLO - C_QHI), k, ID_S, 1);
        }
      } else {
        uint64_t k = sdesc(base + s * STAGE, RNT * 16, 128), q = sdesc(base + QR_OFF, QR_LEAD, 128);
#pragma unroll 1
        for (int ks = 0; ks < D / 16; ++ks, k += RNT * 2, q += 2 * QR_LEAD / 16) {
          mma_ss(dS, q, k, ID_SR, ks > 0);
          mma_ss(dS, q + QR_PLANE / 16, k, ID_SR, 1);
          if (!BF16) mma_ss(dS, q, k + LO_PLANE / 16, ID_SR, 1);
        }
      }
      mma_commit(&sh.sfull[bb]);
      mma_commit(&sh.kempty[s]);
    }
  }
  __device__ void issue_values(const Stretch& u) {
    const Tiles& tl = u.tl;
    const uint32_t base = smem_u32(smem);
    for (int it = u.ta; it < u.tb; ++it, ++gt) {
      const int s = gt % NS, bb = gt & 1;
      if (!held(&sh.pfull[bb], (gt >> 1) & 1) || !held(&sh.vfull[s], (gt / NS) & 1)) return;
      fence_after();
      uint64_t v = sdesc(base + s * STAGE + V_OFF, 2048, 128);
      uint32_t p = tmem + C_S + NT * bb;
      const uint32_t dO = tmem + C_O + D * bb;
      if (it < tl.nqt) {
#pragma unroll 1
        for (int ks = 0; ks < NT / 16; ++ks, v += 256, p += 16) {
          mma_ts(dO, p + 8, v, ID_O, ks > 0);
          mma_ts(dO, p, v, ID_O, 1);
        }
      } else {
#pragma unroll 1
        for (int ks = 0; ks < RNT / 16; ++ks, v += 256, p += 16) {
          mma_ts(dO, p + 8, v, ID_OR, ks > 0);
          if (!BF16) mma_ts(dO, p, v + LO_PLANE / 16, ID_OR, 1);
          mma_ts(dO, p, v, ID_OR, 1);
        }
      }
      mma_commit(&sh.vempty[s]);
      mma_commit(&sh.pvdone[bb]);
    }
  }

  // ---------------------------------------------------------------- operands
  // Lane (r, i) = (lane & 7, lane >> 3): the eight lanes of a store phase write eight rows of one core matrix.
  __device__ void operands(const Stretch& u) {
    const Tiles& tl = u.tl;
    const int ta = u.ta, tb = u.tb;
    const int dw = warp - DQ0, r = lane & 7, i = lane >> 3, h = u.h;
    const int32_t* bt = a.block_table + (size_t)u.b * a.max_pages_per_seq;
    const uint8_t* pages = a.p.pages + ((size_t)u.layer * a.L.n_pages * a.Hkv + h) * a.L.page_bytes;
    const size_t page_step = (size_t)a.Hkv * a.L.page_bytes;
    const int last_q = min(tb, tl.nqt);
    uint4 kw[4], vw[4];
    float2 sc = make_float2(0.f, 0.f);
    auto page_of = [&](int it) { return it < last_q ? __ldg(bt + it) : 0; };
    auto load = [&](int it, int phys, bool keys, uint4 (&w)[4]) {
      // chunk dw + 4 (q & 1) of block q >> 1
#pragma unroll
      for (int q = 0; q < 4; ++q) w[q] = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
      if (keys) sc = make_float2(0.f, 0.f);
      if (it >= last_q || phys < 0 || phys >= a.L.n_pages) return;
      const uint8_t* at = pages + phys * page_step + (keys ? 0 : 4096) + dw * 512 + (r * 4 + i) * 16;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (it * NT + HALF * (q >> 1) < tl.qend)
          w[q] = __ldg(reinterpret_cast<const uint4*>(at + (size_t)(q >> 1) * a.L.half_bytes + (q & 1) * 2048));
      if (keys && dw == 0 && lane < 2 && it * NT + HALF * lane < tl.qend)
        sc = __ldg(reinterpret_cast<const float2*>(pages + phys * page_step + (size_t)lane * a.L.half_bytes + a.L.off_kmeta));
    };
    int phys = page_of(ta), next = page_of(ta + 1);
    load(ta, phys, true, kw);
    load(ta, phys, false, vw);
    for (int it = ta; it < tb; ++it, ++gt) {
      const int s = gt % NS;
      const uint32_t before = ((gt / NS) & 1) ^ 1;  // phase of the stage's previous use
      uint8_t* kp = smem + s * STAGE;
      uint8_t* vp = kp + V_OFF;
      if (gt >= NS && !held(&sh.kempty[s], before)) return;
      if (it < tl.nqt) {
        if ((phys < 0 || phys >= a.L.n_pages) && dw == 0 && lane == 0) atomicOr(a.p.status, KVQ_DEV_BAD_PAGE);
        phys = next;
        next = page_of(it + 2);
        if (dw == 0 && lane < 2) sh.scale[gt & 7][lane] = sc;
        // chunk 4 mt + p (p = dw, mt = q & 1): tokens 16 mt + r and + 8, channels of K-group 4 p + i
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t o = km(32 * (q >> 1) + 16 * (q & 1) + r, 8 * (4 * dw + i), 1024);
          *reinterpret_cast<uint4*>(kp + o) = make_uint4(codes_lo(kw[q].x), codes_lo(kw[q].y), codes_lo(kw[q].z), codes_lo(kw[q].w));
          *reinterpret_cast<uint4*>(kp + o + 128) = make_uint4(codes_hi(kw[q].x), codes_hi(kw[q].y), codes_hi(kw[q].z), codes_hi(kw[q].w));
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(&sh.kfull[s]);
        load(it + 1, phys, true, kw);
        if (gt >= NS && !held(&sh.vempty[s], before)) return;
        // chunk j = dw + 4 (q & 1): channels 16 j + r and + 8, positions of K-group 4 (q >> 1) + i
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t o = km(16 * (dw + 4 * (q & 1)) + r, 8 * (4 * (q >> 1) + i), 2048);
          *reinterpret_cast<uint4*>(vp + o) = make_uint4(codes_lo(vw[q].x), codes_lo(vw[q].y), codes_lo(vw[q].z), codes_lo(vw[q].w));
          *reinterpret_cast<uint4*>(vp + o + 128) = make_uint4(codes_hi(vw[q].x), codes_hi(vw[q].y), codes_hi(vw[q].z), codes_hi(vw[q].w));
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(&sh.vfull[s]);
        load(it + 1, phys, false, vw);
      } else {
        const int j0 = tl.rlo + (it - tl.nqt) * RNT;
        raw(u, j0, j0 - tl.rlo, false, kp);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(&sh.kfull[s]);
        if (gt >= NS && !held(&sh.vempty[s], before)) return;
        raw(u, j0, j0 - tl.rlo, true, vp);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(&sh.vfull[s]);
      }
    }
  }
  // raw keys (K-major) or values (N-major: rows are positions too) of positions j0 .. j0 + RNT - 1 as operand planes, each
  // vector over its power of two.  A bf16 vector's elements that its fp16 plane does not hold exactly are 2^-14 of the
  // largest or smaller and off by 2^-25 of it at most.
  __device__ void raw(const Stretch& u, int j0, int slot0, bool values, uint8_t* plane) {
    const int dw = warp - DQ0, r = lane & 7, i = lane >> 3;
    const int p0 = u.p0;
    const size_t unit = u.unit;
    const void* chunk = values ? a.v : a.k;
    const float* old = values ? a.snap_v : a.snap_k;
#pragma unroll 1
    for (int t = 8 * dw + r; t < RNT; t += 8 * N_DQ) {
      const int j = j0 + t;
      const bool here = j <= u.tl.Pmax;
      const size_t off = j < p0 ? (unit * a.W + j % a.W) * D : (unit * a.T + (j - p0)) * D;
      const void* src = j < p0 ? (const void*)old : chunk;
      const int bf16 = j < p0 ? 0 : a.in_bf16;
      auto load8 = [&](int q, float (&x)[8]) {  // channels 8 (4 q + i) ..
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const float4 f = here ? load4_in(src, off + 8 * (4 * q + i) + e, bf16) : make_float4(0.f, 0.f, 0.f, 0.f);
          x[e] = f.x;
          x[e + 1] = f.y;
          x[e + 2] = f.z;
          x[e + 3] = f.w;
        }
      };
      float m = 0.f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float x[8];
        load8(q, x);
#pragma unroll
        for (int e = 0; e < 8; e += 2) m = max3(m, fabsf(x[e]), fabsf(x[e + 1]));
      }
      m = fmaxf(m, __shfl_xor_sync(FULL, m, 8));
      m = fmaxf(m, __shfl_xor_sync(FULL, m, 16));
      float inv;
      const float s2 = pow2_of(m, inv);
      if (i == 0) (values ? sh.rawv : sh.rawk)[slot0 + t] = here ? s2 : 0.f;
#pragma unroll 2
      for (int q = 0; q < 4; ++q) {
        float x[8];
        load8(q, x);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split2(x[2 * e] * inv, x[2 * e + 1] * inv, hi[e], lo[e]);
        const int kg = 4 * q + i;
        const uint32_t o = values ? (uint32_t)((t >> 3) * 2048 + kg * 128 + (t & 7) * 16) : km(t, 8 * kg, RNT * 16);
        *reinterpret_cast<uint4*>(plane + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if (!BF16) *reinterpret_cast<uint4*>(plane + LO_PLANE + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
  }

  // ---------------------------------------------------------------- softmax
  struct Row {
    float acc[D];  // sum of weights times values over vref, of this group's tiles
    float m, l;    // the weights' reference and their sum
    float vref, rvref;
  };
  // acc += this group's last P V
  __device__ __forceinline__ void drain(Row& w, uint32_t addr) {
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += 32) {
      float o[32];
      tm_ld32(addr + c0, o);
#pragma unroll
      for (int i = 0; i < 32; i += 2) add2(w.acc[c0 + i], w.acc[c0 + i + 1], o[i], o[i + 1]);
    }
  }
  __device__ __forceinline__ void rescale(Row& w, float f) {
#pragma unroll
    for (int i = 0; i < D; i += 2) mul2(w.acc[i], w.acc[i + 1], f, f);
  }
  // a larger logit or a larger scale of values than the references allow for
  __device__ __forceinline__ void follow(Row& w, float mx, float vmax) {
    float f = 1.f;
    if (mx > w.m + (BOOST + RAISE_AT)) {
      const float mnew = mx - BOOST;
      f = w.m == -INFINITY ? 0.f : ex2(w.m - mnew);
      w.l *= f;
      w.m = mnew;
    }
    if (vmax > 4.f * w.vref) {
      float inv;
      const float vnew = pow2_of(vmax, inv);
      f *= w.vref * inv;
      w.vref = vnew;
      w.rvref = inv;
    }
    if (__any_sync(FULL, f != 1.f)) rescale(w, f);
  }
  // the accumulator from the values' quantised space to the heads': s . (c H (sigma . y))
  __device__ __forceinline__ void to_heads(Row& w, const Stretch& u) {
    if (a.sinkhorn) {
      const __half2* sig = reinterpret_cast<const __half2*>(a.p.sigv + ((size_t)u.layer * a.Hkv + u.h) * D);
#pragma unroll
      for (int i = 0; i < D; i += 2) {
        const float2 s = __half22float2(__ldg(sig + i / 2));
        mul2(w.acc[i], w.acc[i + 1], s.x, s.y);
      }
    }
#pragma unroll
    for (int i = 0; i < D; i += 2) {
      const float p = w.acc[i], q = w.acc[i + 1];
      w.acc[i] = p + q;
      w.acc[i + 1] = p - q;
    }
#pragma unroll
    for (int hs = 2; hs < D; hs <<= 1) {
#pragma unroll
      for (int i = 0; i < D; i += 2) {
        if (i & hs) continue;
        bfly2(w.acc[i], w.acc[i + 1], w.acc[i + hs], w.acc[i + hs + 1]);
      }
    }
#pragma unroll
    for (int i = 0; i < D; i += 4) {
      const float4 s = *reinterpret_cast<const float4*>(sh.signs + i);
      mul2(w.acc[i], w.acc[i + 1], C_WHT * s.x, C_WHT * s.y);
      mul2(w.acc[i + 2], w.acc[i + 3], C_WHT * s.z, C_WHT * s.w);
    }
  }
  // a tile of recorded positions; MASKED: some row does not attend to all of them
  template <bool MASKED>
  __device__ __forceinline__ void soften(Row& w, uint32_t sa, const float (&dk)[2], const float (&dv)[2], int j0, int hi) {
    float mx = -INFINITY;
#pragma unroll
    for (int c0 = 0; c0 < NT; c0 += 32) {
      float v[32];
      tm_ld32(sa + c0, v);
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < 32; i += 2)
        m = MASKED ? max3(m, j0 + c0 + i <= hi ? v[i] : -INFINITY, j0 + c0 + i + 1 <= hi ? v[i + 1] : -INFINITY) : max3(m, v[i], v[i + 1]);
      if (!MASKED || j0 + c0 <= hi) mx = fmaxf(mx, m * dk[c0 >> 5]);
    }
    follow(w, mx, fmaxf(dv[0], dv[1]));
    const float m0 = w.m == -INFINITY ? 0.f : w.m;
    // K-step by K-step of P V: the first of a block needs columns 8 n .. + 3, the second 8 n + 4 .. + 7, so the first one's
    // weights wait until the second one's logits are read
#pragma unroll
    for (int c0 = 0; c0 < NT; c0 += 32) {
      const float k = dk[c0 >> 5], f = dv[c0 >> 5] * w.rvref;
      float s0 = 0.f, s1 = 0.f;
      uint32_t pw[32];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float v[16];  // v[4 n + e]: column 8 n + 4 half + e
        tm_ld4x4(sa + c0 + 4 * half, v);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const int c = j0 + c0 + 8 * (i >> 2) + 4 * half + (i & 3);
          fma2(v[i], v[i + 1], k, k, -m0, -m0);
          v[i] = ex2(!MASKED || c <= hi ? v[i] : -INFINITY);
          v[i + 1] = ex2(!MASKED || c + 1 <= hi ? v[i + 1] : -INFINITY);
          add2(s0, s1, v[i], v[i + 1]);
          mul2(v[i], v[i + 1], f, f);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int col = at_place(16 * half + 2 * e), i = 4 * (col >> 3) + (col & 3);
          split2(v[i], v[i + 1], pw[16 * half + e], pw[16 * half + 8 + e]);
        }
      }
      w.l += s0 + s1;
      tm_st32(sa + c0, pw);
    }
  }
  // a tile of raw positions, lo < j <= hi attended
  __device__ __forceinline__ void soften_raw(Row& w, uint32_t sa, float qs, int slot0, int j0, int lo, int hi) {
    float mx = -INFINITY, vmax = 0.f;
#pragma unroll 1
    for (int c0 = 0; c0 < RNT; c0 += 32) {
      float v[32];
      tm_ld32(sa + c0, v);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const int j = j0 + c0 + i;
        if (j > lo && j <= hi) mx = fmaxf(mx, v[i] * (sh.rawk[slot0 + c0 + i] * qs));
        vmax = fmaxf(vmax, sh.rawv[slot0 + c0 + i]);
      }
    }
    follow(w, mx, vmax);
    const float m0 = w.m == -INFINITY ? 0.f : w.m;
#pragma unroll 1
    for (int c0 = 0; c0 < RNT; c0 += 32) {
      float v[32];
      tm_ld32(sa + c0, v);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const int j = j0 + c0 + i;
        const float p = j > lo && j <= hi ? ex2(v[i] * (sh.rawk[slot0 + c0 + i] * qs) - m0) : 0.f;
        w.l += p;
        v[i] = p * (sh.rawv[slot0 + c0 + i] * w.rvref);
      }
      uint32_t pw[32];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) split2(v[16 * k + 2 * e], v[16 * k + 2 * e + 1], pw[16 * k + e], pw[16 * k + 8 + e]);
      tm_st32(sa + c0, pw);
    }
  }
  __device__ void softmax(const Stretch& u, Row& w) {
    const Tiles& tl = u.tl;
    const int grp = warp >> 2, row = 32 * (warp & 3) + lane;
    const uint32_t at = tmem + ((uint32_t)(32 * (warp & 3)) << 16), sa = at + C_S + NT * grp, oa = at + C_O + D * grp;
    // rows past the last query go along with it (and are not written)
    const int P = min(u.p0 + tl.t0 + row / a.g, tl.Pmax), W = a.W;
    const float qs = sh.qscale[row], qr = sh.qraw[row];
#pragma unroll
    for (int i = 0; i < D; ++i) w.acc[i] = 0.f;
    w.m = -INFINITY;
    w.l = w.vref = w.rvref = 0.f;
    bool pending = false, heads = false;
    for (int it = u.ta; it < u.tb; ++it, ++gt) {
      if ((gt & 1) != grp) continue;
      if (pending) {
        if (!held(&sh.pvdone[grp], ((gt - 2) >> 1) & 1)) return;
        fence_after();
        drain(w, oa);
      }
      if (it >= tl.nqt && !heads) {
        if (pending) to_heads(w, u);
        heads = true;
      }
      if (!held(&sh.sfull[grp], (gt >> 1) & 1)) return;
      fence_after();
      if (it < tl.nqt) {
        const float2 s0 = sh.scale[gt & 7][0], s1 = sh.scale[gt & 7][1];
        const float dk[2] = {s0.x * qs, s1.x * qs}, dv[2] = {s0.y, s1.y};
        const int j0 = it * NT, hi = P - W;
        // (a page that is not there has scales of zero: nothing of it is attended to)
        const int top = s0.x == 0.f && s1.x == 0.f && s0.y == 0.f && s1.y == 0.f && page_bad(u, it) ? -1 : hi;
        if (__all_sync(FULL, j0 + NT - 1 <= top)) soften<false>(w, sa, dk, dv, j0, top);
        else soften<true>(w, sa, dk, dv, j0, top);
      } else {
        const int slot0 = (it - tl.nqt) * RNT;
        if (!held(&sh.vfull[gt % NS], (gt / NS) & 1)) return;  // (the values' powers of two are there)
        soften_raw(w, sa, qr, slot0, tl.rlo + slot0, P - W, P);
      }
      tm_wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&sh.pfull[grp]);
      pending = true;
    }
    if (pending) {
      // the group's last tile: the last of the segment or the one before
      const int last = (gt & 1) != grp ? gt - 1 : gt - 2;
      if (!held(&sh.pvdone[grp], (last >> 1) & 1)) return;
      fence_after();
      drain(w, oa);
      if (!heads) to_heads(w, u);
    }
  }
  __device__ __forceinline__ bool page_bad(const Stretch& u, int it) const {
    const int phys = __ldg(a.block_table + (size_t)u.b * a.max_pages_per_seq + it);
    return phys < 0 || phys >= a.L.n_pages;
  }
  __device__ void leave_row(const Row& w) {
    const int grp = warp >> 2, row = 32 * (warp & 3) + lane;
    float* o = reinterpret_cast<float*>(smem + ((size_t)grp * ROWS + row) * O_STRIDE);
#pragma unroll
    for (int i = 0; i < D; i += 4)
      *reinterpret_cast<float4*>(o + i) = make_float4(w.acc[i] * w.vref, w.acc[i + 1] * w.vref, w.acc[i + 2] * w.vref, w.acc[i + 3] * w.vref);
    sh.m[grp][row] = w.m;
    sh.l[grp][row] = w.l;
  }
  // both groups' parts together, to the output or to a partial result
  __device__ void rows_out(const Stretch& u) {
    const Tiles& tl = u.tl;
    float* rec = u.rec < 0 ? nullptr : recs + (size_t)u.rec * REC;
    const int g = a.g, nrows = tl.nq * g;
    const size_t head0 = (size_t)u.unit * g;
#pragma unroll 2
    for (int row = warp; row < nrows; row += THREADS / 32) {
      const float m0 = sh.m[0][row], m1 = sh.m[1][row], M = fmaxf(m0, m1);
      const float f0 = m0 == -INFINITY ? 0.f : ex2(m0 - M), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - M);
      const float l = sh.l[0][row] * f0 + sh.l[1][row] * f1;
      const float4 x = *reinterpret_cast<const float4*>(smem + (size_t)row * O_STRIDE + 16 * lane);
      const float4 y = *reinterpret_cast<const float4*>(smem + (size_t)(ROWS + row) * O_STRIDE + 16 * lane);
      float4 o = make_float4(x.x * f0 + y.x * f1, x.y * f0 + y.y * f1, x.z * f0 + y.z * f1, x.w * f0 + y.w * f1);
      if (rec) {
        *reinterpret_cast<float4*>(rec + row * D + 4 * lane) = o;
        if (lane == 0) {
          rec[ROWS * D + row] = M;
          rec[ROWS * D + ROWS + row] = l;
        }
      } else {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        *reinterpret_cast<float4*>(a.out + ((head0 + row % g) * a.T + tl.t0 + row / g) * D + 4 * lane) = o;
      }
    }
  }

  // ---------------------------------------------------------------- a warp's life: ROLE 0 softmax, 1 operands, 2 logits, 3 values, 4 where to go on
  template <int ROLE>
  __device__ void run() {
    for (int k = 0;; ++k) {
      const Stretch& u = sh.at[k & 1];
      if (u.tb < 0) return;
      queries(u);
      sync_all();
      if (ROLE == 0) queries_to_tmem();
      fence_before();
      sync_all();
      fence_after();
      if constexpr (ROLE == 0) {
        Row w;
        softmax(u, w);
        sync_all();
        if (sh.gone) return;
        leave_row(w);
      } else {
        if (ROLE == 1) operands(u);
        else if (ROLE == 2) issue_logits(u);
        else if (ROLE == 3) issue_values(u);
        else if (warp == NEXT_WARP && lane == 0)
          locate(u.next, work.cut(blockIdx.x), work.cut(blockIdx.x + 1), sh.at[(k + 1) & 1]);
        sync_all();
        if (sh.gone) return;
      }
      sync_all();
      rows_out(u);
      sync_all();
    }
  }
};

template <bool BF16>
__global__ void __launch_bounds__(THREADS, 1) prefill_block_kernel(const __grid_constant__ PrefillArgs a, float* recs) {
  using K = Kernel<BF16>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ typename K::Shared sh;
  Work work;
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid < D) sh.signs[tid] = a.p.signs[tid];
  if (tid == 32) {
    for (int s = 0; s < NS; ++s) {
      bar_init(&sh.kfull[s], N_DQ);
      bar_init(&sh.kempty[s], 1);
      bar_init(&sh.vfull[s], N_DQ);
      bar_init(&sh.vempty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&sh.sfull[i], 1);
      bar_init(&sh.pfull[i], N_SOFT / 2);
      bar_init(&sh.pvdone[i], 1);
      bar_init(&sh.done[i], 1);
    }
    sh.gone = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  plan(a, work, sh.p0, sh.pre, gridDim.x);
  // sequences that are not part of the call, or past capacity: zeros
  for (int b = 0; b < a.batch; ++b) {
    if (sh.p0[b] >= 0) continue;
    const size_t per = (size_t)a.Hkv * a.g * a.T * (D / 4);
    for (int ll = 0; ll < a.n_layers_call; ++ll) {
      float4* o = reinterpret_cast<float4*>(a.out) + ((size_t)ll * a.batch + b) * per;
      for (size_t i = (size_t)blockIdx.x * THREADS + tid; i < per; i += (size_t)gridDim.x * THREADS) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  if (blockIdx.x >= work.n || work.total() == 0) return;
  if (warp == S_WARP) {
    tm_alloc(&sh.tmem, TMEM_COLS);
    fence_before();
  }
  __syncthreads();
  fence_after();
  K k(a, sh, smem, work, recs);
  k.tmem = sh.tmem;
  if (tid == NEXT_WARP * 32) {
    const long long lo = work.cut(blockIdx.x);
    k.locate(lo, lo, work.cut(blockIdx.x + 1), sh.at[0]);
  }
  __syncthreads();
  if (warp < N_SOFT) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SOFT_REGS));
    k.template run<0>();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGS));
    if (warp < DQ0 + N_DQ) k.template run<1>();
    else if (warp == S_WARP) k.template run<2>();
    else if (warp == PV_WARP) k.template run<3>();
    else k.template run<4>();
    // everything that a warp has issued lands before the columns are freed
    if (warp == S_WARP || warp == PV_WARP) {
      uint64_t* bar = &sh.done[warp - S_WARP];
      mma_commit(bar);
      bar_land(bar, 0);
    }
  }
  fence_before();
  part_sync(1, THREADS);
  if (warp == S_WARP) {
    fence_after();
    tm_free(k.tmem, TMEM_COLS);
  }
}

// Joins the partial results of the row tiles that a cut divides.  Block (c, part): cut c + 1, if it is the first within its
// row tile, for a share of the rows; parts in the order of their CTAs.
constexpr int JOIN_SHARES = 8, JOIN_WARPS = ROWS / JOIN_SHARES;
template <bool BF16>
__global__ void __launch_bounds__(JOIN_WARPS * 32) prefill_join_kernel(const __grid_constant__ PrefillArgs a, const float* recs, int ctas) {
  __shared__ int p0s[MAX_BATCH];
  __shared__ long long pre[MAX_BATCH + 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Work w;
  plan(a, w, p0s, pre, ctas);
  const int c = blockIdx.x + 1, lane = threadIdx.x & 31;
  if (c >= w.n || w.total() == 0) return;
  const long long y = w.cut(c);
  const Unit u = w.find(y);
  const Tiles tl(w, u, a.W, Kernel<BF16>::RNT);
  const int at = tl.before(y - u.start);
  if (at == 0 || at == tl.n) return;
  const long long y1 = w.cut(c - 1);
  if (y1 > u.start && tl.before(y1 - u.start) > 0) return;  // an earlier cut within the row tile
  const int row = blockIdx.y * JOIN_WARPS + (threadIdx.x >> 5), g = a.g;
  if (row >= tl.nq * g) return;
  // parts: of CTA c - 1 (its first stretch only if that begins in this row tile), then of those that begin in it
  const long long end = u.start + u.cost;
  auto part_of = [&](int k) { return recs + (size_t)(2 * k + (w.cut(k) >= u.start ? 0 : 1)) * REC; };
  auto empty = [&](int k) {
    const long long lo = w.cut(k), hi = w.cut(k + 1);
    return (lo > u.start ? tl.before(lo - u.start) : 0) >= (hi >= end ? tl.n : tl.before(hi - u.start));
  };
  int last = c;
  while (last + 1 < w.n && w.cut(last + 1) < end) ++last;
  float M = -INFINITY;
  for (int k = c - 1; k <= last; ++k)
    if (!empty(k)) M = fmaxf(M, __ldcg(part_of(k) + ROWS * D + row));
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = c - 1; k <= last; ++k) {
    if (empty(k)) continue;
    const float* rec = part_of(k);
    const float m = __ldcg(rec + ROWS * D + row);
    const float f = m == -INFINITY ? 0.f : ex2(m - M);
    const float4 x = __ldcg(reinterpret_cast<const float4*>(rec + row * D) + lane);
    l += __ldcg(rec + ROWS * D + ROWS + row) * f;
    o.x += x.x * f;
    o.y += x.y * f;
    o.z += x.z * f;
    o.w += x.w * f;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const size_t unit = ((size_t)(u.hl / a.Hkv) * a.batch + u.b) * a.Hkv + u.hl % a.Hkv;
  *reinterpret_cast<float4*>(a.out + ((unit * g + row % g) * a.T + tl.t0 + row / g) * D + 4 * lane) =
      make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
}

template <bool BF16>
cudaError_t launch(const PrefillArgs& a, int sms, cudaStream_t s) {
  cudaError_t e = allow_shared_memory<prefill_block_kernel<BF16>>();
  if (e != cudaSuccess) return e;
  prefill_block_kernel<BF16><<<sms, THREADS, SMEM, s>>>(a, a.parts);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms, JOIN_SHARES);
  cfg.blockDim = dim3(JOIN_WARPS * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefill_join_kernel<BF16>, a, (const float*)a.parts, sms);
}

}  // namespace

size_t prefill_block_scratch_bytes(int sms) { return (size_t)2 * sms * REC * sizeof(float); }

cudaError_t launch_prefill_blocks(const PrefillArgs& a, int sms, cudaStream_t s) {
  return a.in_bf16 ? launch<true>(a, sms, s) : launch<false>(a, sms, s);
}

}  // namespace kvq

// Attention of a prefill chunk over a KVQ_Q8B32 cache: query t of sequence b attends to positions [0, pos[b] + t], the
// newest `window` raw, the rest through the records (what its own single-token step would read), after the chunk's append.
//
//   o = sum_j w_j v_j / sum_j w_j,  w_j = 2^(l_j - m),  l_j = log2(e) / sqrt(128) q.k_j
//   recorded j:  q.k_j = d_k (q~ . c_j), v_j = d_v H c'_j ...: the codes c are the operands, the two scales of a block of 32
//   positions never meet them: logits are multiplied by d_k, weights by d_v before they go to P V, in their exponents:
//   w'_j = 2^(l_j + log2 d_v - R), R a row's running reference of these; sum_j w_j has a reference m of its own
//
// The products run on the 5th-generation tensor cores (tcgen05.mma, kind::f16, fp32 accumulators in tensor memory).  Codes
// are exact in one fp16 plane, so a product takes two passes (hi and lo of the queries, or of the weights: 22 bits) where
// formats whose dequantised values need two planes take three.
//  * Work: a row tile is 128 (query, head) rows of one (layer, sequence, kv-head); its positions go in tiles of 64 recorded
//    ones (a page), then of raw ones.  The call's tiles form one list that is cut into equal ranges, one per CTA (one CTA
//    an SM), whatever the chunk's and the contexts' lengths: a row tile that a cut divides leaves partial results, which a
//    second launch joins in order.  Without the cut 1024 tokens of 24 heads are 200 row tiles on 152 SMs, and three short
//    turns keep 12 of them busy.  Where row tiles are many and not long (take_whole) nothing is cut: CTAs take them one
//    after the other.  (The arithmetic of the list stands in prefill_list.cuh.)
//  * A tile's stored order is the operands' order up to a permutation of channels (keys) or positions (values), which
//    queries and weights follow: 16 stored bytes become two 16-byte operand rows by byte permutes, nothing is transposed.
//  * Raw tiles are taken as they are, not rotated: queries are also kept unrotated (in shared memory), and the output
//    accumulator, a row per thread in registers, is rotated back once, before the first raw tile.
//  * Warps: two groups of four soften alternate tiles (a row a thread: lanes of tensor memory), each with a reference and a
//    sum of its own; four add every tile's P V, which starts from zero, to the output accumulator in registers (the tensor
//    cores' truncating sums stay within a tile, and a reference that moves rescales registers only); four turn bytes into
//    operands; one issues the logits' products, one those of the values.  Registers are shared out among them.
//  * Queries, raw keys and raw values are scaled by powers of two, each vector by its own, and what is kept to fp16's range is
//    a weight together with its value's scale, against the row's own largest: fp16 parts keep their bits at any magnitude, and
//    what a row does not attend to, or hardly, takes none of them.  (One scale for a raw tile, and the largest scale of values
//    for all rows, lost an early row whose chunk had values 2^40 times larger further on.)
//  * A kernel's small first-level cache (shared memory takes the rest) makes spilled registers and code that is run once dear: values
//    for one phase are computed in it (once()), what a row tile does once is done by one group of warps.
//  * Every wait is bounded (kv_set_wait_limit_ns); one that runs out flags the status word, and the CTA makes NaN of the row
//    tiles, or parts of them, that it is at and that it would have come to.
//
// One layer, bf16, window 128: 1024 tokens of 24 heads at position 15001 take 440 us (two passes of the products over recorded
// positions at the measured bf16 rate: 204 us, 46 %), a prompt of 2048 tokens of 32 heads 164 us, three float turns of 37
// tokens of 8 heads at 1000 positions 37 us.  A tile of 64 positions takes 2400 cycles of which both products would take 1024 (the
// tensor pipe is busy 40 % of the time): bound by the weights (1500 cycles a tile and group of warps, two groups) and the rate at
// which instructions come.
#include <cfloat>

#include "prefill_list.cuh"
#include "tc.cuh"

namespace kvq {

namespace {

using namespace tc;
using namespace prefill_list;

constexpr int NS = 3;                // operand stages
constexpr int RS = 2;                // pages under way
constexpr int N_SOFT = 8;            // softmax warps, two groups
constexpr int N_SUM = 4;             // warps that hold the output
constexpr int DQ0 = 12, N_DQ = 4;    // operand warps
constexpr int S_WARP = 16, PV_WARP = 17, PAGE_WARP = 18, NEXT_WARP = 19;
constexpr int THREADS = 640;
constexpr int LAUNCH_REGS = 96;
// registers: 256 x 96 + 128 x (168 + 80 + 40) = 640 x 96, what the block is launched with
constexpr int SOFT_REGS = 96, SUM_REGS = 168, DQ_REGS = 80, ISSUE_REGS = 40;
constexpr uint32_t TMEM_COLS = 512, C_QHI = 0, C_QLO = 64, C_S = 128, C_O = 256;  // Q hi | lo | two S or P | two O
// K-groups of an operand (8 channels of 64 keys, 8 positions of 128 value channels) are 32 bytes further apart than they
// are long, so that lanes which write one row of four neighbouring groups each do not meet in a bank
constexpr uint32_t K_LEAD = NT * 16 + 32, V_LEAD = D * 16 + 32;
constexpr uint32_t V_OFF = 16 * K_LEAD, STAGE = V_OFF + 8 * V_LEAD;  // a stage: keys, values
constexpr uint32_t LO_K = 8192, LO_V = 4 * V_LEAD;      // raw tiles of float caches (32 positions): from hi to lo
constexpr uint32_t Q_STRIDE = 2 * D * 2 + 16;           // query staging row: hi, lo, pad
constexpr uint32_t QR_LEAD = ROWS * 16 + 16;            // unrotated queries: from one 8 channels to the next
constexpr uint32_t QR_PLANE = 16 * QR_LEAD;
constexpr uint32_t QR_OFF = NS * STAGE, PAGE_OFF = QR_OFF + 2 * QR_PLANE, PAGE_SLOT = 2 * 8208;
constexpr uint32_t SMEM = PAGE_OFF + RS * PAGE_SLOT;
static_assert(V_OFF >= 16384, "raw keys fit too");
constexpr uint32_t O_STRIDE = (D + 4) * 4;
static_assert(ROWS * Q_STRIDE <= NS * STAGE && ROWS * O_STRIDE <= NS * STAGE, "what borrows the stages");
// References are whole numbers: a factor between two of them is exact.  One is set BOOST to BOOST + 1 below the largest exponent
// so far and follows when that is RAISE_AT further up: weights stay below 2^15.
constexpr float BOOST = 4.f, RAISE_AT = 10.f;
constexpr int REC = ROWS * D + 3 * ROWS;  // floats of a partial result: O, its reference, l, its reference

// Along K, channels (keys) and positions of a tile (values) stand in the order in which 16-byte chunks hold their codes: which
// of them is at a place, and the place of each
__host__ __device__ constexpr int at_place(int k) {
  return (k & ~31) | (((k >> 2) & 1) << 4) | (((k >> 1) & 1) << 3) | (((k >> 3) & 3) << 1) | (k & 1);
}
__host__ __device__ constexpr int place_of(int c) {
  return (c & ~31) | (((c >> 1) & 3) << 3) | (((c >> 4) & 1) << 2) | (((c >> 3) & 1) << 1) | (c & 1);
}
// (row, k) of a K-major operand whose groups of 8 k are `lead` bytes apart
__device__ __forceinline__ uint32_t km(int row, int k, uint32_t lead) {
  return (uint32_t)(k >> 3) * lead + (uint32_t)((row >> 3) * 128 + (row & 7) * 16 + (k & 7) * 2);
}

// ------------------------------------------------------------------ the list of tiles
// warp 0: positions, active sequences and prefix of the sequences' costs into shared memory; how the CTAs share the list
template <typename Shared>
__device__ void plan(const PrefillArgs& a, Shared& sh, int ctas, int raw_nt) {
  if (threadIdx.x < 32) {
    const List w(a.batch, a.T, a.g, a.Hkv * a.n_layers_call, a.W, raw_nt, sh.p0, sh.pre, sh.act, 0);
    const int lane = threadIdx.x, per = (a.batch + 31) / 32;
    const int b0 = min(a.batch, lane * per), b1 = min(a.batch, b0 + per);
    long long s = 0;
    int far = -1, active = 0;
    for (int b = b0; b < b1; ++b) {
      const int p = a.pos[b];
      sh.p0[b] = p >= 0 && (long long)p + a.T <= a.max_seq_len ? p : -1;
      if (sh.p0[b] >= 0) s += w.upto(b, w.nx);
      far = max(far, sh.p0[b]);
      active += sh.p0[b] >= 0;
    }
    long long incl = s;
    int upto = active;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(FULL, incl, o);
      const int z = __shfl_up_sync(FULL, upto, o);
      if (lane >= o) {
        incl += y;
        upto += z;
      }
    }
    long long run = incl - s;
    int at = upto - active;
    for (int b = b0; b < b1; ++b) {
      sh.pre[b] = run;
      if (sh.p0[b] < 0) continue;
      run += w.upto(b, w.nx);
      sh.act[at++] = (unsigned short)b;
    }
    if (lane == 31) sh.pre[a.batch] = incl;
    far = __reduce_max_sync(FULL, far);
    active = __reduce_add_sync(FULL, active);
    __syncwarp();
    if (lane == 0) {
      List l = w;
      l.n_act = sh.n_act = active;
      sh.whole = l.take_whole(ctas, far);
      sh.parts = l.parts(ctas, sh.whole);
    }
  }
  __syncthreads();
}

// A CTA's stretch of one row tile: tiles ta .. tb - 1 of it, whole or to be joined with others
struct Stretch : Part {
  int unit, layer, h;  // unit: (layer of the call, sequence, kv-head)
  int p0, rec;         // rec: -1: the row tile as a whole
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
__device__ __forceinline__ void tm_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      KVQ_R8(KVQ_IN, 0), KVQ_R8(KVQ_IN, 8)
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// (NaN if one is)
__device__ __forceinline__ float max3nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// A warp's bounded wait, of about `limit` ns at most.  false: this CTA gives up (a wait elsewhere ran out, or this one: flagged).
// NAP false: looks without sleeping, for limits that a single sleep might pass.  (Sleeps of a given length, or a choice between the
// two in every wait, cost 1024 tokens at 15001 positions 7 to 40 us of 438.)
template <bool NAP = true>
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* gone, unsigned* status, unsigned long long limit) {
  bool ok = NAP ? bar_try(bar, parity) : bar_test(bar, parity);
  if (__builtin_expect(!ok, 0)) {
    const unsigned long long t0 = gtimer();
    while (true) {
#pragma unroll 1
      for (int i = 0; i < (NAP ? 64 : 1) && !ok; ++i) ok = NAP ? bar_try(bar, parity) : bar_test(bar, parity);
      if (ok || *gone) break;
      if (gtimer() - t0 > limit) {
        atomicOr(status, KVQ_DEV_TIMEOUT);
        *gone = 1;
        break;
      }
    }
  }
  return __all_sync(FULL, ok);
}
// the largest magnitude of 128 values in four neighbouring lanes
__device__ __forceinline__ float quad_max(const float (&x)[32]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 32; i += 2) m = max3(m, fabsf(x[i]), fabsf(x[i + 1]));
  m = fmaxf(m, __shfl_xor_sync(FULL, m, 1));
  return fmaxf(m, __shfl_xor_sync(FULL, m, 2));
}
// log2 of a finite scale, its fraction to 2^-22 whatever its size; -inf of zero
__device__ __forceinline__ float log2_of(float x) {
  if (!(x > 0.f)) return -INFINITY;
  int e = 0;
  if (x < FLT_MIN) {
    x *= 0x1p24f;
    e = -24;
  }
  const uint32_t u = __float_as_uint(x);
  return (float)(e + (int)(u >> 23) - 127) + __log2f(__uint_as_float((u & 0x7fffffu) | 0x3f800000u));
}
// eight bf16 values
__device__ __forceinline__ void unpack8(uint4 w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(u[e] << 16);
    x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
  }
}

// This warp group's registers per thread from here on (taking more and giving some back are two instructions)
template <int N>
__device__ __forceinline__ void take_registers() {
  static_assert(N % 8 == 0 && 8 * 32 * SOFT_REGS + 4 * 32 * (SUM_REGS + DQ_REGS + ISSUE_REGS) <= THREADS * LAUNCH_REGS, "more than there are");
  if constexpr (N > LAUNCH_REGS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 2^n / l, the factor from sums to outputs (n: between the references of the two sums)
__device__ __forceinline__ float share_of(float n, float l) {
  if (!(l > 0.f) || !(n > -INFINITY)) return 0.f;
  const float h = floorf(0.5f * n);  // (the sum of weights may be as far from 1 as the factor)
  return ex2(h) / l * ex2(n - h);
}

template <bool BF16>
struct Kernel {
  static constexpr int ROW_BYTES = D * (BF16 ? 2 : 4);  // of a raw vector of the call
  static constexpr int RNT = BF16 ? 64 : FULL_NT;  // raw positions of a tile: one plane of a bf16 cache's, hi and lo of a float one's
  static constexpr uint32_t ID_S = idesc(ROWS, NT, false, false), ID_SR = idesc(ROWS, FULL_NT, false, false);
  static_assert(!BF16 || RNT == NT, "as wide as a recorded tile");
  static constexpr uint32_t ID_O = idesc(ROWS, D, false, false), ID_OR = idesc(ROWS, D, false, true);

  // shared by the CTA, besides the stages
  struct Shared {
    uint64_t kfull[NS], kempty[NS], vfull[NS], vempty[NS], sfull[2], pfull[2], pvdone[2], ofree[2], done[2], rfull[RS], rempty[RS], begun[4];
    uint32_t tmem;
    int gone;
    float qscale[ROWS], qraw[ROWS];        // powers of two that the queries were divided by
    float m[2][ROWS], l[2][ROWS], M[ROWS]; // both groups' sums and their references, the output's reference, at the end
    float mt[4][ROWS];                     // a tile's references of its weights
    long long hi;                          // where the CTA's stretch of the cost line ends
    int whole, parts, n_act;               // row tiles are taken whole; CTAs that have work; sequences of the call
    int halves[RS];                        // of a page under way that are read (0: there is no such page)
    alignas(16) float4 blk[8][2];          // of a recorded tile's two blocks: the keys' scale, log2 of the values', both again
    alignas(16) float2 col[8][NT];         // of a raw tile's positions: the keys' power of two, log2 of the values'
    alignas(16) float signs[D];            // (read four at a time)
    int p0[MAX_BATCH];
    unsigned short act[MAX_BATCH];
    long long pre[MAX_BATCH + 1];
    Stretch at[2];                         // this stretch and the next
  };

  static_assert(alignof(Shared) % 16 == 0, "parts of it are read as float4");

  const PrefillArgs& a;
  Shared& sh;
  uint8_t* smem;
  int warp, lane;
  uint32_t tmem;
  int gt = 0, gr = 0, gb = 0;  // tiles so far, slots of pages and raw operands, stretches of two tiles or more

  // Made within each role: nothing is then live where the roles part and their registers are shared out (a value that is
  // takes a register that the smallest share has, or memory)
  __device__ Kernel(const PrefillArgs& args, Shared& s, uint8_t* sm) : a(args), sh(s), smem(sm) {
    uint32_t tid;
    asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));
    warp = tid >> 5;
    lane = tid & 31;
    tmem = *const_cast<volatile uint32_t*>(&s.tmem);
  }
  __device__ __forceinline__ bool held(uint64_t* bar, uint32_t parity) { return wait(bar, parity, &sh.gone, a.p.status, a.wait_ns); }
  __device__ __forceinline__ void sync_all() { part_sync(1, THREADS); }

  __device__ __forceinline__ List list() const {
    return List(a.batch, a.T, a.g, a.Hkv * a.n_layers_call, a.W, RNT, sh.p0, sh.pre, sh.act, sh.n_act);
  }
  // the CTA's first stretch with tiles
  __device__ void locate(Stretch& st) {
    if (sh.whole) {
      grab(blockIdx.x, st);
      return;
    }
    const List l = list();
    long long lo, hi;
    l.cut(blockIdx.x, sh.parts, lo, hi);
    sh.hi = hi;
    fill(l.first(lo, hi, st) ? 0 : 1, st);
  }
  // a value whose derivatives are computed where they are used, and not kept through the tiles of a stretch
  __device__ __forceinline__ static int once(int x) {
    asm volatile("" : "+r"(x));
    return x;
  }
  // Row tile i of the list, or (-1) the next that no CTA has taken.  Which CTA computes a row tile does not change its result.
  __device__ void grab(int i, Stretch& st) const {
    if (i < 0) {
      asm volatile("griddepcontrol.wait;" ::: "memory");  // (the ring's copy clears the count)
      i = gridDim.x + atomicAdd(a.taken, 1);
    }
    list().whole(i, st);
    fill(0, st);
  }
  // the one after it: the next row tiles of the line
  __device__ void follow_up(const Stretch& u, Stretch& st) const {
    list().follow(u, sh.hi, st);
    fill(1, st);
  }
  // what else the CTA goes by
  __device__ __forceinline__ void fill(int slot, Stretch& st) const {
    if (st.tb < 0) return;
    st.rec = st.ta == 0 && st.tb == st.tl.n ? -1 : 2 * (int)blockIdx.x + slot;
    const int l = st.hl / a.Hkv;
    st.h = st.hl - l * a.Hkv;
    st.layer = a.layer0 + l;
    st.unit = (l * a.batch + st.b) * a.Hkv + st.h;
    st.p0 = sh.p0[st.b];
    if (st.rec >= 0) a.keys[st.rec] = make_int2(st.unit, st.x);
  }

  // ---------------------------------------------------------------- queries
  // Four lanes a row with 32 channels each, eight rows a warp and round: unrotated hi and lo to their operand, rotated ones to the
  // staging rows, each over its own power of two
  __device__ void queries(const Stretch& u) {
    const Tiles& tl = u.tl;
    const int g = a.g, lane = once(this->lane), v = lane >> 2, G = lane & 3;
#pragma unroll 1
    for (int round = 0; round < ROWS / (8 * N_SOFT); ++round) {
      const int row = 8 * (warp + N_SOFT * round) + v;
      float x[32];
      if (row < tl.nq * g) {
        const size_t off = (((size_t)u.unit * g + row % g) * a.T + tl.t0 + row / g) * D + 32 * G;
        if (BF16) {
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + off);
          uint4 w[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) w[c] = __ldg(src + c);
#pragma unroll
          for (int c = 0; c < 4; ++c) unpack8(w[c], x + 8 * c);
        } else {
          const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + off);
#pragma unroll
          for (int c = 0; c < 8; ++c) *reinterpret_cast<float4*>(x + 4 * c) = __ldg(src + c);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 32; i += 2) mul2(x[i], x[i + 1], LOGIT_SCALE, LOGIT_SCALE);
      float inv;
      float s2 = pow2_of(quad_max(x), inv);
      if (G == 0) sh.qraw[row] = s2;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split2(x[8 * c + 2 * e] * inv, x[8 * c + 2 * e + 1] * inv, hi[e], lo[e]);
        uint8_t* at = smem + QR_OFF + km(row, 32 * G + 8 * c, QR_LEAD);
        *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(at + QR_PLANE) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      rotate32(x, G, sh.signs, nullptr);
      if (a.sinkhorn) {
        const __half2* sig = reinterpret_cast<const __half2*>(a.p.sigk + ((size_t)u.layer * a.Hkv + u.h) * D + 32 * G);
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float2 f = __half22float2(sig[i / 2]);
          mul2(x[i], x[i + 1], f.x, f.y);
        }
      }
      s2 = pow2_of(quad_max(x), inv);
      if (G == 0) sh.qscale[row] = s2;
      uint8_t* st = smem + (size_t)row * Q_STRIDE + 64 * G;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = at_place(8 * i + 2 * e);
          split2(x[c] * inv, x[c + 1] * inv, hi[e], lo[e]);
        }
        *reinterpret_cast<uint4*>(st + 16 * i) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(st + 2 * D + 16 * i) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
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
#pragma unroll 1
    for (int it = u.ta; it < u.tb; ++it, ++gt) {
      const int s = gt % NS, bb = gt & 1;
      // the stage's keys; the buffer is free once the values' products of two tiles before have read its weights
      if (!held(&sh.kfull[s], (gt / NS) & 1)) return;
      if (gt >= 2 && !held(&sh.pvdone[bb], ((gt - 2) >> 1) & 1)) return;
      fence_after();
      const uint32_t dS = tmem + C_S + NT * bb;
      if (it < tl.nqt) {
        const uint64_t k = sdesc(base + s * STAGE, K_LEAD, 128);
        const uint32_t q = tmem + C_QHI;
#pragma unroll 2
        for (int ks = 0; ks < D / 16; ++ks) {
          mma_ts(dS, q + 8 * ks, k + 2 * K_LEAD / 16 * ks, ID_S, ks > 0);
          mma_ts(dS, q + 8 * ks + (C_QLO - C_QHI), k + 2 * K_LEAD / 16 * ks, ID_S, 1);
        }
      } else {
        const bool full = !BF16 || it < tl.nqt + tl.n_full;
        const uint32_t nt = full ? FULL_NT : RNT, id = full ? ID_SR : ID_S;
        uint64_t k = sdesc(base + s * STAGE, nt * 16, 128), q = sdesc(base + QR_OFF, QR_LEAD, 128);
#pragma unroll 1
        for (int ks = 0; ks < D / 16; ++ks, k += nt * 2, q += 2 * QR_LEAD / 16) {
          mma_ss(dS, q, k, id, ks > 0);
          mma_ss(dS, q + QR_PLANE / 16, k, id, 1);
          if (full) mma_ss(dS, q, k + LO_K / 16, id, 1);
        }
      }
      mma_commit(&sh.sfull[bb]);
      mma_commit(&sh.kempty[s]);
    }
  }
  __device__ void issue_values(const Stretch& u) {
    const Tiles& tl = u.tl;
    const uint32_t base = smem_u32(smem);
#pragma unroll 1
    for (int it = u.ta; it < u.tb; ++it, ++gt) {
      const int s = gt % NS, bb = gt & 1;
      if (!held(&sh.pfull[bb], (gt >> 1) & 1) || !held(&sh.vfull[s], (gt / NS) & 1)) return;
      if (gt >= 2 && !held(&sh.ofree[bb], ((gt - 2) >> 1) & 1)) return;
      fence_after();
      uint32_t p = tmem + C_S + NT * bb;
      const uint32_t dO = tmem + C_O + D * bb;
      if (it < tl.nqt) {
        const uint64_t v = sdesc(base + s * STAGE + V_OFF, V_LEAD, 128);
#pragma unroll 2
        for (int ks = 0; ks < NT / 16; ++ks) {
          mma_ts(dO, p + 16 * ks + 8, v + 2 * V_LEAD / 16 * ks, ID_O, ks > 0);
          mma_ts(dO, p + 16 * ks, v + 2 * V_LEAD / 16 * ks, ID_O, 1);
        }
      } else {
        const bool full = !BF16 || it < tl.nqt + tl.n_full;
        uint64_t v = sdesc(base + s * STAGE + V_OFF, V_LEAD, 128);
#pragma unroll 1
        for (int ks = 0; ks < (full ? FULL_NT : RNT) / 16; ++ks, v += 2 * V_LEAD / 16, p += 16) {
          mma_ts(dO, p + 8, v, ID_OR, ks > 0);
          if (full) mma_ts(dO, p, v + LO_V / 16, ID_OR, 1);
          mma_ts(dO, p, v, ID_OR, 1);
        }
      }
      mma_commit(&sh.vempty[s]);
      mma_commit(&sh.pvdone[bb]);
    }
  }

  // ---------------------------------------------------------------- pages and operands
  // One lane brings the pages of the stretch's recorded tiles, two ahead; the others read the block table ahead of it.
  __device__ void fetch(const Stretch& u) {
    const int32_t* bt = a.block_table + (size_t)u.b * a.max_pages_per_seq;
    const int last = min(u.tb, u.tl.nqt);
#pragma unroll 1
    for (int it0 = u.ta; it0 < last; it0 += 32) {
      const int mine = it0 + lane < last ? __ldg(bt + it0 + lane) : 0;
#pragma unroll 1
      for (int it = it0; it < min(last, it0 + 32); ++it, ++gr) {
        const int phys = __shfl_sync(FULL, mine, it - it0), s = gr % RS;
        if (gr >= RS && !held(&sh.rempty[s], ((gr / RS) & 1) ^ 1)) return;
        if (lane == 0) {
          if (phys < 0 || phys >= a.L.n_pages) {
            atomicOr(a.p.status, KVQ_DEV_BAD_PAGE);
            sh.halves[s] = 0;
            bar_arrive(&sh.rfull[s]);
          } else {
            const int n = it * NT + HALF < u.tl.qend ? 2 : 1;
            sh.halves[s] = n;
            bar_expect(&sh.rfull[s], n * a.L.half_bytes);
            bulk_g2s(smem + PAGE_OFF + s * PAGE_SLOT, a.p.pages + (((size_t)u.layer * a.L.n_pages + phys) * a.Hkv + u.h) * a.L.page_bytes,
                     n * a.L.half_bytes, &sh.rfull[s]);
          }
        }
        __syncwarp();
      }
    }
    // Raw tiles of the call's own tokens come the same way, keys then values, a slot each.  (Loads of their own, which only a
    // tile's other half overlapped, took 3000 cycles each of a raw tile's 10000.)
    static_assert(RNT * ROW_BYTES <= PAGE_SLOT, "a raw operand fits a slot");
#pragma unroll 1
    for (int it = max(u.ta, u.tl.nqt); it < u.tb; ++it) {
      const int j0 = u.tl.raw_at(it - u.tl.nqt, RNT);
      if (j0 < u.p0) continue;
      const uint32_t bytes = min(RNT, u.tl.Pmax - j0 + 1) * ROW_BYTES;
      const size_t off = ((size_t)u.unit * a.T + (j0 - u.p0)) * ROW_BYTES;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv, ++gr) {
        const int s = gr % RS;
        if (gr >= RS && !held(&sh.rempty[s], ((gr / RS) & 1) ^ 1)) return;
        if (lane == 0) {
          bar_expect(&sh.rfull[s], bytes);
          bulk_g2s(smem + PAGE_OFF + s * PAGE_SLOT, static_cast<const uint8_t*>(kv ? a.v : a.k) + off, bytes, &sh.rfull[s]);
        }
        __syncwarp();
      }
    }
  }
  // Lane (r, i) = (lane >> 2, lane & 3) takes the 16 bytes of (r, i) of a chunk, in order.  (A half that is not there, or not
  // read, may hold anything: its codes are finite and its weights zero.)
  __device__ void operands(const Stretch& u) {
    const int dw = warp - DQ0, r = lane >> 2, i = lane & 3;
    const int last_q = min(u.tb, u.tl.nqt);
    int it = u.ta;
#pragma unroll 1
    for (; it < last_q; ++it, ++gt, ++gr) {
      const int s = gt % NS, rs = gr % RS;
      const uint32_t before = ((gt / NS) & 1) ^ 1;  // phase of the stage's previous use
      uint8_t* kp = smem + s * STAGE + km(r, 8 * (4 * dw + i), K_LEAD);
      uint8_t* vp = smem + s * STAGE + V_OFF + km(16 * dw + r, 8 * i, V_LEAD);
      const uint8_t* pg = smem + PAGE_OFF + rs * PAGE_SLOT + dw * 512 + lane * 16;
      if (!held(&sh.rfull[rs], (gr / RS) & 1)) return;
      if (gt >= NS && !held(&sh.kempty[s], before)) return;
      if (dw == 0 && lane < 2) {
        float2 d = lane < sh.halves[rs] ? *reinterpret_cast<const float2*>(smem + PAGE_OFF + rs * PAGE_SLOT + lane * (PAGE_SLOT / 2) + 8192)
                                              : make_float2(0.f, 0.f);
        if (!(d.y < INFINITY)) d = make_float2(NAN, 1.f);  // (as for raw values that are not finite)
        const float e = log2_of(d.y);
        sh.blk[gt & 7][lane] = make_float4(d.x, e, d.x, e);
      }
      // chunk 4 mt + p (p = dw, mt = q & 1) of block q >> 1: tokens 16 mt + r and + 8, channels of K-group 4 p + i
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 w = *reinterpret_cast<const uint4*>(pg + (q >> 1) * (PAGE_SLOT / 2) + (q & 1) * 2048);
        uint8_t* o = kp + (32 * (q >> 1) + 16 * (q & 1)) * 16;
        *reinterpret_cast<uint4*>(o) = make_uint4(codes_lo(w.x), codes_lo(w.y), codes_lo(w.z), codes_lo(w.w));
        *reinterpret_cast<uint4*>(o + 128) = make_uint4(codes_hi(w.x), codes_hi(w.y), codes_hi(w.z), codes_hi(w.w));
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive(&sh.kfull[s]);
      if (gt >= NS && !held(&sh.vempty[s], before)) return;
      // chunk j = dw + 4 (q & 1): channels 16 j + r and + 8, positions of K-group 4 (q >> 1) + i
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 w = *reinterpret_cast<const uint4*>(pg + (q >> 1) * (PAGE_SLOT / 2) + 4096 + (q & 1) * 2048);
        uint8_t* o = vp + 64 * (q & 1) * 16 + 4 * (q >> 1) * V_LEAD;
        *reinterpret_cast<uint4*>(o) = make_uint4(codes_lo(w.x), codes_lo(w.y), codes_lo(w.z), codes_lo(w.w));
        *reinterpret_cast<uint4*>(o + 128) = make_uint4(codes_hi(w.x), codes_hi(w.y), codes_hi(w.z), codes_hi(w.w));
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        bar_arrive(&sh.vfull[s]);
        bar_arrive(&sh.rempty[rs]);
      }
    }
#pragma unroll 1
    for (; it < u.tb; ++it, ++gt) {
      const int s = gt % NS, j0 = u.tl.raw_at(it - u.tl.nqt, RNT);
      const bool full = !BF16 || it < u.tl.nqt + u.tl.n_full;
      const uint32_t before = ((gt / NS) & 1) ^ 1;
#pragma unroll 1
      for (int values = 0; values < 2; ++values) {
        if (gt >= NS && !held(values ? &sh.vempty[s] : &sh.kempty[s], before)) return;
        uint8_t* plane = smem + s * STAGE + (values ? V_OFF : 0);
        if (!(full ? raw<true>(u, j0, plane, values) : raw<false>(u, j0, plane, values))) return;
        fence_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(values ? &sh.vfull[s] : &sh.kfull[s]);
      }
    }
  }
  // Raw keys (K-major) or values (N-major: rows are positions too, in the order of the places) of positions j0 .. as operand
  // planes, each vector over a power of two of its own: FULL: hi and lo of FULL_NT positions, else one of RNT of the call's own
  // bf16 ones.  An element of a bf16 vector that its one fp16 plane does not hold exactly is below 2^-14 of the vector's largest
  // and off by 2^-25 of that at most.
  template <bool FULL>
  __device__ __forceinline__ bool raw(const Stretch& u, int j0, uint8_t* plane, int values) {
    // the lane's q-th eight channels are group 4 ((q + r / 4) mod 4) + (i + r) mod 4: eight lanes' reads of a slot hit all banks
    const int lane = once(this->lane), dw = once(warp) - DQ0, r = lane & 7, b = ((lane >> 3) + r) & 3, q0 = r >> 2;
    const int p0 = u.p0;
    const size_t unit = u.unit;
    constexpr bool PACKED = !FULL;  // kept as bf16
    const bool staged = PACKED || j0 >= p0;
    const int slot = gr % RS;
    if (staged && !held(&sh.rfull[slot], (gr / RS) & 1)) return false;
    const float* old = values ? a.snap_v : a.snap_k;
    const uint8_t* mine = staged ? smem + PAGE_OFF + slot * PAGE_SLOT
                                 : static_cast<const uint8_t*>(values ? a.v : a.k) + ((size_t)unit * a.T * ROW_BYTES + (long long)(j0 - p0) * ROW_BYTES);
    constexpr int TILE = FULL ? FULL_NT : RNT, ROUNDS = TILE / (8 * N_DQ), WORDS = PACKED ? 4 : 8;
    uint4 w[ROUNDS][WORDS];  // bf16 values, or floats; every load of the tile under way at once
#pragma unroll
    for (int n = 0; n < ROUNDS; ++n) {
      const int t = 8 * dw + r + 8 * N_DQ * n, j = j0 + t;
#pragma unroll
      for (int q = 0; q < WORDS; ++q) w[n][q] = make_uint4(0u, 0u, 0u, 0u);
      if (j > u.tl.Pmax) continue;
      if (FULL && j < p0) {
        const float4* f = reinterpret_cast<const float4*>(old + (unit * a.W + j % a.W) * D) + 2 * b;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 x = __ldg(f + 8 * ((q + q0) & 3)), y = __ldg(f + 8 * ((q + q0) & 3) + 1);
          w[n][(2 * q) % WORDS] = *reinterpret_cast<const uint4*>(&x);
          w[n][(2 * q + 1) % WORDS] = *reinterpret_cast<const uint4*>(&y);
        }
      } else {
        const uint4* f = reinterpret_cast<const uint4*>(mine + t * ROW_BYTES) + (BF16 ? 1 : 2) * b;  // (of either memory)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (PACKED) w[n][q] = f[4 * ((q + q0) & 3)];
          else if (BF16) {
            const uint4 x = f[4 * ((q + q0) & 3)];
            w[n][(2 * q) % WORDS] = make_uint4(x.x << 16, x.x & 0xffff0000u, x.y << 16, x.y & 0xffff0000u);
            w[n][(2 * q + 1) % WORDS] = make_uint4(x.z << 16, x.z & 0xffff0000u, x.w << 16, x.w & 0xffff0000u);
          } else {
            w[n][(2 * q) % WORDS] = f[8 * ((q + q0) & 3)];
            w[n][(2 * q + 1) % WORDS] = f[8 * ((q + q0) & 3) + 1];
          }
        }
      }
    }
    auto eight = [&](int n, int q, float (&x)[8]) {  // the q-th channels
      if (PACKED) unpack8(w[n][q], x);
      else {
        *reinterpret_cast<uint4*>(x) = w[n][(2 * q) % WORDS];
        *reinterpret_cast<uint4*>(x + 4) = w[n][(2 * q + 1) % WORDS];
      }
    };
    float most[ROUNDS];  // of each vector (the lanes of r have one)
    unsigned sick = 0;   // those that are not finite
#pragma unroll
    for (int n = 0; n < ROUNDS; ++n) {
      float m = 0.f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float x[8];
        eight(n, q, x);
#pragma unroll
        for (int e = 0; e < 8; e += 2) m = max3nan(m, fabsf(x[e]), fabsf(x[e + 1]));
      }
      m = max3nan(m, m, __shfl_xor_sync(FULL, m, 8));
      most[n] = max3nan(m, m, __shfl_xor_sync(FULL, m, 16));
      if (!(most[n] < INFINITY)) sick |= 1u << n;
    }
    if (lane == 0 && staged) bar_arrive(&sh.rempty[slot]);
    gr += staged;
#pragma unroll
    for (int n = 0; n < ROUNDS; ++n) {
      const int t = 8 * dw + r + 8 * N_DQ * n, k = place_of(t);
      uint8_t* to = plane + (values ? (k >> 3) * V_LEAD + (k & 7) * 16 : (uint32_t)((t >> 3) * 128 + (t & 7) * 16));
      float inv;
      const float s2 = pow2_of(most[n], inv);
      if (lane < 8) {
        float* col = reinterpret_cast<float*>(&sh.col[gt & 7][t]);
        if (!values) col[0] = s2;
        else col[1] = (float)((int)(__float_as_uint(s2) >> 23) - 127);
        if (sick >> n & 1) col[0] = NAN;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float x[8];
        eight(n, q, x);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split2(x[2 * e] * inv, x[2 * e + 1] * inv, hi[e], lo[e]);
        const int kg = 4 * ((q + q0) & 3) + b;
        uint8_t* o = to + kg * (values ? 128 : TILE * 16);
        *reinterpret_cast<uint4*>(o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if (FULL) *reinterpret_cast<uint4*>(o + (values ? LO_V : LO_K)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
    // A vector that is not finite counts as zero in the products, where rows that do not attend to it meet it too; those that do
    // get NaN by the keys' power of two.
    if (__any_sync(FULL, sick != 0)) {
#pragma unroll 1
      for (int i = 0; i < 4 * ROUNDS; ++i) {
        if (!(sick >> (i >> 2) & 1)) continue;
        const int t = 8 * dw + r + 8 * N_DQ * (i >> 2), k = place_of(t), kg = 4 * (i & 3) + b;
        uint8_t* o = plane + (values ? (k >> 3) * V_LEAD + (k & 7) * 16 + kg * 128 : (uint32_t)((t >> 3) * 128 + (t & 7) * 16) + kg * (TILE * 16));
        *reinterpret_cast<uint4*>(o) = make_uint4(0u, 0u, 0u, 0u);
        if (FULL) *reinterpret_cast<uint4*>(o + (values ? LO_V : LO_K)) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    return true;
  }

  // ---------------------------------------------------------------- softmax
  struct Row {
    float m, l;  // the reference of the weights' sum, that sum, of this group's tiles
    float R;     // the reference of the weights with their values' scales
  };
  // a larger logit, or logit with its value's scale, than the references allow for
  __device__ __forceinline__ void follow(Row& w, float mx, float rx) {
    if (mx > w.m + (BOOST + RAISE_AT)) {
      const float mnew = floorf(mx) - BOOST;
      w.l = w.m == -INFINITY ? w.l : w.l * ex2(w.m - mnew);
      w.m = mnew;
    }
    if (rx > w.R + (BOOST + RAISE_AT)) w.R = floorf(rx) - BOOST;
  }
  // The largest logit of a tile that every row attends to as a whole, and that of logits with their values' scales
  __device__ __forceinline__ void top_of(uint32_t sa, const float (&dk)[2], const float (&lv)[2], float& mx, float& rx) {
    mx = rx = -INFINITY;
#pragma unroll
    for (int c0 = 0; c0 < NT; c0 += 32) {
      float t = -INFINITY, v[32];
      tm_ld32(sa + c0, v);
#pragma unroll
      for (int i = 0; i < 32; i += 2) t = max3(t, v[i], v[i + 1]);
      t *= dk[c0 >> 5];
      mx = fmaxf(mx, t);
      rx = fmaxf(rx, t + lv[c0 >> 5]);
    }
  }
  // ... of columns first .. last of any other tile of nt, whose scales of columns c, c + 1 are at[(c >> 5) half + (c / 2 mod 16) step]
  __device__ __forceinline__ void top_of(uint32_t sa, const float4* at, int half, int step, int nt, float qs, int first, int last, float& mx,
                                         float& rx) {
    mx = rx = -INFINITY;
#pragma unroll 1
    for (int c0 = 0; c0 < nt; c0 += 32, at += half) {
      float v[32];
      tm_ld32(sa + c0, v);
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float4 s = at[step * (i / 2)];
        float x = v[i] * (s.x * qs), y = v[i + 1] * (s.z * qs);
        if (c0 + i < first || c0 + i > last) x = -INFINITY;
        if (c0 + i + 1 < first || c0 + i + 1 > last) y = -INFINITY;
        mx = max3(mx, x, y);
        rx = max3(rx, x + s.y, y + s.w);
      }
    }
  }
  // fp16 hi and lo of weights: hi is a weight's upper 11 bits, cut, lo the rest rounded to 11
  __device__ __forceinline__ static void halves_of(float x, float y, uint32_t& hi, uint32_t& lo) {
    const float hx = __uint_as_float(__float_as_uint(x) & 0xffffe000u), hy = __uint_as_float(__float_as_uint(y) & 0xffffe000u);
    sub2(x, y, hx, hy);
    hi = h2u(__floats2half2_rn(hx, hy));
    lo = h2u(__floats2half2_rn(x, y));
  }
  // The weights of a tile that a row attends to as a whole, each with its value's scale in the exponent: w' = 2^(l + lv - R); the
  // sum of a block's weights over 2^m is that of the w' times 2^(R - m - lv).  (A scale so small that its w' would be below 2^-80
  // counts as that: fp16 has no such numbers, but the sum does.)
  __device__ __forceinline__ void weigh(Row& w, uint32_t sa, const float (&dk)[2], const float (&lv)[2]) {
    const float R = w.R == -INFINITY ? w.m : w.R, Rm = R - w.m;
#pragma unroll 1
    for (int c0 = 0; c0 < NT; c0 += 32) {
      const float f = fmaxf(c0 ? lv[1] : lv[0], Rm - 100.f), k = c0 ? dk[1] : dk[0], b = f - R;
      float s0 = 0.f, s1 = 0.f, v[32];
      tm_ld32(sa + c0, v);
      // K-step by K-step of P V, in the order of the places
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        uint32_t pw[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = at_place(16 * ks + 2 * e);
          float x = v[c], y = v[c + 1];
          fma2(x, y, k, k, b, b);
          x = ex2(x);
          y = ex2(y);
          add2(s0, s1, x, y);
          halves_of(x, y, pw[e], pw[8 + e]);
        }
        tm_st16(sa + c0 + 16 * ks, pw);
      }
      w.l += (s0 + s1) * ex2(Rm - f);
    }
  }
  // ... of any other tile (scales as for top_of): weights and their sum each by its own exponent
  __device__ __forceinline__ void weigh(Row& w, uint32_t sa, const float4* at, int half, int step, int nt, float qs, int first, int last) {
    const float m0 = w.m == -INFINITY ? 0.f : w.m, R = w.R == -INFINITY ? m0 : w.R;
#pragma unroll 1
    for (int c0 = 0; c0 < nt; c0 += 32, at += half) {
      float s0 = 0.f, s1 = 0.f, v[32];
      tm_ld32(sa + c0, v);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        uint32_t pw[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = at_place(16 * ks + 2 * e);
          const float4 s = at[step * (c / 2)];
          const bool ox = c0 + c < first || c0 + c > last, oy = c0 + c + 1 < first || c0 + c + 1 > last;
          float x = v[c] * (s.x * qs), y = v[c + 1] * (s.z * qs);
          add2(s0, s1, ex2(ox ? -INFINITY : x - m0), ex2(oy ? -INFINITY : y - m0));
          x = ex2(ox ? -INFINITY : x + (s.y - R));
          y = ex2(oy ? -INFINITY : y + (s.w - R));
          halves_of(x, y, pw[e], pw[8 + e]);
        }
        tm_st16(sa + c0 + 16 * ks, pw);
      }
      w.l += s0 + s1;
    }
  }
  // a tile's reference, for whoever adds its P V
  __device__ __forceinline__ void leave(const Row& w, int row) { sh.mt[gt & 3][row] = w.R; }
  // its weights are in tensor memory
  __device__ __forceinline__ void hand_over(int grp) {
    tm_wait_st();
    fence_before();
    __syncwarp();
    if (lane == 0) bar_arrive(&sh.pfull[grp]);
  }
  // Little lives from tile to tile in registers (a tile takes most of them): the rest is read again from shared memory.
  __device__ void softmax(const Stretch& u) {
    const int grp = warp >> 2, row = 32 * (warp & 3) + lane;
    const uint32_t sa = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + C_S + NT * grp;
    // rows past the last query go along with it (and are not written)
    const int P = min(u.p0 + u.tl.t0 + row / a.g, u.tl.Pmax);
    Row w = {-INFINITY, 0.f, -INFINITY};
    const int first = u.ta + ((gt & 1) != grp), left = u.tb - u.ta;
    gt += first - u.ta;
    int it = first;
#pragma unroll 1
    while (it < u.tb) {
      // recorded tiles that every row attends to as a whole
      bool rec = false;
      float mx, rx;
      const int hi = P - a.W;  // the last recorded position that is attended to, as long as it is there
#pragma unroll 1
      for (; it < u.tb; it += 2, gt += 2) {
        if (!held(&sh.sfull[grp], (gt >> 1) & 1)) return;
        fence_after();
        rec = it < u.tl.nqt;
        const float4 s0 = sh.blk[gt & 7][0], s1 = sh.blk[gt & 7][1];
        // (the first tiles share references, and a page that is not there has scales of zero: below)
        if (!__all_sync(FULL, rec && it > u.ta + 1 && it * NT + NT - 1 <= hi && fmaxf(s0.y, s1.y) > -INFINITY)) break;
        const float qs = sh.qscale[row], dk[2] = {s0.x * qs, s1.x * qs}, lv[2] = {s0.y, s1.y};
        top_of(sa, dk, lv, mx, rx);
        follow(w, mx, rx);
        leave(w, row);
        weigh(w, sa, dk, lv);
        hand_over(grp);
      }
      if (it >= u.tb) break;
      // any other tile: columns first .. last are attended to
      int first, last, half = 1, step = 0, nt = NT;
      const float4* at = sh.blk[gt & 7];
      float qs;
      if (rec) {
        first = 0;
        last = page_bad(u, it) ? -1 : hi - it * NT;
        qs = sh.qscale[row];
      } else {
        if (!held(&sh.vfull[gt % NS], (gt / NS) & 1)) return;  // (all its powers of two are there)
        at = reinterpret_cast<const float4*>(sh.col[gt & 7]);
        half = NT / 4;
        step = 1;
        qs = sh.qraw[row];
        const int r = it - u.tl.nqt, j0 = u.tl.raw_at(r, RNT);
        first = hi + 1 - j0;
        nt = BF16 && r >= u.tl.n_full ? RNT : FULL_NT;
        last = min(P - j0, nt - 1);
      }
      top_of(sa, at, half, step, nt, qs, first, last, mx, rx);
      // The second group begins with the first one's reference: as long as neither moves, their parts add up as they are.
      if (it == u.ta + 1) {
        if (!held(&sh.begun[warp & 3], gb & 1)) return;
        w.R = sh.mt[(gt - 1) & 3][row];
      }
      follow(w, mx, rx);
      leave(w, row);
      if (it == u.ta && left > 1) {
        __syncwarp();
        if (lane == 0) bar_arrive(&sh.begun[warp & 3]);
      }
      weigh(w, sa, at, half, step, nt, qs, first, last);
      hand_over(grp);
      it += 2;
      gt += 2;
    }
    gb += left > 1;
    gt += left - (first - u.ta) - ((left - (first - u.ta) + 1) & ~1);  // tiles of the stretch, whoever softened them
    sh.m[grp][row] = w.m;
    sh.l[grp][row] = w.l;
  }
  __device__ __forceinline__ bool page_bad(const Stretch& u, int it) const {
    const int phys = __ldg(a.block_table + (size_t)u.b * a.max_pages_per_seq + it);
    return phys < 0 || phys >= a.L.n_pages;
  }

  // ---------------------------------------------------------------- the output
  // the accumulator from the values' quantised space to the heads': s . (c H (sigma . y))
  __device__ __forceinline__ void to_heads(float (&acc)[D], const Stretch& u) {
    if (a.sinkhorn) {
      const __half2* sig = reinterpret_cast<const __half2*>(a.p.sigv + ((size_t)u.layer * a.Hkv + u.h) * D);
#pragma unroll
      for (int i = 0; i < D; i += 2) {
        const float2 s = __half22float2(__ldg(sig + i / 2));
        mul2(acc[i], acc[i + 1], s.x, s.y);
      }
    }
#pragma unroll
    for (int i = 0; i < D; i += 2) {
      const float p = acc[i], q = acc[i + 1];
      acc[i] = p + q;
      acc[i + 1] = p - q;
    }
#pragma unroll
    for (int hs = 2; hs < D; hs <<= 1) {
#pragma unroll
      for (int i = 0; i < D; i += 2) {
        if (i & hs) continue;
        bfly2(acc[i], acc[i + 1], acc[i + hs], acc[i + hs + 1]);
      }
    }
#pragma unroll
    for (int i = 0; i < D; i += 4) {
      const float4 s = *reinterpret_cast<const float4*>(sh.signs + i);
      mul2(acc[i], acc[i + 1], C_WHT * s.x, C_WHT * s.y);
      mul2(acc[i + 2], acc[i + 3], C_WHT * s.z, C_WHT * s.w);
    }
  }
  __device__ __forceinline__ void free_output() {
    fence_before();
    __syncwarp();
    if (lane == 0) bar_arrive(&sh.ofree[gt & 1]);
  }
  // acc 2^M is the sum of weights times values so far, of both groups' tiles
  __device__ void sums(const Stretch& u) {
    const int row = 32 * (warp & 3) + lane;
    const uint32_t at = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + C_O;
    float acc[D];
#pragma unroll
    for (int i = 0; i < D; ++i) acc[i] = 0.f;
    float M = -INFINITY;
    int it = u.ta;
    // recorded tiles, then raw ones
#pragma unroll 1
    for (int part = 0; part < 2; ++part) {
      const int end = part ? u.tb : min(u.tb, u.tl.nqt);
#pragma unroll 1
      while (it < end) {
        float m;
        // tiles under the references of those before
#pragma unroll 1
        for (; it < end; ++it, ++gt) {
          if (!held(&sh.pvdone[gt & 1], (gt >> 1) & 1)) return;
          fence_after();
          m = sh.mt[gt & 3][row];
          if (__any_sync(FULL, m != M)) break;
          const uint32_t oa = at + D * (gt & 1);
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 32) {
            float o[32];
            tm_ld32(oa + c0, o);
#pragma unroll
            for (int i = 0; i < 32; i += 2) add2(acc[c0 + i], acc[c0 + i + 1], o[i], o[i + 1]);
          }
          free_output();
        }
        if (it >= end) break;
        const float Mn = fmaxf(M, m);
        // (where nothing was attended to the part is zero)
        const float fa = M == -INFINITY ? 1.f : ex2(M - Mn), fo = m == -INFINITY ? 1.f : ex2(m - Mn);
        M = Mn;
        const uint32_t oa = at + D * (gt & 1);
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 32) {
          float o[32];
          tm_ld32(oa + c0, o);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            mul2(o[i], o[i + 1], fo, fo);
            fma2(acc[c0 + i], acc[c0 + i + 1], fa, fa, o[i], o[i + 1]);
          }
        }
        free_output();
        ++it;
        ++gt;
      }
      if (part == 0 && it > u.ta) to_heads(acc, u);
    }
    // (no operand is in use any more: every product of the stretch has been waited for)
    float* o = reinterpret_cast<float*>(smem + (size_t)row * O_STRIDE);
#pragma unroll
    for (int i = 0; i < D; i += 4) *reinterpret_cast<float4*>(o + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
    sh.M[row] = M;
  }
  // rows to the output, or to a partial result: lane i & 15 knows of the warp's i-th row, then all write each row.  NaN where the CTA
  // has given up.
  __device__ void rows_out(const Stretch& u) {
    static_assert(ROWS == 16 * N_SOFT, "");
    const int g = a.g, nrows = u.tl.nq * g, lane = once(this->lane), warp = once(this->warp), row = warp + N_SOFT * (lane & 15);
    float* dst = a.parts + (size_t)max(u.rec, 0) * REC;
    const bool gone = sh.gone;
    float f = 0.f;
    if (row < nrows) {
      const float M = sh.M[row], m0 = sh.m[0][row], m1 = sh.m[1][row];
      // (alike whichever group had the first tile)
      const float m = fmaxf(m0, m1), l = __fadd_rn(__fmul_rn(sh.l[0][row], m0 == -INFINITY ? 1.f : ex2(m0 - m)),
                                                   __fmul_rn(sh.l[1][row], m1 == -INFINITY ? 1.f : ex2(m1 - m)));
      if (u.rec >= 0) {
        if (lane < 16) {
          dst[ROWS * D + row] = M;
          dst[ROWS * D + ROWS + row] = l;
          dst[ROWS * D + 2 * ROWS + row] = m;
        }
        f = 1.f;
        dst += row * D;
      } else {
        f = share_of(M - m, l);
        dst = a.out + (((size_t)u.unit * g + row % g) * a.T + u.tl.t0 + row / g) * D;
      }
      if (gone) f = NAN;
    }
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
      const float fi = __shfl_sync(FULL, f, i);
      float* to = reinterpret_cast<float*>(__shfl_sync(FULL, reinterpret_cast<unsigned long long>(dst), i));
      if (warp + N_SOFT * i < nrows) {
        const float4 o = *reinterpret_cast<const float4*>(smem + (size_t)(warp + N_SOFT * i) * O_STRIDE + 16 * lane);
        *reinterpret_cast<float4*>(to + 4 * lane) = make_float4(o.x * fi, o.y * fi, o.z * fi, o.w * fi);
      }
    }
  }

  // ---------------------------------------------------------------- a warp's life
  enum { SOFTMAX, SUMS, OPERANDS, LOGITS, VALUES, PAGES, AHEAD };
  template <int ROLE>
  __device__ void run() {
    stretches<ROLE>();
    // everything that a warp has issued lands before the columns are freed
    if (ROLE == LOGITS || ROLE == VALUES) {
      uint64_t* bar = &sh.done[ROLE - LOGITS];
      mma_commit(bar);
      bar_land(bar, 0);
    }
    if (ROLE == PAGES && sh.gone)
      for (int n = max(0, gr - RS); n < gr; ++n) bar_land(&sh.rfull[n % RS], (n / RS) & 1);
    fence_before();
    sync_all();
    if (ROLE == LOGITS) {
      fence_after();
      tm_free(tmem, TMEM_COLS);
    }
  }
  template <int ROLE>
  __device__ void stretches() {
#pragma unroll 1
    for (int k = 0;; ++k) {
      const Stretch& u = sh.at[k & 1];
      if (u.tb < 0) return;
      // (all threads agree: a wait that sets it is behind the barrier that all come to next)
      if (!*const_cast<volatile int*>(&sh.gone)) {
        if (ROLE == SOFTMAX) queries(u);
        sync_all();
        if (ROLE == SOFTMAX) queries_to_tmem();
        if (k == 0) asm volatile("griddepcontrol.wait;" ::: "memory");  // the call's tokens are appended, older ones copied
        fence_before();
        sync_all();
        fence_after();
        if (ROLE == SOFTMAX) softmax(u);
        if (ROLE == SUMS) sums(u);
        if (ROLE == OPERANDS) operands(u);
        if (ROLE == LOGITS) issue_logits(u);
        if (ROLE == VALUES) issue_values(u);
        if (ROLE == PAGES) fetch(u);
        // (the warp that has time keeps a limit below a sleep, with the stretch's first product)
        if (ROLE == AHEAD && a.wait_ns < NAP_NS) wait<false>(&sh.sfull[gt & 1], (gt >> 1) & 1, &sh.gone, a.p.status, a.wait_ns);
        if (ROLE == AHEAD) gt += u.tb - u.ta;
      }
      if (ROLE == AHEAD && lane == 0) {
        if (sh.whole) grab(-1, sh.at[(k + 1) & 1]);
        else follow_up(u, sh.at[(k + 1) & 1]);
      }
      sync_all();
      if (ROLE == SOFTMAX) rows_out(u);
      sync_all();
    }
  }
};

template <bool BF16>
__global__ void __launch_bounds__(THREADS, 1) prefill_block_kernel(const __grid_constant__ PrefillArgs a) {
  using K = Kernel<BF16>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ typename K::Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid < D) sh.signs[tid] = a.p.signs[tid];
  if (tid == 32) {
    for (int s = 0; s < NS; ++s) {
      bar_init(&sh.kfull[s], N_DQ);
      bar_init(&sh.kempty[s], 1);
      bar_init(&sh.vfull[s], N_DQ);
      bar_init(&sh.vempty[s], 1);
    }
    for (int i = 0; i < 4; ++i) bar_init(&sh.begun[i], 1);
    for (int i = 0; i < RS; ++i) {
      bar_init(&sh.rfull[i], 1);
      bar_init(&sh.rempty[i], N_DQ);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&sh.sfull[i], 1);
      bar_init(&sh.pfull[i], N_SOFT / 2);
      bar_init(&sh.pvdone[i], 1);
      bar_init(&sh.ofree[i], N_SUM);
      bar_init(&sh.done[i], 1);
    }
    sh.gone = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  plan(a, sh, gridDim.x, K::RNT);
  if (tid == NEXT_WARP * 32) a.keys[2 * blockIdx.x] = a.keys[2 * blockIdx.x + 1] = make_int2(-1, -1);
  // sequences that are not part of the call, or past capacity: zeros
  for (int b = 0; b < a.batch; ++b) {
    if (sh.p0[b] >= 0) continue;
    const size_t per = (size_t)a.Hkv * a.g * a.T * (D / 4);
    for (int ll = 0; ll < a.n_layers_call; ++ll) {
      float4* o = reinterpret_cast<float4*>(a.out) + ((size_t)ll * a.batch + b) * per;
      for (size_t i = (size_t)blockIdx.x * THREADS + tid; i < per; i += (size_t)gridDim.x * THREADS) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  if ((int)blockIdx.x >= sh.parts) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // (this grid ends after those before it)
    return;
  }
  if (warp == S_WARP) {
    tm_alloc(&sh.tmem, TMEM_COLS);
    fence_before();
  }
  __syncthreads();
  fence_after();
  if (tid == NEXT_WARP * 32) {
    K(a, sh, smem).locate(sh.at[0]);
  }
  __syncthreads();
  if (warp < N_SOFT) {
    take_registers<SOFT_REGS>();
    K(a, sh, smem).template run<K::SOFTMAX>();
  } else if (warp < DQ0) {
    take_registers<SUM_REGS>();
    K(a, sh, smem).template run<K::SUMS>();
  } else if (warp < S_WARP) {
    take_registers<DQ_REGS>();
    K(a, sh, smem).template run<K::OPERANDS>();
  } else {
    take_registers<ISSUE_REGS>();
    if (warp == S_WARP) K(a, sh, smem).template run<K::LOGITS>();
    else if (warp == PV_WARP) K(a, sh, smem).template run<K::VALUES>();
    else if (warp == PAGE_WARP) K(a, sh, smem).template run<K::PAGES>();
    else K(a, sh, smem).template run<K::AHEAD>();
  }
}

// Joins the partial results of the row tiles that a cut divides, a share of the rows a block.  Records stand in the order
// of the cost line (two a CTA: of the row tile that it begins in, of the one that it ends in), those of one row tile have
// its key.  Blocks (c, .) join the row tile whose first record is CTA c's: its last one, or no other is the first of its
// kind.  A warp joins a row.
constexpr int JOIN_SHARES = 8, JOIN_WARPS = ROWS / JOIN_SHARES, MAX_CTAS = 256;
static_assert(2 * MAX_CTAS <= JOIN_WARPS * 32, "a thread for each record");
__global__ void __launch_bounds__(JOIN_WARPS * 32) prefill_join_kernel(const __grid_constant__ PrefillArgs a, int ctas) {
  __shared__ int part[2 * MAX_CTAS], before[JOIN_WARPS + 1];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, g = a.g, qpt = ROWS / g;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int2 k0 = __ldcg(a.keys + 2 * blockIdx.x), k1 = __ldcg(a.keys + 2 * blockIdx.x + 1), key = k1.x >= 0 ? k1 : k0;
  const int2 k = t < 2 * ctas ? __ldcg(a.keys + t) : make_int2(-1, -1);
  if (key.x < 0) return;
  const bool mine = k.x == key.x && k.y == key.y;
  const unsigned same = __ballot_sync(FULL, mine);
  if (lane == 0) before[warp + 1] = __popc(same);
  __syncthreads();
  int at = 0, n = 0;
#pragma unroll
  for (int i = 0; i < JOIN_WARPS; ++i) {
    if (i < warp) at += before[i + 1];
    n += before[i + 1];
  }
  if (mine) part[at + __popc(same & ((1u << lane) - 1))] = t;
  __syncthreads();
  if (part[0] < 2 * (int)blockIdx.x) return;
  const int t0 = key.y * qpt, row = blockIdx.y * JOIN_WARPS + warp;
  if (row >= min(qpt, a.T - t0) * g) return;
  float M = -INFINITY, m = -INFINITY;
  for (int i = lane; i < n; i += 32) {
    const float* rec = a.parts + (size_t)part[i] * REC + ROWS * D + row;
    M = fmaxf(M, __ldcg(rec));
    m = fmaxf(m, __ldcg(rec + 2 * ROWS));
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    M = fmaxf(M, __shfl_xor_sync(FULL, M, o));
    m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
  }
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float* rec = a.parts + (size_t)part[i] * REC;
    const float* refs = rec + ROWS * D + row;
    const float Mi = __ldcg(refs), li = __ldcg(refs + ROWS), mi = __ldcg(refs + 2 * ROWS);
    const float4 x = __ldcg(reinterpret_cast<const float4*>(rec + row * D) + lane);
    const float f = Mi == -INFINITY ? 0.f : ex2(Mi - M);
    l += li * (mi == -INFINITY ? 0.f : ex2(mi - m));
    o.x += x.x * f;
    o.y += x.y * f;
    o.z += x.z * f;
    o.w += x.w * f;
  }
  const float f = share_of(M - m, l);
  *reinterpret_cast<float4*>(a.out + (((size_t)key.x * g + row % g) * a.T + t0 + row / g) * D + 4 * lane) =
      make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
}

template <bool BF16>
cudaError_t launch(const PrefillArgs& a, cudaStream_t s) {
  const int sms = a.sms;
  cudaError_t e = allow_shared_memory<prefill_block_kernel<BF16>>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // (a dependent of the append: it has its queries by the time that the append ends)
  if ((e = cudaLaunchKernelEx(&cfg, prefill_block_kernel<BF16>, a)) != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)sms, JOIN_SHARES);
  cfg.blockDim = dim3(JOIN_WARPS * 32);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, prefill_join_kernel, a, sms);
}

}  // namespace

size_t prefill_block_scratch_bytes(int sms) { return (size_t)2 * sms * (REC * sizeof(float) + sizeof(int2)) + 16; }

void prefill_block_places(PrefillArgs* a) {
  a->sms = a->sms < MAX_CTAS ? a->sms : MAX_CTAS;
  a->keys = reinterpret_cast<int2*>(a->parts + (size_t)2 * a->sms * REC);
  a->taken = reinterpret_cast<int*>(a->keys + (size_t)2 * a->sms);
}

cudaError_t launch_prefill_blocks(const PrefillArgs& a, cudaStream_t s) { return a.in_bf16 ? launch<true>(a, s) : launch<false>(a, s); }

}  // namespace kvq

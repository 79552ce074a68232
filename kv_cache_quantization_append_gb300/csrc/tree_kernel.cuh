// Tree attention: the kernels of one key format (included by one translation unit per format).
//
// A unit's rows (query heads of its nodes, node-major: row = node * g + head) are the N side of the products and
// its positions the M side, so that the tensor cores do work for the rows there are (16 to 64 a CTA, more rows in
// further CTAs) and a position's scales and norms belong to one thread:
//   S^T [128 positions x N rows]  = K~ [128 x 128] Q~^T         (tcgen05.mma, both operands in shared memory)
//   O^T [128 channels x N rows] += V~^T [128 x 128] P^T
// in the quantised records' space (rotated, balanced), where K~ and V~ are the dequantised records, or the window's
// and the drafts' raw vectors taken there once by the first kernel.  The softmax runs in base 2 down a thread's own
// columns against a reference per row that moves only when a logit passes it by 8 (weights stay below 2^8 in fp16):
// no exchange between threads but one vote per tile.
//
// Three launches, each the programmatic dependent of the one before:
//  1. tree_prep_kernel: rotated queries (and their QJL projections) as operand images, the raw tiles' images, and
//     every node's ancestors and depth.
//  2. tree_kernel: the tiles of all units in one list, cut into equal ranges, one per CTA (stream-K).  All warps of a
//     CTA dequantise K~, then V~ while the tensor cores run the logits, then take the softmax, then go on to the next
//     K~ while the tensor cores run P V: the CUDA cores never wait for the products, and two CTAs an SM fill each
//     other's barriers.  A range's part of a unit ends as one partial record (reference, sum, O).
//  3. tree_merge_kernel: joins a row's records in a fixed order, undoes the balancing and the rotation.
//
// Operands: bf16 caches take each of K~, V~, Q~ and P rounded once to fp16 (2^-11, an eighth of the bf16 output's own
// rounding step); float caches split each into fp16 hi and lo and run hi hi + hi lo + lo hi (22 bits).  TQ3 keys need
// no rounding: the centroids and the signs are exact, their two products go to two accumulators, and the thread that
// owns the position joins them as n (S1 + w S2).
#pragma once

#include "tc.cuh"

namespace kvq {
namespace tree {

using namespace tc;

constexpr int TILE = 128;     // positions per tile = MMA M
constexpr int THREADS = 256;
constexpr int MAX_ROWS = 64;  // rows per CTA
constexpr int MERGE_WARPS = 8;
constexpr float NO_REF = -1e30f;  // reference of a row that has met no position yet

// what the launches share: sizes from the host, pointers into the caller's scratch
struct Plan {
  MultiArgs a;
  int rb, N, n_units, G, raw_tiles;  // row blocks of N rows per unit, units (with row blocks), CTAs, raw tiles at most
  int q_image, raw_image;            // bytes: of a row block's queries, of one raw tile (K then V)
  unsigned long long* anc;           // [batch][n] ancestors-or-self, 0: not there
  uint8_t* q_images;                 // [n_units][q_image]
  uint8_t* raw_images;               // [n_units / rb][raw_tiles][raw_image]
  float* records;                    // [n_units + G][2 N + 128 N]
};

__host__ __device__ inline int raw_count(int L, int W, int n) { return (W > 0 ? (L < W - 1 ? L : W - 1) : 0) + n; }
// positions below this may be read through their records by some node (the deepest is at L + n - 1)
__host__ __device__ inline int quant_end(int L, int W, int n) {
  if (W <= 0) return L;
  const int e = L - W + n;
  return e < 0 ? 0 : e > L ? L : e;
}
__device__ __forceinline__ int seq_len(const MultiArgs& a, int b) {
  const int L = a.seq_lens[b];
  return L < 0 || L > a.max_seq_len ? 0 : L;
}
__device__ __forceinline__ int seq_tiles(const MultiArgs& a, int L) {
  return (quant_end(L, a.W, a.n) + TILE - 1) / TILE + (raw_count(L, a.W, a.n) + TILE - 1) / TILE;
}
// warp 0: exclusive prefix of the sequences' tiles, [batch + 1]
__device__ __forceinline__ void tile_prefix(const MultiArgs& a, int* pre) {
  const int lane = threadIdx.x & 31, per = (a.batch + 31) / 32;
  const int b0 = min(a.batch, lane * per), b1 = min(a.batch, b0 + per);
  int s = 0;
  for (int b = b0; b < b1; ++b) s += seq_tiles(a, seq_len(a, b));
  int incl = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(FULL, incl, o);
    if (lane >= o) incl += y;
  }
  int run = incl - s;
  for (int b = b0; b < b1; ++b) {
    pre[b] = run;
    run += seq_tiles(a, seq_len(a, b));
  }
  if (lane == 31) pre[a.batch] = incl;
}

template <int KF, bool F32>
struct Cfg {
  static constexpr bool TQ = KF == KVQ_TQ3_QJL;
  static constexpr int PL = F32 ? 2 : 1;            // fp16 planes per value
  static constexpr int KD = TQ ? 256 : 128;         // width of a query image: [q~] or [q~, S q~]
  static constexpr uint32_t PLANE = TILE * D * 2;   // 32 KB
  // place of channel c within its group of eight, for the key side (values: always nibble_place)
  __host__ __device__ static constexpr int k_place(int c) { return KF == KVQ_Q4G32 ? nibble_place(c) : c; }
};

// byte offset of (row, k) in a K-major operand of R rows
__host__ __device__ constexpr uint32_t km_off(int row, int k, int R) {
  return (uint32_t)((k >> 3) * (R >> 3) * 128 + (row >> 3) * 128 + (row & 7) * 16 + (k & 7) * 2);
}
// byte offset of (m, k) in an M-major operand of 128 m
__host__ __device__ constexpr uint32_t mm_off(int m, int k) {
  return (uint32_t)((k >> 3) * 2048 + (m >> 3) * 128 + (k & 7) * 16 + (m & 7) * 2);
}

// ------------------------------------------------------------------ 1. prep
template <int KF, bool F32>
__global__ void __launch_bounds__(THREADS) tree_prep_kernel(const __grid_constant__ Plan p) {
  using C = Cfg<KF, F32>;
  constexpr int RPW = C::TQ ? 4 : 1;  // query rows per warp: a pass over the projection serves four
  const MultiArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;");
  if ((int)blockIdx.x < a.batch) {
    // ancestors of every node of one sequence
    __shared__ int par[KVQ_MAX_TREE];
    const int b = blockIdx.x, i = threadIdx.x;
    if (i < a.n) par[i] = a.parents[(size_t)b * a.n + i];
    if (i == 0) {
      const int L = a.seq_lens[b];
      if (L < 0 || L > a.max_seq_len) atomicOr(a.p.status, KVQ_DEV_SEQLEN_RANGE);
    }
    __syncthreads();
    if (i < a.n) {
      unsigned long long m = 0;
      for (int j = i; j >= 0;) {
        m |= 1ull << j;
        const int q = par[j];
        if (q < -1 || q >= j) {
          if (q >= j) atomicOr(a.p.status, KVQ_DEV_BAD_NODE);
          m = 0;
          break;
        }
        j = q;
      }
      p.anc[(size_t)b * a.n + i] = m;
    }
    return;
  }
  const long long item = (long long)(blockIdx.x - a.batch) * (THREADS / 32) + warp;
  const int H = a.Hkv, B = a.batch, rows = a.n * a.g;
  const long long q_items = (long long)p.n_units * (p.N / RPW);
  const float4 sg = *reinterpret_cast<const float4*>(a.p.signs + 4 * lane);
  // is node i of sequence b there? (its chain of parents, two to a lane, walked by the whole warp)
  auto there = [&](int b, int i) {
    const int* par = a.parents + (size_t)b * a.n;
    const int lo = lane < a.n ? par[lane] : -2, hi = lane + 32 < a.n ? par[lane + 32] : -2;
    for (int j = i; j >= 0;) {
      const int x = __shfl_sync(FULL, lo, j & 31), y = __shfl_sync(FULL, hi, j & 31);
      const int q = j < 32 ? x : y;
      if (q < -1 || q >= j) return false;
      j = q;
    }
    return true;
  };
  if (item < q_items) {
    const int u = (int)(item / (p.N / RPW)), r0 = (int)(item % (p.N / RPW)) * RPW;
    const int rbi = u % p.rb, h = (u / p.rb) % H, b = (u / (p.rb * H)) % B, ll = u / (p.rb * H * B);
    uint8_t* img = p.q_images + (size_t)u * p.q_image;
    float y[RPW][4];
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
      const int row = rbi * p.N + r0 + r, node = row / a.g;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < rows && there(b, node))  // a node that is not there may hold anything
        x = load4_in(a.q, ((((size_t)ll * B + b) * H * a.g + (size_t)h * a.g + row % a.g) * a.n + node) * D + 4 * lane, a.in_bf16);
      y[r][0] = x.x * sg.x;
      y[r][1] = x.y * sg.y;
      y[r][2] = x.z * sg.z;
      y[r][3] = x.w * sg.w;
      hadamard_warp(y[r][0], y[r][1], y[r][2], y[r][3], lane);
      const __half* sig = a.p.sigk + ((size_t)(a.layer0 + ll) * H + h) * D + 4 * lane;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[r][e] *= C_WHT * LOGIT_SCALE;
        if (a.sinkhorn) y[r][e] *= __half2float(sig[e]);
      }
    }
    const auto put = [&](int r, int c, float v) {
      const __half hi = __float2half_rn(v);
      const uint32_t off = km_off(r, (c & ~7) + C::k_place(c & 7), p.N);
      *reinterpret_cast<__half*>(img + off) = hi;
      if (F32) *reinterpret_cast<__half*>(img + p.N * C::KD * 2 + off) = __float2half_rn(v - __half2float(hi));
    };
#pragma unroll
    for (int r = 0; r < RPW; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) put(r0 + r, 4 * lane + e, y[r][e]);
    if (C::TQ) {
      // projections 4 lane .. + 3 of S q~ (the stored projection is transposed: row j is column j of S)
      float acc[RPW][4] = {};
#pragma unroll 4
      for (int j = 0; j < D; j += 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 s4 = *reinterpret_cast<const float4*>(a.p.qjl_t + (j + e) * D + 4 * lane);
#pragma unroll
          for (int r = 0; r < RPW; ++r) {
            const float qj = __shfl_sync(FULL, y[r][e], j >> 2);
            acc[r][0] += s4.x * qj;
            acc[r][1] += s4.y * qj;
            acc[r][2] += s4.z * qj;
            acc[r][3] += s4.w * qj;
          }
        }
      }
#pragma unroll
      for (int r = 0; r < RPW; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) put(r0 + r, D + 4 * lane + e, acc[r][e]);
    }
    return;
  }
  // raw vectors: x = 0 .. 128 raw_tiles - 1 of each unit's list, K and V
  const long long rest = item - q_items;
  const int per_unit = p.raw_tiles * TILE;
  const long long vec = rest >> 1;
  if (vec >= (long long)(p.n_units / p.rb) * per_unit) return;
  const int kv = (int)(rest & 1), x = (int)(vec % per_unit), u = (int)(vec / per_unit);
  const int h = u % H, b = (u / H) % B, ll = u / (H * B), layer = a.layer0 + ll;
  const int L = seq_len(a, b), nraw = raw_count(L, a.W, a.n), nring = nraw - a.n;
  if (x >= (nraw + TILE - 1) / TILE * TILE) return;  // a tile that this sequence does not have
  float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
  if (x < nring) {
    const float* ring = kv ? a.p.ringv : a.p.ringk;
    w = *reinterpret_cast<const float4*>(ring + ((((size_t)layer * a.max_batch + b) * H + h) * a.W + (L - nring + x) % a.W) * D + 4 * lane);
  } else if (x < nraw && there(b, x - nring)) {
    w = load4_in(kv ? a.v : a.k, ((((size_t)ll * B + b) * H + h) * a.n + x - nring) * D + 4 * lane, a.in_bf16);
  }
  float y[4] = {w.x * sg.x, w.y * sg.y, w.z * sg.z, w.w * sg.w};
  hadamard_warp(y[0], y[1], y[2], y[3], lane);
  const __half* sig = (kv ? a.p.sigv : a.p.sigk) + ((size_t)layer * H + h) * D + 4 * lane;
  uint8_t* img = p.raw_images + ((size_t)u * p.raw_tiles + x / TILE) * p.raw_image + (kv ? C::PL * C::PLANE : 0);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float v = y[e] * C_WHT;
    if (a.sinkhorn) v = __fdiv_rn(v, __half2float(sig[e]));
    const int c = 4 * lane + e, t = x % TILE;
    const uint32_t off = kv ? mm_off((c & ~7) + nibble_place(c & 7), t) : km_off(t, (c & ~7) + C::k_place(c & 7), TILE);
    const __half hi = __float2half_rn(v);
    *reinterpret_cast<__half*>(img + off) = hi;
    if (F32) *reinterpret_cast<__half*>(img + C::PLANE + off) = __float2half_rn(v - __half2float(hi));
  }
}

// ------------------------------------------------------------------ dequantising
// one tile's words of this thread: keys of position t = tid & 127 (half tid >> 7 of its record), values of the
// position pair vp and rows 2 vr, 2 vr + 1
template <int KF>
struct Words {
  uint4 k[KF == KVQ_Q8G32 ? 4 : 2];
  uint4 km;         // Q4: scales and zeros
  uint32_t kx;      // Q8: two scales; TQ: (norm, residual norm)
  uint4 v[2];
  uint32_t vs[4], vz[4];
};

struct Lane {
  int t, hf, vp, vr;
};
__device__ __forceinline__ Lane lane_of(int tid) {
  // values: 8 consecutive lanes write 8 distinct 16-byte slots of their core matrices (the odd rows' lanes take the odd
  // position of the pair first)
  return {tid & 127, tid >> 7, (tid & 3) | ((tid >> 2) & 4) | ((tid >> 2) & 56), (tid >> 2) & 3};
}

// physical pages of a tile (-1: out of range or past the end)
struct Pages {
  int p[2];
};

template <int KF>
__device__ __forceinline__ void load_k(const MultiArgs& a, const uint8_t* unit_pages, size_t page_stride, const Pages& pg,
                                       const Lane& ln, Words<KF>& w) {
  const int tt = ln.t & 31, phys = ln.t & 64 ? pg.p[1] : pg.p[0];
#pragma unroll
  for (int i = 0; i < (KF == KVQ_Q8G32 ? 4 : 2); ++i) w.k[i] = make_uint4(0u, 0u, 0u, 0u);
  w.km = make_uint4(0u, 0u, 0u, 0u);
  w.kx = 0u;
  if (phys < 0) return;
  const uint8_t* hb = unit_pages + (size_t)phys * page_stride + (size_t)((ln.t >> 5) & 1) * a.L.half_bytes;
  if (KF == KVQ_Q8G32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w.k[i] = __ldg(reinterpret_cast<const uint4*>(hb + tt * 128 + 16 * ((2 * i + ln.hf) ^ (tt & 1))));
    w.kx = __ldg(reinterpret_cast<const uint32_t*>(hb + a.L.off_kmeta + tt * 8) + ln.hf);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) w.k[i] = __ldg(reinterpret_cast<const uint4*>(hb + tt * 64 + 32 * ln.hf) + i);
    if (KF == KVQ_Q4G32) {
      w.km = __ldg(reinterpret_cast<const uint4*>(hb + a.L.off_kmeta + tt * 16));
    } else {
      const unsigned short* m = reinterpret_cast<const unsigned short*>(hb + a.L.off_kmeta);
      w.kx = (uint32_t)__ldg(m + tt) | ((uint32_t)__ldg(m + HALF + tt) << 16);
    }
  }
}

template <int KF>
__device__ __forceinline__ void load_v(const MultiArgs& a, const uint8_t* unit_pages, size_t page_stride, const Pages& pg,
                                       const Lane& ln, Words<KF>& w) {
  const int phys = ln.vp & 32 ? pg.p[1] : pg.p[0], pp = ln.vp & 15;
#pragma unroll
  for (int i = 0; i < 2; ++i) w.v[i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = 0; i < 4; ++i) w.vs[i] = w.vz[i] = 0u;
  if (phys < 0) return;
  const uint8_t* hb = unit_pages + (size_t)phys * page_stride + (size_t)((ln.vp >> 4) & 1) * a.L.half_bytes;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w.v[i] = __ldg(reinterpret_cast<const uint4*>(hb + a.L.off_vmain + 128 * pp + 16 * ((2 * ln.vr + i + 2 * (pp & 3)) & 7)));
  const uint32_t* m = reinterpret_cast<const uint32_t*>(hb + a.L.off_vmeta) + pp;
#pragma unroll
  for (int G = 0; G < 4; ++G) {
    w.vs[G] = __ldg(m + 16 * G);
    w.vz[G] = __ldg(m + 64 + 16 * G);
  }
}

__device__ __forceinline__ uint32_t dup_lo(uint32_t x) { return __byte_perm(x, x, 0x1010); }
__device__ __forceinline__ uint32_t dup_hi(uint32_t x) { return __byte_perm(x, x, 0x3232); }

// eight codes of a word times scale plus zero, as one 16-byte chunk (and its lo part)
template <bool F32>
__device__ __forceinline__ void put_nibbles(uint8_t* dst, uint32_t plane, uint32_t word, uint32_t s2, uint32_t z2) {
  __half2 c[4];
  nibbles(word, c);
  uint4 o, l;
  if (!F32) {
    o.x = h2u(__hfma2(c[0], u2h(s2), u2h(z2)));
    o.y = h2u(__hfma2(c[1], u2h(s2), u2h(z2)));
    o.z = h2u(__hfma2(c[2], u2h(s2), u2h(z2)));
    o.w = h2u(__hfma2(c[3], u2h(s2), u2h(z2)));
  } else {
    const float s = __low2float(u2h(s2)), z = __low2float(u2h(z2));
    const float2 f0 = __half22float2(c[0]), f1 = __half22float2(c[1]), f2 = __half22float2(c[2]), f3 = __half22float2(c[3]);
    split2(z + s * f0.x, z + s * f0.y, o.x, l.x);
    split2(z + s * f1.x, z + s * f1.y, o.y, l.y);
    split2(z + s * f2.x, z + s * f2.y, o.z, l.z);
    split2(z + s * f3.x, z + s * f3.y, o.w, l.w);
    *reinterpret_cast<uint4*>(dst + plane) = l;
  }
  *reinterpret_cast<uint4*>(dst) = o;
}

// keys of the thread's position (TQ3: the exact centroids)
template <int KF, bool F32>
__device__ __forceinline__ void put_k(uint8_t* kb, const Lane& ln, const Words<KF>& w, const uint4& cent) {
  constexpr uint32_t PLANE = Cfg<KF, F32>::PLANE;
  uint8_t* dst = kb + km_off(ln.t, 0, TILE);
  if (KF == KVQ_Q4G32) {
    const uint32_t sc[2] = {w.km.x, w.km.y}, zr[2] = {w.km.z, w.km.w};
#pragma unroll
    for (int G = 0; G < 4; ++G) {
      const uint32_t s2 = G & 1 ? dup_hi(sc[G >> 1]) : dup_lo(sc[G >> 1]), z2 = G & 1 ? dup_hi(zr[G >> 1]) : dup_lo(zr[G >> 1]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t word = G == 0 ? w.k[i].x : G == 1 ? w.k[i].y : G == 2 ? w.k[i].z : w.k[i].w;
        put_nibbles<F32>(dst + (4 * G + 2 * ln.hf + i) * 2048, PLANE, word, s2, z2);
      }
    }
  } else if (KF == KVQ_Q8G32) {
    const __half2 off = u2h(0x64806480u);  // 1024 + 128
#pragma unroll
    for (int wi = 0; wi < 4; ++wi) {
      const uint32_t s2 = wi & 2 ? dup_hi(w.kx) : dup_lo(w.kx);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t o[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t word = wi == 0 ? w.k[i].x : wi == 1 ? w.k[i].y : wi == 2 ? w.k[i].z : w.k[i].w;
          const __half2 c = __hsub2(u2h(__byte_perm(word, 0x64646464u, x ? 0x4342 : 0x4140)), off);
          if (F32) {
            const float d = __low2float(u2h(s2));
            const float2 f = __half22float2(c);
            split2(d * f.x, d * f.y, o[i], l[i]);
          } else {
            o[i] = h2u(__hmul2(c, u2h(s2)));
          }
        }
        uint8_t* at = dst + (2 * (4 * ln.hf + wi) + x) * 2048;
        *reinterpret_cast<uint4*>(at) = make_uint4(o[0], o[1], o[2], o[3]);
        if (F32) *reinterpret_cast<uint4*>(at + PLANE) = make_uint4(l[0], l[1], l[2], l[3]);
      }
    }
  } else {
    // the eight centroids' bytes in two register pairs (low bytes: cent.x, .y; high bytes: cent.z, .w), picked by
    // byte permutes with the codes as selectors
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4& q = w.k[i >> 2];
      const uint32_t word = (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
      const uint32_t sel = (word & 0x07070707u) | ((word << 1) & 0x70707070u);
      const uint32_t l0 = __byte_perm(cent.x, cent.y, sel), h0 = __byte_perm(cent.z, cent.w, sel);
      const uint32_t l1 = __byte_perm(cent.x, cent.y, sel >> 16), h1 = __byte_perm(cent.z, cent.w, sel >> 16);
      *reinterpret_cast<uint4*>(dst + (8 * ln.hf + i) * 2048) =
          make_uint4(__byte_perm(l0, h0, 0x5140), __byte_perm(l0, h0, 0x7362), __byte_perm(l1, h1, 0x5140), __byte_perm(l1, h1, 0x7362));
    }
  }
}

// TQ3: the signs of the residual's projections, exactly +-1 (bit 6: projection 2j, bit 7: 2j + 1; set: +1)
__device__ __forceinline__ void put_signs(uint8_t* kb, const Lane& ln, const Words<KVQ_TQ3_QJL>& w) {
  uint8_t* dst = kb + km_off(ln.t, 0, TILE);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint4& q = w.k[i >> 2];
    const uint32_t hi = (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
    const uint32_t lo = hi << 1;  // bit 6 of each byte to its top
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // bytes 1 and 3: all ones where the bit is set (a permute that spreads the sign bit)
      const uint32_t sel = (uint32_t)((8 + k) << 4) | (uint32_t)((12 + k) << 12);
      uint32_t m;
      asm("prmt.b32 %0, %1, %2, %3;" : "=r"(m) : "r"(lo), "r"(hi), "r"(sel));
      o[k] = 0xBC00BC00u ^ (m & 0x80008000u);
    }
    *reinterpret_cast<uint4*>(dst + (8 * ln.hf + i) * 2048) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// values of the thread's two positions, eight channels of each group; positions from `left` on (of the pair) are zero
template <int KF, bool F32>
__device__ __forceinline__ void put_v(uint8_t* vb, const Lane& ln, const Words<KF>& w, int left) {
  constexpr uint32_t PLANE = Cfg<KF, F32>::PLANE;
  const uint32_t keep = left >= 2 ? 0xffffffffu : left == 1 ? 0x0000ffffu : 0u;  // (records there may hold anything)
#pragma unroll
  for (int G = 0; G < 4; ++G) {
    const uint32_t w0 = G == 0 ? w.v[0].x : G == 1 ? w.v[0].y : G == 2 ? w.v[0].z : w.v[0].w;
    const uint32_t w1 = G == 0 ? w.v[1].x : G == 1 ? w.v[1].y : G == 2 ? w.v[1].z : w.v[1].w;
    const uint32_t vs = w.vs[G] & keep, vz = w.vz[G] & keep;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = i ^ (ln.vr & 1);
      const uint32_t word = __byte_perm(w0, w1, e ? 0x7531 : 0x6420);
      put_nibbles<F32>(vb + mm_off(32 * G + 8 * ln.vr, 2 * ln.vp + e), PLANE, word, e ? dup_hi(vs) : dup_lo(vs),
                       e ? dup_hi(vz) : dup_lo(vz));
    }
  }
}

// ------------------------------------------------------------------ 2. the tiles
// dynamic shared memory: K planes | V planes | query image | P planes | small state.  TQ3 keys, whose query image is
// twice as wide, take the weights P into the key buffer (free once the logits are done), so that two CTAs of 64 rows fit
// an SM; their next keys then wait for P V.
template <int KF, bool F32>
struct Smem {
  using C = Cfg<KF, F32>;
  static constexpr bool P_IN_K = C::TQ;
  static constexpr uint32_t K = 0, V = C::PL * C::PLANE, Q = 2 * C::PL * C::PLANE;
  static __host__ __device__ constexpr uint32_t P(int N) { return P_IN_K ? K : Q + N * C::KD * 2 * C::PL; }
  static __host__ __device__ constexpr uint32_t total(int N) {
    return Q + N * C::KD * 2 * C::PL + (P_IN_K ? 0 : N * TILE * 2 * C::PL);
  }
};

template <int KF, int NH, bool F32>
__global__ void __launch_bounds__(THREADS, F32 ? 1 : 2) tree_kernel(const __grid_constant__ Plan p) {
  using C = Cfg<KF, F32>;
  using SM = Smem<KF, F32>;
  constexpr int N = 2 * NH;
  constexpr bool TQ = C::TQ;
  constexpr uint32_t S_COLS = TQ ? 2 * N : N, C_O = S_COLS;
  constexpr uint32_t TM_COLS = S_COLS + N <= 32 ? 32 : S_COLS + N <= 64 ? 64 : S_COLS + N <= 128 ? 128 : 256;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t qk_bar, pv_bar, load_bar;
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh;
  __shared__ float mref[N], wmax[4][N];
  __shared__ int lim[N];
  __shared__ unsigned long long anc[N];
  const MultiArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int* pre = reinterpret_cast<int*>(smem + SM::total(N));

  if (tid == 0) {
    bar_init(&qk_bar, 1);
    bar_init(&pv_bar, 1);
    bar_init(&load_bar, 1);
    abort_sh = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) tile_prefix(a, pre);
  if (warp == 1) tm_alloc(&tmem_sh, TM_COLS);
  fence_before();
  asm volatile("griddepcontrol.launch_dependents;");
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_sh;
  const uint32_t sbase = smem_u32(smem);

  // this CTA's range of the list of tiles
  const long long per_layer = (long long)pre[a.batch] * a.Hkv * p.rb, total = per_layer * a.n_layers_call;
  const long long G = min((long long)p.G, total);  // no range is empty: the merge reads every range between a unit's ends
  long long t = blockIdx.x < G ? total * blockIdx.x / G : 0;
  const long long t_end = blockIdx.x < G ? total * (blockIdx.x + 1) / G : 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const Lane ln = lane_of(tid);
  const size_t page_stride = (size_t)a.Hkv * a.L.page_bytes;
  uint4 cent = make_uint4(0u, 0u, 0u, 0u);
  if (TQ) {
    const uint4 c = *reinterpret_cast<const uint4*>(a.p.cb->cent);
    cent.x = __byte_perm(c.x, c.y, 0x6420);
    cent.y = __byte_perm(c.z, c.w, 0x6420);
    cent.z = __byte_perm(c.x, c.y, 0x7531);
    cent.w = __byte_perm(c.z, c.w, 0x7531);
  }
  uint32_t qk_phase = 0, pv_phase = 0, load_phase = 0;
  bool pv_pending = false;
  const int col0 = (warp >> 2) * NH;                                  // this thread's columns (rows of the unit)
  const uint32_t lane_addr = tmem + ((uint32_t)(32 * (warp & 3)) << 16);  // its tensor-memory lane: position ln.t, channel ln.t
  bool ok = true;

  while (t < t_end && ok) {
    // ---- the next unit: its sequence, head and row block, and this CTA's tiles of it
    const int ll = (int)(t / per_layer);
    const long long in_layer = t - ll * per_layer;
    int lo = 0, hi = a.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((long long)pre[mid] * a.Hkv * p.rb <= in_layer) lo = mid;
      else hi = mid - 1;
    }
    const int b = lo, tiles = pre[b + 1] - pre[b];
    const long long r = in_layer - (long long)pre[b] * a.Hkv * p.rb;
    const int hr = (int)(r / tiles), it0 = (int)(r - (long long)hr * tiles);
    const int h = hr / p.rb, rbi = hr - h * p.rb;
    const int it1 = (int)min((long long)tiles, it0 + (t_end - t));
    const int u = ((ll * a.batch + b) * a.Hkv + h) * p.rb + rbi;
    const int L = seq_len(a, b), qend = quant_end(L, a.W, a.n), nq = (qend + TILE - 1) / TILE;
    const int nraw = raw_count(L, a.W, a.n), nring = nraw - a.n;
    const int full_end = a.W > 0 ? L - a.W + 1 : L;  // positions below are read through records by every node
    const uint8_t* unit_pages = a.p.pages + ((size_t)(a.layer0 + ll) * a.L.n_pages * a.Hkv + h) * (size_t)a.L.page_bytes;
    const int* bt = a.block_table + (size_t)b * a.max_pages_per_seq;
    const auto pages_of = [&](int it) {
      Pages g;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = it * TILE + i * PAGE;
        const int x = it < nq && j < qend ? __ldg(bt + j / PAGE) : -1;
        g.p[i] = x < a.L.n_pages ? x : -1;
        if (it < nq && j < qend && (x < 0 || x >= a.L.n_pages) && tid == 0) atomicOr(a.p.status, KVQ_DEV_BAD_PAGE);
      }
      return g;
    };
    Words<KF> w;
    Pages pg = pages_of(it0), pg1 = pages_of(it0 + 1);
    load_k<KF>(a, unit_pages, page_stride, pg, ln, w);
    load_v<KF>(a, unit_pages, page_stride, pg, ln, w);
    if (tid == 0) {
      bar_expect(&load_bar, (uint32_t)p.q_image);
      bulk_g2s(smem + SM::Q, p.q_images + (size_t)u * p.q_image, (uint32_t)p.q_image, &load_bar);
    }
    if (tid < N) {
      const int row = rbi * N + tid, node = row / a.g;
      const unsigned long long m = row < a.n * a.g ? p.anc[(size_t)b * a.n + node] : 0ull;
      anc[tid] = m;
      mref[tid] = NO_REF;
      lim[tid] = m ? (a.W > 0 ? min(L - 1, L + __popcll(m) - 1 - a.W) : L - 1) : -1;
    }
    float l[NH];
#pragma unroll
    for (int c = 0; c < NH; ++c) l[c] = 0.f;
    bar_wait(&load_bar, load_phase, &abort_sh, a.p.status);
    load_phase ^= 1;

    for (int it = it0; it < it1; ++it) {
      const bool raw = it >= nq;
      const auto wait_pv = [&] {
        if (pv_pending) {
          bar_wait(&pv_bar, pv_phase, &abort_sh, a.p.status);
          pv_phase ^= 1;
          pv_pending = false;
        }
      };
      // ---- keys (the previous tile's logits are done: its softmax has read them)
      if (SM::P_IN_K) wait_pv();
      uint32_t ng = 0;  // TQ3: norm and residual norm of this thread's position
      bool valid = true;
      if (!raw) {
        put_k<KF, F32>(smem + SM::K, ln, w, cent);
        ng = w.kx;
        valid = (ln.t & 64 ? pg.p[1] : pg.p[0]) >= 0;
        fence_async_smem();
      } else {
        const uint8_t* img = p.raw_images + ((size_t)(u / p.rb) * p.raw_tiles + (it - nq)) * p.raw_image;
        if (tid == 0) {
          bar_expect(&load_bar, C::PL * C::PLANE);
          bulk_g2s(smem + SM::K, img, C::PL * C::PLANE, &load_bar);
        }
        bar_wait(&load_bar, load_phase, &abort_sh, a.p.status);
        load_phase ^= 1;
      }
      fence_before();
      __syncthreads();
      if (warp == 0) {
        fence_after();
        // logits: k-step of 16 channels = 4096 bytes of K, 32 N of the queries
        uint64_t ka = sdesc(sbase + SM::K, 2048, 128), qa = sdesc(sbase + SM::Q, N * 16, 128);
        const uint64_t lo_k = C::PLANE >> 4, lo_q = (N * C::KD * 2) >> 4;
#pragma unroll 1
        for (int ks = 0; ks < D / 16; ++ks, ka += 256, qa += 2 * N) {
          mma_ss(tmem, ka, qa, idesc(TILE, N, false, false), ks > 0);
          if (F32) {
            mma_ss(tmem, ka, qa + lo_q, idesc(TILE, N, false, false), 1);
            if (!TQ || raw) mma_ss(tmem, ka + lo_k, qa, idesc(TILE, N, false, false), 1);
          }
        }
        mma_commit(&qk_bar);
      }
      // ---- values, while the logits run (the previous tile's P V must be done with the buffer)
      wait_pv();
      if (!raw) {
        put_v<KF, F32>(smem + SM::V, ln, w, qend - it * TILE - 2 * ln.vp);
      } else if (tid == 0) {
        const uint8_t* img = p.raw_images + ((size_t)(u / p.rb) * p.raw_tiles + (it - nq)) * p.raw_image + C::PL * C::PLANE;
        bar_expect(&load_bar, C::PL * C::PLANE);
        bulk_g2s(smem + SM::V, img, C::PL * C::PLANE, &load_bar);
      }
      if (TQ && !raw) {
        // the projections' signs take the centroids' place
        bar_wait(&qk_bar, qk_phase, &abort_sh, a.p.status);
        qk_phase ^= 1;
        if constexpr (TQ) put_signs(smem + SM::K, ln, w);
        fence_async_smem();
        __syncthreads();
        if (warp == 0) {
          fence_after();
          uint64_t ka = sdesc(sbase + SM::K, 2048, 128), qa = sdesc(sbase + SM::Q + N * 256, N * 16, 128);
          const uint64_t lo_q = (N * C::KD * 2) >> 4;
#pragma unroll 1
          for (int ks = 0; ks < D / 16; ++ks, ka += 256, qa += 2 * N) {
            mma_ss(tmem + N, ka, qa, idesc(TILE, N, false, false), ks > 0);
            if (F32) mma_ss(tmem + N, ka, qa + lo_q, idesc(TILE, N, false, false), 1);
          }
          mma_commit(&qk_bar);
        }
      }
      // the next tile's words (its page numbers were read a tile earlier)
      if (it + 1 < it1) {
        load_k<KF>(a, unit_pages, page_stride, pg1, ln, w);
        load_v<KF>(a, unit_pages, page_stride, pg1, ln, w);
        pg = pg1;
        pg1 = it + 2 < it1 ? pages_of(it + 2) : pg1;
      }
      // ---- softmax down the thread's columns
      bar_wait(&qk_bar, qk_phase, &abort_sh, a.p.status);
      qk_phase ^= 1;
      fence_after();
      const int j = (raw ? it - nq : it) * TILE + ln.t;  // position, or place in the raw list
      const bool no_mask = !raw && (it + 1) * TILE <= full_end && valid;
      const float nn = TQ && !raw ? __low2float(u2h(ng)) : 1.f;
      const float nw = TQ && !raw ? nn * QJL_CONST * __high2float(u2h(ng)) : 0.f;
      uint8_t* pbuf = smem + SM::P(N) + (ln.t >> 3) * (N * 16) + (ln.t & 7) * 16 + col0 * 16;
      // logits of eight columns from tensor memory
      const auto logits = [&](int c, float (&x)[8]) {
        tm_ld8(lane_addr + col0 + c, x);
        if (TQ && !raw) {
          float y[8];
          tm_ld8(lane_addr + N + col0 + c, y);
          tm_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * nn + y[i] * nw;
        } else {
          tm_wait_ld();
        }
        if (!no_mask) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int cc = col0 + c + i;
            bool on;
            if (!raw) on = valid && j <= lim[cc];
            else if (j < nring) on = anc[cc] != 0 && L - nring + j > lim[cc];
            else on = j < nraw && ((anc[cc] >> (j - nring)) & 1ull);
            if (!on) x[i] = -INFINITY;
          }
        }
      };
      uint32_t over = 0;  // by groups of eight columns: some lane of the warp passed a reference; those are not summed yet
#pragma unroll
      for (int c = 0; c < NH; c += 8) {
        float x[8];
        logits(c, x);
        uint32_t ph[4], pl[4];
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] -= mref[col0 + c + i];
          top = fmaxf(top, x[i]);
          x[i] = ex2(x[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (F32) split2(x[2 * i], x[2 * i + 1], ph[i], pl[i]);
          else ph[i] = h2u(__floats2half2_rn(x[2 * i], x[2 * i + 1]));
        }
        *reinterpret_cast<uint4*>(pbuf + c * 16) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
        if (F32) *reinterpret_cast<uint4*>(pbuf + N * TILE * 2 + c * 16) = make_uint4(pl[0], pl[1], pl[2], pl[3]);
        if (__any_sync(FULL, top > 8.f)) {
          over |= 1u << (c / 8);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) l[c + i] += x[i];
        }
      }
      if (raw) {  // the raw values have landed before their product
        bar_wait(&load_bar, load_phase, &abort_sh, a.p.status);
        load_phase ^= 1;
      }
      fence_async_smem();
      fence_before();
      if (__syncthreads_or(over)) {
        // ---- a row's logit passed its reference by more than 8 (its first ones do): raise the references to the
        // tile's maxima, rescale what has been summed, and take the weights again
#pragma unroll
        for (int c = 0; c < NH; c += 8) {
          float x[8];
          logits(c, x);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (!(over >> (c / 8) & 1)) l[c + i] -= ex2(x[i] - mref[col0 + c + i]);
            float m = x[i];
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
            if (lane == 0) wmax[warp & 3][col0 + c + i] = m;
          }
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < NH; c += 8) {
          float x[8], f[8];
          logits(c, x);
          uint32_t ph[4], pl[4];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int cc = col0 + c + i;
            const float top = fmaxf(fmaxf(wmax[0][cc], wmax[1][cc]), fmaxf(wmax[2][cc], wmax[3][cc]));
            const float m0 = mref[cc], m1 = top > m0 + 8.f ? top : m0;
            f[i] = ex2(m0 - m1);
            x[i] = ex2(x[i] - m1);
            l[c + i] = l[c + i] * f[i] + x[i];
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (F32) split2(x[2 * i], x[2 * i + 1], ph[i], pl[i]);
            else ph[i] = h2u(__floats2half2_rn(x[2 * i], x[2 * i + 1]));
          }
          *reinterpret_cast<uint4*>(pbuf + c * 16) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
          if (F32) *reinterpret_cast<uint4*>(pbuf + N * TILE * 2 + c * 16) = make_uint4(pl[0], pl[1], pl[2], pl[3]);
          if (it > it0) {
            float o[8];
            tm_ld8(lane_addr + C_O + col0 + c, o);
            tm_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] *= f[i];
            tm_st8(lane_addr + C_O + col0 + c, o);
          }
        }
        tm_wait_st();
        fence_async_smem();
        fence_before();
        __syncthreads();
        if (tid < N) {
          const float top = fmaxf(fmaxf(wmax[0][tid], wmax[1][tid]), fmaxf(wmax[2][tid], wmax[3][tid]));
          if (top > mref[tid] + 8.f) mref[tid] = top;
        }
      }
      if (abort_sh) {  // raised before the barrier above by whoever gave up: the whole CTA leaves together
        ok = false;
        break;
      }
      if (warp == 0) {
        fence_after();
        // O += V^T P: k-step of 16 positions = 4096 bytes of V, 32 N of P
        uint64_t va = sdesc(sbase + SM::V, 2048, 128), pa = sdesc(sbase + SM::P(N), N * 16, 128);
        const uint64_t lo_v = C::PLANE >> 4, lo_p = (N * TILE * 2) >> 4;
#pragma unroll 1
        for (int ks = 0; ks < TILE / 16; ++ks, va += 256, pa += 2 * N) {
          mma_ss(tmem + C_O, va, pa, idesc(D, N, true, true), it > it0 || ks > 0);
          if (F32) {
            mma_ss(tmem + C_O, va + lo_v, pa, idesc(D, N, true, true), 1);
            mma_ss(tmem + C_O, va, pa + lo_p, idesc(D, N, true, true), 1);
          }
        }
        mma_commit(&pv_bar);
      }
      pv_pending = true;
    }
    if (!ok) break;
    // ---- the range's part of the unit: reference, sum and O of every row
    bar_wait(&pv_bar, pv_phase, &abort_sh, a.p.status);
    pv_phase ^= 1;
    pv_pending = false;
    fence_after();
    float* rec = p.records + (size_t)(u + blockIdx.x) * (2 * N + D * N);
    __syncthreads();  // the last tile's references are up to date, and their maxima read
#pragma unroll
    for (int c = 0; c < NH; ++c) {
      float s = l[c];
#pragma unroll
      for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(FULL, s, o);
      if (lane == 0) wmax[warp & 3][col0 + c] = s;
    }
#pragma unroll
    for (int c = 0; c < NH; c += 8) {
      float o[8];
      tm_ld8(lane_addr + C_O + col0 + c, o);
      tm_wait_ld();
      // tensor-memory lane = place of the channel: back to its own
      const int ch = (ln.t & ~7) + nibble_channel(ln.t & 7);
#pragma unroll
      for (int i = 0; i < 8; ++i) rec[2 * N + (col0 + c + i) * D + ch] = o[i];
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (tid < N) {
      rec[tid] = mref[tid];
      rec[N + tid] = wmax[0][tid] + wmax[1][tid] + wmax[2][tid] + wmax[3][tid];
    }
    __syncthreads();
    t += it1 - it0;
  }
  // products still running (a CTA that gave up) land before the columns are freed; the wait is bounded
  if (warp == 0 && !ok) {
    mma_commit(&pv_bar);
    const unsigned long long t0 = gtimer();
    while (!bar_try(&pv_bar, pv_phase) && gtimer() - t0 < WAIT_NS) {
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    tm_free(tmem, TM_COLS);
  }
}

// ------------------------------------------------------------------ 3. merge
// WIDE: a CTA per row, its warps on slices of the row's records; else a warp per row
template <bool WIDE>
__global__ void __launch_bounds__(MERGE_WARPS * 32) tree_merge_kernel(const __grid_constant__ Plan p) {
  __shared__ float part[MERGE_WARPS][D + 2];
  extern __shared__ int pre[];
  const MultiArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) tile_prefix(a, pre);
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int rows = a.n * a.g;
  const long long idx = WIDE ? blockIdx.x : (long long)blockIdx.x * MERGE_WARPS + warp;
  if (idx >= (long long)(p.n_units / p.rb) * rows) return;
  const int row = (int)(idx % rows), unit = (int)(idx / rows);
  const int h = unit % a.Hkv, b = (unit / a.Hkv) % a.batch, ll = unit / (a.Hkv * a.batch);
  const int u = unit * p.rb + row / p.N, col = row % p.N, node = row / a.g;
  const long long per_layer = (long long)pre[a.batch] * a.Hkv * p.rb, total = per_layer * a.n_layers_call;
  const int tiles = pre[b + 1] - pre[b];
  const long long first = ll * per_layer + (long long)pre[b] * a.Hkv * p.rb + (long long)(h * p.rb + row / p.N) * tiles;
  // range c holds tile x for c = floor(((x + 1) G - 1) / total)
  const long long G = min((long long)p.G, total);
  const int c0 = (int)(((first + 1) * G - 1) / total), c1 = (int)(((first + tiles) * G - 1) / total);
  const size_t rec_floats = 2 * p.N + (size_t)D * p.N;
  float M = NO_REF, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int c = c0 + (WIDE ? warp : 0); c <= c1; c += WIDE ? MERGE_WARPS : 1) {
    const float* rec = p.records + (size_t)(u + c) * rec_floats;
    const float m = rec[col], s = rec[p.N + col];
    const float4 x = *reinterpret_cast<const float4*>(rec + 2 * p.N + (size_t)col * D + 4 * lane);
    const float mn = fmaxf(M, m), f0 = ex2(M - mn), f1 = ex2(m - mn);
    M = mn;
    l = l * f0 + s * f1;
    o[0] = o[0] * f0 + x.x * f1;
    o[1] = o[1] * f0 + x.y * f1;
    o[2] = o[2] * f0 + x.z * f1;
    o[3] = o[3] * f0 + x.w * f1;
  }
  if (WIDE) {
#pragma unroll
    for (int e = 0; e < 4; ++e) part[warp][4 * lane + e] = o[e];
    if (lane == 0) {
      part[warp][D] = M;
      part[warp][D + 1] = l;
    }
    __syncthreads();
    if (warp != 0) return;
    const int nw = min(MERGE_WARPS, c1 - c0 + 1);
    for (int k = 1; k < nw; ++k) {
      const float m = part[k][D], mn = fmaxf(M, m), f0 = ex2(M - mn), f1 = ex2(m - mn);
      M = mn;
      l = l * f0 + part[k][D + 1] * f1;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = o[e] * f0 + part[k][4 * lane + e] * f1;
    }
  }
  const bool there = p.anc[(size_t)b * a.n + node] != 0;
  const float inv = there && l > 0.f ? 1.f / l : 0.f;
  const __half* sig = a.p.sigv + ((size_t)(a.layer0 + ll) * a.Hkv + h) * D + 4 * lane;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    o[e] = there ? o[e] * inv : 0.f;
    if (a.sinkhorn) o[e] *= __half2float(sig[e]);
  }
  hadamard_warp(o[0], o[1], o[2], o[3], lane);
  const float4 sg = *reinterpret_cast<const float4*>(a.p.signs + 4 * lane);
  const float y[4] = {o[0] * C_WHT * sg.x, o[1] * C_WHT * sg.y, o[2] * C_WHT * sg.z, o[3] * C_WHT * sg.w};
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
template <typename... A>
cudaError_t go(void (*kernel)(A...), unsigned grid, unsigned threads, size_t smem, bool dependent, cudaStream_t s, A... args) {
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// sizes of a call, and its pointers into scratch (base may be null: sizes only); returns the scratch bytes
template <int KF, bool F32>
size_t make_plan(const MultiArgs& a, int sms, Plan* p) {
  using C = Cfg<KF, F32>;
  const int rows = a.n * a.g;
  p->a = a;
  p->rb = (rows + MAX_ROWS - 1) / MAX_ROWS;
  p->N = ((rows + p->rb - 1) / p->rb + 15) / 16 * 16;
  p->n_units = a.n_layers_call * a.batch * a.Hkv * p->rb;
  // two CTAs an SM where their shared memory allows (1 KB each is the system's)
  const size_t smem = Smem<KF, F32>::total(p->N) + (size_t)(a.batch + 1) * 4 + 2048;
  p->G = sms * (!F32 && 2 * (smem + 1024) <= 228 * 1024 ? 2 : 1);
  p->raw_tiles = (raw_count(a.max_seq_len, a.W, a.n) + TILE - 1) / TILE;
  p->q_image = p->N * C::KD * 2 * C::PL;
  p->raw_image = 2 * C::PL * C::PLANE;
  size_t o = 0;
  const auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return a.scratch ? a.scratch + at : nullptr;
  };
  p->anc = reinterpret_cast<unsigned long long*>(take((size_t)a.batch * a.n * 8));
  p->q_images = take((size_t)p->n_units * p->q_image);
  p->raw_images = take((size_t)(p->n_units / p->rb) * p->raw_tiles * p->raw_image);
  p->records = reinterpret_cast<float*>(take((size_t)(p->n_units + p->G) * (2 * p->N + D * p->N) * 4));
  return o;
}

template <int KF, bool F32>
cudaError_t launch(const MultiArgs& a, int sms, cudaStream_t s) {
  constexpr int RPW = Cfg<KF, F32>::TQ ? 4 : 1;
  Plan p;
  make_plan<KF, F32>(a, sms, &p);
  const long long items = (long long)p.n_units * (p.N / RPW) + 2LL * (p.n_units / p.rb) * p.raw_tiles * TILE;
  const long long blocks = a.batch + (items + 7) / 8, out_rows = (long long)(p.n_units / p.rb) * a.n * a.g;
  if (blocks > 0x7fffffffLL || out_rows > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaError_t e = go(tree_prep_kernel<KF, F32>, (unsigned)blocks, THREADS, 0, false, s, p);
  if (e != cudaSuccess) return e;
  const size_t smem = Smem<KF, F32>::total(p.N) + (size_t)(a.batch + 1) * 4;
  e = p.N == 16   ? go(tree_kernel<KF, 8, F32>, (unsigned)p.G, THREADS, smem, true, s, p)
      : p.N == 32 ? go(tree_kernel<KF, 16, F32>, (unsigned)p.G, THREADS, smem, true, s, p)
      : p.N == 48 ? go(tree_kernel<KF, 24, F32>, (unsigned)p.G, THREADS, smem, true, s, p)
                  : go(tree_kernel<KF, 32, F32>, (unsigned)p.G, THREADS, smem, true, s, p);
  if (e != cudaSuccess) return e;
  // many records a row (few units over all CTAs): a CTA per row, else a warp per row
  const size_t pre = (size_t)(a.batch + 1) * 4;
  if (p.G > 8 * p.n_units) return go(tree_merge_kernel<true>, (unsigned)out_rows, MERGE_WARPS * 32, pre, true, s, p);
  return go(tree_merge_kernel<false>, (unsigned)((out_rows + MERGE_WARPS - 1) / MERGE_WARPS), MERGE_WARPS * 32, pre, true, s, p);
}

}  // namespace tree
}  // namespace kvq

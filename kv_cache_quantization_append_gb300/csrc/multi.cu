// Attention of several queries per sequence over the cache as it stands: trees of drafted tokens
// (kv_tree_attention) and the weight that cached positions receive (kv_attention_weights).
//
// A simple form: one CTA per 8 (query, head) rows of a unit, tiles of 32 positions dequantised to fp32 in
// shared memory, plain fp32 products, online softmax in base 2.
#include "kvq_internal.cuh"

namespace kvq {

namespace {

constexpr int ROWS = 8, TILE = 32, LD = D + 4, THREADS = 256;
constexpr int MAX_N = KVQ_MAX_TREE;

struct Smem {
  float q[ROWS][LD], sq[ROWS][LD], raw_q[ROWS][LD], k[TILE][LD], k2[TILE][LD], v[TILE][LD], p[ROWS][TILE + 1];
  unsigned long long anc[MAX_N];
  int depth[MAX_N], dmax;
};

struct Unit {
  int ll, b, h, layer, L;
};
__device__ __forceinline__ Unit unit_of(const MultiArgs& a, int u) {
  Unit x;
  x.h = u % a.Hkv;
  x.b = (u / a.Hkv) % a.batch;
  x.ll = u / (a.Hkv * a.batch);
  x.layer = a.layer0 + x.ll;
  x.L = a.seq_lens[x.b];
  if (x.L < 0 || x.L > a.max_seq_len) {
    if (threadIdx.x == 0) atomicOr(a.p.status, KVQ_DEV_SEQLEN_RANGE);
    x.L = 0;
  }
  return x;
}

// ancestors-or-self of every node (0: not there) and depths
__device__ void tree_masks(const MultiArgs& a, int b, Smem& s) {
  const int* par = a.parents + (size_t)b * a.n;
  if (threadIdx.x == 0) s.dmax = -1;
  __syncthreads();
  if (threadIdx.x < a.n) {
    unsigned long long m = 0;
    int i = threadIdx.x;
    while (i >= 0) {
      m |= 1ull << i;
      const int p = par[i];
      if (p < -1 || p >= i) {
        if (p >= i) atomicOr(a.p.status, KVQ_DEV_BAD_NODE);
        m = 0;
        break;
      }
      i = p;
    }
    s.anc[threadIdx.x] = m;
    s.depth[threadIdx.x] = __popcll(m) - 1;
    if (m) atomicMax(&s.dmax, __popcll(m) - 1);
  }
  __syncthreads();
}

template <int KF>
__device__ void load_rows(const MultiArgs& a, const Unit& u, int r0, int nrows, Smem& s) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, Hq = a.Hkv * a.g;
  const float4 sg = *reinterpret_cast<const float4*>(a.p.signs + 4 * lane);
  const int r = r0 + warp;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (r < nrows)
    x = load4_in(a.q, ((((size_t)u.ll * a.batch + u.b) * Hq + (size_t)u.h * a.g + r % a.g) * a.n + r / a.g) * D + 4 * lane, a.in_bf16);
  float y0 = x.x * sg.x, y1 = x.y * sg.y, y2 = x.z * sg.z, y3 = x.w * sg.w;
  hadamard_warp(y0, y1, y2, y3, lane);
  float y[4] = {y0 * C_WHT * LOGIT_SCALE, y1 * C_WHT * LOGIT_SCALE, y2 * C_WHT * LOGIT_SCALE, y3 * C_WHT * LOGIT_SCALE};
  if (a.sinkhorn) {
    const __half* sig = a.p.sigk + ((size_t)u.layer * a.Hkv + u.h) * D + 4 * lane;
    for (int e = 0; e < 4; ++e) y[e] *= __half2float(sig[e]);
  }
  const float raw[4] = {x.x, x.y, x.z, x.w};
  for (int e = 0; e < 4; ++e) {
    s.q[warp][4 * lane + e] = y[e];
    s.raw_q[warp][4 * lane + e] = raw[e] * LOGIT_SCALE;
  }
  __syncwarp();
  if (KF == KVQ_TQ3_QJL) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < D; ++j)
      for (int e = 0; e < 4; ++e) acc[e] += a.p.qjl_t[j * D + 4 * lane + e] * s.q[warp][j];
    for (int e = 0; e < 4; ++e) s.sq[warp][4 * lane + e] = acc[e];
  }
}

// Dequantise the half-page of positions j0 .. j0 + 31 (rotated, balanced space; zeros from position `end` on,
// where records may hold anything); false: bad page
template <int KF, bool VALUES>
__device__ bool load_half(const MultiArgs& a, const Unit& u, int j0, int end, Smem& s) {
  const int phys = a.block_table[(size_t)u.b * a.max_pages_per_seq + j0 / PAGE];
  if (phys < 0 || phys >= a.L.n_pages) {
    if (threadIdx.x == 0) atomicOr(a.p.status, KVQ_DEV_BAD_PAGE);
    return false;
  }
  const uint8_t* hb = a.p.pages + (((size_t)u.layer * a.L.n_pages + phys) * a.Hkv + u.h) * (size_t)a.L.page_bytes +
                      (size_t)((j0 % PAGE) / HALF) * a.L.half_bytes;
  for (int i = threadIdx.x; i < TILE * D; i += THREADS) {
    const int t = i / D, c = i % D, G = c >> 5, w = c & 31;
    if (j0 + t >= end) {
      s.k[t][c] = s.k2[t][c] = s.v[t][c] = 0.f;
      continue;
    }
    const __half* km = reinterpret_cast<const __half*>(hb + a.L.off_kmeta);
    if (KF == KVQ_Q4G32) {
      const uint8_t by = hb[64 * t + 16 * (w >> 3) + 4 * G + ((w & 7) >> 1)];
      const int code = c & 1 ? by >> 4 : by & 15;
      s.k[t][c] = __half2float(km[8 * t + 4 + G]) + __half2float(km[8 * t + G]) * code;
    } else if (KF == KVQ_Q8G32) {
      const int kk = c >> 4, x = c & 15, m = 2 * ((x & 7) >> 1) + (kk >> 2);
      const int code = (int)hb[128 * t + 16 * (m ^ (t & 1)) + 4 * (kk & 3) + (x & 1) + 2 * (x >> 3)] - 128;
      s.k[t][c] = __half2float(km[4 * t + G]) * code;
    } else {
      const uint8_t by = hb[64 * t + (c >> 1)];
      const float n = __half2float(km[t]), gm = __half2float(km[HALF + t]);
      s.k[t][c] = n * __half2float(a.p.cb->cent[c & 1 ? (by >> 3) & 7 : by & 7]);
      s.k2[t][c] = ((by >> (6 + (c & 1))) & 1) ? n * QJL_CONST * gm : -n * QJL_CONST * gm;
    }
    if (VALUES) {
      const int r = w >> 2, p = t >> 1;
      const uint8_t by = hb[a.L.off_vmain + 128 * p + 16 * ((r + 2 * (p & 3)) & 7) + 4 * G + (t & 1) + (w & 2)];
      const __half* vm = reinterpret_cast<const __half*>(hb + a.L.off_vmeta);
      s.v[t][c] = __half2float(vm[4 * HALF + G * HALF + t]) + __half2float(vm[G * HALF + t]) * (c & 1 ? by >> 4 : by & 15);
    }
  }
  return true;
}

// raw position x of the unit's raw list: ring positions rlo .. L - 1, then (tree) the drafts; keys as they are
template <bool TREE>
__device__ void load_raw(const MultiArgs& a, const Unit& u, int x0, int nraw, int rlo, Smem& s) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nring = u.L - rlo;
  const float4 sg = *reinterpret_cast<const float4*>(a.p.signs + 4 * lane);
  for (int t = warp; t < TILE; t += THREADS / 32) {
    const int x = x0 + t;
    float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
    if (x >= 0 && x < nring) {
      const size_t o = ((((size_t)u.layer * a.max_batch + u.b) * a.Hkv + u.h) * a.W + (rlo + x) % a.W) * D + 4 * lane;
      k = *reinterpret_cast<const float4*>(a.p.ringk + o);
      v = *reinterpret_cast<const float4*>(a.p.ringv + o);
    } else if (TREE && x >= nring && x < nraw && s.anc[x - nring]) {  // nodes that are not there may hold anything
      const size_t o = ((((size_t)u.ll * a.batch + u.b) * a.Hkv + u.h) * a.n + x - nring) * D + 4 * lane;
      k = load4_in(a.k, o, a.in_bf16);
      v = load4_in(a.v, o, a.in_bf16);
    }
    *reinterpret_cast<float4*>(&s.k[t][4 * lane]) = k;
    if (TREE) {
      // values join the quantised ones in rotated, balanced space
      float y0 = v.x * sg.x, y1 = v.y * sg.y, y2 = v.z * sg.z, y3 = v.w * sg.w;
      hadamard_warp(y0, y1, y2, y3, lane);
      float y[4] = {y0 * C_WHT, y1 * C_WHT, y2 * C_WHT, y3 * C_WHT};
      if (a.sinkhorn) {
        const __half* sig = a.p.sigv + ((size_t)u.layer * a.Hkv + u.h) * D + 4 * lane;
        for (int e = 0; e < 4; ++e) y[e] = __fdiv_rn(y[e], __half2float(sig[e]));
      }
      *reinterpret_cast<float4*>(&s.v[t][4 * lane]) = make_float4(y[0], y[1], y[2], y[3]);
    }
  }
}

template <int KF>
__device__ float row_logit(const Smem& s, int r, int t, bool raw) {
  float d = 0.f;
  for (int c = 0; c < D; ++c) d += (raw ? s.raw_q : s.q)[r][c] * s.k[t][c];
  if (KF == KVQ_TQ3_QJL && !raw)
    for (int c = 0; c < D; ++c) d += s.sq[r][c] * s.k2[t][c];
  return d;
}

template <int KF, bool TREE>
__global__ void __launch_bounds__(THREADS) rows_kernel(const __grid_constant__ MultiArgs a) {
  extern __shared__ __align__(16) uint8_t raw_smem[];
  Smem& s = *reinterpret_cast<Smem*>(raw_smem);
  const Unit u = unit_of(a, blockIdx.y);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nrows = a.n * a.g, r0 = blockIdx.x * ROWS;
  if (TREE) tree_masks(a, u.b, s);
  load_rows<KF>(a, u, r0, nrows, s);
  const int row = r0 + warp, node = row / a.g;
  const bool live = row < nrows && (!TREE || s.anc[node < a.n ? node : 0] != 0);
  // the row's position, records up to hi, ring from lo
  const int P = TREE ? u.L + (live ? s.depth[node] : 0) : u.L - a.n + node;
  const int hi = TREE ? (a.W > 0 ? P - a.W : u.L - 1) : min(P, u.L - a.W - 1);
  const int qend = TREE ? (a.W > 0 ? max(0, min(u.L, u.L + s.dmax - a.W + 1)) : u.L) : max(0, u.L - a.W);
  const int rlo = a.W > 0 ? max(0, TREE ? u.L - a.W + 1 : u.L - a.W) : u.L;
  const int nraw = u.L - rlo + (TREE ? a.n : 0);
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  const int nq = (qend + TILE - 1) / TILE, nt = nq + (nraw + TILE - 1) / TILE;
  for (int it = 0; it < nt; ++it) {
    const bool raw = it >= nq;
    const int x0 = (raw ? it - nq : it) * TILE;
    __syncthreads();
    bool ok = true;
    if (raw) load_raw<TREE>(a, u, x0, nraw, rlo, s);
    else ok = load_half<KF, TREE>(a, u, x0, qend, s);
    __syncthreads();
    if (!ok) continue;
    const int x = x0 + lane;
    bool valid = live;
    if (!raw) valid = valid && x <= hi && x < qend;
    else if (x < u.L - rlo) valid = valid && rlo + x <= P && (!TREE || rlo + x > P - a.W);
    else valid = valid && TREE && x < nraw && ((s.anc[node] >> (x - (u.L - rlo))) & 1);
    const float lg = valid ? row_logit<KF>(s, warp, lane, raw) : -INFINITY;
    float mx = lg;
    for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, d));
    const float mn = fmaxf(m, mx);
    if (mn == -INFINITY) continue;
    const float al = exp2f(m - mn), p = exp2f(lg - mn);
    m = mn;
    float ps = p;
    for (int d = 16; d; d >>= 1) ps += __shfl_xor_sync(FULL, ps, d);
    l = l * al + ps;
    if (TREE) {
      s.p[warp][lane] = p;
      __syncwarp();
      for (int e = 0; e < 4; ++e) o[e] *= al;
      for (int t = 0; t < TILE; ++t)
        for (int e = 0; e < 4; ++e) o[e] += s.p[warp][t] * s.v[t][4 * lane + e];
      __syncwarp();
    }
  }
  if (row >= nrows) return;
  if (!TREE) {
    if (lane == 0) reinterpret_cast<float*>(a.scratch)[(size_t)blockIdx.y * nrows + row] = l > 0.f ? m + log2f(l) : INFINITY;
    return;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int e = 0; e < 4; ++e) o[e] *= inv;
  if (a.sinkhorn) {
    const __half* sig = a.p.sigv + ((size_t)u.layer * a.Hkv + u.h) * D + 4 * lane;
    for (int e = 0; e < 4; ++e) o[e] *= __half2float(sig[e]);
  }
  hadamard_warp(o[0], o[1], o[2], o[3], lane);
  const float4 sg = *reinterpret_cast<const float4*>(a.p.signs + 4 * lane);
  const float y[4] = {o[0] * C_WHT * sg.x, o[1] * C_WHT * sg.y, o[2] * C_WHT * sg.z, o[3] * C_WHT * sg.w};
  const int Hq = a.Hkv * a.g;
  const size_t at = ((((size_t)u.ll * a.batch + u.b) * Hq + (size_t)u.h * a.g + row % a.g) * a.n + node) * D + 4 * lane;
  for (int e = 0; e < 4; ++e) {
    if (a.in_bf16) static_cast<__nv_bfloat16*>(a.out)[at + e] = __float2bfloat16_rn(y[e]);
    else static_cast<float*>(a.out)[at + e] = y[e];
  }
}

// weights of positions 32 blockIdx.x .. +31 of a unit: the rows' normalised softmax values, summed in order
template <int KF>
__global__ void __launch_bounds__(THREADS) sum_kernel(const __grid_constant__ MultiArgs a) {
  extern __shared__ __align__(16) uint8_t raw_smem[];
  Smem& s = *reinterpret_cast<Smem*>(raw_smem);
  const Unit u = unit_of(a, blockIdx.y);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nrows = a.n * a.g;
  const int j0 = blockIdx.x * TILE;
  if (j0 >= u.L) return;
  const int qend = max(0, u.L - a.W);
  const float* lse = reinterpret_cast<const float*>(a.scratch) + (size_t)blockIdx.y * nrows;
  float sum = 0.f;
  for (int part = 0; part < 2; ++part) {  // records, then ring
    const bool raw = part == 1;
    if (raw ? j0 + TILE <= qend : j0 >= qend) continue;
    __syncthreads();
    bool ok = true;
    if (raw) load_raw<false>(a, u, j0 - qend, u.L - qend, qend, s);
    else ok = load_half<KF, false>(a, u, j0, qend, s);
    if (!ok) continue;
    for (int r0 = 0; r0 < nrows; r0 += ROWS) {
      __syncthreads();
      load_rows<KF>(a, u, r0, nrows, s);
      __syncthreads();
      const int row = r0 + warp, j = j0 + lane;
      const bool valid = row < nrows && j <= u.L - a.n + row / a.g && (raw ? j >= qend : j < qend);
      s.p[warp][lane] = valid ? exp2f(row_logit<KF>(s, warp, lane, raw) - lse[row]) : 0.f;
      __syncthreads();
      if (warp == 0)
        for (int r = 0; r < ROWS; ++r) sum += s.p[r][lane];
    }
  }
  if (warp == 0 && j0 + lane < u.L) {
    float* w = a.weights + (size_t)blockIdx.y * a.max_seq_len + j0 + lane;
    *w = a.decay != 0.f ? a.decay * *w + sum : sum;
  }
}

template <typename K>
cudaError_t go(K kernel, dim3 grid, const MultiArgs& a, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem));
  if (e != cudaSuccess) return e;
  kernel<<<grid, THREADS, sizeof(Smem), s>>>(a);
  return cudaGetLastError();
}

template <int KF>
cudaError_t launch_weights_kf(const MultiArgs& a, cudaStream_t s) {
  const unsigned units = (unsigned)(a.n_layers_call * a.batch * a.Hkv);
  const cudaError_t e = go(rows_kernel<KF, false>, dim3((a.n * a.g + ROWS - 1) / ROWS, units), a, s);
  return e != cudaSuccess ? e : go(sum_kernel<KF>, dim3((a.max_seq_len + TILE - 1) / TILE, units), a, s);
}
template <int KF>
cudaError_t launch_tree_kf(const MultiArgs& a, cudaStream_t s) {
  const unsigned units = (unsigned)(a.n_layers_call * a.batch * a.Hkv);
  return go(rows_kernel<KF, true>, dim3((a.n * a.g + ROWS - 1) / ROWS, units), a, s);
}

}  // namespace

size_t tree_scratch_q4(const MultiArgs& a, int sms);
size_t tree_scratch_q8(const MultiArgs& a, int sms);
size_t tree_scratch_tq3(const MultiArgs& a, int sms);
cudaError_t launch_tree_q4(const MultiArgs& a, int sms, cudaStream_t s);
cudaError_t launch_tree_q8(const MultiArgs& a, int sms, cudaStream_t s);
cudaError_t launch_tree_tq3(const MultiArgs& a, int sms, cudaStream_t s);

size_t tree_scratch_bytes(const MultiArgs& a, int sms) {
  return a.k_format == KVQ_TQ3_QJL ? tree_scratch_tq3(a, sms) : a.k_format == KVQ_Q8G32 ? tree_scratch_q8(a, sms) : tree_scratch_q4(a, sms);
}
cudaError_t launch_tree(const MultiArgs& a, int sms, cudaStream_t s) {
  return a.k_format == KVQ_TQ3_QJL ? launch_tree_tq3(a, sms, s)
         : a.k_format == KVQ_Q8G32 ? launch_tree_q8(a, sms, s)
                                   : launch_tree_q4(a, sms, s);
}
size_t weights_scratch_bytes(const MultiArgs& a) {
  return align256((size_t)a.n_layers_call * a.batch * a.Hkv * a.n * a.g * sizeof(float));
}
cudaError_t launch_weights(const MultiArgs& a, cudaStream_t s) {
  return a.k_format == KVQ_TQ3_QJL ? launch_weights_kf<KVQ_TQ3_QJL>(a, s)
         : a.k_format == KVQ_Q8G32 ? launch_weights_kf<KVQ_Q8G32>(a, s)
                                   : launch_weights_kf<KVQ_Q4G32>(a, s);
}

}  // namespace kvq

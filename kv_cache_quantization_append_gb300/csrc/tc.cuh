// Helpers of the tensor-core kernels (prefill, trees of drafts, attention weights): mbarriers and bounded waits, tcgen05
// products issued by a warp's elected lane, tensor-memory loads and stores, and the conversion of stored codes to fp16
// operands.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {
namespace tc {

constexpr unsigned long long LAND_NS = 1000000000ull;  // what is under way when a CTA gives up has ~1 s to land

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ unsigned long long gtimer() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// try_wait that may sleep up to about NAP_NS for the phase
constexpr unsigned NAP_NS = 20000;
__device__ __forceinline__ bool bar_sleep(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(NAP_NS)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool bar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// A warp's wait on a phase, of at most about `limit` ns (one shorter than a nap asks again and again).  One that gives up
// flags the status word and the CTA's abort flag, at which every other wait of the CTA gives up too.
__device__ __forceinline__ void bar_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned* status,
                                         unsigned long long limit) {
  const bool nap = limit >= NAP_NS;
  if (!nap || !bar_sleep(bar, parity)) {
    const unsigned long long t0 = gtimer();
    while (nap ? !bar_sleep(bar, parity) : !bar_test(bar, parity)) {
      if (*abort_flag) break;
      if (gtimer() - t0 > limit) {
        atomicOr(status, KVQ_DEV_TIMEOUT);
        *abort_flag = 1;
        break;
      }
    }
  }
  __syncwarp();
}
// A warp's wait for what it has under way when its CTA gives up
__device__ __forceinline__ void bar_land(uint64_t* bar, uint32_t parity) {
  const unsigned long long t0 = gtimer();
  while (!bar_try(bar, parity) && gtimer() - t0 < LAND_NS) {
  }
  __syncwarp();
}
__device__ __forceinline__ void bar_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_g2s(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
// to L2 only (16-byte aligned, a multiple of 16 bytes)
__device__ __forceinline__ void prefetch(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// barriers of a part of the CTA: `count` threads meet at barrier `id`
__device__ __forceinline__ void part_sync(int id, int count) { asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(count) : "memory"); }
__device__ __forceinline__ bool part_or(int id, int count, bool v) {
  uint32_t r;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 p, %3, 0;\nbarrier.cta.red.or.pred q, %1, %2, p;\nselp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"(id), "r"(count), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}
// makes this thread's shared-memory writes visible to the tensor cores and bulk copies (async proxy)
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// shared-memory matrix descriptor, no swizzle: core matrices of 8 x 16 bytes, `lead` and `stride` bytes apart.
// K-major operand: lead along K, stride along M or N; M- or N-major operand: lead along K, stride along M or N.
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lead >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((stride >> 4) & 0x3FFFu) << 32) | (1ull << 46);
}
// kind::f16, fp32 accumulator, fp16 operands
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
constexpr uint32_t BF16_OPERANDS = (1u << 7) | (1u << 10);  // or'ed to it: both operands bf16
// D[tmem] (+)= A[smem] B[smem]^T; the whole warp calls, its elected lane issues (from a single-lane branch a product of
// M128 N64 K16 took 58 cycles instead of 35)
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p, e;\nelect.sync _|e, 0xffffffff;\nsetp.ne.b32 p, %4, 0;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
// the same with A in tensor memory (lane = row, column = two consecutive elements)
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p, e;\nelect.sync _|e, 0xffffffff;\nsetp.ne.b32 p, %4, 0;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
// arrives on bar once all that the elected lane has issued is done (it is the lowest lane, as for the products)
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "{\n.reg .pred e;\nelect.sync _|e, 0xffffffff;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tm_alloc(uint32_t* slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tm_free(uint32_t base, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
}
// this warp's 32 lanes x 4 or 8 consecutive columns
__device__ __forceinline__ void tm_ld(uint32_t taddr, float (&f)[2]) {
  uint32_t r[2];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(taddr));
  f[0] = __uint_as_float(r[0]);
  f[1] = __uint_as_float(r[1]);
}
__device__ __forceinline__ void tm_ld(uint32_t taddr, float (&f)[4]) {
  uint32_t r[4];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tm_ld(uint32_t taddr, float (&f)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tm_st4(uint32_t taddr, uint4 a) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w)
               : "memory");
}
__device__ __forceinline__ void tm_st8(uint32_t taddr, uint4 a, uint4 b) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(a.x), "r"(a.y),
               "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
// fp16 hi and lo of a pair: hi = fp16(v), lo = fp16(v - hi)
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 hf = __half22float2(h);
  hi = h2u(h);
  lo = h2u(__floats2half2_rn(a - hf.x, b - hf.y));
}

// a byte permute whose selector is taken as it is (the intrinsic masks it first)
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

// Eight 4-bit codes of a word whose byte k holds codes 2k (low nibble) and 2k + 1, as exact fp16 in the order
// 0 4 1 5 2 6 3 7: a low nibble under the exponent of 1024 is 1024 + c, a high one under that of 64 is 64 + c.
// (The fp8 conversion instructions run at 16 a cycle and SM here, these at the rate of the fp16 pipe.)
__device__ __forceinline__ void nibbles(uint32_t w, __half2 (&c)[4]) {
  const uint32_t y = w >> 8;
  const __half2 k = u2h(0x64006400u), k16 = u2h(0x54005400u);
  c[0] = __hsub2(u2h((w & 0x000F000Fu) | 0x64006400u), k);    // codes 0, 4
  c[1] = __hsub2(u2h((w & 0x00F000F0u) | 0x54005400u), k16);  // codes 1, 5
  c[2] = __hsub2(u2h((y & 0x000F000Fu) | 0x64006400u), k);    // codes 2, 6
  c[3] = __hsub2(u2h((y & 0x00F000F0u) | 0x54005400u), k16);  // codes 3, 7
}
// channel (0..7) at each place of that order, and the place of each channel
__host__ __device__ constexpr int nibble_channel(int place) { return (place >> 1) + 4 * (place & 1); }
__host__ __device__ constexpr int nibble_place(int channel) { return 2 * (channel & 3) + (channel >> 2); }

}  // namespace tc
}  // namespace kvq

// common.cuh - device helpers shared by the kernels of libattn.so.
//
// Element conversion, the RoPE angle, the bounded-wait status word and thin
// wrappers over the sm_100-family PTX used by the tensor-core kernels
// (mbarrier, TMA, tcgen05).  Nothing here is exported.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace attn {

// Status bits a kernel ORs into the caller-visible status word.
enum : unsigned int { STATUS_TIMEOUT = 1u, STATUS_LAYOUT = 2u };  // LAYOUT: shared memory not as required

// Frequencies of the RoPE pairs, in turns per position: f_i = theta_i / (2*pi)
// with theta_i = base^(-2i / D_r).  Each f_i is split into hi + lo floats by the
// host (computed in double) so that pos * f_i keeps ~48 bits before reduction.
// Pair p of a rotated span of 2 * n_pairs dims is (2p, 2p + 1) within the span,
// or with `half` set (p, p + n_pairs): the split-halves layout.  Either way it
// turns by pos * theta_p.
constexpr int kMaxRopePairs = 128;
struct RopeFreq {
  int n_pairs;  // 0: no rotation
  int half;     // 1: pair p is (p, p + n_pairs); 0: (2p, 2p + 1)
  float hi[kMaxRopePairs];
  float lo[kMaxRopePairs];
};

// Span-relative dims of rotation pair p.
__device__ __forceinline__ int2 rope_pair_dims(const RopeFreq& f, int p) {
  return f.half ? make_int2(p, p + f.n_pairs) : make_int2(2 * p, 2 * p + 1);
}

// sin/cos of the angle pos * theta_i.  The product pos * f_i (turns) is formed
// with an exact two-product, its integer part removed exactly (Sterbenz), and
// the remaining fraction handed to sincospif, which is accurate for any
// argument; the angle error is ~1e-7 rad for positions up to 2^24.
__device__ __forceinline__ void rope_sincos(int pos, float f_hi, float f_lo, float* s, float* c) {
  const float p = static_cast<float>(pos);
  const float a = p * f_hi;
  const float e = fmaf(p, f_hi, -a);
  const float t = (a - rintf(a)) + fmaf(p, f_lo, e);
  sincospif(2.0f * t, s, c);
}

// The same angle, reduced the same way, but its sin/cos taken by the hardware
// approximations (__sincosf on 2*pi*t, |2*pi*t| <= pi, where CUDA documents an
// absolute error of about 2^-21.4): a few instructions instead of a polynomial
// pair.  Used where the rotated value is rounded to bf16 right after (relative
// step 2^-9), so the difference cannot show; the query rows rotated inside the
// prefill kernel, whose rotation sits between two work items on the MMA chain.
__device__ __forceinline__ void rope_sincos_fast(int pos, float f_hi, float f_lo, float* s, float* c) {
  const float p = static_cast<float>(pos);
  const float a = p * f_hi;
  const float e = fmaf(p, f_hi, -a);
  const float t = (a - rintf(a)) + fmaf(p, f_lo, e);
  __sincosf(6.28318530717958647692f * t, s, c);
}

// The paged calls take any 32-bit position.  Behind 2^24 it is split into a float and a rest of 7 bits, and the
// products of both with both words of f_i are reduced one by one: the angle is off by the error of f_i, |pos| * 2^-48
// rad at most, and by some 1e-6 from these sums.  Nearer positions give the bits of the two functions above.
__device__ __forceinline__ bool rope_is_far(int pos) { return pos > (1 << 24) || pos < -(1 << 24); }
__device__ __forceinline__ void rope_sincos_far(int pos, float f_hi, float f_lo, float* s, float* c) {
  const float p = __int2float_rz(pos);                              // not beyond pos
  const float r = static_cast<float>(pos - static_cast<int>(p));
  const float a = __fmul_rn(p, f_hi), b = __fmul_rn(p, f_lo), d = __fmul_rn(r, f_hi);
  const float ae = fmaf(p, f_hi, -a), be = fmaf(p, f_lo, -b), de = fmaf(r, f_hi, -d);
  const float t = (a - rintf(a)) + (ae - rintf(ae)) + (b - rintf(b)) + (d - rintf(d)) + fmaf(r, f_lo, be + de);
  sincospif(2.0f * t, s, c);
}
// f(angle), where angle(f_hi, f_lo, &s, &c) gives a pair's sine and cosine at pos: FAST by rope_sincos_fast, ANY at any
// position.  f's code is there twice then, so that nearer positions do not ask pair by pair (which made 8 MLA queries
// behind 1000 keys each 2.5 us slower).
template <bool ANY, bool FAST, typename F>
__device__ __forceinline__ void with_angles(int pos, const F& f) {
  if (ANY && rope_is_far(pos))
    f([=](float f_hi, float f_lo, float* s, float* c) { rope_sincos_far(pos, f_hi, f_lo, s, c); });
  else if (FAST)
    f([=](float f_hi, float f_lo, float* s, float* c) { rope_sincos_fast(pos, f_hi, f_lo, s, c); });
  else
    f([=](float f_hi, float f_lo, float* s, float* c) { rope_sincos(pos, f_hi, f_lo, s, c); });
}

// Rotate the pair (x0, x1) = (x_{2i}, x_{2i+1}) by the angle with sin s, cos c.
__device__ __forceinline__ void rotate_pair(float& x0, float& x1, float s, float c) {
  const float r0 = x0 * c - x1 * s;
  const float r1 = x0 * s + x1 * c;
  x0 = r0;
  x1 = r1;
}

// ---------------------------------------------------------------- elements
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// Exchange a 16-byte value with the lane whose index differs by the bits of mask.
__device__ __forceinline__ uint4 shfl_xor_u4(uint4 v, int mask) {
  return make_uint4(__shfl_xor_sync(0xffffffffu, v.x, mask), __shfl_xor_sync(0xffffffffu, v.y, mask),
                    __shfl_xor_sync(0xffffffffu, v.z, mask), __shfl_xor_sync(0xffffffffu, v.w, mask));
}

// max(a, b, c) in one instruction (three-input max.f32, sm_100 family).
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 8 bf16 packed in a uint4 <-> 8 floats.  bf16 is the upper half of an fp32,
// so widening is a shift / mask.
__device__ __forceinline__ void bf16x8_to_f32(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);  // .x (low half) = lo
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint4 f32_to_bf16x8(const float* f) {
  uint4 u;
  u.x = pack_bf16x2(f[0], f[1]);
  u.y = pack_bf16x2(f[2], f[3]);
  u.z = pack_bf16x2(f[4], f[5]);
  u.w = pack_bf16x2(f[6], f[7]);
  return u;
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint64_t globaltimer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// ---------------------------------------------------------------- smem / mbarrier
__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Shared abort state of one CTA: set when any wait of the CTA gives up, after
// which every other wait of the CTA returns false at its next check.
struct WaitCtl {
  volatile int* abort_flag;     // in shared memory
  unsigned int* status;         // caller-visible status word (global)
  unsigned long long limit_ns;  // per-wait limit
};

// Wait for the phase with the given parity to complete, giving up after
// limit_ns (then flagging the CTA and the status word).  Returns false on
// give-up or when another wait of the CTA already gave up.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, const WaitCtl& w) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0u) {
      if (*w.abort_flag) return false;
      if (globaltimer_ns() - t0 > w.limit_ns) {
        *w.abort_flag = 1;
        atomicOr(w.status, STATUS_TIMEOUT);
        return false;
      }
    }
  }
}

// ---------------------------------------------------------------- fences
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void named_barrier_sync(uint32_t id, uint32_t nthreads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

// ---------------------------------------------------------------- TMA
__device__ __forceinline__ void tma_prefetch_desc(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int c0,
                                            int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}

// Ask the TMA unit to pull a box into L2 ahead of its real load (no shared
// memory, no barrier; coordinates outside the tensor are clipped).
__device__ __forceinline__ void tma_prefetch_l2_4d(const CUtensorMap* map, int c0, int c1, int c2, int c3) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}
__device__ __forceinline__ void tma_prefetch_l2_3d(const CUtensorMap* map, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// ---------------------------------------------------------------- tcgen05
// Shared-memory matrix descriptor for a 128-byte-swizzled operand tile whose
// 8-row swizzle atoms (8 x 128 B) are 1024-byte aligned.
//   K-major (rows of the matrix contiguous along K): lbo unused, sbo = byte
//     distance between consecutive 8-row groups.
//   MN-major (contiguous along M/N): lbo = byte distance between 64-element
//     column blocks along M/N, sbo = byte distance between 8-row groups along K.
__host__ __device__ constexpr uint64_t sdesc_sw128(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((lbo_bytes >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>((sbo_bytes >> 4) & 0x3FFFu) << 32;
  d |= static_cast<uint64_t>(1) << 46;  // descriptor version for tcgen05
  d |= static_cast<uint64_t>(2) << 61;  // 128-byte swizzle
  return d;
}

// Instruction descriptor of tcgen05.mma kind::f16 with bf16 A/B and fp32 D.
// A is K-major; B is K-major or (b_mn_major) MN-major.
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4)                                    // D format f32
         | (1u << 7)                                  // A format bf16
         | (1u << 10)                                 // B format bf16
         | ((b_mn_major ? 1u : 0u) << 16)             // B major-ness
         | (static_cast<uint32_t>(N >> 3) << 17)      // N / 8
         | (static_cast<uint32_t>(M >> 4) << 24);     // M / 16
}

__device__ __forceinline__ void tmem_alloc(uint32_t* smem_result, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_result)),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// D[tmem] (+)= A[smem] * B[smem]
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Per-warpgroup register budget (all warps of a warpgroup execute the same one).
template <int N> __device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N> __device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}

// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive once on bar when every tcgen05 operation issued so far by this thread completes.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_u32(bar))
               : "memory");
}

// 32 consecutive 32-bit TMEM columns of this warp's 32 lanes (one lane per thread).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

}  // namespace attn

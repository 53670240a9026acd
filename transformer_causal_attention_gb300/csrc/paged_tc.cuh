// paged_tc.cuh - what the tensor-core kernels over a paged cache share: bounded waits, MMAs by short
// descriptors, the stage ring, TMEM row helpers and the early launch.
#pragma once

#include "common.cuh"

namespace attn {
namespace {

// ------------------------------------------------------------------------------------- waits
// A wait whose slow part is out of line: two dozen inlined copies of it were a quarter of the code.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, const WaitCtl* w) {
  return mbar_wait(bar, parity, *w);
}
__device__ __forceinline__ bool lane_wait(uint64_t* bar, uint32_t parity, const WaitCtl* w) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, w);
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtl* w) {
  const bool ok = lane_wait(bar, parity, w);
  return __all_sync(0xffffffffu, ok);
}
// In line, for the softmax warps (beside their tile loops the compiler finds no registers for a call),
// and short: what they wait for comes from the other roles, whose waits keep the time and raise the
// abort flag; the count only bounds the loop should none of them be left.
__device__ __forceinline__ bool row_wait(uint64_t* bar, uint32_t parity, const WaitCtl* w) {
  bool ok = false;
#pragma unroll 1
  for (uint32_t it = 0; it < (1u << 26) && !(ok = mbar_try_wait(bar, parity)) && !*w->abort_flag; ++it) {
  }
  return __all_sync(0xffffffffu, ok);
}

__device__ __noinline__ void drain_wait(uint64_t* bar, uint32_t parity, unsigned long long limit_ns) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > limit_ns) return;
  }
}

// The MMAs with shared-memory descriptors by their low words (address and leading offset): the high words of all
// tiles here are the same, and a burst's descriptors differ by constants that never carry.  Half the instructions
// per MMA of 64-bit descriptors.
constexpr uint32_t kDescHigh = static_cast<uint32_t>(sdesc_sw128(0, 16, 1024) >> 32);
__device__ __forceinline__ void mma_ss_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_ts_lo(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}

struct Ring {
  uint32_t st = 0, ph = 0;
  __device__ __forceinline__ void next(uint32_t n) {
    if (++st == n) {
      st = 0;
      ph ^= 1u;
    }
  }
};

// ------------------------------------------------------------------------------------- TMEM rows
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// This thread's row of O times alpha, before the tile's P V; the P V before has completed (the
// tile's scores were committed after it).
template <int D>
__device__ __forceinline__ void rescale_o(uint32_t o_addr, float alpha) {
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    uint32_t orow[32];
    tmem_ld32(o_addr + c * 32, orow);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) orow[e] = __float_as_uint(__uint_as_float(orow[e]) * alpha);
    tmem_st32(o_addr + c * 32, orow);
  }
}

// Among four lanes (lj = lane & 3): piece e of lane k becomes piece k of lane e.
__device__ __forceinline__ void transpose_pieces(uint4* pc, int lj) {
  const bool b1 = (lj & 2) != 0, b0 = (lj & 1) != 0;
  const uint4 r0 = shfl_xor_u4(b1 ? pc[0] : pc[2], 2), r1 = shfl_xor_u4(b1 ? pc[1] : pc[3], 2);
  pc[0] = b1 ? r0 : pc[0];
  pc[1] = b1 ? r1 : pc[1];
  pc[2] = b1 ? pc[2] : r0;
  pc[3] = b1 ? pc[3] : r1;
  const uint4 q0 = shfl_xor_u4(b0 ? pc[0] : pc[1], 1), q1 = shfl_xor_u4(b0 ? pc[2] : pc[3], 1);
  pc[0] = b0 ? q0 : pc[0];
  pc[1] = b0 ? pc[1] : q0;
  pc[2] = b0 ? q1 : pc[2];
  pc[3] = b0 ? pc[3] : q1;
}

// Launches a kernel that may start before the one in front of it has ended.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t st, bool early,
                         A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace
}  // namespace attn

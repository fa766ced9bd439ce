// Fifth-generation tensor core instructions: tensor memory, asynchronous matrix products,
// their descriptors. sm_103a only.
#pragma once

#include "pkv_common.cuh"

namespace pkv {

// ---- tensor memory: 128 lanes of 512 32-bit columns per SM; an address is lane << 16 | column

// Called by one whole warp; the base address goes to shared memory. The same warp frees it.
__device__ __forceinline__ void tmem_alloc(uint32_t smem_dst, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(columns) : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_before_sync() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_after_sync() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// 32 columns of the warp's 32 lanes: lane l of the warp gets columns of its own TMEM lane. The
// registers hold the values only after tmem_wait_ld of them.
__device__ __forceinline__ void tmem_ld_32(uint32_t addr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(addr)
      : "memory");
}
// Waits for the thread's loads. The registers go through it, so that nothing that reads them can be
// moved before it.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
        "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
        "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),
        "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]),
        "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
      :
      : "memory");
}
__device__ __forceinline__ void tmem_st_32(uint32_t addr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

// mbar_wait_warp for waits that a chain of products hangs on: the clock and the abort flag are looked at only every
// 32 polls, so that a phase that completes is seen at once.
__device__ __forceinline__ bool mbar_wait_close(uint32_t bar, uint32_t parity, volatile int* abort_flag, int32_t* error_flag,
                                                unsigned long long limit_ns) {
  if (limit_ns < kShortWaitLimitNs) return mbar_wait_warp(bar, parity, abort_flag, error_flag, limit_ns);
  unsigned long long start = 0;
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    int stop = 0;
    if ((threadIdx.x & 31) == 0) {
      const unsigned long long now = global_timer_ns();
      if (start == 0) start = now;
      if (*abort_flag) {
        stop = 1;
      } else if (now - start > limit_ns) {
        *abort_flag = 1;
        if (error_flag) atomicOr(error_flag, kDevErrTimeout);
        stop = 1;
      }
    }
    if (__shfl_sync(0xffffffffu, stop, 0)) return false;
  }
}

// ---- matrix products

// Shared-memory operand in 128-byte rows with the 128-byte swizzle, tiles 1024-byte aligned.
// Groups of 8 rows are 1024 bytes apart. lead: for an operand whose rows run along the
// contracted dim (64 columns of the other dim per row), the distance between runs of 64 columns.
__device__ __forceinline__ uint64_t umma_desc(uint32_t smem, uint32_t lead) {
  return static_cast<uint64_t>((smem & 0x3FFFFu) >> 4) | static_cast<uint64_t>((lead & 0x3FFFFu) >> 4) << 16 |
         static_cast<uint64_t>(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

// kind::f16 with f32 sums, M = 128; operands bf16, or fp16 with `half`. b_columns: B's rows run along the
// contracted dim. negate: -A.
__device__ __forceinline__ constexpr uint32_t umma_instr(int n, bool b_columns, bool negate, bool half) {
  return 1u << 4 | (half ? 0u : 1u << 7 | 1u << 10) | (negate ? 1u << 13 : 0u) | (b_columns ? 1u << 16 : 0u) |
         static_cast<uint32_t>(n >> 3) << 17 | 8u << 24;
}

// Whether this lane issues for its warp, which is converged.
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is;
}

// D (TMEM) = A B^T + (accumulate ? D : 0) over 16 contracted values. Called by a whole converged warp and
// issued by the lane with `leader`: operands that the compiler sees to be the same in all lanes stay in uniform
// registers, where the instruction wants them (behind a branch on the lane each would be moved there first).
__device__ __forceinline__ void umma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t instr,
                                        bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "setp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(instr), "r"(static_cast<uint32_t>(accumulate)), "r"(leader)
      : "memory");
}
// The same with A in tensor memory: two 16-bit values per column.
__device__ __forceinline__ void umma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t instr,
                                        bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "setp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(instr), "r"(static_cast<uint32_t>(accumulate)), "r"(leader)
      : "memory");
}
// The mbarrier gets one arrival once every product this thread has issued is done.
__device__ __forceinline__ void umma_commit(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(leader)
      : "memory");
}

}  // namespace pkv

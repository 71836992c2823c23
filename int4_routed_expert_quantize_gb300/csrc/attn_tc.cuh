// Tensor-core helpers of the attention kernels for many rows: tensor memory as a thread's row, descriptors, query copies, output stores.
#pragma once

#include "attn_device.cuh"

namespace coli {

#define COLI_LD32(taddr, r)                                                                          \
  asm volatile(                                                                                      \
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "                                                      \
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "                       \
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"       \
      : "=f"((r)[0]), "=f"((r)[1]), "=f"((r)[2]), "=f"((r)[3]), "=f"((r)[4]), "=f"((r)[5]),          \
        "=f"((r)[6]), "=f"((r)[7]), "=f"((r)[8]), "=f"((r)[9]), "=f"((r)[10]), "=f"((r)[11]),        \
        "=f"((r)[12]), "=f"((r)[13]), "=f"((r)[14]), "=f"((r)[15]), "=f"((r)[16]), "=f"((r)[17]),    \
        "=f"((r)[18]), "=f"((r)[19]), "=f"((r)[20]), "=f"((r)[21]), "=f"((r)[22]), "=f"((r)[23]),    \
        "=f"((r)[24]), "=f"((r)[25]), "=f"((r)[26]), "=f"((r)[27]), "=f"((r)[28]), "=f"((r)[29]),    \
        "=f"((r)[30]), "=f"((r)[31])                                                                 \
      : "r"(taddr)                                                                                   \
      : "memory")
// a wait that names 32 loaded registers, so that no use of them can move before it
#define COLI_LDWAIT32(r)                                                                             \
  asm volatile("tcgen05.wait::ld.sync.aligned;"                                                      \
               : "+f"((r)[0]), "+f"((r)[1]), "+f"((r)[2]), "+f"((r)[3]), "+f"((r)[4]), "+f"((r)[5]), \
                 "+f"((r)[6]), "+f"((r)[7]), "+f"((r)[8]), "+f"((r)[9]), "+f"((r)[10]),              \
                 "+f"((r)[11]), "+f"((r)[12]), "+f"((r)[13]), "+f"((r)[14]), "+f"((r)[15]),          \
                 "+f"((r)[16]), "+f"((r)[17]), "+f"((r)[18]), "+f"((r)[19]), "+f"((r)[20]),          \
                 "+f"((r)[21]), "+f"((r)[22]), "+f"((r)[23]), "+f"((r)[24]), "+f"((r)[25]),          \
                 "+f"((r)[26]), "+f"((r)[27]), "+f"((r)[28]), "+f"((r)[29]), "+f"((r)[30]),          \
                 "+f"((r)[31])                                                                       \
               :                                                                                     \
               : "memory")

#define COLI_ST32(taddr, r)                                                                          \
  asm volatile(                                                                                      \
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "                                                \
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "                     \
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr), \
      "f"((r)[0]), "f"((r)[1]), "f"((r)[2]), "f"((r)[3]), "f"((r)[4]), "f"((r)[5]), "f"((r)[6]),     \
      "f"((r)[7]), "f"((r)[8]), "f"((r)[9]), "f"((r)[10]), "f"((r)[11]), "f"((r)[12]), "f"((r)[13]), \
      "f"((r)[14]), "f"((r)[15]), "f"((r)[16]), "f"((r)[17]), "f"((r)[18]), "f"((r)[19]),            \
      "f"((r)[20]), "f"((r)[21]), "f"((r)[22]), "f"((r)[23]), "f"((r)[24]), "f"((r)[25]),            \
      "f"((r)[26]), "f"((r)[27]), "f"((r)[28]), "f"((r)[29]), "f"((r)[30]), "f"((r)[31])             \
      : "memory")

__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Instruction descriptor of kind::f16, fp32 accumulator, M = 128: A and B format 1 = bf16, 0 = fp16; bit
// 16: B is stored with N contiguous.
template <class T>
__device__ constexpr uint32_t mma_desc(int n, bool b_n_major) {
  constexpr uint32_t fmt = T::kExp == 0x7F807F80u ? 1u : 0u;
  return (1u << 4) | (fmt << 7) | (fmt << 10) | ((b_n_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         (8u << 24);
}

// Shared-memory descriptor of a value tile as the N-contiguous operand: boxes of 64 values (128 swizzled
// bytes) x 128 keys.  8 keys make one 1024-byte atom; the next 8 keys follow at 1024 bytes, the next 64
// values at one box (16 KB).  p = first key of the 16 that one MMA takes.
__device__ __forceinline__ uint64_t smem_desc_values(const void* p) {
  const uint64_t a = (smem_addr(p) >> 4) & 0x3FFFu;
  return a | ((uint64_t)((kTileKeys * 128) >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
         (2ull << 61);
}

// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1 : 0)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

// true in one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// the n lowest bits (n may be out of 0..32)
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
}

// 32 bytes of a thread's row at once: a full sector per thread.  p on a 32-byte boundary
__device__ __forceinline__ void st_sector(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// The same of the caller's output, whose heads start on 16-byte boundaries: in one store where they all start on 32, else
// in two.  8192 tokens, window 4096, back to back: 449 us in one store, 487 in two.
__device__ __forceinline__ void st_out(void* p, const uint32_t (&v)[8], bool sectors) {
  if (sectors) {
    st_sector(p, v);
  } else {
    uint4* q = static_cast<uint4*>(p);
    q[0] = make_uint4(v[0], v[1], v[2], v[3]), q[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

}  // namespace coli

// Device helpers of the attention kernels: 16-bit types, mma.sync fragments, 4-D tensor copies.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_sched.cuh"
#include "coli_tc.cuh"

namespace coli {

struct Bf16 {
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float lo(uint32_t v) { return __uint_as_float(v << 16); }
  static __device__ __forceinline__ float hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
  static constexpr uint32_t kExp = 0x7F807F80u, kExpInc = 0x00800080u;
};

struct Fp16 {
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float lo(uint32_t v) {
    return __half2float(__ushort_as_half((unsigned short)(v & 0xFFFFu)));
  }
  static __device__ __forceinline__ float hi(uint32_t v) {
    return __half2float(__ushort_as_half((unsigned short)(v >> 16)));
  }
  static constexpr uint32_t kExp = 0x7C007C00u, kExpInc = 0x04000400u;
};

// A bounded wait by a whole warp: every lane sees the phase, and the lanes are together afterwards
// (the instructions that follow are warp-wide).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  return __all_sync(FULL, mbar_wait_bounded(bar, parity, abort_flag, status));
}

// nonzero when one of the two 16-bit values is infinite or NaN (all exponent bits set: adding
// one to the exponent field carries into the sign bit, which the mask had cleared)
template <class T>
__device__ __forceinline__ uint32_t nonfinite2(uint32_t v) {
  return ((v & T::kExp) + T::kExpInc) & 0x80008000u;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// c += a (16 x 16, row major) * b (16 x 8, column major)
template <class T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<Bf16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<Fp16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// 4-D tensor copy global -> shared of one box of the cache: coordinates value, slot, head, page
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int slot,
                                            int head, int page, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(slot), "r"(head), "r"(page),
      "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// One warp fills one stage: the boxes of a KT-key tile of K (and of V after it) that hold keys
// some row of the block sees.  Pages whose id is out of range read as zeros (page coordinate
// past the end) and are reported.
template <int KT, int D>
__device__ __forceinline__ void fill_boxes(const AttnParams& p, const CUtensorMap* map, uint8_t* dst,
                                           uint64_t* bar, int64_t table_row, int p0, int p1, int j0,
                                           int head, int lane) {
  constexpr int kSlabs = D / 64;
  const int page = 1 << p.page_shift;
  const int rows = min(page, KT);  // slots per box
  const int boxes = KT / rows;     // per slab
  bool need = false;
  int id = p.n_pages;
  if (lane < boxes) {
    const int a = j0 + lane * rows, e = a + rows - 1;  // the box's keys
    // some_sees of some key in [a, e]
    if (a <= p1 && p1 >= 0 && (e > p0 - p.window || a < p.sinks)) {
      need = true;
      id = __ldg(p.table + table_row + (a >> p.page_shift));
      if (id < 0 || id >= p.n_pages) {
        id = p.n_pages;
        atomicExch(p.status, COLI_EINVAL);
      }
    }
  }
  if (need) {
    const int slot = (j0 + lane * rows) & (page - 1);
#pragma unroll
    for (int s = 0; s < kSlabs; ++s)
      tma_load_4d(dst + s * KT * 128 + lane * rows * 128, map, s * 64, slot, head, id, bar);
  }
}

// bytes fill_boxes will copy for this tile
template <int KT, int D>
__device__ __forceinline__ uint32_t fill_bytes(const AttnParams& p, int p0, int p1, int j0, int lane) {
  const int rows = min(1 << p.page_shift, KT);
  const int boxes = KT / rows;
  const int a = j0 + lane * rows, e = a + rows - 1;
  const bool need = lane < boxes && a <= p1 && p1 >= 0 && (e > p0 - p.window || a < p.sinks);
  return (uint32_t)__popc(__ballot_sync(FULL, need)) * (uint32_t)rows * D * 2;
}

}  // namespace coli

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
// (the instructions that follow are warp-wide).  The rules of mbar_wait_bounded, but inline: a call would
// tie the kernels that split their registers by role to one count.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) {
    const uint64_t t0 = global_ns();
#pragma unroll 1
    for (uint32_t it = 1; !*abort_flag; ++it) {
      if (mbar_try_wait(bar, parity)) {
        ok = true;
        break;
      }
      if ((it & 63u) == 0 && global_ns() - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        atomicExch(status, COLI_ETIMEOUT);
      }
    }
  }
  return __all_sync(FULL, ok);
}

// The same by one lane on its own; a wait that gives up returns all the same (the abort flag is up then).
__device__ __forceinline__ void lane_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = global_ns();
#pragma unroll 1
  for (uint32_t it = 1; !mbar_try_wait(bar, parity) && !*abort_flag; ++it)
    if ((it & 63u) == 0 && global_ns() - t0 > kWaitLimitNs) {
      *abort_flag = 1;
      atomicExch(status, COLI_ETIMEOUT);
    }
}

// drain_fills, inline for the same reason
__device__ __forceinline__ void drain_ring(uint64_t* full, int stages, int issued) {
#pragma unroll 1
  for (int it = max(0, issued - stages); it < issued; ++it) {
    const uint64_t t0 = global_ns();
#pragma unroll 1
    while (!mbar_try_wait(full + it % stages, (uint32_t)((it / stages) & 1)))
      if (global_ns() - t0 > kWaitLimitNs / 8) break;
  }
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

// the page table of a list entry
__device__ __forceinline__ const int32_t* table_of(const AttnParams& p, int b) {
  return b < p.n_seqs ? p.table + (int64_t)b * p.table_stride : p.pre_table;
}

// One warp fills the stage of a KT-key tile: the boxes that hold keys some row of the block sees.  Lane i takes box i, from
// `map` to dst and (N = 2) from `second` to dst + KT * D * 2.  Pages whose id is out of
// range read as zeros (page coordinate past the end) and are reported.
template <int KT, int D, int N>
__device__ __forceinline__ void fill_boxes(const AttnParams& p, const CUtensorMap* map, const CUtensorMap* second,
                                           uint8_t* dst, uint64_t* bar, const int32_t* table, int p0, int p1, int j0, int head, int lane) {
  const int page = 1 << p.page_shift;
  const int rows = min(page, KT);  // slots per box
  const int boxes = KT / rows;     // per 64 values
  const int a = j0 + lane * rows, e = a + rows - 1;  // the lane's keys
  const bool need = lane < boxes && a <= p1 && (e > p0 - p.window || a < p.sinks);
  int id = 0;
  if (need) id = __ldg(table + (a >> p.page_shift));
  const uint32_t bytes = (uint32_t)__popc(__ballot_sync(FULL, need)) * (uint32_t)rows * D * 2;
  if (lane == 0) mbar_expect_tx(bar, N * bytes);
  __syncwarp();
  if (need) {
    if (id < 0 || id >= p.n_pages) {
      id = p.n_pages;
      atomicExch(p.status, COLI_EINVAL);
    }
    const int slot = a & (page - 1);
    dst += lane * rows * 128;
#pragma unroll
    for (int s = 0; s < D / 64; ++s) tma_load_4d(dst + s * KT * 128, map, s * 64, slot, head, id, bar);
    if (N == 2)
#pragma unroll
      for (int s = 0; s < D / 64; ++s)
        tma_load_4d(dst + KT * D * 2 + s * KT * 128, second, s * 64, slot, head, id, bar);
  }
  __syncwarp();
}

}  // namespace coli

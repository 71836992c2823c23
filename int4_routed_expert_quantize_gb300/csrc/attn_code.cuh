// Device helpers of the attention kernels over an 8-bit cache: codes to 16-bit values, and the copies of code tiles and their scales.
#pragma once

#include "attn_device.cuh"
#include "bulk.cuh"

namespace coli {

// widen: four codes of a word -> two pairs of type T: bytes 0 and 2, bytes 1 and 3.  A code is `unit` times its value, which is exact.
template <int CODE>
struct Code;

template <>
struct Code<COLI_ATTN_CODE_INT8> {
  static constexpr float unit = 1.f;
  template <class T>
  static __device__ __forceinline__ void widen(uint32_t w, uint32_t& even, uint32_t& odd) {
    if constexpr (T::kExp == Bf16::kExp) {
      even = less(__byte_perm(w, 0x43434343u, 0x4240)), odd = less(__byte_perm(w, 0x43434343u, 0x4341));
    } else {  // offset by 128, the byte is the mantissa of 1024 + c + 128
      const uint32_t u = w ^ 0x80808080u;
      even = minus(__byte_perm(u, 0x64646464u, 0x4240));
      odd = minus(__byte_perm(u, 0x64646464u, 0x4341));
    }
  }
  static __device__ __forceinline__ uint32_t minus(uint32_t v) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x64806480u));  // 1152
    return r;
  }
  // codes under bf16's exponent of 128: 128 + (c & 127), less 128 or, for a negative c, 256
  static __device__ __forceinline__ uint32_t less(uint32_t v) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v & 0xFF7FFF7Fu), "r"(v & 0xFF80FF80u));
    return r;
  }
};

template <>
struct Code<COLI_ATTN_CODE_E4M3> {
  static constexpr float unit = 256.f;
  // e4m3's exponent and mantissa are fp16's, whose exponent is offset by 8 more (so subnormal codes are subnormal too); or bf16's
  // at its lowest exponents.  Codes 0x7F and 0xFF come out finite, so that a slot that no row sees cannot spoil a product with its
  // zero weight.
  template <class T>
  static __device__ __forceinline__ void widen(uint32_t w, uint32_t& even, uint32_t& odd) {
    if constexpr (T::kExp == Bf16::kExp) {
      even = raise(((w << 4) & 0x07F007F0u) | ((w << 8) & 0x80008000u));
      odd = raise(((w >> 4) & 0x07F007F0u) | (w & 0x80008000u));
    } else {
      even = ((w << 7) & 0x3F803F80u) | ((w << 8) & 0x80008000u);
      odd = ((w >> 1) & 0x3F803F80u) | (w & 0x80008000u);
    }
  }
  static __device__ __forceinline__ uint32_t raise(uint32_t v) {  // times 2^112
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(0x77807780u));
    return v;
  }
};

// A finite scale as it is, any other as NaN: the sign of a score would make an infinite one's weight 0.
__device__ __forceinline__ float spoil(float scale) { return fmaf(scale, 0.f, scale); }

// log2 |value scale|; not below -80, so that weights of values of (next to) 0 keep their sum in fp32's range
__device__ __forceinline__ float scale_log(float scale) {
  const float l = __log2f(fabsf(scale));
  return l < -80.f ? -80.f : l;  // NaN stays
}

// One warp fills the stage of a KT-key tile: the boxes that hold keys some row of the block sees, lane i box i: the keys' codes
// to `keys`, the values' to `vals`, their scales to scales[0..KT-1] and scales[KT..2KT-1].  A page whose id is out of range
// reads as zeros, scales included, and is reported.
template <int KT, int D>
__device__ __forceinline__ void fill_codes(const AttnParams& p, const CUtensorMap* kmap, const CUtensorMap* vmap, uint8_t* keys,
                                           uint8_t* vals, float* scales, uint64_t* bar, const int32_t* table, int p0, int p1,
                                           int j0, int head, int lane) {
  const int page = 1 << p.page_shift;
  const int rows = min(page, KT);  // slots per box
  const int boxes = KT / rows;
  const int a = j0 + lane * rows, e = a + rows - 1;  // the lane's keys
  const bool need = lane < boxes && a <= p1 && (e > p0 - p.window || a < p.sinks);
  int id = 0;
  if (need) id = __ldg(table + (a >> p.page_shift));
  const bool bad = need && (id < 0 || id >= p.n_pages);
  if (bad) {
    id = p.n_pages;  // the tensor copies' coordinate past the end
    atomicExch(p.status, COLI_EINVAL);
    for (int i = 0; i < rows; ++i) scales[lane * rows + i] = scales[KT + lane * rows + i] = 0.f;
    fence_proxy_async_smem();  // a later tile's copies go to the same place
  }
  const int n = __popc(__ballot_sync(FULL, need)), good = n - __popc(__ballot_sync(FULL, bad));
  __syncwarp();
  if (lane == 0) mbar_expect_tx(bar, (uint32_t)rows * (uint32_t)(n * 2 * D + good * 8));
  __syncwarp();
  if (need) {
    const int slot = a & (page - 1);
    tma_load_4d(keys + lane * rows * D, kmap, 0, slot, head, id, bar);
    tma_load_4d(vals + lane * rows * D, vmap, 0, slot, head, id, bar);
    if (!bad) {
      bulk_load(scales + lane * rows, p.k_scale + id * p.ks_page + head * p.ks_head + slot, rows * 4, bar);
      bulk_load(scales + KT + lane * rows, p.v_scale + id * p.vs_page + head * p.vs_head + slot, rows * 4, bar);
    }
  }
  __syncwarp();
}

}  // namespace coli

// New keys and values into the paged cache, keys and queries rotated by their position on the way.
//
// Pair i of a token at position p turns by p * f_i.  The angle is reduced before it becomes a float: f_i
// is kept as a fraction of a turn in 64-bit fixed point, and the product with p modulo 2^64 is the
// angle's fraction of a turn to 2^-33 of a turn at any int32 position, where p * f_i in fp32 is off by
// 1e-3 radians at position 16384 already.  One rounding to the cache's type at the end.
//
// A lane holds 16 values (8 pairs) of a head, so D/16 lanes make a head and a warp 4 or 8 heads; its 8 sines
// and cosines serve all heads that the warp handles for its token.  Bound by HBM: q, k, v are read
// once, q', k', v written once, in 16-byte accesses.  16384 tokens of 48 query and 8 key heads of 128: 537 MB in 83 us,
// 6.5 TB/s (a copy reaches 6.78); 16 tokens 2.6 us, which is the launch.
// Into an 8-bit cache (codes and scales as coli_attn.h defines them) 504 MB in 87 us: issue slots are 68 % used beside HBM at 5.8 TB/s.
#include "attn_device.cuh"

namespace coli {

namespace {

// warps a block: the warps share nothing, and small blocks spread evenly and start as others end; us with 1 / 2 / 8: 16 tokens
// 2.6 / 2.6 / 2.9, 700 5.2 / 5.3 / 6.0, 4000 24.3 / 26.8 / 27.8, 16384 83.1 / 82.6 / 82.6
constexpr int kAppendWarps = 1;
// groups of heads a warp has in flight; us with 2 / 3 / 4: 700 tokens 5.6 / 5.5 / 5.3, 2000 15.9 / 15.1 /
// 14.6, 16384 83.8 / 83.7 / 82.6 (8 take so many registers that 16384 take 82.8 and 500 10.4 / 8.5)
// Into an 8-bit cache 2, with registers for 28 blocks an SM, and two warps a token: 16384 tokens 86.5 us (4 ahead, 18 blocks, one warp 94.8; 3
// ahead with 28 blocks 89.9, and two warps 85.9, where 16 tokens take 3.6 for 3.2).
__host__ __device__ constexpr int ahead(int code) { return code ? 2 : 4; }
constexpr int blocks_per_sm(int code) { return code ? 28 : 0; }  // 0: as many as come

template <class T>
__device__ __forceinline__ void rotate8(uint4& a, uint4& b, const float (&cs)[8], const float (&sn)[8],
                                        bool interleaved) {
  uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (interleaved) {  // word w = pair w
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const float u = T::lo(x[w]), v = T::hi(x[w]);
      x[w] = T::pack(u * cs[w] - v * sn[w], v * cs[w] + u * sn[w]);
    }
  } else {  // word w of a and of b hold the halves of pairs 2w, 2w+1
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float u0 = T::lo(x[w]), u1 = T::hi(x[w]), v0 = T::lo(x[w + 4]), v1 = T::hi(x[w + 4]);
      x[w] = T::pack(u0 * cs[2 * w] - v0 * sn[2 * w], u1 * cs[2 * w + 1] - v1 * sn[2 * w + 1]);
      x[w + 4] = T::pack(v0 * cs[2 * w] + u0 * sn[2 * w], v1 * cs[2 * w + 1] + u1 * sn[2 * w + 1]);
    }
  }
  a = make_uint4(x[0], x[1], x[2], x[3]);
  b = make_uint4(x[4], x[5], x[6], x[7]);
}

// 16 values as fp32: word w of x[0], x[1] hold values 2w, 2w + 1
template <class T>
__device__ __forceinline__ void widen(const uint4& a, const uint4& b, float (&f)[16]) {
  const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int w = 0; w < 8; ++w) f[2 * w] = T::lo(x[w]), f[2 * w + 1] = T::hi(x[w]);
}
// rotate8 without the rounding
__device__ __forceinline__ void rotate16(float (&f)[16], const float (&cs)[8], const float (&sn)[8], bool interleaved) {
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    // pair w: values 2w and 2w + 1, or w and w + 8
    const float u = interleaved ? f[2 * w] : f[w], v = interleaved ? f[2 * w + 1] : f[w + 8];
    const float p = u * cs[w] - v * sn[w], q = v * cs[w] + u * sn[w];
    if (interleaved) f[2 * w] = p, f[2 * w + 1] = q;
    else f[w] = p, f[w + 8] = q;
  }
}

// 16 of a head's values -> codes and, by the head's first lane, the scale.  LPH consecutive lanes hold a head; all lanes of
// the warp take part, those without a destination too.
template <int CODE, int LPH>
__device__ __forceinline__ void store_codes(float (&f)[16], uint8_t* d0, uint8_t* d1, float* scale, bool first) {
  constexpr float top = CODE == COLI_ATTN_CODE_INT8 ? 127.f : 448.f;
  uint32_t bits = 0;  // of the largest |x|: as integers, infinity and NaN are larger than all others
#pragma unroll
  for (int i = 0; i < 16; ++i) bits = max(bits, __float_as_uint(f[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 1; o < LPH; o <<= 1) bits = max(bits, __shfl_xor_sync(FULL, bits, o));
  if (!d0) return;
  float m = __uint_as_float(bits);
  const bool finite = bits < 0x7F800000u;
  if (first) *scale = finite ? __fdiv_rn(m, top) : __uint_as_float(0x7FFFFFFFu);
  // neither top * x may overflow nor a residual underflow
  const float fit = m >= 0x1p100f ? 0x1p-20f : m < 0x1p-60f ? 0x1p64f : 1.f;
  if (!finite || bits == 0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = 0.f;
    m = 1.f;
  } else if (fit != 1.f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] *= fit;
    m *= fit;
  }
  const float r = __frcp_rn(m);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float t = top * f[4 * k + i], q = t * r;
      y[i] = fmaf(fmaf(-q, m, t), r, q);
    }
    if constexpr (CODE == COLI_ATTN_CODE_INT8) {  // under the exponent of 2^23 the lowest byte is the nearest integer
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(y[i] + 12582912.f);
      w[k] = __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
    } else {
      uint16_t lo, hi;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y[1]), "f"(y[0]));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y[3]), "f"(y[2]));
      w[k] = (uint32_t)lo | (uint32_t)hi << 16;
    }
  }
  *reinterpret_cast<uint2*>(d0) = make_uint2(w[0], w[1]);
  *reinterpret_cast<uint2*>(d1) = make_uint2(w[2], w[3]);
}

// warps_per_token consecutive warps share a token's heads.  CODE: the type of an 8-bit cache, or 0
template <class T, int D, int CODE>
__global__ void __launch_bounds__(kAppendWarps * 32, blocks_per_sm(CODE)) attn_append_kernel(const AttnAppend a, int warps_per_token) {
  constexpr int LPH = D / 16, HPW = 32 / LPH;  // lanes per head, heads per warp
  constexpr int kAhead = ahead(CODE);
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t gw = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  const int token = (int)(gw / warps_per_token), part = (int)(gw - (int64_t)token * warps_per_token);
  if (token >= a.n_tokens) return;
  const int e = lane % LPH, sub = lane / LPH;  // 16 values e of head sub of a group of HPW heads
  const bool rot = e < a.rot / 16;
  // first value of the lane's two 8-value vectors
  const int i0 = rot && !a.interleaved ? 8 * e : 16 * e;
  const int i1 = rot && !a.interleaved ? a.rot / 2 + 8 * e : 16 * e + 8;
  const int nq = a.q ? a.n_q : 0;
  const int groups = (nq + 2 * a.n_kv + HPW - 1) / HPW;
  const auto source = [&](int h) -> const uint16_t* {
    if (h < nq) return static_cast<const uint16_t*>(a.q) + token * a.q_stride + (int64_t)h * D;
    if ((h -= nq) < a.n_kv) return static_cast<const uint16_t*>(a.k) + token * a.k_stride + (int64_t)h * D;
    if ((h -= a.n_kv) < a.n_kv) return static_cast<const uint16_t*>(a.v) + token * a.v_stride + (int64_t)h * D;
    return nullptr;
  };
  // the first values are asked for before the token's place is looked up
  uint4 x[kAhead], y[kAhead];
  const auto load = [&](int g) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int gk = g + k * warps_per_token;
      const uint16_t* src = gk < groups ? source(gk * HPW + sub) : nullptr;
      x[k] = y[k] = make_uint4(0, 0, 0, 0);
      if (src) {
        x[k] = __ldg(reinterpret_cast<const uint4*>(src + i0));
        y[k] = __ldg(reinterpret_cast<const uint4*>(src + i1));
      }
    }
  };
  load(part);

  int b = 0;  // the first sequence that ends after the token
  for (int b0 = 0; b0 < a.n_seqs; b0 += 32) {
    const bool before = b0 + lane < a.n_seqs && __ldg(a.q_start + b0 + lane + 1) <= token;
    const int n = __popc(__ballot_sync(FULL, before));
    b += n;
    if (n < 32) break;
  }
  if (b >= a.n_seqs) {  // the offsets end before n_tokens
    if (lane == 0) atomicExch(a.status, COLI_EINVAL);
    return;
  }
  const int start = __ldg(a.q_start + b), end = __ldg(a.q_start + b + 1), len = __ldg(a.kv_len + b);
  const int pos = len - (end - token);
  bool store = pos >= 0;
  // (where the offsets do not ascend, the sequence found need not hold the token)
  if (token < start || token >= end || end > a.n_tokens || len < 0 || (pos >> a.page_shift) >= a.max_pages) {
    if (lane == 0) atomicExch(a.status, COLI_EINVAL);
    store = false;
  }
  int64_t page = 0;
  if (store) page = __ldg(a.table + (int64_t)b * a.table_stride + (pos >> a.page_shift));
  float cs[8], sn[8];
#pragma unroll
  for (int w = 0; w < 8; ++w) cs[w] = 1.f, sn[w] = 0.f;
  if (rot) {
    const int64_t at = pos + (int64_t)(a.pos_base ? __ldg(a.pos_base) : 0);
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const uint64_t turn = __ldg(a.turn + 8 * e + w) * (uint64_t)at;
      // the top 32 bits as a signed fraction of a turn, times 2: in units of pi
      sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn[w], &cs[w]);
    }
  }
  if (store && (page < 0 || page >= a.n_pages)) {
    if (lane == 0) atomicExch(a.status, COLI_EINVAL);
    store = false;
  }
  const int64_t slot = pos & ((1 << a.page_shift) - 1);

#pragma unroll 1
  for (int g = part;;) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int gk = g + k * warps_per_token;
      if (gk >= groups) break;
      int h = gk * HPW + sub;
      if constexpr (CODE != 0) {
        if (gk * HPW + HPW > nq) {  // some of the warp's heads are keys or values
          float f[16], *scale = nullptr;
          uint8_t* d = nullptr;
          widen<T>(x[k], y[k], f);
          int g = h - nq;
          const bool value = g >= a.n_kv;
          if (rot && !value) rotate16(f, cs, sn, a.interleaved);
          if (value) g -= a.n_kv;
          if (store && h >= nq && g < a.n_kv) {
            d = static_cast<uint8_t*>(value ? a.vc : a.kc) + page * (value ? a.vp : a.kp) + g * (value ? a.vh : a.kh) +
                slot * (value ? a.vs : a.ks);
            scale = (value ? a.v_scale : a.k_scale) + page * (value ? a.vsp : a.ksp) + g * (value ? a.vsh : a.ksh) + slot;
          }
          // (a value's head is not rotated: its lanes hold the same columns, which are stored where they belong)
          store_codes<CODE, LPH>(f, d ? d + i0 : nullptr, d ? d + i1 : nullptr, scale, e == 0);
          if (h >= nq) continue;
        }
      }
      uint16_t* dst = nullptr;
      bool turn = rot;
      if (h < nq) {
        dst = static_cast<uint16_t*>(a.q_out) + token * a.q_out_stride + (int64_t)h * D;
      } else if ((h -= nq) < a.n_kv) {
        if (CODE == 0 && store) dst = static_cast<uint16_t*>(a.kc) + page * a.kp + h * a.kh + slot * a.ks;
      } else if ((h -= a.n_kv) < a.n_kv) {
        if (CODE == 0 && store) dst = static_cast<uint16_t*>(a.vc) + page * a.vp + h * a.vh + slot * a.vs;
        turn = false;
      }
      if (dst) {
        if (turn) rotate8<T>(x[k], y[k], cs, sn, a.interleaved);
        *reinterpret_cast<uint4*>(dst + i0) = x[k];
        *reinterpret_cast<uint4*>(dst + i1) = y[k];
      }
    }
    g += kAhead * warps_per_token;
    if (g >= groups) break;
    load(g);
  }
}

template <class T, int D, int CODE>
cudaError_t launch(const AttnAppend& a, int num_sms, cudaStream_t stream) {
  const int groups = ((a.q ? a.n_q : 0) + 2 * a.n_kv + 32 * 16 / D - 1) / (32 * 16 / D);
  // Enough warps to fill the GPU from few tokens, otherwise as few as possible per token, since each computes its token's
  // angles: double them up to 6 an SM.  us with 1 warp a token / up to 3, 6, 12, 32 an SM: 16 tokens 6.7 / 3.0, 3.0, 3.0, 3.0;
  // 250 - / 4.7, 3.6, 4.6, 5.9; 500 6.9 / 6.9, 4.7, 5.5, 8.5; 700 - / 6.8, 6.1, 5.6, 7.3; 2000 14.9 / 15.0 for all.
  // Into an 8-bit cache two at least, where a token has work for them (quantising takes more instructions).
  int wpt = CODE && groups >= 8 ? 2 : 1;
  while (wpt < groups && (int64_t)a.n_tokens * wpt < (int64_t)num_sms * 6) wpt *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((int64_t)a.n_tokens * wpt + kAppendWarps - 1) / kAppendWarps));
  cfg.blockDim = dim3(kAppendWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_append_kernel<T, D, CODE>, a, wpt);
}

template <class T, int D>
cudaError_t launch_code(const AttnAppend& a, int num_sms, cudaStream_t stream) {
  if (a.code == COLI_ATTN_CODE_INT8) return launch<T, D, COLI_ATTN_CODE_INT8>(a, num_sms, stream);
  if (a.code == COLI_ATTN_CODE_E4M3) return launch<T, D, COLI_ATTN_CODE_E4M3>(a, num_sms, stream);
  return launch<T, D, 0>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_attn_append(const AttnAppend& a, int dtype, int num_sms, cudaStream_t stream) {
  if (dtype == COLI_ATTN_BF16)
    return a.head_dim == 64 ? launch_code<Bf16, 64>(a, num_sms, stream) : launch_code<Bf16, 128>(a, num_sms, stream);
  return a.head_dim == 64 ? launch_code<Fp16, 64>(a, num_sms, stream) : launch_code<Fp16, 128>(a, num_sms, stream);
}

}  // namespace coli

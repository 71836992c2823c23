// Attention of few query rows over a paged cache: o = softmax(scale q K^T) V with a running
// maximum and sum, one pass over the keys.
//
// A block is up to 16 or 32 rows: the query heads of one key head times the tokens of one sequence.  At such
// sizes every key and value byte is used by few rows, so the kernel is bound by HBM and is built around the
// copies: one warp keeps a ring of key tiles (64 keys, K and V) full with tensor copies straight from the
// pages, and the other four each take 16 or 32 keys of a tile for 16 rows with mma.sync and a running
// softmax of their own, joined once at the end of the unit, so nothing but the ring synchronises them.
// Legacy mma.sync suffices: the tensor pipe is 15 % busy while DRAM is at its limit, and its fragments keep
// P in registers.  Two CTAs an SM: while one joins its warps the other's copies run on.  The list of all
// units' key tiles is cut into equal stretches, one per CTA, so a single long sequence and many short ones
// fill the GPU alike.
//
// Measured, with the combine kernel: 64 sequences' next tokens, 6 query heads a key head, 8 key heads of 128,
// windows of 4096 keys: 1.08 GB in 174 us, 6.2 TB/s (a copy reaches 6.78).  One sequence and 516 keys: 9.2 us, of
// which two launches, the placement and the first tile's way from DRAM take nearly all.
#include "attn_device.cuh"

namespace coli {

namespace {

template <int D, int RG>
struct SplitCfg {
  static constexpr int KG = 4 / RG;  // key groups: warps that share 16 rows
  static constexpr int warps = 4;
  static constexpr int threads = (warps + 1) * 32;
  static constexpr int rows = RG * 16;
  static constexpr int kw = kSplitKeys / KG;  // keys per warp and tile
  static constexpr int ctas = 2;  // per SM
  static constexpr int tile_bytes = kSplitKeys * D * 2;
  static constexpr int stages = 98304 / (2 * tile_bytes);
  static constexpr int merge_bytes = 4 * (8 * D + 32) * 4;  // a buffer a warp: half its columns
  static constexpr int smem = stages * 2 * tile_bytes + merge_bytes + 2 * stages * 8 + (int)sizeof(UnitRing) + 24;
};

// 16 rows, at positions p0..p1, x kw keys of one tile for one warp.  bad: a value that is not finite and that
// only some of the rows see has gone into products with the others' zero weights.
template <class T, int D, int RG, bool Masked>
__device__ __forceinline__ void tile_step(const AttnParams& p, uint32_t ks, uint32_t vs, int key0,
                                          int p0, int p1, const int (&pos)[2],
                                          const uint32_t (&qf)[D / 16][4], float (&o)[D / 8][4],
                                          float (&mx)[2], float (&sum)[2], uint32_t& bad, int lane) {
  using C = SplitCfg<D, RG>;
  constexpr int NT = C::kw / 8;
  const int c2 = (lane & 3) * 2;
  float s[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
  const int kloc = key0 & (kSplitKeys - 1);  // the warp's first key within the tile
#pragma unroll
  for (int n = 0; n < NT; n += 2) {
    const int row = kloc + n * 8 + ((lane >> 4) << 3) + (lane & 7);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const int ch = (k * 2 + ((lane >> 3) & 1));
      uint32_t b[4];
      ldsm4(ks + (ch >> 3) * kSplitKeys * 128 + row * 128 + (((ch & 7) ^ (row & 7)) << 4), b);
      mma16816<T>(s[n], qf[k], b[0], b[1]);
      mma16816<T>(s[n + 1], qf[k], b[2], b[3]);
    }
  }
  if (Masked) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!sees(p, pos[i >> 1], key0 + n * 8 + c2 + (i & 1))) s[n][i] = -INFINITY;
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    float m = mx[r];
#pragma unroll
    for (int n = 0; n < NT; ++n) m = fmaxf(m, fmaxf(s[n][2 * r], s[n][2 * r + 1]));
    m = fmaxf(m, __shfl_xor_sync(FULL, m, 1));
    m = fmaxf(m, __shfl_xor_sync(FULL, m, 2));
    const float base = m == -INFINITY ? 0.f : m * p.scale_log2;
    const float fix = ex2(mx[r] * p.scale_log2 - base);  // mx = -inf: 0, and o, sum are 0
    mx[r] = m;
    float a = 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float e = ex2(fmaf(s[n][2 * r + i], p.scale_log2, -base));
        s[n][2 * r + i] = e;
        a += e;
      }
    sum[r] = fmaf(sum[r], fix, a);  // this thread's share of the row; joined at the end
#pragma unroll
    for (int d = 0; d < D / 8; ++d) {
      o[d][2 * r] *= fix;
      o[d][2 * r + 1] *= fix;
    }
  }
#pragma unroll
  for (int n = 0; n < NT; n += 2) {
    const uint32_t pf[4] = {T::pack(s[n][0], s[n][1]), T::pack(s[n][2], s[n][3]),
                            T::pack(s[n + 1][0], s[n + 1][1]), T::pack(s[n + 1][2], s[n + 1][3])};
    const int row = kloc + n * 8 + (lane & 15);
    const int kk = key0 + n * 8 + c2;
    uint32_t z0 = 0xFFFFFFFFu, z1 = 0xFFFFFFFFu;  // values of keys that no row sees become 0
    if (Masked) {
      z0 = (some_sees(p, p0, p1, kk) ? 0xFFFFu : 0u) | (some_sees(p, p0, p1, kk + 1) ? 0xFFFF0000u : 0u);
      z1 = (some_sees(p, p0, p1, kk + 8) ? 0xFFFFu : 0u) |
           (some_sees(p, p0, p1, kk + 9) ? 0xFFFF0000u : 0u);
    }
#pragma unroll
    for (int d = 0; d < D / 16; ++d) {
      const int ch = d * 2 + (lane >> 4);
      uint32_t b[4];
      ldsm4t(vs + (ch >> 3) * kSplitKeys * 128 + row * 128 + (((ch & 7) ^ (row & 7)) << 4), b);
      if (Masked) {
        b[0] &= z0, b[2] &= z0;
        b[1] &= z1, b[3] &= z1;
        bad |= nonfinite2<T>(b[0]) | nonfinite2<T>(b[1]) | nonfinite2<T>(b[2]) | nonfinite2<T>(b[3]);
      }
      mma16816<T>(o[2 * d], pf, b[0], b[1]);
      mma16816<T>(o[2 * d + 1], pf, b[2], b[3]);
    }
  }
}

// Buffer of a warp: H 8-column groups of its 16 rows in fragment order, then the rows' maxima and sums.
template <int D, int H>
__device__ __forceinline__ void hand_over(float* merge, int buffer, const float (&o)[D / 8][4], int first,
                                          const float (&mx)[2], const float (&sum)[2], int lane) {
  float* base = merge + buffer * (8 * D + 32);
  float4* buf = reinterpret_cast<float4*>(base);
#pragma unroll
  for (int d = 0; d < D / 8; ++d)
    if ((d / H) * H == first) buf[(d % H) * 32 + lane] = make_float4(o[d][0], o[d][1], o[d][2], o[d][3]);
  if ((lane & 3) == 0) {
    float2* ml = reinterpret_cast<float2*>(base + 8 * D);
    ml[lane >> 2] = make_float2(mx[0], sum[0]);
    ml[(lane >> 2) + 8] = make_float2(mx[1], sum[1]);
  }
}
template <int D, int H>
__device__ __forceinline__ void take_over(const float* merge, int buffer, float (&o)[D / 8][4], int first,
                                          float scale_log2, float (&mx)[2], float (&sum)[2], int lane) {
  const float* base = merge + buffer * (8 * D + 32);
  const float4* buf = reinterpret_cast<const float4*>(base);
  const float2* ml = reinterpret_cast<const float2*>(base + 8 * D);
  float fa[2], fb[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const float2 other = ml[(lane >> 2) + r * 8];
    const float m = fmaxf(mx[r], other.x);
    const float base2 = m == -INFINITY ? 0.f : m * scale_log2;
    fa[r] = ex2(mx[r] * scale_log2 - base2);
    fb[r] = ex2(other.x * scale_log2 - base2);
    mx[r] = m;
    sum[r] = sum[r] * fa[r] + other.y * fb[r];
  }
#pragma unroll
  for (int d = 0; d < D / 8; ++d)
    if ((d / H) * H == first) {
      const float4 v = buf[(d % H) * 32 + lane];
      o[d][0] = o[d][0] * fa[0] + v.x * fb[0];
      o[d][1] = o[d][1] * fa[0] + v.y * fb[0];
      o[d][2] = o[d][2] * fa[1] + v.z * fb[1];
      o[d][3] = o[d][3] * fa[1] + v.w * fb[1];
    }
}

template <class T, int D, int RG>
__global__ void __launch_bounds__(SplitCfg<D, RG>::threads, SplitCfg<D, RG>::ctas)
    attn_split_kernel(const AttnParams p, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap) {
  using C = SplitCfg<D, RG>;
  constexpr int NST = C::stages;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* merge = reinterpret_cast<float*>(smem + NST * 2 * C::tile_bytes);
  UnitRing* units = reinterpret_cast<UnitRing*>(smem + NST * 2 * C::tile_bytes + C::merge_bytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(units + 1);
  uint64_t *empty = full + NST, *met = empty + NST;
  // (no static shared memory: with it, two CTAs of 16 rows would no longer fit one SM)
  int* abort_flag = reinterpret_cast<int*>(met + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const auto wait = [&](uint64_t* bar, uint32_t parity) { return warp_wait(bar, parity, abort_flag, p.status); };

  if (tid == 0) {
    *abort_flag = 0;
    units->init(C::warps);
    for (int i = 0; i < NST; ++i) mbar_init(full + i, 1), mbar_init(empty + i, C::warps);
    mbar_init(met, C::warps);
    fence_barrier_init();
    prefetch_map(&kmap);
    prefetch_map(&vmap);
  }
  uint32_t* weights = reinterpret_cast<uint32_t*>(smem);  // in the ring, before the first copy
  const bool few = n_lists(p) <= 32;
  Walk<kSplitKeys> walk;
  if (few) {
    __syncthreads();
    if (warp == C::warps) {
#pragma unroll 1
      for (int real = 0; real < 2; ++real) {
        if (real) griddep_wait();
        walk.start_few(p, lane, real);
      }
    } else {
      griddep_wait();
    }
  } else {
    griddep_wait();
    weigh<kSplitKeys>(p, weights);
  }
  griddep_launch_dependents();

  if (warp == C::warps) {  // ---- copies
    if (!few) walk.start(p, weights, lane);
    if (lane == 0) p.rec[blockIdx.x].first_cta = -1;
    __syncwarp();
    fence_proxy_async_smem();
    int it = 0, n = 0;
    Unit u;
    bool ok = true;
    while (ok && walk.next(p, u)) {
      ok = give_unit(units, u, n++, lane, wait);
      const int32_t* row = table_of(p, u.b);
#pragma unroll 1
      for (int i = u.i0; i < u.i1 && ok; ++i, ++it) {
        const int sgi = it % NST;
        if (it >= NST) ok = wait(empty + sgi, ((it / NST) + 1) & 1);
        if (!ok) break;
        uint8_t* dst = smem + sgi * 2 * C::tile_bytes;
        fill_boxes<kSplitKeys, D, 2>(p, &kmap, &vmap, dst, full + sgi, row, u.p0, u.p1, u.tile(i) * kSplitKeys, u.head, lane);
      }
    }
    u.i1 = 0;
    if (ok) give_unit(units, u, n, lane, wait);
    // the CTA's shared memory must not go while copies to it are on their way, even when the other warps have given up
    drain_ring(full, NST, it);
    return;
  }

  // ---- products
  const int rg = warp % RG, kg = warp / RG;
  const int row0 = rg * 16;  // this warp's rows of the block
  uint32_t meetings = 0;
  // the product warps wait for one another (bounded: one that gave up must not leave the others behind)
  const auto meet = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(met);
    return wait(met, meetings++ & 1);
  };
  int it = 0;
  Unit u;
  for (int n = 0; take_unit(units, u, n, lane, wait); ++n) {
    const int tok0 = u.tok0, nt = u.nt, p0 = u.p0;
    const bool causal = u.flags & kCausal, whole = u.flags & kWhole;
    float* const dense_o = p.dense_o[causal ? 0 : 1];
    float2* const dense_ml = p.dense_ml[causal ? 0 : 1];
    int pos[2], tok[2];
    bool live[2];
    uint32_t qf[D / 16][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = row0 + (lane >> 2) + r * 8;
      tok[r] = row / p.group;
      live[r] = tok[r] < nt;
      pos[r] = causal ? p0 + tok[r] : p0;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(
          static_cast<const uint16_t*>(p.q) + (int64_t)(tok0 + tok[r]) * p.q_stride +
          (int64_t)(u.head * p.group + row - tok[r] * p.group) * D);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qf[k][r] = live[r] ? __ldg(src + k * 8 + (lane & 3)) : 0u;
        qf[k][r + 2] = live[r] ? __ldg(src + k * 8 + 4 + (lane & 3)) : 0u;
      }
    }
    // the warp's own tokens and their positions
    const int tok_lo = row0 / p.group, tok_hi = min(nt - 1, (row0 + 15) / p.group);
    const int w0 = causal ? p0 + tok_lo : p0, w1 = causal ? p0 + tok_hi : p0;
    uint32_t bad = 0;
    float o[D / 8][4], mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
    for (int d = 0; d < D / 8; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[d][i] = 0.f;

#pragma unroll 1
    for (int i = u.i0; i < u.i1; ++i, ++it) {
      const int sgi = it % NST;
      if (!wait(full + sgi, (it / NST) & 1)) return;
      {
        const uint32_t ks = smem_addr(smem + sgi * 2 * C::tile_bytes), vs = ks + C::tile_bytes;
        const int key0 = u.tile(i) * kSplitKeys + kg * C::kw;
        if (tok_lo >= nt) {
        } else if (all_see(p, w0, w1, key0, key0 + C::kw - 1)) {
          tile_step<T, D, RG, false>(p, ks, vs, key0, w0, w1, pos, qf, o, mx, sum, bad, lane);
        } else {
          tile_step<T, D, RG, true>(p, ks, vs, key0, w0, w1, pos, qf, o, mx, sum, bad, lane);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + sgi);
    }
    if (tok_hi > tok_lo && __any_sync(FULL, bad != 0)) flag_unit(p, u, lane);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      sum[r] += __shfl_xor_sync(FULL, sum[r], 1);
      sum[r] += __shfl_xor_sync(FULL, sum[r], 2);
    }
    // Join the KG warps that share these rows.  Each step halves the columns a warp keeps: it hands the other
    // half to its partner and takes its own half's counterpart, so the last step leaves every warp
    // D / KG finished columns.  Buffer A_w holds what was handed to warp w; only w reads it in the first step and
    // writes its second handover there.
    constexpr int NC = D / 8 / C::KG;  // 8-column groups a warp ends with
    int col = 0;                       // the first of them
    {
      constexpr int H = D / 16;
      if (!meet()) return;  // the buffers are free
      const int other = rg + RG * (kg ^ (C::KG / 2));
      const bool up = kg & (C::KG / 2);
      hand_over<D, H>(merge, other, o, up ? 0 : H, mx, sum, lane);
      if (!meet()) return;
      take_over<D, H>(merge, warp, o, up ? H : 0, p.scale_log2, mx, sum, lane);
      col = up ? H : 0;
    }
    if (C::KG > 2) {
      constexpr int H = D / 32;
      const bool up = kg & 1;
      hand_over<D, H>(merge, warp, o, col + (up ? 0 : H), mx, sum, lane);
      if (!meet()) return;
      take_over<D, H>(merge, rg + RG * (kg ^ 1), o, col + (up ? H : 0), p.scale_log2, mx, sum, lane);
      col += up ? H : 0;
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = row0 + (lane >> 2) + r * 8;
      const float m2 = mx[r] * p.scale_log2;  // -inf stays -inf
      const int hq = u.head * p.group + row - tok[r] * p.group;
      if (whole && !live[r]) continue;
      if (whole && !dense_o) {
        const float inv = sum[r] == 0.f ? 0.f : 1.f / sum[r];
        uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) +
                                                    (int64_t)(tok0 + tok[r]) * p.out_stride + (int64_t)hq * D);
#pragma unroll
        for (int d = 0; d < D / 8; ++d)
          if ((d / NC) * NC == col)
            dst[d * 4 + (lane & 3)] = T::pack(o[d][2 * r] * inv, o[d][2 * r + 1] * inv);
        if (p.lse && kg == 0 && (lane & 3) == 0)
          p.lse[(int64_t)(tok0 + tok[r]) * p.n_q + hq] =
              sum[r] == 0.f ? -INFINITY : (m2 + log2f(sum[r])) * 0.69314718055994530942f;
      } else {
        const int64_t at = whole ? (int64_t)(tok0 + tok[r]) * p.n_q + hq
                                 : ((int64_t)blockIdx.x * 2 + (u.i0 > 0 ? 0 : 1)) * C::rows + row;
        float* dst = whole ? dense_o : p.part_o;
#pragma unroll
        for (int d = 0; d < D / 8; ++d)
          if ((d / NC) * NC == col)
            *reinterpret_cast<float2*>(dst + at * D + d * 8 + (lane & 3) * 2) =
                make_float2(o[d][2 * r], o[d][2 * r + 1]);
        if (kg == 0 && (lane & 3) == 0) (whole ? dense_ml : p.part_ml)[at] = make_float2(m2, sum[r]);
      }
    }
  }
}

template <class T, int D, int RG>
cudaError_t configure() {
  return cudaFuncSetAttribute(attn_split_kernel<T, D, RG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              SplitCfg<D, RG>::smem);
}

template <class T, int D, int RG>
cudaError_t launch(const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, int grid,
                   cudaStream_t stream) {
  using C = SplitCfg<D, RG>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(C::threads);
  cfg.dynamicSmemBytes = C::smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_split_kernel<T, D, RG>, p, k, v);
}

template <class T, int D>
cudaError_t launch_rows(const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, int rows,
                        int grid, cudaStream_t stream) {
  return rows == 16 ? launch<T, D, 1>(p, k, v, grid, stream) : launch<T, D, 2>(p, k, v, grid, stream);
}

}  // namespace

int split_rows(int64_t rows) { return rows <= 16 ? 16 : kSplitMaxRows; }
int split_grid(int num_sms) { return 2 * num_sms; }

cudaError_t configure_attn_split() {
  cudaError_t e = cudaSuccess;
#define COLI_CFG(T, D)                                  \
  if (e == cudaSuccess) e = configure<T, D, 1>();       \
  if (e == cudaSuccess) e = configure<T, D, 2>();
  COLI_CFG(Bf16, 64) COLI_CFG(Bf16, 128) COLI_CFG(Fp16, 64) COLI_CFG(Fp16, 128)
#undef COLI_CFG
  return e;
}

cudaError_t launch_attn_split(const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v,
                              int rows, int dtype, int num_sms, cudaStream_t stream) {
  const int grid = split_grid(num_sms);
  if (dtype == COLI_ATTN_BF16)
    return p.head_dim == 64 ? launch_rows<Bf16, 64>(p, k, v, rows, grid, stream)
                            : launch_rows<Bf16, 128>(p, k, v, rows, grid, stream);
  return p.head_dim == 64 ? launch_rows<Fp16, 64>(p, k, v, rows, grid, stream)
                          : launch_rows<Fp16, 128>(p, k, v, rows, grid, stream);
}

}  // namespace coli

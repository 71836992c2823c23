// Attention of few query rows over a paged cache of 8-bit codes with a scale for each token and key head:
//   s_j = scale * ks_j * (q . kc_j),  o = sum_j softmax(s)_j vs_j vc_j
// in one pass over the keys, with attn_split.cu's plan: a warp copies tiles of 64 keys, four warps take 16 or 32 of a
// tile's keys for 16 rows each, the list of all units' tiles is cut into equal stretches.
//
// The codes are widened on their way from shared memory to mma.sync, which is exact: keys to the queries' type, values to fp16, the
// weights' type.  Weights: 2^(s_j - m) vs_j, where m follows the row's largest s_j + log2 |vs_j| to within 2^8, so that they do not run
// out of fp16's range, and neither what a row does not see nor a large value without weight has a part in it; they are rounded to fp16
// once.  m rarely grows, and the accumulators are rescaled only then.
//
// A lane's codes of a key are contiguous in shared memory (the order of the products' inner dimension is free as long as the
// queries follow it), and a 16-bit transposing load of the values brings two columns' codes of a key in one half, so
// both operands take one widening of a word for four codes: to fp16 5 instructions (int8) or 7 (e4m3), to bf16 8 or 9.
//
// Measured, with the combine kernel: 64 sequences' next tokens, 6 query heads a key head, 8 key heads of 128, windows of 4096 keys: 556 MB
// in bf16 with int8 117 us, 4.8 TB/s, with e4m3 122.2, in fp16 105.9 and 121.0; the copies alone take 97 (pages of 8 KB a head in random
// order).  Keys as fp16 for bf16 queries too took 6 us less (and 0.5 us more for one token), which holds only queries whose values are within
// 2^31 of one another.  Beside 111 of an earlier form: three CTAs an SM (128 registers) 112, 32 keys a warp of every other tile 110 and
// 11.4 instead of 10.1 for one token, the queries' fragments in registers 141.
#include "attn_code.cuh"

namespace coli {

namespace {

constexpr float kSlack = 8.f;  // of a row's m

template <int D, int RG>
struct QSplitCfg {
  static constexpr int KG = 4 / RG;  // key groups: warps that share 16 rows
  static constexpr int warps = 4;
  static constexpr int threads = (warps + 1) * 32;
  static constexpr int rows = RG * 16;
  static constexpr int kw = kSplitKeys / KG;  // keys per warp and tile
  static constexpr int ctas = 2;  // per SM
  static constexpr int tile_bytes = kSplitKeys * D;
  static constexpr int stages = 81920 / (2 * tile_bytes);
  static constexpr int scale_bytes = stages * 2 * kSplitKeys * 4;
  // a buffer a warp, of half its columns; between joins, the queries' fragments of RG x 16 rows
  static constexpr int merge_bytes = 4 * (8 * D + 32) * 4;
  static_assert(merge_bytes >= RG * (D / 16) * 512, "the queries fit");
  static constexpr int smem =
      stages * 2 * tile_bytes + scale_bytes + merge_bytes + 2 * stages * 8 + (int)sizeof(UnitRing) + 24;
};


// 16-byte chunk `ch` of row `row` of a code tile, as the tensor copies swizzle it: rows of 128 bytes by row % 8, of 64
// bytes by row / 2 % 4
template <int D>
__device__ __forceinline__ uint32_t code_chunk(int row, int ch) {
  return D == 128 ? row * 128 + ((ch ^ (row & 7)) << 4) : row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// the larger of two, NaN where one is
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// What a thread keeps of its two rows (lane / 4 and 8 more).
template <int D>
struct Rows {
  float o[D / 8][4];  // columns 16 c + 4 (lane % 4) + 0, 2 in o[2c], 1, 3 in o[2c + 1]
  float m[2], sum[2];  // o and sum are in units of 2^m
};

// 16 rows at positions pos x kw keys of one tile for one warp; rs: score of a product of codes and q, times log2(e); q: its rows' fragments, ks: the keys' codes (the values' D * 64 bytes
// further), all shared-memory addresses.  Step k of the fragments: of the D / 4 values from (lane % 4) D / 4 on, values 4k and 4k + 2,
// 4k + 1 and 4k + 3
template <class T, int CODE, int D, int RG, bool Masked>
__device__ __forceinline__ void tile_step(const AttnParams& p, float rs, uint32_t q, uint32_t ks, const float* scales, int key0,
                                          const int (&pos)[2], Rows<D>& r, int lane) {
  using C = QSplitCfg<D, RG>;
  constexpr int NT = C::kw / 8;
  const int c2 = (lane & 3) * 2;
  const int kloc = key0 & (kSplitKeys - 1);  // the warp's first key within the tile
  float s[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
#pragma unroll
  for (int h = 0; h < D / 64; ++h) {
    uint4 v[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) v[n] = lds128(ks + code_chunk<D>(kloc + n * 8 + (lane >> 2), (lane & 3) * (D / 64) + h));
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint4 f = lds128(q + (h * 4 + t) * 512 + lane * 16);
      const uint32_t a[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t b0, b1;
        Code<CODE>::template widen<T>(t == 0 ? v[n].x : t == 1 ? v[n].y : t == 2 ? v[n].z : v[n].w, b0, b1);
        mma16816<T>(s[n], a, b0, b1);
      }
    }
  }
  uint32_t see = 0xFFFFFFFFu;  // bit 4n + i: the row sees the key of s[n][i]
  if (Masked) {
    see = 0;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (sees(p, pos[i >> 1], key0 + n * 8 + c2 + (i & 1))) see |= 1u << (4 * n + i);
  }
  float vs[NT][2], m[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float2 k2 = *reinterpret_cast<const float2*>(scales + kloc + n * 8 + c2);
    const float2 v2 = *reinterpret_cast<const float2*>(scales + kSplitKeys + kloc + n * 8 + c2);
    vs[n][0] = v2.x, vs[n][1] = v2.y;
    const float k[2] = {spoil(k2.x) * rs, spoil(k2.y) * rs}, lv[2] = {scale_log(v2.x), scale_log(v2.y)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[n][i] *= k[i & 1];
      if (Masked && !(see >> (4 * n + i) & 1)) s[n][i] = -INFINITY;
      else m[i >> 1] = max_nan(m[i >> 1], s[n][i] + lv[i & 1]);
    }
  }
  // (a NaN is above any m)
  if (__any_sync(FULL, !(m[0] <= r.m[0] + kSlack) || !(m[1] <= r.m[1] + kSlack))) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float a = max_nan(m[i], r.m[i]);
      a = max_nan(a, __shfl_xor_sync(FULL, a, 1));
      a = max_nan(a, __shfl_xor_sync(FULL, a, 2));
      // A row moves when its own keys ask for it, whatever the others of the warp do: rows without a token see slots that nobody has
      // asked for, and a row's roundings must not depend on those.
      if (a <= r.m[i] + kSlack) continue;
      if (!(a < INFINITY)) {  // a scale or score that is not finite
        r.sum[i] = NAN;
        continue;
      }
      const float fix = ex2(r.m[i] - a);  // m = -inf: 0, and o, sum are 0
      r.m[i] = a, r.sum[i] *= fix;
#pragma unroll
      for (int d = 0; d < D / 8; ++d) r.o[d][2 * i] *= fix, r.o[d][2 * i + 1] *= fix;
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float base = r.m[i] == -INFINITY ? 0.f : r.m[i];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float e = ex2(s[n][2 * i + k] - base);
        r.sum[i] += e;  // this thread's share of the row; joined at the end
        float w = e * vs[n][k];
        if (Masked && !(see >> (4 * n + 2 * i + k) & 1)) w = 0.f;  // (its scale may be NaN)
        s[n][2 * i + k] = w;
      }
  }
#pragma unroll
  for (int n = 0; n < NT; n += 2) {
    const uint32_t pf[4] = {Fp16::pack(s[n][0], s[n][1]), Fp16::pack(s[n][2], s[n][3]),
                            Fp16::pack(s[n + 1][0], s[n + 1][1]), Fp16::pack(s[n + 1][2], s[n + 1][3])};
    const int row = kloc + n * 8 + (lane & 15);
#pragma unroll
    for (int c = 0; c < D / 16; c += 2) {
      uint32_t b[4], x[2], y[2];
      ldsm4t(ks + kSplitKeys * D + code_chunk<D>(row, c + (lane >> 4)), b);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        Code<CODE>::template widen<Fp16>(b[2 * h], x[0], y[0]);
        Code<CODE>::template widen<Fp16>(b[2 * h + 1], x[1], y[1]);
        mma16816<Fp16>(r.o[2 * (c + h)], pf, x[0], x[1]);
        mma16816<Fp16>(r.o[2 * (c + h) + 1], pf, y[0], y[1]);
      }
    }
  }
}

// Buffer of a warp: H 8-column groups of its 16 rows in fragment order, then the rows' units and sums.
template <int D, int H>
__device__ __forceinline__ void hand_over(float* merge, int buffer, const Rows<D>& r, int first, int lane) {
  float* base = merge + buffer * (8 * D + 32);
  float4* buf = reinterpret_cast<float4*>(base);
#pragma unroll
  for (int d = 0; d < D / 8; ++d)
    if ((d / H) * H == first) buf[(d % H) * 32 + lane] = make_float4(r.o[d][0], r.o[d][1], r.o[d][2], r.o[d][3]);
  if ((lane & 3) == 0) {
    float2* ml = reinterpret_cast<float2*>(base + 8 * D);
    ml[lane >> 2] = make_float2(r.m[0], r.sum[0]);
    ml[(lane >> 2) + 8] = make_float2(r.m[1], r.sum[1]);
  }
}
template <int D, int H>
__device__ __forceinline__ void take_over(const float* merge, int buffer, Rows<D>& r, int first, int lane) {
  const float* base = merge + buffer * (8 * D + 32);
  const float4* buf = reinterpret_cast<const float4*>(base);
  const float2* ml = reinterpret_cast<const float2*>(base + 8 * D);
  float fa[2], fb[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 other = ml[(lane >> 2) + i * 8];
    const float m = fmaxf(r.m[i], other.x), at = m == -INFINITY ? 0.f : m;
    fa[i] = ex2(r.m[i] - at);
    fb[i] = ex2(other.x - at);
    r.m[i] = m;
    r.sum[i] = r.sum[i] * fa[i] + other.y * fb[i];
  }
#pragma unroll
  for (int d = 0; d < D / 8; ++d)
    if ((d / H) * H == first) {
      const float4 v = buf[(d % H) * 32 + lane];
      r.o[d][0] = r.o[d][0] * fa[0] + v.x * fb[0];
      r.o[d][1] = r.o[d][1] * fa[0] + v.y * fb[0];
      r.o[d][2] = r.o[d][2] * fa[1] + v.z * fb[1];
      r.o[d][3] = r.o[d][3] * fa[1] + v.w * fb[1];
    }
}

template <class T, int CODE, int D, int RG>
__global__ void __launch_bounds__(QSplitCfg<D, RG>::threads, QSplitCfg<D, RG>::ctas)
    attn_qsplit_kernel(const AttnParams p, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap) {
  using C = QSplitCfg<D, RG>;
  constexpr int NST = C::stages;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* scales = reinterpret_cast<float*>(smem + NST * 2 * C::tile_bytes);
  float* merge = reinterpret_cast<float*>(smem + NST * 2 * C::tile_bytes + C::scale_bytes);
  UnitRing* units = reinterpret_cast<UnitRing*>(smem + NST * 2 * C::tile_bytes + C::scale_bytes + C::merge_bytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(units + 1);
  uint64_t *empty = full + NST, *met = empty + NST;
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
        fill_codes<kSplitKeys, D>(p, &kmap, &vmap, dst, dst + C::tile_bytes, scales + sgi * 2 * kSplitKeys, full + sgi, row,
                                  u.p0, u.p1, u.tile(i) * kSplitKeys, u.head, lane);
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
    if (n > 0 && !meet()) return;  // the last unit's sums have been taken over
    const int tok0 = u.tok0, nt = u.nt, p0 = u.p0;
    const bool whole = u.flags & kWhole;
    int pos[2], tok[2];
    bool live[2];
    Rows<D> r;
    const float rs = p.scale_log2 * Code<CODE>::unit;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = row0 + (lane >> 2) + i * 8;
      tok[i] = row / p.group;
      live[i] = tok[i] < nt;
      pos[i] = p0 + tok[i];
      uint32_t x[D / 8];
#pragma unroll
      for (int k = 0; k < D / 8; ++k) x[k] = 0;
      if (live[i]) {
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(p.q) + (int64_t)(tok0 + tok[i]) * p.q_stride +
            (int64_t)(u.head * p.group + row - tok[i] * p.group) * D + (lane & 3) * (D / 4));
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          const uint4 v = __ldg(src + k);
          x[4 * k] = v.x, x[4 * k + 1] = v.y, x[4 * k + 2] = v.z, x[4 * k + 3] = v.w;
        }
      }
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        if (k % C::KG != kg) continue;  // the others' share
        uint32_t* at = reinterpret_cast<uint32_t*>(merge) + ((rg * (D / 16) + k) * 32 + lane) * 4 + i;
        at[0] = __byte_perm(x[2 * k], x[2 * k + 1], 0x5410);
        at[2] = __byte_perm(x[2 * k], x[2 * k + 1], 0x7632);
      }
      r.m[i] = -INFINITY, r.sum[i] = 0.f;
    }
    if (!meet()) return;  // all fragments are there
    const uint32_t q_at = smem_addr(merge) + rg * (D / 16) * 512;
    // the warp's own tokens and their positions
    const int tok_lo = row0 / p.group, tok_hi = min(nt - 1, (row0 + 15) / p.group);
    const int w0 = p0 + tok_lo, w1 = p0 + tok_hi;
#pragma unroll
    for (int d = 0; d < D / 8; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) r.o[d][i] = 0.f;

#pragma unroll 1
    for (int i = u.i0; i < u.i1; ++i, ++it) {
      const int sgi = it % NST;
      if (!wait(full + sgi, (it / NST) & 1)) return;
      if (tok_lo < nt) {
        const uint32_t ks = smem_addr(smem + sgi * 2 * C::tile_bytes);
        const float* sc = scales + sgi * 2 * kSplitKeys;
        const int key0 = u.tile(i) * kSplitKeys + kg * C::kw;
        if (all_see(p, w0, w1, key0, key0 + C::kw - 1))
          tile_step<T, CODE, D, RG, false>(p, rs, q_at, ks, sc, key0, pos, r, lane);
        else
          tile_step<T, CODE, D, RG, true>(p, rs, q_at, ks, sc, key0, pos, r, lane);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + sgi);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      r.sum[i] += __shfl_xor_sync(FULL, r.sum[i], 1);
      r.sum[i] += __shfl_xor_sync(FULL, r.sum[i], 2);
    }
    // Join the KG warps that share these rows.  Each step halves the columns a warp keeps: it hands the other
    // half to its partner and takes its own half's counterpart, so the last step leaves every warp
    // D / KG finished columns.  Buffer A_w holds what was handed to warp w; only w reads it in the first step and
    // writes its second handover there.
    constexpr int NC = D / 8 / C::KG;  // 8-column groups a warp ends with
    int col = 0;                       // the first of them
    {
      constexpr int H = D / 16;
      if (!meet()) return;  // nobody reads the queries any more
      const int other = rg + RG * (kg ^ (C::KG / 2));
      const bool up = kg & (C::KG / 2);
      hand_over<D, H>(merge, other, r, up ? 0 : H, lane);
      if (!meet()) return;
      take_over<D, H>(merge, warp, r, up ? H : 0, lane);
      col = up ? H : 0;
    }
    if (C::KG > 2) {
      constexpr int H = D / 32;
      const bool up = kg & 1;
      hand_over<D, H>(merge, warp, r, col + (up ? 0 : H), lane);
      if (!meet()) return;
      take_over<D, H>(merge, rg + RG * (kg ^ 1), r, col + (up ? H : 0), lane);
      col += up ? H : 0;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = row0 + (lane >> 2) + i * 8;
      const float m2 = r.m[i], unit = Code<CODE>::unit;
      const int hq = u.head * p.group + row - tok[i] * p.group;
      if (whole && !live[i]) continue;
      if (whole) {
        const float inv = r.sum[i] == 0.f ? 0.f : unit / r.sum[i];
        uint16_t* dst = static_cast<uint16_t*>(p.out) + (int64_t)(tok0 + tok[i]) * p.out_stride + (int64_t)hq * D;
#pragma unroll
        for (int d = 0; d < D / 8; d += 2)
          if ((d / NC) * NC == col)
            *reinterpret_cast<uint2*>(dst + d * 8 + (lane & 3) * 4) =
                make_uint2(T::pack(r.o[d][2 * i] * inv, r.o[d + 1][2 * i] * inv),
                           T::pack(r.o[d][2 * i + 1] * inv, r.o[d + 1][2 * i + 1] * inv));
        if (p.lse && kg == 0 && (lane & 3) == 0)
          p.lse[(int64_t)(tok0 + tok[i]) * p.n_q + hq] =
              r.sum[i] == 0.f ? -INFINITY : (m2 + log2f(r.sum[i])) * 0.69314718055994530942f;
      } else {
        const int64_t at = ((int64_t)blockIdx.x * 2 + (u.i0 > 0 ? 0 : 1)) * C::rows + row;
#pragma unroll
        for (int d = 0; d < D / 8; d += 2)
          if ((d / NC) * NC == col)
            *reinterpret_cast<float4*>(p.part_o + at * D + d * 8 + (lane & 3) * 4) =
                make_float4(r.o[d][2 * i] * unit, r.o[d + 1][2 * i] * unit, r.o[d][2 * i + 1] * unit, r.o[d + 1][2 * i + 1] * unit);
        if (kg == 0 && (lane & 3) == 0) p.part_ml[at] = make_float2(m2, r.sum[i]);
      }
    }
  }
}

template <class T, int CODE, int D, int RG>
cudaError_t configure() {
  return cudaFuncSetAttribute(attn_qsplit_kernel<T, CODE, D, RG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              QSplitCfg<D, RG>::smem);
}

template <class T, int CODE, int D, int RG>
cudaError_t launch(const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, int grid, cudaStream_t stream) {
  using C = QSplitCfg<D, RG>;
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
  return cudaLaunchKernelEx(&cfg, attn_qsplit_kernel<T, CODE, D, RG>, p, k, v);
}

template <class T, int CODE>
cudaError_t launch_rows(const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, int rows, int grid,
                        cudaStream_t stream) {
  if (p.head_dim == 64)
    return rows == 16 ? launch<T, CODE, 64, 1>(p, k, v, grid, stream) : launch<T, CODE, 64, 2>(p, k, v, grid, stream);
  return rows == 16 ? launch<T, CODE, 128, 1>(p, k, v, grid, stream) : launch<T, CODE, 128, 2>(p, k, v, grid, stream);
}

template <class T>
cudaError_t launch_code(const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, int rows, int code, int grid,
                        cudaStream_t stream) {
  return code == COLI_ATTN_CODE_INT8 ? launch_rows<T, COLI_ATTN_CODE_INT8>(p, k, v, rows, grid, stream)
                                     : launch_rows<T, COLI_ATTN_CODE_E4M3>(p, k, v, rows, grid, stream);
}

}  // namespace

cudaError_t configure_attn_qsplit() {
  cudaError_t e = cudaSuccess;
#define COLI_CFG(T, D)                                                  \
  if (e == cudaSuccess) e = configure<T, COLI_ATTN_CODE_INT8, D, 1>();  \
  if (e == cudaSuccess) e = configure<T, COLI_ATTN_CODE_INT8, D, 2>();  \
  if (e == cudaSuccess) e = configure<T, COLI_ATTN_CODE_E4M3, D, 1>();  \
  if (e == cudaSuccess) e = configure<T, COLI_ATTN_CODE_E4M3, D, 2>();
  COLI_CFG(Bf16, 64) COLI_CFG(Bf16, 128) COLI_CFG(Fp16, 64) COLI_CFG(Fp16, 128)
#undef COLI_CFG
  return e;
}

cudaError_t launch_attn_qsplit(const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, int rows, int dtype, int code,
                               int num_sms, cudaStream_t stream) {
  const int grid = split_grid(num_sms);
  return dtype == COLI_ATTN_BF16 ? launch_code<Bf16>(p, k, v, rows, code, grid, stream)
                                 : launch_code<Fp16>(p, k, v, rows, code, grid, stream);
}

}  // namespace coli

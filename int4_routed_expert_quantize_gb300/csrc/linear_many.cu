// y = W x for more than 16 tokens, W in 4-bit codes with scales of 128 columns, on the fifth-generation tensor cores.
//
// A pass takes up to 16 tiles of the store: 128 rows, which are the lanes of tensor memory.  Two warpgroups take the blocks of 128
// columns in turn; thread = row: its 128 codes become 16-bit values (exact) in tensor memory, the A operand; x of 32 or 64 tokens
// is B.  A block's product is complete in a D of its own; the thread of the row reads it, multiplies it by the block's
// scale and adds it up in fp32, one block behind the codes that it widens.  At the end of a pass the two warpgroups' sums are added.
//
//   tensor memory (512 columns)   A of 4 blocks | D of 4 blocks, 64 columns each
//   warps 0-3, 4-7   codes to A, D to sums: even and odd blocks
//   warp 8           issues every product; warp 9 copies weights, 4 blocks of every tile a stage; warp 10 copies x, a block at a time
//
// The weights are read once for 64 tokens.  A block takes 800 to 900 cycles, in which HBM could bring two and a half, however few tokens there
// are.  Four warpgroups in place of two took as long (100000 rows, 32 tokens: 109 us for 108), and nothing is near its limit (64 tokens: tensor pipe
// 32 %, issue slots 53 %, L2 18 %, DRAM 26 %), so what is left is the chain of eight products of a block, each of which waits for the one before it.
// So 16 tokens are better off with linear.cu's kernel, and groups of 32 or 64, whose D would not all fit, at any number.  us, here / there, groups of 128:
//   8192 x 6144    16 tokens 20.1 / 12.7   24 19.5 / 23.4   64 21.5 / 47.8   128 42.2 / 95.2
//   100000 x 6144  16 tokens 109 / 79      24 107 / 156     64 118 / 313     128 235 / 626
// A start at another column for each CTA, against all asking for the same x at once, changed nothing.
#include "attn_tc.cuh"
#include "coli_linear.h"
#include "linear_store.cuh"

namespace coli {

namespace {

constexpr int kThreadsMany = 11 * 32;
constexpr int kTiles = 16;       // of a pass
constexpr int kStageBlocks = 4;  // of a stage of weights

constexpr int BLK = block_bytes(128);

template <int N>
struct ManyCfg {
  // a tile's blocks of a stage: an odd number of 16 bytes apart, so that 8 lanes that read 8 tiles meet all banks
  static constexpr int piece = kStageBlocks * BLK + 16;
  static constexpr int stages = N == 64 ? 3 : 4;
  static constexpr int stage_bytes = kTiles * piece;
  static constexpr int x_bytes = N * 256;  // of a block
  static constexpr int x_slots = 4;
  static constexpr int swap_bytes = N * 128 * 4;
  static constexpr int bars = 2 * stages + 2 * x_slots + 8 + 3;
  static constexpr int smem = x_slots * x_bytes + stages * stage_bytes + swap_bytes + bars * 8 + 16;
  static_assert(piece / 16 % 2 == 1 && smem <= 232448, "");
};

// 8 codes of a word as four pairs of neighbours.  fp16: under the exponent of 1024 a nibble in bits 0-3 is 1024 + u, one in bits 4-7 is
// 1024 + 16 u; bf16: under the exponent of 128 a nibble in bits 0-3 is 128 + u.  u - 8 is exact.
template <class T>
__device__ __forceinline__ void widen_word(uint32_t w, uint32_t* v) {
  if constexpr (T::kExp == Fp16::kExp) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t u = i ? w >> 8 : w, lo = (u & 0x000F000Fu) | 0x64006400u, hi = (u & 0x00F000F0u) | 0x64006400u;
      asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(v[2 * i]) : "r"(lo), "r"(0x64086408u));
      asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(v[2 * i + 1]) : "r"(hi), "r"(0x2C002C00u), "r"(0xD480D480u));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
      asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(v[i]) : "r"(u), "r"(0x43084308u));
    }
  }
}

template <class T, int N>
__global__ void __launch_bounds__(kThreadsMany, 1)
    linear_many_kernel(const LinearParams p, int step, const __grid_constant__ CUtensorMap xmap) {
  using C = ManyCfg<N>;
  constexpr int NS = C::stages, XS = C::x_slots;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *xs = smem, *ring = xs + XS * C::x_bytes;
  float* swap = reinterpret_cast<float*>(ring + NS * C::stage_bytes);  // [warpgroup][N / 2][row]: sums for the other one
  uint64_t* w_full = reinterpret_cast<uint64_t*>(swap + N * 128);
  uint64_t *w_empty = w_full + NS, *x_full = w_empty + NS, *x_empty = x_full + XS, *a_full = x_empty + XS, *d_full = a_full + 4,
           *given = d_full + 4, *taken = given + 1, *drain = taken + 1;
  int* abort_flag = reinterpret_cast<int*>(drain + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(abort_flag + 1);
  const int tid = threadIdx.x, warp = __shfl_sync(FULL, tid >> 5, 0), lane = tid & 31;
  const auto wait = [&](uint64_t* bar, uint32_t parity) { return ring_wait(bar, parity, abort_flag, p.status); };
  if (tid == 0) {
    *abort_flag = 0;
    for (int i = 0; i < NS; ++i) mbar_init(w_full + i, 1), mbar_init(w_empty + i, 8);
    for (int i = 0; i < XS; ++i) mbar_init(x_full + i, 1), mbar_init(x_empty + i, 1);
    for (int i = 0; i < 4; ++i) mbar_init(a_full + i, 4), mbar_init(d_full + i, 1);
    mbar_init(given, 8), mbar_init(taken, 8), mbar_init(drain, 1);
    fence_barrier_init();
    prefetch_map(&xmap);
  }
  if (warp == 8) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  const int t0 = (int)((int64_t)p.tiles * blockIdx.x / gridDim.x), t1 = (int)((int64_t)p.tiles * (blockIdx.x + 1) / gridDim.x);
  const int tok0 = blockIdx.y * N, nt = min(N, p.n_tokens - tok0);

  if (warp == 9) {  // ---- weights
    int it = 0;
    bool ok = true;
#pragma unroll 1
    for (int t = t0; t < t1 && ok; t += step) {
      const int n = min(step, t1 - t);
      const uint8_t* src = p.store + (int64_t)(t + lane) * p.blocks * BLK;
#pragma unroll 1
      for (int k = 0; k < p.blocks; k += kStageBlocks, ++it) {
        const int sg = it % NS, bytes = min(kStageBlocks, p.blocks - k) * BLK;
        if (it >= NS) ok = wait(w_empty + sg, ((it / NS) + 1) & 1);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(w_full + sg, (uint32_t)(n * bytes));
        __syncwarp();
        if (lane < n) bulk_load(ring + sg * C::stage_bytes + lane * C::piece, src + (int64_t)k * BLK, bytes, w_full + sg);
      }
    }
    drain_ring(w_full, NS, it);  // shared memory must not go while copies to it are on their way
  } else if (warp == 10) {  // ---- x
    griddep_wait();
    int it = 0;
    bool ok = true;
#pragma unroll 1
    for (int t = t0; t < t1 && ok; t += step)
#pragma unroll 1
      for (int k = 0; k < p.blocks; ++k, ++it) {
        const int sg = it % XS;
        if (it >= XS) ok = wait(x_empty + sg, ((it / XS) + 1) & 1);
        if (!ok) break;
        if (lane == 0) {
          mbar_expect_tx(x_full + sg, C::x_bytes);
          tma_load_2d(xs + sg * C::x_bytes, &xmap, k * 128, tok0, x_full + sg);
          tma_load_2d(xs + sg * C::x_bytes + N * 128, &xmap, k * 128 + 64, tok0, x_full + sg);
        }
        __syncwarp();
      }
    drain_ring(x_full, XS, it);
  } else if (warp == 8) {  // ---- products
    constexpr uint32_t idesc = mma_desc<T>(N, false);
    const uint64_t x_desc = smem_desc_sw128(xs);
    uint32_t phases = 0, x_phase = 0;  // a bit for each of the four A
    int sg = 0;
    bool ok = true;
#pragma unroll 1
    for (int t = t0; t < t1 && ok; t += step)
#pragma unroll 1
      for (int k = 0; k < p.blocks; ++k) {
        const int j = k % kStageBlocks;
        ok = wait(x_full + sg, x_phase) && wait(a_full + j, phases >> j & 1);
        if (!ok) break;
        phases ^= 1u << j;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t b = x_desc + sg * (C::x_bytes >> 4);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            tc_mma_ts(tmem + 256 + j * 64, tmem + j * 64 + i * 8, b + (((i >> 2) * N * 128 + (i & 3) * 32) >> 4), idesc, i > 0);
          tc_commit(d_full + j);
          tc_commit(x_empty + sg);
        }
        __syncwarp();
        if (++sg == XS) sg = 0, x_phase ^= 1;
      }
    if (elect_one()) tc_commit(drain);  // nor tensor memory while products write to it
    __syncwarp();
    drain_ring(drain, 1, 1);
  } else {  // ---- codes to A, D to sums
    const int wg = warp >> 2, quarter = warp & 3;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    // the thread's row: row n of tile `tile` of the pass; 8 lanes that read shared memory together take 8 tiles
    const int tile = (quarter & 1) * 8 + (lane & 7), n = (quarter >> 1) * 4 + (lane >> 3), row = quarter * 32 + lane;
    float* mine = swap + wg * (N / 2) * 128 + row;
    const float* its = swap + (wg ^ 1) * (N / 2) * 128 + row;
    int it = 0, pass = 0;
    uint32_t phases = 0;
    bool ok = true;
#pragma unroll 1
    for (int t = t0; t < t1 && ok; t += step, ++pass) {
      float acc[N];
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = 0.f;
      int behind = -1;  // the block whose D is to be added: its place, and the row's scale
      float scale = 0.f;
      const auto add = [&]() {
        if (!wait(d_full + behind, phases >> behind & 1)) return false;
        phases ^= 1u << behind;
        tc_fence_after();
        const uint32_t at = lanes + 256 + behind * 64;
#pragma unroll
        for (int i = 0; i < N; i += 16) {
          float d[16];
          tmem_ld16(at + i, d);
#pragma unroll
          for (int e = 0; e < 16; e += 2) fma2_rn(d[e], d[e + 1], scale, scale, acc[i + e], acc[i + e + 1]);
        }
        return true;
      };
#pragma unroll 1
      for (int k = 0; k < p.blocks && ok; k += kStageBlocks, ++it) {
        const int sg = it % NS, nb = min(kStageBlocks, p.blocks - k);
        ok = wait(w_full + sg, (it / NS) & 1);
        if (!ok) break;
        const uint8_t* src = ring + sg * C::stage_bytes + tile * C::piece;
        if (wg >= nb && lane == 0) mbar_arrive(w_empty + sg);
#pragma unroll 1
        for (int j = wg; j < nb; j += 2) {
          uint4 w[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) w[c] = *reinterpret_cast<const uint4*>(src + j * BLK + n * 64 + c * 16);
          const uint16_t s = *reinterpret_cast<const uint16_t*>(src + j * BLK + kBlockCodes + n * 2);
          __syncwarp();
          if (j + 2 >= nb && lane == 0) mbar_arrive(w_empty + sg);
#pragma unroll
          for (int q = 0; q < 4; ++q) {  // 32 columns in order
            uint32_t v[16];
#pragma unroll
            for (int m = 0; m < 4; ++m) widen_word<T>(m == 0 ? w[q].x : m == 1 ? w[q].y : m == 2 ? w[q].z : w[q].w, v + 4 * m);
            tmem_st16u(lanes + j * 64 + q * 16, v);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(a_full + j);
          if (behind >= 0) ok = add();
          if (!ok) break;
          behind = j, scale = T::lo(s);
        }
      }
      if (ok && behind >= 0) ok = add();
      // either warpgroup gives the other half of the tokens' sums away
      if (ok && pass > 0) ok = wait(taken, (pass - 1) & 1);
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) mine[i * 128] = wg ? acc[i] : acc[N / 2 + i];
      __syncwarp();
      if (lane == 0) mbar_arrive(given);
      ok = wait(given, pass & 1);
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) acc[i] = wg ? its[i * 128] + acc[N / 2 + i] : acc[i] + its[i * 128];
      __syncwarp();
      if (lane == 0) mbar_arrive(taken);
      griddep_wait();  // (the launch before this one may still read or write y)
      const int at = (t + tile) * 8 + n, first = wg * (N / 2);
      if (tile < min(step, t1 - t) && at < p.rows) {
        uint16_t* dst = p.y + (int64_t)(tok0 + first) * p.y_stride + at;
#pragma unroll
        for (int i = 0; i < N / 2; i += 2) {
          const uint32_t v = T::pack(acc[i], acc[i + 1]);
          if (first + i < nt) dst[i * p.y_stride] = (uint16_t)v;
          if (first + i + 1 < nt) dst[(i + 1) * p.y_stride] = (uint16_t)(v >> 16);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

template <class T, int N>
cudaError_t launch(const LinearParams& p, int num_sms, cudaStream_t stream) {
  CUtensorMap map;
  if (!rows_map(&map, p.x, T::kExp == Bf16::kExp ? COLI_ATTN_BF16 : COLI_ATTN_FP16, p.cols, p.n_tokens, p.x_stride, N))
    return cudaErrorUnknown;
  cudaLaunchConfig_t cfg = {};
  const int grid = num_sms < p.tiles ? num_sms : p.tiles, most = (p.tiles + grid - 1) / grid;
  const int passes = (most + kTiles - 1) / kTiles;
  cfg.gridDim = dim3(grid, (p.n_tokens + N - 1) / N);
  cfg.blockDim = dim3(kThreadsMany);
  cfg.dynamicSmemBytes = ManyCfg<N>::smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, linear_many_kernel<T, N>, p, (most + passes - 1) / passes, map);
}

template <class T, int N>
cudaError_t configure() {
  return cudaFuncSetAttribute(linear_many_kernel<T, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, ManyCfg<N>::smem);
}

}  // namespace

cudaError_t configure_linear_many() {
  cudaError_t e = configure<Bf16, 32>();
  if (e == cudaSuccess) e = configure<Bf16, 64>();
  if (e == cudaSuccess) e = configure<Fp16, 32>();
  if (e == cudaSuccess) e = configure<Fp16, 64>();
  return e;
}

cudaError_t launch_linear_many(const LinearParams& p, int dtype, int num_sms, cudaStream_t stream) {
  if (dtype == COLI_ATTN_BF16) return p.n_tokens <= 32 ? launch<Bf16, 32>(p, num_sms, stream) : launch<Bf16, 64>(p, num_sms, stream);
  return p.n_tokens <= 32 ? launch<Fp16, 32>(p, num_sms, stream) : launch<Fp16, 64>(p, num_sms, stream);
}

}  // namespace coli

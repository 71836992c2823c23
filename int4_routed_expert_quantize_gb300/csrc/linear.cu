// y = W x for few tokens, W in 4-bit codes with a scale for each row and group of columns:
//   y[t,n] = sum_g s[n,g] sum_{k in g} c[n,k] x[t,k]
//
// At up to 16 tokens every weight byte is used by few products, so HBM bounds it and the kernel is built around one stream
// of weights: a persistent CTA an SM, in which one lane keeps a ring of some 180 KB full with bulk copies.  The weights are the
// handle's, written by load alone, so the first copies start before the launch that makes x has ended.
//
// The store.  8 rows x 128 columns are a block: 32 lanes x 16 bytes of codes (+ 8, so that they are unsigned), then the 8 rows'
// scales of each group.  A tile of 8 rows is its blocks one after another, so a ring stage is one copy, and a lane's
// 16 bytes are what it feeds to the matrix instructions.  Lane (n = lane / 4, c = lane % 4) holds 4 words of 8 columns of row n, all of one
// group for all c: groups of 128 take columns 32 c + 8 j (word j), of 64 columns 64 (j / 2) + 16 c + 8 (j % 2), of 32 columns 32 j + 8 c.
// Nibble i of a word is column 2 i (i < 4) or 2 i - 7, so that (w >> 4 i) & 0x000F000F is a pair of neighbours.
//
// A warp has nb of a tile's blocks, the same ones of every tile: their share of x stays in its registers, as the A operand of
// mma.sync (16 tokens, or 8 and zeros), and the weights are B: 8 rows a step, so tiles are narrow and the SMs
// end together.  A code becomes bf16 or fp16 exactly, by its bits under the exponent of 128 or 1024; a group's sum is fp32 and
// its scale multiplies it in fp32.  The warps' sums of a tile meet in shared memory, where a warp of its own adds them in order.
// Columns beyond what the registers of one CTA hold (48 blocks at 8 tokens, 32 at 16) are split over a cluster, whose CTAs send
// their sums to the first one.
#include <algorithm>
#include <new>

#include "attn_device.cuh"
#include "bulk.cuh"
#include "coli_linear.h"

using namespace coli;

struct coli_linear {
  coli_linear_config cfg{};
  int device = 0, num_sms = 0, tiles = 0, blocks = 0;  // of 8 rows; of 128 columns
  bool loaded = false;
  uint8_t* store = nullptr;
  int32_t* status = nullptr;
};

namespace {

constexpr int kProduct = 16;                // product warps
constexpr int kThreads = (kProduct + 2) * 32;  // and one that copies, one that adds
constexpr int kRing = 184320;               // bytes of the ring, at most
constexpr int kMaxStages = 16;
constexpr int kSums = 4;                    // buffers of the warps' sums
constexpr int kMaxParts = 8;                // CTAs of a cluster
constexpr int kBlockCodes = 512;

__host__ __device__ constexpr int block_bytes(int group) { return kBlockCodes + 16 * (128 / group); }

__host__ __device__ constexpr int max_blocks(int mt) { return mt == 1 ? 3 : 2; }  // of a warp

struct LinearParams {
  const uint8_t* store;
  const uint16_t* x;
  uint16_t* y;
  int64_t x_stride, y_stride;
  int n_tokens, rows, cols;
  int tiles, blocks;   // of the whole matrix
  int part;            // blocks of a CTA of the cluster (the last one may have fewer)
  int nb, kw, rw;      // blocks a warp, warps a tile, tiles a stage
  int stages;
  int* status;
};

// column of a lane's word j within a block
template <int G>
__device__ __forceinline__ int word_col(int c, int j) {
  return G == 128 ? 32 * c + 8 * j : G == 64 ? 64 * (j >> 1) + 16 * c + 8 * (j & 1) : 32 * j + 8 * c;
}

// 8 codes of a word as four pairs of neighbours
template <class T>
__device__ __forceinline__ void unpack(uint32_t w, uint32_t (&v)[4]);
template <>
__device__ __forceinline__ void unpack<Bf16>(uint32_t w, uint32_t (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(v[i]) : "r"(u), "r"(0x43084308u));  // 136
  }
}
template <>
__device__ __forceinline__ void unpack<Fp16>(uint32_t w, uint32_t (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = ((w >> (4 * i)) & 0x000F000Fu) | 0x64006400u;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(v[i]) : "r"(u), "r"(0x64086408u));  // 1032
  }
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// the address of this CTA's shared memory at `p` in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t peer(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void peer_store(uint32_t addr, float2 v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(v.x), "f"(v.y) : "memory");
}
__device__ __forceinline__ void peer_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// a bounded wait for what another CTA's peer_arrive releases
__device__ __forceinline__ bool peer_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  const uint64_t t0 = global_ns();
  bool ok = false;
#pragma unroll 1
  for (uint32_t it = 1; !*abort_flag; ++it) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    if (r) {
      ok = true;
      break;
    }
    if ((it & 63u) == 0 && global_ns() - t0 > kWaitLimitNs) {
      *abort_flag = 1;
      atomicExch(status, COLI_ETIMEOUT);
    }
  }
  return __all_sync(FULL, ok);
}

// MT: 1 for up to 8 tokens, 2 for up to 16.  A warp's blocks: at most 3 or 2, 48 or 64 registers of x (18 warps leave 96).
template <class T, int G, int MT>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const LinearParams p) {
  constexpr int NB = max_blocks(MT), BLK = block_bytes(G), GPB = 128 / G, OUT = MT * 64;  // OUT: sums of a tile
  extern __shared__ __align__(128) uint8_t smem[];
  const int parts = (p.blocks + p.part - 1) / p.part;  // the cluster's size
  const int stage_bytes = p.rw * p.part * BLK, warps = p.kw * p.rw;
  float* sums = reinterpret_cast<float*>(smem + (size_t)p.stages * stage_bytes);  // [kSums][warps][OUT]
  float* inbox = sums + kSums * warps * OUT;                                       // [kSums][parts - 1][rw][OUT]
  uint64_t* full = reinterpret_cast<uint64_t*>(inbox + kSums * (parts - 1) * p.rw * OUT);
  uint64_t *empty = full + kMaxStages, *sum_full = empty + kMaxStages, *sum_empty = sum_full + kSums,
           *in_full = sum_empty + kSums, *in_empty = in_full + kSums;
  int* abort_flag = reinterpret_cast<int*>(in_empty + kSums);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const auto wait = [&](uint64_t* bar, uint32_t parity) { return warp_wait(bar, parity, abort_flag, p.status); };

  if (tid == 0) {
    *abort_flag = 0;
    for (int i = 0; i < p.stages; ++i) mbar_init(full + i, 1), mbar_init(empty + i, warps);
    for (int i = 0; i < kSums; ++i) {
      mbar_init(sum_full + i, warps), mbar_init(sum_empty + i, 1);
      mbar_init(in_full + i, parts > 1 ? parts - 1 : 1), mbar_init(in_empty + i, 1);
    }
    fence_barrier_init();
  }
  const int rank = parts > 1 ? (int)cluster_rank() : 0;
  __syncwarp();
  if (parts > 1) cluster_sync();
  else __syncthreads();
  griddep_launch_dependents();

  const int cluster = blockIdx.x / parts, clusters = gridDim.x / parts;
  const int groups = (p.tiles + p.rw - 1) / p.rw;  // stages' worth of tiles
  const int g0 = (int)((int64_t)groups * cluster / clusters), g1 = (int)((int64_t)groups * (cluster + 1) / clusters);
  const int here = min(p.part, p.blocks - rank * p.part);  // blocks of this CTA
  const int tok0 = blockIdx.y * 8 * MT, nt = min(8 * MT, p.n_tokens - tok0);

  if (warp == kProduct) {  // ---- copies
    int it = 0;
    bool ok = true;
#pragma unroll 1
    for (int g = g0; g < g1; ++g, ++it) {
      const int s = it % p.stages, n = min(p.rw, p.tiles - g * p.rw);
      if (it >= p.stages) ok = wait(empty + s, (it / p.stages + 1) & 1);
      if (!ok) break;
      if (lane == 0) {
        mbar_expect_tx(full + s, (uint32_t)(n * here * BLK));
        for (int r = 0; r < n; ++r)
          bulk_load(smem + (size_t)s * stage_bytes + r * p.part * BLK,
                    p.store + ((int64_t)(g * p.rw + r) * p.blocks + rank * p.part) * BLK, here * BLK, full + s);
      }
      __syncwarp();
    }
    drain_ring(full, p.stages, it);  // shared memory must not go while copies are on their way
  } else if (warp == kProduct + 1) {  // ---- sums
    griddep_wait();  // (the launch before this one may still read or write y)
    int it = 0;
    bool ok = true;
#pragma unroll 1
    for (int g = g0; g < g1 && ok; ++g, ++it) {
      const int buf = it % kSums, n = min(p.rw, p.tiles - g * p.rw);
      const uint32_t phase = (it / kSums) & 1;
      ok = wait(sum_full + buf, phase);
      if (ok && rank == 0 && parts > 1) ok = peer_wait(in_full + buf, phase, abort_flag, p.status);
      if (ok && rank > 0 && it >= kSums) ok = peer_wait(in_empty + buf, phase ^ 1, abort_flag, p.status);
      if (!ok) break;
#pragma unroll 1
      for (int r = 0; r < n; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const float* src = sums + (size_t)(buf * warps + r * p.kw) * OUT + m * 64 + lane * 2;
          float2 v = make_float2(0.f, 0.f);
#pragma unroll 4
          for (int k = 0; k < p.kw; ++k) {
            const float2 u = *reinterpret_cast<const float2*>(src + k * OUT);
            v.x += u.x, v.y += u.y;
          }
          if (rank > 0) {
            peer_store(peer(inbox, 0) + (uint32_t)(((buf * (parts - 1) + rank - 1) * p.rw + r) * OUT + m * 64 + lane * 2) * 4, v);
            continue;
          }
#pragma unroll 1
          for (int q = 0; q + 1 < parts; ++q) {
            const float2 u = *reinterpret_cast<const float2*>(inbox + ((buf * (parts - 1) + q) * p.rw + r) * OUT + m * 64 + lane * 2);
            v.x += u.x, v.y += u.y;
          }
          const int t = m * 8 + (lane >> 2), row = (g * p.rw + r) * 8 + (lane & 3) * 2;
          if (t < nt) {
            uint16_t* dst = p.y + (tok0 + t) * p.y_stride + row;
            const uint32_t w = T::pack(v.x, v.y);
            if (row < p.rows) dst[0] = (uint16_t)w;
            if (row + 1 < p.rows) dst[1] = (uint16_t)(w >> 16);
          }
        }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(sum_empty + buf);
        if (rank > 0) peer_arrive(peer(in_full + buf, 0));
        else
          for (int q = 1; q < parts; ++q) peer_arrive(peer(in_empty + buf, q));
      }
      __syncwarp();
    }
  } else if (warp < warps) {  // ---- products
    const int first = (warp % p.kw) * p.nb, tile = warp / p.kw;  // the warp's blocks of the part; its tile of a stage
    const int nb = max(0, min(p.nb, here - first));
    griddep_wait();
    uint32_t x[NB][8][2 * MT];  // A fragments: step 2j + h is columns 4h..4h+3 of word j
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int t = m * 8 + (lane >> 2), col = (rank * p.part + first + b) * 128 + word_col<G>(lane & 3, j);
          uint4 v = make_uint4(0, 0, 0, 0);
          if (b < nb && t < nt && col < p.cols)
            v = __ldg(reinterpret_cast<const uint4*>(p.x + (tok0 + t) * p.x_stride + col));
          x[b][2 * j][m] = v.x, x[b][2 * j][MT + m] = v.y;
          x[b][2 * j + 1][m] = v.z, x[b][2 * j + 1][MT + m] = v.w;
        }
    const uint8_t* base = smem + (size_t)(tile * p.part + first) * BLK;
    int it = 0;
#pragma unroll 1
    for (int g = g0; g < g1; ++g, ++it) {
      const int s = it % p.stages, buf = it % kSums;
      if (!wait(full + s, (it / p.stages) & 1)) break;
      float tot[4] = {0.f, 0.f, 0.f, 0.f};
      if (g * p.rw + tile < p.tiles) {
        const uint8_t* at = base + (size_t)s * stage_bytes;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if (b < nb) {
            const uint4 w4 = *reinterpret_cast<const uint4*>(at + b * BLK + lane * 16);
            const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
            float acc[GPB][4];
#pragma unroll
            for (int q = 0; q < GPB; ++q)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[q][i] = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t v[4];
              unpack<T>(w[j], v);
              float(&a)[4] = acc[j * GPB / 4];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t(&xs)[2 * MT] = x[b][2 * j + h];
                const uint32_t f[4] = {xs[0], MT == 2 ? xs[1] : 0u, xs[MT], MT == 2 ? xs[MT + 1] : 0u};
                mma16816<T>(a, f, v[2 * h], v[2 * h + 1]);
              }
            }
#pragma unroll
            for (int q = 0; q < GPB; ++q) {
              const uint32_t sc = *reinterpret_cast<const uint32_t*>(at + b * BLK + kBlockCodes + q * 16 + (lane & 3) * 4);
              const float s0 = T::lo(sc), s1 = T::hi(sc);
              tot[0] = fmaf(acc[q][0], s0, tot[0]), tot[1] = fmaf(acc[q][1], s1, tot[1]);
              if (MT == 2) tot[2] = fmaf(acc[q][2], s0, tot[2]), tot[3] = fmaf(acc[q][3], s1, tot[3]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + s);
      if (it >= kSums && !wait(sum_empty + buf, (it / kSums + 1) & 1)) break;
      float* dst = sums + (size_t)(buf * warps + warp) * OUT + lane * 2;
      *reinterpret_cast<float2*>(dst) = make_float2(tot[0], tot[1]);
      if (MT == 2) *reinterpret_cast<float2*>(dst + 64) = make_float2(tot[2], tot[3]);
      __syncwarp();
      if (lane == 0) mbar_arrive(sum_full + buf);
    }
  }
  __syncwarp();
  if (parts > 1) cluster_sync();  // a CTA's shared memory stays until the others are done with it
}

// one 16-byte unit of the store, or the scales of a block, a thread; the grid covers tiles * blocks * 33 units
template <int G>
__global__ void repack_kernel(const uint8_t* packed, const uint16_t* scales, uint8_t* store, int rows, int cols, int tiles,
                              int blocks) {
  constexpr int GPB = 128 / G;
  const int64_t at = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, block = at / 33;
  const int unit = (int)(at - block * 33);
  if (block >= (int64_t)tiles * blocks) return;
  const int64_t tile = block / blocks;
  const int kb = (int)(block - tile * blocks);
  uint8_t* dst = store + block * block_bytes(G);
  if (unit < 32) {
    const int64_t row = tile * 8 + (unit >> 2);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = kb * 128 + word_col<G>(unit & 3, j);
      const uint32_t v =
          (row < rows && col < cols ? *reinterpret_cast<const uint32_t*>(packed + (row * cols + col) / 2) : 0u) ^ 0x88888888u;
      w[j] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[j] |= ((v >> (8 * i)) & 15u) << (4 * i) | ((v >> (8 * i + 4)) & 15u) << (4 * i + 16);
    }
    *reinterpret_cast<uint4*>(dst + unit * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    for (int i = 0; i < GPB * 8; ++i) {
      const int64_t row = tile * 8 + (i & 7);
      const int g = kb * GPB + (i >> 3);
      reinterpret_cast<uint16_t*>(dst + kBlockCodes)[i] = row < rows && g * G < cols ? scales[row * (cols / G) + g] : 0;
    }
  }
}

// a warp a group
template <class T>
__global__ void quantize_kernel(const float* w, int64_t groups, int group, uint8_t* packed, uint16_t* scales) {
  const int64_t g = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (g >= groups) return;
  const float* src = w + g * group;
  float m = 0.f;
  for (int i = lane; i < group; i += 32) m = fmaxf(m, fabsf(src[i]));
  const uint32_t s = T::pack(__fdiv_rn(warp_max(m), 7.f), 0.f) & 0xFFFFu;
  const float d = T::lo(s);
  if (lane == 0) scales[g] = (uint16_t)s;
  for (int i = lane; i < group / 2; i += 32) {
    uint32_t b = 0;
    for (int k = 0; k < 2; ++k) {
      const int q = d == 0.f ? 0 : max(-7, min(7, (int)roundf(__fdiv_rn(src[2 * i + k], d))));
      b |= ((uint32_t)q & 15u) << (4 * k);
    }
    packed[g * (group / 2) + i] = (uint8_t)b;
  }
}

int check_device(int device) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return COLI_ECUDA;
  return dev == device ? COLI_OK : COLI_ESTATE;
}

size_t smem_bytes(const LinearParams& p, int group, int mt, int parts) {
  return (size_t)p.stages * p.rw * p.part * block_bytes(group) +
         (size_t)kSums * (p.kw * p.rw + (parts - 1) * p.rw) * mt * 64 * 4 + (2 * kMaxStages + 4 * kSums) * 8 + 16;
}

template <class T, int G, int MT>
cudaError_t launch(LinearParams p, int num_sms, cudaStream_t stream) {
  constexpr int NB = max_blocks(MT);
  // the cluster: as few CTAs as hold x in registers; the warps: as few blocks each as that takes
  int parts = (p.blocks + kProduct * NB - 1) / (kProduct * NB);
  p.part = (p.blocks + parts - 1) / parts;
  parts = (p.blocks + p.part - 1) / p.part;
  p.nb = (p.part + kProduct - 1) / kProduct;
  p.kw = (p.part + p.nb - 1) / p.nb;
  // narrow matrices: several tiles at a time, while every cluster still gets some
  const int clusters = num_sms / parts;
  p.rw = std::max(1, std::min(kProduct / p.kw, (p.tiles + clusters - 1) / clusters));
  p.stages = std::min(kMaxStages, kRing / (p.rw * p.part * block_bytes(G)));
  const int groups = (p.tiles + p.rw - 1) / p.rw;
  const size_t smem = smem_bytes(p, G, MT, parts);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(std::min(clusters, groups) * parts, (p.n_tokens + 8 * MT - 1) / (8 * MT));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = parts, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = parts > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, linear_kernel<T, G, MT>, p);
}

static_assert(kProduct * 3 * block_bytes(32) * 6 <= kRing, "at least six stages");

template <class T, int G, int MT>
cudaError_t configure() {
  // the device's limit; a launch's own need is below it: the ring, sums of 16 warps (16 or 32 KB) and of 7 other CTAs (7 or 14 KB)
  return cudaFuncSetAttribute(linear_kernel<T, G, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
}

template <class T, int G>
cudaError_t launch_tokens(const LinearParams& p, int num_sms, cudaStream_t stream) {
  return p.n_tokens <= 8 ? launch<T, G, 1>(p, num_sms, stream) : launch<T, G, 2>(p, num_sms, stream);
}
template <class T>
cudaError_t launch_group(const LinearParams& p, int group, int num_sms, cudaStream_t stream) {
  return group == 128  ? launch_tokens<T, 128>(p, num_sms, stream)
         : group == 64 ? launch_tokens<T, 64>(p, num_sms, stream)
                       : launch_tokens<T, 32>(p, num_sms, stream);
}

cudaError_t configure_device() {
  cudaError_t e = cudaSuccess;
#define COLI_CFG(T, G)                                 \
  if (e == cudaSuccess) e = configure<T, G, 1>();      \
  if (e == cudaSuccess) e = configure<T, G, 2>();
  COLI_CFG(Bf16, 32) COLI_CFG(Bf16, 64) COLI_CFG(Bf16, 128) COLI_CFG(Fp16, 32) COLI_CFG(Fp16, 64) COLI_CFG(Fp16, 128)
#undef COLI_CFG
  return e;
}

// Whether rows of `wa` values every `sa` from a and of `wb` every `sb` from b (n of either) share memory; rows of the same
// stride may lie between one another.
bool collide(const void* a, int64_t sa, int64_t wa, const void* b, int64_t sb, int64_t wb, int64_t n) {
  const int64_t x = (int64_t)((uintptr_t)a / 2), y = (int64_t)((uintptr_t)b / 2);
  if (x + (n - 1) * sa + wa <= y || y + (n - 1) * sb + wb <= x) return false;
  if (sa != sb || n == 1) return true;
  const int64_t gap = (((y - x) % sa) + sa) % sa;  // b's row starts so far behind one of a's
  return gap < wa || gap + wb > sa;
}

}  // namespace

extern "C" int coli_linear_create(const coli_linear_config* cfg, coli_linear** out) {
  if (out) *out = nullptr;
  if (!cfg || !out) return COLI_EINVAL;
  const coli_linear_config& c = *cfg;
  if (c.rows < 1 || c.rows > 16777216 || c.cols < 1 || c.group < 1 || c.cols % c.group || c.max_tokens < 1 ||
      c.max_tokens > 1000000)
    return COLI_EINVAL;
  if ((c.group != 32 && c.group != 64 && c.group != 128) || (c.dtype != COLI_ATTN_BF16 && c.dtype != COLI_ATTN_FP16) ||
      c.cols > kMaxParts * kProduct * 2 * 128)
    return COLI_EUNSUPPORTED;
  coli_linear* h = new (std::nothrow) coli_linear();
  if (!h) return COLI_ENOMEM;
  h->cfg = c;
  h->tiles = (c.rows + 7) / 8, h->blocks = (c.cols + 127) / 128;
  int rc = COLI_OK;
  if (cudaGetDevice(&h->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess ||
      configure_device() != cudaSuccess)
    rc = COLI_ECUDA;
  if (!rc) {
    const size_t size = (size_t)h->tiles * h->blocks * block_bytes(c.group);  // a multiple of 16
    void* p = nullptr;
    if (cudaMalloc(&p, size + 16) != cudaSuccess) {
      rc = COLI_ENOMEM;
    } else {
      h->store = static_cast<uint8_t*>(p);
      h->status = reinterpret_cast<int32_t*>(h->store + size);
      if (cudaMemset(h->status, 0, 16) != cudaSuccess || cudaStreamSynchronize(cudaStreamLegacy) != cudaSuccess) rc = COLI_ECUDA;
    }
  }
  if (rc) {
    cudaGetLastError();
    if (h->store) cudaFree(h->store);
    delete h;
    return rc;
  }
  *out = h;
  return COLI_OK;
}

extern "C" void coli_linear_destroy(coli_linear* h) {
  if (!h) return;
  cudaDeviceSynchronize();
  cudaFree(h->store);
  delete h;
}

extern "C" int coli_linear_load(coli_linear* h, const uint8_t* packed, const void* scales, void* stream) {
  if (!h || !packed || !scales || ((uintptr_t)packed & 3u) || ((uintptr_t)scales & 1u)) return COLI_EINVAL;
  const int rc = check_device(h->device);
  if (rc) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  const int64_t units = (int64_t)h->tiles * h->blocks * 33;
  const int threads = 256;
  const auto kernel = h->cfg.group == 128 ? repack_kernel<128> : h->cfg.group == 64 ? repack_kernel<64> : repack_kernel<32>;
  kernel<<<(unsigned)((units + threads - 1) / threads), threads, 0, st>>>(
      packed, static_cast<const uint16_t*>(scales), h->store, h->cfg.rows, h->cfg.cols, h->tiles, h->blocks);
  if (cudaGetLastError() != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess) return COLI_ECUDA;
  h->loaded = true;
  return COLI_OK;
}

extern "C" int coli_linear_forward(const coli_linear* h, const void* x, int64_t x_stride, int n_tokens, void* y, int64_t y_stride,
                                   void* stream) {
  if (!h || n_tokens < 0 || n_tokens > h->cfg.max_tokens) return COLI_EINVAL;
  if (!h->loaded) return COLI_ESTATE;
  if (n_tokens == 0) return COLI_OK;
  const coli_linear_config& c = h->cfg;
  if (!x || !y || ((uintptr_t)x & 15u) || (x_stride & 7) || ((uintptr_t)y & 1u) || x_stride < c.cols || y_stride < c.rows ||
      x_stride >= (1LL << 38) || y_stride >= (1LL << 38) || collide(x, x_stride, c.cols, y, y_stride, c.rows, n_tokens))
    return COLI_EINVAL;
  const int rc = check_device(h->device);
  if (rc) return rc;
  LinearParams p = {};
  p.store = h->store, p.x = static_cast<const uint16_t*>(x), p.y = static_cast<uint16_t*>(y);
  p.x_stride = x_stride, p.y_stride = y_stride;
  p.n_tokens = n_tokens, p.rows = c.rows, p.cols = c.cols, p.tiles = h->tiles, p.blocks = h->blocks;
  p.status = h->status;
  const cudaError_t e = c.dtype == COLI_ATTN_BF16 ? launch_group<Bf16>(p, c.group, h->num_sms, (cudaStream_t)stream)
                                                  : launch_group<Fp16>(p, c.group, h->num_sms, (cudaStream_t)stream);
  return e == cudaSuccess ? COLI_OK : COLI_ECUDA;
}

extern "C" int coli_linear_status(coli_linear* h, void* stream) {
  if (!h) return COLI_EINVAL;
  const int rc = check_device(h->device);
  if (rc) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  int32_t v = 0;
  if (cudaMemcpyAsync(&v, h->status, sizeof(v), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaMemsetAsync(h->status, 0, sizeof(v), st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess)
    return COLI_ECUDA;
  return v;
}

extern "C" int coli_linear_quantize(const float* w, int64_t rows, int cols, int group, int dtype, uint8_t* packed, void* scales,
                                    void* stream) {
  if (!w || !packed || !scales || rows < 0 || rows > 16777216 || cols < 1 || group < 1 || cols % group || cols > 1048576 ||
      ((uintptr_t)w & 3u) || ((uintptr_t)scales & 1u))
    return COLI_EINVAL;
  if ((group != 32 && group != 64 && group != 128) || (dtype != COLI_ATTN_BF16 && dtype != COLI_ATTN_FP16))
    return COLI_EUNSUPPORTED;
  const int64_t groups = rows * (cols / group);
  if (groups == 0) return COLI_OK;
  const int64_t ctas = (groups + 7) / 8;
  if (ctas > 0x7FFFFFFF) return COLI_EUNSUPPORTED;
  const auto kernel = dtype == COLI_ATTN_BF16 ? quantize_kernel<Bf16> : quantize_kernel<Fp16>;
  kernel<<<(unsigned)ctas, 256, 0, (cudaStream_t)stream>>>(w, groups, group, packed, static_cast<uint16_t*>(scales));
  return cudaGetLastError() == cudaSuccess ? COLI_OK : COLI_ECUDA;
}

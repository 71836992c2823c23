// y = W x for few tokens (more than 16 with groups of 128: linear_many.cu), W in 4-bit codes with a scale for each row and group of columns:
//   y[t,n] = sum_g s[n,g] sum_{k in g} c[n,k] x[t,k]
//
// At up to 16 tokens every weight byte is used by few products, so HBM bounds it, and next to it the instructions that make 16-bit
// values of 4-bit codes: a word of 8 takes 5 on the ALU and 4 on the fp16 pipe (to bf16 7 and 4), and mma.sync gets in their way (fp16:
// together 73 cycles a block and SM partition, where HBM takes 98).  So the 12 product warps of an SM stay clear of one another: each keeps a ring of its own in shared
// memory full with bulk copies and waits for nobody else, x stays in its registers, and the sums that it shares with others go to
// warps that do nothing but add.  The weights are the handle's, written by load alone, so the first copies start before the launch that
// makes x has ended.
//
// A warp has NB blocks of every tile that it takes, the same ones each time, 2 or 4 tiles a step: two tiles' weights are the A operand of
// mma.sync, x of 8 or 2 x 8 tokens is B.  A CTA has a range of tiles, so the CTAs end together to within 8 rows.  Columns beyond what
// the registers of one CTA hold (48 blocks at 8 tokens, 24 at 16) are split over a cluster, whose CTAs send their sums to the first one.
//
// Measured, groups of 128, bf16: 8192 x 6144 for one token 8.0 us, of which 3.3 are launch and prologue; from 20000 to 40000 rows 11.8 us
// more, 5.4 TB/s (fp16 10.6, 6.0 TB/s; a copy reaches 6.79).  100000 x 6144 for 16 tokens 78.6 us (fp16 73), 4.1 TB/s: there the
// instructions bound it.
//
// A code becomes a value of x's type exactly, so products are exact whatever the sizes of x; a group's sum is fp32, and its scale
// multiplies it in fp32.  (bf16 x as fp16 times a power of two for each token and warp, which saves two shifts a word, lost what was 2^39 below the
// largest value: back to back, 100000 rows 55.8 us for one token instead of 60.4, 78.1 for 16
// instead of 79.0, 8192 rows 8.7 and 13.1 instead of 8.4 and 12.7.)
#include <algorithm>
#include <new>

#include "coli_linear.h"
#include "linear_store.cuh"

using namespace coli;

namespace {

struct Room {
  int num_sms = 0;
  int clusters[2] = {};  // that run at once, of calls of up to 8 and up to 16 tokens; 0: not asked yet
};

}  // namespace

struct coli_linear {
  coli_linear_config cfg{};
  int device = 0, tiles = 0, blocks = 0;  // of 8 rows; of 128 columns
  Room room;
  bool loaded = false;
  uint8_t* store = nullptr;
  int32_t* status = nullptr;
};

namespace {

constexpr int kProduct = 12;  // product warps
constexpr int kAdd = 4;       // warps that add their sums: 16 in all, of up to 128 registers
constexpr int kThreads = (kProduct + kAdd) * 32;
constexpr int kSmem = 232448;  // of a CTA
constexpr int kMaxSlots = 8;  // of a warp's ring
constexpr int kRing = 106496;  // bytes of all rings that are enough
constexpr int kIn = 4;        // buffers of the other CTAs' sums
constexpr int kMaxParts = 8;  // CTAs of a cluster
constexpr int kLaunchTokens = 8 * 65535;  // of one launch: a grid's y goes up to 65535, at 8 tokens or more each

__host__ __device__ constexpr int step_tiles(int mt) { return 2 * mt; }    // of a warp
__host__ __device__ constexpr int sum_buffers(int mt) { return mt == 1 ? 4 : 2; }

// Masks and exponents, in registers of their own (as immediates, one of two would be moved to a register each time).
template <class T>
struct Bits {
  uint32_t lo, hi, exp;
  __device__ __forceinline__ Bits() {
    asm volatile("mov.b32 %0, 0x000F000F;" : "=r"(lo));
    asm volatile("mov.b32 %0, 0x00F000F0;" : "=r"(hi));
    if constexpr (T::kExp == Fp16::kExp) asm volatile("mov.b32 %0, 0x64006400;" : "=r"(exp));
    else asm volatile("mov.b32 %0, 0x43004300;" : "=r"(exp));
  }
};
// 8 codes of a word as four pairs of neighbours, exactly.  fp16: under the exponent of 1024 a nibble in bits 0-3 is 1024 + u, one in
// bits 4-7 is 1024 + 16 u, so a word takes one shift; bf16 has 7 bits under the exponent of 128, so a word takes three.
template <class T>
__device__ __forceinline__ void unpack(const Bits<T>& k, uint32_t w, uint32_t (&v)[4]) {
  if constexpr (T::kExp == Fp16::kExp) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t u = i ? w >> 8 : w;
      uint32_t lo, hi;
      asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(lo) : "r"(u), "r"(k.lo), "r"(k.exp));  // u & mask | exp
      asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(hi) : "r"(u), "r"(k.hi), "r"(k.exp));
      asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(v[2 * i]) : "r"(lo), "r"(0x64086408u));                          // 1032
      asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(v[2 * i + 1]) : "r"(hi), "r"(0x2C002C00u), "r"(0xD480D480u));  // / 16 - 72
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t u;
      asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(u) : "r"(w >> (4 * i)), "r"(k.lo), "r"(k.exp));
      asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(v[i]) : "r"(u), "r"(0x43084308u));  // 136
    }
  }
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ uint16_t lds16(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void sts64(uint32_t at, float a, float b) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(a), "f"(b) : "memory");
}

// bounded waits for copies number done .. ahead - 1 of a ring
__device__ __noinline__ void drain_slots(uint64_t* bars, int slots, int done, int ahead) {
  for (int i = done; i < ahead; ++i) {
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait(bars + i % slots, (uint32_t)((i / slots) & 1)))
      if (global_ns() - t0 > kWaitLimitNs / 8) break;
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
// 8 bytes there, which its barrier counts when they have come
__device__ __forceinline__ void peer_store(uint32_t addr, float2 v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(addr), "f"(v.x),
               "f"(v.y), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void peer_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// MT: 1 for up to 8 tokens, 2 for up to 16.  NB: a warp's blocks, at most 4 or 2: 64 registers of x.
template <class T, int G, int MT, int NB>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const LinearParams p) {
  constexpr int BLK = block_bytes(G), GPB = 128 / G, OUT = MT * 64, TP = step_tiles(MT), SUMS = sum_buffers(MT);
  constexpr int slot_bytes = TP * NB * BLK;  // OUT: sums of a tile
  extern __shared__ __align__(128) uint8_t smem[];
  const int parts = (p.blocks + p.part - 1) / p.part;  // the cluster's size
  const int warps = p.kw * p.rw, step = p.rw * TP;
  const int sum_floats = step * p.kw * OUT, in_floats = step * OUT;
  // rings [warps][slots], sums [SUMS][step][kw][OUT], the other CTAs' [kIn][parts - 1][step][OUT], barriers
  float* sums = reinterpret_cast<float*>(smem + warps * p.slots * slot_bytes);
  float* inbox = sums + SUMS * sum_floats;
  uint64_t* full = reinterpret_cast<uint64_t*>(inbox + kIn * (parts - 1) * in_floats);
  uint64_t *sum_full = full + kProduct * kMaxSlots, *sum_empty = sum_full + SUMS, *in_full = sum_empty + SUMS,
           *in_empty = in_full + kIn;
  int* abort_flag = reinterpret_cast<int*>(in_empty + kIn);
  const int tid = threadIdx.x, warp = __shfl_sync(FULL, tid >> 5, 0), lane = tid & 31;
  const auto wait = [&](uint64_t* bar, uint32_t parity) { return ring_wait(bar, parity, abort_flag, p.status); };

  if (tid == 0) {
    *abort_flag = 0;
    for (int i = 0; i < SUMS; ++i) mbar_init(sum_full + i, warps), mbar_init(sum_empty + i, kAdd);
    for (int i = 0; i < kIn; ++i) mbar_init(in_full + i, 1), mbar_init(in_empty + i, kAdd);
  }
  if (warp < kProduct && lane < kMaxSlots) mbar_init(full + warp * kMaxSlots + lane, 1);
  fence_barrier_init();
  griddep_launch_dependents();
  const int rank = parts > 1 ? (int)cluster_rank() : 0;
  const int cluster = blockIdx.x / parts, clusters = gridDim.x / parts;
  const int t0 = (int)((int64_t)p.tiles * cluster / clusters), t1 = (int)((int64_t)p.tiles * (cluster + 1) / clusters);
  const int here = min(p.part, p.blocks - rank * p.part);  // blocks of this CTA
  const int tok0 = blockIdx.y * 8 * MT, nt = min(8 * MT, p.n_tokens - tok0);

  if (warp < warps) {  // ---- products
    const int sub = warp / p.kw, ki = warp - sub * p.kw, first = ki * NB;  // the warp's tiles of a step, its blocks of the part
    const int nb = max(0, min(NB, here - first));  // of which the part has so many; what is behind has x = 0
    const int64_t tile_bytes = (int64_t)p.blocks * BLK;
    const uint8_t* src = p.store + (int64_t)(t0 + sub * TP) * tile_bytes + (int64_t)(rank * p.part + first) * BLK;
    uint8_t* ring = smem + warp * p.slots * slot_bytes;
    uint64_t* bars = full + warp * kMaxSlots;
    // what is behind a narrower last share is never copied; its scales must not be NaN
    for (int i = nb * GPB * 8 + lane; nb < NB && i < NB * GPB * 8; i += 32)
      for (int k = 0; k < p.slots * TP; ++k)
        *reinterpret_cast<uint16_t*>(ring + (k * NB + i / (GPB * 8)) * BLK + kBlockCodes + i % (GPB * 8) * 2) = 0;
    __syncwarp();  // and the barriers that this warp has made
    int lt = t0 + sub * TP, ls = 0, ahead = 0;  // the copies' tile and slot
    const auto copy = [&]() {
      const int n = min(TP, t1 - lt);
      if (n <= 0) return;
      if (lane == 0) mbar_expect_tx(bars + ls, (uint32_t)(n * nb * BLK));
      __syncwarp();
      if (lane < n && nb > 0) bulk_load(ring + ls * slot_bytes + lane * NB * BLK, src + lane * tile_bytes, nb * BLK, bars + ls);
      src += step * tile_bytes, lt += step, ++ahead;
      if (++ls == p.slots) ls = 0;
    };
#pragma unroll 1
    for (int i = 0; i < p.slots; ++i) copy();
    // the sums' barriers, and the other CTAs'
    if (parts > 1) cluster_sync();
    else __syncthreads();

    griddep_wait();
    // B fragments: x[b][2j + e][m] are columns 4e..4e+3 of word j for token 8m + lane / 4
    uint32_t x[NB][8][MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int t = m * 8 + (lane >> 2);
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int col = (rank * p.part + first + b) * 128 + word_col<G>(lane & 3, j);
          uint4 v = make_uint4(0, 0, 0, 0);
          if (b < nb && t < nt && col < p.cols)
            v = *reinterpret_cast<const uint4*>(p.x + (tok0 + t) * p.x_stride + col);
          x[b][2 * j][m][0] = v.x, x[b][2 * j][m][1] = v.y;
          x[b][2 * j + 1][m][0] = v.z, x[b][2 * j + 1][m][1] = v.w;
        }
    }

    const Bits<T> bits;
    const uint32_t sum_at = smem_addr(sums) + ((sub * TP * p.kw + ki) * OUT + lane * 2) * 4;
    int s = 0, buf = 0, done = 0;
    uint32_t phase = 0, sum_phase = 1;
    bool ok = true;
#pragma unroll 1
    for (int t = t0; t < t1; t += step) {
      ok = wait(sum_empty + buf, sum_phase);
      if (!ok) break;
      if (t + sub * TP < t1) {  // (else: no tile for this warp in the last step)
        ok = wait(bars + s, phase);
        if (!ok) break;
        const uint32_t at = smem_addr(ring) + s * slot_bytes;
        uint32_t dst = sum_at + buf * sum_floats * 4;
        // two tiles are the upper and lower rows of the products (those behind t1 are not there: what they give is not read)
#pragma unroll
        for (int h = 0; h < MT; ++h) {
          float tot[MT][4] = {};  // rows lane / 4 of the first tile [0, 1] and of the second, tokens 8m + 2 (lane % 4) + 0, 1
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint32_t at0 = at + (2 * h * NB + b) * BLK, at1 = at0 + NB * BLK;
            const uint4 w0 = lds128(at0 + lane * 16), w1 = lds128(at1 + lane * 16);
#pragma unroll
            for (int q = 0; q < GPB; ++q) {
              float acc[MT][4] = {};
#pragma unroll
              for (int j = q * 4 / GPB; j < (q + 1) * 4 / GPB; ++j) {
                uint32_t u[4], v[4];
                unpack(bits, j == 0 ? w0.x : j == 1 ? w0.y : j == 2 ? w0.z : w0.w, u);
                unpack(bits, j == 0 ? w1.x : j == 1 ? w1.y : j == 2 ? w1.z : w1.w, v);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t f[4] = {u[2 * e], v[2 * e], u[2 * e + 1], v[2 * e + 1]};
#pragma unroll
                  for (int m = 0; m < MT; ++m) mma16816<T>(acc[m], f, x[b][2 * j + e][m][0], x[b][2 * j + e][m][1]);
                }
              }
              const uint32_t sc = kBlockCodes + (lane >> 2) * 2 * GPB + q * 2;
              const float s0 = T::lo(lds16(at0 + sc)), s1 = T::lo(lds16(at1 + sc));
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                tot[m][0] = fmaf(acc[m][0], s0, tot[m][0]), tot[m][1] = fmaf(acc[m][1], s0, tot[m][1]);
                tot[m][2] = fmaf(acc[m][2], s1, tot[m][2]), tot[m][3] = fmaf(acc[m][3], s1, tot[m][3]);
              }
            }
          }
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            sts64(dst + m * 256, tot[m][0], tot[m][1]);
            sts64(dst + m * 256 + p.kw * OUT * 4, tot[m][2], tot[m][3]);
          }
          dst += 2 * p.kw * OUT * 4;
        }
        ++done;
        if (++s == p.slots) s = 0, phase ^= 1;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sum_full + buf);
      copy();  // into the slot that has just been read
      if (++buf == SUMS) buf = 0, sum_phase ^= 1;
    }
    // a wait that gave up: shared memory must not go while copies to it are on their way
    if (!ok) drain_slots(bars, p.slots, done, ahead);
  } else {
    if (parts > 1) cluster_sync();
    else __syncthreads();
    if (warp >= kProduct) {  // ---- sums
      griddep_wait();        // (the launch before this one may still read or write y)
      uint32_t phase = 0, in_phase = 0;
      int buf = 0, in = 0;
      bool ok = true;
      const int first = warp - kProduct;
      const auto add = [&](int i) {  // this CTA's sum of tile i / MT of the step, tokens 8 (i % MT) ..
        const float* src = sums + buf * sum_floats + i / MT * p.kw * OUT + i % MT * 64 + lane * 2;
        float2 v = make_float2(0.f, 0.f);
#pragma unroll 6
        for (int k = 0; k < p.kw; ++k) {
          const float2 u = *reinterpret_cast<const float2*>(src + k * OUT);
          v.x += u.x, v.y += u.y;
        }
        return v;
      };
      const auto write = [&](int t, int i, float2 v) {
        const int tok = i % MT * 8 + (lane & 3) * 2, row = (t + i / MT) * 8 + (lane >> 2);
        if (tok >= nt || row >= p.rows) return;
        uint16_t* dst = p.y + (tok0 + tok) * p.y_stride + row;
        const uint32_t w = T::pack(v.x, v.y);
        dst[0] = (uint16_t)w;
        if (tok + 1 < nt) dst[p.y_stride] = (uint16_t)(w >> 16);
      };
#pragma unroll 1
      for (int t = t0; t < t1; t += step) {
        const int n = min(step, t1 - t) * MT;
        ok = wait(sum_full + buf, phase);
        if (!ok) break;
        if (parts == 1) {
#pragma unroll 1
          for (int i = first; i < n; i += kAdd) write(t, i, add(i));
          __syncwarp();
          if (lane == 0) mbar_arrive(sum_empty + buf);
        } else {  // (rw is 1: at most 2 results a warp)
          float2 v[2];
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (first + h * kAdd < n) v[h] = add(first + h * kAdd);
          __syncwarp();
          if (lane == 0) mbar_arrive(sum_empty + buf);
          if (rank > 0) {
            ok = wait(in_empty + in, in_phase ^ 1);  // at once in the first round
            if (!ok) break;
            const uint32_t dst = peer(inbox, 0) + (uint32_t)((in * (parts - 1) + rank - 1) * in_floats + lane * 2) * 4;
            const uint32_t bar = peer(in_full + in, 0);
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (first + h * kAdd < n) peer_store(dst + (first + h * kAdd) * 256, v[h], bar);
          } else {
            if (first == 0 && lane == 0) mbar_expect_tx(in_full + in, (uint32_t)((parts - 1) * n * 256));
            ok = wait(in_full + in, in_phase);
            if (!ok) break;
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (first + h * kAdd < n)
#pragma unroll 1
                for (int q = 0; q + 1 < parts; ++q) {
                  const float2 u = *reinterpret_cast<const float2*>(inbox + (in * (parts - 1) + q) * in_floats +
                                                                    (first + h * kAdd) * 64 + lane * 2);
                  v[h].x += u.x, v[h].y += u.y;
                }
            __syncwarp();
            if (lane > 0 && lane < parts) peer_arrive(peer(in_empty + in, lane));
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (first + h * kAdd < n) write(t, first + h * kAdd, v[h]);
          }
          __syncwarp();
          if (++in == kIn) in = 0, in_phase ^= 1;
        }
        if (++buf == SUMS) buf = 0, phase ^= 1;
      }
    }
  }
  __syncwarp();
  if (parts > 1) {  // a CTA's shared memory stays until the others are done with it
    cluster_sync();
    // Sums that nobody has waited for may still be on their way when a wait gave up.
    if (rank == 0 && *reinterpret_cast<volatile int*>(abort_flag))
      for (const uint64_t t0 = global_ns(); global_ns() - t0 < 100000;) {}
  }
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
      const int64_t row = tile * 8 + i / GPB;
      const int g = kb * GPB + i % GPB;
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

// ask: nothing is launched; the clusters that run at once go there
template <class T, int G, int MT>
cudaError_t launch(LinearParams p, const Room& room, Room* ask, cudaStream_t stream) {
  constexpr int NB = 4 / MT, BLK = block_bytes(G), TP = step_tiles(MT);
  // the cluster: as few CTAs as hold x in registers
  int parts = (p.blocks + kProduct * NB - 1) / (kProduct * NB);
  p.part = (p.blocks + parts - 1) / parts;
  parts = (p.blocks + p.part - 1) / p.part;
  // A range of tiles for each cluster that runs at once.  A cluster's CTAs, one an SM, sit in one of the GPU's processor clusters of up to
  // 20 SMs, so that 152 SMs do not hold 152 / parts of them (of 3 46, of 6 23, of 8 15); one that waits for another to end takes as long
  // again.  us with ranges for 152 / parts clusters / for those that fit: 16 tokens of 8192 x 8192 27.8 / 17.8, x 12288 34.2 / 19.2,
  // x 24576 59.8 / 38.0, of 40000 x 8192 95 / 59; one of 40000 x 16384 144 / 87.
  const int fit = room.clusters[MT - 1] ? room.clusters[MT - 1] : room.num_sms / parts;
  // The warps: as many of a tile's blocks each as keeps most of them busy (fewer warps a tile are fewer sums to add), several
  // steps' tiles at once where a tile takes few warps, while every cluster still gets some.
  const int clusters = std::min(fit, p.tiles), most = (p.tiles + clusters - 1) / clusters;
  int best = -1, blocks = 1;
  for (int nb = 1; nb <= NB; ++nb) {
    const int kw = (p.part + nb - 1) / nb;
    if (kw > kProduct) continue;
    const int rw = std::max(1, std::min(kProduct / kw, (most + TP - 1) / TP)), busy = p.part * rw * 12 / nb;  // (12 / nb is whole)
    if (busy >= best) best = busy, blocks = nb, p.kw = kw, p.rw = rw;
  }
  const int step = p.rw * TP, ring = p.kw * p.rw * TP * blocks * BLK;  // of one slot of every warp
  const int rest = step * (sum_buffers(MT) * p.kw + kIn * (parts - 1)) * MT * 64 * 4 +
                   (kProduct * kMaxSlots + 2 * sum_buffers(MT) + 2 * kIn) * 8 + 16;
  // Two slots a warp, more while they are small: deeper rings delay x, which waits in the same queues.  us with 2 / 3 / 4 slots of 50 KB:
  // 8192 x 6144 for one token 8.6 / 9.2 / 9.7, 40000 rows 26.4 / 27.5 / 27.7.
  p.slots = std::max(2, std::min({kMaxSlots, kRing / ring, (most + step - 1) / step}));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(clusters * parts, (p.n_tokens + 8 * MT - 1) / (8 * MT));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = p.slots * ring + rest;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = parts, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = parts > 1 ? 2 : 1;
  void (*kernel)(LinearParams) = blocks == 2 ? linear_kernel<T, G, MT, 2> : linear_kernel<T, G, MT, 1>;
  if constexpr (MT == 1) kernel = blocks == 4 ? linear_kernel<T, G, 1, 4> : blocks == 3 ? linear_kernel<T, G, 1, 3> : kernel;
  if (!ask) return cudaLaunchKernelEx(&cfg, kernel, p);
  int n = room.num_sms;
  const cudaError_t e = parts > 1 ? cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) : cudaSuccess;
  ask->clusters[MT - 1] = std::max(1, std::min(n, room.num_sms / parts));
  return e;
}

template <class T, int G, int MT, int NB>
cudaError_t configure() {
  return cudaFuncSetAttribute(linear_kernel<T, G, MT, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
}

template <class T, int G>
cudaError_t launch_tokens(const LinearParams& p, bool few, const Room& room, Room* ask, cudaStream_t stream) {
  // (x of 16 tokens and more columns than a cluster holds: 8 tokens at a time)
  return few || p.blocks > kMaxParts * kProduct * 2 ? launch<T, G, 1>(p, room, ask, stream) : launch<T, G, 2>(p, room, ask, stream);
}
template <class T>
cudaError_t launch_group(const LinearParams& p, int group, bool few, const Room& room, Room* ask, cudaStream_t stream) {
  return group == 128  ? launch_tokens<T, 128>(p, few, room, ask, stream)
         : group == 64 ? launch_tokens<T, 64>(p, few, room, ask, stream)
                       : launch_tokens<T, 32>(p, few, room, ask, stream);
}
cudaError_t launch_type(const LinearParams& p, const coli_linear_config& c, bool few, const Room& room, Room* ask, cudaStream_t stream) {
  return c.dtype == COLI_ATTN_BF16 ? launch_group<Bf16>(p, c.group, few, room, ask, stream)
                                   : launch_group<Fp16>(p, c.group, few, room, ask, stream);
}

LinearParams params(const coli_linear* h) {
  LinearParams p = {};
  p.store = h->store, p.status = h->status;
  p.rows = h->cfg.rows, p.cols = h->cfg.cols, p.tiles = h->tiles, p.blocks = h->blocks;
  return p;
}

// how many clusters of the handle's shape run at once
cudaError_t ask_room(coli_linear* h) {
  LinearParams p = params(h);
  p.n_tokens = 8;
  const Room room = h->room;
  const cudaError_t e = launch_type(p, h->cfg, true, room, &h->room, nullptr);
  return e == cudaSuccess ? launch_type(p, h->cfg, false, room, &h->room, nullptr) : e;
}

cudaError_t configure_device() {
  cudaError_t e = cudaSuccess;
#define COLI_CFG(T, G)                                \
  if (e == cudaSuccess) e = configure<T, G, 1, 1>();  \
  if (e == cudaSuccess) e = configure<T, G, 1, 2>();  \
  if (e == cudaSuccess) e = configure<T, G, 1, 3>();  \
  if (e == cudaSuccess) e = configure<T, G, 1, 4>();  \
  if (e == cudaSuccess) e = configure<T, G, 2, 1>();  \
  if (e == cudaSuccess) e = configure<T, G, 2, 2>();
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
      c.cols > 32768)
    return COLI_EUNSUPPORTED;
  coli_linear* h = new (std::nothrow) coli_linear();
  if (!h) return COLI_ENOMEM;
  h->cfg = c;
  h->tiles = (c.rows + 7) / 8, h->blocks = (c.cols + 127) / 128;
  int rc = COLI_OK;
  if (cudaGetDevice(&h->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&h->room.num_sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess ||
      configure_device() != cudaSuccess || configure_linear_many() != cudaSuccess || ask_room(h) != cudaSuccess)
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
  LinearParams p = params(h);
  p.x_stride = x_stride, p.y_stride = y_stride;
  cudaError_t e = cudaSuccess;
  for (int at = 0; at < n_tokens && e == cudaSuccess; at += kLaunchTokens) {
    p.x = static_cast<const uint16_t*>(x) + at * x_stride, p.y = static_cast<uint16_t*>(y) + at * y_stride;
    p.n_tokens = std::min(n_tokens - at, kLaunchTokens);
    if (n_tokens > 16 && c.group == 128)  // both sides' times: linear_many.cu
      e = launch_linear_many(p, c.dtype, h->room.num_sms, (cudaStream_t)stream);
    else
      e = launch_type(p, c, n_tokens <= 8, h->room, nullptr, (cudaStream_t)stream);
  }
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

// Attention of many query rows over a paged cache on the fifth-generation tensor cores.
//
// A block is 2 x 128 rows (tokens x query heads of one key head, whole tokens only).  For every tile
// of 128 keys S = Q K^T goes to tensor memory, a warpgroup per 128 rows (one thread a row, so neither
// maxima nor sums cross threads) turns it into P = 2^(scale S - m), written over S in 16 bits, and
// O += P V reads P from tensor memory and stays there.  The two row tiles alternate: while one's
// scores are in the softmax the other's products run, and the matrix unit is meant never to wait.
//
//   tensor memory (512 columns)   S0/P0 | S1/P1 | O0 | O1
//   shared memory                 Q0, Q1 and a ring of key and value tiles, 128-byte swizzled boxes
//   warps 0-3, 4-7   softmax, rescaling and the epilogue of row tile 0, 1
//   warp 8           issues every product; warp 9 every copy
//   warps 10, 11     look at value tiles with keys that not every row sees
//
// The maximum that P refers to is only raised when a row's scores outgrow it by 2^8 (O is rescaled then,
// in fp32): P stays within 2^8, far inside the 16-bit types' range, and rescaling is rare.
//
// Rows that do not see a key have P = 0 there, and 0 * inf is NaN: so values of keys that no row of the
// block sees are set to zero in shared memory, and a block of which some rows see a non-finite value
// and others do not is put on a list and computed again, row by row, by the kernel that follows.
//
// The list of all blocks' key tiles is cut into one equal stretch per SM (attn_sched.cuh), so few long
// rows fill the GPU as well as many short ones.
//
// Measured: 8192 new tokens, 6 query heads a key head, 8 key heads of 128, window 4096: calls in a row 450 us, under the
// power cap, 1.37 PFLOP/s of the scores that rows see; the first ones after a pause 420 us, 1.47 PFLOP/s (1.59 of those
// computed; cuBLAS reaches 1.94 in bf16, 1.71 under the cap).  After a pause a key tile takes both row tiles 1.53 us
// (8.4 MFLOP of each): the products alone 1.0, the rest is what the two softmax chains leave uncovered; the tensor
// pipe is 60 % busy at 4096 tokens, where units of few tiles at the start of the sequence cost more.  A block that
// fills one row tile takes about 1.2 us a tile, its products and softmax one after another: below the 1.47 us that its
// keys and values take from DRAM when every SM reads others.
#include <float.h>

#include "attn_tc.cuh"

namespace coli {

namespace {

constexpr int kThreadsTile = 12 * 32;
constexpr int kTileSmemRing = 163840;

template <int D>
struct TileCfg {
  static constexpr int tile_bytes = kTileKeys * D * 2;  // K or V of one stage; Q of one row tile
  static constexpr int stages = kTileSmemRing / tile_bytes;
  static constexpr int q_bytes = 2 * tile_bytes;
  // barriers: ring full/empty/checked, q full/empty, scores, weights (first half, all), output, drain
  static constexpr int bars = 3 * stages + 4 + 2 + 4 + 2 + 1;
  static constexpr int smem = kTileSmemRing + q_bytes + (int)sizeof(UnitRing) + bars * 8 + 16;
  static constexpr uint32_t o_col = 256;  // first column of O0; O1 follows after D columns
};

template <class T, int D>
__global__ void __launch_bounds__(kThreadsTile, 1)
    attn_tile_kernel(const AttnParams p, const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using C = TileCfg<D>;
  constexpr int NST = C::stages;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem;  // key tile i is item 2i, value tile i item 2i + 1
  uint8_t* qs = smem + kTileSmemRing;
  UnitRing* units = reinterpret_cast<UnitRing*>(qs + C::q_bytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(units + 1);
  uint64_t *empty = full + NST, *checked = empty + NST, *q_full = checked + NST, *q_empty = q_full + 2,
           *s_full = q_empty + 2, *p_half = s_full + 2, *p_full = p_half + 2, *o_full = p_full + 2, *drain = o_full + 2;
  int* abort_flag = reinterpret_cast<int*>(drain + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(abort_flag + 1);
  // (the shuffle tells the compiler that a warp's number, and with it every role's control flow, is uniform)
  const int tid = threadIdx.x, warp = __shfl_sync(FULL, tid >> 5, 0), lane = tid & 31;
  const auto wait = [&](uint64_t* bar, uint32_t parity) { return warp_wait(bar, parity, abort_flag, p.status); };

  if (tid == 0) {
    *abort_flag = 0;
    units->init(11);  // every warp but the copying one
#pragma unroll 1
    for (int i = 0; i < NST; ++i) mbar_init(full + i, 1), mbar_init(empty + i, 1), mbar_init(checked + i, 2);
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {
      mbar_init(q_full + s, 1), mbar_init(q_empty + s, 1), mbar_init(s_full + s, 1);
      mbar_init(p_half + s, 4), mbar_init(p_full + s, 4), mbar_init(o_full + s, 1);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
    prefetch_map(&qmap), prefetch_map(&kmap), prefetch_map(&vmap);
  }
  if (warp == 8) tmem_alloc(tmem_slot, 512);
  const bool few = n_lists(p) <= 32;
  Walk<kTileKeys> walk;
  if (few && warp == 9) walk.start_few(p, lane, p.late_wait);  // without the late wait: the dry run
  uint32_t* weights = reinterpret_cast<uint32_t*>(smem);  // in the ring, before the first copy
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (!p.late_wait) griddep_wait();
  if (few && warp == 9 && !p.late_wait) walk.start_few(p, lane, true);
  if (!few) weigh<kTileKeys>(p, weights);
  griddep_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  const int half_tokens = p.block_tokens / 2;  // tokens of one row tile

  // registers: 200 for each of the 256 softmax threads, 104 for the others: the 384 x 168 of the launch
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    Unit u;
    bool ok = true;
    if (warp == 9) {  // ---- copies
      if (!few) walk.start(p, weights, lane);
      if (lane == 0) p.rec[blockIdx.x].first_cta = -1;
      __syncwarp();
      fence_proxy_async_smem();
      int it = 0, n = 0, qn0 = 0, qn1 = 0;  // items, units, queries of either row tile
      const uint32_t qb = (uint32_t)(p.group * half_tokens) * D * 2;
#pragma unroll 1
      while (ok && walk.next(p, u)) {
        ok = give_unit(units, u, n++, lane, wait);
#pragma unroll 1
        for (int s = 0; s < 2 && ok && u.nt > s * half_tokens; ++s) {
          const int qn = s ? qn1 : qn0;
          if (qn > 0) ok = wait(q_empty + s, (qn - 1) & 1);
          if (!ok) break;
          s ? ++qn1 : ++qn0;
          if (lane == 0) {
            mbar_expect_tx(q_full + s, qb);
#pragma unroll
            for (int sl = 0; sl < D / 64; ++sl)
              tma_load_3d(qs + s * C::tile_bytes + sl * kTileKeys * 128, &qmap, sl * 64, u.head * p.group,
                          u.tok0 + s * half_tokens, q_full + s);
          }
          __syncwarp();
        }
        const int32_t* row = table_of(p, u.b);
#pragma unroll 1
        for (int i = 2 * u.i0; i < 2 * u.i1 && ok; ++i, ++it) {
          const int j0 = u.tile(i >> 1) * kTileKeys, sg = it % NST;
          if (it >= NST) ok = wait(empty + sg, ((it / NST) + 1) & 1);
          if (!ok) break;
          fill_boxes<kTileKeys, D, 1>(p, i & 1 ? &vmap : &kmap, nullptr, ring + sg * C::tile_bytes, full + sg, row, u.p0, u.p1, j0, u.head, lane);
        }
      }
      u.i1 = 0;
      if (ok) give_unit(units, u, n, lane, wait);
      // the CTA's shared memory must not go while copies to it are on their way, even when the other warps have given up
      drain_ring(full, NST, it);
      drain_ring(q_full, 1, qn0);
      drain_ring(q_full + 1, 1, qn1);
    } else if (warp == 8) {  // ---- products (one lane issues; the warp waits together)
      constexpr uint32_t qk_idesc = mma_desc<T>(kTileKeys, false), pv_idesc = mma_desc<T>(D, true);
      // descriptors of the first tiles; others are a whole number of 16-byte units further (no carry out of
      // the 14-bit address field: shared memory ends below 2^18 bytes)
      const uint64_t q_desc = smem_desc_sw128(qs), k_desc = smem_desc_sw128(ring), v_desc = smem_desc_values(ring);
      // Scores run one key tile ahead of values: a_* is the unit they are in (a_left tiles to go, a_first: none
      // yet), b_* the values' one.  Each round issues, for either row tile, values of one tile and scores of the
      // next.  This warp's instructions are what the matrix unit waits for, so a round is one elected lane's, with
      // everything that is the same for all lanes worked out before it, and a wait that gives up does not leave
      // the loop: the later ones then return at once.
      int units_taken = 0;
      int vs = NST - 1, ks = 0;  // stages of the value and the key tile (the first round has no values)
      uint32_t vphase = 1, kphase = 0, pphase0 = 0, pphase1 = 0, qphase0 = 0, qphase1 = 0;
      int a_left = 0, b_left = 0;
      bool a_two = false, b_two = false, a_first = false, b_first = false;
      const auto take = [&]() {
        if (!take_unit(units, u, units_taken++, lane, wait)) return false;
        a_left = u.i1 - u.i0, a_two = u.nt > half_tokens, a_first = true;
        return true;
      };
      const auto wait1 = [&](uint64_t* bar, uint32_t parity) { lane_wait(bar, parity, abort_flag, p.status); };
      bool more = take();
#pragma unroll 1
      while (more || b_left > 0) {
        const uint64_t bv = v_desc + vs * (C::tile_bytes >> 4), bk = k_desc + ks * (C::tile_bytes >> 4);
        const bool pv0 = b_left > 0, pv1 = pv0 && b_two, qk1 = more && a_two, o_last = b_left == 1, s_last = a_left == 1;
        if (elect_one()) {
          if (pv0) wait1(checked + vs, vphase);
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (s ? pv1 : pv0) {
              const uint32_t d = tmem + C::o_col + s * D, a = tmem + s * 128;
              wait1(p_half + s, s ? pphase1 : pphase0);  // the first 64 keys' weights are there
              tc_fence_after();
              tc_mma_ts(d, a, bv, pv_idesc, !b_first);
#pragma unroll
              for (int k = 1; k < 4; ++k) tc_mma_ts(d, a + k * 8, bv + k * (2048 >> 4), pv_idesc, true);
              wait1(p_full + s, s ? pphase1 : pphase0);
              tc_fence_after();
#pragma unroll
              for (int k = 4; k < 8; ++k) tc_mma_ts(d, a + k * 8, bv + k * (2048 >> 4), pv_idesc, true);
              if (o_last) tc_commit(o_full + s);
              if (s == 1 || !pv1) tc_commit(empty + vs);
            }
            if (s ? qk1 : more) {
              if (a_first) wait1(q_full + s, s ? qphase1 : qphase0);
              if (s == 0) wait1(checked + ks, kphase);
              tc_fence_after();
              const uint64_t a = q_desc + s * (C::tile_bytes >> 4);
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const int off = ((k >> 2) * kTileKeys * 128 + (k & 3) * 32) >> 4;
                tc_mma_bf16(tmem + s * 128, a + off, bk + off, qk_idesc, k > 0);
              }
              tc_commit(s_full + s);
              if (s_last) tc_commit(q_empty + s);
            }
          }
          if (more) tc_commit(empty + ks);
        }
        __syncwarp();
        pphase0 ^= pv0, pphase1 ^= pv1;
        if (a_first) qphase0 ^= more, qphase1 ^= qk1;
        if ((vs += 2) >= NST) vs -= NST, vphase ^= 1;
        if ((ks += 2) >= NST) ks -= NST, kphase ^= 1;
        if (b_left > 0) --b_left, b_first = false;
        if (b_left == 0 && more) b_left = a_left, b_two = a_two, b_first = true;  // the scores of its first tile are out
        if (more) {
          a_first = false;
          if (--a_left == 0) more = take();
        }
      }
      // Nor must tensor memory while products write to it: usually the softmax warps have waited for them, but not when they
      // gave up.  (With a limit of its own.)
      if (elect_one()) tc_commit(drain);
      __syncwarp();
      drain_ring(drain, 1, 1);
    } else {
      // ---- values that not every row sees.  These warps pass every item of the ring on to the products' warp, key
      // tiles too: a waiter that skipped items could meet a stage whose previous item is still on its way
      // and take the barrier's older phase for the one it wants.
      int it = 0;
#pragma unroll 1
      for (int n = 0; ok && take_unit(units, u, n, lane, wait); ++n) {
        uint32_t bad = 0;
#pragma unroll 1
        for (int i = 2 * u.i0; i < 2 * u.i1; ++i, ++it) {
          const int sg = it % NST;
          ok = wait(full + sg, (it / NST) & 1);
          if (!ok) break;
          const int j0 = u.tile(i >> 1) * kTileKeys;
          if ((i & 1) && !all_see(p, u.p0, u.p1, j0, j0 + kTileKeys - 1)) {
            // warp 10 takes the even keys, 11 the odd ones; 8 lanes a 128-byte row
#pragma unroll 1
            for (int r = (warp - 10) + (lane >> 3) * 2; r < kTileKeys; r += 8) {
              if (all_see(p, u.p0, u.p1, j0 + r, j0 + r)) continue;
              const bool some = some_sees(p, u.p0, u.p1, j0 + r);
#pragma unroll
              for (int sl = 0; sl < D / 64; ++sl) {
                uint4* v = reinterpret_cast<uint4*>(ring + sg * C::tile_bytes + sl * kTileKeys * 128 + r * 128) + (lane & 7);
                if (some) {
                  const uint4 x = *v;
                  bad |= nonfinite2<T>(x.x) | nonfinite2<T>(x.y) | nonfinite2<T>(x.z) | nonfinite2<T>(x.w);
                } else {
                  *v = make_uint4(0, 0, 0, 0);
                }
              }
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(checked + sg);
        }
        if (__any_sync(FULL, bad != 0)) flag_unit(p, u, lane);
      }
    }
  } else {  // ---- softmax of row tile s; thread = row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int s = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t st_addr = tmem + lane_base + s * 128, ot_addr = tmem + lane_base + C::o_col + s * D;
    const int tok = row / p.group;
    const float slack = fminf(8.f / p.scale_log2, FLT_MAX);  // finite: -inf + inf would never let the first keys in
    uint32_t sn = 0, on = 0;
    Unit u;
#pragma unroll 1
    for (int n = 0; take_unit(units, u, n, lane, wait); ++n) {
      const int nt = min(half_tokens, u.nt - s * half_tokens);
      if (nt <= 0) continue;
      const bool causal = u.flags & kCausal, whole = u.flags & kWhole;
      float* const dense_o = p.dense_o[causal ? 0 : 1];
      const int pa = causal ? u.p0 + s * half_tokens : u.p0;  // the row tile's positions
      const int pb = causal ? pa + nt - 1 : pa;
      const int pos = causal ? pa + tok : pa;
      float ref = -INFINITY, sum0 = 0.f, sum1 = 0.f;
      bool ok = true;
#pragma unroll 1
      for (int i = u.i0; i < u.i1; ++i) {
        ok = wait(s_full + s, sn & 1);
        ++sn;
        if (!ok) break;
        tc_fence_after();
        const int j0 = u.tile(i) * kTileKeys;
        float x[128];
        COLI_LD32(st_addr, x);
        COLI_LD32(st_addr + 32, x + 32);
        COLI_LD32(st_addr + 64, x + 64);
        COLI_LD32(st_addr + 96, x + 96);
        float m0 = -INFINITY, m1 = m0, m2 = m0, m3 = m0;
        const bool masked = !all_see(p, pa, pb, j0, j0 + kTileKeys - 1);
        const int hi = pos - j0, lo = pos - p.window - j0, sk = p.sinks - j0;
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          COLI_LDWAIT32(x + c);
          if (masked) {  // bit k: the row sees key c + k
            const uint32_t see = low_bits(hi + 1 - c) & (~low_bits(lo + 1 - c) | low_bits(sk - c));
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!(see & (1u << k))) x[c + k] = -INFINITY;
          }
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            m0 = max3(m0, x[c + k], x[c + k + 1]);
            m1 = max3(m1, x[c + k + 2], x[c + k + 3]);
            m2 = max3(m2, x[c + k + 4], x[c + k + 5]);
            m3 = max3(m3, x[c + k + 6], x[c + k + 7]);
          }
        }
        const float top = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
        const bool grow = top > ref + slack;  // ref = -inf: the row's first keys
        if (__any_sync(FULL, grow)) {
          float fix = 1.f;
          if (grow) {
            fix = ref == -INFINITY ? 1.f : ex2((ref - top) * p.scale_log2);  // nothing added up yet: 1
            ref = top;
            sum0 *= fix, sum1 *= fix;
          }
          // the scores' commit also covers the products before them: O is complete
          if (i > u.i0 && __any_sync(FULL, fix != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float o[32];
              COLI_LD32(ot_addr + c, o);
              COLI_LDWAIT32(o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] *= fix;
              COLI_ST32(ot_addr + c, o);
            }
          }
        }
        const float base = ref == -INFINITY ? 0.f : -ref * p.scale_log2;
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float e = base, f = base;
            fma2_rn(x[c + 2 * k], x[c + 2 * k + 1], p.scale_log2, p.scale_log2, e, f);
            e = ex2(e), f = ex2(f);
            x[c + 2 * k] = e, x[c + 2 * k + 1] = f;
            w[k] = T::pack(e, f);
          }
          tmem_st16u(st_addr + c / 2, w);
          if (c == 32) {  // the products of the first 64 keys can start
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_half + s);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + s);
        float s2 = 0.f, s3 = 0.f;  // the sum is not needed before the end of the unit
#pragma unroll
        for (int c = 0; c < 128; c += 4) {
          add2_rn(x[c], x[c + 1], sum0, sum1);
          add2_rn(x[c + 2], x[c + 3], s2, s3);
        }
        sum0 += s2, sum1 += s3;
      }
      if (!ok) break;
      ok = wait(o_full + s, on & 1);
      ++on;
      if (!ok) break;
      tc_fence_after();
      const float sum = sum0 + sum1, m2 = ref * p.scale_log2;
      const int token = u.tok0 + s * half_tokens + tok, hq = u.head * p.group + row - tok * p.group;
      const bool live = tok < nt;
      if (whole && !dense_o) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        uint16_t* dst = static_cast<uint16_t*>(p.out) + (int64_t)token * p.out_stride + (int64_t)hq * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          COLI_LD32(ot_addr + c, o);
          COLI_LDWAIT32(o);
          if (live) {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = T::pack(o[2 * k] * inv, o[2 * k + 1] * inv);
            st_out(dst + c, w, p.out_sectors);
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = T::pack(o[16 + 2 * k] * inv, o[17 + 2 * k] * inv);
            st_out(dst + c + 16, w, p.out_sectors);
          }
        }
        if (live && p.lse)
          p.lse[(int64_t)token * p.n_q + hq] = sum == 0.f ? -INFINITY : (m2 + log2f(sum)) * 0.69314718055994530942f;
      } else {
        // a cut unit's rows are numbered over both row tiles: row tile 1 starts at half_tokens * group
        const int64_t at = whole ? (int64_t)token * p.n_q + hq
                                   : ((int64_t)blockIdx.x * 2 + (u.i0 > 0 ? 0 : 1)) * kTileRows +
                                         s * half_tokens * p.group + row;
        float* dst = (whole ? dense_o : p.part_o) + at * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          COLI_LD32(ot_addr + c, o);
          COLI_LDWAIT32(o);
          if (live) {
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(o[k + e]);
              st_sector(dst + c + k, w);
            }
          }
        }
        if (live) (whole ? p.dense_ml[causal ? 0 : 1] : p.part_ml)[at] = make_float2(m2, sum);
      }
      tc_fence_before();  // the next unit's products overwrite O after this row tile's next arrival
    }
  }
  // With a late wait this grid starts as the one before it leaves the SMs, and is done only when that one is: whoever
  // waits for this grid then has waited for both.
  if (p.late_wait) griddep_wait();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

template <class T, int D>
cudaError_t launch(const AttnParams& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, int grid,
                   cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreadsTile);
  cfg.dynamicSmemBytes = TileCfg<D>::smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_tile_kernel<T, D>, p, q, k, v);
}

template <class T, int D>
cudaError_t configure() {
  return cudaFuncSetAttribute(attn_tile_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              TileCfg<D>::smem);
}

}  // namespace

cudaError_t configure_attn_tile() {
  cudaError_t e = configure<Bf16, 64>();
  if (e == cudaSuccess) e = configure<Bf16, 128>();
  if (e == cudaSuccess) e = configure<Fp16, 64>();
  if (e == cudaSuccess) e = configure<Fp16, 128>();
  return e;
}

int tile_block_tokens(int group) { return 2 * (128 / group); }

cudaError_t launch_attn_tile(const AttnParams& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                             int dtype, int num_sms, cudaStream_t stream) {
  if (dtype == COLI_ATTN_BF16)
    return p.head_dim == 64 ? launch<Bf16, 64>(p, q, k, v, num_sms, stream) : launch<Bf16, 128>(p, q, k, v, num_sms, stream);
  return p.head_dim == 64 ? launch<Fp16, 64>(p, q, k, v, num_sms, stream) : launch<Fp16, 128>(p, q, k, v, num_sms, stream);
}

}  // namespace coli

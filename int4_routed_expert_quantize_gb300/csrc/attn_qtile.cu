// Attention of many query rows over a paged cache of 8-bit codes on the fifth-generation tensor cores: attn_tile.cu's plan, with
// a warpgroup that widens the code tiles on their way to the products.
//
//   tensor memory (512 columns)   S0/P0 | S1/P1 | O0 | O1
//   shared memory                 Q0, Q1; a ring of key and value tiles; scales
//   warps 0-3, 4-7   softmax, rescaling and the epilogue of row tile 0, 1
//   warps 8-11       widen, in place: the codes come into the second half of their tile's place; a thread makes one key's into D
//                    16-bit values where a tensor copy would have put them
//   warp 12          issues every product; warp 13 every copy
//
// The codes are exact in the products: keys in the queries' type, values in fp16.  A score is multiplied by its key's scale in fp32; a
// weight is 2^(s - m) vs, with m the row's largest s + log2 |vs|, to within 11, so that it is at most 2^11 and rounds to fp16 well.
// m moves rarely, and the output in tensor memory is rescaled only then.  So a tile's scores become exponents in one step, t = acc ks - m,
// and a tile whose largest t and largest |vs| could make too large a weight is the exception in which the row looks for its largest t + log2 |vs|.
// What a row does not see has weight 0; codes are always finite, and values' scales that are not become 0 and a bit that spoils the
// sums of the rows that see them, so nothing is computed again here.
//
// Measured, with the combine kernel: 8192 tokens, window 4096, 48 query and 8 key heads of 128, int8: 838 us (0.74 PFLOP/s; 450 over a 16-bit cache), e4m3 769.  A
// round of both row tiles takes 6300 cycles, the products of it 2050: they wait for weights, whose softmax takes 4000.  Beside 831 of an earlier form: two threads a row 930,
// a second pass over tensor memory instead of 128 registers 1047, one pass over 64 keys and another where m moves 828, four rows a thread 860.
//
// The softmax loop is long straight code and shares the instruction cache with the other roles', so what only masked tiles need is
// kept out of it.
#include <float.h>

#include "attn_code.cuh"
#include "attn_tc.cuh"

namespace coli {

namespace {

constexpr int kThreadsQTile = 16 * 32;
constexpr float kRoom = 11.f;  // log2 of the largest weight

struct TileScales {
  float keys[kTileKeys], values[kTileKeys];
  float logs[kTileKeys];  // scale_log of the values'
  float top[4];     // of 32 keys each: the largest of these
  uint32_t bad[4];  // and which of them were not finite
};

template <int D>
struct QTileCfg {
  static constexpr int tile_bytes = kTileKeys * D * 2;  // of a widened tile; Q of one row tile
  static constexpr int raw_bytes = kTileKeys * D;       // of a code tile
  static constexpr int stages = 131072 / tile_bytes;
  static constexpr int q_bytes = 2 * tile_bytes;
  // Scales of a tile's keys and values.  A tile's are asked for when the key tile stages / 2 before it has been multiplied, so
  // the tile before that one has left the softmax.
  static constexpr int scale_slots = stages / 2 + 1;
  // barriers: ring codes/full/empty, q full/empty, scores, weights (first half, all), output, drain, reading, scales
  static constexpr int bars = 3 * stages + 4 + 2 + 4 + 2 + 2 + scale_slots;
  static constexpr int smem =
      stages * tile_bytes + q_bytes + scale_slots * (int)sizeof(TileScales) + (int)sizeof(UnitRing) + bars * 8 + 16;
  static constexpr uint32_t o_col = 256;  // first column of O0; O1 follows after D columns
};

// (a0, a1) *= (b0, b1)
__device__ __forceinline__ void mul2_rn(float b0, float b1, float& a0, float& a1) {
  asm("{\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tmul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}

// One warp fills a stage of the ring with the codes of a 128-key tile, keys or values, and (keys) the scales of both: as fill_codes
template <int D, bool KEYS>
__device__ __forceinline__ void fill_item(const AttnParams& p, const CUtensorMap* map, uint8_t* dst, float* scales, uint64_t* bar,
                                          const int32_t* table, int p0, int p1, int j0, int head, int lane) {
  const int page = 1 << p.page_shift;
  const int rows = min(page, kTileKeys), boxes = kTileKeys / rows;
  const int a = j0 + lane * rows, e = a + rows - 1;  // the lane's keys
  const bool need = lane < boxes && a <= p1 && (e > p0 - p.window || a < p.sinks);
  int id = 0;
  if (need) id = __ldg(table + (a >> p.page_shift));
  const bool bad = need && (id < 0 || id >= p.n_pages);
  if (bad) {
    id = p.n_pages;
    if (KEYS) {
      atomicExch(p.status, COLI_EINVAL);
      for (int i = 0; i < rows; ++i) scales[lane * rows + i] = scales[kTileKeys + lane * rows + i] = 0.f;
      fence_proxy_async_smem();
    }
  }
  const int n = __popc(__ballot_sync(FULL, need)), good = KEYS ? n - __popc(__ballot_sync(FULL, bad)) : 0;
  __syncwarp();
  if (lane == 0) mbar_expect_tx(bar, (uint32_t)rows * (uint32_t)(n * D + good * 8));
  __syncwarp();
  if (need) {
    const int slot = a & (page - 1);
    tma_load_4d(dst + lane * rows * D, map, 0, slot, head, id, bar);
    if (KEYS && !bad) {
      bulk_load(scales + lane * rows, p.k_scale + id * p.ks_page + head * p.ks_head + slot, rows * 4, bar);
      bulk_load(scales + kTileKeys + lane * rows, p.v_scale + id * p.vs_page + head * p.vs_head + slot, rows * 4, bar);
    }
  }
  __syncwarp();
}

// Four codes of a word -> two pairs in order, in the type of `T`; a code is Code<CODE>::unit times the value.
template <class T, int CODE>
__device__ __forceinline__ void widen_pairs(uint32_t w, uint32_t& a, uint32_t& b) {
  constexpr bool bf16 = T::kExp == Bf16::kExp;
  if constexpr (CODE == COLI_ATTN_CODE_INT8) {
    if constexpr (bf16) {  // 128 + (c & 127), less 128 or, for a negative c, 256
      const uint32_t r[2] = {__byte_perm(w, 0x43434343u, 0x4140), __byte_perm(w, 0x43434343u, 0x4342)};
      asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(r[0] & 0xFF7FFF7Fu), "r"(r[0] & 0xFF80FF80u));
      asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(r[1] & 0xFF7FFF7Fu), "r"(r[1] & 0xFF80FF80u));
    } else {
      const uint32_t u = w ^ 0x80808080u;
      a = Code<CODE>::minus(__byte_perm(u, 0x64646464u, 0x4140));
      b = Code<CODE>::minus(__byte_perm(u, 0x64646464u, 0x4342));
    }
  } else {
    const uint32_t t = __byte_perm(w, 0u, 0x1404), u = __byte_perm(w, 0u, 0x3424);  // the codes as high bytes
    if constexpr (bf16) {  // exponent and mantissa at bf16's lowest exponents, times 2^112
      a = ((t >> 4) & 0x07F007F0u) | (t & 0x80008000u), b = ((u >> 4) & 0x07F007F0u) | (u & 0x80008000u);
      asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(0x77807780u));
      asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(b) : "r"(0x77807780u));
    } else {
      a = ((t >> 1) & 0x3F803F80u) | (t & 0x80008000u), b = ((u >> 1) & 0x3F803F80u) | (u & 0x80008000u);
    }
  }
}

// 16 codes as two 16-byte chunks of a widened row
template <class T, int CODE>
__device__ __forceinline__ void write_chunks(const uint4& v, uint8_t* row_at, int ch, int row) {
  uint4 x, y;
  widen_pairs<T, CODE>(v.x, x.x, x.y), widen_pairs<T, CODE>(v.y, x.z, x.w);
  widen_pairs<T, CODE>(v.z, y.x, y.y), widen_pairs<T, CODE>(v.w, y.z, y.w);
  *reinterpret_cast<uint4*>(row_at + ((ch ^ (row & 7)) << 4)) = x;
  *reinterpret_cast<uint4*>(row_at + (((ch + 1) ^ (row & 7)) << 4)) = y;
}

// One key's row: its codes, as the tensor copies swizzle them in the second half of the tile's place, to boxes of 64 values x 128 keys.
// A row of 128 codes lies just where its own second 64 values go, chunk by chunk behind those that have been read, so nothing is
// overwritten before its time; rows of 64 codes lie where others' values go, and `meet` makes all threads wait until all have read
// theirs.  (In a loop: unrolled by 2 or 4 its instructions came late, 866 / 934 / 966 us for 8192 tokens.)
template <class T, int CODE, int D, class Meet>
__device__ __forceinline__ bool widen_row(uint8_t* tile, int row, Meet meet) {
  const uint8_t* raw = tile + kTileKeys * D;
  if constexpr (D == 128) {
    uint4 next = *reinterpret_cast<const uint4*>(raw + row * 128 + ((row & 7) << 4));
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
      const uint4 v = next;
      if (c < 7) next = *reinterpret_cast<const uint4*>(raw + row * 128 + (((c + 1) ^ (row & 7)) << 4));
      write_chunks<T, CODE>(v, tile + (c >> 2) * kTileKeys * 128 + row * 128, 2 * c & 7, row);
    }
  } else {
    uint4 v[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = *reinterpret_cast<const uint4*>(raw + row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
    if (!meet()) return false;
#pragma unroll
    for (int c = 0; c < 4; ++c) write_chunks<T, CODE>(v[c], tile + row * 128, 2 * c, row);
  }
  return true;
}

template <class T, int CODE, int D>
__global__ void __launch_bounds__(kThreadsQTile, 1)
    attn_qtile_kernel(const AttnParams p, const __grid_constant__ CUtensorMap qmap,
                      const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using C = QTileCfg<D>;
  constexpr int NST = C::stages, NSC = C::scale_slots;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem;  // key tile i is item 2i, value tile i item 2i + 1
  uint8_t* qs = smem + NST * C::tile_bytes;
  TileScales* scales = reinterpret_cast<TileScales*>(qs + C::q_bytes);  // [NSC]
  UnitRing* units = reinterpret_cast<UnitRing*>(scales + NSC);
  uint64_t* full = reinterpret_cast<uint64_t*>(units + 1);
  uint64_t *empty = full + NST, *codes = empty + NST, *sc_full = codes + NST,
           *q_full = sc_full + NSC, *q_empty = q_full + 2, *s_full = q_empty + 2, *p_half = s_full + 2, *p_full = p_half + 2,
           *o_full = p_full + 2, *drain = o_full + 2, *met = drain + 1;
  int* abort_flag = reinterpret_cast<int*>(met + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(abort_flag + 1);
  // (the shuffle tells the compiler that a warp's number, and with it every role's control flow, is uniform)
  const int tid = threadIdx.x, warp = __shfl_sync(FULL, tid >> 5, 0), lane = tid & 31;
  const auto wait = [&](uint64_t* bar, uint32_t parity) { return ring_wait(bar, parity, abort_flag, p.status); };

  if (tid == 0) {
    *abort_flag = 0;
    units->init(13);  // warps 0 to 12
#pragma unroll 1
    for (int i = 0; i < NST; ++i) mbar_init(full + i, 4), mbar_init(empty + i, 1), mbar_init(codes + i, 1);
#pragma unroll 1
    for (int i = 0; i < NSC; ++i) mbar_init(sc_full + i, 4);
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {
      mbar_init(q_full + s, 1), mbar_init(q_empty + s, 1), mbar_init(s_full + s, 1);
      mbar_init(p_half + s, 4), mbar_init(p_full + s, 4), mbar_init(o_full + s, 1);
    }
    mbar_init(drain, 1), mbar_init(met, 4);
    fence_barrier_init();
    prefetch_map(&qmap), prefetch_map(&kmap), prefetch_map(&vmap);
  }
  if (warp == 12) tmem_alloc(tmem_slot, 512);
  const bool few = n_lists(p) <= 32;
  Walk<kTileKeys> walk;
  if (few && warp == 13) walk.start_few(p, lane, false);
  uint32_t* weights = reinterpret_cast<uint32_t*>(smem);  // in the ring, before the first copy
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  if (few && warp == 13) walk.start_few(p, lane, true);
  if (!few) weigh<kTileKeys>(p, weights);
  griddep_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  const int half_tokens = p.block_tokens / 2;  // tokens of one row tile

  // registers: 184 for each of the 256 softmax threads, 72 for the others: the 512 x 128 of the launch
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    Unit u;
    bool ok = true;
    if (warp == 13) {  // ---- copies
      if (!few) walk.start(p, weights, lane);
      if (lane == 0) p.rec[blockIdx.x].first_cta = -1;
      __syncwarp();
      fence_proxy_async_smem();
      int tile = 0;  // of the scales' ring
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
          uint8_t* dst = ring + sg * C::tile_bytes + C::raw_bytes;
          float* sc = scales[tile].keys;
          if (i & 1) {
            fill_item<D, false>(p, &vmap, dst, sc, codes + sg, row, u.p0, u.p1, j0, u.head, lane);
            if (++tile == NSC) tile = 0;
          } else {
            fill_item<D, true>(p, &kmap, dst, sc, codes + sg, row, u.p0, u.p1, j0, u.head, lane);
          }
        }
      }
      u.i1 = 0;
      if (ok) give_unit(units, u, n, lane, wait);
      // the CTA's shared memory must not go while copies to it are on their way, even when the other warps have given up
      drain_ring(codes, NST, it);
      drain_ring(q_full, 1, qn0);
      drain_ring(q_full + 1, 1, qn1);
    } else if (warp == 12) {  // ---- products (one lane issues; the warp waits together)
      constexpr uint32_t qk_idesc = mma_desc<T>(kTileKeys, false), pv_idesc = mma_desc<Fp16>(D, true);
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
          if (pv0) wait1(full + vs, vphase);
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
              if (s == 0) wait1(full + ks, kphase);
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
    } else if (warp < 12) {  // ---- codes to 16-bit values; thread = key
      const int row = (warp - 8) * 32 + lane;
      const float rs = p.scale_log2 * Code<CODE>::unit;  // of a product of codes and q times its key's scale: log2 units
      int it = 0, slot = 0;
#pragma unroll 1
      for (int n = 0; ok && take_unit(units, u, n, lane, wait); ++n) {
#pragma unroll 1
        for (int i = 2 * u.i0; i < 2 * u.i1; ++i, ++it) {
          const int sg = it % NST;
          ok = wait(codes + sg, (it / NST) & 1);
          if (!ok) break;
          if (!(i & 1)) {  // both scales have come with the keys
            scales[slot].keys[row] = spoil(scales[slot].keys[row]) * rs;
            float* value = scales[slot].values + row;
            float v = fabsf(*value);
            const bool bad = !(v < INFINITY);
            if (bad) *value = v = 0.f;
            scales[slot].logs[row] = scale_log(v);
            const float top = scale_log(__uint_as_float(__reduce_max_sync(FULL, __float_as_uint(v))));
            const uint32_t which = __ballot_sync(FULL, bad);
            if (lane == 0) scales[slot].top[warp - 8] = top, scales[slot].bad[warp - 8] = which;
            __syncwarp();
            if (lane == 0) mbar_arrive(sc_full + slot);
            if (++slot == NSC) slot = 0;
          }
          const auto meet = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(met);
            return wait(met, it & 1);
          };
          uint8_t* dst = ring + sg * C::tile_bytes;
          ok = i & 1 ? widen_row<Fp16, CODE, D>(dst, row, meet) : widen_row<T, CODE, D>(dst, row, meet);
          if (!ok) break;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(full + sg);
        }
      }
    }
  } else {  // ---- softmax of row tile s; thread = row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    const int s = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t st_addr = tmem + lane_base + s * 128, ot_addr = tmem + lane_base + C::o_col + s * D;
    const int tok = row / p.group;
    uint32_t sn = 0, on = 0, sc_phase = 0;
    int slot = 0;
    Unit u;
#pragma unroll 1
    for (int n = 0; take_unit(units, u, n, lane, wait); ++n) {
      const int nt = min(half_tokens, u.nt - s * half_tokens);
      if (nt <= 0) {  // the other row tile's alone
        for (slot += u.i1 - u.i0; slot >= NSC; slot -= NSC) sc_phase ^= 1;
        continue;
      }
      const bool whole = u.flags & kWhole;
      const int pa = u.p0 + s * half_tokens, pb = pa + nt - 1, pos = pa + tok;  // the row tile's positions, the row's
      // -m; the t + log2 |vs| from which the row needs another m: kRoom, or -inf before its first key
      float off = 0.f, limit = -INFINITY, sum0 = 0.f, sum1 = 0.f;
      bool ok = true;
#pragma unroll 1
      for (int i = u.i0; i < u.i1; ++i) {
        ok = wait(sc_full + slot, sc_phase);
        if (ok) ok = wait(s_full + s, sn & 1);
        ++sn;
        if (!ok) break;
        tc_fence_after();
        const TileScales& sc = scales[slot];
        const float *ks = sc.keys, *vs = sc.values;
        if (++slot == NSC) slot = 0, sc_phase ^= 1;
        const int j0 = u.tile(i) * kTileKeys;
        float x[128];
        COLI_LD32(st_addr, x);
        COLI_LD32(st_addr + 32, x + 32);
        COLI_LD32(st_addr + 64, x + 64);
        COLI_LD32(st_addr + 96, x + 96);
        float m0 = -INFINITY, m1 = m0, m2 = m0, m3 = m0;
        const bool masked = !all_see(p, pa, pb, j0, j0 + kTileKeys - 1);
        const int hi = pos - j0, lo = pos - p.window - j0, sk = p.sinks - j0;
        // the tile's largest log2 |vs|, and whether the row sees a value's scale that is not finite
        const float4 tops = *reinterpret_cast<const float4*>(sc.top);
        const uint4 bads = *reinterpret_cast<const uint4*>(sc.bad);
        const float lv = fmaxf(fmaxf(tops.x, tops.y), fmaxf(tops.z, tops.w));
        bool spoilt = (bads.x | bads.y | bads.z | bads.w) != 0;
        if (masked && spoilt) {
          spoilt = false;
#pragma unroll 1
          for (int c = 0; c < 128; c += 32)
            spoilt |= (sc.bad[c >> 5] & low_bits(hi + 1 - c) & (~low_bits(lo + 1 - c) | low_bits(sk - c))) != 0;
        }
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          COLI_LDWAIT32(x + c);
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            const float4 v = *reinterpret_cast<const float4*>(ks + c + k);
            float a = off, b = off, e = off, f = off;
            fma2_rn(x[c + k], x[c + k + 1], v.x, v.y, a, b);
            fma2_rn(x[c + k + 2], x[c + k + 3], v.z, v.w, e, f);
            x[c + k] = a, x[c + k + 1] = b, x[c + k + 2] = e, x[c + k + 3] = f;
          }
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
        if (spoilt) sum0 = NAN;
        const bool grow = top + lv > limit;
        if (__any_sync(FULL, grow)) {
          float u0 = -INFINITY, u1 = u0;  // the largest t + log2 |vs|
#pragma unroll
          for (int c = 0; c < 128; c += 4) {
            float4 l = *reinterpret_cast<const float4*>(sc.logs + c);
            add2_rn(x[c], x[c + 1], l.x, l.y);
            add2_rn(x[c + 2], x[c + 3], l.z, l.w);
            u0 = max3(u0, l.x, l.y);
            u1 = max3(u1, l.z, l.w);
          }
          float fix = 1.f, by = 0.f;  // by: added to the row's t
          if (fmaxf(u0, u1) > limit) {
            by = -fmaxf(u0, u1);
            if (limit == kRoom) fix = ex2(by);
            off += by, limit = kRoom;
            sum0 *= fix, sum1 *= fix;
          }
#pragma unroll
          for (int c = 0; c < 128; c += 2) add2_rn(by, by, x[c], x[c + 1]);
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
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            const float4 v = *reinterpret_cast<const float4*>(vs + c + 2 * k);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float e = ex2(x[c + 2 * (k + h)]), f = ex2(x[c + 2 * (k + h) + 1]);
              x[c + 2 * (k + h)] = e, x[c + 2 * (k + h) + 1] = f;
              mul2_rn(h ? v.z : v.x, h ? v.w : v.y, e, f);
              w[k + h] = Fp16::pack(e, f);
            }
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
      const float sum = sum0 + sum1, m2 = limit == -INFINITY ? -INFINITY : -off;
      const int token = u.tok0 + s * half_tokens + tok, hq = u.head * p.group + row - tok * p.group;
      const bool live = tok < nt;
      if (whole) {
        const float inv = sum == 0.f ? 0.f : Code<CODE>::unit / sum;
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
        const int64_t at =
            ((int64_t)blockIdx.x * 2 + (u.i0 > 0 ? 0 : 1)) * kTileRows + s * half_tokens * p.group + row;
        float* dst = p.part_o + at * D;
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
              for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(o[k + e] * Code<CODE>::unit);
              st_sector(dst + c + k, w);
            }
          }
        }
        if (live) p.part_ml[at] = make_float2(m2, sum);
      }
      tc_fence_before();  // the next unit's products overwrite O after this row tile's next arrival
    }
  }
  __syncthreads();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

template <class T, int CODE, int D>
cudaError_t launch(const AttnParams& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, int grid,
                   cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreadsQTile);
  cfg.dynamicSmemBytes = QTileCfg<D>::smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_qtile_kernel<T, CODE, D>, p, q, k, v);
}

template <class T, int CODE>
cudaError_t launch_dim(const AttnParams& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, int grid,
                       cudaStream_t stream) {
  return p.head_dim == 64 ? launch<T, CODE, 64>(p, q, k, v, grid, stream) : launch<T, CODE, 128>(p, q, k, v, grid, stream);
}

template <class T>
cudaError_t launch_code(const AttnParams& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, int code, int grid,
                        cudaStream_t stream) {
  return code == COLI_ATTN_CODE_INT8 ? launch_dim<T, COLI_ATTN_CODE_INT8>(p, q, k, v, grid, stream)
                                     : launch_dim<T, COLI_ATTN_CODE_E4M3>(p, q, k, v, grid, stream);
}

template <class T, int CODE, int D>
cudaError_t configure() {
  return cudaFuncSetAttribute(attn_qtile_kernel<T, CODE, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, QTileCfg<D>::smem);
}

}  // namespace

cudaError_t configure_attn_qtile() {
  cudaError_t e = cudaSuccess;
#define COLI_CFG(T, D)                                               \
  if (e == cudaSuccess) e = configure<T, COLI_ATTN_CODE_INT8, D>();  \
  if (e == cudaSuccess) e = configure<T, COLI_ATTN_CODE_E4M3, D>();
  COLI_CFG(Bf16, 64) COLI_CFG(Bf16, 128) COLI_CFG(Fp16, 64) COLI_CFG(Fp16, 128)
#undef COLI_CFG
  return e;
}

cudaError_t launch_attn_qtile(const AttnParams& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, int dtype,
                              int code, int num_sms, cudaStream_t stream) {
  return dtype == COLI_ATTN_BF16 ? launch_code<Bf16>(p, q, k, v, code, num_sms, stream)
                                 : launch_code<Fp16>(p, q, k, v, code, num_sms, stream);
}

}  // namespace coli

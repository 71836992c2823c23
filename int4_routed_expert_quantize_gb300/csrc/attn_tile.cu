// Attention of many query rows over a paged cache on the fifth-generation tensor cores.
//
// A block is 2 x 128 rows (tokens x query heads of one key head, whole tokens only).  For every tile
// of 128 keys S = Q K^T goes to tensor memory, a warpgroup per 128 rows (one thread a row, so neither
// maxima nor sums cross threads) turns it into P = 2^(scale S - m), written over S in 16 bits, and
// O += P V reads P from tensor memory and stays there.  The two row tiles alternate: while one's
// scores are in the softmax the other's products run, and the matrix unit is meant never to wait.
//
//   tensor memory (512 columns)   S0/P0 | S1/P1 | O0 | O1
//   shared memory                 Q0, Q1, a ring of key and a ring of value tiles, 128-byte swizzled boxes
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
#include "attn_device.cuh"

namespace coli {

namespace {

constexpr int kThreadsTile = 12 * 32;
constexpr int kTileSmemRing = 163840;

template <int D>
struct TileCfg {
  static constexpr int tile_bytes = kTileKeys * D * 2;  // K or V of one stage; Q of one row tile
  // Two rings, each with waiters that see every one of its tiles in order: with one ring for both, a
  // waiter for value tiles alone could meet a stage whose previous (key) tile is still on its way and take
  // the barrier's older phase for the one it wants.
  static constexpr int k_stages = 2 * (kTileSmemRing / 5 / tile_bytes);
  static constexpr int v_stages = 3 * (kTileSmemRing / 5 / tile_bytes);
  static constexpr int q_bytes = 2 * tile_bytes;
  // barriers: keys full/empty, values full/empty/checked, q full/empty, scores, weights, output, drain
  static constexpr int bars = 2 * k_stages + 3 * v_stages + 4 + 6 + 1;
  static constexpr int smem = kTileSmemRing + q_bytes + bars * 8 + 128;
  static constexpr uint32_t o_col = 256;  // first column of O0; O1 follows after D columns
};

#define COLI_LD32(taddr, r)                                                                          \
  asm volatile(                                                                                      \
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "                                                      \
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "                       \
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"       \
      : "=f"((r)[0]), "=f"((r)[1]), "=f"((r)[2]), "=f"((r)[3]), "=f"((r)[4]), "=f"((r)[5]),          \
        "=f"((r)[6]), "=f"((r)[7]), "=f"((r)[8]), "=f"((r)[9]), "=f"((r)[10]), "=f"((r)[11]),        \
        "=f"((r)[12]), "=f"((r)[13]), "=f"((r)[14]), "=f"((r)[15]), "=f"((r)[16]), "=f"((r)[17]),    \
        "=f"((r)[18]), "=f"((r)[19]), "=f"((r)[20]), "=f"((r)[21]), "=f"((r)[22]), "=f"((r)[23]),    \
        "=f"((r)[24]), "=f"((r)[25]), "=f"((r)[26]), "=f"((r)[27]), "=f"((r)[28]), "=f"((r)[29]),    \
        "=f"((r)[30]), "=f"((r)[31])                                                                 \
      : "r"(taddr)                                                                                   \
      : "memory")
// a wait that names 32 loaded registers, so that no use of them can move before it
#define COLI_LDWAIT32(r)                                                                             \
  asm volatile("tcgen05.wait::ld.sync.aligned;"                                                      \
               : "+f"((r)[0]), "+f"((r)[1]), "+f"((r)[2]), "+f"((r)[3]), "+f"((r)[4]), "+f"((r)[5]), \
                 "+f"((r)[6]), "+f"((r)[7]), "+f"((r)[8]), "+f"((r)[9]), "+f"((r)[10]),              \
                 "+f"((r)[11]), "+f"((r)[12]), "+f"((r)[13]), "+f"((r)[14]), "+f"((r)[15]),          \
                 "+f"((r)[16]), "+f"((r)[17]), "+f"((r)[18]), "+f"((r)[19]), "+f"((r)[20]),          \
                 "+f"((r)[21]), "+f"((r)[22]), "+f"((r)[23]), "+f"((r)[24]), "+f"((r)[25]),          \
                 "+f"((r)[26]), "+f"((r)[27]), "+f"((r)[28]), "+f"((r)[29]), "+f"((r)[30]),          \
                 "+f"((r)[31])                                                                       \
               :                                                                                     \
               : "memory")

#define COLI_ST32(taddr, r)                                                                          \
  asm volatile(                                                                                      \
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "                                                \
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "                     \
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr), \
      "f"((r)[0]), "f"((r)[1]), "f"((r)[2]), "f"((r)[3]), "f"((r)[4]), "f"((r)[5]), "f"((r)[6]),     \
      "f"((r)[7]), "f"((r)[8]), "f"((r)[9]), "f"((r)[10]), "f"((r)[11]), "f"((r)[12]), "f"((r)[13]), \
      "f"((r)[14]), "f"((r)[15]), "f"((r)[16]), "f"((r)[17]), "f"((r)[18]), "f"((r)[19]),            \
      "f"((r)[20]), "f"((r)[21]), "f"((r)[22]), "f"((r)[23]), "f"((r)[24]), "f"((r)[25]),            \
      "f"((r)[26]), "f"((r)[27]), "f"((r)[28]), "f"((r)[29]), "f"((r)[30]), "f"((r)[31])             \
      : "memory")

__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Instruction descriptor of kind::f16, fp32 accumulator, M = 128: A and B format 1 = bf16, 0 = fp16; bit
// 16: B is stored with N contiguous.
template <class T>
__device__ constexpr uint32_t mma_desc(int n, bool b_n_major) {
  constexpr uint32_t fmt = T::kExp == 0x7F807F80u ? 1u : 0u;
  return (1u << 4) | (fmt << 7) | (fmt << 10) | ((b_n_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         (8u << 24);
}

// Shared-memory descriptor of a value tile as the N-contiguous operand: boxes of 64 values (128 swizzled
// bytes) x 128 keys.  8 keys make one 1024-byte atom; the next 8 keys follow at 1024 bytes, the next 64
// values at one box (16 KB).  p = first key of the 16 that one MMA takes.
__device__ __forceinline__ uint64_t smem_desc_values(const void* p) {
  const uint64_t a = (smem_addr(p) >> 4) & 0x3FFFu;
  return a | ((uint64_t)((kTileKeys * 128) >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
         (2ull << 61);
}

// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1 : 0)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

// 32 bytes of a thread's row at once: a full sector per thread
__device__ __forceinline__ void st_sector(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

template <class T, int D>
__global__ void __launch_bounds__(kThreadsTile, 1)
    attn_tile_kernel(const AttnParams p, const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using C = TileCfg<D>;
  constexpr int KST = C::k_stages, VST = C::v_stages;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *kring = smem, *vring = smem + KST * C::tile_bytes;
  uint8_t* qs = smem + kTileSmemRing;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(qs + C::q_bytes);
  uint64_t *k_empty = k_full + KST, *v_full = k_empty + KST, *v_empty = v_full + VST, *checked = v_empty + VST,
           *q_full = checked + VST, *q_empty = q_full + 2,
           *s_full = q_empty + 2, *p_full = s_full + 2, *o_full = p_full + 2, *drain = o_full + 2;
  Stretch* stretch = reinterpret_cast<Stretch*>(drain + 1);
  int* abort_flag = reinterpret_cast<int*>(stretch + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(abort_flag + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    *abort_flag = 0;
    for (int i = 0; i < KST; ++i) mbar_init(k_full + i, 1), mbar_init(k_empty + i, 1);
    for (int i = 0; i < VST; ++i) mbar_init(v_full + i, 1), mbar_init(v_empty + i, 1), mbar_init(checked + i, 2);
    for (int s = 0; s < 2; ++s) {
      mbar_init(q_full + s, 1), mbar_init(q_empty + s, 1), mbar_init(s_full + s, 1);
      mbar_init(p_full + s, 4), mbar_init(o_full + s, 1);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
    prefetch_map(&qmap), prefetch_map(&kmap), prefetch_map(&vmap);
  }
  if (warp == 8) tmem_alloc(tmem_slot, 512);
  griddep_wait();
  griddep_launch_dependents();
  const Stretch st = schedule<kTileKeys>(p, reinterpret_cast<int64_t*>(smem), stretch);
  if (warp == 9 && lane == 0) write_record<kTileKeys>(p, st);
  fence_proxy_async_smem();  // the copies overwrite what schedule() kept in the rings
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int half_tokens = p.block_tokens / 2;  // tokens of one row tile

  Cursor<kTileKeys> cur;
  cur.start(p, st);
  // tokens of row tile s of the current unit
  const auto tokens = [&](const Cursor<kTileKeys>& c, int s) {
    return max(0, min(half_tokens, c.s.n - c.blk * p.block_tokens - s * half_tokens));
  };

  if (warp == 9) {  // ---- copies
    int it = 0, kt = 0, qn[2] = {0, 0};  // value, key and query tiles asked for
    bool ok = true;
    for (; cur.valid() && ok; cur.next(p)) {
      const int64_t row = (int64_t)cur.b * p.table_stride;
      const int tok0 = cur.s.start + cur.blk * p.block_tokens;
      const uint32_t qb = (uint32_t)(p.group * half_tokens) * D * 2;
      for (int s = 0; s < 2 && ok; ++s) {
        if (tokens(cur, s) == 0) continue;
        if (qn[s] > 0) ok = warp_wait(q_empty + s, (qn[s] - 1) & 1, abort_flag, p.status);
        if (!ok) break;
        ++qn[s];
        if (lane == 0) {
          mbar_expect_tx(q_full + s, qb);
          for (int sl = 0; sl < D / 64; ++sl)
            tma_load_3d(qs + s * C::tile_bytes + sl * kTileKeys * 128, &qmap, sl * 64, cur.head * p.group,
                        tok0 + s * half_tokens, q_full + s);
        }
        __syncwarp();
      }
      for (int i = cur.i0; i < cur.i1 && ok; ++i, ++it) {
        const int j0 = cur.t.tile(i) * kTileKeys;
        const uint32_t bytes = fill_bytes<kTileKeys, D>(p, cur.t.p0, cur.t.p1, j0, lane);
        const int ks = it % KST, vs = it % VST;
        if (it >= KST) ok = warp_wait(k_empty + ks, ((it / KST) + 1) & 1, abort_flag, p.status);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(k_full + ks, bytes);
        __syncwarp();
        fill_boxes<kTileKeys, D>(p, &kmap, kring + ks * C::tile_bytes, k_full + ks, row, cur.t.p0, cur.t.p1, j0,
                                 cur.head, lane);
        ++kt;
        if (it >= VST) ok = warp_wait(v_empty + vs, ((it / VST) + 1) & 1, abort_flag, p.status);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(v_full + vs, bytes);
        __syncwarp();
        fill_boxes<kTileKeys, D>(p, &vmap, vring + vs * C::tile_bytes, v_full + vs, row, cur.t.p0, cur.t.p1, j0,
                                 cur.head, lane);
      }
    }
    if (!ok) {
      drain_fills(k_full, KST, kt);
      drain_fills(v_full, VST, it);
      for (int s = 0; s < 2; ++s)
        if (qn[s] > 0) drain_fills(q_full + s, 1, qn[s]);
    }
  } else if (warp == 8) {  // ---- products (lane 0 issues; the warp waits together)
    constexpr uint32_t qk_desc = mma_desc<T>(kTileKeys, false), pv_desc = mma_desc<T>(D, true);
    Cursor<kTileKeys> nxt = cur;  // the unit and tile whose scores come next
    int ni = nxt.i0, nit = 0, qn[2] = {0, 0}, pn[2] = {0, 0};
    bool ok = true, more = nxt.valid();
    const auto scores = [&](int s) {  // S_s of tile ni of nxt; nit: its number
      if (tokens(nxt, s) == 0) return;
      if (ni == nxt.i0) {
        ok = ok && warp_wait(q_full + s, qn[s] & 1, abort_flag, p.status);
        ++qn[s];
      }
      const int sg = nit % KST;
      ok = ok && warp_wait(k_full + sg, (nit / KST) & 1, abort_flag, p.status);
      if (!ok) return;
      tc_fence_after();
      if (lane == 0) {
#pragma unroll 1
        for (int k = 0; k < D / 16; ++k) {
          const int off = (k >> 2) * kTileKeys * 128 + (k & 3) * 32;
          tc_mma_bf16(tmem + s * 128, smem_desc_sw128(qs + s * C::tile_bytes + off),
                      smem_desc_sw128(kring + sg * C::tile_bytes + off), qk_desc, k > 0);
        }
        tc_commit(s_full + s);
        if (ni == nxt.i1 - 1) tc_commit(q_empty + s);
      }
      __syncwarp();
    };
    const auto step = [&]() {  // nxt's key tile is done with
      if (lane == 0) tc_commit(k_empty + nit % KST);
      __syncwarp();
      ++nit;
      if (++ni == nxt.i1) {
        nxt.next(p);
        more = nxt.valid();
        ni = more ? nxt.i0 : 0;
      }
    };
    if (more) {
      scores(0), scores(1);
      if (ok) step();
    }
    int it = 0;
    for (; cur.valid() && ok; cur.next(p))
      for (int i = cur.i0; i < cur.i1 && ok; ++i, ++it) {
        const int sg = it % VST;
        for (int s = 0; s < 2 && ok; ++s) {
          if (tokens(cur, s) > 0) {
            ok = warp_wait(checked + sg, (it / VST) & 1, abort_flag, p.status) &&
                 warp_wait(p_full + s, pn[s] & 1, abort_flag, p.status);
            ++pn[s];
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll 1
              for (int k = 0; k < kTileKeys / 16; ++k)
                tc_mma_ts(tmem + C::o_col + s * D, tmem + s * 128 + k * 8,
                          smem_desc_values(vring + sg * C::tile_bytes + k * 2048), pv_desc, i > cur.i0 || k > 0);
              if (i == cur.i1 - 1) tc_commit(o_full + s);
            }
            __syncwarp();
          }
          if (more) scores(s);
        }
        if (!ok) break;
        if (lane == 0) tc_commit(v_empty + sg);
        __syncwarp();
        if (more) step();
      }
    if (!ok) {  // wait, with a limit of its own, for the products in flight
      if (lane == 0) tc_commit(drain);
      drain_fills(drain, 1, 1);
    }
  } else if (warp >= 10) {  // ---- values that not every row sees
    int it = 0;
    bool ok = true;
    for (; cur.valid() && ok; cur.next(p)) {
      bool listed = false;
      for (int i = cur.i0; i < cur.i1; ++i, ++it) {
        const int sg = it % VST;
        ok = warp_wait(v_full + sg, (it / VST) & 1, abort_flag, p.status);
        if (!ok) break;
        const int j0 = cur.t.tile(i) * kTileKeys;
        if (!all_see(p, cur.t.p0, cur.t.p1, j0, j0 + kTileKeys - 1)) {
          uint32_t bad = 0;
          // warp 10 takes the even keys, 11 the odd ones; 8 lanes a 128-byte row
          for (int r = (warp - 10) + (lane >> 3) * 2; r < kTileKeys; r += 8) {
            const bool some = some_sees(p, cur.t.p0, cur.t.p1, j0 + r);
            const bool all = all_see(p, cur.t.p0, cur.t.p1, j0 + r, j0 + r);
            if (all) continue;
#pragma unroll
            for (int sl = 0; sl < D / 64; ++sl) {
              uint4* v = reinterpret_cast<uint4*>(vring + sg * C::tile_bytes + sl * kTileKeys * 128 + r * 128) + (lane & 7);
              if (some) {
                const uint4 x = *v;
                bad |= nonfinite2<T>(x.x) | nonfinite2<T>(x.y) | nonfinite2<T>(x.z) | nonfinite2<T>(x.w);
              } else {
                *v = make_uint4(0, 0, 0, 0);
              }
            }
          }
          fence_proxy_async_smem();
          if (__any_sync(FULL, bad != 0) && !listed) {
            listed = true;
            if (lane == 0 && p.redo) {
              const int at = atomicAdd(p.redo_count, 1);
              if (at < p.redo_cap) p.redo[at] = make_int4(cur.b, cur.blk, cur.head, 0);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(checked + sg);
      }
    }
  } else {  // ---- softmax of row tile s; thread = row
    const int s = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t st_addr = tmem + lane_base + s * 128, ot_addr = tmem + lane_base + C::o_col + s * D;
    const int tok = row / p.group;
    const float slack = 8.f / p.scale_log2;
    int sn = 0, on = 0;
    bool ok = true;
    for (; cur.valid() && ok; cur.next(p)) {
      const int nt = tokens(cur, s);
      if (nt == 0) continue;
      const int pa = p.causal ? cur.t.p0 + s * half_tokens : cur.t.p0;  // the row tile's positions
      const int pb = p.causal ? pa + nt - 1 : pa;
      const int pos = p.causal ? pa + tok : pa;
      float ref = -INFINITY, sum0 = 0.f, sum1 = 0.f;
      for (int i = cur.i0; i < cur.i1; ++i) {
        ok = warp_wait(s_full + s, sn & 1, abort_flag, p.status);
        ++sn;
        if (!ok) break;
        tc_fence_after();
        const int j0 = cur.t.tile(i) * kTileKeys;
        const bool masked = !all_see(p, pa, pb, j0, j0 + kTileKeys - 1);
        const int hi = pos - j0, lo = pos - p.window - j0, sk = p.sinks - j0;
        // Scores are read twice, for the maximum and for the weights: holding all 128 would spill.
        float m0 = -INFINITY, m1 = m0, m2 = m0, m3 = m0;
        {
          float x[128];
          COLI_LD32(st_addr, x);
          COLI_LD32(st_addr + 32, x + 32);
          COLI_LD32(st_addr + 64, x + 64);
          COLI_LD32(st_addr + 96, x + 96);
          COLI_LDWAIT32(x);
          COLI_LDWAIT32(x + 32);
          COLI_LDWAIT32(x + 64);
          COLI_LDWAIT32(x + 96);
          if (masked) {
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (c > hi || (c <= lo && c >= sk)) x[c] = -INFINITY;
          }
#pragma unroll
          for (int c = 0; c < 128; c += 8) {
            m0 = fmaxf(m0, fmaxf(x[c], x[c + 1]));
            m1 = fmaxf(m1, fmaxf(x[c + 2], x[c + 3]));
            m2 = fmaxf(m2, fmaxf(x[c + 4], x[c + 5]));
            m3 = fmaxf(m3, fmaxf(x[c + 6], x[c + 7]));
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
          if (i > cur.i0 && __any_sync(FULL, fix != 1.f)) {
#pragma unroll
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
        float y[2][32];
        COLI_LD32(st_addr, y[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float* x = y[c & 1];
          COLI_LDWAIT32(x);
          if (c < 3) COLI_LD32(st_addr + 32 * (c + 1), y[(c + 1) & 1]);
          if (masked) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (c * 32 + k > hi || (c * 32 + k <= lo && c * 32 + k >= sk)) x[k] = -INFINITY;
          }
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float e = base, f = base;
            fma2_rn(x[2 * k], x[2 * k + 1], p.scale_log2, p.scale_log2, e, f);
            e = ex2(e), f = ex2(f);
            add2_rn(e, f, sum0, sum1);
            w[k] = T::pack(e, f);
          }
          tmem_st16u(st_addr + 16 * c, w);  // over scores that have been read
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + s);
      }
      if (!ok) break;
      ok = warp_wait(o_full + s, on & 1, abort_flag, p.status);
      ++on;
      if (!ok) break;
      tc_fence_after();
      const float sum = sum0 + sum1, m2 = ref * p.scale_log2;
      const int tok0 = cur.s.start + cur.blk * p.block_tokens + s * half_tokens;
      const int hq = cur.head * p.group + row - tok * p.group;
      const bool live = tok < nt;
      if (cur.whole() && !p.dense_o) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        uint16_t* dst = static_cast<uint16_t*>(p.out) + (int64_t)(tok0 + tok) * p.out_stride + (int64_t)hq * D;
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          float o[32];
          COLI_LD32(ot_addr + c, o);
          COLI_LDWAIT32(o);
          if (live) {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = T::pack(o[2 * k] * inv, o[2 * k + 1] * inv);
            st_sector(dst + c, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = T::pack(o[16 + 2 * k] * inv, o[17 + 2 * k] * inv);
            st_sector(dst + c + 16, w);
          }
        }
        if (live && p.lse)
          p.lse[(int64_t)(tok0 + tok) * p.n_q + hq] =
              sum == 0.f ? -INFINITY : (m2 + log2f(sum)) * 0.69314718055994530942f;
      } else {
        const bool dense = cur.whole();
        // a cut unit's rows, numbered over both row tiles: row tile 1 starts at half_tokens * group
        const int64_t at = dense ? (int64_t)(tok0 + tok) * p.n_q + hq
                                 : ((int64_t)blockIdx.x * 2 + (cur.first ? 0 : 1)) * kTileRows +
                                       s * half_tokens * p.group + row;
        float* dst = (dense ? p.dense_o : p.part_o) + at * D;
#pragma unroll
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
        if (live) (dense ? p.dense_ml : p.part_ml)[at] = make_float2(m2, sum);
      }
      tc_fence_before();  // the next unit's products overwrite O after this row tile's next arrival
    }
  }
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

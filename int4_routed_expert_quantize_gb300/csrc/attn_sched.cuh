// The work list of the attention kernels: which key tiles each block of queries needs, and which
// stretch of the list over all blocks a CTA takes.  Everything is read from the batch's
// device arrays, so the host knows no lengths.
#pragma once

#include "attn_internal.h"
#include "attn_stretch.h"
#include "coli_device.cuh"

namespace coli {

struct SeqInfo {
  int start, n, len;  // first query token, query tokens, cached tokens
  bool causal;        // false: the prefix, of which every query sees every key
};

// (past L1: a line read before the launch's inputs were final must not be met again)
__device__ __forceinline__ SeqInfo seq_info(const AttnParams& p, int b) {
  SeqInfo s;
  const bool own = b < p.n_seqs;
  s.causal = own;
  if (own) {
    const int a = __ldcg(p.q_start + b), e = __ldcg(p.q_start + b + 1);
    s.start = min(max(a, 0), p.n_tokens);
    s.n = min(max(e, s.start), p.n_tokens) - s.start;
  } else {
    s.start = 0;
    s.n = p.n_tokens;
  }
  const int64_t cap = (int64_t)(own ? p.max_pages : p.pre_pages) << p.page_shift;
  const int l = __ldcg(own ? p.kv_len + b : p.pre_len);
  s.len = max(l, 0);
  if (s.len > cap) s.len = (int)cap;
  return s;
}

__device__ __forceinline__ int n_lists(const AttnParams& p) { return p.n_seqs + (p.pre_len ? 1 : 0); }

// what seq_info clamps, and more new tokens than announced, is reported once per call
__device__ __forceinline__ void seq_check(const AttnParams& p, int b) {
  const bool own = b < p.n_seqs;
  const int l = __ldg(own ? p.kv_len + b : p.pre_len);
  bool bad = l < 0 || (int64_t)l > ((int64_t)(own ? p.max_pages : p.pre_pages) << p.page_shift);
  if (own) {
    const int a = __ldg(p.q_start + b), e = __ldg(p.q_start + b + 1);
    bad = bad || a < 0 || e < a || e > p.n_tokens || e - a > p.max_q || (b == 0 && a != 0) ||
          (b == p.n_seqs - 1 && e != p.n_tokens);
  }
  if (bad) atomicExch(p.status, COLI_EINVAL);
}

// The key tiles of one block of queries: tiles 0..sink-1, then `base`, base+1, ... (count in all, at
// least one so that every block writes its rows; a block that sees nothing gets a tile in which
// everything is masked).
template <int KT>
struct Tiles {
  int count, sink, base;
  int p0, p1;  // positions of the block's first and last query (causal), or the last key twice
  __device__ __forceinline__ void set(const AttnParams& p, const SeqInfo& s, int blk) {
    const int t0 = blk * p.block_tokens;
    const int nt = min(p.block_tokens, s.n - t0);
    p0 = s.causal ? s.len - s.n + t0 : s.len - 1;
    p1 = s.causal ? p0 + nt - 1 : s.len - 1;
    const int hi = p1 < 0 ? -1 : p1 / KT;
    const int lo = p.window >= kAttnNoWindow ? 0 : max(0, p0 - p.window + 1) / KT;
    sink = p.sinks > 0 ? min((p.sinks - 1) / KT, hi) + 1 : 0;
    if (lo <= sink) sink = 0, base = 0;
    else base = lo;
    count = max(1, sink + max(0, hi - base + 1));
  }
  __device__ __forceinline__ int tile(int i) const { return i < sink ? i : base + i - sink; }
};

// rows of a block see key j iff j <= p && (j > p - window || j < sinks)
__device__ __forceinline__ bool sees(const AttnParams& p, int pos, int j) {
  return j <= pos && (j > pos - p.window || j < p.sinks);
}
// some row of a block with positions p0..p1 sees key j
__device__ __forceinline__ bool some_sees(const AttnParams& p, int p0, int p1, int j) {
  return j <= p1 && (j > p0 - p.window || j < p.sinks);
}
// every row sees every key of [j0, j1]
__device__ __forceinline__ bool all_see(const AttnParams& p, int p0, int p1, int j0, int j1) {
  return j1 <= p0 && (j0 > p1 - p.window || j1 < p.sinks);
}

// ---- the list ----
// A unit is one block with one key head.  On the list it takes unit_cost positions (what it costs besides
// its tiles: queries in, results out) and then one position a tile; a CTA's stretch is `per` positions,
// and a tile belongs to the CTA whose stretch holds its position.  Order: sequences, blocks, key heads.

// One unit's tiles i0..i1-1, for the roles of a CTA.
struct alignas(16) Unit {
  int tok0, nt;      // first query token (of all), tokens
  int p0, p1;        // Tiles
  int sink, base;
  int i0, i1;        // i1 = 0: the end
  int head, b, blk;
  int flags;         // kWhole: all of its tiles (otherwise a part goes to slot (i0 > 0 ? 0 : 1) of the workspace)
  __device__ __forceinline__ int tile(int i) const { return i < sink ? i : base + i - sink; }
};
constexpr int kWhole = 1, kCausal = 2;  // Unit::flags
static_assert(sizeof(Unit) == 48, "three 16-byte words");

constexpr int kUnitSlots = 4;
struct UnitRing {  // one warp fills it, every warp of the other roles reads it
  Unit u[kUnitSlots];
  uint64_t full[kUnitSlots], empty[kUnitSlots];
  __device__ __forceinline__ void init(int readers) {
    for (int i = 0; i < kUnitSlots; ++i) mbar_init(full + i, 1), mbar_init(empty + i, readers);
  }
};

constexpr int kSerialBlocks = 4;

// Positions of each sequence into pos[b + 1] (shared memory; may overlay memory that is used only
// afterwards), by all threads of the CTA; the caller synchronises.
template <int KT>
__device__ __forceinline__ void weigh(const AttnParams& p, uint32_t* pos) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarps = blockDim.x >> 5;
  bool any_long = false;
#pragma unroll 1
  for (int b = tid; b < n_lists(p); b += blockDim.x) {
    const SeqInfo s = seq_info(p, b);
    if (blockIdx.x == 0) seq_check(p, b);
    uint32_t w = 0;
    const int nb = (s.n + p.block_tokens - 1) / p.block_tokens;
#pragma unroll 1
    for (int blk = 0; blk < nb && nb <= kSerialBlocks; ++blk) {
      Tiles<KT> t;
      t.set(p, s, blk);
      w += t.count + p.unit_cost;
    }
    any_long |= nb > kSerialBlocks;
    pos[b + 1] = nb > kSerialBlocks ? 0xFFFFFFFFu : w * p.n_kv;
  }
  if (!__syncthreads_or(any_long)) return;
#pragma unroll 1
  for (int b = warp; b < n_lists(p); b += nwarps) {  // long sequences: one warp over the blocks
    const uint32_t have = pos[b + 1];
    __syncwarp();
    if (have != 0xFFFFFFFFu) continue;
    const SeqInfo s = seq_info(p, b);
    const int nb = (s.n + p.block_tokens - 1) / p.block_tokens;
    uint32_t w = 0;
#pragma unroll 1
    for (int blk = lane; blk < nb; blk += 32) {
      Tiles<KT> t;
      t.set(p, s, blk);
      w += t.count + p.unit_cost;
    }
    w = __reduce_add_sync(FULL, w);
    if (lane == 0) pos[b + 1] = w * p.n_kv;
  }
  __syncthreads();
}

__device__ __forceinline__ uint32_t warp_scan(uint32_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(FULL, v, o);
    if (lane >= o) v = list_add(v, u);
  }
  return v;
}

// Walks a CTA's stretch; one warp, all lanes alike.
template <int KT>
struct Walk {
  SeqInfo s;
  Tiles<KT> t;
  uint32_t begin, end, per, at;  // at: the current unit's first position
  int b, blk, head;
  __device__ __forceinline__ void cut(const AttnParams& p, uint32_t run, int longest, bool real) {
    per = list_stretch(run, gridDim.x, longest);
    if (run == kListFull) {  // no place is known: nothing is computed, and the joining kernel finds every row in one piece
      if (blockIdx.x == 0 && (threadIdx.x & 31) == 0 && real) atomicExch(p.status, COLI_EINVAL);
      run = 0, per = 0xFFFFFFFFu;
    }
    begin = min(blockIdx.x * per, run);
    end = min(begin + per, run);
    b = blk = head = 0;
    at = end;  // nothing to do
  }
  // More than 32 sequences: pos as weigh() left it; becomes their first positions.
  __device__ __forceinline__ void start(const AttnParams& p, uint32_t* pos, int lane) {
    const int ns = n_lists(p);
    uint32_t run = 0;
    if (lane == 0) pos[0] = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < ns; b0 += 32) {
      const uint32_t v = warp_scan(b0 + lane < ns ? pos[b0 + lane + 1] : 0, lane);
      if (b0 + lane < ns) pos[b0 + lane + 1] = list_add(run, v);
      run = list_add(run, __shfl_sync(FULL, v, 31));
    }
    __syncwarp();
    cut(p, run, 0, true);
    if (blockIdx.x == 0 && p.seq_pos) {
#pragma unroll 1
      for (int i = lane; i <= ns; i += 32) p.seq_pos[i] = pos[i];
      if (lane == 0) p.seq_pos[ns + 1] = per;
    }
    if (begin >= end) return;
    int hi = ns - 1;  // the sequence with pos[b] <= begin < pos[b+1]
#pragma unroll 1
    while (b < hi) {
      const int mid = (b + hi + 1) >> 1;
      if (pos[mid] <= begin) b = mid;
      else hi = mid - 1;
    }
    s = seq_info(p, b);
    find_block(p, pos[b], lane);
  }
  // Up to 32 sequences: one a lane, nothing through shared memory, and the other warps need not wait.  It is run twice:
  // first (real = false) while the launches before this one still run, on whatever the lengths are then and with
  // nothing written, so that its instructions are in the caches when its inputs are final.  us with start() for all / this:
  // one token 9.8 / 9.4, 13 sequences of 5 14.3 / 13.5, 4 answers behind 7036 tokens 22.2 / 15.0.
  __device__ __forceinline__ void start_few(const AttnParams& p, int lane, bool real) {
    const int ns = n_lists(p);
    SeqInfo mine = {0, 0, 0, true};
    if (lane < ns) {
      mine = seq_info(p, lane);
      if (blockIdx.x == 0 && real) seq_check(p, lane);
    }
    const int nb = (mine.n + p.block_tokens - 1) / p.block_tokens;
    uint32_t w = 0;
    int longest = 0;
#pragma unroll 1
    for (int i = 0; i < nb && nb <= kSerialBlocks; ++i) {
      Tiles<KT> x;
      x.set(p, mine, i);
      w += x.count + p.unit_cost;
      if (KT == kSplitKeys) longest = x.count;
    }
    unsigned many = __ballot_sync(FULL, nb > kSerialBlocks);
#pragma unroll 1
    for (; many; many &= many - 1) {
      const int l = __ffs(many) - 1;
      take_lane(mine, l);
      const int n = __shfl_sync(FULL, nb, l);
      uint32_t sum = 0;
#pragma unroll 1
      for (int i = lane; i < n; i += 32) {
        Tiles<KT> x;
        x.set(p, s, i);
        sum += x.count + p.unit_cost;
      }
      sum = __reduce_add_sync(FULL, sum);
      if (lane == l) w = sum;
    }
    w *= p.n_kv;
    const uint32_t v = warp_scan(w, lane);
    cut(p, __shfl_sync(FULL, v, 31), __reduce_max_sync(FULL, longest), real);
    if (blockIdx.x == 0 && p.seq_pos && real) {
      if (lane <= ns && lane < 31) p.seq_pos[lane] = v - w;
      if (lane == 31) p.seq_pos[31] = v - w, p.seq_pos[32] = v;
      __syncwarp();
      if (lane == 0) p.seq_pos[ns + 1] = per;
    }
    if (begin >= end) return;
    b = __ffs(__ballot_sync(FULL, begin < v)) - 1;
    take_lane(mine, b);
    find_block(p, __shfl_sync(FULL, v - w, b), lane);
  }
  __device__ __forceinline__ void take_lane(const SeqInfo& mine, int l) {
    s.start = __shfl_sync(FULL, mine.start, l);
    s.n = __shfl_sync(FULL, mine.n, l);
    s.len = __shfl_sync(FULL, mine.len, l);
    s.causal = __shfl_sync(FULL, (int)mine.causal, l);
  }
  // the block and key head at `begin` in sequence b, whose first position is `first`
  __device__ __forceinline__ void find_block(const AttnParams& p, uint32_t first, int lane) {
    at = first;
    const int nb = (s.n + p.block_tokens - 1) / p.block_tokens;
#pragma unroll 1
    for (int blk0 = 0; blk0 < nb && nb > 1; blk0 += 32) {
      uint32_t w = 0;
      if (blk0 + lane < nb) {
        t.set(p, s, blk0 + lane);
        w = (t.count + p.unit_cost) * p.n_kv;
      }
      const uint32_t v = warp_scan(w, lane);
      const unsigned in = __ballot_sync(FULL, begin < at + v);
      if (in) {
        const int l = __ffs(in) - 1;
        blk = blk0 + l;
        at += __shfl_sync(FULL, v - w, l);
        break;
      }
      at += __shfl_sync(FULL, v, 31);
    }
    t.set(p, s, blk);
    const uint32_t cost = t.count + p.unit_cost;
    head = (begin - at) / cost;
    at += head * cost;
  }
  // the next unit of which a tile belongs to this CTA; false at the end
  __device__ __forceinline__ bool next(const AttnParams& p, Unit& u) {
    while (at < end) {
      const int first = at + p.unit_cost;  // the first tile's position
      u.i0 = max(0, (int)begin - first);
      u.i1 = min(t.count, (int)end - first);
      u.head = head, u.b = b, u.blk = blk;
      u.p0 = t.p0, u.p1 = t.p1, u.sink = t.sink, u.base = t.base;
      u.tok0 = s.start + blk * p.block_tokens;
      u.nt = min(p.block_tokens, s.n - blk * p.block_tokens);
      u.flags = (u.i0 == 0 && u.i1 == t.count ? kWhole : 0) | (s.causal ? kCausal : 0);
      const uint32_t here = at;
      at += t.count + p.unit_cost;
      if (++head == p.n_kv && at < end) {
        head = 0;
        if (++blk * p.block_tokens >= s.n) {
          blk = 0;
#pragma unroll 1
          do {
            ++b;
            s = seq_info(p, b);
          } while (s.n == 0);  // a later sequence has tokens: the stretch ends inside the list
        }
        t.set(p, s, blk);
      }
      if (u.i1 > u.i0) {
        if (u.i0 > 0) record(p, u, here + p.unit_cost, at - here - p.unit_cost);
        return true;
      }
    }
    return false;
  }
  // a unit whose first part is the previous CTA's: the combine kernel learns of it from here
  __device__ __forceinline__ void record(const AttnParams& p, const Unit& u, uint32_t first, uint32_t count) const {
    const int c0 = first / per;
    if (c0 + 1 != (int)blockIdx.x || (threadIdx.x & 31) != 0) return;
    AttnRec r;
    r.first_cta = c0, r.last_cta = (first + count - 1) / per;
    r.token0 = u.tok0, r.tokens = u.nt, r.head = u.head;
    p.rec[blockIdx.x] = r;
  }
};

// A block in which a value that is not finite met rows that do not see it: its rows are computed again, one by one,
// by the kernel that joins the parts (0 * inf = NaN has spoilt them here).
__device__ __forceinline__ void flag_unit(const AttnParams& p, const Unit& u, int lane) {
#pragma unroll 1
  for (int i = lane; i < u.nt; i += 32) p.redo[(int64_t)(u.tok0 + i) * p.n_kv + u.head] = 1;
  if (lane == 0) atomicExch(p.redo_any, 1);
}

// The copying warp hands unit u (number n of the CTA) to the other roles; false: a wait gave up.
template <class Wait>
__device__ __forceinline__ bool give_unit(UnitRing* r, const Unit& u, int n, int lane, Wait wait) {
  const int slot = n % kUnitSlots;
  if (n >= kUnitSlots && !wait(r->empty + slot, (n / kUnitSlots + 1) & 1)) return false;
  if (lane == 0) {
    const int4* src = reinterpret_cast<const int4*>(&u);
    int4* dst = reinterpret_cast<int4*>(r->u + slot);
    dst[0] = src[0], dst[1] = src[1], dst[2] = src[2];
    mbar_arrive(r->full + slot);
  }
  __syncwarp();
  return true;
}
// A warp of another role takes its n-th unit; false: the end, or a wait gave up.
template <class Wait>
__device__ __forceinline__ bool take_unit(UnitRing* r, Unit& u, int n, int lane, Wait wait) {
  const int slot = n % kUnitSlots;
  if (!wait(r->full + slot, (n / kUnitSlots) & 1)) return false;
  int4* dst = reinterpret_cast<int4*>(&u);
  const int4* src = reinterpret_cast<const int4*>(r->u + slot);
  dst[0] = src[0], dst[1] = src[1], dst[2] = src[2];
  __syncwarp();
  if (lane == 0) mbar_arrive(r->empty + slot);
  return u.i1 > 0;
}

}  // namespace coli

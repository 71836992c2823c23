// The work list of the attention kernels: which key tiles each block of queries needs, and which
// stretch of the list over all blocks a CTA takes.  Everything is read from the batch's
// device arrays, so the host knows no lengths.
#pragma once

#include "attn_internal.h"
#include "coli_device.cuh"

namespace coli {

struct SeqInfo {
  int start, n, len;  // first query token, query tokens, cached tokens
};

__device__ __forceinline__ SeqInfo seq_info(const AttnParams& p, int b) {
  SeqInfo s;
  if (p.q_start) {
    const int a = __ldg(p.q_start + b), e = __ldg(p.q_start + b + 1);
    s.start = min(max(a, 0), p.n_tokens);
    s.n = min(max(e, s.start), p.n_tokens) - s.start;
    const int64_t rows = (int64_t)s.n * p.group;
    if (rows <= p.rows_lo || rows > p.rows_hi) s.n = 0;
  } else {
    s.start = 0;
    s.n = p.n_tokens;
  }
  const int64_t cap = (int64_t)p.max_pages << p.page_shift;
  const int l = __ldg(p.kv_len + b);
  s.len = max(l, 0);
  if (s.len > cap) s.len = (int)cap;
  return s;
}

// what seq_info clamps is reported once per call
__device__ __forceinline__ void seq_check(const AttnParams& p, int b) {
  const int l = __ldg(p.kv_len + b);
  bool bad = l < 0 || (int64_t)l > ((int64_t)p.max_pages << p.page_shift);
  if (p.q_start) {
    const int a = __ldg(p.q_start + b), e = __ldg(p.q_start + b + 1);
    bad = bad || a < 0 || e < a || e > p.n_tokens || (b == 0 && a != 0);
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
    p0 = p.causal ? s.len - s.n + t0 : s.len - 1;
    p1 = p.causal ? p0 + nt - 1 : s.len - 1;
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

// list positions of one sequence: blocks in order, each block's key heads in order
template <int KT>
__device__ __forceinline__ int64_t seq_weight_serial(const AttnParams& p, const SeqInfo& s) {
  int64_t w = 0;
  const int nb = (s.n + p.block_tokens - 1) / p.block_tokens;
  for (int blk = 0; blk < nb; ++blk) {
    Tiles<KT> t;
    t.set(p, s, blk);
    w += t.count;
  }
  return w * p.n_kv;
}

struct Stretch {
  int64_t begin, end, per, total;
  int b, blk, head, off;  // the unit at `begin` and the tile within it
};

constexpr int kSchedSerialBlocks = 4;

// All threads of the CTA take part.  pos: shared, [n_seqs + 1] (may overlay memory that is used
// only afterwards).  Returns this CTA's stretch; CTA 0 also writes the list positions to
// the workspace (p.seq_pos).
template <int KT>
__device__ Stretch schedule(const AttnParams& p, int64_t* pos, Stretch* shared_out) {
  const int nthreads = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nwarps = nthreads >> 5;
  for (int b = tid; b < p.n_seqs; b += nthreads) {
    const SeqInfo s = seq_info(p, b);
    if (blockIdx.x == 0) seq_check(p, b);
    const int nb = (s.n + p.block_tokens - 1) / p.block_tokens;
    pos[b + 1] = nb <= kSchedSerialBlocks ? seq_weight_serial<KT>(p, s) : -1;
  }
  __syncthreads();
  for (int b = warp; b < p.n_seqs; b += nwarps) {  // long sequences: one warp over the blocks
    if (pos[b + 1] >= 0) continue;
    const SeqInfo s = seq_info(p, b);
    const int nb = (s.n + p.block_tokens - 1) / p.block_tokens;
    int64_t w = 0;
    for (int blk = lane; blk < nb; blk += 32) {
      Tiles<KT> t;
      t.set(p, s, blk);
      w += t.count;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) w += __shfl_xor_sync(FULL, w, o);
    __syncwarp();
    if (lane == 0) pos[b + 1] = w * p.n_kv;
  }
  __syncthreads();
  if (warp == 0) {
    int64_t run = 0;
    for (int b0 = 0; b0 < p.n_seqs; b0 += 32) {
      int64_t v = b0 + lane < p.n_seqs ? pos[b0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(FULL, v, o);
        if (lane >= o) v += u;
      }
      if (b0 + lane < p.n_seqs) pos[b0 + lane + 1] = run + v;
      run += __shfl_sync(FULL, v, 31);
    }
    if (lane == 0) pos[0] = 0;
    __syncwarp();
    Stretch st;
    st.total = run;
    st.per = max((int64_t)1, (run + gridDim.x - 1) / gridDim.x);
    st.begin = min((int64_t)blockIdx.x * st.per, run);
    st.end = min(st.begin + st.per, run);
    st.b = st.blk = st.head = st.off = 0;
    if (st.begin < st.end) {
      int lo = 0, hi = p.n_seqs - 1;  // the sequence with pos[b] <= begin < pos[b+1]
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pos[mid] <= st.begin) lo = mid;
        else hi = mid - 1;
      }
      st.b = lo;
      int64_t x = st.begin - pos[lo];
      const SeqInfo s = seq_info(p, lo);
      const int nb = (s.n + p.block_tokens - 1) / p.block_tokens;
      for (int blk0 = 0; blk0 < nb; blk0 += 32) {
        Tiles<KT> t;
        int64_t w = 0;
        if (blk0 + lane < nb) {
          t.set(p, s, blk0 + lane);
          w = (int64_t)t.count * p.n_kv;
        }
        int64_t v = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t u = __shfl_up_sync(FULL, v, o);
          if (lane >= o) v += u;
        }
        const unsigned in = __ballot_sync(FULL, x < v);
        if (in) {
          const int l = __ffs(in) - 1;
          st.blk = blk0 + l;
          x -= __shfl_sync(FULL, v - w, l);
          const int cnt = __shfl_sync(FULL, (int)(w / p.n_kv), l);
          st.head = (int)(x / cnt);
          st.off = (int)(x % cnt);
          break;
        }
        x -= __shfl_sync(FULL, v, 31);
      }
    }
    if (lane == 0) *shared_out = st;
    if (blockIdx.x == 0) {
      for (int b = lane; b <= p.n_seqs; b += 32) p.seq_pos[b] = pos[b];
      if (lane == 0) p.seq_pos[p.n_seqs + 1] = st.per;
    }
  }
  __syncthreads();
  return *shared_out;
}

// Walks the units of a stretch; every role of a CTA runs its own copy.
template <int KT>
struct Cursor {
  SeqInfo s;
  Tiles<KT> t;
  int b, blk, head, i0, i1;  // tiles i0..i1-1 of the unit are this CTA's
  int64_t pos, end;
  bool first;
  __device__ __forceinline__ void start(const AttnParams& p, const Stretch& st) {
    b = st.b, blk = st.blk, head = st.head, i0 = st.off;
    pos = st.begin, end = st.end;
    first = true;
    if (pos < end) {
      s = seq_info(p, b);
      t.set(p, s, blk);
      i1 = (int)min((int64_t)t.count, i0 + (end - pos));
    }
  }
  __device__ __forceinline__ bool valid() const { return pos < end; }
  __device__ __forceinline__ bool whole() const { return i0 == 0 && i1 == t.count; }
  __device__ __forceinline__ void next(const AttnParams& p) {
    pos += i1 - i0;
    first = false;
    if (pos >= end) return;
    i0 = 0;
    if (++head == p.n_kv) {
      head = 0;
      const int nb = (s.n + p.block_tokens - 1) / p.block_tokens;
      if (++blk >= nb) {
        blk = 0;
        do {
          ++b;
          s = seq_info(p, b);
        } while (s.n == 0);  // a later sequence has tokens: the stretch ends inside the list
      }
      t.set(p, s, blk);
    }
    i1 = (int)min((int64_t)t.count, end - pos);
  }
};

// The record of a CTA: filled when its stretch starts inside a unit whose first part lies in
// the previous CTA's stretch.
template <int KT>
__device__ __forceinline__ void write_record(const AttnParams& p, const Stretch& st) {
  AttnRec r;
  r.first_cta = -1;
  r.last_cta = r.first_slot = r.token0 = r.tokens = r.head = 0;
  r.seq = r.blk = 0;
  if (st.begin < st.end && st.off > 0 && st.off <= st.per) {
    Cursor<KT> c;
    c.start(p, st);
    const int64_t unit = st.begin - st.off;
    r.first_cta = blockIdx.x - 1;
    r.first_slot = unit == st.begin - st.per ? 0 : 1;
    r.last_cta = (int)((unit + c.t.count - 1) / st.per);
    r.token0 = c.s.start + c.blk * p.block_tokens;
    r.tokens = min(p.block_tokens, c.s.n - c.blk * p.block_tokens);
    r.head = c.head, r.seq = c.b, r.blk = c.blk;
  }
  p.rec[blockIdx.x] = r;
}

}  // namespace coli

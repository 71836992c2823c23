// Joins partial attention results of the same query rows:
//   m = max m_i,  o = sum 2^(m_i - m) o_i / sum 2^(m_i - m) l_i
// with o_i unnormalised, m_i the partial's maximum in log2 units and l_i its sum.  Parts are added in
// the order of the keys, so equal calls give equal bits.  The parts of few rows are read by a warp a row, the (m, l)
// pairs one per lane and the outputs two or four values per lane; of many rows by a warp for four rows, where every load is a
// whole line.  The kernels are bound by the latency of their L2 reads: after the last part is written, 3 to 5 us of a
// small call pass before the output is (record, parts, join, store), so every address is worked out while the launch
// before still runs, and as many parts are on their way as registers allow.
#include "attn_device.cuh"

namespace coli {

namespace {

constexpr int kWarps = 4;
// Parts on their way: more hide more of the L2's latency, and cost registers, so warps.  A row's parts are many where the
// split kernel has few rows, so there a warp takes one row with 16 of its parts on their way; elsewhere four rows with 4 each
// (combine), or one with 8 (join).
// Combine, us, one row a warp / four, after the split kernel: one token 9.4 / 9.8, one sequence of 5 new tokens (240 rows)
// 17.4 / 18.9, 8 of 4 (1536 rows) 13.9 / 13.0; after the tensor-memory kernel: one of 16 (768 rows) 19.7 / 18.1, 8 of 32
// 56.3 / 49.3.  Join, 16 / 8 on their way: 32 chats 37.0 / 34.6, 64 sequences behind 2000 tokens 32.5 / 30.1, 256 286 / 276;
// after the split kernel alone, 24 rows a key head: 14.1 / 14.9.
constexpr int64_t kSmallCombine = 1024;  // rows (tokens x heads) after the split kernel up to which a warp takes one

// one part of a row: its unnormalised output, and its maximum and sum
struct Part {
  const float* o;
  const float2* ml;
};

// running join of one row over a warp; lane holds D/32 consecutive values
template <int D, int Loads>
struct Join {
  static constexpr int V = D / 32;
  static constexpr int kLoads = Loads;  // parts in flight
  float m = -INFINITY, l = 0.f, o[V];
  __device__ __forceinline__ Join() {
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = 0.f;
  }
  template <class At>
  static __device__ __forceinline__ void load(float (&v)[kLoads][V], int c, int n, int lane, At at) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[j][i] = 0.f;
      if (j < n) {
        const float* src = at(c + j).o + lane * V;
        if constexpr (V == 4) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(src));
          v[j][0] = x.x, v[j][1] = x.y, v[j][2] = x.z, v[j][3] = x.w;
        } else {
          const float2 x = __ldcg(reinterpret_cast<const float2*>(src));
          v[j][0] = x.x, v[j][1] = x.y;
        }
      }
    }
  }
  // parts at(0..n-1)
  template <class At>
  __device__ __forceinline__ void add(int n, int lane, At at) {
#pragma unroll 1
    for (int c = 0; c < n; c += 32) {
      const int k = min(32, n - c);
      float first[kLoads][V];  // asked for before the weights are known
      load(first, c, k, lane, at);
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < k) ml = __ldcg(at(c + lane).ml);
      float top = fmaxf(m, warp_max(ml.x));
      const float base = top == -INFINITY ? 0.f : top;
      const float keep = ex2(m - base);
      const float w = ml.y == 0.f ? 0.f : ex2(ml.x - base);  // a NaN sum stays
      float add_l = w * ml.y;
#pragma unroll
      for (int s = 16; s; s >>= 1) add_l += __shfl_xor_sync(FULL, add_l, s);
      l = l * keep + add_l;
      m = top;
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] *= keep;
#pragma unroll 1
      for (int j0 = 0; j0 < k; j0 += kLoads) {
        if (j0 > 0) load(first, c + j0, k - j0, lane, at);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
          const float wj = __shfl_sync(FULL, w, j0 + j);  // 0 past the end, and for a part without keys
          if (wj != 0.f)
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = fmaf(wj, first[j][i], o[i]);
        }
      }
    }
  }
  template <class T>
  __device__ __forceinline__ void write(const AttnParams& p, int token, int hq, int lane) const {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + (int64_t)token * p.out_stride +
                                                (int64_t)hq * D) +
                    lane * (V / 2);
#pragma unroll
    for (int i = 0; i < V; i += 2) dst[i / 2] = T::pack(o[i] * inv, o[i + 1] * inv);
    if (p.lse && lane == 0)
      p.lse[(int64_t)token * p.n_q + hq] =
          l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
  }
};

// Adds one query row's attention to its own cache, from the definition, by one warp: for the rare blocks with
// values that are not finite and that only some of the block's rows see.  qf: D floats of shared memory.
template <class T, int D, class J>
__device__ __noinline__ void add_direct(J& r, const AttnParams& p, const SeqInfo& s, int b, int i, int hq,
                                        float* qf, int lane) {
  constexpr int V = D / 32;
  const int pos = s.len - s.n + i, head = hq / p.group;
  const uint16_t* q = static_cast<const uint16_t*>(p.q) + (int64_t)(s.start + i) * p.q_stride + (int64_t)hq * D;
  __syncwarp();
  for (int d = lane * 2; d < D; d += 64) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(q + d);
    qf[d] = T::lo(v), qf[d + 1] = T::hi(v);
  }
  __syncwarp();
  const int lo = p.window >= kAttnNoWindow ? 0 : max(0, pos - p.window + 1);
  const auto slot = [&](const void* base, int64_t sp, int64_t sh, int64_t ss, int j) -> const uint16_t* {
    const int id = __ldg(p.table + (int64_t)b * p.table_stride + (j >> p.page_shift));
    if (id < 0 || id >= p.n_pages) return nullptr;  // reads as zeros
    return static_cast<const uint16_t*>(base) + id * sp + head * sh + (j & ((1 << p.page_shift) - 1)) * ss;
  };
  for (int j0 = 0; j0 <= pos; j0 += 32) {
    if (j0 >= p.sinks && j0 + 31 < lo) {
      j0 = (lo & ~31) - 32;
      continue;
    }
    const int j = j0 + lane;
    float x = -INFINITY;
    if (sees(p, pos, j)) {
      const uint16_t* k = slot(p.kc, p.k_page, p.k_head, p.k_slot, j);
      x = 0.f;
      for (int d = 0; k && d < D; d += 2) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(k + d);
        x = fmaf(qf[d], T::lo(v), fmaf(qf[d + 1], T::hi(v), x));
      }
      x *= p.scale_log2;
    }
    const float top = fmaxf(r.m, warp_max(x)), base = top == -INFINITY ? 0.f : top;
    const float keep = ex2(r.m - base), w = ex2(x - base);
    float sum = w;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
    r.l = r.l * keep + sum;
    r.m = top;
#pragma unroll
    for (int e = 0; e < V; ++e) r.o[e] *= keep;
    for (int n = 0; n < 32; ++n) {
      if (!sees(p, pos, j0 + n)) continue;
      const float wn = __shfl_sync(FULL, w, n);
      const uint16_t* v = slot(p.vc, p.v_page, p.v_head, p.v_slot, j0 + n);
      if (!v) continue;
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        const uint32_t y = *reinterpret_cast<const uint32_t*>(v + lane * V + e);
        r.o[e] = fmaf(wn, T::lo(y), r.o[e]), r.o[e + 1] = fmaf(wn, T::hi(y), r.o[e + 1]);
      }
    }
  }
}

// the sequence of a token: the first one that ends after it (n_seqs: none)
__device__ __forceinline__ int seq_of(const AttnParams& p, int token, int lane) {
  int b = 0;
  for (int b0 = 0; b0 < p.n_seqs; b0 += 32) {
    const bool before = b0 + lane < p.n_seqs && __ldg(p.q_start + b0 + lane + 1) <= token;
    const int n = __popc(__ballot_sync(FULL, before));
    b += n;
    if (n < 32) break;
  }
  return b;
}

// the last block to get here clears the flags for the next call
__device__ __noinline__ void clear_flags(const AttnParams& p) {
  __shared__ int last;
  __syncthreads();  // this block has read what it needs
  if (threadIdx.x == 0) last = atomicAdd(p.redo_any + 1, 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  for (int64_t k = threadIdx.x; k < (int64_t)p.n_tokens * p.n_kv; k += blockDim.x) p.redo[k] = 0;
  if (threadIdx.x == 0) p.redo_any[0] = p.redo_any[1] = 0;
}

// Four rows of one cut unit by one warp, eight lanes a row, each with a running maximum and sum of its own: nothing crosses
// lanes, and every load is a whole line.  A lane holds columns 32 k + 4 (lane % 8) .. + 3.
template <class T, int D>
__device__ __forceinline__ void join_four(const AttnParams& p, int rows, const AttnRec& r, int row, int lane) {
  constexpr int K = D / 32, kAtOnce = 4;
  const int tok = row / p.group, n = r.last_cta - r.first_cta + 1, lane8 = lane & 7;
  if (tok >= r.tokens) return;
  float m = -INFINITY, sum = 0.f;
  float4 o[K];
#pragma unroll
  for (int k = 0; k < K; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int c = 0; c < n; c += kAtOnce) {
    float4 v[kAtOnce][K];
    float2 ml[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      ml[j] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int k = 0; k < K; ++k) v[j][k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c + j < n) {
        const int64_t at = ((int64_t)(r.first_cta + c + j) * 2 + (c + j == 0 ? 1 : 0)) * rows + row;
        ml[j] = __ldcg(p.part_ml + at);
#pragma unroll
        for (int k = 0; k < K; ++k) v[j][k] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * D) + k * 8 + lane8);
      }
    }
    float top = m;
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) top = fmaxf(top, ml[j].x);
    const float ref = top == -INFINITY ? 0.f : top, keep = ex2(m - ref);
    m = top;
    sum *= keep;
#pragma unroll
    for (int k = 0; k < K; ++k) o[k].x *= keep, o[k].y *= keep, o[k].z *= keep, o[k].w *= keep;
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      if (ml[j].y == 0.f) continue;  // no part, or one without keys; a NaN sum stays
      const float w = ex2(ml[j].x - ref);
      sum = fmaf(w, ml[j].y, sum);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        o[k].x = fmaf(w, v[j][k].x, o[k].x), o[k].y = fmaf(w, v[j][k].y, o[k].y);
        o[k].z = fmaf(w, v[j][k].z, o[k].z), o[k].w = fmaf(w, v[j][k].w, o[k].w);
      }
    }
  }
  const int token = r.token0 + tok, hq = r.head * p.group + row - tok * p.group;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (int64_t)token * p.out_stride + (int64_t)hq * D);
#pragma unroll
  for (int k = 0; k < K; ++k)
    dst[k * 8 + lane8] = make_uint2(T::pack(o[k].x * inv, o[k].y * inv), T::pack(o[k].z * inv, o[k].w * inv));
  if (p.lse && lane8 == 0)
    p.lse[(int64_t)token * p.n_q + hq] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.69314718055994530942f;
}

// SMALL: a warp a row; otherwise four rows a warp
template <class T, int D, bool SMALL>
__global__ void __launch_bounds__(kWarps * 32) attn_combine_kernel(const AttnParams p, int rows, int ctas, int block_rows) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const AttnRec r = p.rec[blockIdx.x % ctas];
  const bool redo = __ldcg(p.redo_any) != 0;
  if (r.first_cta >= 0 && !(redo && __ldcg(p.redo + (int64_t)r.token0 * p.n_kv + r.head)))
    for (int i = SMALL ? warp : warp * 4 + (lane >> 3); i < block_rows; i += SMALL ? kWarps : kWarps * 4) {
      const int row = blockIdx.x / ctas * block_rows + i;
      if (!SMALL) {
        join_four<T, D>(p, rows, r, row, lane);
        continue;
      }
      const int tok = row / p.group;
      if (tok >= r.tokens) break;
      Join<D, 16> j;
      j.add(r.last_cta - r.first_cta + 1, lane, [&](int c) {
        const int64_t at = ((int64_t)(r.first_cta + c) * 2 + (c == 0 ? 1 : 0)) * rows + row;
        return Part{p.part_o + at * D, p.part_ml + at};
      });
      j.template write<T>(p, r.token0 + tok, r.head * p.group + row - tok * p.group, lane);
    }
  if (!redo) return;
  __shared__ float qf[kWarps][D];
  for (int64_t k = (int64_t)blockIdx.x * kWarps + warp; k < (int64_t)p.n_tokens * p.n_kv;
       k += (int64_t)gridDim.x * kWarps) {
    if (!__ldcg(p.redo + k)) continue;
    const int token = (int)(k / p.n_kv), b = seq_of(p, token, lane);
    if (b >= p.n_seqs) continue;  // (only where the offsets do not ascend, which is reported)
    const SeqInfo s = seq_info(p, b);
    const int i = token - s.start;
    if (i < 0 || i >= s.n) continue;  // (likewise: its position would lie outside the sequence's pages)
    for (int g = 0; g < p.group; ++g) {
      Join<D, 4> j;
      const int hq = (int)(k % p.n_kv) * p.group + g;
      add_direct<T, D>(j, p, s, b, i, hq, qf[warp], lane);
      j.template write<T>(p, token, hq, lane);
    }
  }
  clear_flags(p);
}

// where one row's results of one source are
struct Parts {
  int n;       // parts; dense: the row sits in the dense buffer
  bool dense;
  int first_cta, rows, row;
};

// Where token i of a sequence is on the list, from the sequence's first position on: the first tile of its unit, the
// unit's tiles and the row within its block.
struct Place {
  uint32_t first;
  int tiles, row;
};
template <int KT>
__device__ __forceinline__ Place find_place(const AttnParams& p, const SeqInfo& s, int i, int head, int g) {
  const int blk = i / p.block_tokens;
  Tiles<KT> t;
  Place r;
  r.first = 0;
  if (s.causal) {
#pragma unroll 1
    for (int k = 0; k < blk; ++k) {
      t.set(p, s, k);
      r.first += (t.count + p.unit_cost) * p.n_kv;
    }
    t.set(p, s, blk);
  } else {  // every block has the same tiles
    t.set(p, s, blk);
    r.first = blk * (t.count + p.unit_cost) * p.n_kv;
  }
  r.first += head * (t.count + p.unit_cost) + p.unit_cost;
  r.tiles = t.count;
  r.row = (i - blk * p.block_tokens) * p.group + g;
  return r;
}
// its parts, once the sequence's first position and the stretch are known
__device__ __forceinline__ Parts find_parts(const Place& w, int rows, uint32_t at, uint32_t per) {
  Parts r;
  r.row = w.row;
  r.rows = rows;
  at += w.first;
  const int c0 = at / per, c1 = (at + w.tiles - 1) / per;
  r.dense = c0 == c1;
  r.n = c1 - c0 + 1;
  r.first_cta = c0;
  return r;
}

// part c of them; which: own (0) or prefix (1), for the dense buffer
template <int D>
__device__ __forceinline__ Part part_of(const AttnParams& p, const Parts& r, int which, int64_t dense_row, int c) {
  if (r.dense) return Part{p.dense_o[which] + dense_row * D, p.dense_ml[which] + dense_row};
  const int64_t at = ((int64_t)(r.first_cta + c) * 2 + (c == 0 ? 1 : 0)) * r.rows + r.row;
  return Part{p.part_o + at * D, p.part_ml + at};
}

// Every row is the join of its own sequence's parts and the prefix's, which one launch with KT-key tiles has made, or (KT = 0)
// two: the split kernel's for the sequences, the tensor-memory kernel's for the prefix.  Rows are looked up while those run
// (they had waited for whatever wrote the lengths).
template <class T, int D, int KT, int Loads>
__global__ void __launch_bounds__(kWarps * 32)
    attn_join_kernel(const AttnParams own, int own_rows, const AttnParams shared, int shared_ctas) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const bool live = row < (int64_t)own.n_tokens * own.n_q;
  const int token = live ? (int)(row / own.n_q) : 0, hq = live ? (int)(row - (int64_t)token * own.n_q) : 0;
  const int head = hq / own.group, g = hq - head * own.group;
  const int b = seq_of(own, token, lane);
  const SeqInfo pre = seq_info(shared, shared.n_seqs);
  SeqInfo s = {0, 0, 0, true};
  if (b < own.n_seqs) s = seq_info(own, b);
  const int i = token - s.start;
  const bool has_own = i >= 0 && i < s.n;
  const Place far = find_place<KT ? KT : kTileKeys>(shared, pre, token, head, g);
  Place near = {0, 1, 0};
  if (has_own) near = find_place<KT ? KT : kSplitKeys>(own, s, i, head, g);
  uint32_t far_per = 1;
  if (!KT) {  // the prefix alone on its list: the stretch follows from its length
    const uint32_t blocks = (pre.n + shared.block_tokens - 1) / shared.block_tokens;
    const uint32_t total = blocks * shared.n_kv * (far.tiles + shared.unit_cost);
    far_per = list_stretch(total, shared_ctas, 0);
  }
  griddep_wait();
  griddep_launch_dependents();
  const bool redo = __ldcg(own.redo_any) != 0;
  const uint32_t per = __ldcg(own.seq_pos + n_lists(own) + 1), near_at = has_own ? __ldcg(own.seq_pos + b) : 0;
  const uint32_t far_at = KT ? __ldcg(own.seq_pos + own.n_seqs) : 0;
  Join<D, Loads> j;
  if (live) {
    const Parts f = KT ? find_parts(far, own_rows, far_at, per) : find_parts(far, kTileRows, 0, far_per);
    Parts e = find_parts(near, own_rows, near_at, per);
    if (!has_own) e.n = 0;
    if (redo && has_own && __ldcg(own.redo + (int64_t)token * own.n_kv + head)) {
      __shared__ float qf[kWarps][D];
      add_direct<T, D>(j, own, s, b, i, hq, qf[threadIdx.x >> 5], lane);
      e.n = 0;
    }
    j.add(f.n + e.n, lane,
          [&](int c) { return c < f.n ? part_of<D>(shared, f, 1, row, c) : part_of<D>(own, e, 0, row, c - f.n); });
    j.template write<T>(own, token, hq, lane);
  }
  if (redo) clear_flags(own);
}

template <class K, class... A>
cudaError_t go(K kernel, dim3 grid, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <class T, int D>
cudaError_t join(const AttnParams& own, int own_rows, const AttnParams& shared, bool same, int shared_ctas,
                 cudaStream_t stream) {
  const dim3 grid((unsigned)(((int64_t)own.n_tokens * own.n_q + kWarps - 1) / kWarps));
  const auto kernel = !same                     ? attn_join_kernel<T, D, 0, 8>
                      : own_rows == kTileRows ? attn_join_kernel<T, D, kTileKeys, 8>
                                              : attn_join_kernel<T, D, kSplitKeys, 16>;
  return go(kernel, grid, stream, own, own_rows, shared, shared_ctas);
}

template <class T, int D>
cudaError_t combine(const AttnParams& p, int rows, int live, int ctas, cudaStream_t stream) {
  const bool small = rows <= kSplitMaxRows && (int64_t)p.n_tokens * p.n_q <= kSmallCombine;
  const int block_rows = small ? 4 : 16;
  const dim3 grid(ctas * ((live + block_rows - 1) / block_rows));
  return small ? go(attn_combine_kernel<T, D, true>, grid, stream, p, rows, ctas, block_rows)
               : go(attn_combine_kernel<T, D, false>, grid, stream, p, rows, ctas, block_rows);
}

}  // namespace

cudaError_t launch_attn_combine(const AttnParams& p, int rows, int live, int ctas, int dtype, cudaStream_t stream) {
  if (dtype == COLI_ATTN_BF16)
    return p.head_dim == 64 ? combine<Bf16, 64>(p, rows, live, ctas, stream) : combine<Bf16, 128>(p, rows, live, ctas, stream);
  return p.head_dim == 64 ? combine<Fp16, 64>(p, rows, live, ctas, stream) : combine<Fp16, 128>(p, rows, live, ctas, stream);
}

cudaError_t launch_attn_join(const AttnParams& own, int own_rows, const AttnParams& shared, bool same_list,
                             int shared_ctas, int dtype, cudaStream_t stream) {
  if (dtype == COLI_ATTN_BF16)
    return own.head_dim == 64 ? join<Bf16, 64>(own, own_rows, shared, same_list, shared_ctas, stream)
                              : join<Bf16, 128>(own, own_rows, shared, same_list, shared_ctas, stream);
  return own.head_dim == 64 ? join<Fp16, 64>(own, own_rows, shared, same_list, shared_ctas, stream)
                            : join<Fp16, 128>(own, own_rows, shared, same_list, shared_ctas, stream);
}

}  // namespace coli

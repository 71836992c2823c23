// Joins partial attention results of the same query rows:
//   m = max m_i,  o = sum 2^(m_i - m) o_i / sum 2^(m_i - m) l_i
// with o_i unnormalised, m_i the partial's maximum in log2 units and l_i its sum.  Parts are added in
// the order of the keys, so equal calls give equal bits.  One warp takes one row: the parts'
// (m, l) pairs are read one per lane, the outputs four values per lane.  The kernels are bound by the
// L2 reads of the parts.
#include "attn_device.cuh"

namespace coli {

namespace {

constexpr int kWarps = 4;

// running join of one row over a warp; lane holds D/32 consecutive values
template <int D>
struct Join {
  static constexpr int V = D / 32;
  float m = -INFINITY, l = 0.f, o[V];
  __device__ __forceinline__ Join() {
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = 0.f;
  }
  // parts i = 0..n-1 of the row at o_base + at(i) * D, ml_base[at(i)]
  template <class At>
  __device__ __forceinline__ void add(const float* ob, const float2* mlb, int n, int lane, At at) {
    for (int c = 0; c < n; c += 32) {
      const int k = min(32, n - c);
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < k) ml = __ldcg(mlb + at(c + lane));
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
#pragma unroll 4
      for (int j = 0; j < k; ++j) {
        const float wj = __shfl_sync(FULL, w, j);
        const float* src = ob + at(c + j) * D + lane * V;
        float v[V];
        if constexpr (V == 4) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(src));
          v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        } else {
          const float2 x = __ldcg(reinterpret_cast<const float2*>(src));
          v[0] = x.x, v[1] = x.y;
        }
        if (wj != 0.f)  // a part without keys holds zeros
#pragma unroll
          for (int i = 0; i < V; ++i) o[i] = fmaf(wj, v[i], o[i]);
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
template <class T, int D>
__device__ __noinline__ void add_direct(Join<D>& r, const AttnParams& p, const SeqInfo& s, int b, int i, int hq,
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
  if (threadIdx.x == 0) last = atomicAdd(p.redo_any + 1, 1) == (int)(gridDim.x * gridDim.y) - 1;
  __syncthreads();
  if (!last) return;
  for (int64_t k = threadIdx.x; k < (int64_t)p.n_tokens * p.n_kv; k += blockDim.x) p.redo[k] = 0;
  if (threadIdx.x == 0) p.redo_any[0] = p.redo_any[1] = 0;
}

template <class T, int D>
__device__ __forceinline__ void join_parts(const AttnParams& p, const AttnRec& r, int rows, int rows_per_block,
                                           int warp, int lane) {
  for (int i = warp; i < rows_per_block; i += kWarps) {
    const int row = blockIdx.y * rows_per_block + i;
    const int tok = row / p.group;
    if (tok >= r.tokens) break;
    Join<D> j;
    j.add(p.part_o, p.part_ml, r.last_cta - r.first_cta + 1, lane, [&](int c) {
      return ((int64_t)(r.first_cta + c) * 2 + (c == 0 ? 1 : 0)) * rows + row;
    });
    j.template write<T>(p, r.token0 + tok, r.head * p.group + row - tok * p.group, lane);
  }
}

template <class T, int D>
__global__ void __launch_bounds__(kWarps * 32)
    attn_combine_kernel(const AttnParams p, int rows, int rows_per_block) {
  griddep_wait();
  griddep_launch_dependents();
  const AttnRec r = p.rec[blockIdx.x];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool redo = __ldcg(p.redo_any) != 0;
  if (r.first_cta >= 0 && !(redo && __ldcg(p.redo + (int64_t)r.token0 * p.n_kv + r.head)))
    join_parts<T, D>(p, r, rows, rows_per_block, warp, lane);
  if (!redo) return;
  __shared__ float qf[kWarps][D];
  const int64_t stride = (int64_t)gridDim.x * gridDim.y * kWarps;
  for (int64_t k = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kWarps + warp; k < (int64_t)p.n_tokens * p.n_kv;
       k += stride) {
    if (!__ldcg(p.redo + k)) continue;
    const int token = (int)(k / p.n_kv), b = seq_of(p, token, lane);
    const SeqInfo s = seq_info(p, b);
    for (int g = 0; g < p.group; ++g) {
      Join<D> j;
      const int hq = (int)(k % p.n_kv) * p.group + g;
      add_direct<T, D>(j, p, s, b, token - s.start, hq, qf[warp], lane);
      j.template write<T>(p, token, hq, lane);
    }
  }
  clear_flags(p);
}

// where one row's results of one source are
struct Parts {
  int n;        // parts; 1 with dense: the row sits in the dense buffer
  bool dense;
  int first_cta, rows, row;
};

template <int KT>
__device__ __forceinline__ Parts find_parts(const AttnParams& p, int rows, int b, int i, int head, int g) {
  // token i of sequence b
  const SeqInfo s = seq_info(p, b);
  const uint32_t per = __ldcg(p.seq_pos + p.n_seqs + 1);
  const int blk = i / p.block_tokens;
  uint32_t at = __ldcg(p.seq_pos + b);
  Tiles<KT> t;
  if (p.causal) {
#pragma unroll 1
    for (int k = 0; k < blk; ++k) {
      t.set(p, s, k);
      at += (t.count + p.unit_cost) * p.n_kv;
    }
    t.set(p, s, blk);
  } else {  // every block has the same tiles
    t.set(p, s, blk);
    at += blk * (t.count + p.unit_cost) * p.n_kv;
  }
  at += head * (t.count + p.unit_cost) + p.unit_cost;
  Parts r;
  r.row = (i - blk * p.block_tokens) * p.group + g;
  r.rows = rows;
  const int c0 = at / per, c1 = (at + t.count - 1) / per;
  r.dense = c0 == c1;
  r.n = c1 - c0 + 1;
  r.first_cta = c0;
  return r;
}

template <int D>
__device__ __forceinline__ void add_parts(Join<D>& j, const AttnParams& p, const Parts& r, int64_t dense_row,
                                          int lane) {
  if (r.dense)
    j.add(p.dense_o, p.dense_ml, 1, lane, [&](int) { return dense_row; });
  else
    j.add(p.part_o, p.part_ml, r.n, lane, [&](int c) {
      return ((int64_t)(r.first_cta + c) * 2 + (c == 0 ? 1 : 0)) * r.rows + r.row;
    });
}

template <class T, int D, int OWN, int SHARED>
__device__ __forceinline__ void join_row(const AttnParams& own, int own_rows, const AttnParams& shared, int shared_rows,
                                         int64_t row, int lane, bool redo) {
  const int token = (int)(row / own.n_q), hq = (int)(row - (int64_t)token * own.n_q);
  const int head = hq / own.group, g = hq - head * own.group;
  Join<D> j;
  add_parts(j, shared, find_parts<SHARED>(shared, shared_rows, 0, token, head, g), row, lane);
  const int b = seq_of(own, token, lane);
  if (b < own.n_seqs) {
    const SeqInfo s = seq_info(own, b);
    const int i = token - s.start;
    if (i >= 0 && i < s.n) {
      if (redo && __ldcg(own.redo + (int64_t)token * own.n_kv + head)) {
        __shared__ float qf[kWarps][D];
        add_direct<T, D>(j, own, s, b, i, hq, qf[threadIdx.x >> 5], lane);
      } else {
        add_parts(j, own, find_parts<OWN>(own, own_rows, b, i, head, g), row, lane);
      }
    }
  }
  j.template write<T>(own, token, hq, lane);
}

template <class T, int D, int OWN, int SHARED>
__global__ void __launch_bounds__(kWarps * 32)
    attn_join_kernel(const AttnParams own, int own_rows, const AttnParams shared, int shared_rows) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const bool redo = __ldcg(own.redo_any) != 0;
  if (row < (int64_t)own.n_tokens * own.n_q) join_row<T, D, OWN, SHARED>(own, own_rows, shared, shared_rows, row, lane, redo);
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
cudaError_t join(const AttnParams& own, int own_rows, const AttnParams& shared, int shared_rows, int ot,
                 int st, cudaStream_t stream) {
  const dim3 grid((unsigned)(((int64_t)own.n_tokens * own.n_q + kWarps - 1) / kWarps));
  if (ot == kSplitKeys && st == kSplitKeys)
    return go(attn_join_kernel<T, D, kSplitKeys, kSplitKeys>, grid, stream, own, own_rows, shared, shared_rows);
  if (ot == kSplitKeys && st == kTileKeys)
    return go(attn_join_kernel<T, D, kSplitKeys, kTileKeys>, grid, stream, own, own_rows, shared, shared_rows);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_attn_combine(const AttnParams& p, int rows, int ctas, int dtype, cudaStream_t stream) {
  const int rpb = rows >= 64 ? 16 : 4;
  const dim3 grid(ctas, rows / rpb);
  if (dtype == COLI_ATTN_BF16)
    return p.head_dim == 64 ? go(attn_combine_kernel<Bf16, 64>, grid, stream, p, rows, rpb)
                            : go(attn_combine_kernel<Bf16, 128>, grid, stream, p, rows, rpb);
  return p.head_dim == 64 ? go(attn_combine_kernel<Fp16, 64>, grid, stream, p, rows, rpb)
                          : go(attn_combine_kernel<Fp16, 128>, grid, stream, p, rows, rpb);
}

cudaError_t launch_attn_join(const AttnParams& own, int own_rows, const AttnParams& shared,
                             int shared_rows, int own_tile, int shared_tile, int dtype,
                             cudaStream_t stream) {
  if (dtype == COLI_ATTN_BF16)
    return own.head_dim == 64 ? join<Bf16, 64>(own, own_rows, shared, shared_rows, own_tile, shared_tile, stream)
                              : join<Bf16, 128>(own, own_rows, shared, shared_rows, own_tile, shared_tile, stream);
  return own.head_dim == 64 ? join<Fp16, 64>(own, own_rows, shared, shared_rows, own_tile, shared_tile, stream)
                            : join<Fp16, 128>(own, own_rows, shared, shared_rows, own_tile, shared_tile, stream);
}

}  // namespace coli

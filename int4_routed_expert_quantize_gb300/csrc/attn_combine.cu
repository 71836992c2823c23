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

template <class T, int D>
__global__ void __launch_bounds__(kWarps * 32)
    attn_combine_kernel(const AttnParams p, int rows, int rows_per_block) {
  griddep_wait();
  griddep_launch_dependents();
  const AttnRec r = p.rec[blockIdx.x];
  if (r.first_cta < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = warp; i < rows_per_block; i += kWarps) {
    const int row = blockIdx.y * rows_per_block + i;
    const int tok = row / p.group;
    if (tok >= r.tokens) break;
    Join<D> j;
    j.add(p.part_o, p.part_ml, r.last_cta - r.first_cta + 1, lane, [&](int c) {
      return ((int64_t)(r.first_cta + c) * 2 + (c == 0 ? r.first_slot : 0)) * rows + row;
    });
    j.template write<T>(p, r.token0 + tok, r.head * p.group + row - tok * p.group, lane);
  }
}

// where one row's results of one source are
struct Parts {
  int n;        // parts; 1 with dense: the row sits in the dense buffer
  bool dense;
  int first_cta, first_slot, rows, row;
};

template <int KT>
__device__ __forceinline__ Parts find_parts(const AttnParams& p, int rows, int b, int i, int head, int g) {
  // token i of sequence b
  const SeqInfo s = seq_info(p, b);
  const int64_t per = __ldcg(p.seq_pos + p.n_seqs + 1);
  const int blk = i / p.block_tokens;
  int64_t at = __ldcg(p.seq_pos + b);
  Tiles<KT> t;
  if (p.causal) {
    for (int k = 0; k < blk; ++k) {
      t.set(p, s, k);
      at += (int64_t)t.count * p.n_kv;
    }
    t.set(p, s, blk);
  } else {  // every block has the same tiles
    t.set(p, s, blk);
    at += (int64_t)blk * t.count * p.n_kv;
  }
  at += (int64_t)head * t.count;
  Parts r;
  r.row = (i - blk * p.block_tokens) * p.group + g;
  r.rows = rows;
  const int64_t c0 = at / per, c1 = (at + t.count - 1) / per;
  r.dense = c0 == c1;
  r.n = (int)(c1 - c0) + 1;
  r.first_cta = (int)c0;
  r.first_slot = at == c0 * per ? 0 : 1;
  return r;
}

template <int D>
__device__ __forceinline__ void add_parts(Join<D>& j, const AttnParams& p, const Parts& r, int64_t dense_row,
                                          int lane) {
  if (r.dense)
    j.add(p.dense_o, p.dense_ml, 1, lane, [&](int) { return dense_row; });
  else
    j.add(p.part_o, p.part_ml, r.n, lane, [&](int c) {
      return ((int64_t)(r.first_cta + c) * 2 + (c == 0 ? r.first_slot : 0)) * r.rows + r.row;
    });
}

template <class T, int D, int OWN, int SHARED>
__global__ void __launch_bounds__(kWarps * 32)
    attn_join_kernel(const AttnParams own, int own_rows, const AttnParams shared, int shared_rows) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= (int64_t)own.n_tokens * own.n_q) return;
  const int token = (int)(row / own.n_q), hq = (int)(row - (int64_t)token * own.n_q);
  const int head = hq / own.group, g = hq - head * own.group;
  Join<D> j;
  add_parts(j, shared, find_parts<SHARED>(shared, shared_rows, 0, token, head, g), row, lane);
  int b = 0;  // the first sequence that ends after the token
  for (int b0 = 0; b0 < own.n_seqs; b0 += 32) {
    const bool before = b0 + lane < own.n_seqs && __ldg(own.q_start + b0 + lane + 1) <= token;
    const int n = __popc(__ballot_sync(FULL, before));
    b += n;
    if (n < 32) break;
  }
  if (b < own.n_seqs) {
    const SeqInfo s = seq_info(own, b);
    const int i = token - s.start;
    if (i >= 0 && i < s.n)
      add_parts(j, own, find_parts<OWN>(own, own_rows, b, i, head, g), row, lane);
  }
  j.template write<T>(own, token, hq, lane);
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

// Pieces the paged attention kernels share: the mask of a query, the key
// tiles a range of queries walks, and the stream-K split of a ragged batch.
#pragma once

#include "paged.cuh"
#include "ptx.cuh"

namespace rc {

// Keys [lo, hi) and, under a window, [0, sink_tok) within hi.
struct RowMask {
  int lo, hi;
};

// at: the query's position (negative: it sees nothing); L: tokens in the pages.
__device__ __forceinline__ RowMask row_mask(const MaskView& m, int at, int L) {
  if (at < 0) return RowMask{0, 0};
  const int f = m.frame == 1 ? at : at / m.frame;
  const int lo = m.window > 0 && f >= m.window ? (f - m.window + 1) * m.frame : 0;
  return RowMask{lo, min(L, (f + 1) * m.frame)};
}

// The key tiles (TK keys each, tile k = keys [k TK, k TK + TK)) that queries
// at positions [first, last] walk: those of the sinks, then those from the
// first window start to the last query's end.
template <int TK>
struct TileSpan {
  int n_sink, from, n;
  int lo_min, hi_max;  // some query sees: [lo_min, hi_max) and the sinks below hi_max
  int lo_max, hi_min;  // every query sees: [lo_max, hi_min) and the sinks below hi_min
  __device__ __forceinline__ void init(const MaskView& m, int first, int last, int L) {
    const RowMask a = row_mask(m, first, L), b = row_mask(m, last, L);
    lo_min = a.lo;
    lo_max = b.lo;
    hi_min = a.hi;
    hi_max = b.hi;
    const int n_end = (hi_max + TK - 1) / TK;
    n_sink = 0;
    from = 0;
    if (m.window > 0) {
      n_sink = min((m.sink_tok + TK - 1) / TK, n_end);
      from = max(n_sink, lo_min / TK);
    }
    n = n_sink + max(0, n_end - from);
  }
  __device__ __forceinline__ int key(int j) const { return (j < n_sink ? j : from + j - n_sink) * TK; }
};

// One sequence of the batch, with whatever the device arrays hold brought
// into range: rows [q0, q0 + n) of q, L tokens in the pages. `bad` says that
// something was out of range. Where cu_q descends (`falls`), rows could be
// claimed many times over and the sums of the split pass 32 bits: the
// attention kernels then do nothing but record it.
struct Seq {
  int q0, n, L;
  bool bad, falls;
};

__device__ __forceinline__ Seq load_seq(const BatchView& v, int n_tok, int b) {
  const int a = __ldg(v.cu_q + b), e = __ldg(v.cu_q + b + 1), l = __ldg(v.kv_len + b);
  Seq s;
  s.q0 = min(max(a, 0), n_tok);
  s.n = min(max(e - s.q0, 0), n_tok - s.q0);
  s.L = min(max(l, 0), v.max_pages << v.page_log2);
  s.falls = e < a;
  s.bad = s.falls || s.q0 != a || e - a != s.n || s.L != l || (b == 0 && a != 0);
  return s;
}

// What a CTA's range of tiles left in the partial rows. Slot 2c holds the part
// of the unit its range begins inside (x: kHasHead if there is one, kHeadEnds if
// that unit ends in the range); slot 2c + 1 the first part of a unit that begins
// in the range and goes on in the next CTA's: rows [y, y + z) of q (z 0: there
// is none) and query heads from w on.
using PartRecord = int4;
constexpr int kHasHead = 1, kHeadEnds = 2;

// Exclusive prefix sums of f(0..n-1) into pre[0..n] (shared memory), by all
// threads of the block.
template <int THREADS, typename T, typename Fn>
__device__ __forceinline__ void block_prefix(T* pre, int n, T* warp_sums, Fn f) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (n + THREADS - 1) / THREADS;
  const int i0 = min(tid * per, n), i1 = min(i0 + per, n);
  T sum = 0;
  for (int i = i0; i < i1; ++i) {
    const T w = f(i);
    pre[i] = sum;
    sum += w;
  }
  T inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  T base = inc - sum;
  for (int w = 0; w < warp; ++w) base += warp_sums[w];
  for (int i = i0; i < i1; ++i) pre[i] += base;
  if (i0 < i1 && i1 == n) pre[n] = base + sum;
  if (n == 0 && tid == 0) pre[0] = 0;
  __syncthreads();
}

// Launches a kernel of an attention call; chained: as a programmatic dependent
// of the call's kernel before it, so that its start overlaps that one's end. Such a
// kernel calls grid_wait before it reads or overwrites what that one wrote, and before its last block ends.
template <typename Params>
inline cudaError_t launch_chained(void (*kernel)(const Params), const Params& p, dim3 grid, int threads, size_t smem,
                                  bool chained, cudaStream_t s, int cluster = 1) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2]{};
  if (chained) {
    at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    at[cfg.numAttrs++].val.clusterDim = {(unsigned)cluster, 1, 1};
  }
  cfg.attrs = at;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// A row's sum of exponentials over some keys, sum_j 2^(c x_j) = y 2^(c x) with the raw score x of its running maximum
// (-inf: it has none; y is then 0, or NaN of NaN scores) and c = scale_log2. Apart, because their one
// logarithm c x + log2 y, in fp32, loses y and even the differences of scores where c x is large: two parts are
// weighed by 2^(c (x1 - x2)), whose difference is taken between the scores themselves.
using RowSum = float2;

__device__ __forceinline__ float row_lse2(RowSum s, float c) { return s.y == 0.f ? -INFINITY : s.x * c + log2f(s.y); }

// Where a row's result goes, and what it is merged with (PagedAttnParams' fields).
struct RowOutput {
  uint8_t* out;
  long long tok_stride, head_stride;  // bytes
  float* lse;
  const float* prev_o;
  const RowSum* prev_sum;
  float* pre_o;
  RowSum* pre_sum;
  int n_tok, heads;
  float c;
};

__device__ __forceinline__ RowOutput row_output(const PagedAttnParams& p) {
  return RowOutput{p.out.data, p.out.tok_stride, p.out.head_stride, p.lse,   p.prev_o,   p.prev_sum,
                   p.pre_o,    p.pre_sum,        p.n_tok,           p.Hk * p.G, p.scale_log2};
}

// Merges 8 columns of a row (divided by its sum) with the same row's result over the shared prefix.
template <int D>
__device__ __forceinline__ void merge_prev(const RowOutput& p, int tok, int head, int col, float (&acc)[8],
                                           RowSum& sum) {
  const RowSum ps = __ldcg(p.prev_sum + (size_t)head * p.n_tok + tok);
  const float m = fmaxf(sum.x, ps.x), ref = m == -INFINITY ? 0.f : m;
  const float4* src = reinterpret_cast<const float4*>(p.prev_o + ((size_t)tok * p.heads + head) * D + col);
  const float4 a = __ldcg(src), b = __ldcg(src + 1);
  const float w = sum.y * ptx::ex2((sum.x - ref) * p.c), wp = ps.y * ptx::ex2((ps.x - ref) * p.c), l = w + wp;
  const float inv = l == 0.f ? 0.f : 1.f / l;  // neither side saw a key: both are zeros
  const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = (acc[k] * w + x[k] * wp) * inv;
  sum = make_float2(m, l);
}

// The last write of 8 columns of a row: the output, or the prefix pass's fp32 result.
template <int D, bool BF16>
__device__ __forceinline__ void store_row(const RowOutput& p, int tok, int head, int col, const float (&acc)[8],
                                          RowSum sum) {
  if (p.pre_o) {
    float4* dst = reinterpret_cast<float4*>(p.pre_o + ((size_t)tok * p.heads + head) * D + col);
    dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    if (col == 0) p.pre_sum[(size_t)head * p.n_tok + tok] = sum;
    return;
  }
  uint4 u;
  u.x = ptx::pack16x2<BF16>(acc[0], acc[1]);
  u.y = ptx::pack16x2<BF16>(acc[2], acc[3]);
  u.z = ptx::pack16x2<BF16>(acc[4], acc[5]);
  u.w = ptx::pack16x2<BF16>(acc[6], acc[7]);
  *reinterpret_cast<uint4*>(p.out + tok * p.tok_stride + head * p.head_stride + col * 2) = u;
  if (p.lse && col == 0) p.lse[(size_t)head * p.n_tok + tok] = row_lse2(sum, p.c) * 0.69314718055994531f;
}

}  // namespace rc

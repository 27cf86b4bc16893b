// Merges the parts of the units that the paged attention kernels cut between
// CTAs: O = sum_i w_i O_i, w_i = l_i 2^(c m_i) / sum_k l_k 2^(c m_k) with each part's
// sum l_i 2^(c m_i) (RowSum), in fp32 and in a fixed order. Block (c, y) takes rows of the unit that begins in CTA
// c's range and goes on in the next; the unit's parts are slot 2c + 1 and
// slots 2(c + 1), 2(c + 2), ... up to the CTA whose record says that the unit
// ends there. First every part's weight for every row, in shared memory, then
// the weighted sum: a thread holds 8 columns of a row and several parts'
// loads are in flight at once; where the rows are few, groups of threads share the parts.
//
// Launched as a programmatic dependent of the attention kernel: its blocks are
// resident when that grid ends. Bound by that start-up and two dependent reads
// (records and sums, then the parts), from L2: 4.3 us behind the attention
// kernel for 12 units of one row, 16 us for 148 units of 256 rows (39 MB of parts;
// blocks of 64 threads that ask for the first parts along with the records: the same).
#include "paged_common.cuh"

namespace rc {

namespace {

constexpr int kCombThreads = 256;

// weight[i][r], l[i][r] from the two halves of RowSums to the shares of their sum, in weight, for sources i < n
// and rows r < rows, a warp a row; sum[r]: the sum. A source whose l is 0 gets the
// weight 0 whatever the others hold (a NaN among them included): it may not exist, and is not read.
template <int ROWS>
__device__ __forceinline__ void normalise(float (*weight)[ROWS], const float (*ls)[ROWS], int n, int rows, float c,
                                          RowSum* sum) {
  const int lane = threadIdx.x & 31;
  for (int r = threadIdx.x >> 5; r < rows; r += kCombThreads / 32) {
    float m = -INFINITY, l = 0.f;
    for (int i = lane; i < n; i += 32) m = fmaxf(m, weight[i][r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float ref = m == -INFINITY ? 0.f : m;
    for (int i = lane; i < n; i += 32) {
      const float x = ls[i][r] == 0.f ? 0.f : ls[i][r] * ptx::ex2((weight[i][r] - ref) * c);
      weight[i][r] = x;
      l += x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int i = lane; i < n; i += 32) {
      const float x = weight[i][r];
      weight[i][r] = x == 0.f ? 0.f : x * inv;
    }
    if (lane == 0) sum[r] = make_float2(m, l);
  }
}

// DECODE: up to 16 rows a unit, all in block y = 0; else 256 rows, 16 a block
// (few units cut over many CTAs: with 32 a block, 8 units of 18 parts took 22 us).
template <int D, bool BF16, bool DECODE>
__global__ void __launch_bounds__(kCombThreads) paged_combine_kernel(const __grid_constant__ PagedAttnParams p) {
  constexpr int kChunks = D / 8;
  constexpr int kUnitRows = DECODE ? kDecodeRows : kPrefillRows;
  constexpr int kRows = 16;
  constexpr int kEarly = kCombThreads / kRows;
  __shared__ int last_sh, flags_sh[kCombThreads];
  __shared__ float weight[kMaxPersistentCtas][kRows];
  static_assert(kMaxPersistentCtas <= kCombThreads, "a thread a CTA");
  __shared__ RowSum sum_sh[kRows];
  // the parts' second halves, and behind the weights the threads' sums: small enough that the block
  // is resident beside the attention kernel's
  constexpr int kScratch = kMaxPersistentCtas * kRows > kCombThreads * 9 ? kMaxPersistentCtas * kRows : kCombThreads * 9;
  __shared__ float scratch[kScratch];
  float(*ls)[kRows] = reinterpret_cast<float(*)[kRows]>(scratch);
  float(*so)[9] = reinterpret_cast<float(*)[9]>(scratch);
  const int tid = threadIdx.x, c = blockIdx.x, row_lo = blockIdx.y * kRows;
  if (tid == 0) last_sh = p.n_ctas - 1;
  auto part_row = [&](int i) { return (size_t)(2 * (c + i) + (i == 0)) * kUnitRows + row_lo; };
  ptx::grid_wait();
  // records and parts come from L2 (ld.cg): this block's SM may have cached
  // their addresses before the attention kernel wrote them. The first parts'
  // sums are asked for along with the records, before it is known which of them exist
  const PartRecord rec = __ldcg(p.rec + c);
  const int ahead = c + 1 + tid < p.n_ctas ? __ldcg(&p.rec[c + 1 + tid].x) : 0;
  const RowSum none = make_float2(-INFINITY, 0.f);
  RowSum early = none;
  if (tid < kEarly * kRows && c + tid / kRows < p.n_ctas) early = __ldcg(p.part_sum + part_row(tid / kRows) + tid % kRows);
  if (rec.z <= 0) return;
  flags_sh[tid] = ahead;
  __syncthreads();
  if (ahead & kHeadEnds) atomicMin(&last_sh, c + 1 + tid);
  const int n_rows = DECODE ? rec.z * p.G : kUnitRows, head0 = rec.w;
  __syncthreads();
  const int parts = last_sh - c + 1;
  const int rows = min(kRows, n_rows - row_lo);
  if (rows <= 0) return;
  for (int x = tid; x < parts * kRows; x += kCombThreads) {
    const int i = x / kRows, r = x % kRows;
    // a CTA whose range is empty left no part
    const bool there = r < rows && (i == 0 || (flags_sh[i - 1] & kHasHead));
    const RowSum s = !there ? none : (x < kEarly * kRows ? early : __ldcg(p.part_sum + part_row(i) + r));
    weight[i][r] = s.x;
    ls[i][r] = s.y;
  }
  __syncthreads();
  normalise(weight, ls, parts, rows, p.scale_log2, sum_sh);
  __syncthreads();
  const RowOutput to = row_output(p);
  const int items = rows * kChunks, groups = max(1, kCombThreads / items);
  for (int item0 = 0; item0 < items; item0 += kCombThreads) {
    const int item = groups > 1 ? tid % items : item0 + tid, grp = groups > 1 ? tid / items : 0;
    const bool on = item < items && grp < groups;
    const int r = on ? item / kChunks : 0, col = item % kChunks * 8;
    float acc[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = 0.f;
    if (on) {
#pragma unroll 4
      for (int i = grp; i < parts; i += groups) {
        const float w = weight[i][r];
        // nothing was written where the weight is 0: such a load goes to the first part
        const float4* src = reinterpret_cast<const float4*>(p.part_o + (part_row(w != 0.f ? i : 0) + r) * D + col);
        const float4 a = __ldcg(src), b = __ldcg(src + 1);
        const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = fmaf(x[k], w, acc[k]);
      }
    }
    if (groups > 1) {
#pragma unroll
      for (int k = 0; k < 8; ++k) so[tid][k] = acc[k];
      __syncthreads();
      if (on && grp == 0)
        for (int g = 1; g < groups; ++g)
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[k] += so[g * items + item][k];
    }
    if (!on || grp != 0) continue;
    const int row = row_lo + r;
    int i, h;
    if constexpr (DECODE) {
      i = row / p.G;
      h = row - i * p.G;
    } else {
      const int tpt = 128 / p.G, rr = row & 127;
      i = (row >> 7) * tpt + rr / p.G;
      h = rr % p.G;
      if (rr >= tpt * p.G || i >= rec.z) continue;
    }
    store_row<D, BF16>(to, rec.y + i, head0 + h, col, acc, sum_sh[r]);
  }
}

// One result over some of the keys of a unit: where it lies whole, and where in parts.
struct JoinSide {
  const float* o;
  const RowSum* sum;  // whole rows: [n_tok][q_heads][d] and [q_heads][n_tok]
  const float* part_o;
  const RowSum* part_sum;
  const int4* rec;
  int n_ctas;
};
struct JoinParams {
  BatchView b;
  RowOutput to;
  JoinSide own, pre;
  int n_tok, Hk, G;
};

constexpr int kJoinSources = 2 * kMaxPersistentCtas + 2;

// Block (b, h): the rows of sequence b and key head h (at most 16). A row's
// sources are its unit's parts in the decode pass, or its whole row, and the
// parts, or the whole row, of the query pair its token lies in in the pass over the prefix.
// As in the combine kernel: all sources' weights first, then the weighted sum.
// 48 sequences of 8 key heads, the prefix in 18 parts a head: 8 to 10 us behind the kernels.
template <int D, bool BF16>
__global__ void __launch_bounds__(kCombThreads) paged_join_kernel(const __grid_constant__ JoinParams p) {
  constexpr int kChunks = D / 8;
  __shared__ int first_sh[3], last_sh[3];  // the decode unit's, and the first and last token's pair's
  // small enough that two blocks are resident beside the decode kernel's (with the sums' other
  // halves here too, one: 0.7 us more)
  __shared__ float scratch[kJoinSources * kDecodeRows];
  __shared__ float most_sh[kCombThreads / 32][kDecodeRows], l_sh[kCombThreads / 32][kDecodeRows];  // each warp's, of the rows
  __shared__ uint8_t there[2][kMaxPersistentCtas];  // the CTAs' records' flags
  float(*weight)[kDecodeRows] = reinterpret_cast<float(*)[kDecodeRows]>(scratch);
  float(*so)[9] = reinterpret_cast<float(*)[9]>(scratch);  // after the weights
  static_assert(kCombThreads * 9 <= kJoinSources * kDecodeRows, "the sums fit");
  const int tid = threadIdx.x;
  const int b = blockIdx.x / p.Hk, h = blockIdx.x - b * p.Hk;
  const Seq s = load_seq(p.b, p.n_tok, b);
  const int R = min(s.n, 16 / p.G) * p.G, heads = p.Hk * p.G;
  const int per_pair = 2 * (128 / p.G);
  const int pair0 = s.q0 / per_pair, pair1 = R > 0 ? (s.q0 + R / p.G - 1) / per_pair : pair0;
  if (tid < 3) {
    first_sh[tid] = -1;
    last_sh[tid] = (tid == 0 ? p.own : p.pre).n_ctas - 1;
  }
  ptx::grid_wait();
  if (R == 0) return;
  __syncthreads();
  const int most = max(p.own.n_ctas, p.pre.n_ctas);
  for (int c = tid; c < most; c += kCombThreads) {
    const int4 none = make_int4(0, 0, 0, 0);
    const int4 x = c < p.own.n_ctas ? __ldcg(p.own.rec + c) : none, y = c < p.pre.n_ctas ? __ldcg(p.pre.rec + c) : none;
    if (x.z > 0 && x.y == s.q0 && x.w == h * p.G) first_sh[0] = c;
    if (y.z > 0 && y.y == pair0 * per_pair && y.w == h * p.G) first_sh[1] = c;
    if (y.z > 0 && y.y == pair1 * per_pair && y.w == h * p.G) first_sh[2] = c;
    there[0][c] = x.x;
    there[1][c] = y.x;
  }
  __syncthreads();
  for (int c = tid; c < most; c += kCombThreads)
    for (int k = 0; k < 3; ++k)
      if (first_sh[k] >= 0 && c > first_sh[k] && (there[k > 0][c] & kHeadEnds)) atomicMin(&last_sh[k], c);
  __syncthreads();
  const int n_own = first_sh[0] < 0 ? 1 : last_sh[0] - first_sh[0] + 1;
  const int n_pre0 = first_sh[1] < 0 ? 1 : last_sh[1] - first_sh[1] + 1;
  const int n_pre1 = first_sh[2] < 0 ? 1 : last_sh[2] - first_sh[2] + 1;
  const int n = n_own + max(n_pre0, n_pre1);
  // Row r's values and sum on one side: whole (c < 0), or in the parts
  // from CTA c on, whose slots lie `unit` rows apart.
  struct Rows {
    const float* o;
    const RowSum* l;
    int c, last, unit;
  };
  auto rows_of = [&](int r, bool own) {
    const int i = r / p.G, g = r - i * p.G, tok = s.q0 + i, head = h * p.G + g;
    const JoinSide& side = own ? p.own : p.pre;
    const int in_pair = tok % per_pair;
    const int k = own ? 0 : (tok - in_pair == pair0 * per_pair ? 1 : 2);
    Rows x;
    x.c = first_sh[k];
    x.last = last_sh[k];
    x.unit = own ? kDecodeRows : kPrefillRows;
    const int tpt = per_pair / 2, tile = in_pair >= tpt;
    const size_t at = x.c < 0 ? (size_t)tok * heads + head
                              : (size_t)(own ? r : tile * 128 + (in_pair - tile * tpt) * p.G + g);
    x.o = (x.c < 0 ? side.o : side.part_o) + at * D;
    x.l = x.c < 0 ? side.sum + (size_t)head * p.n_tok + tok : side.part_sum + at;
    return x;
  };
  auto slot = [](const Rows& x, int e) { return x.c < 0 ? (size_t)0 : (size_t)(2 * (x.c + e) + (e == 0)) * x.unit; };
  // a row's largest m, then its sources' l 2^(c (m - that)) and their sum; a source that does not exist has the
  // weight 0, whatever the others hold, and is not read
  {
    const int r = tid % kDecodeRows, warp = tid >> 5;  // the row of all of a thread's sources
    const int e0 = tid / kDecodeRows, step = kCombThreads / kDecodeRows;
    const Rows own = rows_of(min(r, R - 1), true), pre = rows_of(min(r, R - 1), false);
    auto source = [&](int e) {
      const bool mine = e < n_own;
      const Rows& x = mine ? own : pre;
      const int i = mine ? e : e - n_own;
      // a CTA whose range is empty left no part
      const bool is = e < n && r < R && (i == 0 || (x.c >= 0 && x.c + i <= x.last && (there[!mine][x.c + i] & kHasHead)));
      return is ? __ldcg(x.l + slot(x, i)) : make_float2(-INFINITY, 0.f);
    };
    const RowSum first = source(e0), second = source(e0 + step);  // kept; the rest is loaded twice
    float m = fmaxf(first.x, second.x), l = 0.f;
    for (int e = e0 + 2 * step; e < n; e += step) m = fmaxf(m, source(e).x);
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, kDecodeRows));
    most_sh[warp][r] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kCombThreads / 32; ++w) m = fmaxf(m, most_sh[w][r]);
    const float ref = m == -INFINITY ? 0.f : m;
    for (int e = e0; e < n; e += step) {
      const RowSum x = e == e0 ? first : (e == e0 + step ? second : source(e));
      const float w = x.y == 0.f ? 0.f : x.y * ptx::ex2((x.x - ref) * p.to.c);
      weight[e][r] = w;
      l += w;
    }
    l += __shfl_xor_sync(0xffffffffu, l, kDecodeRows);
    l_sh[warp][r] = l;
  }
  __syncthreads();
  const int items = R * kChunks, groups = kCombThreads / items;
  const int item = tid % items, grp = tid / items;
  const int r = item / kChunks, col = item % kChunks * 8;
  float acc[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.f;
  if (grp < groups) {
    const Rows own = rows_of(r, true), pre = rows_of(r, false);
#pragma unroll 4
    for (int e = grp; e < n; e += groups) {
      const float w = weight[e][r];
      const bool mine = e < n_own;
      // nothing was written where the weight is 0: such a load goes to the side's first source
      const int i = w != 0.f ? (mine ? e : e - n_own) : 0;
      const float4* src = reinterpret_cast<const float4*>((mine ? own.o + slot(own, i) * D : pre.o + slot(pre, i) * D) + col);
      const float4 a = __ldcg(src), c = __ldcg(src + 1);
      const float x[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = fmaf(x[k], w, acc[k]);
    }
  }
  RowSum sum = make_float2(-INFINITY, 0.f);
#pragma unroll
  for (int w = 0; w < kCombThreads / 32; ++w) sum = make_float2(fmaxf(sum.x, most_sh[w][r]), sum.y + l_sh[w][r]);
  const float inv = sum.y == 0.f ? 0.f : 1.f / sum.y;
  if (groups > 1) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) so[tid][k] = acc[k];
    __syncthreads();
    if (grp == 0)
      for (int g = 1; g < groups; ++g)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] += so[g * items + item][k];
  }
  if (grp != 0) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] *= inv;
  const int i = r / p.G;
  store_row<D, BF16>(p.to, s.q0 + i, h * p.G + r - i * p.G, col, acc, sum);
}

template <int D, bool BF16>
cudaError_t join_d(const JoinParams& p, cudaStream_t s) {
  return launch_chained(paged_join_kernel<D, BF16>, p, dim3(p.b.n_seqs * p.Hk), kCombThreads, 0, true, s);
}

// out = the merge of the results in (pre_o, pre_sum) and (prev_o, prev_sum), 8
// columns of a row a thread, rows of no sequence left alone. Bound by HBM and L2: 768
// rows of 32 heads of 128, 31 MB, 6.2 us.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) paged_merge_kernel(const __grid_constant__ PagedAttnParams p) {
  constexpr int kChunks = D / 8;
  const long long x = (long long)blockIdx.x * 256 + threadIdx.x;
  const int heads = p.Hk * p.G;
  const long long row = x / kChunks;
  const int tok = (int)(row / heads), head = (int)(row - (long long)tok * heads), col = (int)(x % kChunks) * 8;
  if (tok >= min(p.n_tok, __ldg(p.b.cu_q + p.b.n_seqs)) || tok < __ldg(p.b.cu_q)) return;
  const float4* src = reinterpret_cast<const float4*>(p.pre_o + (size_t)row * D + col);
  const float4 a = src[0], b = src[1];
  float acc[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  RowSum sum = p.pre_sum[(size_t)head * p.n_tok + tok];
  RowOutput to = row_output(p);
  to.pre_o = nullptr;
  merge_prev<D>(to, tok, head, col, acc, sum);
  store_row<D, BF16>(to, tok, head, col, acc, sum);
}

template <int D, bool BF16>
cudaError_t merge_d(const PagedAttnParams& p, cudaStream_t s) {
  const long long threads = (long long)p.n_tok * p.Hk * p.G * (D / 8);
  paged_merge_kernel<D, BF16><<<(unsigned)((threads + 255) / 256), 256, 0, s>>>(p);
  return cudaGetLastError();
}

template <int D, bool BF16>
cudaError_t combine_d(const PagedAttnParams& p, bool decode, cudaStream_t s) {
  const dim3 grid(p.n_ctas, decode ? 1 : kPrefillRows / 16);
  return decode ? launch_chained(paged_combine_kernel<D, BF16, true>, p, grid, kCombThreads, 0, true, s)
                : launch_chained(paged_combine_kernel<D, BF16, false>, p, grid, kCombThreads, 0, true, s);
}

}  // namespace

cudaError_t launch_paged_combine(const PagedAttnParams& p, bool bf16, int head_dim, bool decode, cudaStream_t s) {
  if (head_dim == 64) return bf16 ? combine_d<64, true>(p, decode, s) : combine_d<64, false>(p, decode, s);
  return bf16 ? combine_d<128, true>(p, decode, s) : combine_d<128, false>(p, decode, s);
}

cudaError_t launch_paged_join(const PagedAttnParams& own, const PagedAttnParams& pre, bool bf16, int head_dim,
                              cudaStream_t s) {
  JoinParams p{};
  p.b = own.b;
  p.to = RowOutput{own.out.data, own.out.tok_stride, own.out.head_stride, own.lse,        nullptr,       nullptr,
                   nullptr,      nullptr,            own.n_tok,           own.Hk * own.G, own.scale_log2};
  p.own = JoinSide{own.pre_o, own.pre_sum, own.part_o, own.part_sum, own.rec, own.n_ctas};
  p.pre = JoinSide{pre.pre_o, pre.pre_sum, pre.part_o, pre.part_sum, pre.rec, pre.n_ctas};
  p.n_tok = own.n_tok;
  p.Hk = own.Hk;
  p.G = own.G;
  if (head_dim == 64) return bf16 ? join_d<64, true>(p, s) : join_d<64, false>(p, s);
  return bf16 ? join_d<128, true>(p, s) : join_d<128, false>(p, s);
}

cudaError_t launch_paged_merge(const PagedAttnParams& p, bool bf16, int head_dim, cudaStream_t s) {
  if (head_dim == 64) return bf16 ? merge_d<64, true>(p, s) : merge_d<64, false>(p, s);
  return bf16 ? merge_d<128, true>(p, s) : merge_d<128, false>(p, s);
}

}  // namespace rc

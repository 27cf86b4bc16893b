// Merges the parts of the units that the paged attention kernels cut between
// CTAs: O = sum_i 2^(lse_i - lse) O_i, lse = log2 sum_i 2^(lse_i), in fp32 and
// in a fixed order. Block (c, y) takes rows of the unit that begins in CTA
// c's range and goes on in the next; the unit's parts are slot 2c + 1 and
// slots 2(c + 1), 2(c + 2), ... up to the CTA whose record says that the unit
// ends there. First every part's weight for every row, in shared memory, then
// the weighted sum: a thread holds 8 columns of a row and several parts'
// loads are in flight at once; where the rows are few, groups of threads share the parts.
//
// Launched as a programmatic dependent of the attention kernel: its blocks are
// resident when that grid ends. Bound by that start-up and two dependent reads
// (records and log-sum-exps, then the parts), from L2.
#include "paged_common.cuh"

namespace rc {

namespace {

constexpr int kCombThreads = 256;

// DECODE: up to 16 rows a unit, all in block y = 0; else 256 rows, 16 a block
// (few units cut over many CTAs: with 32 a block, 8 units of 18 parts took 22 us).
template <int D, bool BF16, bool DECODE>
__global__ void __launch_bounds__(kCombThreads) paged_combine_kernel(const __grid_constant__ PagedAttnParams p) {
  constexpr int kChunks = D / 8;
  constexpr int kUnitRows = DECODE ? kDecodeRows : kPrefillRows;
  constexpr int kRows = 16;
  __shared__ int last_sh;
  __shared__ float weight[kMaxPersistentCtas][kRows];
  __shared__ float lse_sh[kRows];
  __shared__ float so[kCombThreads][9];
  const int tid = threadIdx.x, lane = tid & 31, c = blockIdx.x;
  if (tid == 0) last_sh = p.n_ctas - 1;
  ptx::grid_launch_dependents();
  ptx::grid_wait();
  // records and parts come from L2 (ld.cg): this block's SM may have cached
  // their addresses before the attention kernel wrote them
  const PartRecord rec = __ldcg(p.rec + c);
  if (rec.z < 0 || rec.z >= p.b.n_seqs) return;
  __syncthreads();
  for (int i = c + 1 + tid; i < p.n_ctas; i += kCombThreads)
    if (__ldcg(&p.rec[i].y)) atomicMin(&last_sh, i);
  // the unit's rows
  int n_rows, head0, pair = 0;
  Seq s;
  if constexpr (DECODE) {
    s = load_seq(p.b, p.n_tok, rec.z);
    n_rows = min(s.n, 16 / p.G) * p.G;
    head0 = rec.w * p.G;
  } else {
    if (p.batch_pass) {
      s.q0 = 0;
      s.n = min(max(__ldg(p.b.cu_q + p.b.n_seqs), 0), p.n_tok);
    } else {
      s = load_seq(p.b, p.n_tok, rec.z);
    }
    const int tpt = 128 / p.G, pairs = max((s.n + 2 * tpt - 1) / (2 * tpt), 1);
    pair = rec.w % pairs;
    head0 = rec.w / pairs * p.G;
    n_rows = kUnitRows;
  }
  __syncthreads();
  const int parts = last_sh - c + 1;
  const int row_lo = blockIdx.y * kRows;
  const int rows = min(kRows, n_rows - row_lo);
  if (rows <= 0) return;
  auto part_row = [&](int i) { return (size_t)(2 * (c + i) + (i == 0)) * kUnitRows + row_lo; };
  for (int x = tid; x < parts * kRows; x += kCombThreads) {
    const int i = x / kRows, r = x % kRows;
    // a CTA whose range is empty left no part
    const bool there = r < rows && (i == 0 || __ldcg(&p.rec[c + i].x));
    weight[i][r] = there ? __ldcg(p.part_lse + part_row(i) + r) : -INFINITY;
  }
  __syncthreads();
  for (int r = tid >> 5; r < rows; r += kCombThreads / 32) {
    float m = -INFINITY, l = 0.f;
    for (int i = lane; i < parts; i += 32) m = fmaxf(m, weight[i][r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float ref = m == -INFINITY ? 0.f : m;
    for (int i = lane; i < parts; i += 32) l += exp2f(weight[i][r] - ref);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int i = lane; i < parts; i += 32) weight[i][r] = exp2f(weight[i][r] - ref) * inv;
    if (lane == 0) lse_sh[r] = l == 0.f ? -INFINITY : ref + log2f(l);
  }
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
      i = (pair * 2 + (row >> 7)) * tpt + rr / p.G;
      h = rr % p.G;
      if (rr >= tpt * p.G || i >= s.n) continue;
    }
    float lse2 = lse_sh[r];
    if (DECODE && to.prev_o) merge_prev<D>(to, s.q0 + i, head0 + h, col, acc, lse2);
    store_row<D, BF16>(to, s.q0 + i, head0 + h, col, acc, lse2);
  }
}

// out = the merge of the results in (pre_o, pre_lse) and (prev_o, prev_lse), 8
// columns of a row a thread, rows behind the last sequence left alone.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) paged_merge_kernel(const __grid_constant__ PagedAttnParams p) {
  constexpr int kChunks = D / 8;
  const long long x = (long long)blockIdx.x * 256 + threadIdx.x;
  const int heads = p.Hk * p.G;
  const long long row = x / kChunks;
  const int tok = (int)(row / heads), head = (int)(row - (long long)tok * heads), col = (int)(x % kChunks) * 8;
  if (tok >= min(p.n_tok, __ldg(p.b.cu_q + p.b.n_seqs))) return;
  const float4* src = reinterpret_cast<const float4*>(p.pre_o + (size_t)row * D + col);
  const float4 a = src[0], b = src[1];
  float acc[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float lse2 = p.pre_lse[(size_t)head * p.n_tok + tok];
  RowOutput to = row_output(p);
  to.pre_o = nullptr;
  merge_prev<D>(to, tok, head, col, acc, lse2);
  store_row<D, BF16>(to, tok, head, col, acc, lse2);
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

cudaError_t launch_paged_merge(const PagedAttnParams& p, bool bf16, int head_dim, cudaStream_t s) {
  if (head_dim == 64) return bf16 ? merge_d<64, true>(p, s) : merge_d<64, false>(p, s);
  return bf16 ? merge_d<128, true>(p, s) : merge_d<128, false>(p, s);
}

}  // namespace rc

// Merges the parts of the units that the paged attention kernels cut between
// CTAs: O = sum_i 2^(lse_i - lse) O_i, lse = log2 sum_i 2^(lse_i), in fp32 and
// in a fixed order. Block (c, y) takes rows of the unit that begins in CTA
// c's range and goes on in the next; the unit's parts are slot 2c + 1 and
// slots 2(c + 1), 2(c + 2), ... up to the CTA whose record says that the unit
// ends there. A thread holds 8 columns of a row; where the rows are few,
// groups of threads share the parts, so that a single long sequence cut over
// every CTA is not summed part after part by one thread.
//
// Launched as a programmatic dependent of the attention kernel: its blocks are
// resident when that grid ends. Bound by that start-up and one dependent read
// of the records and the parts (L2).
#include "paged_common.cuh"

namespace rc {

namespace {

constexpr int kCombThreads = 256;

// DECODE: up to 16 rows a unit, all in block y = 0; else 256 rows, 8 a block.
template <int D, bool BF16, bool DECODE>
__global__ void __launch_bounds__(kCombThreads) paged_combine_kernel(const __grid_constant__ PagedAttnParams p) {
  constexpr int kChunks = D / 8;
  constexpr int kUnitRows = DECODE ? kDecodeRows : kPrefillRows;
  constexpr int kRows = DECODE ? kDecodeRows : 8;
  __shared__ int last_sh;
  __shared__ float sm[kCombThreads], sl[kCombThreads];
  __shared__ float so[kCombThreads][9];
  const int tid = threadIdx.x, c = blockIdx.x;
  if (tid == 0) last_sh = p.n_ctas - 1;
  ptx::grid_wait();
  // records and parts come from L2 (ld.cg): this block's SM may have cached
  // their addresses before the attention kernel wrote them
  const PartRecord rec = __ldcg(p.rec + c);
  if (rec.z < 0 || rec.z >= p.b.n_seqs) return;
  __syncthreads();
  for (int i = c + 1 + tid; i < p.n_ctas; i += kCombThreads) {
    const PartRecord r = __ldcg(p.rec + i);
    if (r.y) atomicMin(&last_sh, i);
  }
  __syncthreads();
  const int parts = last_sh - c + 1;
  // the unit's rows
  int tok0, n_rows, head0;
  Seq s;
  int pair = 0;
  if constexpr (DECODE) {
    s = load_seq(p.b, p.n_tok, rec.z);
    n_rows = min(s.n, 16 / p.G) * p.G;
    head0 = rec.w * p.G;
  } else {
    if (p.pre_o) {
      s.q0 = 0;
      s.n = min(max(__ldg(p.b.cu_q + p.b.n_seqs), 0), p.n_tok);
    } else {
      s = load_seq(p.b, p.n_tok, rec.z);
    }
    const int tpt = 128 / p.G, pairs = (s.n + 2 * tpt - 1) / (2 * tpt);
    pair = rec.w % pairs;
    head0 = rec.w / pairs * p.G;
    n_rows = kUnitRows;
  }
  const int row_lo = blockIdx.y * kRows;
  const int rows = min(kRows, n_rows - row_lo);
  if (rows <= 0) return;
  const int items = rows * kChunks, groups = kCombThreads / items;
  const int item = tid % items, grp = tid / items;
  const int row = row_lo + item / kChunks, col = item % kChunks * 8;
  float m = -INFINITY, l = 0.f, acc[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.f;
  if (grp < groups) {
    for (int i = grp; i < parts; i += groups) {
      if (i > 0 && !__ldcg(&p.rec[c + i].x)) continue;  // a CTA whose range is empty
      const size_t at = (size_t)(2 * (c + i) + (i == 0)) * kUnitRows + row;
      const float pl = __ldcg(p.part_lse + at);
      const float4* src = reinterpret_cast<const float4*>(p.part_o + at * D + col);
      const float4 a = __ldcg(src), b = __ldcg(src + 1);
      if (pl == -INFINITY) continue;
      const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      const float mn = fmaxf(m, pl), f = exp2f(m - mn), w = exp2f(pl - mn);
      m = mn;
      l = l * f + w;
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = acc[k] * f + x[k] * w;
    }
  }
  if (groups > 1) {
    sm[tid] = m;
    sl[tid] = l;
#pragma unroll
    for (int k = 0; k < 8; ++k) so[tid][k] = acc[k];
    __syncthreads();
    if (grp == 0) {
      float gm = m;
      for (int g = 1; g < groups; ++g) gm = fmaxf(gm, sm[g * items + item]);
      l = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = 0.f;
      for (int g = 0; g < groups; ++g) {
        const int t = g * items + item;
        if (sl[t] == 0.f) continue;
        const float f = exp2f(sm[t] - gm);
        l += sl[t] * f;
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] += so[t][k] * f;
      }
      m = gm;
    }
  }
  if (grp != 0) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] *= inv;
  int i, h;
  if constexpr (DECODE) {
    i = row / p.G;
    h = row - i * p.G;
  } else {
    const int tpt = 128 / p.G, rr = row & 127;
    i = (pair * 2 + (row >> 7)) * tpt + rr / p.G;
    h = rr % p.G;
    if (rr >= tpt * p.G || i >= s.n) return;
  }
  const RowOutput to = row_output(p);
  if (to.prev_o) merge_prev<D>(to, s.q0 + i, head0 + h, col, acc, lse2);
  store_row<D, BF16>(to, s.q0 + i, head0 + h, col, acc, lse2);
}

template <int D, bool BF16>
cudaError_t combine_d(const PagedAttnParams& p, bool decode, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.n_ctas, decode ? 1 : kPrefillRows / 8);
  cfg.blockDim = dim3(kCombThreads);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return decode ? cudaLaunchKernelEx(&cfg, paged_combine_kernel<D, BF16, true>, p)
                : cudaLaunchKernelEx(&cfg, paged_combine_kernel<D, BF16, false>, p);
}

}  // namespace

cudaError_t launch_paged_combine(const PagedAttnParams& p, bool bf16, int head_dim, bool decode, cudaStream_t s) {
  if (head_dim == 64) return bf16 ? combine_d<64, true>(p, decode, s) : combine_d<64, false>(p, decode, s);
  return bf16 ? combine_d<128, true>(p, decode, s) : combine_d<128, false>(p, decode, s);
}

}  // namespace rc

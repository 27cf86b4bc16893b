// Rotary positions over several axes, alone and on the way into the pages of
// a cache.
//
// Pair m of a head's d / 2 pairs belongs to one axis (the first pairs[0] to
// axis 0, the next pairs[1] to axis 1, ...) and turns by the angle whose
// (cos, sin) its axis's table holds at the token's position on that axis:
//   (a, b) -> (a c - b s, a s + b c).
// Adjacent pairing takes (a, b) = (x[2m], x[2m + 1]), halves pairing
// (x[m], x[m + d/2]). The turn is orthogonal, so its gradient is the turn by
// the opposite angle: the same kernel with the sine's sign changed.
//
// Bound by HBM: each element is read and written once. A group of d / 2E lanes
// holds one token (E elements to 16 bytes, two such chunks a lane, d / 2 apart, so that
// every load and store of the group is one contiguous run and both pairings
// find their partners in one lane). The lane's (cos, sin) pairs are loaded
// once and serve every head that the group visits; `splits` groups share a
// token's heads when there are too few tokens to fill the GPU. Products are
// fp32, rounded once at the store. Measured: 18720 tokens of 24 heads of 128, 230 MB
// in 35.6 us, 6.5 TB/s (the copy rate); four chunks' append, 345 MB in 56 us.
#include "paged.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace rc {

namespace {

// 16 bytes of a row as fp32 values.
template <int DT>
struct Chunk;
template <>
struct Chunk<RC_BF16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void load(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 store(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Chunk<RC_F16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void load(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
  static __device__ __forceinline__ uint4 store(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Chunk<RC_F32> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void load(const uint4& u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 store(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// The (cos, sin) of the lane's E pairs at token `tok`. A position outside its
// table is clamped to it (no read leaves the table) and recorded.
template <int E, int LN, bool HALVES>
__device__ __forceinline__ void load_angles(const AxisTables& ax, int tok, int lane, float sign, int* status,
                                            float (&c)[E], float (&s)[E]) {
  const float2* row[3];
  bool bad = false;
#pragma unroll
  for (int a = 0; a < 3; ++a) {
    row[a] = nullptr;
    if (a < ax.n_axes) {
      const int p = __ldg(ax.pos + (size_t)tok * ax.n_axes + a);
      const int q = min(max(p, 0), ax.n_pos[a] - 1);
      bad |= p != q;
      row[a] = ax.table[a] + (size_t)q * ax.pairs[a];
    }
  }
  if (bad && status) atomicCAS(status, 0, (int)RC_ERANGE);
#pragma unroll
  for (int j = 0; j < E; ++j) {
    int m = HALVES ? lane * E + j : (j < E / 2 ? lane * (E / 2) + j : (lane + LN) * (E / 2) + j - E / 2);
    const float2* r = row[0];
    if (m >= ax.pairs[0]) {
      m -= ax.pairs[0];
      r = row[1];
      if (m >= ax.pairs[1]) {
        m -= ax.pairs[1];
        r = row[2];
      }
    }
    const float2 v = __ldg(r + m);
    c[j] = v.x;
    s[j] = sign * v.y;
  }
}

// Turns the lane's two chunks of a row in place.
template <int E, bool HALVES>
__device__ __forceinline__ void turn(float (&a)[E], float (&b)[E], const float (&c)[E], const float (&s)[E]) {
  if constexpr (HALVES) {
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float x = a[j], y = b[j];
      a[j] = x * c[j] - y * s[j];
      b[j] = x * s[j] + y * c[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      const float x = a[2 * j], y = a[2 * j + 1];
      a[2 * j] = x * c[j] - y * s[j];
      a[2 * j + 1] = x * s[j] + y * c[j];
      const float u = b[2 * j], v = b[2 * j + 1];
      b[2 * j] = u * c[E / 2 + j] - v * s[E / 2 + j];
      b[2 * j + 1] = u * s[E / 2 + j] + v * c[E / 2 + j];
    }
  }
}

constexpr int kUnroll = 4;  // heads in flight per lane
constexpr int kRopeThreads = 256;

template <int DT, int D, bool HALVES>
__global__ void __launch_bounds__(kRopeThreads) rope_axes_kernel(const __grid_constant__ RopeAxesParams p) {
  using C = Chunk<DT>;
  constexpr int E = C::E, LN = D / 2 / E;
  const long long idx = (long long)blockIdx.x * kRopeThreads + threadIdx.x;
  const int lane = (int)(idx % LN);
  const long long g = idx / LN;
  if (g >= (long long)p.n_tok * p.splits) return;
  const int tok = (int)(g / p.splits), s0 = (int)(g - (long long)tok * p.splits);
  const int NH = p.x[0].heads + p.x[1].heads;
  float c[E], s[E];
  bool have = false;
  for (int h0 = s0; h0 < NH; h0 += p.splits * kUnroll) {
    uint4 u[kUnroll][2];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int hh = h0 + i * p.splits;
      if (hh >= NH) break;
      const int w = hh >= p.x[0].heads;
      const uint8_t* src = p.x[w].data + tok * p.x[w].tok_stride + (hh - (w ? p.x[0].heads : 0)) * p.x[w].head_stride;
      u[i][0] = *reinterpret_cast<const uint4*>(src + lane * 16);
      u[i][1] = *reinterpret_cast<const uint4*>(src + (lane + LN) * 16);
    }
    if (!have) load_angles<E, LN, HALVES>(p.ax, tok, lane, p.sign, p.status, c, s);
    have = true;
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int hh = h0 + i * p.splits;
      if (hh >= NH) break;
      const int w = hh >= p.x[0].heads;
      float a[E], b[E];
      C::load(u[i][0], a);
      C::load(u[i][1], b);
      turn<E, HALVES>(a, b, c, s);
      uint8_t* dst = p.y[w].data + tok * p.y[w].tok_stride + (hh - (w ? p.x[0].heads : 0)) * p.y[w].head_stride;
      *reinterpret_cast<uint4*>(dst + lane * 16) = C::store(a);
      *reinterpret_cast<uint4*>(dst + (lane + LN) * 16) = C::store(b);
    }
  }
}

// The sequence of token `tok`: the largest b < n_seqs with cu_q[b] <= tok.
__device__ __forceinline__ int seq_of(const BatchView& v, int tok) {
  int lo = 0, hi = v.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(v.cu_q + mid) <= tok) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The append: head index hh walks the query heads (turned, to q_out), then
// the key heads (turned, into the token's page row), then the value heads
// (copied there). Tokens behind the last sequence are left alone, those of no sequence before
// that too, with RC_ERANGE; a token whose place does not exist (a position before 0, past the table, or an
// entry that is no page) keeps its keys and values out of the pool and
// records RC_ERANGE.
template <int DT, int D, bool HALVES>
__global__ void __launch_bounds__(kRopeThreads) paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
  using C = Chunk<DT>;
  constexpr int E = C::E, LN = D / 2 / E;
  const long long idx = (long long)blockIdx.x * kRopeThreads + threadIdx.x;
  const int lane = (int)(idx % LN);
  const long long g = idx / LN;
  if (g >= (long long)p.n_tok * p.splits) return;
  const int tok = (int)(g / p.splits), s0 = (int)(g - (long long)tok * p.splits);
  // sequences that begin before the first row or end behind the last
  if (idx == 0 && p.status && (__ldg(p.b.cu_q) != 0 || __ldg(p.b.cu_q + p.b.n_seqs) > p.n_tok))
    atomicCAS(p.status, 0, (int)RC_ERANGE);
  const int Hq = p.q.heads, Hk = p.k.heads, NH = Hq + 2 * Hk;
  const bool rotate = p.ax.n_axes > 0;
  float c[E], s[E];
  bool have = false, inside = true;
  long long krow = 0, vrow = 0;
  for (int h0 = s0; h0 < NH && inside; h0 += p.splits * kUnroll) {
    uint4 u[kUnroll][2];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int hh = h0 + i * p.splits;
      if (hh >= NH) break;
      const RowsView& r = hh < Hq ? p.q : (hh < Hq + Hk ? p.k : p.v);
      const int h = hh < Hq ? hh : (hh < Hq + Hk ? hh - Hq : hh - Hq - Hk);
      const uint8_t* src = r.data + tok * r.tok_stride + h * r.head_stride;
      u[i][0] = *reinterpret_cast<const uint4*>(src + lane * 16);
      u[i][1] = *reinterpret_cast<const uint4*>(src + (lane + LN) * 16);
    }
    if (!have) {
      have = true;
      const int b = seq_of(p.b, tok);
      const int q0 = __ldg(p.b.cu_q + b), q1 = __ldg(p.b.cu_q + b + 1);
      inside = tok >= q0 && tok < q1;
      krow = vrow = -1;
      if (inside) {
        const int at = __ldg(p.b.kv_len + b) - (q1 - tok);
        const int slot = at >> p.b.page_log2;
        int page = -1;
        if (at >= 0 && slot < p.b.max_pages) page = __ldg(p.b.page_table + b * p.b.table_stride + slot);
        if (page >= 0 && page < p.b.n_pages) {
          const int row = at & ((1 << p.b.page_log2) - 1);
          krow = page * p.kp.page_stride + row * p.kp.row_stride;
          vrow = page * p.vp.page_stride + row * p.vp.row_stride;
        } else if (p.status) {
          atomicCAS(p.status, 0, (int)RC_ERANGE);
        }
        if (rotate) load_angles<E, LN, HALVES>(p.ax, tok, lane, 1.f, p.status, c, s);
      }
    }
    if (!inside) {  // of no sequence, and before the last one's end
      if (p.status && tok < __ldg(p.b.cu_q + p.b.n_seqs)) atomicCAS(p.status, 0, (int)RC_ERANGE);
      break;
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int hh = h0 + i * p.splits;
      if (hh >= NH) break;
      uint8_t* dst;
      if (hh < Hq) {
        dst = p.q_out.data + tok * p.q_out.tok_stride + hh * p.q_out.head_stride;
      } else if (krow < 0) {
        continue;
      } else if (hh < Hq + Hk) {
        dst = p.kp.data + krow + (hh - Hq) * p.kp.head_stride;
      } else {
        dst = p.vp.data + vrow + (hh - Hq - Hk) * p.vp.head_stride;
      }
      if (rotate && hh < Hq + Hk) {
        float a[E], b[E];
        C::load(u[i][0], a);
        C::load(u[i][1], b);
        turn<E, HALVES>(a, b, c, s);
        u[i][0] = C::store(a);
        u[i][1] = C::store(b);
      }
      *reinterpret_cast<uint4*>(dst + lane * 16) = u[i][0];
      *reinterpret_cast<uint4*>(dst + (lane + LN) * 16) = u[i][1];
    }
  }
}

// Groups that share a token's heads: one while the tokens alone give every SM
// 768 threads, more for fewer tokens, at most one per head. (1536 threads: 6000
// tokens of 24 heads 23 us instead of 20.5, 18720 tokens 44 instead of 45, the
// append of four chunks 65.5 instead of 64.5; every group loads its angles anew.)
int head_splits(int n_tok, int lanes, int heads) {
  const long long want = 148LL * 768, have = (long long)n_tok * lanes;
  const long long s = (want + have - 1) / have;
  return (int)(s < 1 ? 1 : (s > heads ? heads : s));
}

template <typename P, typename K>
cudaError_t launch(K kernel, const P& p, int lanes, cudaStream_t s) {
  const long long threads = (long long)p.n_tok * p.splits * lanes;
  kernel<<<(unsigned)((threads + kRopeThreads - 1) / kRopeThreads), kRopeThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <int DT, int D>
cudaError_t rope_d(const RopeAxesParams& p0, bool halves, cudaStream_t s) {
  constexpr int lanes = D / 2 / Chunk<DT>::E;
  RopeAxesParams p = p0;
  p.splits = head_splits(p.n_tok, lanes, p.x[0].heads + p.x[1].heads);
  return halves ? launch(rope_axes_kernel<DT, D, true>, p, lanes, s)
                : launch(rope_axes_kernel<DT, D, false>, p, lanes, s);
}

template <int DT, int D>
cudaError_t append_d(const PagedAppendParams& p0, bool halves, cudaStream_t s) {
  constexpr int lanes = D / 2 / Chunk<DT>::E;
  PagedAppendParams p = p0;
  p.splits = head_splits(p.n_tok, lanes, p.q.heads + 2 * p.k.heads);
  return halves ? launch(paged_append_kernel<DT, D, true>, p, lanes, s)
                : launch(paged_append_kernel<DT, D, false>, p, lanes, s);
}

}  // namespace

cudaError_t launch_rope_axes(const RopeAxesParams& p, int dtype, int head_dim, bool halves, cudaStream_t s) {
  if (p.n_tok == 0 || p.x[0].heads + p.x[1].heads == 0) return cudaSuccess;
  switch (dtype * 2 + (head_dim == 128)) {
    case RC_BF16 * 2: return rope_d<RC_BF16, 64>(p, halves, s);
    case RC_BF16 * 2 + 1: return rope_d<RC_BF16, 128>(p, halves, s);
    case RC_F16 * 2: return rope_d<RC_F16, 64>(p, halves, s);
    case RC_F16 * 2 + 1: return rope_d<RC_F16, 128>(p, halves, s);
    case RC_F32 * 2: return rope_d<RC_F32, 64>(p, halves, s);
    default: return rope_d<RC_F32, 128>(p, halves, s);
  }
}

cudaError_t launch_paged_append(const PagedAppendParams& p, int dtype, int head_dim, bool halves, cudaStream_t s) {
  if (p.n_tok == 0 || p.b.n_seqs == 0) return cudaSuccess;
  switch (dtype * 2 + (head_dim == 128)) {
    case RC_BF16 * 2: return append_d<RC_BF16, 64>(p, halves, s);
    case RC_BF16 * 2 + 1: return append_d<RC_BF16, 128>(p, halves, s);
    case RC_F16 * 2: return append_d<RC_F16, 64>(p, halves, s);
    default: return append_d<RC_F16, 128>(p, halves, s);
  }
}

}  // namespace rc

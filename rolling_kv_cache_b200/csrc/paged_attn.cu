// Attention over pages for many query rows per key head (tcgen05 + TMEM + TMA):
// prompts, chunks of video frames, and a batch's queries against a shared
// prefix.
//
//   o = sum_j exp(x_j) v_j / sum_j exp(x_j),  x_j = scale q . k_j,
// over the keys the mask leaves, one pass, running maximum and sum. Bound by the tensor cores and
// the exponentials: 4 * head_dim operations and one exponential a pair.
//
// A unit of work is a pair of 128-row query tiles (Q0, Q1) of one key head,
// sharing every K/V tile. A tile's rows are (query, query head of the key
// head) pairs, query-major: 128 / G whole queries of G heads each, brought by one TMA box per
// 64 dims, so that shared key heads are read once for all their query heads.
//   warps 0-7   softmax of Q0 and epilogue: 32 query rows (TMEM lanes) x
//               64 keys per warp
//   warps 8-15  softmax of Q1, epilogue
//   warp 16     TMA producer: Q0/Q1 once per unit, K and V tiles (128 keys, a
//               box per page and 64 dims) into separate 2-stage rings
//   warp 17     TMEM allocator; one thread issues every tcgen05.mma
// TMEM (512 columns): S0 [0,128), S1 [128,256), O0 [256,256+d), O1 [384,384+d).
// P_i (16-bit) overwrites columns [0,32) and [64,96) of S_i and is the A operand of
// O_i += P_i V. MMA issue order per KV tile j: PV0(j), S0(j+1), PV1(j), S1(j+1),
// so that while one softmax group turns S into P the tensor core runs the
// other group's two products. P comes in two halves (the first and the last 32
// keys of each warp's 64), each with its barrier: PV of the first runs while the
// exponentials of the second do (video chunk 847 -> 818 us; a third step, 851).
//
// Measured: 4680 queries against 18 frames of 1560 keys, 12 heads of 128, 852 GFLOP:
// 912 us, 934 TFLOP/s back to back (835 us the first times, before the power cap); tensor
// pipe and exponentials are each 54 % busy, a tile's softmax (from S to P) being longer than
// the other tile's two products beside it.
//
// Schedule, found by every CTA from the lengths on the device: units in
// (sequence, key head, pair) order; CTA c of G first takes whole units c, c + G,
// ... for as many rounds as leave no CTA above the average of the whole
// batch's tiles (the pairs of a head then walk its K/V tiles together, which
// come from DRAM once), and the tiles of the units left over, in order, are
// cut into one range per CTA, sized so that every CTA's total is the
// average (units differ in length: ragged batches, causal and window masks).
// A unit cut between CTAs leaves its parts for the combine kernel.
//
// Keys that a query does not see are masked in S (-inf, written back to TMEM by a tile's softmax warps before
// they use it, in boundary tiles only); V rows behind the sequence or before the
// pair's windows are zeroed in shared memory before the product, so that what their bits hold stays out; pages that are none are
// filled with zeros by an out-of-range copy and masked.
//
// Every wait is bounded (2 s) and reports RC_ETIMEOUT through the status
// word; no trap.
#include "paged_common.cuh"

namespace rc {

namespace {

constexpr int kTileRows = 128;
constexpr uint32_t kSubTileBytes = 128 * 64 * 2;  // 128 rows x 64 dims = one 128-byte-swizzle box
constexpr int kSoftmaxWarps = 16;
constexpr int kProducerWarp = 16;
constexpr int kMmaWarp = 17;
constexpr int kPreThreads = 18 * 32;
constexpr float kRescaleLog2 = 8.0f;
// A row's reference c m is rounded, to R. Below this its rounding is at most 1, and the row's sums
// stand for what they are times 2^R; beyond, for that times 2^(c m), whose exponents take more steps (steep_scores).
constexpr float kSteepLog2 = 16777216.f;
constexpr int kMaxRounds = 64;
// What a unit costs beside its tiles, in tiles (its queries, its first tile's
// start and its last writes; ragged prompts 254 us with 1, 246 with 2, 3 or 4)
constexpr int kPairCost = 2;
constexpr int kPlanSeqs = 512;

template <int D>
struct PreLayout {
  static constexpr int kSub = D / 64;
  static constexpr uint32_t kTile = kSubTileBytes * kSub;
  static constexpr uint32_t kQ = 0;              // Q0, Q1
  static constexpr uint32_t kK = 2 * kTile;      // 2 stages
  static constexpr uint32_t kV = 4 * kTile;      // 2 stages
  static constexpr uint32_t kBytes = 6 * kTile;
  static constexpr uint32_t kDynSmem = kBytes + 1024;
  // the schedule's sums, gone before the first load: tiles (low half) and pairs
  // (high half) of the sequences before each, the first sequences themselves,
  // and each CTA's tiles after each round
  static constexpr uint32_t kBefore = 0;
  static constexpr uint32_t kSeqs = kBefore + ((kMaxSeqs + 1) * 8 + 15) / 16 * 16;
  static constexpr uint32_t kLoads = kSeqs + kPlanSeqs * 16;
  static_assert(kLoads + kMaxRounds * kMaxPersistentCtas * 4 <= kBytes, "the schedule fits the tiles' memory");
};

// KV tiles [kv_lo, kv_hi) of one pair of query tiles of key head h of
// sequence b. slot >= 0: the job covers part of its unit and leaves
// (O / l, its RowSum) in that slot; slot < 0: it writes the output.
struct Job {
  int b, h, q0;      // q0: row of q of the pair's first query
  int tokens, at0;   // queries of the pair, position of the first
  int L, kv_lo, kv_hi, slot;
  bool has1, head, tail;  // head: begins inside the unit; tail: ends inside it
  int lead, total;        // tiles of the prefix that it walks first, and in all
  TileSpan<kTileRows> sp;
};

// The batch as the kernel sees it: the sequences, or, in a pass over a shared
// prefix alone, one sequence of every query that sees the prefix whole (the host
// sets a frame beyond every position and no window).
__device__ __forceinline__ Seq pre_seq(const PagedAttnParams& p, int b) {
  if (p.batch_pass) {
    Seq s;
    const int n = __ldg(p.b.cu_q + p.b.n_seqs);
    s.q0 = 0;
    s.n = min(max(n, 0), p.n_tok);
    s.L = p.prefix_len;
    s.falls = s.bad = false;  // the pass over the sequences' own tokens reports
    return s;
  }
  return load_seq(p.b, p.n_tok, b);
}

__device__ __forceinline__ void pair_span(const PagedAttnParams& p, const Seq& s, int pair, int tpt, Job& j) {
  const int i0 = pair * 2 * tpt;
  j.tokens = min(2 * tpt, s.n - i0);
  j.at0 = (p.batch_pass ? 0 : s.L - s.n) + i0;
  j.sp.init(p.mask, j.at0, j.at0 + j.tokens - 1, s.L);
  j.lead = (p.lead_len + kTileRows - 1) / kTileRows;
  j.total = j.lead + j.sp.n;
}

// A unit as the softmax and MMA warps need it.
struct JobInfo {
  int tiles;              // its key tiles; -1: the last unit is past
  int two;                // it has a second query tile
  int tokens, q0, head0;  // queries, row of q of the first, query head of the tile's first row
  int at0, L, slot, lo_min, hi_max;
};
constexpr int kJobRing = 4;
constexpr int kLeadTile = 1 << 16;  // in a tile's page bits: it is the prefix's

// A unit, and a position within it: 0, or kPairCost + a tile after the first.
struct Start {
  int b, h, pair, off;
};

// This CTA's work: `rounds` whole units from `whole` on, G apart, then the
// positions [pos, end) of the batch, which begin at `range`; a unit of n tiles
// takes kPairCost + n. A bound that falls among a unit's cost is moved to the unit's
// start, alike for the CTAs on both sides.
struct Plan {
  Start whole, range;
  int rounds, pos, end;
};

struct PairWalk {
  const PagedAttnParams* p;
  int n_seqs, tpt, pos, end, rounds;
  int b, h, pair, off, pairs;
  Start range;
  Seq s;

  __device__ __forceinline__ void load() {
    s = pre_seq(*p, b);
    pairs = (s.n + 2 * tpt - 1) / (2 * tpt);
  }
  __device__ __forceinline__ void go(const Start& st) {
    b = st.b;
    h = st.h;
    pair = st.pair;
    off = st.off;
    load();
  }
  __device__ __forceinline__ void init(const PagedAttnParams& prm, const Plan& pl) {
    p = &prm;
    n_seqs = prm.batch_pass ? 1 : prm.b.n_seqs;
    tpt = kTileRows / prm.G;
    pos = pl.pos;
    end = pl.end;
    rounds = pl.rounds;
    range = pl.range;
    if (rounds > 0) go(pl.whole);
    else if (pos < end) go(range);
  }
  __device__ __forceinline__ bool next(Job& j) {
    if (rounds > 0) {
      pair_span(*p, s, pair, tpt, j);
      fill(j, 0, max(j.total, 1));
      if (--rounds > 0) {
        int i = h * pairs + pair + (int)gridDim.x;
        while (i >= p->Hk * pairs) {
          i -= p->Hk * pairs;
          ++b;
          load();
        }
        h = i / pairs;
        pair = i - h * pairs;
      } else if (pos < end) {
        go(range);
      }
      return true;
    }
    if (pos >= end) return false;
    while (pair >= pairs) {
      pair = 0;
      if (pairs == 0 || ++h == p->Hk) {
        h = 0;
        if (++b >= n_seqs) return false;
        load();
      }
    }
    pair_span(*p, s, pair, tpt, j);
    const int len = min(max(j.total, 1) + kPairCost - off, end - pos), lo = max(off - kPairCost, 0);
    fill(j, lo, off + len - kPairCost - lo);
    pos += len;
    off = 0;
    ++pair;
    return true;
  }
  __device__ __forceinline__ void fill(Job& j, int lo, int len) const {
    j.b = b;
    j.h = h;
    j.q0 = s.q0 + pair * 2 * tpt;
    j.L = s.L;
    j.kv_lo = lo;
    j.kv_hi = min(lo + len, j.total);
    j.has1 = j.tokens > tpt;
    j.head = lo > 0;
    j.tail = lo + len < max(j.total, 1);
    j.slot = j.head ? 2 * (int)blockIdx.x : (j.tail ? 2 * (int)blockIdx.x + 1 : -1);
  }
};

__device__ __forceinline__ int tiles_of(unsigned long long x) { return (int)(uint32_t)x; }
__device__ __forceinline__ int pairs_of(unsigned long long x) { return (int)(x >> 32); }

// The largest b < n with per * of(before[b]) <= x.
template <typename Fn>
__device__ __forceinline__ int last_at_most(const unsigned long long* before, int n, int per, int x, Fn of) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (per * of(before[mid]) <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The schedule, by all threads; `mem` is scratch as the layout lays it out.
template <int D>
__device__ __forceinline__ void make_plan(const PagedAttnParams& p, uint8_t* mem, unsigned long long* warp_sums,
                                          int* most, int* sums, Plan* plan) {
  using L = PreLayout<D>;
  unsigned long long* before = reinterpret_cast<unsigned long long*>(mem + L::kBefore);
  int4* seqs = reinterpret_cast<int4*>(mem + L::kSeqs);
  int* loads = reinterpret_cast<int*>(mem + L::kLoads);  // [round][CTA]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_seqs = p.b.n_seqs, tpt = kTileRows / p.G;
  const int G = gridDim.x, c = blockIdx.x;
  if (p.batch_pass) {
    // units all alike: no sums to take (3.1 us less of a short pass)
    if (tid == 0) {
      const Seq s = pre_seq(p, 0);
      const int pairs = (s.n + 2 * tpt - 1) / (2 * tpt), U = p.Hk * pairs;
      const int w = (p.prefix_len + kTileRows - 1) / kTileRows + kPairCost, W = U * w;
      const int rounds = min(U / G, kMaxRounds);
      auto bound = [&](int i, Start* at) {
        int x = (int)((long long)W * i / G) + rounds * w * (G - i);
        const int u = x / w, off = x - u * w;
        if (off <= kPairCost) x -= off;
        if (at && x < W) *at = Start{0, u / pairs, u % pairs, off <= kPairCost ? 0 : off};
        return x;
      };
      plan->rounds = rounds;
      if (rounds > 0) plan->whole = Start{0, c / pairs, c % pairs, 0};
      plan->pos = bound(c, &plan->range);
      plan->end = bound(c + 1, nullptr);
    }
    __syncthreads();
    return;
  }
  auto seq = [&](int b) {
    if (b >= kPlanSeqs) return load_seq(p.b, p.n_tok, b);
    const int4 x = seqs[b];
    return Seq{x.x, x.y, x.z, false, false};
  };
  if (tid < kMaxRounds) most[tid] = 0;
  if (tid < 3) sums[tid] = 0;
  __syncthreads();
  // tiles and pairs of each sequence (one key head), a warp a sequence
  for (int b = warp; b < n_seqs; b += kPreThreads / 32) {
    const Seq s = load_seq(p.b, p.n_tok, b);
    const int pairs = (s.n + 2 * tpt - 1) / (2 * tpt);
    int sum = 0;
    for (int q = lane; q < pairs; q += 32) {
      Job j;
      pair_span(p, s, q, tpt, j);
      sum += max(j.total, 1) + kPairCost;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      if (s.falls) sums[2] = 1;
      if (s.bad && p.status) atomicCAS(p.status, 0, (int)RC_ERANGE);  // also where it is left without a unit
      before[b] = (unsigned long long)pairs << 32 | (uint32_t)sum;
      if (b < kPlanSeqs) seqs[b] = make_int4(s.q0, s.n, s.L, 0);
    }
  }
  __syncthreads();
  block_prefix<kPreThreads>(before, n_seqs, warp_sums, [&](int b) { return before[b]; });
  const bool falls = sums[2];
  const int W = falls ? 0 : p.Hk * tiles_of(before[n_seqs]), U = falls ? 0 : p.Hk * pairs_of(before[n_seqs]);
  const int r_max = min(U / G, kMaxRounds);
  int rounds = 0, own = 0;
  if (r_max > 0) {
    // each CTA's tiles after each round, and the most any has
    for (int u = tid; u < r_max * G; u += kPreThreads) {
      const int b = last_at_most(before, n_seqs, p.Hk, u, pairs_of);
      const int first = pairs_of(before[b]);
      Job j;
      pair_span(p, seq(b), (u - p.Hk * first) % (pairs_of(before[b + 1]) - first), tpt, j);
      loads[u] = max(j.total, 1) + kPairCost;
    }
    __syncthreads();
    if (tid < G) {
      int load = 0;
      for (int r = 0; r < r_max; ++r) {
        load += loads[r * G + tid];
        loads[r * G + tid] = load;
        atomicMax(&most[r], load);
      }
    }
    __syncthreads();
    while (rounds < r_max && most[rounds] <= W / G) ++rounds;
    // range of this CTA: what brings it, and those before it, to the average
    if (rounds > 0 && tid < G) {
      const int load = loads[(rounds - 1) * G + tid];
      atomicAdd(&sums[0], load);
      if (tid < c) atomicAdd(&sums[1], load);
    }
    __syncthreads();
    if (rounds > 0) own = loads[(rounds - 1) * G + c];
  }
  if (warp == 0 && lane == 0) {
    plan->rounds = rounds;
    if (rounds > 0) {
      const int b = last_at_most(before, n_seqs, p.Hk, c, pairs_of);
      const int first = pairs_of(before[b]), pairs = pairs_of(before[b + 1]) - first, i = c - p.Hk * first;
      plan->whole = Start{b, i / pairs, i % pairs, 0};
    }
  }
  if (warp < 2) {  // the range's begin, and its end
    int x = warp == 0 ? (int)((long long)W * c / G) - sums[1] + sums[0]
                      : (int)((long long)W * (c + 1) / G) - sums[1] - own + sums[0];
    if (x < W) {
      const int b = last_at_most(before, n_seqs, p.Hk, x, tiles_of);
      const int w = tiles_of(before[b + 1]) - tiles_of(before[b]);
      const int rem = x - p.Hk * tiles_of(before[b]), h = rem / w;
      int left = rem - h * w;
      const Seq s = seq(b);
      const int pairs = pairs_of(before[b + 1]) - pairs_of(before[b]);
      for (int q0 = 0; q0 < pairs; q0 += 32) {
        int t = 0;
        if (q0 + lane < pairs) {
          Job j;
          pair_span(p, s, q0 + lane, tpt, j);
          t = max(j.total, 1) + kPairCost;
        }
        int inc = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        const int sum = __shfl_sync(0xffffffffu, inc, 31);
        if (left < sum) {
          const uint32_t here = __ballot_sync(0xffffffffu, left >= inc - t && left < inc);
          const int src = __ffs(here) - 1;
          int off = left - __shfl_sync(0xffffffffu, inc - t, src);
          if (off <= kPairCost) {
            x -= off;
            off = 0;
          }
          if (warp == 0 && lane == 0) plan->range = Start{b, h, q0 + src, off};
          break;
        }
        left -= sum;
      }
    }
    if (lane == 0) (warp == 0 ? plan->pos : plan->end) = x;
  }
}

// The masking of a boundary tile stays out of line, so that its registers are
// not the tile loop's.

// -inf over the scores of one row's 64 keys from h0 on (TMEM columns tS ..)
// that the row does not see or whose page is none; returns the largest other score.
__device__ __noinline__ float mask_scores(uint32_t tS, int h0, RowMask rm, int sink, uint32_t pages, int page_log2) {
  auto below = [](int x) { return x >= 64 ? ~0ull : (x <= 0 ? 0ull : (1ull << x) - 1); };
  unsigned long long v = below(rm.hi - h0) & (~below(rm.lo - h0) | below(sink - h0));
  const int step = min(64, 1 << page_log2);
  for (int k = 0; k < 64; k += step)
    if (!((pages >> (k >> page_log2)) & 1)) v &= ~(below(step) << k);
  float mx = -INFINITY;
#pragma unroll 1
  for (int cc = 0; cc < 2; ++cc) {
    const uint32_t vis = (uint32_t)(v >> (32 * cc));
    uint32_t r[32];
    ptx::tmem_ld32(tS + cc * 32, r);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 32; ++k) r[k] = (vis >> k) & 1u ? r[k] : 0xff800000u;
#pragma unroll
    for (int k = 0; k < 16; ++k) mx = ptx::fmax3(mx, __uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1]));
    if (!__all_sync(0xffffffffu, vis == 0xffffffffu)) ptx::tmem_st32(tS + cc * 32, r);
  }
  ptx::tmem_st_wait();
  return mx;
}

// c m - R of a row's reference (see kSteepLog2)
__device__ __forceinline__ float reference_gap(float m, float c) {
  const float r = m * c;
  return fabsf(r) < kSteepLog2 ? fmaf(m, c, -r) : 0.f;
}

// Writes the exponents of one row's 64 scores (TMEM columns tS ..) over them, where some row's of the warp
// is steep: the difference first, so that the product's rounding is relative to the exponent.
__device__ __noinline__ void steep_scores(uint32_t tS, float m, float c) {
  const float r = m * c;
  const bool steep = !(fabsf(r) < kSteepLog2);
#pragma unroll 1
  for (int cc = 0; cc < 64; cc += 16) {
    uint32_t s[16];
    ptx::tmem_ld16(tS + cc, s);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float x = __uint_as_float(s[k]);
      s[k] = __float_as_uint(steep ? (x - m) * c : fmaf(x, c, -r));
    }
    ptx::tmem_st16(tS + cc, s);
  }
  ptx::tmem_st_wait();
}

// Zeros the V rows of a tile (from key t0 on, one row to two threads) outside [lo, hi) and the sinks.
template <int D>
__device__ __noinline__ void zero_values(uint8_t* v, int t0, int lo, int hi, int sink) {
  const int row = (int)threadIdx.x >> 1, key = t0 + row;
  if (!(key < hi && (key >= lo || key < sink))) {
    uint8_t* dst = v + row * 128 + (threadIdx.x & 1) * 64;
#pragma unroll
    for (int k = 0; k < PreLayout<D>::kSub; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(dst + k * kSubTileBytes + i * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  ptx::fence_proxy_async_smem();
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kPreThreads, 1) paged_prefill_kernel(const __grid_constant__ PagedAttnParams p) {
  using L = PreLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bar_q, bar_qe, bar_kf[2], bar_vf[2], bar_ke[2], bar_ve[2], bar_s[2], bar_h[2], bar_p[2], bar_o[2],
      bar_fin, bar_pair[8];
  __shared__ float swap_buf[2][2][2][kTileRows];  // [group][exchange parity][column half][row]
  // what the softmax has to know of tile g, at g % 4: its first key, its pages
  // that are there (a bit each), whether every query sees all of it, whether it has V
  // rows behind the sequence or before the pair's windows
  __shared__ int4 tile_info[4];
  // the units' descriptions, written by the producer (which alone walks the
  // schedule: the walk's state in 18 warps' local memory would not fit L1)
  __shared__ JobInfo jobs[kJobRing];
  __shared__ uint64_t bar_jf[kJobRing], bar_je[kJobRing];
  __shared__ unsigned long long warp_sums[18];
  __shared__ int most[kMaxRounds], sums[3];
  __shared__ Plan plan;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base_u32 = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_u32 - ptx::smem_u32(smem_raw));

  if (threadIdx.x == 0) {
    ptx::mbar_init(&bar_q, 1);
    ptx::mbar_init(&bar_qe, 1);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&bar_kf[i], 1);
      ptx::mbar_init(&bar_vf[i], 1);
      ptx::mbar_init(&bar_ke[i], 1);
      ptx::mbar_init(&bar_ve[i], 1);
      ptx::mbar_init(&bar_s[i], 1);
      ptx::mbar_init(&bar_h[i], 256);
      ptx::mbar_init(&bar_p[i], 256);
      ptx::mbar_init(&bar_o[i], 1);
    }
    ptx::mbar_init(&bar_fin, 1);
    for (int i = 0; i < 8; ++i) ptx::mbar_init(&bar_pair[i], 64);
    for (int i = 0; i < kJobRing; ++i) {
      ptx::mbar_init(&bar_jf[i], 1);
      ptx::mbar_init(&bar_je[i], kSoftmaxWarps + 1);
    }
    abort_sh = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(&tmem_base_sh, 512);
    ptx::tmem_relinquish();
  }
  ptx::grid_launch_dependents();
  make_plan<D>(p, base, warp_sums, most, sums, &plan);
  ptx::fence_proxy_async_smem();  // the plan's scratch is where copies land
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  const int tpt = kTileRows / p.G;
  volatile int* abort = &abort_sh;
  int dummy_abort = 0;
  volatile int* noabort = reinterpret_cast<volatile int*>(&dummy_abort);
  if (warp == kProducerWarp) {
    // ---------------------------------------------------------- producer
    if (lane == 0) {
      ptx::tma_prefetch_desc(&p.tm_q);
      ptx::tma_prefetch_desc(&p.tm_k);
      ptx::tma_prefetch_desc(&p.tm_v);
    }
    int nq = 0, g = 0, nw = 0;
    PartRecord rec = make_int4(0, 0, 0, 0);
    PairWalk walk;
    walk.init(p, plan);
    Job jb;
    // K/V tiles are read by every pair of their head: keep them in L2; Q is read once
    const uint64_t pol_q = ptx::l2_policy(false), pol_kv = ptx::l2_policy(true);
    // a tile is `boxes` pages; a lane copies one page's 64 dims of K, then of V
    const int boxes = kTileRows >> p.b.page_log2;
    const int box = lane & (boxes - 1), plane = lane / boxes;
    const bool copies = plane < L::kSub;
    const uint32_t dst0 = plane * kSubTileBytes + (box << p.b.page_log2) * 128;
    int j = 0, n = 0, page = -1;
    bool ok = true, v_missing = false, want = false, fresh = false;
    // describes the next unit to the other warps; n < 0: there is none
    auto publish = [&](int tiles) {
      const int slot = nw % kJobRing;
      if (nw >= kJobRing) {
        ok = ptx::mbar_wait(&bar_je[slot], (nw / kJobRing - 1) & 1, abort, p.status, RC_ETIMEOUT);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
      }
      if (lane == 0) {
        jobs[slot] = JobInfo{tiles, jb.has1, jb.tokens, jb.q0, jb.h * p.G, jb.at0, jb.L, jb.slot, jb.sp.lo_min, jb.sp.hi_max};
        ptx::mbar_arrive(&bar_jf[slot]);
      }
      ++nw;
    };
    // the next tile, with the load of its page entry under way; fresh: it is its unit's first
    auto advance = [&]() -> bool {
      fresh = false;
      for (++j; j >= n;) {
        if (!walk.next(jb)) {
          publish(-1);
          return false;
        }
        if (jb.head) rec.x = kHasHead | (jb.tail ? 0 : kHeadEnds);
        else if (jb.tail) rec = make_int4(rec.x, jb.q0, jb.tokens, jb.h * p.G);
        j = jb.kv_lo;
        n = jb.kv_hi;
        fresh = true;
        publish(max(0, n - j));
        if (!ok) return false;
      }
      const int in_tile = box << p.b.page_log2;
      if (j < jb.lead) {
        const int k0 = j * kTileRows + in_tile;
        want = k0 < p.lead_len;
        page = want ? __ldg(p.lead_table + (k0 >> p.b.page_log2)) : -1;
      } else {
        const int k0 = jb.sp.key(j - jb.lead) + in_tile;
        want = k0 < jb.sp.hi_max &&
               (k0 + (1 << p.b.page_log2) > jb.sp.lo_min || (p.mask.window > 0 && k0 < p.mask.sink_tok));
        page = want ? __ldg(p.b.page_table + jb.b * p.b.table_stride + (k0 >> p.b.page_log2)) : -1;
      }
      return true;
    };
    for (bool more = advance(); more; ++g) {
      const int st = g & 1;
      const uint32_t free_par = ((g >> 1) - 1) & 1;
      const bool good = page >= 0 && page < p.b.n_pages;
      if (want && !good && p.status) atomicCAS(p.status, 0, (int)RC_ERANGE);
      const uint32_t pages = __ballot_sync(0xffffffffu, good) & 0xffu;
      const int pg = good ? page : p.b.n_pages;  // a page that is none: read out of bounds on purpose, zeros
      const int h = jb.h;
      const bool all = __all_sync(0xffffffffu, good);
      int4 info;
      if (j < jb.lead) {
        const int t0 = j * kTileRows, hidden = t0 + kTileRows > p.lead_len;
        info = make_int4(t0, (int)pages | kLeadTile, !hidden && all, hidden);
      } else {
        const int t0 = jb.sp.key(j - jb.lead), t1 = t0 + kTileRows;
        const bool in_sink = p.mask.window > 0 && t1 <= p.mask.sink_tok;
        info = make_int4(t0, (int)pages, t1 <= jb.sp.hi_min && (t0 >= jb.sp.lo_max || in_sink) && all,
                         !(t1 <= jb.L && (t0 >= jb.sp.lo_min || in_sink)));
      }
      if (fresh) {
        ok = nq == 0 || ptx::mbar_wait(&bar_qe, (nq - 1) & 1, abort, p.status, RC_ETIMEOUT);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          const int nt = jb.has1 ? 2 : 1;
          ptx::mbar_arrive_expect_tx(&bar_q, nt * L::kSub * tpt * p.G * 128);
          for (int i = 0; i < nt; ++i)
            for (int k = 0; k < L::kSub; ++k)
              ptx::tma_load_3d_hint(&p.tm_q, &bar_q, base + L::kQ + i * L::kTile + k * kSubTileBytes, 64 * k,
                                    h * p.G, jb.q0 + i * tpt, pol_q);
        }
        ++nq;
      }
      ok = g < 2 || ptx::mbar_wait(&bar_ke[st], free_par, abort, p.status, RC_ETIMEOUT);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (lane == 0) {
        // S of tile g - 2 is complete, issued after the P of tile g - 3: the
        // softmax is past tile g - 4, whose word this was
        tile_info[g & 3] = info;
        ptx::mbar_arrive_expect_tx(&bar_kf[st], L::kTile);
      }
      __syncwarp();
      if (copies)
        ptx::tma_load_4d_hint(&p.tm_k, &bar_kf[st], base + L::kK + st * L::kTile + dst0, 64 * plane, 0, h, pg, pol_kv);
      ok = g < 2 || ptx::mbar_wait(&bar_ve[st], free_par, abort, p.status, RC_ETIMEOUT);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        ++g;  // its K is in flight, its V is not
        v_missing = true;
        break;
      }
      if (lane == 0) ptx::mbar_arrive_expect_tx(&bar_vf[st], L::kTile);
      __syncwarp();
      if (copies)
        ptx::tma_load_4d_hint(&p.tm_v, &bar_vf[st], base + L::kV + st * L::kTile + dst0, 64 * plane, 0, h, pg, pol_kv);
      __syncwarp();
      // only with this tile's loads out: a unit is published once the fourth
      // before it is done, which may be this tile's when the units between are empty
      more = advance();
    }
    if (lane == 0) {
      p.rec[blockIdx.x] = rec;
      // never leave a copy in flight: wait (bounded, ignoring abort) for the last ones
      if (nq) ptx::mbar_wait(&bar_q, (nq - 1) & 1, noabort, p.status, RC_ETIMEOUT);
      for (int k = max(0, g - 2); k < g; ++k) {
        ptx::mbar_wait(&bar_kf[k & 1], (k >> 1) & 1, noabort, p.status, RC_ETIMEOUT);
        if (!(v_missing && k + 1 == g)) ptx::mbar_wait(&bar_vf[k & 1], (k >> 1) & 1, noabort, p.status, RC_ETIMEOUT);
      }
    }
  } else if (warp == kMmaWarp && lane == 0) {
    // ---------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc_s = ptx::idesc_f16(BF16, 128, 128, 0, 0);
    constexpr uint32_t idesc_o = ptx::idesc_f16(BF16, 128, D, 0, 1);
    const uint32_t sQ = base_u32 + L::kQ;
    auto issue_s = [&](int i, int st) {
      const uint32_t sQi = sQ + i * L::kTile;
      const uint32_t sK = base_u32 + L::kK + st * L::kTile;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t off = (ks >> 2) * kSubTileBytes + (ks & 3) * 32;
        ptx::mma_ss(tmem + i * 128, ptx::sdesc_sw128(sQi + off, 16, 1024), ptx::sdesc_sw128(sK + off, 16, 1024),
                    idesc_s, ks > 0);
      }
      ptx::mma_commit(&bar_s[i]);
    };
    // O_i += P_i V; committed for the epilogue after a job's last PV only (a
    // softmax that rescales O at tile j has waited for S_i(j), issued after PV_i(j-1))
    auto issue_pv = [&](int i, int st, int part, bool acc) {
      const uint32_t sV = base_u32 + L::kV + st * L::kTile;
      // P of keys [16 ks, 16 ks + 16): column (ks / 4) * 64 + (ks % 4) * 8 of S_i
#pragma unroll
      for (int k = 0; k < kTileRows / 32; ++k) {
        const int ks = (k >> 1) * 4 + part * 2 + (k & 1);
        ptx::mma_ts(tmem + 256 + i * 128, tmem + i * 128 + (ks >> 2) * 64 + (ks & 3) * 8,
                    ptx::sdesc_sw128(sV + ks * 2048, kSubTileBytes, 1024), idesc_o, acc || part > 0 || k > 0);
      }
    };
    int nq = 0, g = 0, gp[2] = {0, 0};
    bool ok = true;
    for (int nw = 0; ok; ++nw) {
      const int slot = nw % kJobRing;
      if (!ptx::mbar_wait(&bar_jf[slot], (nw / kJobRing) & 1, abort, p.status, RC_ETIMEOUT)) break;
      const int n = jobs[slot].tiles;
      const bool two = jobs[slot].two;
      ptx::mbar_arrive(&bar_je[slot]);
      if (n < 0) break;
      if (n == 0) continue;
      if (!ptx::mbar_wait(&bar_q, nq & 1, abort, p.status, RC_ETIMEOUT)) break;
      ++nq;
      if (!ptx::mbar_wait(&bar_kf[g & 1], (g >> 1) & 1, abort, p.status, RC_ETIMEOUT)) break;
      ptx::tc_fence_after();
      issue_s(0, g & 1);
      if (two) issue_s(1, g & 1);
      ptx::mma_commit(&bar_ke[g & 1]);
      if (n == 1) ptx::mma_commit(&bar_qe);
      for (int j = 0; j < n; ++j, ++g) {
        const int st = g & 1, st1 = (g + 1) & 1;
        const bool more = j + 1 < n;
        if (!ptx::mbar_wait(&bar_vf[st], (g >> 1) & 1, abort, p.status, RC_ETIMEOUT)) { ok = false; break; }
        if (!ptx::mbar_wait(&bar_h[0], gp[0] & 1, abort, p.status, RC_ETIMEOUT)) { ok = false; break; }
        ptx::tc_fence_after();
        issue_pv(0, st, 0, j > 0);
        if (!ptx::mbar_wait(&bar_p[0], gp[0] & 1, abort, p.status, RC_ETIMEOUT)) { ok = false; break; }
        ptx::tc_fence_after();
        issue_pv(0, st, 1, true);
        if (!more) ptx::mma_commit(&bar_o[0]);
        ++gp[0];
        if (!two) ptx::mma_commit(&bar_ve[st]);
        if (more) {
          if (!ptx::mbar_wait(&bar_kf[st1], ((g + 1) >> 1) & 1, abort, p.status, RC_ETIMEOUT)) { ok = false; break; }
          ptx::tc_fence_after();
          issue_s(0, st1);
          if (!two) {
            ptx::mma_commit(&bar_ke[st1]);
            if (j + 2 == n) ptx::mma_commit(&bar_qe);
          }
        }
        if (two) {
          if (!ptx::mbar_wait(&bar_h[1], gp[1] & 1, abort, p.status, RC_ETIMEOUT)) { ok = false; break; }
          ptx::tc_fence_after();
          issue_pv(1, st, 0, j > 0);
          if (!ptx::mbar_wait(&bar_p[1], gp[1] & 1, abort, p.status, RC_ETIMEOUT)) { ok = false; break; }
          ptx::tc_fence_after();
          issue_pv(1, st, 1, true);
          if (!more) ptx::mma_commit(&bar_o[1]);
          ++gp[1];
          ptx::mma_commit(&bar_ve[st]);
          if (more) {
            issue_s(1, st1);
            ptx::mma_commit(&bar_ke[st1]);
            if (j + 2 == n) ptx::mma_commit(&bar_qe);
          }
        }
      }
    }
    ptx::mma_commit(&bar_fin);
    ptx::mbar_wait(&bar_fin, 0, noabort, p.status, RC_ETIMEOUT);
  } else if (warp < kSoftmaxWarps) {
    // ---------------------------------------------------------- softmax
    // group g = warp / 8 owns query tile g. Warp w reads TMEM lane quarter
    // w % 4 (32 rows) and column half ch = (w / 4) % 2: keys [64 ch, 64 ch + 64)
    // of S and output columns [ch D/2, ch D/2 + D/2) of O. The two warps of a
    // row block (partners) swap their partial row maxima every tile and their
    // partial row sums once per unit through shared memory and a 64-thread
    // mbarrier.
    const int grp = warp >> 3;
    const int ch = (warp >> 2) & 1;
    const int wq = warp & 3;
    const int row = wq * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + grp * 128 + ch * 64;
    const uint32_t tO = tmem + lane_off + 256 + grp * 128 + ch * (D / 2);
    uint64_t* pbar = &bar_pair[grp * 4 + wq];
    const float c = p.scale_log2;
    const float thresh = kRescaleLog2 / c;
    int gs = 0;  // this group's tiles so far (phase of bar_s / bar_p)
    int gt = 0;  // the CTA's tiles so far (stage of K and V)
    int nj = 0;  // this group's jobs so far (phase of bar_o: one commit per job)
    int nx = 0;  // partner exchanges so far (phase of pbar, slot of swap_buf)
    bool alive = true;
    // A bounded wait, with one answer for the warp: lanes that gave up alone would leave
    // the others at the next warp-wide step for good (and a warp that is whole again
    // after each wait runs faster: video chunk 819 -> 811 us)
    auto wait = [&](uint64_t* bar, int phase) {
      alive = __all_sync(0xffffffffu, ptx::mbar_wait(bar, phase & 1, abort, p.status, RC_ETIMEOUT));
      return alive;
    };
    // writes v, returns the partner's value
    auto swap = [&](float v, float& other) -> bool {
      float(*buf)[128] = swap_buf[grp][nx & 1];
      buf[ch][row] = v;
      ptx::mbar_arrive(pbar);
      if (!wait(pbar, nx)) return false;
      ++nx;
      other = buf[ch ^ 1][row];
      return true;
    };
    for (int nw = 0;; ++nw) {
      const int slot = nw % kJobRing;
      if (!wait(&bar_jf[slot], nw / kJobRing)) break;
      const JobInfo& jb = jobs[slot];
      const int n_tiles = jb.tiles;
      if (n_tiles < 0) break;
      if (grp == 1 && !jb.two) {
        gt += n_tiles;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bar_je[slot]);
        continue;
      }
      float m = -INFINITY, l = 0.f;  // l: this half's share of the row sum
      bool steep = false;            // some row of the warp is (kSteepLog2)
      for (int left = n_tiles; left > 0; --left) {
        if (!wait(&bar_s[grp], gs)) break;
        ptx::tc_fence_after();
        const int4 info = tile_info[gt & 3];
        uint32_t ra[32];
        float mx = -INFINITY;
        if (info.z) {
          // S in halves, read again for the exponentials: 32 scores at a time leave
          // the loop's state in registers
          ptx::tmem_ld32(tS, ra);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 16; ++k) mx = ptx::fmax3(mx, __uint_as_float(ra[2 * k]), __uint_as_float(ra[2 * k + 1]));
          ptx::tmem_ld32(tS + 32, ra);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 16; ++k) mx = ptx::fmax3(mx, __uint_as_float(ra[2 * k]), __uint_as_float(ra[2 * k + 1]));
        } else {
          // some key of the tile is hidden from some row: those scores become
          // -inf in TMEM, and the rest of the tile's work needs no mask. Rows of no
          // query take the widest mask
          RowMask rm{jb.lo_min, jb.hi_max};
          const int qi = grp * tpt + row / p.G;  // this row's query within the pair
          const bool lead = info.y & kLeadTile;
          if (lead) rm = RowMask{0, p.lead_len};
          else if (row < tpt * p.G && qi < jb.tokens) rm = row_mask(p.mask, jb.at0 + qi, jb.L);
          mx = mask_scores(tS, info.x + ch * 64, rm, p.mask.window > 0 && !lead ? p.mask.sink_tok : 0,
                           (uint32_t)info.y >> ((ch * 64) >> p.b.page_log2), p.b.page_log2);
        }
        float mo;
        if (!swap(mx, mo)) break;
        const float m_new = ptx::fmax3(m, mx, mo);
        const bool need = m_new > m + thresh;      // also true for the first visible tile
        const bool real = need && m != -INFINITY;  // O already holds weighted values
        if (__any_sync(0xffffffffu, need)) {
          if (__any_sync(0xffffffffu, real)) {
            // PV of the previous tile is complete: it was issued before this
            // tile's S, which the wait above saw complete
            const float alpha = real ? ptx::ex2(fmaf(m - m_new, c, reference_gap(m_new, c) - reference_gap(m, c))) : 1.f;
#pragma unroll
            for (int cc = 0; cc < D / 64; ++cc) {
              uint32_t o[32];
              ptx::tmem_ld32(tO + cc * 32, o);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
              ptx::tmem_st32(tO + cc * 32, o);
            }
            ptx::tmem_st_wait();
            l *= alpha;
          }
          if (need) m = m_new;
          // rows of no query hold anything: they do not count
          steep = __any_sync(0xffffffffu, m != -INFINITY && !(fabsf(m * c) < kSteepLog2) && row < tpt * p.G);
        }
        // P = 2^(s c - R), R = c m rounded, as packed 16-bit pairs over the first 32 columns of
        // this half of S (already read): keys h0 + 2i, h0 + 2i + 1 -> column i. One
        // rounding, relative to the exponent; what R is off by is the same for the row's sums, and
        // put right where they meet others (with (s - m) c for all, video chunk 912 -> 930 us).
        // P is rounded to the values' type, the product's operand: off by at most
        // 2^-8 (bf16) or 2^-11 (fp16) of each weight; the sum l is taken before it.
        // Every exponential is the SFU's: with one pair in eight or two on the FMA pipe the
        // video chunk takes 834 and 835 us instead of 819 (head_dim 128; 64, which has half the products
        // to as many exponentials, was not measured)
        const float ref = m == -INFINITY ? 0.f : m;
        float ce = c, re = ref * c;
        if (steep) {
          steep_scores(tS, ref, c);
          ce = 1.f;
          re = 0.f;
        }
        float sum = 0.f;
        auto emit = [&](const uint32_t (&r)[32], int k0) {
          uint32_t pk[16];
          const float2 c2 = make_float2(ce, ce), nr2 = make_float2(-re, -re);
          float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 x =
                ptx::ffma2(make_float2(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1])), c2, nr2);
            const float2 e = make_float2(ptx::ex2(x.x), ptx::ex2(x.y));
            s2 = ptx::fadd2(s2, e);
            pk[k] = ptx::pack16x2<BF16>(e.x, e.y);
          }
          sum += s2.x + s2.y;
          ptx::tmem_st16(tS + k0 / 2, pk);
        };
        ptx::tmem_ld32(tS, ra);
        ptx::tmem_ld_wait();
        emit(ra, 0);
        // V rows behind the sequence or before the windows may hold anything: zero, before group 0's P lets the
        // product start (a key that only later queries see is data, and meets P = 0)
        if (grp == 0 && tile_info[gt & 3].w) {
          const int st = gt & 1;
          if (!wait(&bar_vf[st], gt >> 1)) break;
          const int4 info = tile_info[gt & 3];
          const bool lead = info.y & kLeadTile;
          zero_values<D>(base + L::kV + st * L::kTile, info.x, lead ? 0 : jb.lo_min, lead ? p.lead_len : jb.L,
                         p.mask.window > 0 && !lead ? p.mask.sink_tok : 0);
        }
        ptx::tmem_ld32(tS + 32, ra);
        ptx::tmem_st_wait();
        ptx::tmem_ld_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(&bar_h[grp]);
        emit(ra, 32);
        ptx::tmem_st_wait();
        l += sum;
        ptx::tc_fence_before();
        ptx::mbar_arrive(&bar_p[grp]);
        ++gs;
        ++gt;
      }
      // epilogue: O / l to the output (or, fp32 with its RowSum, to the prefix
      // pass's result or to this CTA's partial slot); each warp writes its D/2 columns
      float l_other = 0.f;
      if (!alive || !swap(l, l_other)) break;
      const float lt = l + l_other;
      const bool have_o = n_tiles > 0;
      if (have_o && !wait(&bar_o[grp], nj)) break;
      nj += have_o;
      ptx::tc_fence_after();
      // a row that saw nothing has l = 0: zeros and -inf; a NaN sum stays NaN
      const bool none = lt == 0.f;
      const float inv_l = none ? 0.f : 1.f / lt;
      const int qi = grp * tpt + row / p.G, tok = jb.q0 + qi, head = jb.head0 + row % p.G;
      const bool live = row < tpt * p.G && qi < jb.tokens;
      const float a = have_o ? inv_l : 0.f;
      uint8_t* dst;  // this warp's half of the row
      RowSum* dst_sum = nullptr;
      const bool f32 = jb.slot >= 0 || p.pre_o;
      if (jb.slot >= 0) {
        const size_t at = (size_t)jb.slot * kPrefillRows + grp * kTileRows + row;
        dst = reinterpret_cast<uint8_t*>(p.part_o + at * D) + ch * (D * 2);
        dst_sum = p.part_sum + at;
      } else if (p.pre_o) {
        dst = reinterpret_cast<uint8_t*>(p.pre_o + ((size_t)tok * p.Hk * p.G + head) * D) + ch * (D * 2);
        dst_sum = p.pre_sum + (size_t)head * p.n_tok + tok;
      } else {
        dst = p.out.data + tok * p.out.tok_stride + head * p.out.head_stride + ch * D;
      }
      const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;  // fp32 rows always are
      // the job's words are read: its slot is free (before the stores, which an
      // arrive behind them would wait for)
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bar_je[slot]);
      if (live && ch == 0) {
        const RowSum sum = make_float2(m, lt * ptx::ex2(-reference_gap(m, c)));
        if (f32) *dst_sum = sum;
        else if (p.lse) p.lse[(size_t)head * p.n_tok + tok] = row_lse2(sum, c) * 0.69314718055994531f;
      }
#pragma unroll 4
      for (int cc = 0; cc < D / 2; cc += 16) {
        uint32_t o[16];
        if (have_o) {
          ptx::tmem_ld16(tO + cc, o);
          ptx::tmem_ld_wait();
        }
        if (!live) continue;
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = a != 0.f ? __float_as_uint(__uint_as_float(o[k]) * a) : 0u;
        if (f32) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = o[8 * k + e];
            ptx::stg8(dst + cc * 4 + 32 * k, y);
          }
        } else {
          uint32_t y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            y[e] = ptx::pack16x2<BF16>(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
          if (wide) {
            ptx::stg8(dst + cc * 2, y);
          } else {
            *reinterpret_cast<uint4*>(dst + cc * 2) = make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4*>(dst + cc * 2 + 16) = make_uint4(y[4], y[5], y[6], y[7]);
          }
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int D, bool BF16>
cudaError_t launch_d(const PagedAttnParams& p, cudaStream_t s) {
  static PerDevice attr_set;
  int done = 0;
  cudaError_t e = attr_set.get(&done, [](int, int* x) {
    *x = 1;
    return cudaFuncSetAttribute(paged_prefill_kernel<D, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)PreLayout<D>::kDynSmem);
  });
  if (e != cudaSuccess) return e;
  return launch_chained(paged_prefill_kernel<D, BF16>, p, dim3(p.n_ctas), kPreThreads, PreLayout<D>::kDynSmem,
                        false, s);
}

}  // namespace

cudaError_t launch_paged_prefill(const PagedAttnParams& p, bool bf16, int head_dim, cudaStream_t s) {
  if (head_dim == 64) return bf16 ? launch_d<64, true>(p, s) : launch_d<64, false>(p, s);
  return bf16 ? launch_d<128, true>(p, s) : launch_d<128, false>(p, s);
}

}  // namespace rc

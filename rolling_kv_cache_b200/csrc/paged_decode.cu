// Attention over pages for few query rows per key head (rows = queries of a
// sequence x query heads of a key head <= 16): single tokens, short drafts.
//
//   o = sum_j exp(x_j) v_j / sum_j exp(x_j),  x_j = scale q . k_j,
// over the keys the mask leaves, in one pass with the running maximum and
// sum. Every key and value is read once for all the rows of its key head, so
// the bound is HBM: 2 * keys * head_dim * 2 bytes per (sequence, key head).
//
// The units (sequence, key head) are cut into 64-key tiles, and the tiles of
// the whole batch, in order, into one range per CTA (one CTA per SM), equal to
// a tile, a unit's start and end counted as kUnitCost more: a ragged batch and a single long
// sequence keep every SM reading alike. Each CTA finds its range from the lengths on the device. A unit cut
// between CTAs leaves parts for the combine kernel. Or, for few short units (CLUSTER), each unit's
// tiles are shared equally by the CTAs of a cluster, whose first merges the others' results
// out of their shared memory.
//
// Two warps (one for K, one for V) issue TMA copies of the tiles' pages (a box per page, its 64-dim
// planes one after the other, 128-byte swizzle) into a ring of 128 KB, running ahead across units, so
// that about that much of HBM reads is in flight per SM. Two groups of four warps
// take alternate tiles; a warp owns 16 keys of its tile: S = Q K^T and O += P V
// by warp-level 16 x 8 x 16 matrix steps on ldmatrix fragments (the 16 rows
// are the padded query rows; with so few rows a tcgen05 tile of 128 would be
// nearly all padding), with its own running maximum, sum and O, so that no warp waits
// for another within a unit. At a unit's end the eight warps' results meet
// in shared memory in a fixed order.
//
// Measured: 64 streams of 300 to 16384 tokens, 8 key heads of 128: 2.19 GB in 331 us,
// 6.6 TB/s, the copy rate. A tile takes its group of warps 1500 cycles, a unit 5000
// more (its place and lengths 1400, its queries 900, its merge and write 2700),
// which the ring hides from HBM but not in units of a tile or two. 12 heads of
// one stream of 777 tokens, in clusters of 8: 6.6 us.
//
// Rows of a tile that no query of the unit sees (behind the sequence, before
// the window, on a page that is not one) get weight 0 and their V fragments
// are zeroed, so whatever their bits hold, NaN included, stays out.
#include "paged_common.cuh"

namespace rc {

namespace {

constexpr int kTK = 64;                       // keys per tile
constexpr int kConsumers = 8;                 // warps
constexpr int kDecThreads = (kConsumers + 2) * 32;  // and two producers
constexpr int kRingBytes = 128 * 1024;
constexpr float kDecRescaleLog2 = 8.f;
// What a unit costs beside its tiles, in tiles (its queries, its merge and its
// writes: 5000 cycles to a tile's 1500)
constexpr int kUnitCost = 3;
constexpr int kMaxCluster = 8;

template <int D>
struct DecLayout {
  static constexpr int kSub = D / 64;
  static constexpr uint32_t kTile = kTK * 128 * kSub;    // K or V of a tile: [box][64-dim plane][box row][128 bytes]
  static constexpr uint32_t kStage = 2 * kTile;
  static constexpr int kStages = kRingBytes / kStage;    // 4 at d = 128, 8 at d = 64
  // Tiles alternate between the two groups of warps, so an even number of
  // stages gives each stage to one group. With an odd number a group that waits
  // for its tile in a stage whose last tile, the other group's, has not
  // landed would see the completed phase before that one, of the same parity,
  // and go on with stale data.
  static_assert(kStages % 2 == 0, "a stage belongs to one group of warps");
  static constexpr int kOPad = D + 8;                    // row stride of a merge buffer: spreads rows over banks
  static constexpr uint32_t kMerge = kRingBytes;         // 4 buffers [16][kOPad] fp32
  static constexpr uint32_t kPre = kMerge + 4 * 16 * kOPad * 4;
  static constexpr uint32_t kBytes = kPre + (kMaxSeqs + 1) * 4;
  static constexpr uint32_t kDynSmem = kBytes + 1024;
};

struct DecUnit {
  int b, h, lo, hi, total;  // tiles [lo, hi) of the unit's `total`
};

// Walks the units of positions [pos, end): a unit of w tiles takes kUnitCost + w
// positions, and position Hk * pre[b] + h * (pre[b + 1] - pre[b]) is the first of head h of
// sequence b. A range that begins or ends among a unit's cost is moved to the
// unit's start, alike for the CTAs on both sides.
struct DecWalk {
  const int* pre;
  int Hk, pos, end, b;
  __device__ __forceinline__ int at(int x, int n, int* seq) const {
    int lo = 0, hi = n - 1;
    while (lo < hi) {  // the largest b with Hk * pre[b] <= x
      const int mid = (lo + hi + 1) >> 1;
      if (Hk * pre[mid] <= x) lo = mid;
      else hi = mid - 1;
    }
    *seq = lo;
    if (x >= Hk * pre[n]) return x;
    const int off = (x - Hk * pre[lo]) % (pre[lo + 1] - pre[lo]);
    return off <= kUnitCost ? x - off : x;
  }
  __device__ __forceinline__ void init(const int* pre_, int n, int Hk_, int pos_, int end_) {
    pre = pre_;
    Hk = Hk_;
    int unused;
    end = at(end_, n, &unused);
    pos = at(pos_, n, &b);
  }
  __device__ __forceinline__ bool next(DecUnit& u) {
    if (pos >= end) return false;
    while (Hk * pre[b + 1] <= pos) ++b;
    const int w = pre[b + 1] - pre[b], rem = pos - Hk * pre[b];
    u.b = b;
    u.h = rem / w;
    const int off = rem - u.h * w, len = min(w - off, end - pos);
    u.total = w - kUnitCost;
    u.lo = max(off - kUnitCost, 0);
    u.hi = max(off + len - kUnitCost, 0);
    pos += len;
    return true;
  }
};

template <int D, bool BF16, bool CLUSTER>
__global__ void __launch_bounds__(kDecThreads, 1) paged_decode_kernel(const __grid_constant__ PagedAttnParams p) {
  using L = DecLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bar_full[L::kStages], bar_empty[L::kStages];
  __shared__ uint32_t readable[L::kStages];  // bit i: page i of the stage's tile is one
  __shared__ float wm[2][kConsumers][16], wl[2][kConsumers][16];
  __shared__ int warp_sums[kConsumers + 2];
  __shared__ int abort_sh, falls_sh;
  __shared__ RowSum own_sum[16];  // CLUSTER: of this CTA's tiles
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* base = smem_raw + (((ptx::smem_u32(smem_raw) + 1023u) & ~1023u) - ptx::smem_u32(smem_raw));
  const uint32_t base_u32 = ptx::smem_u32(base);
  int* pre = reinterpret_cast<int*>(base + L::kPre);
  if (tid == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      ptx::mbar_init(&bar_full[i], 2);
      ptx::mbar_init(&bar_empty[i], 4);
    }
    abort_sh = 0;
    falls_sh = 0;
    ptx::fence_mbar_init();
  }
  __syncthreads();
  ptx::grid_launch_dependents();
  DecWalk walk;
  DecUnit u, mine;
  bool taken = false;
  const int lead = CLUSTER ? (p.lead_len + kTK - 1) / kTK : 0;  // the prefix's tiles
  if constexpr (CLUSTER) {
    // an equal share of one unit's tiles, a prefix's first
    const int unit = blockIdx.x / p.cluster, rank = blockIdx.x - unit * p.cluster;
    mine.b = unit / p.Hk;
    mine.h = unit - mine.b * p.Hk;
    const Seq s = load_seq(p.b, p.n_tok, mine.b);
    if (tid == 0 && s.bad && p.status) atomicCAS(p.status, 0, (int)RC_ERANGE);
    if (s.n == 0) return;  // the whole cluster
    TileSpan<kTK> sp;
    sp.init(p.mask, s.L - s.n, s.L - 1, s.L);
    mine.total = lead + sp.n;
    const int each = (mine.total + p.cluster - 1) / p.cluster;
    mine.lo = min(rank * each, mine.total);
    mine.hi = min(mine.lo + each, mine.total);
  } else {
    // tiles of each sequence, and this CTA's range of the batch's
    block_prefix<kDecThreads>(pre, p.b.n_seqs, warp_sums, [&](int b) {
      const Seq s = load_seq(p.b, p.n_tok, b);
      if (s.falls) falls_sh = 1;
      if (s.bad && p.status) atomicCAS(p.status, 0, (int)RC_ERANGE);  // also where it is left without a unit
      if (s.n == 0) return 0;
      TileSpan<kTK> sp;
      sp.init(p.mask, s.L - s.n, s.L - 1, s.L);
      return max(sp.n, 1) + kUnitCost;
    });
    const int W = falls_sh ? 0 : p.Hk * pre[p.b.n_seqs];
    const int pos = (int)((long long)W * blockIdx.x / gridDim.x);
    const int end = (int)((long long)W * (blockIdx.x + 1) / gridDim.x);
    walk.init(pre, p.b.n_seqs, p.Hk, pos, end);
  }
  auto next_unit = [&](DecUnit& v) {
    if constexpr (!CLUSTER) return walk.next(v);
    if (taken) return false;
    taken = true;
    v = mine;
    return true;
  };
  volatile int* abort = &abort_sh;

  if (warp >= kConsumers) {
    // ----------------------------------------------------------- producers
    const bool is_v = warp > kConsumers;
    const CUtensorMap* map = is_v ? &p.tm_v : &p.tm_k;
    if (lane == 0) ptx::tma_prefetch_desc(map);
    const uint64_t pol = ptx::l2_policy(false);
    // A tile is `boxes` runs of box_rows keys, each in one page; a lane copies one. Page
    // entries are loaded a batch at a time, as many tiles of one unit as 32 lanes
    // cover, and the next batch's behind this one's second copy, so that an empty ring
    // fills without a load's latency between the tiles (64 streams 354 -> 349 us, 200
    // short ones 94 -> 89)
    const int boxes = kTK / p.box_rows, in_batch = 32 / boxes;
    const int in_page = (1 << p.b.page_log2) - 1;
    const int box = lane & (boxes - 1), ahead = lane / boxes;
    const uint32_t dst0 = (is_v ? L::kTile : 0) + box * p.box_rows * 128 * L::kSub;
    struct Batch {
      int tiles, h;     // 0: there is no more
      int k0, page;     // this lane's box: its first key, its page entry
      uint32_t wanted;  // bit of a lane: its page is to be read
    };
    int g = 0, j = 0, n = 0;
    bool ok = true;
    PartRecord rec = make_int4(0, 0, 0, 0);
    TileSpan<kTK> sp;
    auto fetch = [&]() -> Batch {
      Batch t{0, 0, 0, -1, 0u};
      while (j >= n) {
        if (!next_unit(u)) return t;
        const Seq s = load_seq(p.b, p.n_tok, u.b);
        sp.init(p.mask, s.L - s.n, s.L - 1, s.L);
        if (CLUSTER) {
        } else if (u.lo > 0) rec.x = kHasHead | (u.hi == u.total ? kHeadEnds : 0);
        else if (u.hi < u.total) rec = make_int4(rec.x, s.q0, min(s.n, 16 / p.G), u.h * p.G);
        j = u.lo;
        n = min(u.hi, lead + sp.n);
      }
      t.tiles = min(in_batch, n - j);
      t.h = u.h;
      const bool pre = CLUSTER && j + ahead < lead;
      t.k0 = (pre ? (j + ahead) * kTK : sp.key(j + ahead - lead)) + box * p.box_rows;
      const bool want = ahead < t.tiles &&
                        (pre ? t.k0 < p.lead_len
                             : t.k0 < sp.hi_max && (t.k0 + p.box_rows > sp.lo_min ||
                                                    (p.mask.window > 0 && t.k0 < p.mask.sink_tok)));
      const int32_t* table = pre ? p.lead_table : p.b.page_table + u.b * p.b.table_stride;
      if (want) t.page = __ldg(table + (t.k0 >> p.b.page_log2));
      t.wanted = __ballot_sync(0xffffffffu, want);
      j += t.tiles;
      return t;
    };
    for (Batch now = fetch(); now.tiles > 0 && ok;) {
      Batch next{0, 0, 0, -1, 0u};
      for (int t = 0; t < now.tiles; ++t, ++g) {
        const int from = t * boxes + box;
        const int pg = __shfl_sync(0xffffffffu, now.page, from), row0 = __shfl_sync(0xffffffffu, now.k0, from) & in_page;
        const bool good = pg >= 0 && pg < p.b.n_pages;
        if (((now.wanted >> from) & 1u) && !good && p.status) atomicCAS(p.status, 0, (int)RC_ERANGE);
        const uint32_t pages = __ballot_sync(0xffffffffu, good);
        const int st = g % L::kStages;
        if (g >= L::kStages) {
          ok = ptx::mbar_wait(&bar_empty[st], (g / L::kStages - 1) & 1, abort, p.status, RC_ETIMEOUT);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        if (lane == 0) {
          if (!is_v) readable[st] = pages;
          ptx::mbar_arrive_expect_tx(&bar_full[st], L::kTile);
        }
        __syncwarp();
        // a page that is none is read out of bounds on purpose: the copy fills zeros
        if (lane < boxes)
          ptx::tma_load_5d_hint(map, &bar_full[st], base + st * L::kStage + dst0, 0, good ? row0 : 0, 0, now.h,
                                good ? pg : p.b.n_pages, pol);
        __syncwarp();
        if (t == min(1, now.tiles - 1)) next = fetch();  // not before the first copies: the walk would hold them up
      }
      now = next;
    }
    if (lane == 0) {
      if (!CLUSTER && !is_v) p.rec[blockIdx.x] = rec;
      // leave no copy in flight (bounded, whether or not the others gave up)
      int dummy = 0;
      for (int k = max(0, g - L::kStages); k < g; ++k)
        ptx::mbar_wait(&bar_full[k % L::kStages], (k / L::kStages) & 1, &dummy, p.status, RC_ETIMEOUT);
      if (!is_v) ptx::grid_wait();  // in a chain, this grid ends after the one before it
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int grp = warp >> 2, kw = (warp & 3) * 16;  // this warp's keys of its group's tiles
  const int r0 = lane >> 2, r1 = r0 + 8, cq = (lane & 3) * 2;
  // the warp's 16 keys lie in one box: its start, their first row in it, and the box's plane stride
  const uint32_t plane = p.box_rows * 128, box0 = (kw / p.box_rows) * plane * L::kSub;
  const int krow0 = kw & (p.box_rows - 1);
  const float c = p.scale_log2, thresh = kDecRescaleLog2 / c;
  const int i0 = r0 / p.G, i1 = r1 / p.G, h0 = r0 - i0 * p.G, h1 = r1 - i1 * p.G;  // query and head of the rows
  int g = 0, nu = 0;
  bool alive = true;  // a warp whose wait gave up still meets the others at the merges' barriers
  // A unit's Q fragments (rows r0 and r1, zero behind the last row). The next
  // unit's sequence is loaded before the current one's tiles and its Q before the
  // current one's merge, which hides their latencies
  Seq s;
  uint32_t qf[D / 16][4];
  auto fetch = [&](const DecUnit& v, const Seq& sv, uint32_t (&f)[D / 16][4]) {
    const int rows = min(sv.n, 16 / p.G) * p.G;
    const uint8_t* q0 = p.q.data + (sv.q0 + i0) * p.q.tok_stride + (v.h * p.G + h0) * p.q.head_stride + cq * 2;
    const uint8_t* q1 = p.q.data + (sv.q0 + i1) * p.q.tok_stride + (v.h * p.G + h1) * p.q.head_stride + cq * 2;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      f[k][0] = r0 < rows ? __ldg(reinterpret_cast<const uint32_t*>(q0 + k * 32)) : 0u;
      f[k][1] = r1 < rows ? __ldg(reinterpret_cast<const uint32_t*>(q1 + k * 32)) : 0u;
      f[k][2] = r0 < rows ? __ldg(reinterpret_cast<const uint32_t*>(q0 + k * 32 + 16)) : 0u;
      f[k][3] = r1 < rows ? __ldg(reinterpret_cast<const uint32_t*>(q1 + k * 32 + 16)) : 0u;
    }
  };
  bool more = next_unit(u);
  if (more) {
    s = load_seq(p.b, p.n_tok, u.b);
    fetch(u, s, qf);
  }
  while (more) {
    DecUnit un = u;
    Seq sn = s;
    more = next_unit(un);
    if (more) sn = load_seq(p.b, p.n_tok, un.b);
    TileSpan<kTK> sp;
    sp.init(p.mask, s.L - s.n, s.L - 1, s.L);
    const int nq = min(s.n, 16 / p.G), R = nq * p.G;
    if (nq < s.n && tid == 0 && p.status) atomicCAS(p.status, 0, (int)RC_ERANGE);
    const RowMask m0 = row_mask(p.mask, s.L - s.n + i0, s.L), m1 = row_mask(p.mask, s.L - s.n + i1, s.L);
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float mx0 = -INFINITY, mx1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    const int n = min(u.hi, lead + sp.n);
    for (int j = u.lo; j < n && alive; ++j, ++g) {
      if ((g & 1) != grp) continue;
      const int st = g % L::kStages;
      alive = ptx::mbar_wait(&bar_full[st], (g / L::kStages) & 1, abort, p.status, RC_ETIMEOUT);
      alive = __all_sync(0xffffffffu, alive);
      if (!alive) break;
      const bool pre = CLUSTER && j < lead;
      const int t0 = pre ? j * kTK : sp.key(j - lead), w0 = t0 + kw;
      const uint32_t sK = base_u32 + st * L::kStage, sV = sK + L::kTile;
      float x[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      {
        const int row = krow0 + (lane >> 4) * 8 + (lane & 7);
        const uint32_t a = sK + box0 + row * 128;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t kf[4];
          ptx::ldsm4(kf, a + (k >> 2) * plane + ((((k & 3) * 2 + ((lane >> 3) & 1)) ^ (row & 7)) << 4));
          ptx::mma16816<BF16>(x[0], qf[k], kf[0], kf[1]);
          ptx::mma16816<BF16>(x[1], qf[k], kf[2], kf[3]);
        }
      }
      // keep: bit pairs of this lane's 4 keys (w0 + cq, +1, +8, +9) that some row sees
      const uint32_t pages = readable[st];
      const bool whole = (pre ? w0 + 16 <= p.lead_len
                              : w0 + 16 <= sp.hi_min &&
                                    (w0 >= sp.lo_max || (p.mask.window > 0 && w0 + 16 <= p.mask.sink_tok))) &&
                         ((pages >> (kw / p.box_rows)) & 1u);
      uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
      if (!whole) {
        const bool page_ok = (pages >> (kw / p.box_rows)) & 1u;  // a warp's 16 keys lie in one page
        const int sink = p.mask.window > 0 ? p.mask.sink_tok : 0;
        uint32_t kb[2] = {0u, 0u};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = w0 + i * 8 + cq + e;
            const bool v0 = page_ok && (pre ? key < p.lead_len : key < m0.hi && (key >= m0.lo || key < sink));
            const bool v1 = page_ok && (pre ? key < p.lead_len : key < m1.hi && (key >= m1.lo || key < sink));
            if (!v0) x[i][e] = -INFINITY;
            if (!v1) x[i][2 + e] = -INFINITY;
            if (page_ok && (pre ? key < p.lead_len : key < sp.hi_max && (key >= sp.lo_min || key < sink)))
              kb[i] |= 0xffffu << (16 * e);
          }
        keep0 = kb[0];
        keep1 = kb[1];
      }
      float t_0 = ptx::fmax3(fmaxf(x[0][0], x[0][1]), x[1][0], x[1][1]);
      float t_1 = ptx::fmax3(fmaxf(x[0][2], x[0][3]), x[1][2], x[1][3]);
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        t_0 = fmaxf(t_0, __shfl_xor_sync(0xffffffffu, t_0, d));
        t_1 = fmaxf(t_1, __shfl_xor_sync(0xffffffffu, t_1, d));
      }
      // the maximum moves only when it grows by more than 2^8: numerator and
      // denominator share the stale one, and P stays below 256
      const bool n0 = t_0 > mx0 + thresh, n1 = t_1 > mx1 + thresh;
      if (__any_sync(0xffffffffu, n0 || n1)) {
        const float a0 = n0 ? ptx::ex2((mx0 - t_0) * c) : 1.f, a1 = n1 ? ptx::ex2((mx1 - t_1) * c) : 1.f;
        if (n0) mx0 = t_0;
        if (n1) mx1 = t_1;
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= a0;
          o[i][1] *= a0;
          o[i][2] *= a1;
          o[i][3] *= a1;
        }
      }
      // the difference first: the product's rounding is then relative to the exponent, whatever c is
      const float b0 = mx0 == -INFINITY ? 0.f : mx0, b1 = mx1 == -INFINITY ? 0.f : mx1;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[i][0] = ptx::ex2((x[i][0] - b0) * c);
        x[i][1] = ptx::ex2((x[i][1] - b0) * c);
        x[i][2] = ptx::ex2((x[i][2] - b1) * c);
        x[i][3] = ptx::ex2((x[i][3] - b1) * c);
      }
      l0 += (x[0][0] + x[0][1]) + (x[1][0] + x[1][1]);
      l1 += (x[0][2] + x[0][3]) + (x[1][2] + x[1][3]);
      // P is rounded to the values' type, the matrix step's operand: off by at
      // most 2^-8 (bf16) or 2^-11 (fp16) of each weight; the sums l are not
      const uint32_t pf[4] = {ptx::pack16x2<BF16>(x[0][0], x[0][1]), ptx::pack16x2<BF16>(x[0][2], x[0][3]),
                              ptx::pack16x2<BF16>(x[1][0], x[1][1]), ptx::pack16x2<BF16>(x[1][2], x[1][3])};
      {
        const int row = krow0 + (lane & 15);
        const uint32_t a = sV + box0 + row * 128;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t vf[4];
          ptx::ldsm4_t(vf, a + (k >> 2) * plane + ((((k & 3) * 2 + (lane >> 4)) ^ (row & 7)) << 4));
          ptx::mma16816<BF16>(o[2 * k], pf, vf[0] & keep0, vf[1] & keep1);
          ptx::mma16816<BF16>(o[2 * k + 1], pf, vf[2] & keep0, vf[3] & keep1);
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bar_empty[st]);
    }
    const DecUnit done = u;
    const Seq ds = s;
    u = un;
    s = sn;
    if (more) fetch(u, s, qf);
    // ------------------------------------------------- merge of the 8 warps
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    float(*um)[16] = wm[nu & 1];
    float(*ul)[16] = wl[nu & 1];
    ++nu;
    if ((lane & 3) == 0) {
      um[warp][r0] = mx0;
      um[warp][r1] = mx1;
      ul[warp][r0] = l0;
      ul[warp][r1] = l1;
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    float* buf = reinterpret_cast<float*>(base + L::kMerge) + (warp & 3) * 16 * L::kOPad;
    float g0 = -INFINITY, g1 = -INFINITY;
#pragma unroll
    for (int w = 0; w < kConsumers; ++w) {
      g0 = fmaxf(g0, um[w][r0]);
      g1 = fmaxf(g1, um[w][r1]);
    }
    const float f0 = mx0 == -INFINITY ? 0.f : ptx::ex2((mx0 - g0) * c);
    const float f1 = mx1 == -INFINITY ? 0.f : ptx::ex2((mx1 - g1) * c);
    if (warp >= 4) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        if (r0 < R) *reinterpret_cast<float2*>(buf + r0 * L::kOPad + i * 8 + cq) = make_float2(o[i][0] * f0, o[i][1] * f0);
        if (r1 < R) *reinterpret_cast<float2*>(buf + r1 * L::kOPad + i * 8 + cq) = make_float2(o[i][2] * f1, o[i][3] * f1);
      }
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (warp < 4) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        if (r0 < R) {
          float2* d = reinterpret_cast<float2*>(buf + r0 * L::kOPad + i * 8 + cq);
          *d = make_float2(fmaf(o[i][0], f0, d->x), fmaf(o[i][1], f0, d->y));
        }
        if (r1 < R) {
          float2* d = reinterpret_cast<float2*>(buf + r1 * L::kOPad + i * 8 + cq);
          *d = make_float2(fmaf(o[i][2], f1, d->x), fmaf(o[i][3], f1, d->y));
        }
      }
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    const int row = tid / (D / 8), col = (tid % (D / 8)) * 8;
    if (row < R) {
      const float* b = reinterpret_cast<const float*>(base + L::kMerge) + row * L::kOPad + col;
      float acc[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        acc[k] = (b[k] + b[16 * L::kOPad + k]) + (b[32 * L::kOPad + k] + b[48 * L::kOPad + k]);
      float gm = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) gm = fmaxf(gm, um[w][row]);
#pragma unroll
      for (int w = 0; w < kConsumers; ++w)  // a warp without a maximum: 0, or NaN of NaN scores
        l += um[w][row] == -INFINITY ? ul[w][row] : ul[w][row] * ptx::ex2((um[w][row] - gm) * c);
      // a row that sees nothing has l = 0: zeros and -inf; a NaN sum stays NaN
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const RowSum sum = make_float2(gm, l);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] *= inv;
      if constexpr (CLUSTER) {
        // where this thread alone has read: the first buffer's place of the row
        float4* dst = reinterpret_cast<float4*>(base + L::kMerge + (row * L::kOPad + col) * 4);
        dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (col == 0) own_sum[row] = sum;
      } else if (done.lo > 0 || done.hi < done.total) {
        const size_t at = (size_t)(2 * blockIdx.x + (done.lo > 0 ? 0 : 1)) * kDecodeRows + row;
        float4* dst = reinterpret_cast<float4*>(p.part_o + at * D + col);
        dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (col == 0) p.part_sum[at] = sum;
      } else {
        const int i = row / p.G, head = done.h * p.G + row - i * p.G, tok = ds.q0 + i;
        store_row<D, BF16>(row_output(p), tok, head, col, acc, sum);
      }
    }
    if constexpr (CLUSTER) {
      // O = sum_i w_i O_i over the cluster's CTAs, w_i each one's share of the sums, by the first of them
      ptx::cluster_sync();
      if (row < R && (int)blockIdx.x % p.cluster == 0) {
        const uint32_t at_sum = ptx::smem_u32(&own_sum[row]), at = base_u32 + L::kMerge + (row * L::kOPad + col) * 4;
        float w[kMaxCluster], ls[kMaxCluster], m = -INFINITY, sum = 0.f, acc[8];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          const RowSum s = r < p.cluster ? ptx::cluster_ld2(ptx::cluster_addr(at_sum, r)) : make_float2(-INFINITY, 0.f);
          w[r] = s.x;
          ls[r] = s.y;
          m = fmaxf(m, s.x);
        }
        const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          w[r] = ls[r] * ptx::ex2((w[r] - ref) * c);
          sum += w[r];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = 0.f;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          if (r >= p.cluster) continue;
          const uint32_t src = ptx::cluster_addr(at, r);
          const float4 x = ptx::cluster_ld4(src), y = ptx::cluster_ld4(src + 16);
          const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[k] = fmaf(v[k], w[r], acc[k]);
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] *= inv;
        const int i = row / p.G;
        store_row<D, BF16>(row_output(p), ds.q0 + i, done.h * p.G + row - i * p.G, col, acc, make_float2(m, sum));
      }
      ptx::cluster_sync();  // no CTA's memory goes before it has been read
    }
  }
}

}  // namespace

template <int D, bool BF16, bool CLUSTER>
static cudaError_t launch_d(const PagedAttnParams& p, bool chained, cudaStream_t s) {
  static PerDevice attr_set;
  int done = 0;
  cudaError_t e = attr_set.get(&done, [](int, int* x) {
    *x = 1;
    return cudaFuncSetAttribute(paged_decode_kernel<D, BF16, CLUSTER>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)DecLayout<D>::kDynSmem);
  });
  if (e != cudaSuccess) return e;
  return launch_chained(paged_decode_kernel<D, BF16, CLUSTER>, p,
                        dim3(CLUSTER ? p.b.n_seqs * p.Hk * p.cluster : p.n_ctas), kDecThreads, DecLayout<D>::kDynSmem,
                        chained, s, CLUSTER ? p.cluster : 1);
}

cudaError_t paged_decode_clusters(int log2, int* n) {
  static PerDevice cache[4];
  if (log2 < 1 || log2 > 3) return cudaErrorInvalidValue;
  auto query = [](int log2, int* x) {
    const auto kernel = paged_decode_kernel<128, true, true>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)DecLayout<128>::kDynSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(1u << log2);
    cfg.blockDim = dim3(kDecThreads);
    cfg.dynamicSmemBytes = DecLayout<128>::kDynSmem;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim = {1u << log2, 1, 1};
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(x, kernel, &cfg);
  };
  return cache[log2].get(n, [&](int, int* x) { return query(log2, x); });
}

cudaError_t launch_paged_decode(const PagedAttnParams& p, bool bf16, int head_dim, bool chained, cudaStream_t s) {
  const auto launch = p.cluster > 1 ? (head_dim == 64 ? (bf16 ? launch_d<64, true, true> : launch_d<64, false, true>)
                                                      : (bf16 ? launch_d<128, true, true> : launch_d<128, false, true>))
                                    : (head_dim == 64 ? (bf16 ? launch_d<64, true, false> : launch_d<64, false, false>)
                                                      : (bf16 ? launch_d<128, true, false> : launch_d<128, false, false>));
  return launch(p, chained, s);
}

}  // namespace rc

// C entries of the paged-cache operators (include/rc.h): argument checks,
// TMA descriptors, workspace layout and launches. Host code.
#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <exception>
#include <initializer_list>
#include <mutex>
#include <string>
#include <utility>

#include "paged.cuh"

namespace rc {
rc_status SetLastError(rc_status st, const char* message);  // api.cu
}

namespace {

using rc::SetLastError;

rc_status invalid(const char* m) { return SetLastError(RC_EINVAL, m); }

rc_status cuda_failed(cudaError_t e, const char* what) {
  return SetLastError(RC_ECUDA, (std::string(what) + ": " + cudaGetErrorString(e)).c_str());
}

// Runs an entry's body; nothing it throws crosses the C ABI.
template <typename Fn>
rc_status guarded(Fn f) {
  try {
    return f();
  } catch (const std::exception& e) {
    return SetLastError(RC_ENOMEM, e.what());
  } catch (...) {
    return SetLastError(RC_ENOMEM, "unknown exception");
  }
}

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

int elem_size(int dtype) { return dtype == RC_F32 ? 4 : 2; }

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
bool aligned4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

// Whether entries of `row` elements at every combination of indices i[k] < n[k] and strides are apart: dimension by
// dimension, smallest stride first, each steps over all that the ones before it cover.
bool apart(std::initializer_list<std::pair<int64_t, int64_t>> dims, int64_t row) {
  std::pair<int64_t, int64_t> d[3];  // (stride, entries)
  int n = 0;
  for (const auto& x : dims)
    if (x.second > 1) d[n++] = x;
  std::sort(d, d + n);
  __int128 extent = row;
  for (int i = 0; i < n; ++i) {
    if (d[i].first < extent) return false;
    extent += (__int128)(d[i].second - 1) * d[i].first;
  }
  return true;
}

// How a call uses rows: plain loads take any strides, a TMA copy's are at least a row, written rows are apart.
enum class Use { kRead, kCopied, kWritten };

rc_status check_rows(const rc_rows& r, int n_tok, int d, int size, Use use, const char* what) {
  const std::string name(what);
  if (r.heads < 0 || r.heads > 16384) return invalid((name + ": heads out of range").c_str());
  if (r.heads == 0 || n_tok == 0) return RC_OK;
  if (!r.data) return invalid((name + ": null tensor").c_str());
  if (!aligned16(r.data) || r.tok_stride * size % 16 || r.head_stride * size % 16)
    return invalid((name + ": start and strides must be multiples of 16 bytes").c_str());
  const int64_t most = (int64_t)1 << 40;
  if (r.tok_stride < 0 || r.head_stride < 0 || r.tok_stride > most || r.head_stride > most)
    return invalid((name + ": stride out of range").c_str());
  if (use == Use::kCopied && ((n_tok > 1 && r.tok_stride < d) || (r.heads > 1 && r.head_stride < d)))
    return invalid((name + ": strides must be at least a row").c_str());
  if (use == Use::kWritten && !apart({{r.tok_stride, n_tok}, {r.head_stride, r.heads}}, d))
    return invalid((name + ": the rows overlap").c_str());
  return RC_OK;
}

rc::RowsView view(const rc_rows& r, int size) {
  return rc::RowsView{static_cast<uint8_t*>(r.data), r.tok_stride * size, r.head_stride * size, r.heads};
}

rc_status make_axes(const rc_rope* rope, int n_tok, int head_dim, rc::AxisTables* ax) {
  std::memset(ax, 0, sizeof(*ax));
  if (!rope || rope->n_axes == 0) return RC_OK;
  if (rope->n_axes < 0 || rope->n_axes > 3) return invalid("rope: n_axes must be 1 to 3");
  if (rope->pairing != RC_PAIR_ADJACENT && rope->pairing != RC_PAIR_HALVES) return invalid("rope: unknown pairing");
  if (n_tok > 0 && (!rope->pos || !aligned4(rope->pos))) return invalid("rope: null or misaligned positions");
  int sum = 0;
  for (int a = 0; a < rope->n_axes; ++a) {
    if (rope->pairs[a] < 0 || rope->pairs[a] > head_dim / 2) return invalid("rope: pairs out of range");
    if (rope->n_pos[a] < 1) return invalid("rope: an empty table");
    if (rope->pairs[a] > 0 && !rope->table[a]) return invalid("rope: null table");
    if (reinterpret_cast<uintptr_t>(rope->table[a]) % 8)
      return invalid("rope: misaligned table");
    sum += rope->pairs[a];
    ax->table[a] = reinterpret_cast<const float2*>(rope->table[a]);
    ax->n_pos[a] = rope->n_pos[a];
    ax->pairs[a] = rope->pairs[a];
  }
  if (sum != head_dim / 2) return invalid("rope: pairs must sum to head_dim / 2");
  ax->pos = rope->pos;
  ax->n_axes = rope->n_axes;
  return RC_OK;
}

// The pool and the batch; *b receives the kernels' view.
rc_status check_paged(const rc_paged* p, int n_tok, rc::BatchView* b) {
  if (!p) return invalid("null argument");
  if (p->dtype != RC_BF16 && p->dtype != RC_F16) return invalid("pages are bf16 or fp16");
  if (p->head_dim != 64 && p->head_dim != 128) return invalid("head_dim must be 64 or 128");
  if (p->page_size != 16 && p->page_size != 32 && p->page_size != 64 && p->page_size != 128)
    return invalid("page_size must be 16, 32, 64 or 128");
  if (p->kv_heads < 1 || p->kv_heads > 1024) return invalid("kv_heads must be in [1, 1024]");
  if (p->n_pages < 1) return invalid("an empty pool");
  if (!p->k_pages || !p->v_pages || !aligned16(p->k_pages) || !aligned16(p->v_pages))
    return invalid("the pages must be 16-byte aligned");
  const int entries[3] = {p->n_pages, p->kv_heads, p->page_size};
  for (const int64_t* st : {p->k_stride, p->v_stride})
    for (int i = 0; i < 3; ++i)
      if (entries[i] > 1 && (st[i] < p->head_dim || st[i] % 8 || st[i] >= ((int64_t)1 << 38)))
        return invalid("page strides must be multiples of 16 bytes, of at least a row");
  if (n_tok < 0 || n_tok > (1 << 30)) return invalid("n_tok out of range");
  if (p->n_seqs < 0 || p->n_seqs > rc::kMaxSeqs) return invalid("n_seqs must be in [0, 4096]");
  if (p->n_seqs > 0 && (!p->cu_q || !p->kv_len)) return invalid("null cu_q or kv_len");
  if (!aligned4(p->cu_q) || !aligned4(p->kv_len) || !aligned4(p->page_table))
    return invalid("misaligned cu_q, kv_len or page_table");
  if (p->max_pages < 0) return invalid("max_pages must not be negative");
  if ((int64_t)p->max_pages * p->page_size > (1 << 30))
    return SetLastError(RC_ERANGE, "max_pages * page_size exceeds 2^30");
  if (p->n_seqs > 0 && p->max_pages > 0 && !p->page_table) return invalid("null page_table");
  if (p->table_stride < 0 || (p->n_seqs > 1 && p->table_stride < p->max_pages && p->table_stride != 0))
    return invalid("table_stride below max_pages");
  int lg = 4;
  while ((1 << lg) < p->page_size) ++lg;
  *b = rc::BatchView{p->cu_q, p->kv_len, p->page_table, p->table_stride, p->n_seqs, p->max_pages, p->n_pages, lg};
  return RC_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// A map over `rank` dimensions, innermost first; strides in elements of dimensions 1..rank - 1. A dimension of one
// entry may come with any stride: it gets one that the encoder takes.
rc_status encode(CUtensorMap* map, void* base, int dtype, int rank, const int64_t* dims, const int64_t* strides,
                 const int* box) {
  auto fn = encode_fn();
  if (!fn) return SetLastError(RC_ECUDA, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t d[5], st[4];
  cuuint32_t bx[5], es[5];
  for (int i = 0; i < rank; ++i) {
    d[i] = (cuuint64_t)dims[i];
    bx[i] = (cuuint32_t)box[i];
    es[i] = 1;
    if (i > 0) st[i - 1] = (cuuint64_t)(dims[i] > 1 ? strides[i - 1] : dims[0]) * 2;
  }
  const CUresult r = fn(map, dtype == RC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                        rank, base, d, st, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return SetLastError(RC_ECUDA, ("cuTensorMapEncodeTiled failed: " + std::to_string(r)).c_str());
  return RC_OK;
}

cudaError_t sm_count(int* n) {
  static rc::PerDevice cache;
  return cache.get(n, [](int dev, int* x) { return cudaDeviceGetAttribute(x, cudaDevAttrMultiProcessorCount, dev); });
}

// Where the parts of an attention call lie in its workspace.
struct Work {
  bool decode;    // the kernel for few rows
  bool lead;      // a prefix is walked by every unit first
  bool two_pass;  // a prefix has a pass of its own
  int n_ctas, group;
  int x_ctas;     // of the prefix's own pass
  int cluster;    // CTAs to a unit of the kernel for few rows; 1: cut evenly
  size_t part_o, part_sum, rec, total;
  size_t x_part_o, x_part_sum, x_rec, pre_o, pre_sum;  // two passes: the prefix's parts and its result
  size_t own_o, own_sum;                                // and that over the sequences' own tokens
};

// Tiles of 64 keys that a CTA of a cluster takes at most (plan_work)
constexpr int kClusterTiles = 16;

rc_status plan_work(const rc_paged* p, const rc_paged_mask* m, int n_tok, int q_heads, Work* w) {
  *w = Work{};
  rc::BatchView b;
  if (rc_status st = check_paged(p, n_tok, &b)) return st;
  if (!m) return invalid("null mask");
  if (q_heads < 1 || q_heads % p->kv_heads) return invalid("q_heads must be a multiple of kv_heads");
  w->group = q_heads / p->kv_heads;
  if (w->group > 128) return invalid("q_heads / kv_heads must be at most 128");
  if (m->frame_seqlen < 1 || m->frame_seqlen > (1 << 30)) return invalid("frame_seqlen must be in [1, 2^30]");
  if (m->sink_frames < 0 || m->window_frames < 0) return invalid("sink_frames and window_frames must not be negative");
  if (m->sink_frames > 0 && m->window_frames == 0) return invalid("sink_frames need a window");
  if (m->max_q < 0) return invalid("max_q must not be negative");
  // within these bounds its product with the log2 of e, and what is divided by that, are finite and normal; an
  // exponential's argument is the product of that with a difference of scores, which is right at either end
  if (m->scale != 0.f && !(m->scale >= 1e-30f && m->scale <= 1e30f)) return invalid("scale must be 0 or in [1e-30, 1e30]");
  if (m->prefix_len < 0 || m->prefix_pages < 0) return invalid("prefix_len must not be negative");
  if (m->prefix_len > 0 &&
      (!m->prefix_table || (int64_t)m->prefix_pages * p->page_size < m->prefix_len || m->prefix_len > (1 << 30)))
    return invalid("prefix_table must list the pages of prefix_len tokens");
  if (!aligned4(m->prefix_table)) return invalid("misaligned prefix_table");
  // The kernel for few rows while a unit's rows fit its one 16-row matrix step: 64
  // streams of up to 16384 keys, 4 query heads a key head, take 355 us there and 494
  // in the other kernel with one query each, 363 and 498 with four (16 rows).
  w->decode = (int64_t)std::max(1, m->max_q) * w->group <= rc::kDecodeRows;
  const int per_pair = 2 * (128 / w->group);
  // positions of the stream-K split are 32-bit: tiles of every unit, summed
  const int64_t tiles = ((int64_t)p->max_pages + (m->prefix_len > 0 ? m->prefix_pages : 0)) * p->page_size / 64 + 6;
  const int64_t pairs = (int64_t)n_tok / per_pair + p->n_seqs + 1;
  if ((w->decode ? tiles * p->n_seqs : tiles * pairs) * p->kv_heads >= INT_MAX)
    return SetLastError(RC_ERANGE, "the batch has too many key tiles for one call");
  int sms = 0;
  if (cudaError_t e = sm_count(&sms)) return cuda_failed(e, "device attribute");
  w->n_ctas = std::min(sms, rc::kMaxPersistentCtas);
  // Few short units, by the table's width, the window and the prefix: a cluster of CTAs for each,
  // which merges its parts in shared memory, in one launch and without a workspace. As
  // many CTAs a unit as run at once (a cluster lies in one part of the GPU: 15 of 8 CTAs fit; 16
  // units take 17.1 us in clusters of 8 and 12.3 in clusters of 4), and 16 tiles a CTA at most:
  // 12 units of 777 keys take 10.2 us in clusters and 14.3 cut evenly, of 8000 18.4 and
  // 20.4, of 16000 26.6 and 24.6; one unit of 4000 12.3 and 16.4, of 8000 16.8 and 16.7, of
  // 12000 22.5 and 18.4; 60 units of 2000 18.4 and 22.5, of 8000 43.0 and 41.0. With a
  // prefix, whose other way is two passes and a join, 32 tiles: 8 units over 4000 prefix
  // tokens 16.4 and 37, over 15000 28.7 and 53; 64 over 3300 27 and 39.
  w->cluster = 1;
  if (w->decode) {
    int64_t keys = (int64_t)p->max_pages * p->page_size;
    if (m->window_frames > 0)
      keys = std::min(keys, ((int64_t)m->sink_frames + m->window_frames) * m->frame_seqlen + m->max_q + 64);
    keys += m->prefix_len;
    const int64_t most = (m->prefix_len > 0 ? 2 : 1) * kClusterTiles * 64;
    for (int log2 = 3; log2 > 0 && w->cluster == 1; --log2) {
      int room = 0;
      if (cudaError_t e = rc::paged_decode_clusters(log2, &room)) return cuda_failed(e, "cluster occupancy");
      if ((int64_t)p->n_seqs * p->kv_heads <= room && keys <= (most << log2)) w->cluster = 1 << log2;
    }
  }
  // A prefix and many rows (few rows: walked in clusters, else two passes): each sequence's units walk the prefix's tiles themselves
  // (from L2; no second pass and no merge), or the whole batch's rows are packed into
  // tiles for a pass over the prefix, and three kernels and the results in fp32 go on
  // top. The first where what its units walk beside a packed pass's is no more than the second costs:
  // per CTA 14 tiles and 20 bytes of traffic an element of q. In two passes and
  // walked, us: 48 sequences, 64-token pairs, 7021 prefix tokens: 16 tokens each 191 and
  // 338, 48 each 381 and 379, 63 each 466 and 382; 20 each over 300 prefix tokens 90 and 73, over
  // 1500 115 and 120; 48 each over 30000 1112 and 1331. 256-token pairs: 6 sequences of 30
  // over 5000 74 and 79; 16 of 100 over 3000 109 and 109, over 9360 177 and 231; 16 of 200
  // over 9360 279 and 256, over 30000 621 and 683; 3 of 50 over 1000 61 and 35.
  const int64_t each = p->n_seqs > 0 ? ((int64_t)n_tok + p->n_seqs - 1) / p->n_seqs : 0;
  const int64_t walked = p->n_seqs * ((each + per_pair - 1) / per_pair), packed = ((int64_t)n_tok + per_pair - 1) / per_pair;
  const double more = (double)(walked - packed) * p->kv_heads * ((m->prefix_len + 127) / 128);
  w->lead = m->prefix_len > 0 && (w->decode ? w->cluster > 1
                                            : more <= w->n_ctas * (14 + 1.64e-6 * n_tok * q_heads * p->head_dim));
  w->two_pass = m->prefix_len > 0 && !w->lead;
  // One SM is left to the pass that follows, whose first block is then in place and
  // the rest start without delay as the prefix's end: 48 continuations 62 us with
  // 147 CTAs (63 with 136 or 110), 68 with all 148
  w->x_ctas = w->two_pass && w->decode ? std::max(1, w->n_ctas - 1) : w->n_ctas;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes);
    return at;
  };
  auto parts = [&](int unit_rows, size_t* po, size_t* ps, size_t* rec) {
    const size_t rows = (size_t)2 * w->n_ctas * unit_rows;
    *po = take(rows * p->head_dim * 4);
    *ps = take(rows * sizeof(float2));
    *rec = take((size_t)w->n_ctas * sizeof(int4));
  };
  if (w->cluster == 1)
    parts(w->decode ? rc::kDecodeRows : rc::kPrefillRows, &w->part_o, &w->part_sum, &w->rec);
  if (w->two_pass) {
    // its own regions: the kernels of the call overlap at their ends
    parts(rc::kPrefillRows, &w->x_part_o, &w->x_part_sum, &w->x_rec);
    w->pre_o = take((size_t)n_tok * q_heads * p->head_dim * 4);
    w->pre_sum = take((size_t)n_tok * q_heads * sizeof(float2));
    w->own_o = take((size_t)n_tok * q_heads * p->head_dim * 4);
    w->own_sum = take((size_t)n_tok * q_heads * sizeof(float2));
  }
  w->total = o;
  return RC_OK;
}

}  // namespace

extern "C" {

rc_status rc_rope_axes(const rc_rope* rope, int dtype, int n_tok, int head_dim, int inverse, const rc_rows x[2],
                       const rc_rows y[2], int32_t* status, void* stream) {
  return guarded([&]() -> rc_status {
    if (!rope || !x || !y) return invalid("null argument");
    if (dtype != RC_BF16 && dtype != RC_F16 && dtype != RC_F32) return invalid("unknown dtype");
    if (head_dim != 64 && head_dim != 128) return invalid("head_dim must be 64 or 128");
    if (n_tok < 0 || n_tok > (1 << 30)) return invalid("n_tok out of range");
    rc::RopeAxesParams p{};
    if (rope->n_axes == 0) return invalid("rope: n_axes must be 1 to 3");
    if (!aligned4(status)) return invalid("misaligned status");
    if (rc_status st = make_axes(rope, n_tok, head_dim, &p.ax)) return st;
    const int size = elem_size(dtype);
    for (int i = 0; i < 2; ++i) {
      if (rc_status st = check_rows(x[i], n_tok, head_dim, size, Use::kRead, "x")) return st;
      if (rc_status st = check_rows(y[i], n_tok, head_dim, size, Use::kWritten, "y")) return st;
      if (x[i].heads != y[i].heads) return invalid("x and y differ in heads");
      p.x[i] = view(x[i], size);
      p.y[i] = view(y[i], size);
    }
    if (n_tok > 0 && y[0].heads > 0 && y[1].heads > 0 && y[0].data == y[1].data)
      return invalid("y: the two tensors are one");
    p.status = status;
    p.n_tok = n_tok;
    p.sign = inverse ? -1.f : 1.f;
    if (cudaError_t e = rc::launch_rope_axes(p, dtype, head_dim, rope->pairing == RC_PAIR_HALVES,
                                             static_cast<cudaStream_t>(stream)))
      return cuda_failed(e, "rope launch");
    return RC_OK;
  });
}

rc_status rc_paged_append(const rc_paged* pg, const rc_rope* rope, int n_tok, const rc_rows* q, const rc_rows* k,
                          const rc_rows* v, const rc_rows* q_out, int32_t* status, void* stream) {
  return guarded([&]() -> rc_status {
    rc::PagedAppendParams p{};
    if (rc_status st = check_paged(pg, n_tok, &p.b)) return st;
    if (!q || !k || !v || !q_out) return invalid("null argument");
    if (!aligned4(status)) return invalid("misaligned status");
    if (rc_status st = make_axes(rope, n_tok, pg->head_dim, &p.ax)) return st;
    if (rc_status st = check_rows(*q, n_tok, pg->head_dim, 2, Use::kRead, "q")) return st;
    if (rc_status st = check_rows(*q_out, n_tok, pg->head_dim, 2, Use::kWritten, "q_out")) return st;
    if (rc_status st = check_rows(*k, n_tok, pg->head_dim, 2, Use::kRead, "k")) return st;
    if (rc_status st = check_rows(*v, n_tok, pg->head_dim, 2, Use::kRead, "v")) return st;
    if (q->heads != q_out->heads) return invalid("q and q_out differ in heads");
    for (const int64_t* st : {pg->k_stride, pg->v_stride})
      if (!apart({{st[0], pg->n_pages}, {st[1], pg->kv_heads}, {st[2], pg->page_size}}, pg->head_dim))
        return invalid("the pages' rows overlap");
    if (k->heads != pg->kv_heads || v->heads != pg->kv_heads) return invalid("k and v must have the pool's heads");
    if (pg->k_pages == pg->v_pages) return invalid("k_pages and v_pages are one tensor");
    p.q = view(*q, 2);
    p.q_out = view(*q_out, 2);
    p.k = view(*k, 2);
    p.v = view(*v, 2);
    p.kp = rc::PageView{static_cast<uint8_t*>(pg->k_pages), pg->k_stride[0] * 2, pg->k_stride[1] * 2, pg->k_stride[2] * 2};
    p.vp = rc::PageView{static_cast<uint8_t*>(pg->v_pages), pg->v_stride[0] * 2, pg->v_stride[1] * 2, pg->v_stride[2] * 2};
    p.status = status;
    p.n_tok = n_tok;
    const bool halves = p.ax.n_axes > 0 && rope->pairing == RC_PAIR_HALVES;
    if (cudaError_t e = rc::launch_paged_append(p, pg->dtype, pg->head_dim, halves, static_cast<cudaStream_t>(stream)))
      return cuda_failed(e, "append launch");
    return RC_OK;
  });
}

rc_status rc_paged_workspace(const rc_paged* p, const rc_paged_mask* mask, int n_tok, int q_heads, size_t* bytes) {
  return guarded([&]() -> rc_status {
    if (!bytes) return invalid("null argument");
    Work w;
    if (rc_status st = plan_work(p, mask, n_tok, q_heads, &w)) return st;
    *bytes = w.total;
    return RC_OK;
  });
}

rc_status rc_paged_attention(const rc_paged* pg, const rc_paged_mask* m, int n_tok, const rc_rows* q,
                             const rc_rows* out, float* lse, void* workspace, size_t workspace_bytes, int32_t* status,
                             void* stream) {
  return guarded([&]() -> rc_status {
    if (!q || !out) return invalid("null argument");
    if (!aligned4(status) || !aligned4(lse)) return invalid("misaligned status or lse");
    rc::PagedAttnParams p;
    std::memset(&p, 0, sizeof(p));
    if (rc_status st = check_paged(pg, n_tok, &p.b)) return st;
    const int d = pg->head_dim;
    if (rc_status st = check_rows(*q, n_tok, d, 2, Use::kCopied, "q")) return st;
    if (rc_status st = check_rows(*out, n_tok, d, 2, Use::kWritten, "out")) return st;
    if (q->heads != out->heads) return invalid("q and out differ in heads");
    Work w;
    if (rc_status st = plan_work(pg, m, n_tok, q->heads, &w)) return st;
    if (n_tok == 0 || pg->n_seqs == 0) return RC_OK;
    if (w.total > 0 && (!workspace || reinterpret_cast<uintptr_t>(workspace) % kAlign))
      return invalid("the workspace must be 256-byte aligned");
    if (workspace_bytes < w.total) return SetLastError(RC_ENOMEM, "workspace smaller than rc_paged_workspace()");
    const bool bf16 = pg->dtype == RC_BF16;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.q = view(*q, 2);
    p.out = view(*out, 2);
    p.mask.frame = m->frame_seqlen;
    p.mask.sink_tok = (int)std::min<int64_t>((int64_t)m->sink_frames * m->frame_seqlen, 1 << 30);
    p.mask.window = m->window_frames;
    p.lse = lse;
    p.status = status;
    p.part_o = reinterpret_cast<float*>(ws + w.part_o);
    p.part_sum = reinterpret_cast<float2*>(ws + w.part_sum);
    p.rec = reinterpret_cast<int4*>(ws + w.rec);
    p.n_tok = n_tok;
    p.Hk = pg->kv_heads;
    p.G = w.group;
    p.n_ctas = w.n_ctas;
    p.cluster = w.cluster;
    const double scale = m->scale > 0.f ? (double)m->scale : 1.0 / std::sqrt((double)d);
    p.scale_log2 = (float)(1.4426950408889634 * scale);
    cudaStream_t s = static_cast<cudaStream_t>(stream);

    auto maps = [&](bool planes, int box_rows) -> rc_status {
      p.box_rows = box_rows;
      for (int i = 0; i < 2; ++i) {
        const int64_t* st = i ? pg->v_stride : pg->k_stride;
        CUtensorMap* map = i ? &p.tm_v : &p.tm_k;
        void* base = i ? pg->v_pages : pg->k_pages;
        const int64_t d4[4] = {d, pg->page_size, pg->kv_heads, pg->n_pages}, s4[3] = {st[2], st[1], st[0]};
        const int64_t d5[5] = {64, pg->page_size, d / 64, pg->kv_heads, pg->n_pages}, s5[4] = {st[2], 64, st[1], st[0]};
        const int b4[4] = {64, box_rows, 1, 1}, b5[5] = {64, box_rows, d / 64, 1, 1};
        if (rc_status e = planes ? encode(map, base, pg->dtype, 5, d5, s5, b5)
                                 : encode(map, base, pg->dtype, 4, d4, s4, b4))
          return e;
      }
      return RC_OK;
    };
    auto prefill = [&](const rc::PagedAttnParams& x) -> rc_status {
      if (cudaError_t e = rc::launch_paged_prefill(x, bf16, d, s)) return cuda_failed(e, "paged attention launch");
      if (cudaError_t e = rc::launch_paged_combine(x, bf16, d, false, s)) return cuda_failed(e, "combine launch");
      return RC_OK;
    };
    if (w.two_pass || !w.decode) {
      const int64_t dims[3] = {d, q->heads, n_tok};
      const int64_t st3[2] = {q->head_stride, q->tok_stride};
      const int box[3] = {64, w.group, 128 / w.group};
      if (rc_status st = encode(&p.tm_q, q->data, pg->dtype, 3, dims, st3, box)) return st;
      if (rc_status st = maps(false, pg->page_size)) return st;
    }
    if (w.lead) {
      p.lead_table = m->prefix_table;
      p.lead_len = m->prefix_len;
    }
    if (!w.two_pass && !w.decode) return prefill(p);
    rc::PagedAttnParams x = p;  // two passes: every query of the batch against the prefix's pages
    if (w.two_pass) {
      x.b.page_table = m->prefix_table;
      x.b.max_pages = m->prefix_pages;
      x.b.table_stride = 0;
      x.batch_pass = 1;
      x.n_ctas = w.x_ctas;
      x.prefix_len = m->prefix_len;
      x.mask = rc::MaskView{1 << 30, 0, 0};
      x.part_o = reinterpret_cast<float*>(ws + w.x_part_o);
      x.part_sum = reinterpret_cast<float2*>(ws + w.x_part_sum);
      x.rec = reinterpret_cast<int4*>(ws + w.x_rec);
      x.pre_o = reinterpret_cast<float*>(ws + w.pre_o);
      x.pre_sum = reinterpret_cast<float2*>(ws + w.pre_sum);
      p.pre_o = reinterpret_cast<float*>(ws + w.own_o);
      p.pre_sum = reinterpret_cast<float2*>(ws + w.own_sum);
    }
    if (!w.decode) {
      if (rc_status st = prefill(x)) return st;
      if (rc_status st = prefill(p)) return st;
      p.prev_o = x.pre_o;
      p.prev_sum = x.pre_sum;
      if (cudaError_t e = rc::launch_paged_merge(p, bf16, d, s)) return cuda_failed(e, "merge launch");
      return RC_OK;
    }
    if (rc_status st = maps(true, std::min(pg->page_size, 64))) return st;
    // the prefix first, its CTAs end together: 48 continuations 65 us the other way round, 62 so
    if (w.two_pass)
      if (cudaError_t e = rc::launch_paged_prefill(x, bf16, d, s)) return cuda_failed(e, "prefix launch");
    if (cudaError_t e = rc::launch_paged_decode(p, bf16, d, w.two_pass, s)) return cuda_failed(e, "paged attention launch");
    if (w.two_pass) {
      if (cudaError_t e = rc::launch_paged_join(p, x, bf16, d, s)) return cuda_failed(e, "join launch");
      return RC_OK;
    }
    if (w.cluster > 1) return RC_OK;
    if (cudaError_t e = rc::launch_paged_combine(p, bf16, d, true, s)) return cuda_failed(e, "combine launch");
    return RC_OK;
  });
}

}  // extern "C"

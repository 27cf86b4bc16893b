// Kernel parameter blocks and launchers of the paged-cache operators: rotary
// positions over several axes, the append that rotates keys into the pages,
// and attention over pages. Metadata of a call travels by value; lengths,
// page tables and positions are device arrays, so that a captured call sees
// their values of each replay.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/rc.h"
#include "kernels.cuh"

namespace rc {

// Most sequences one attention call takes: their tile counts are scanned in shared memory.
constexpr int kMaxSeqs = 4096;

struct AxisTables {
  const int32_t* pos;      // [n_tok][n_axes]
  const float2* table[3];  // [n_pos][pairs] (cos, sin)
  int n_pos[3];
  int pairs[3];
  int n_axes;
};

struct RowsView {
  uint8_t* data;
  long long tok_stride, head_stride;  // bytes
  int heads;
};

// Rotary positions of up to two tensors of rows (queries and keys).
struct RopeAxesParams {
  AxisTables ax;
  RowsView x[2], y[2];
  int* status;
  int n_tok, splits;
  float sign;  // of the sine: -1 turns back (the transpose)
};

struct PageView {
  uint8_t* data;
  long long page_stride, head_stride, row_stride;  // bytes
};

struct BatchView {
  const int32_t* cu_q;        // [n_seqs + 1]
  const int32_t* kv_len;      // [n_seqs]
  const int32_t* page_table;  // [n_seqs][table_stride]
  long long table_stride;
  int n_seqs, max_pages, n_pages;
  int page_log2;
};

struct PagedAppendParams {
  AxisTables ax;
  RowsView q, k, v, q_out;
  PageView kp, vp;
  BatchView b;
  int* status;
  int n_tok, splits;
};

// The mask: with f = position / frame, a query sees the keys of frames <= its
// own, and under a window (> 0 frames) only the last `window` of those frames
// and the first sink_tok tokens.
struct MaskView {
  int frame, sink_tok, window;
};

// Attention over pages: one call's inputs and outputs.
struct alignas(64) PagedAttnParams {
  CUtensorMap tm_q;    // prefill only: q as (d, q_heads, n_tok), box {64, G, 128 / G}
  // prefill: pages as (d, page, heads, n_pages), box {64, page, 1, 1}; decode: as
  // (64, page, d / 64, heads, n_pages), box {64, box_rows, d / 64, 1, 1}
  CUtensorMap tm_k;
  CUtensorMap tm_v;
  BatchView b;
  RowsView q, out;     // byte strides
  MaskView mask;
  float* lse;          // [q_heads][n_tok] or null
  int* status;
  float* part_o;       // [2 * n_ctas][rows][d] fp32: parts of units cut between CTAs, each divided by its sum
  float2* part_sum;    // [2 * n_ctas][rows], each part's sum of exponentials (RowSum)
  int4* rec;           // [n_ctas] what of its range a CTA left in parts (PartRecord)
  // A prefix that the whole batch sees. Prefill, and decode in clusters: lead_len > 0 tokens in the pages of
  // lead_table, which every unit walks first.
  const int32_t* lead_table;
  int lead_len;
  // Or in a pass of its own (batch_pass): one sequence of every query of the batch against keys [0, prefix_len) of
  // table row 0.
  int batch_pass, prefix_len;
  // null, or where the result goes instead of out and lse: fp32 [n_tok][q_heads][d], RowSum [q_heads][n_tok]
  float* pre_o;
  float2* pre_sum;
  // the merge kernel's: such a result that it merges with pre_o, pre_sum
  const float* prev_o;
  const float2* prev_sum;
  int n_tok, Hk, G;
  int box_rows;        // rows of a page per TMA box
  float scale_log2;    // log2(e) * scale
  int n_ctas;
  int cluster;         // decode: CTAs that share a unit (1: the whole batch is cut evenly)
};

// part_o / part_sum rows of one unit in the two attention kernels
constexpr int kDecodeRows = 16;
constexpr int kPrefillRows = 256;

// How many clusters of 2^log2 CTAs of the decode kernel the current device runs at once (asked of one of its
// instantiations: every one has an SM to a CTA, by its shared memory).
cudaError_t paged_decode_clusters(int log2, int* n);
// chained: as a programmatic dependent of the kernel before it, whose results it does not read
cudaError_t launch_paged_decode(const PagedAttnParams& p, bool bf16, int head_dim, bool chained, cudaStream_t s);
cudaError_t launch_paged_prefill(const PagedAttnParams& p, bool bf16, int head_dim, cudaStream_t s);
// out from a decode pass over the sequences' own tokens (`own`) and a pass of the batch over their prefix (`pre`),
// from whole results (pre_o, pre_sum of each) and parts alike. Launched as a programmatic dependent.
cudaError_t launch_paged_join(const PagedAttnParams& own, const PagedAttnParams& pre, bool bf16, int head_dim,
                              cudaStream_t s);
// out = the merge of two results in fp32 (prev_o, prev_sum; pre_o, pre_sum), for the rows of sequences.
cudaError_t launch_paged_merge(const PagedAttnParams& p, bool bf16, int head_dim, cudaStream_t s);
cudaError_t launch_paged_combine(const PagedAttnParams& p, bool bf16, int head_dim, bool decode, cudaStream_t s);

cudaError_t launch_rope_axes(const RopeAxesParams& p, int dtype, int head_dim, bool halves, cudaStream_t s);
cudaError_t launch_paged_append(const PagedAppendParams& p, int dtype, int head_dim, bool halves, cudaStream_t s);

}  // namespace rc

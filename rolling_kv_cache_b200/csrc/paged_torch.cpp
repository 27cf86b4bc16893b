// Python's way to the paged-cache operators: torch tensors to the C entries of
// include/rc.h. Checks what only tensors know (device, type, shape), allocates
// outputs and workspaces from torch's caching allocator, and carries the
// rotation's gradient. It is native because a decoding step's call is short:
// the same marshalling in Python took 16 us of host time, and the rotation's
// forward and backward 126 us. Every computation is the library's.
#include <ATen/ATen.h>
#include <ATen/TracerMode.h>
#include <ATen/cuda/CUDAContext.h>
#include <ATen/cuda/CUDAGraphsUtils.cuh>
#include <c10/core/AutogradState.h>
#include <c10/core/InferenceMode.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDAGuard.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/utils/pybind.h>

#include <mutex>
#include <optional>
#include <stdexcept>
#include <string>
#include <vector>

#include "../../include/rc.h"

namespace py = pybind11;

namespace {

using at::Tensor;
using Tensors = std::vector<Tensor>;

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

// A failed rc_* call: Python's RcError where the caller holds the interpreter
// (an operator's call), a runtime error in autograd's threads.
void check(rc_status st) {
  if (st == RC_OK) return;
  const std::string msg = rc_last_error();
  if (!PyGILState_Check()) throw std::runtime_error("rc status " + std::to_string(st) + ": " + msg);
  const py::object type = py::module_::import("rolling_kv_cache_b200.binding").attr("RcError");
  const py::object e = type(static_cast<int>(st), msg);
  PyErr_SetObject(type.ptr(), e.ptr());
  throw py::error_already_set();
}

constexpr int kMaxDevices = 64;

// One status word per device for every call of this module; never freed.
struct Words {
  std::mutex m;
  Tensor word[kMaxDevices];
};
Words& words() {
  static Words* w = new Words;
  return *w;
}

int32_t* status_word(int device) {
  if (device < 0 || device >= kMaxDevices) refuse("device index out of range");
  Words& w = words();
  std::lock_guard<std::mutex> lock(w.m);
  if (!w.word[device].defined()) {
    if (at::cuda::currentStreamCaptureStatus() != at::cuda::CaptureStatus::None)
      throw std::runtime_error("run one paged call on this device before capturing one");
    // a plain tensor whatever the mode of the first call: one made in inference mode could not be cleared outside it
    const c10::InferenceMode plain(false);
    const at::NoGradGuard no_grad;
    Tensor t = at::zeros({1}, at::TensorOptions().dtype(at::kInt).device(at::kCUDA, device));
    at::cuda::getCurrentCUDAStream(device).synchronize();
    w.word[device] = t;
  }
  return w.word[device].data_ptr<int32_t>();
}

std::optional<Tensor> existing_word(int device) {
  if (device < 0 || device >= kMaxDevices) refuse("device index out of range");
  Words& w = words();
  std::lock_guard<std::mutex> lock(w.m);
  if (!w.word[device].defined()) return std::nullopt;
  return w.word[device];
}

// The one CUDA device that every tensor of a call is on. Refuses what torch would take for an answer although the
// kernels are not part of it: tangents of forward mode, recordings of a call, and views whose memory holds
// the values negated.
struct Device {
  int index = -1;
  Device() {
    using c10::impl::TorchDispatchModeKey;
    if (at::tracer::impl::is_dispatch_enabled() || c10::impl::TorchDispatchModeTLS::get_mode(TorchDispatchModeKey::PROXY))
      refuse("paged operators cannot be recorded by a trace");
  }
  void add(const Tensor& t) {
    if (!t.defined()) return;
    if (c10::AutogradState::get_tls_state().get_fw_grad_mode() && t._fw_grad(0).defined())
      refuse("paged operators have no forward-mode derivative");
    if (t.is_neg()) refuse("paged operators do not take negated views (resolve_neg() makes a tensor of one)");
    if (!t.is_cuda()) refuse("paged operators take CUDA tensors");
    const int i = t.get_device();
    if (index >= 0 && i != index) refuse("tensors on more than one device");
    index = i;
  }
  void add(const std::optional<Tensor>& t) {
    if (t) add(*t);
  }
};

int dtype_of(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return RC_BF16;
    case at::kHalf: return RC_F16;
    case at::kFloat: return RC_F32;
    default: return -1;
  }
}

rc_rows rows_of(const Tensor& t, const char* what) {
  if (t.dim() != 3) refuse(std::string(what) + " must be [tokens, heads, head_dim]");
  if (t.stride(2) != 1) refuse(std::string(what) + " must have a contiguous last dimension");
  return rc_rows{t.data_ptr(), t.stride(0), t.stride(1), static_cast<int32_t>(t.size(1))};
}

bool is_int32(const Tensor& t, int dim) { return t.scalar_type() == at::kInt && t.dim() == dim; }

// The tables have no gradient: one that is asked for must not come out missing.
void constant(const Tensors& tables) {
  if (!at::GradMode::is_enabled()) return;
  for (const Tensor& t : tables)
    if (t.requires_grad()) refuse("the rotation tables have no gradient; detach them");
}

rc_rope rope_of(const Tensor& pos, const Tensors& tables, bool halves, int64_t n_tok, int64_t head_dim) {
  const int64_t n = static_cast<int64_t>(tables.size());
  if (n < 1 || n > 3) refuse("1 to 3 rotation tables");
  if (!is_int32(pos, 2) || pos.size(0) != n_tok || pos.size(1) != n || !pos.is_contiguous())
    refuse("pos must be a contiguous int32 tensor [tokens, axes]");
  rc_rope r{};
  r.pos = static_cast<const int32_t*>(pos.data_ptr());
  r.n_axes = static_cast<int32_t>(n);
  r.pairing = halves ? RC_PAIR_HALVES : RC_PAIR_ADJACENT;
  int64_t pairs = 0;
  for (int64_t a = 0; a < n; ++a) {
    const Tensor& t = tables[a];
    if (t.scalar_type() != at::kFloat || t.dim() != 3 || t.size(2) != 2 || !t.is_contiguous() || t.size(0) > INT32_MAX)
      refuse("a rotation table is a contiguous fp32 tensor [positions, pairs, 2]");
    r.table[a] = static_cast<const float*>(t.data_ptr());
    r.n_pos[a] = static_cast<int32_t>(t.size(0));
    r.pairs[a] = static_cast<int32_t>(t.size(1));
    pairs += t.size(1);
  }
  if (2 * pairs != head_dim) refuse("the tables' pairs must sum to head_dim / 2");
  return r;
}

int32_t tokens_of(const Tensor& t) {
  if (t.size(0) > INT32_MAX) refuse("too many tokens");
  return static_cast<int32_t>(t.size(0));
}

// Tells autograd that the library wrote to t.
void written(const Tensor& t) {
  if (!t.is_inference()) torch::autograd::impl::bump_version(t);
}

Tensor new_like(const Tensor& t) { return at::empty(t.sizes(), t.options()); }

// ---------------------------------------------------------------- rotation

void turn(const Tensors& xs, const Tensors& outs, const Tensor& pos, const Tensors& tables, bool halves, bool inverse) {
  Device dev;
  for (const Tensor& t : xs) dev.add(t);
  for (const Tensor& t : outs) dev.add(t);
  for (const Tensor& t : tables) dev.add(t);
  dev.add(pos);
  const Tensor& x = xs[0];
  const int dtype = dtype_of(x);
  if (dtype < 0) refuse("rope_axes takes bf16, fp16 or fp32");
  if (x.dim() != 3) refuse("x must be [tokens, heads, head_dim]");
  const int64_t d = x.size(2);
  rc_rows rx[2] = {}, ry[2] = {};
  for (size_t i = 0; i < xs.size(); ++i) {
    if (xs[i].scalar_type() != x.scalar_type() || outs[i].scalar_type() != x.scalar_type() || xs[i].dim() != 3 ||
        xs[i].size(0) != x.size(0) || xs[i].size(2) != d || outs[i].sizes() != xs[i].sizes())
      refuse("tensors differ in type, tokens or head_dim");
    rx[i] = rows_of(xs[i], "x");
    ry[i] = rows_of(outs[i], "out");
  }
  const rc_rope r = rope_of(pos, tables, halves, x.size(0), d);
  const c10::cuda::CUDAGuard guard(dev.index);
  check(rc_rope_axes(&r, dtype, tokens_of(x), static_cast<int>(d), inverse, rx, ry, status_word(dev.index),
                     at::cuda::getCurrentCUDAStream(dev.index).stream()));
}

// The tensor itself where the kernels can read it, else a contiguous copy (a
// gradient may come expanded, transposed, negated or at any offset).
Tensor readable(const Tensor& t) {
  if (t.dim() == 3 && t.stride(2) == 1 && !t.is_neg()) {
    const int64_t size = t.element_size();
    if (t.stride(0) >= 0 && t.stride(1) >= 0 && t.stride(0) * size % 16 == 0 && t.stride(1) * size % 16 == 0 &&
        reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0)
      return t;
  }
  return t.resolve_neg().clone(at::MemoryFormat::Contiguous);
}

Tensors turned(const Tensors& xs, const Tensor& pos, const Tensors& tables, bool halves, bool inverse);

// The gradients of x, from those of y that are there.
Tensors turned_back(torch::autograd::AutogradContext* ctx, const torch::autograd::variable_list& grads) {
  const auto saved = ctx->get_saved_variables();
  const Tensors tables(saved.begin() + 1, saved.end());
  Tensors gs;
  std::vector<size_t> at;
  for (size_t i = 0; i < grads.size(); ++i)
    if (grads[i].defined() && ctx->needs_input_grad(i)) {
      gs.push_back(readable(grads[i]));
      at.push_back(i);
    }
  Tensors out(grads.size());
  if (!gs.empty()) {
    const Tensors t = turned(gs, saved[0], tables, ctx->saved_data["halves"].toBool(), !ctx->saved_data["inverse"].toBool());
    for (size_t i = 0; i < at.size(); ++i) out[at[i]] = t[i];
  }
  return out;
}

Tensors turned_forward(torch::autograd::AutogradContext* ctx, const Tensors& xs, const Tensor& pos,
                       const Tensors& tables, bool halves, bool inverse) {
  Tensors keep{pos};
  keep.insert(keep.end(), tables.begin(), tables.end());
  ctx->save_for_backward(keep);
  ctx->saved_data["halves"] = halves;
  ctx->saved_data["inverse"] = inverse;
  ctx->set_materialize_grads(false);
  Tensors outs;
  for (const Tensor& x : xs) outs.push_back(new_like(x));
  turn(xs, outs, pos, tables, halves, inverse);
  return outs;
}

struct Turn1 : torch::autograd::Function<Turn1> {
  static torch::autograd::variable_list forward(torch::autograd::AutogradContext* ctx, const Tensor& x,
                                                const Tensor& pos, const Tensors& tables, bool halves, bool inverse) {
    return turned_forward(ctx, {x}, pos, tables, halves, inverse);
  }
  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx,
                                                 torch::autograd::variable_list grads) {
    const Tensors g = turned_back(ctx, grads);
    return {g[0], Tensor(), Tensor(), Tensor(), Tensor()};
  }
};

struct Turn2 : torch::autograd::Function<Turn2> {
  static torch::autograd::variable_list forward(torch::autograd::AutogradContext* ctx, const Tensor& x,
                                                const Tensor& z, const Tensor& pos, const Tensors& tables,
                                                bool halves, bool inverse) {
    return turned_forward(ctx, {x, z}, pos, tables, halves, inverse);
  }
  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx,
                                                 torch::autograd::variable_list grads) {
    const Tensors g = turned_back(ctx, grads);
    return {g[0], g[1], Tensor(), Tensor(), Tensor(), Tensor()};
  }
};

// While a graph is captured: refuses a leaf that an earlier graph of another
// stream still holds. The captured backward would hand its gradient to that
// graph's node on that stream, and a wait that leaves the capture ends the process.
void no_older_graph(const Tensors& xs) {
  if (!xs[0].is_cuda()) return;
  const c10::cuda::CUDAGuard guard(xs[0].get_device());
  if (at::cuda::currentStreamCaptureStatus() == at::cuda::CaptureStatus::None) return;
  for (const Tensor& x : xs) {
    if (!x.requires_grad() || !x.is_leaf()) continue;
    const auto node = torch::autograd::impl::try_get_grad_accumulator(x);
    const auto stream = node ? node->stream() : std::nullopt;
    if (stream && *stream != at::cuda::getCurrentCUDAStream(xs[0].get_device()).unwrap())
      refuse("an earlier autograd graph of this tensor, made on another stream, is alive: free it before the capture");
  }
}

Tensors turned(const Tensors& xs, const Tensor& pos, const Tensors& tables, bool halves, bool inverse) {
  if (at::GradMode::is_enabled()) {
    bool any = false;
    for (const Tensor& x : xs) any |= x.requires_grad();
    if (any) no_older_graph(xs);
    if (any)
      return xs.size() == 1 ? Turn1::apply(xs[0], pos, tables, halves, inverse)
                            : Turn2::apply(xs[0], xs[1], pos, tables, halves, inverse);
  }
  Tensors outs;
  for (const Tensor& x : xs) outs.push_back(new_like(x));
  turn(xs, outs, pos, tables, halves, inverse);
  return outs;
}

Tensors rope_axes(const Tensors& xs, const Tensor& pos, const Tensors& tables, bool halves, bool inverse,
                  const std::optional<Tensors>& out) {
  if (xs.empty() || xs.size() > 2) refuse("one tensor or a pair");
  constant(tables);
  if (!out) return turned(xs, pos, tables, halves, inverse);
  if (out->size() != xs.size()) refuse("one out for each x");
  if (at::GradMode::is_enabled())
    for (const Tensors* ts : {&xs, &*out})
      for (const Tensor& t : *ts)
        if (t.requires_grad()) refuse("out= takes no part in autograd; call it under torch.no_grad()");
  turn(xs, *out, pos, tables, halves, inverse);
  for (const Tensor& t : *out) written(t);
  return *out;
}

// ------------------------------------------------------------- paged cache

void no_grad(std::initializer_list<const Tensor*> ts) {
  if (!at::GradMode::is_enabled()) return;
  for (const Tensor* t : ts)
    if (t && t->defined() && t->requires_grad())
      refuse("the paged cache serves; it has no gradient (call it under torch.no_grad())");
}

rc_paged paged_of(const Tensor& k, const Tensor& v, const Tensor& cu_q, const Tensor& kv_len, const Tensor& table) {
  if (k.dim() != 4 || v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type())
    refuse("k_pages and v_pages must be [n_pages, kv_heads, page_size, head_dim] alike");
  const int dtype = dtype_of(k);
  if (dtype != RC_BF16 && dtype != RC_F16) refuse("pages are bf16 or fp16");
  if (!is_int32(cu_q, 1) || !is_int32(kv_len, 1) || !is_int32(table, 2))
    refuse("cu_q [n + 1], kv_len [n] and page_table [n, pages] must be int32");
  const int64_t n = table.size(0), width = table.size(1);
  if (kv_len.size(0) != n || cu_q.size(0) != n + 1)
    refuse("cu_q has one entry more than kv_len, page_table as many rows");
  if (k.stride(3) != 1 || v.stride(3) != 1 || (table.stride(1) != 1 && width > 1) || !cu_q.is_contiguous() ||
      !kv_len.is_contiguous())
    refuse("pages must have a contiguous last dimension; cu_q, kv_len and rows of page_table too");
  for (int64_t s : {k.size(0), k.size(1), k.size(2), k.size(3), n, width})
    if (s > INT32_MAX) refuse("a size passes 32 bits");
  rc_paged p{};
  p.k_pages = k.data_ptr();
  p.v_pages = v.data_ptr();
  for (int i = 0; i < 3; ++i) {
    p.k_stride[i] = k.stride(i);
    p.v_stride[i] = v.stride(i);
  }
  p.n_pages = static_cast<int32_t>(k.size(0));
  p.kv_heads = static_cast<int32_t>(k.size(1));
  p.page_size = static_cast<int32_t>(k.size(2));
  p.head_dim = static_cast<int32_t>(k.size(3));
  p.dtype = dtype;
  p.n_seqs = static_cast<int32_t>(n);
  p.cu_q = static_cast<const int32_t*>(cu_q.data_ptr());
  p.kv_len = static_cast<const int32_t*>(kv_len.data_ptr());
  p.page_table = static_cast<const int32_t*>(table.data_ptr());
  p.table_stride = table.stride(0);
  p.max_pages = static_cast<int32_t>(width);
  return p;
}

std::optional<Tensor> append(const std::optional<Tensor>& q, const Tensor& k, const Tensor& v, const Tensor& k_pages,
                             const Tensor& v_pages, const Tensor& cu_q, const Tensor& kv_len, const Tensor& page_table,
                             const std::optional<Tensor>& pos, const std::optional<Tensors>& tables, bool halves,
                             const std::optional<Tensor>& q_out) {
  no_grad({q ? &*q : nullptr, &k, &v, &k_pages, &v_pages, q_out ? &*q_out : nullptr});
  if (pos.has_value() != tables.has_value()) refuse("pos and tables go together");
  if (tables) constant(*tables);
  Device dev;
  for (const Tensor* t : {&k, &v, &k_pages, &v_pages, &cu_q, &kv_len, &page_table}) dev.add(*t);
  dev.add(q);
  dev.add(q_out);
  dev.add(pos);
  if (tables)
    for (const Tensor& t : *tables) dev.add(t);
  const rc_paged p = paged_of(k_pages, v_pages, cu_q, kv_len, page_table);
  const auto dt = k_pages.scalar_type();
  if (k.dim() != 3 || v.sizes() != k.sizes() || k.size(2) != k_pages.size(3) || k.scalar_type() != dt ||
      v.scalar_type() != dt)
    refuse("k and v must be [tokens, kv_heads, head_dim] alike, of the pages' type and head_dim");
  rc_rows rq{}, ro{};
  std::optional<Tensor> out;
  if (q) {
    if (q->scalar_type() != dt || q->dim() != 3 || q->size(0) != k.size(0) || q->size(2) != k.size(2))
      refuse("q must be [tokens, q_heads, head_dim] of k's type, tokens and head_dim");
    out = q_out ? *q_out : new_like(*q);
    if (out->sizes() != q->sizes() || out->scalar_type() != dt) refuse("q_out differs from q in shape or type");
    rq = rows_of(*q, "q");
    ro = rows_of(*out, "q_out");
  } else if (q_out) {
    refuse("q_out without q");
  }
  rc_rope r{};
  if (pos) r = rope_of(*pos, *tables, halves, k.size(0), k.size(2));
  const rc_rows rk = rows_of(k, "k"), rv = rows_of(v, "v");
  const c10::cuda::CUDAGuard guard(dev.index);
  check(rc_paged_append(&p, pos ? &r : nullptr, tokens_of(k), &rq, &rk, &rv, &ro, status_word(dev.index),
                        at::cuda::getCurrentCUDAStream(dev.index).stream()));
  written(k_pages);
  written(v_pages);
  if (q_out) written(*q_out);
  return out;
}

std::pair<Tensor, std::optional<Tensor>> attention(const Tensor& q, const Tensor& k_pages, const Tensor& v_pages,
                                                   const Tensor& cu_q, const Tensor& kv_len, const Tensor& page_table,
                                                   std::optional<int64_t> max_q, int64_t frame_seqlen,
                                                   int64_t sink_frames, int64_t window_frames,
                                                   std::optional<double> scale, const std::optional<Tensor>& out_,
                                                   bool return_lse, const std::optional<Tensor>& prefix_table,
                                                   int64_t prefix_len) {
  no_grad({&q, &k_pages, &v_pages, out_ ? &*out_ : nullptr});
  Device dev;
  for (const Tensor* t : {&q, &k_pages, &v_pages, &cu_q, &kv_len, &page_table}) dev.add(*t);
  dev.add(prefix_table);
  dev.add(out_);
  const rc_paged p = paged_of(k_pages, v_pages, cu_q, kv_len, page_table);
  if (q.scalar_type() != k_pages.scalar_type() || q.dim() != 3 || q.size(2) != k_pages.size(3))
    refuse("q must be [tokens, q_heads, head_dim] of the pages' type and head_dim");
  const int32_t n_tok = tokens_of(q);
  for (int64_t v : {max_q.value_or(0), frame_seqlen, sink_frames, window_frames, prefix_len})
    if (v < 0 || v > INT32_MAX) refuse("max_q, frames and prefix_len must be 32-bit and not negative");
  if (scale && !(*scale >= 1e-30 && *scale <= 1e30)) refuse("scale must be in [1e-30, 1e30]");
  rc_paged_mask m{};
  m.frame_seqlen = static_cast<int32_t>(frame_seqlen);
  m.sink_frames = static_cast<int32_t>(sink_frames);
  m.window_frames = static_cast<int32_t>(window_frames);
  m.max_q = max_q ? static_cast<int32_t>(*max_q) : n_tok;
  m.scale = static_cast<float>(scale.value_or(0.0));
  if (prefix_table) {
    if (!is_int32(*prefix_table, 1) || !prefix_table->is_contiguous() || prefix_table->size(0) > INT32_MAX)
      refuse("prefix_table must be a contiguous int32 tensor [pages]");
    if (prefix_len < 1) refuse("prefix_len must be positive");
    m.prefix_len = static_cast<int32_t>(prefix_len);
    m.prefix_table = static_cast<const int32_t*>(prefix_table->data_ptr());
    m.prefix_pages = static_cast<int32_t>(prefix_table->size(0));
  }
  const Tensor out = out_ ? *out_ : new_like(q);
  if (out.sizes() != q.sizes() || out.scalar_type() != q.scalar_type()) refuse("out differs from q in shape or type");
  const rc_rows rq = rows_of(q, "q"), ro = rows_of(out, "out");
  const c10::cuda::CUDAGuard guard(dev.index);
  std::optional<Tensor> lse;
  if (return_lse) lse = at::empty({q.size(1), q.size(0)}, q.options().dtype(at::kFloat));
  size_t bytes = 0;
  check(rc_paged_workspace(&p, &m, n_tok, rq.heads, &bytes));
  // freed on return: the allocator hands it out again on this stream only
  Tensor work;
  if (bytes) work = at::empty({static_cast<int64_t>(bytes)}, q.options().dtype(at::kByte));
  check(rc_paged_attention(&p, &m, n_tok, &rq, &ro, lse ? lse->data_ptr<float>() : nullptr, bytes ? work.data_ptr() : nullptr, bytes,
                           status_word(dev.index), at::cuda::getCurrentCUDAStream(dev.index).stream()));
  if (out_) written(out);
  return {out, lse};
}

}  // namespace

PYBIND11_MODULE(_paged, m) {
  m.def("rope_axes", &rope_axes);
  m.def("append", &append);
  m.def("attention", &attention);
  m.def("status_word", &existing_word);
}

// The calls of a serving step over a paged cache for torch tensors: argument
// checks, output tensors and the C ABI call (attn_f16.h), in C++.
//
// A step of token generation makes these calls once per layer and its kernels
// take a few microseconds, so the call itself must not take longer: checking
// eight tensors, allocating an output and marshalling thirty arguments in
// Python took 19 to 22 us a call.  Here the maps take 6.3 (3.0 into given
// outputs), the rotation 4.5 to 4.9 (2.5) and the attention 8.0 (4.1; a step for
// both kernels, with four launches, 12.6 and 7.5).  Nothing is computed here.  A bad tensor raises ValueError; a code of the C ABI is returned as a
// number for the caller to raise.
#include <torch/extension.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <string>
#include <vector>

#include "attn_f16.h"

namespace py = pybind11;

namespace {

using at::Tensor;
using c10::cuda::CUDAStream;

constexpr int64_t D = ATTN_F16_HEAD_DIM;

[[noreturn]] void refuse(const std::string& what) { throw py::value_error(what); }

// A tensor of this type and rank on the plan's device, its last dimension
// contiguous.
void need(const Tensor& x, const char* name, at::ScalarType type, int64_t dims, int device) {
  if (x.scalar_type() != type || x.dim() != dims)
    refuse(std::string(name) + " must be a " + std::to_string(dims) + "-dimensional " +
           c10::toString(type) + " tensor");
  if (!x.is_cuda() || x.get_device() != device)
    refuse(std::string(name) + " must be on the plan's device");
  if (x.size(-1) > 1 && x.stride(-1) != 1)
    refuse(std::string(name) + "'s last dimension must be contiguous");
}

void need_count(const Tensor& x, const char* name, int64_t n) {
  if (x.size(0) != n)
    refuse(std::string(name) + " must have " + std::to_string(n) + " entries");
}

// [tokens, heads, 256] binary16.
void need_heads(const Tensor& x, const char* name, int device, int64_t tokens = -1) {
  need(x, name, at::kHalf, 3, device);
  if (x.size(2) != D || (tokens >= 0 && x.size(0) != tokens))
    refuse(std::string(name) + " must be [tokens, heads, 256]");
}

// [pages, page_size, kv_heads, 256] binary16 each.
void need_caches(const Tensor& k, const Tensor& v, int device) {
  need(k, "K_cache", at::kHalf, 4, device);
  need(v, "V_cache", at::kHalf, 4, device);
  if (k.sizes() != v.sizes() || k.size(3) != D)
    refuse("K_cache and V_cache must be [pages, page_size, kv_heads, 256]");
}

int narrow(int64_t n, const char* what) {
  if (n > INT32_MAX || n < INT32_MIN) refuse(std::string(what) + " does not fit 32 bits");
  return (int)n;
}

struct Strides {
  int64_t v[3];
  explicit Strides(const Tensor& x) {
    for (int i = 0; i < 3; ++i) v[i] = i < x.dim() - 1 ? x.stride(i) : 0;
  }
};

// The stream of a call: torch's current one on the plan's device, or the one
// given, which then also owns the tensors that the call allocates.
struct OnStream {
  CUDAStream stream;
  c10::cuda::OptionalCUDAStreamGuard guard;
  OnStream(const c10::optional<int64_t>& handle, int device)
      : stream(handle ? c10::cuda::getStreamFromExternal(
                            reinterpret_cast<cudaStream_t>(static_cast<intptr_t>(*handle)),
                            (c10::DeviceIndex)device)
                      : c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device)) {
    if (handle) guard.reset_stream(stream);
  }
  gemm_f16_stream_t raw() const { return stream.stream(); }
};

Tensor output(const Tensor& x, const c10::optional<Tensor>& out, const char* name, int device) {
  if (!out) return at::empty(x.sizes(), x.options());
  need_heads(*out, "out", device);
  if (out->sizes() != x.sizes()) refuse(std::string("out must have the shape of ") + name);
  return *out;
}

gemm_f16_plan_t plan_of(int64_t handle) {
  return reinterpret_cast<gemm_f16_plan_t>(static_cast<intptr_t>(handle));
}
const int32_t* ints(const Tensor& x) { return static_cast<const int32_t*>(x.const_data_ptr()); }
int32_t* ints_out(const Tensor& x) { return static_cast<int32_t*>(x.data_ptr()); }
const uint64_t* words(const Tensor& x) {
  return static_cast<const uint64_t*>(x.const_data_ptr());
}

py::object done(int rc, py::object result) {
  return rc < 0 ? py::object(py::int_(rc)) : std::move(result);
}

// Numbers at .. at + n - 1 of a one-dimensional tensor, as narrow() gives them
// but without the dispatcher (five of these are most of a call's time with it).
Tensor piece(const Tensor& x, int64_t at, int64_t n) {
  const int64_t one = 1;
  Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      c10::TensorImpl::VIEW, c10::Storage(x.storage()), x.key_set(), x.dtype());
  t.unsafeGetTensorImpl()->set_sizes_and_strides(c10::IntArrayRef(&n, 1),
                                                 c10::IntArrayRef(one), x.storage_offset() + at);
  return t;
}

// -> (starts, kv_lens, positions, slots, free_head), or an error code.
py::object paged_maps(int64_t plan, int device, const Tensor& cached, const Tensor& added,
                      const Tensor& table, const Tensor& free_pages, const Tensor& free_head,
                      int64_t page_size, int64_t max_tokens,
                      const c10::optional<std::vector<Tensor>>& out,
                      const c10::optional<int64_t>& stream) {
  need(cached, "cached", at::kInt, 1, device);
  need(added, "added", at::kInt, 1, device);
  need(table, "block_table", at::kInt, 2, device);
  need(free_pages, "free_pages", at::kInt, 1, device);
  need(free_head, "free_head", at::kInt, 1, device);
  const int64_t batch = cached.size(0);
  if (added.size(0) != batch || table.size(0) != batch || free_head.size(0) != 1)
    refuse("shape mismatch: cached [B], added [B], block_table [B, P], free_head [1]");
  OnStream on(stream, device);
  Tensor starts, lens, positions, slots, head;
  const int64_t most = std::max<int64_t>(max_tokens, 0);
  if (out) {
    if (out->size() != 5) refuse("out must be a PagedMaps");
    starts = (*out)[0];
    lens = (*out)[1];
    positions = (*out)[2];
    slots = (*out)[3];
    head = (*out)[4];
    const char* names[5] = {"out.starts", "out.kv_lens", "out.positions", "out.slots",
                            "out.free_head"};
    const int64_t counts[5] = {batch + 1, batch, most, most, 1};
    for (int i = 0; i < 5; ++i) {
      need((*out)[i], names[i], at::kInt, 1, device);
      need_count((*out)[i], names[i], counts[i]);
    }
  } else {
    // One allocation; positions and slots begin at 16-byte boundaries.
    const int64_t room = (most + 3) / 4 * 4;
    const Tensor buf = at::empty({2 * room + 2 * batch + 2}, cached.options());
    positions = piece(buf, 0, most);
    slots = piece(buf, room, most);
    starts = piece(buf, 2 * room, batch + 1);
    lens = piece(buf, 2 * room + batch + 1, batch);
    head = piece(buf, 2 * room + 2 * batch + 1, 1);
  }
  const int rc = attn_f16_paged_maps(
      plan_of(plan), narrow(batch, "batch"), ints(cached), ints(added), ints_out(table),
      batch > 1 ? table.stride(0) : table.size(1), narrow(table.size(1), "max_pages"),
      ints(free_pages), narrow(free_pages.size(0), "free_pages"), ints(free_head),
      narrow(page_size, "page_size"), narrow(max_tokens, "max_tokens"), ints_out(starts),
      ints_out(lens), ints_out(positions), ints_out(slots), ints_out(head), on.raw());
  return done(rc, py::make_tuple(starts, lens, positions, slots, head));
}

void need_positions(const Tensor& positions, const Tensor& turns, int64_t tokens, int device) {
  need(positions, "positions", at::kInt, 1, device);
  need(turns, "turns", at::kLong, 1, device);
  need_count(positions, "positions", tokens);
}

py::object rotary(int64_t plan, int device, const Tensor& x, const Tensor& positions,
                  const Tensor& turns, const c10::optional<Tensor>& out_, int layout, double factor,
                  bool inverse, const c10::optional<int64_t>& stream) {
  need_heads(x, "X", device);
  need_positions(positions, turns, x.size(0), device);
  OnStream on(stream, device);
  const Tensor out = output(x, out_, "X", device);
  const Strides xs(x), os(out);
  const int rc = attn_f16_rope(
      plan_of(plan), narrow(x.size(0), "tokens"), narrow(x.size(1), "heads"), 0, (int)D,
      narrow(2 * turns.size(0), "turns"), layout, inverse, (float)factor, words(turns),
      ints(positions), x.const_data_ptr(), xs.v, out.data_ptr(), os.v, nullptr, nullptr, nullptr,
      nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, 0, on.raw());
  return done(rc, py::cast(out));
}

py::object rotary_to_cache(int64_t plan, int device, const Tensor& q, const Tensor& k,
                           const Tensor& v, const Tensor& positions, const Tensor& slots,
                           const Tensor& turns, const Tensor& kc, const Tensor& vc,
                           const c10::optional<Tensor>& out_, int layout, double factor,
                           const c10::optional<int64_t>& stream) {
  need_heads(q, "Q", device);
  const int64_t tokens = q.size(0);
  need_heads(k, "K", device, tokens);
  need_heads(v, "V", device, tokens);
  need_caches(kc, vc, device);
  if (k.sizes() != v.sizes() || k.size(1) != kc.size(2))
    refuse("K, V and the caches must have the same heads");
  need_positions(positions, turns, tokens, device);
  need(slots, "slots", at::kInt, 1, device);
  need_count(slots, "slots", tokens);
  OnStream on(stream, device);
  const Tensor out = output(q, out_, "Q", device);
  const Strides qs(q), os(out), ks(k), vs(v), kcs(kc), vcs(vc);
  const int rc = attn_f16_rope(
      plan_of(plan), narrow(tokens, "tokens"), narrow(q.size(1), "heads"),
      narrow(k.size(1), "heads"), (int)D, narrow(2 * turns.size(0), "turns"), layout, 0,
      (float)factor, words(turns), ints(positions), q.const_data_ptr(), qs.v, out.data_ptr(), os.v,
      k.const_data_ptr(), ks.v, v.const_data_ptr(), vs.v, ints(slots), kc.data_ptr(), kcs.v,
      vc.data_ptr(), vcs.v, narrow(kc.size(0), "pages"), narrow(kc.size(1), "page_size"), on.raw());
  return done(rc, py::cast(out));
}

py::object paged_attention(int64_t plan, int device, const Tensor& q, const Tensor& kc,
                           const Tensor& vc, const Tensor& table, const Tensor& starts,
                           const Tensor& lens, int64_t max_q, const c10::optional<Tensor>& out_,
                           double scale, int64_t window, int64_t sinks,
                           const c10::optional<int64_t>& stream) {
  need_heads(q, "Q", device);
  need_caches(kc, vc, device);
  need(table, "block_table", at::kInt, 2, device);
  need(starts, "starts", at::kInt, 1, device);
  need(lens, "kv_lens", at::kInt, 1, device);
  const int64_t batch = lens.size(0);
  if (starts.size(0) != batch + 1 || table.size(0) != batch)
    refuse("shape mismatch: block_table [B, P], starts [B + 1], kv_lens [B]");
  OnStream on(stream, device);
  const Tensor out = output(q, out_, "Q", device);
  const Strides qs(q), os(out), kcs(kc), vcs(vc);
  const int rc = attn_f16_paged_fwd(
      plan_of(plan), narrow(batch, "batch"), narrow(q.size(0), "tokens"), narrow(max_q, "max_q"),
      narrow(q.size(1), "heads"), narrow(kc.size(2), "heads"), (int)D, q.const_data_ptr(), qs.v,
      kc.const_data_ptr(), kcs.v, vc.const_data_ptr(), vcs.v, narrow(kc.size(0), "pages"),
      narrow(kc.size(1), "page_size"), ints(table), batch > 1 ? table.stride(0) : table.size(1),
      narrow(table.size(1), "max_pages"), ints(starts), ints(lens), out.data_ptr(), os.v,
      (float)scale, narrow(window, "window"), narrow(sinks, "sinks"), on.raw());
  return done(rc, py::cast(out));
}

}  // namespace

#include "torch_f8.h"

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
  m.doc() = "attn_f16.h's paged-cache calls and gemm_f8.h's calls for torch tensors";
  m.def("paged_maps", &paged_maps);
  m.def("rotary", &rotary);
  m.def("rotary_to_cache", &rotary_to_cache);
  m.def("paged_attention", &paged_attention);
  add_f8_calls(m);
}

// gemm_f8.h's calls for torch tensors: argument checks, output tensors and the
// C ABI call, in C++ for the same reason as torch_calls.cpp (a generation
// step makes several of them per layer).  Nothing is computed here.  A bad
// tensor raises ValueError; a code of the C ABI is returned as a number for
// the caller to raise.  The differentiable calls are autograd functions in C++
// too: in Python a dense layer's step, forward and backward, took 330 us for
// kernels of 109.
//
// Part of torch_calls.cpp (and of its module), after the helpers there.
#pragma once

#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>

#include "gemm_f8.h"

namespace {

// A code of the C ABI on its way to a binding (raised there) or, from a backward
// pass, to Python as a RuntimeError.
struct CallError : std::runtime_error {
  int code;
  CallError(int rc, const char* where)
      : std::runtime_error(std::string(where) + ": " + gemm_f16_strerror(rc)), code(rc) {}
};
void check(int rc, const char* where) {
  if (rc < 0) throw CallError(rc, where);
}

// A call's result for Python: what `f` returns, or the code of the C ABI.
template <typename F>
py::object answer(const F& f) {
  try {
    return f();
  } catch (const CallError& e) {
    return py::int_(e.code);
  }
}

void on_device(const Tensor& x, const char* name, int device) {
  if (!x.is_cuda() || x.get_device() != device)
    refuse(std::string(name) + " must be on the plan's device");
}

// GEMM_F8_F16, _BF16 or _F32.
int type_of(at::ScalarType t, const char* name) {
  if (t == at::kHalf) return GEMM_F8_F16;
  if (t == at::kBFloat16) return GEMM_F8_BF16;
  if (t == at::kFloat) return GEMM_F8_F32;
  refuse(std::string(name) + " must be float16, bfloat16 or float32");
}

int format_of(at::ScalarType t, const char* name) {
  if (t == at::kFloat8_e4m3fn) return GEMM_F8_E4M3;
  if (t == at::kFloat8_e5m2) return GEMM_F8_E5M2;
  refuse(std::string(name) + " must be float8_e4m3fn or float8_e5m2");
}

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
int64_t blocks_of(int64_t n) { return (n + 127) / 128; }

// ------------------------------------------------------------------ quantize

struct Quantized {
  Tensor q, s, q2, s2;     // q2, s2: the columns' of BOTH
};

Quantized quantize(int64_t plan, int device, const Tensor& x_, int blocks, at::ScalarType dtype,
                   const c10::optional<Tensor>& source = {}, int64_t choices = 1,
                   const c10::optional<int64_t>& stream = {}) {
  const int type = type_of(x_.scalar_type(), "X"), format = format_of(dtype, "dtype");
  on_device(x_, "X", device);
  if (x_.dim() != 2 && x_.dim() != 3) refuse("X must be [rows, cols] or [matrices, rows, cols]");
  if (x_.dim() == 3 && (blocks == GEMM_F8_BOTH || source))
    refuse("several matrices have blocks of one kind and no maps");
  // A transposed view is quantised as it is stored.
  const bool turned = !(x_.size(-1) <= 1 || x_.stride(-1) == 1) && x_.stride(-2) == 1;
  if (turned && source) refuse("X must be row-major where maps are given");
  const Tensor x = turned ? x_.transpose(-1, -2) : x_;
  if (x.size(-1) > 1 && x.stride(-1) != 1) refuse("X must be row-major or a transposed row-major view");
  const int64_t cols = x.size(-1), batch = x.dim() == 3 ? x.size(0) : 1;
  if (cols < 1) refuse("X must have columns");
  if (turned) blocks = blocks == GEMM_F8_ROWS ? GEMM_F8_COLUMNS : blocks == GEMM_F8_COLUMNS ? GEMM_F8_ROWS : blocks;
  if (source) need(*source, "maps.source", at::kInt, 1, device);
  const int64_t rows = source ? source->size(0) : x.size(-2);
  OnStream on(stream, device);
  const int64_t pitch = up(cols, 16);
  const auto codes = [&] {
    Tensor q = x.dim() == 3 ? at::empty({batch, rows, pitch}, x.options().dtype(dtype))
                            : at::empty({rows, pitch}, x.options().dtype(dtype));
    return pitch == cols ? q : q.narrow(-1, 0, cols);
  };
  const auto scales = [&](int kind) {
    const int64_t r = kind == GEMM_F8_ROWS ? rows : blocks_of(rows);
    const int64_t c = kind == GEMM_F8_COLUMNS ? cols : blocks_of(cols);
    return x.dim() == 3 ? at::empty({batch, r, c}, x.options().dtype(at::kFloat))
                        : at::empty({r, c}, x.options().dtype(at::kFloat));
  };
  const bool both = blocks == GEMM_F8_BOTH;
  Tensor q = codes(), s = scales(both ? GEMM_F8_ROWS : blocks), q2, s2;
  if (both) {
    q2 = codes();
    s2 = scales(GEMM_F8_COLUMNS);
  }
  check(gemm_f8_quantize(
            plan_of(plan), blocks, format, type, narrow(batch, "matrices"), narrow(rows, "rows"),
            narrow(cols, "cols"), x.const_data_ptr(), x.size(-2) > 1 ? x.stride(-2) : pitch,
            batch > 1 ? x.stride(0) : 0, source ? ints(*source) : nullptr,
            narrow(choices, "choices"), narrow(x.size(-2), "rows"), q.data_ptr(), pitch,
            rows * pitch, s.data_ptr<float>(), both ? q2.data_ptr() : nullptr,
            both ? s2.data_ptr<float>() : nullptr, on.raw()),
        "gemm_f8_quantize");
  if (turned) {
    q = q.transpose(-1, -2);
    s = s.transpose(-1, -2);
    if (both) return {q2.transpose(-1, -2), s2.transpose(-1, -2), q, s};
  }
  return {q, s, q2, s2};
}

// ------------------------------------------------------------------ product

// Codes [.., rows, cols] with scales; `inner_last`: the inner dimension is the
// last one (A), else the one before (B).
gemm_f8_operand operand(const Tensor& x, const Tensor& s, const char* name, bool inner_last,
                        int device) {
  gemm_f8_operand o = {};
  o.format = format_of(x.scalar_type(), name);
  on_device(x, name, device);
  on_device(s, name, device);
  if (s.scalar_type() != at::kFloat || s.dim() != x.dim())
    refuse(std::string(name) + "'s scales must be float32 and have its codes' dimensions");
  const int64_t rows = x.size(-2), cols = x.size(-1);
  if (x.stride(-1) == 1 && (rows <= 1 || x.stride(-2) >= cols)) {
    o.ld = rows > 1 ? x.stride(-2) : up(cols, 16);
  } else if (x.stride(-2) == 1 && (cols <= 1 || x.stride(-1) >= rows)) {
    o.transposed = 1;
    o.ld = cols > 1 ? x.stride(-1) : up(rows, 16);
  } else if (rows > 0 && cols > 0) {
    refuse(std::string(name) + " must be row-major or a transposed row-major view");
  }
  o.data = x.const_data_ptr();
  o.scales = s.const_data_ptr<float>();
  const int64_t inner = inner_last ? cols : rows, outer = inner_last ? rows : cols;
  const int64_t s_inner = s.size(inner_last ? -1 : -2), s_outer = s.size(inner_last ? -2 : -1);
  if (s_inner != blocks_of(inner) || (s_outer != outer && s_outer != blocks_of(outer)))
    refuse(std::string(name) +
           "'s scales must have an entry for each 128 of the inner dimension, and for each or "
           "each 128 of the other");
  o.tiles = s_outer != outer;
  o.s_inner = s.stride(inner_last ? -1 : -2);
  o.s_outer = s.stride(inner_last ? -2 : -1);
  if (x.dim() == 3) {
    if (s.size(0) != x.size(0)) refuse(std::string(name) + "'s scales must be one set for each matrix");
    o.batch = x.stride(0);
    o.s_batch = s.stride(0);
  }
  return o;
}

Tensor matmul_f8(int64_t plan, int device, const Tensor& a, const Tensor& sa, const Tensor& b,
                 const Tensor& sb, const c10::optional<Tensor>& out_, at::ScalarType dtype,
                 const c10::optional<Tensor>& starts, bool accumulate = false,
                 const c10::optional<int64_t>& stream = {}) {
  if (a.dim() != 2 || (b.dim() != 2 && !(b.dim() == 3 && starts)))
    refuse("A must be [M, K] and B [K, N], or [experts, K, N] with starts");
  const int form = !starts ? GEMM_F8_DENSE : b.dim() == 3 ? GEMM_F8_BY_ROWS : GEMM_F8_BY_INNER;
  const int64_t M = a.size(0), K = a.size(1), N = b.size(-1);
  if (b.size(-2) != K) refuse("A and B must have the same inner dimension");
  int64_t experts = 1;
  if (starts) {
    need(*starts, "starts", at::kInt, 1, device);
    experts = starts->size(0) - 1;
    if (experts < 1 || (form == GEMM_F8_BY_ROWS && b.size(0) != experts))
      refuse("starts must have an entry more than there are experts");
  }
  const gemm_f8_operand A = operand(a, sa, "A", true, device);
  const gemm_f8_operand B = operand(b, sb, "B", false, device);
  OnStream on(stream, device);
  Tensor c;
  if (out_) {
    c = *out_;
    on_device(c, "C", device);
    const bool shape = form == GEMM_F8_BY_INNER
                           ? c.dim() == 3 && c.size(0) == experts && c.size(1) == M && c.size(2) == N
                           : c.dim() == 2 && c.size(0) == M && c.size(1) == N;
    if (!shape || (N > 1 && c.stride(-1) != 1)) refuse("C must be row-major and of the product's shape");
    // An expanded tensor: several experts' matrices in the same place.
    if (c.dim() == 3 && experts > 1 && c.stride(0) == 0 && c.numel() > 0)
      refuse("C must have a place for each expert's matrix");
  } else {
    if (accumulate) refuse("accumulate needs C");
    const auto o = a.options().dtype(dtype);
    c = form == GEMM_F8_BY_INNER ? at::empty({experts, M, N}, o) : at::empty({M, N}, o);
  }
  const int type = type_of(c.scalar_type(), "C");
  if (accumulate && type != GEMM_F8_F32) refuse("accumulate needs a float32 C");
  if (c.numel() == 0) return c;
  const gemm_f16_plan_t p = plan_of(plan);
  const int m = narrow(M, "M"), n = narrow(N, "N"), k = narrow(K, "K"), e = narrow(experts, "experts");
  const size_t bytes = gemm_f8_workspace(p, form, m, n, k, e, A.transposed);
  Tensor ws;
  if (bytes > 0) ws = at::empty({(int64_t)bytes}, a.options().dtype(at::kByte));
  check(gemm_f8_run(p, form, m, n, k, e, starts ? ints(*starts) : nullptr, &A, &B, c.data_ptr(),
                    M > 1 ? c.stride(-2) : N, c.dim() == 3 ? c.stride(0) : 0, type, accumulate,
                    bytes > 0 ? ws.data_ptr() : nullptr, bytes, on.raw()),
        "gemm_f8_run");
  // A graph that has saved C must not use it as it is now.
  if (out_ && !c.is_inference()) c.unsafeGetTensorImpl()->bump_version();
  return c;
}

// ------------------------------------------------------------------ experts

// -> (starts, rows, source), or an error code.
py::object expert_maps(int64_t plan, int device, const Tensor& picks, int64_t num_experts,
                       int64_t align, const c10::optional<int64_t>& stream) {
  const bool wide = picks.scalar_type() == at::kLong;
  need(picks, "experts", wide ? at::kLong : at::kInt, 2, device);
  if (!picks.is_contiguous()) refuse("experts must be contiguous");
  const int64_t entries = picks.numel();
  const int64_t most = experts_max_rows(narrow(entries, "experts"), narrow(num_experts, "num_experts"),
                                        narrow(align, "align"));
  if (most < 0) return py::int_(most);
  OnStream on(stream, device);
  const auto o = picks.options().dtype(at::kInt);
  const Tensor starts = at::empty({num_experts + 1}, o), rows = at::empty(picks.sizes(), o),
               source = at::empty({most}, o);
  const int rc = experts_maps(plan_of(plan), (int)entries, picks.const_data_ptr(), wide,
                              (int)num_experts, (int)align, narrow(most, "rows"),
                              starts.data_ptr<int32_t>(), rows.data_ptr<int32_t>(),
                              source.data_ptr<int32_t>(), on.raw());
  return done(rc, py::make_tuple(starts, rows, source));
}

int64_t row_stride(const Tensor& x) { return x.size(0) > 1 ? x.stride(0) : x.size(1); }

void need_rows(const Tensor& x, const char* name, int device) {
  type_of(x.scalar_type(), name);
  need(x, name, x.scalar_type(), 2, device);
}

void need_maps(const Tensor& rows, const Tensor& source, int device) {
  need(rows, "maps.rows", at::kInt, 2, device);
  need(source, "maps.source", at::kInt, 1, device);
  if (!rows.is_contiguous() || rows.size(1) < 1) refuse("maps.rows must be contiguous [tokens, choices]");
}

Tensor expert_gather(int64_t plan, int device, const Tensor& x, const Tensor& rows,
                     const Tensor& source) {
  need_rows(x, "X", device);
  need_maps(rows, source, device);
  if (x.size(0) != rows.size(0)) refuse("X must have a row for each token of the maps");
  OnStream on({}, device);
  const Tensor y = at::empty({source.size(0), x.size(1)}, x.options());
  check(experts_gather(plan_of(plan), type_of(x.scalar_type(), "X"), narrow(source.size(0), "rows"),
                       narrow(x.size(1), "cols"), x.const_data_ptr(), row_stride(x),
                       narrow(x.size(0), "rows"), narrow(rows.size(1), "choices"), ints(source),
                       y.data_ptr(), x.size(1), on.raw()),
        "experts_gather");
  return y;
}

// w: undefined where all weights are 1.
int weights_type(const Tensor& w, const Tensor& s, const Tensor& rows, int device) {
  if (!w.defined()) return GEMM_F8_F32;
  on_device(w, "weights", device);
  if (w.sizes() != rows.sizes() || !w.is_contiguous() ||
      (w.scalar_type() != at::kFloat && w.scalar_type() != s.scalar_type()))
    refuse("weights must be contiguous [tokens, choices], float32 or of the rows' type");
  return type_of(w.scalar_type(), "weights");
}

Tensor expert_combine(int64_t plan, int device, const Tensor& s, const Tensor& rows,
                      const Tensor& source, const Tensor& weights) {
  need_rows(s, "S", device);
  need_maps(rows, source, device);
  if (s.size(0) != source.size(0)) refuse("S must have a row for each row of the maps");
  const int wt = weights_type(weights, s, rows, device);
  OnStream on({}, device);
  const Tensor y = at::empty({rows.size(0), s.size(1)}, s.options());
  check(experts_combine(plan_of(plan), type_of(s.scalar_type(), "S"), narrow(rows.size(0), "tokens"),
                        narrow(rows.size(1), "choices"), narrow(s.size(1), "cols"),
                        s.const_data_ptr(), row_stride(s), narrow(s.size(0), "rows"), ints(rows),
                        weights.defined() ? weights.const_data_ptr() : nullptr, wt, y.data_ptr(),
                        s.size(1), on.raw()),
        "experts_combine");
  return y;
}

// -> the gradients of S and of the weights, undefined where not wanted.
std::pair<Tensor, Tensor> expert_combine_gradient(int64_t plan, int device, const Tensor& dy,
                                                  const Tensor& s, const Tensor& rows,
                                                  const Tensor& source, const Tensor& weights,
                                                  bool want_s, bool want_w) {
  const int64_t n = source.size(0), cols = dy.size(1);
  const int wt = weights_type(weights, dy, rows, device);
  OnStream on({}, device);
  Tensor ds, dw;
  if (want_s) ds = at::empty({n, cols}, dy.options());
  if (want_w) dw = at::empty(weights.sizes(), weights.options());
  check(experts_combine_gradient(
            plan_of(plan), type_of(dy.scalar_type(), "dY"), narrow(rows.size(0), "tokens"),
            narrow(rows.size(1), "choices"), narrow(cols, "cols"), dy.const_data_ptr(),
            row_stride(dy), want_w ? s.const_data_ptr() : nullptr, want_w ? row_stride(s) : 0,
            narrow(n, "rows"), ints(rows), ints(source), weights.const_data_ptr(), wt,
            want_s ? ds.data_ptr() : nullptr, cols, want_w ? dw.data_ptr() : nullptr, on.raw()),
        "experts_combine_gradient");
  return {ds, dw};
}

// ------------------------------------------------------------------ gradients

using torch::autograd::AutogradContext;
using torch::autograd::variable_list;

// A graph of gradients keeps its plan: the Python object, whose handle is None
// once it has been closed.
struct PlanRef : torch::CustomClassHolder {
  py::object plan;
  int device;
  PlanRef(py::object p, int d) : plan(std::move(p)), device(d) {}
  ~PlanRef() override {
    if (!Py_IsInitialized()) {
      plan.release();
      return;
    }
    py::gil_scoped_acquire gil;
    plan = py::object();
  }
  int64_t handle() const {
    py::gil_scoped_acquire gil;
    const py::object h = plan.attr("handle");
    if (h.is_none()) throw std::runtime_error("the plan was closed before the backward pass");
    return h.cast<int64_t>();
  }
};
using Keep = c10::intrusive_ptr<PlanRef>;

void keep(AutogradContext* ctx, const Keep& plan) {
  ctx->saved_data["plan"] = c10::IValue::make_capsule(plan);
}
Keep kept(AutogradContext* ctx) {
  return c10::static_intrusive_pointer_cast<PlanRef>(ctx->saved_data["plan"].toCapsule());
}

// Forward-mode derivatives have no kernels.  torch refuses them where one of its
// functions in C++ is applied, which is only where a gradient is wanted: without
// this a tangent would be lost in silence everywhere else.
void no_tangent(const Tensor& x) {
  TORCH_CHECK_NOT_IMPLEMENTED(
      !x.defined() || !x._fw_grad(0).defined(),
      "8-bit products and experts' rows have no forward-mode derivatives");
}

// A gradient as the calls take it (it may be one number for all of a tensor).
Tensor dense(const Tensor& x) {
  no_tangent(x);
  return x.contiguous();
}

// Gradients that have none of their own: an error where one is asked for.
variable_list once(variable_list grads) {
  if (!at::GradMode::is_enabled()) return grads;
  variable_list some;
  for (const Tensor& g : grads)
    if (g.defined()) some.push_back(g.detach().set_requires_grad(true));
  auto fn = std::make_shared<torch::autograd::DelayedError>(
      "8-bit products and weighted sums of experts' rows have first gradients only",
      (int)some.size());
  some = (*fn)(std::move(some));
  size_t at = 0;
  for (Tensor& g : grads)
    if (g.defined()) g = some[at++];
  return grads;
}

// Y = X W^T; formats[0] that of X and W, [1] that of dY.  Without w, W comes as
// codes and scales of tiles.
struct LinearCall {
  Keep plan;
  Tensor codes, scales;
  c10::optional<Tensor> starts;
  at::ScalarType formats[2];
  bool want_x, want_w;     // gradients that a backward pass may ask for
};

struct Linear : torch::autograd::Function<Linear> {
  static Tensor run(AutogradContext* ctx, const Tensor& x, const c10::optional<Tensor>& w,
                    const LinearCall& call) {
    const int64_t plan = call.plan->handle();
    const int device = call.plan->device;
    const Quantized qw = w ? quantize(plan, device, *w, GEMM_F8_TILES, call.formats[0])
                           : Quantized{call.codes, call.scales, {}, {}};
    const Quantized qx =
        quantize(plan, device, x, call.want_w ? GEMM_F8_BOTH : GEMM_F8_ROWS, call.formats[0]);
    if (ctx) {
      keep(ctx, call.plan);
      ctx->saved_data["x"] = x.scalar_type();
      ctx->saved_data["w"] = w ? w->scalar_type() : x.scalar_type();
      ctx->saved_data["format"] = call.formats[1];
      ctx->save_for_backward({qx.q2, qx.s2, call.want_x ? qw.q : Tensor(),
                              call.want_x ? qw.s : Tensor(), call.starts ? *call.starts : Tensor()});
    }
    return matmul_f8(plan, device, qx.q, qx.s, qw.q.transpose(-1, -2), qw.s.transpose(-1, -2), {},
                     x.scalar_type(), call.starts);
  }
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const c10::optional<Tensor>& w,
                        const LinearCall& call) {
    return run(ctx, x, w, call);
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const variable_list saved = ctx->get_saved_variables();
    const Tensor &xq = saved[0], &xs = saved[1], &wq = saved[2], &ws = saved[3];
    const auto starts = saved[4].defined() ? c10::optional<Tensor>(saved[4]) : c10::nullopt;
    const auto type = [&](const char* key) {
      return static_cast<at::ScalarType>(ctx->saved_data[key].toInt());
    };
    const bool want_x = wq.defined() && ctx->needs_input_grad(0);
    const bool want_w = xq.defined() && ctx->needs_input_grad(1);
    variable_list out(3);
    if (!want_x && !want_w) return out;
    const Keep plan = kept(ctx);
    const int64_t h = plan->handle();
    {
      at::AutoGradMode off(false);
      const Tensor dy = dense(grads[0]);
      if (dy.size(1) == 0) {     // W has no rows: there is nothing to quantise
        if (want_x) out[0] = at::zeros({dy.size(0), wq.size(-1)}, dy.options().dtype(type("x")));
        if (want_w) {
          std::vector<int64_t> shape = {0, xq.size(1)};
          if (starts) shape.insert(shape.begin(), starts->size(0) - 1);
          out[1] = at::zeros(shape, dy.options().dtype(type("w")));
        }
        return once(std::move(out));
      }
      const Quantized g =
          quantize(h, plan->device, dy,
                   want_x && want_w ? GEMM_F8_BOTH : want_x ? GEMM_F8_ROWS : GEMM_F8_COLUMNS,
                   type("format"));
      if (want_x) out[0] = matmul_f8(h, plan->device, g.q, g.s, wq, ws, {}, type("x"), starts);
      if (want_w) {
        const Tensor &q = want_x ? g.q2 : g.q, &s = want_x ? g.s2 : g.s;
        out[1] = matmul_f8(h, plan->device, q.transpose(-1, -2), s.transpose(-1, -2), xq, xs, {},
                           type("w"), starts);
      }
    }
    return once(std::move(out));
  }
};

Tensor gather_call(const Keep& plan, const Tensor& x, const Tensor& rows, const Tensor& source);
Tensor combine_call(const Keep& plan, const Tensor& s, const Tensor& weights, const Tensor& rows,
                    const Tensor& source);

struct MapsCall {
  Keep plan;
  Tensor rows, source;
};

// The gradients of these two are one another, and so have gradients themselves.
struct Gather : torch::autograd::Function<Gather> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const MapsCall& call) {
    keep(ctx, call.plan);
    ctx->save_for_backward({call.rows, call.source});
    return expert_gather(call.plan->handle(), call.plan->device, x, call.rows, call.source);
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const variable_list saved = ctx->get_saved_variables();
    return {combine_call(kept(ctx), dense(grads[0]), {}, saved[0], saved[1]), {}};
  }
};

struct Combine : torch::autograd::Function<Combine> {
  static Tensor forward(AutogradContext* ctx, const Tensor& s, const c10::optional<Tensor>& weights,
                        const MapsCall& call) {
    keep(ctx, call.plan);
    const Tensor w = weights ? *weights : Tensor();
    ctx->save_for_backward({w.defined() && w.requires_grad() ? s : Tensor(), w, call.rows, call.source});
    return expert_combine(call.plan->handle(), call.plan->device, s, call.rows, call.source, w);
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const variable_list saved = ctx->get_saved_variables();
    const Tensor &s = saved[0], &weights = saved[1], &rows = saved[2], &source = saved[3];
    const Keep plan = kept(ctx);
    variable_list out(3);
    if (!weights.defined()) {
      out[0] = gather_call(plan, dense(grads[0]), rows, source);
      return out;
    }
    const bool want_s = ctx->needs_input_grad(0), want_w = s.defined() && ctx->needs_input_grad(1);
    if (!want_s && !want_w) return out;
    {
      at::AutoGradMode off(false);
      std::tie(out[0], out[1]) =
          expert_combine_gradient(plan->handle(), plan->device, dense(grads[0]), s, rows, source,
                                  weights, want_s, want_w);
    }
    return once(std::move(out));
  }
};

bool wants(const Tensor& x) {
  return at::GradMode::is_enabled() && x.defined() && x.requires_grad();
}

Tensor gather_call(const Keep& plan, const Tensor& x, const Tensor& rows, const Tensor& source) {
  no_tangent(x);
  if (wants(x)) return Gather::apply(x, MapsCall{plan, rows, source});
  return expert_gather(plan->handle(), plan->device, x, rows, source);
}
Tensor combine_call(const Keep& plan, const Tensor& s, const Tensor& weights, const Tensor& rows,
                    const Tensor& source) {
  no_tangent(s);
  no_tangent(weights);
  if (wants(s) || wants(weights))
    return Combine::apply(s, weights.defined() ? c10::optional<Tensor>(weights) : c10::nullopt,
                          MapsCall{plan, rows, source});
  return expert_combine(plan->handle(), plan->device, s, rows, source, weights);
}

Tensor linear_f8(const py::object& plan, int device, const Tensor& x_, const Tensor& w,
                 const Tensor& codes, const Tensor& scales, const c10::optional<Tensor>& starts,
                 at::ScalarType format, at::ScalarType grad_format) {
  if (x_.dim() < 1) refuse("X must be [.., K]");
  if (starts && x_.dim() != 2) refuse("X must be [rows, K] where starts are given");
  const Tensor& W = w.defined() ? w : codes;
  if (W.dim() != (starts ? 3 : 2)) refuse("W must be [N, K], or [experts, N, K] with starts");
  if (!w.defined() && (scales.dim() != W.dim() || scales.size(-2) != blocks_of(W.size(-2)) ||
                       scales.size(-1) != blocks_of(W.size(-1))))
    refuse("W's blocks must be tiles");
  no_tangent(x_);
  no_tangent(w);
  const Tensor x = x_.dim() == 2 ? x_ : x_.reshape({x_.numel() / std::max<int64_t>(x_.size(-1), 1), x_.size(-1)});
  const LinearCall call = {c10::make_intrusive<PlanRef>(plan, device), codes, scales, starts,
                           {format, grad_format}, wants(x), wants(w)};
  const c10::optional<Tensor> given = w.defined() ? c10::optional<Tensor>(w) : c10::nullopt;
  const Tensor y = call.want_x || call.want_w ? Linear::apply(x, given, call)
                                              : Linear::run(nullptr, x, given, call);
  if (x_.dim() == 2) return y;
  std::vector<int64_t> shape(x_.sizes().begin(), x_.sizes().end());
  shape.back() = y.size(1);
  return y.view(shape);
}

at::ScalarType codes_type(int format) {
  return format == GEMM_F8_E5M2 ? at::kFloat8_e5m2 : at::kFloat8_e4m3fn;
}
Tensor or_none(const c10::optional<Tensor>& x) { return x ? *x : Tensor(); }

void add_f8_calls(py::module_& m) {
  // -> (codes, scales) or, for BOTH, (codes, scales, codes, scales)
  m.def("quantize", [](int64_t plan, int device, const Tensor& x, int blocks, int format,
                       const c10::optional<Tensor>& source, int64_t choices,
                       const c10::optional<int64_t>& stream) {
    return answer([&]() -> py::object {
      const Quantized r =
          quantize(plan, device, x, blocks, codes_type(format), source, choices, stream);
      return blocks == GEMM_F8_BOTH ? py::make_tuple(r.q, r.s, r.q2, r.s2)
                                    : py::make_tuple(r.q, r.s);
    });
  });
  m.def("matmul_f8", [](int64_t plan, int device, const Tensor& a, const Tensor& sa, const Tensor& b,
                        const Tensor& sb, const c10::optional<Tensor>& out, int type,
                        const c10::optional<Tensor>& starts, bool accumulate,
                        const c10::optional<int64_t>& stream) {
    return answer([&]() -> py::object {
      return py::cast(matmul_f8(plan, device, a, sa, b, sb, out,
                                type == GEMM_F8_F16    ? at::kHalf
                                : type == GEMM_F8_BF16 ? at::kBFloat16
                                                       : at::kFloat,
                                starts, accumulate, stream));
    });
  });
  m.def("linear_f8", [](const py::object& plan, int device, const Tensor& x,
                        const c10::optional<Tensor>& w, const c10::optional<Tensor>& codes,
                        const c10::optional<Tensor>& scales, const c10::optional<Tensor>& starts,
                        int format, int grad_format) {
    return answer([&]() -> py::object {
      return py::cast(linear_f8(plan, device, x, or_none(w), or_none(codes), or_none(scales), starts,
                                codes_type(format), codes_type(grad_format)));
    });
  });
  m.def("expert_maps", &expert_maps);
  m.def("expert_gather", [](const py::object& plan, int device, const Tensor& x, const Tensor& rows,
                            const Tensor& source) {
    return answer([&]() -> py::object {
      return py::cast(
          gather_call(c10::make_intrusive<PlanRef>(plan, device), x, rows, source));
    });
  });
  m.def("expert_combine", [](const py::object& plan, int device, const Tensor& s, const Tensor& rows,
                             const Tensor& source, const c10::optional<Tensor>& weights) {
    return answer([&]() -> py::object {
      return py::cast(combine_call(c10::make_intrusive<PlanRef>(plan, device), s, or_none(weights),
                                   rows, source));
    });
  });
}

}  // namespace

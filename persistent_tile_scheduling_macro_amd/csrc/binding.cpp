// torch binding of the routed operators and the 4-bit product (module _ops).
//
// Checks shapes and types, makes the outputs and passes pointers to the C ABI
// on torch's current stream: what a call of a few microseconds on the GPU can
// afford on the host (a combine of 16 tokens took 10.7 us of Python). No
// arithmetic happens here. Shapes that do not belong together raise
// ValueError, wrong types TypeError, a refusal of the library PgemmError, a
// forward-mode tangent NotImplementedError.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/AutogradState.h>
#include <c10/hip/HIPGraphsC10Utils.h>
#include <c10/hip/HIPGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/utils/pybind.h>

#include <mutex>
#include <sstream>
#include <string>
#include <vector>

#include "../../include/pgemm.h"

namespace py = pybind11;
using at::Tensor;

namespace {

std::string join(std::initializer_list<std::string> parts) {
  std::string s;
  for (const auto& p : parts) s += p;
  return s;
}
std::string shape(const Tensor& t) {
  std::ostringstream s;
  s << t.sizes();
  return s.str();
}
std::string num(int64_t v) { return std::to_string(v); }
[[noreturn]] void value(const std::string& s) { throw py::value_error(s); }
[[noreturn]] void type(const std::string& s) { throw py::type_error(s); }

int dtype_of(const Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return PGEMM_BF16;
  if (t.scalar_type() == at::kHalf) return PGEMM_F16;
  type(join({name, " is ", c10::toString(t.scalar_type()), ", not float16 or bfloat16"}));
}

// A tangent of t would be lost: the kernels read values only. (Inside an autograd function torch has turned
// forward mode off and refuses the tangent itself.)
void no_tangent(const Tensor& t, const char* name) {
  if (!c10::AutogradState::get_tls_state().get_fw_grad_mode() || !t._fw_grad(0).defined()) return;
  PyErr_SetString(PyExc_NotImplementedError, join({name, " carries a tangent: forward-mode derivatives are not implemented"}).c_str());
  throw py::error_already_set();
}

// A 2-D fp16/bf16 tensor whose rows are contiguous (a copy of one whose are not).
Tensor rows_of(const Tensor& t, const char* name) {
  dtype_of(t, name);
  no_tangent(t, name);
  if (t.dim() != 2) value(join({name, " has shape ", shape(t), ", not two dimensions"}));
  // a negative stride cannot occur in torch; one that repeats a row (0) is fine
  return t.stride(1) == 1 || t.size(1) <= 1 ? t : t.contiguous();
}

void on_device(const char* name, std::initializer_list<const Tensor*> tensors) {
  const Tensor& first = **tensors.begin();
  for (const Tensor* t : tensors) {
    if (!t->is_cuda()) value(join({name, ": every tensor must be on the GPU"}));
    if (t->device() != first.device()) value(join({name, ": tensors on ", first.device().str(), " and ", t->device().str()}));
  }
}

Tensor make(at::IntArrayRef sizes, const Tensor& like, at::ScalarType type) {
  return at::empty(sizes, at::TensorOptions().dtype(type).device(like.device()));
}

// One handle per device, made at its first use. `lock` is held from binding
// the stream to the last launch; the GIL is not held meanwhile.
struct Handle {
  pgemm_handle_t h = nullptr;
  void* stream = nullptr;
};
std::mutex lock;
std::vector<Handle> handles;

void raise(int status, const std::string& detail) {
  py::object cls = py::module_::import("persistent_tile_scheduling_macro_amd").attr("PgemmError");
  py::object e = cls(status, detail);
  PyErr_SetObject(cls.ptr(), e.ptr());
  throw py::error_already_set();
}

// Runs call(handle) with the handle of t's device bound to the current stream there.
template <class F>
void run(const Tensor& t, F call) {
  const int device = t.device().index();
  void* stream = c10::hip::getCurrentHIPStream(device).stream();
  int status = PGEMM_OK;
  std::string detail;
  bool early = false;
  {
    py::gil_scoped_release no_gil;
    std::lock_guard<std::mutex> guard(lock);
    if (handles.size() <= (size_t)device) handles.resize(device + 1);
    Handle& k = handles[device];
    if (!k.h) {
      if (c10::hip::currentStreamCaptureStatusMayInitCtx() != c10::hip::CaptureStatus::None) {
        early = true;
      } else {
        c10::hip::HIPGuard keep(device); // pgemm_create makes its device current
        status = pgemm_create(&k.h, device);
        k.stream = nullptr;
      }
    }
    if (k.h && status == PGEMM_OK) {
      if (k.stream != stream) {
        status = pgemm_set_stream(k.h, stream);
        k.stream = stream;
      }
      if (status == PGEMM_OK) status = call(k.h);
      if (status != PGEMM_OK) detail = pgemm_last_error(k.h);
    }
  }
  if (early) throw std::runtime_error("call an operator once outside graph capture first: the device's handle is made then");
  if (status != PGEMM_OK) raise(status, detail);
}

template <class T = void>
T* ptr(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// ------------------------------------------------------------------ routing
struct Plan {
  const Tensor &offsets, &order, &pos;
  int64_t k, T, n;
};
Plan check_plan(const char* name, const Tensor& offsets, const Tensor& order, const Tensor& pos, int64_t k) {
  const std::pair<const char*, const Tensor*> all[] = {{"offsets", &offsets}, {"order", &order}, {"pos", &pos}};
  for (const auto& p : all)
    if (p.second->scalar_type() != at::kInt || p.second->dim() != 1 || !p.second->is_contiguous())
      value(join({name, ": plan.", p.first, " must be a contiguous int32 vector"}));
  const int64_t n = pos.numel();
  if (k < 1 || n % k || order.numel() != n || offsets.numel() < 2)
    value(join({name, ": the plan's sizes do not belong together"}));
  return {offsets, order, pos, k, n / k, n};
}

std::tuple<Tensor, Tensor, Tensor, Tensor> dispatch(const Tensor& x_, const Tensor& ids_, int64_t E) {
  const Tensor x = rows_of(x_, "x");
  const int64_t T = x.size(0), H = x.size(1);
  if (ids_.scalar_type() != at::kInt && ids_.scalar_type() != at::kLong)
    type(join({"ids are ", c10::toString(ids_.scalar_type()), ", not int32 or int64"}));
  if (ids_.dim() != 2 || ids_.size(0) != T || ids_.size(1) < 1)
    value(join({"ids have shape ", shape(ids_), ", not [", num(T), ", k]"}));
  if (E < 1) value(join({"num_experts is ", num(E)}));
  on_device("dispatch", {&x, &ids_});
  const Tensor ids = ids_.contiguous();
  const int64_t k = ids.size(1), n = T * k;
  int64_t bytes = 0;
  const int rc = pgemm_moe_dispatch_workspace(T, k, E, &bytes);
  if (rc != PGEMM_OK) raise(rc, "dispatch of " + num(n) + " slots to " + num(E) + " experts");
  const Tensor offsets = make({E + 1}, x, at::kInt), order = make({n}, x, at::kInt), pos = make({n}, x, at::kInt);
  const Tensor xs = make({n, H}, x, x.scalar_type());
  Tensor work;
  if (bytes) work = make({bytes}, x, at::kByte);
  run(x, [&](pgemm_handle_t h) {
    return pgemm_moe_dispatch(h, ptr(x), x.stride(0), ptr(ids), ids.scalar_type() == at::kInt ? PGEMM_IDS_I32 : PGEMM_IDS_I64, T,
                              k, E, H, dtype_of(x, "x"), ptr<int32_t>(offsets), ptr<int32_t>(order), ptr<int32_t>(pos), ptr(xs),
                              bytes ? ptr(work) : nullptr, bytes);
  });
  return {xs, offsets, order, pos};
}

Tensor dispatch_backward(const Tensor& dxs_, const Tensor& offsets, const Tensor& order, const Tensor& pos, int64_t k) {
  const Plan p = check_plan("dispatch_backward", offsets, order, pos, k);
  const Tensor dxs = rows_of(dxs_, "dxs");
  if (dxs.size(0) != p.n) value(join({"dxs has ", num(dxs.size(0)), " rows, the plan ", num(p.n)}));
  on_device("dispatch_backward", {&dxs, &pos});
  const int64_t H = dxs.size(1);
  const Tensor dx = make({p.T, H}, dxs, dxs.scalar_type());
  run(dxs, [&](pgemm_handle_t h) {
    return pgemm_moe_dispatch_backward(h, ptr(dxs), dxs.stride(0), ptr<int32_t>(pos), p.T, k, H, dtype_of(dxs, "dxs"), ptr(dx));
  });
  return dx;
}

// (ys, weights) as the combine steps take them.
std::pair<Tensor, Tensor> check_combine(const char* name, const Tensor& ys_, const Tensor& w, const Plan& p) {
  Tensor ys = rows_of(ys_, "ys");
  if (ys.size(0) != p.n) value(join({name, ": ys has ", num(ys.size(0)), " rows, the plan ", num(p.n)}));
  if (w.scalar_type() != at::kFloat) type(join({name, ": weights are ", c10::toString(w.scalar_type()), ", not float32"}));
  no_tangent(w, "weights");
  if (w.dim() != 2 || w.size(0) != p.T || w.size(1) != p.k)
    value(join({name, ": weights have shape ", shape(w), ", not [", num(p.T), ", ", num(p.k), "]"}));
  return {ys, w.contiguous()};
}

Tensor combine(const Tensor& ys_, const Tensor& w_, const Tensor& offsets, const Tensor& order, const Tensor& pos, int64_t k) {
  const Plan p = check_plan("combine", offsets, order, pos, k);
  const auto [ys, w] = check_combine("combine", ys_, w_, p);
  on_device("combine", {&ys, &w, &pos});
  const int64_t H = ys.size(1);
  const Tensor out = make({p.T, H}, ys, ys.scalar_type());
  run(ys, [&, &ys = ys, &w = w](pgemm_handle_t h) {
    return pgemm_moe_combine(h, ptr(ys), ys.stride(0), ptr<float>(w), ptr<int32_t>(pos), p.T, k, H, dtype_of(ys, "ys"), ptr(out));
  });
  return out;
}

std::tuple<Tensor, Tensor> combine_backward(const Tensor& dout_, const Tensor& ys_, const Tensor& w_, const Tensor& offsets,
                                            const Tensor& order, const Tensor& pos, int64_t k) {
  const Plan p = check_plan("combine_backward", offsets, order, pos, k);
  const auto [ys, w] = check_combine("combine_backward", ys_, w_, p);
  const int64_t H = ys.size(1);
  const Tensor dout = rows_of(dout_, "dout");
  if (dout.size(0) != p.T || dout.size(1) != H)
    value(join({"dout has shape ", shape(dout), ", not [", num(p.T), ", ", num(H), "]"}));
  if (dout.scalar_type() != ys.scalar_type())
    type(join({"combine_backward: dout is ", c10::toString(dout.scalar_type()), ", ys ", c10::toString(ys.scalar_type())}));
  on_device("combine_backward", {&ys, &dout, &w, &pos, &order, &offsets});
  const Tensor dys = make({p.n, H}, ys, ys.scalar_type()), dw = make({p.T, k}, ys, at::kFloat);
  run(ys, [&, &ys = ys, &w = w](pgemm_handle_t h) {
    return pgemm_moe_combine_backward_plan(h, ptr(dout), dout.stride(0), ptr(ys), ys.stride(0), ptr<float>(w),
                                           ptr<int32_t>(offsets), ptr<int32_t>(order), ptr<int32_t>(pos), p.T, k,
                                           offsets.numel() - 1, H, dtype_of(ys, "ys"), ptr(dys), ptr<float>(dw));
  });
  return {dys, dw};
}

// ----------------------------------------------------------- experts' products
struct Grouped {
  Tensor x, w, offsets;
  int64_t R, E, K, N;
};
Grouped check_grouped(const char* name, const Tensor& x_, const Tensor& w, const Tensor& offsets, bool nk) {
  const Tensor x = rows_of(x_, "x");
  if (w.scalar_type() != x.scalar_type())
    type(join({name, ": w is ", c10::toString(w.scalar_type()), ", x ", c10::toString(x.scalar_type())}));
  no_tangent(w, "w");
  const int64_t K = x.size(1);
  if (w.dim() != 3 || w.size(0) < 1 || w.size(nk ? 2 : 1) != K)
    value(join({name, ": w has shape ", shape(w), " for rows of ", num(K), " and layout ", nk ? "'nk'" : "'kn'"}));
  if (offsets.scalar_type() != at::kInt || offsets.dim() != 1 || offsets.size(0) != w.size(0) + 1)
    value(join({name, ": offsets must be int32 of shape [", num(w.size(0) + 1), "]"}));
  on_device(name, {&x, &w, &offsets});
  return {x, w.contiguous(), offsets.contiguous(), x.size(0), w.size(0), K, w.size(nk ? 1 : 2)};
}

Tensor grouped_rows(const Tensor& x, const Tensor& w, const Tensor& offsets, int64_t E, int64_t K, int64_t N, bool nk) {
  const Tensor y = make({x.size(0), N}, x, x.scalar_type());
  run(x, [&](pgemm_handle_t h) {
    return pgemm_grouped_run(h, ptr(x), x.stride(0), ptr(w), ptr<int32_t>(offsets), ptr(y), x.size(0), E, K, N,
                             nk ? PGEMM_B_NK : PGEMM_B_KN, dtype_of(x, "x"));
  });
  return y;
}

Tensor grouped(const Tensor& x, const Tensor& w, const Tensor& offsets, bool nk) {
  const Grouped g = check_grouped("grouped_matmul", x, w, offsets, nk);
  return grouped_rows(g.x, g.w, g.offsets, g.E, g.K, g.N, nk);
}

std::tuple<c10::optional<Tensor>, c10::optional<Tensor>> grouped_backward(const Tensor& dy_, const Tensor& x, const Tensor& w,
                                                                          const Tensor& offsets, bool nk, bool need_dx,
                                                                          bool need_dw) {
  const Tensor dy = rows_of(dy_, "dy");
  const Grouped g = check_grouped("grouped_matmul_backward", x, w, offsets, nk);
  if (dy.size(0) != g.R || dy.size(1) != g.N)
    value(join({"dy has shape ", shape(dy), ", not [", num(g.R), ", ", num(g.N), "]"}));
  if (dy.scalar_type() != g.x.scalar_type())
    type(join({"grouped_matmul_backward: dy is ", c10::toString(dy.scalar_type()), ", x ", c10::toString(g.x.scalar_type())}));
  on_device("grouped_matmul_backward", {&g.x, &dy});
  c10::optional<Tensor> dx, dw;
  if (need_dx) dx = grouped_rows(dy, g.w, g.offsets, g.E, g.N, g.K, !nk);
  if (need_dw) {
    const Tensor &a = nk ? dy : g.x, &b = nk ? g.x : dy;
    dw = make({g.E, a.size(1), b.size(1)}, a, a.scalar_type());
    int64_t bytes = 0;
    const int rc = pgemm_grouped_weight_grad_workspace(g.R, g.E, a.size(1), b.size(1), &bytes);
    if (rc != PGEMM_OK) raise(rc, "gradient of " + num(g.E) + " matrices");
    Tensor work;
    if (bytes) work = make({bytes}, a, at::kByte);
    run(a, [&](pgemm_handle_t h) {
      return pgemm_grouped_weight_grad(h, ptr(a), a.stride(0), ptr(b), b.stride(0), ptr<int32_t>(g.offsets), ptr(*dw), g.R, g.E,
                                       a.size(1), b.size(1), dtype_of(a, "x"), bytes ? ptr(work) : nullptr, bytes);
    });
  }
  return {dx, dw};
}

// --------------------------------------------------------------- 4-bit product
Tensor w4(const Tensor& x_, const Tensor& q_, const Tensor& scales_, const c10::optional<Tensor>& zeros_, int64_t group, int fmt,
          const c10::optional<Tensor>& offsets_) {
  const Tensor x = rows_of(x_, "x");
  const int64_t M = x.size(0), K = x.size(1);
  if (group != 32 && group != 64 && group != 128) value(join({"group ", num(group), " is not 32, 64 or 128"}));
  if (q_.scalar_type() != at::kByte) type(join({"q is ", c10::toString(q_.scalar_type()), ", not uint8"}));
  if (scales_.scalar_type() != x.scalar_type())
    type(join({"scales are ", c10::toString(scales_.scalar_type()), ", x ", c10::toString(x.scalar_type())}));
  no_tangent(scales_, "scales");
  const int lead = offsets_ ? 1 : 0;
  if (q_.dim() != lead + 2 || q_.size(-1) != (K + 1) / 2)
    value(join({"q has shape ", shape(q_), " for K = ", num(K), offsets_ ? " and offsets" : ""}));
  const int64_t N = q_.size(-2), E = offsets_ ? q_.size(0) : 1, groups = (K + group - 1) / group;
  auto per_group = [&](const Tensor& t) {
    return t.dim() == lead + 2 && t.size(-1) == groups && t.size(-2) == N && (!lead || t.size(0) == E);
  };
  if (!per_group(scales_)) value(join({"scales have shape ", shape(scales_), " for q of ", shape(q_), " and groups of ", num(group)}));
  if (zeros_) {
    if (fmt != PGEMM_W4_INT4) value("e2m1 weights have no zero points");
    if (zeros_->scalar_type() != at::kByte) type(join({"zeros are ", c10::toString(zeros_->scalar_type()), ", not uint8"}));
    if (!per_group(*zeros_)) value(join({"zeros have shape ", shape(*zeros_), ", scales ", shape(scales_)}));
    on_device("w4.matmul", {&x, &*zeros_});
  }
  if (offsets_) {
    if (offsets_->scalar_type() != at::kInt || offsets_->dim() != 1 || offsets_->size(0) != E + 1)
      value(join({"offsets must be int32 of shape [", num(E + 1), "]"}));
    if (E < 1) value("q holds no expert");
    on_device("w4.matmul", {&x, &*offsets_});
  }
  on_device("w4.matmul", {&x, &q_, &scales_});
  const Tensor q = q_.contiguous(), scales = scales_.contiguous();
  const Tensor zeros = zeros_ ? zeros_->contiguous() : Tensor(), offsets = offsets_ ? offsets_->contiguous() : Tensor();
  const Tensor y = make({M, N}, x, x.scalar_type());
  run(x, [&](pgemm_handle_t h) {
    return pgemm_w4_run(h, ptr(x), x.stride(0), ptr(q), ptr(scales), zeros_ ? ptr(zeros) : nullptr,
                        offsets_ ? ptr<int32_t>(offsets) : nullptr, ptr(y), M, N, K, E, (int)group, fmt, dtype_of(x, "x"));
  });
  return y;
}

} // namespace

PYBIND11_MODULE(_ops, m) {
  m.def("dispatch", &dispatch);
  m.def("dispatch_backward", &dispatch_backward);
  m.def("combine", &combine);
  m.def("combine_backward", &combine_backward);
  m.def("grouped", &grouped);
  m.def("grouped_backward", &grouped_backward);
  m.def("w4", &w4);
}

// Differentiable attention as a node of PyTorch's graph: allocates outputs and workspace, calls
// fa_fwd_sinks and fa_bwd_sinks on the current stream. It holds no arithmetic.
//
// A step over short sequences is host time: B2 Hq6 Hkv2 T1500 D64 with a window is 47 us of kernels,
// and took 334 us with forward and backward written in Python. The backward runs in a thread of
// PyTorch's own, which in Python has to wait for the interpreter's lock besides. Here 188 to 210 us, of which
// PyTorch takes 105 for a graph of one node.
#pragma once

#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/accumulate_grad.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/graph_task.h>

namespace attention {

// Sets FaError(status, what) as the Python error (the interpreter's lock is held).
inline void set_status_error(int status, const char* what) {
  PyObject* package = PyImport_ImportModule("attention_fa_fwd_03_gb300");
  PyObject* type = package ? PyObject_GetAttrString(package, "FaError") : nullptr;
  PyObject* error = type ? PyObject_CallFunction(type, "is", status, what) : nullptr;
  if (error) PyErr_SetObject(type, error);  // (else the error that there is)
  Py_XDECREF(error);
  Py_XDECREF(type);
  Py_XDECREF(package);
}

// Throws the status as a Python error, from a thread that does not hold the lock.
inline void check_status(fa_status status, const char* what) {
  if (status == FA_OK) return;
  pybind11::gil_scoped_acquire lock;
  set_status_error(status, what);
  python_error error;
  error.persist();
  throw std::move(error);
}

inline cudaStream_t current_stream(const at::Tensor& t) {
  return c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
}

// A leaf's gradient is added, or handed out, on the stream on which the leaf was first used, as long
// as a graph of that time lives. Within a capture that must not be the legacy default stream: CUDA
// refuses it, and PyTorch may end the process over that. So such a backward is refused here.
inline void refuse_leaves_of_default_stream(const c10::cuda::CUDAStream& current) {
  if (c10::cuda::currentStreamCaptureStatusMayInitCtx() == c10::cuda::CaptureStatus::None) return;
  const std::shared_ptr<torch::autograd::Node> node = torch::autograd::get_current_node();
  if (!node) return;
  const auto* info = torch::autograd::get_current_graph_task_exec_info();
  for (const torch::autograd::Edge& edge : node->next_edges()) {
    auto* leaf = dynamic_cast<torch::autograd::AccumulateGrad*>(edge.function.get());
    if (!leaf) continue;
    if (info && !info->empty()) {  // gradients of named tensors only
      const auto it = info->find(leaf);
      if (it == info->end() || !it->second.should_execute()) continue;
    }
    const auto stream = leaf->stream();
    if (stream && *stream != current.unwrap() && c10::cuda::CUDAStream(*stream).stream() == nullptr)
      throw std::runtime_error(
          "flash_attention: this backward pass is being captured into a CUDA graph while an eager graph of the same leaves "
          "from the default stream lives; delete its outputs first");
  }
}

// The gradients are kernels' outputs without a graph. Where one is being made of them
// (create_graph) they get a node that raises if it is differentiated: without it a second
// derivative would leave attention's part out without a word.
inline torch::autograd::variable_list not_differentiable_again(torch::autograd::variable_list grads) {
  if (!at::GradMode::is_enabled()) return grads;
  for (at::Tensor& g : grads) g.requires_grad_();
  const auto raise = std::make_shared<torch::autograd::DelayedError>(
      "flash_attention has no second derivative: its gradients cannot be differentiated", static_cast<int64_t>(grads.size()));
  return (*raise)(std::move(grads));
}

struct Sizes {
  int B, Hq, Hkv, Tq, Tkv, D;
  fa_dtype dt;
  Sizes(const at::Tensor& q, const at::Tensor& k)
      : B(n(q, 0)), Hq(n(q, 1)), Hkv(n(k, 1)), Tq(n(q, 2)), Tkv(n(k, 2)), D(n(q, 3)),
        dt(q.scalar_type() == at::kBFloat16 ? FA_BF16 : FA_FP16) {}
  // (beyond 32 bits the library refuses, as it does 0)
  static int n(const at::Tensor& t, int i) { return t.size(i) > INT_MAX ? 0 : static_cast<int>(t.size(i)); }
};

class Node : public torch::autograd::Function<Node> {
 public:
  using Context = torch::autograd::AutogradContext;
  using List = torch::autograd::variable_list;

  static List forward(Context* ctx, const at::Tensor& q, const at::Tensor& k, const at::Tensor& v, double scale,
                      bool causal, int64_t window, int64_t sinks) {
    const c10::cuda::CUDAGuard on(q.device());
    const Sizes s(q, k);
    at::Tensor o = at::empty_like(q), lse = at::empty({q.size(0), q.size(1), q.size(2)}, q.options().dtype(at::kFloat));
    check_status(fa_fwd_sinks(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr<float>(), s.B, s.Hq,
                              s.Hkv, s.Tq, s.Tkv, s.D, static_cast<float>(scale), causal, static_cast<int>(window),
                              static_cast<int>(sinks), s.dt, current_stream(q)),
                 "fa_fwd");
    ctx->save_for_backward({q, k, v, o, lse});
    ctx->saved_data["scale"] = scale;
    ctx->saved_data["causal"] = causal;
    ctx->saved_data["window"] = window;
    ctx->saved_data["sinks"] = sinks;
    ctx->mark_non_differentiable({lse});
    return {o, lse};
  }

  static List backward(Context* ctx, List grads) {
    const List saved = ctx->get_saved_variables();
    refuse_leaves_of_default_stream(c10::cuda::getCurrentCUDAStream(saved[0].get_device()));
    const at::Tensor &q = saved[0], &k = saved[1], &v = saved[2], &o = saved[3], &lse = saved[4];
    const c10::cuda::CUDAGuard on(q.device());
    const Sizes s(q, k);
    const int window = static_cast<int>(ctx->saved_data["window"].toInt());
    const int sinks = static_cast<int>(ctx->saved_data["sinks"].toInt());
    const at::Tensor d_o = grads[0].contiguous();
    at::Tensor dq = at::empty_like(q), dk = at::empty_like(k), dv = at::empty_like(v);
    const size_t bytes = sinks ? fa_bwd_sinks_workspace_size(s.B, s.Hq, s.Hkv, s.Tq, s.Tkv, s.D, window, sinks)
                               : fa_bwd_workspace_size(s.B, s.Hq, s.Tq);
    at::Tensor workspace = at::empty({static_cast<int64_t>(bytes)}, q.options().dtype(at::kByte));
    check_status(fa_bwd_sinks(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), d_o.data_ptr(), lse.data_ptr<float>(),
                              dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), s.B, s.Hq, s.Hkv, s.Tq, s.Tkv, s.D,
                              static_cast<float>(ctx->saved_data["scale"].toDouble()), ctx->saved_data["causal"].toBool(),
                              window, sinks, s.dt, workspace.data_ptr(), bytes, current_stream(q)),
                 "fa_bwd");
    List out = not_differentiable_again({dq, dk, dv});
    out.resize(7);  // (none of scale, causal, window and sinks)
    return out;
  }
};

}  // namespace attention

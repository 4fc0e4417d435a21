// What the binding's files share: checks of tensors, where a call runs and allocates, its scratch.
#pragma once

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include <climits>
#include <string>
#include <type_traits>
#include <utility>

#include "wtconv.h"
#include "wtconv_scan.h"

namespace py = pybind11;
using at::Tensor;
using c10::optional;

namespace binding {

[[noreturn]] inline void refuse(const std::string &why) { throw py::value_error(why); }

inline void check_status(int status, const char *where) {
    if (status == WTCONV_OK) return;
    const py::object type = py::module_::import("memory_bound_cnn_gb300.wtconv").attr("WTConvError");
    const py::object error = type(status, where);
    PyErr_SetObject(type.ptr(), error.ptr());
    throw py::error_already_set();
}

inline int dtype_code(at::ScalarType t) {
    return t == at::kFloat ? WTCONV_F32 : t == at::kBFloat16 ? WTCONV_BF16 : t == at::kHalf ? WTCONV_F16 : -1;
}

inline std::string text(c10::IntArrayRef shape) {
    std::string s = "(";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + ")";
}

// Where a call runs: on the tensors' device, on its current stream or on the one that the caller gives.
// There the call's scratch and new tensors are allocated under that stream, so that no other stream's
// earlier or later use of their memory meets this one, and every tensor is recorded on the stream that it
// does not belong to: memory that the caller lets go of is not used again before the work has ended.  (Not on
// an ExternalStream, which may end before the tensors do: its owner keeps them.)
class Call {
  public:
    Call(const py::object &stream, c10::Device device)
        : device_(device), guard_(device), current_(c10::cuda::getCurrentCUDAStream(device.index())), stream_(current_) {
        if (stream.is_none()) return;
        const py::object where = py::getattr(stream, "device", py::none());
        if (!where.is_none() && py::cast<c10::Device>(where) != device) refuse("stream is on another device than the tensors");
        stream_ = c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(py::cast<uintptr_t>(stream.attr("cuda_stream"))),
                                                   device.index());
        if (stream_.stream() == current_.stream()) return;
        under_.reset_stream(stream_);
        const py::object cuda = py::module_::import("torch.cuda");
        records_ = py::isinstance(stream, cuda.attr("Stream")) && !py::isinstance(stream, cuda.attr("ExternalStream"));
    }
    wtconv_stream_t stream() const { return reinterpret_cast<wtconv_stream_t>(stream_.stream()); }
    // The caller's tensors that the work reads or writes.
    template <typename... Ts> void uses(const Ts &...ts) const {
        if (records_) (record(ts, stream_), ...);
    }
    // A new tensor that the caller gets.
    Tensor empty(c10::IntArrayRef shape, at::ScalarType dtype) const {
        Tensor t = at::detail::empty_cuda(shape, dtype, device_, c10::nullopt);
        if (records_) record(t, current_);
        return t;
    }
    // Scratch that ends with the call.
    Tensor scratch(size_t bytes) const { return at::detail::empty_cuda({(int64_t)bytes}, at::kByte, device_, c10::nullopt); }

  private:
    static void record(const Tensor &t, const c10::cuda::CUDAStream &stream) {
        c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), stream);
    }
    static void record(const optional<Tensor> &t, const c10::cuda::CUDAStream &stream) {
        if (t.has_value()) record(*t, stream);
    }
    c10::Device device_;
    c10::cuda::CUDAGuard guard_;
    c10::cuda::OptionalCUDAStreamGuard under_;
    c10::cuda::CUDAStream current_, stream_;
    bool records_ = false;
};

// One activation of the scan as strides of its batch and row axes.
struct Act {
    void *p;
    int64_t batch, row;
};
inline Act activation(const Tensor &t, const char *name, bool planes, const Tensor *like = nullptr) {
    if (!t.is_cuda() || dtype_code(t.scalar_type()) < 0)
        refuse(std::string(name) + " must be a CUDA tensor of fp32, bf16 or fp16");
    if (like != nullptr && (t.sizes() != like->sizes() || t.scalar_type() != like->scalar_type() || t.device() != like->device()))
        refuse(std::string(name) + " must match x's shape, dtype and device");
    if (t.dim() != 3 && !(t.dim() == 4 && planes))
        refuse(std::string(name) + " must be (B, C, T) or (B, C, H, W) planes, or (B, T, C) tokens");
    if (t.numel() == 0) refuse(std::string(name) + " is empty");
    if (t.dim() == 4 && ((t.stride(3) != 1 && t.size(3) > 1) || (t.stride(2) != t.size(3) && t.size(2) > 1)))
        refuse(std::string(name) + ": the pixels of a plane must be contiguous");
    if (t.dim() == 3 && t.stride(2) != 1 && t.size(2) > 1) refuse(std::string(name) + ": the innermost axis must be contiguous");
    return {t.data_ptr(), t.stride(0), t.stride(1)};
}

struct Dims {
    int B, T, C, layout, dtype;
};
inline bool is_planes(const std::string &layout) {
    if (layout != "planes" && layout != "tokens") refuse("layout must be 'planes' or 'tokens', not '" + layout + "'");
    return layout == "planes";
}
inline Dims dims_of(const Tensor &x, bool planes) {
    const int64_t last = x.dim() == 4 ? x.size(2) * x.size(3) : x.size(2);
    const int64_t T = planes ? last : x.size(1), C = planes ? x.size(1) : last;
    if (x.size(0) > INT_MAX || T > INT_MAX || C > INT_MAX) refuse("x is too large");
    return {(int)x.size(0), (int)T, (int)C, planes ? WTCONV_SCAN_PLANES : WTCONV_SCAN_TOKENS, dtype_code(x.scalar_type())};
}

template <typename V>
V *array(const optional<Tensor> &t, const char *name, c10::IntArrayRef shape, c10::Device device) {
    if (!t.has_value()) return nullptr;
    const at::ScalarType want = std::is_same<V, int>::value ? at::kInt : at::kFloat;
    if (t->device() != device || t->scalar_type() != want || t->sizes() != shape || !t->is_contiguous())
        refuse(std::string(name) + " must be a contiguous " + (want == at::kInt ? "int32" : "fp32") + " tensor of shape " +
               text(shape) + " on " + device.str());
    return static_cast<V *>(t->data_ptr());
}

// The caller's scratch or a new one of `need` bytes.
struct Scratch {
    Tensor t;
    void *p = nullptr;
    size_t bytes = 0;
};
inline Scratch scratch(const optional<Tensor> &given, size_t need, c10::Device device, const Call &call) {
    Scratch s;
    if (given.has_value()) {
        if (given->device() != device) refuse("workspace is on " + given->device().str() + ", the tensors on " + device.str());
        if (!given->is_contiguous()) refuse("workspace must be contiguous");
        s.t = *given;
        call.uses(s.t);
    } else if (need > 0) {
        s.t = call.scratch(need);
    }
    if (s.t.defined()) s.p = s.t.data_ptr(), s.bytes = s.t.nbytes();
    return s;
}

// A tensor of the caller's that a kernel has written: autograd then sees that a value it saved has changed.
inline void written(const Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
inline void written(const optional<Tensor> &t) {
    if (t.has_value()) written(*t);
}

}  // namespace binding

// The dense 8-bit operators on torch tensors: argument checks, output allocation and the C calls, in C++
// because a one-token call lasts a few microseconds on the device: the same checks and allocations from
// Python took 13 to 18 us a call, three to eight times the kernels' own time.
//
// Nothing here computes; every function ends in one call of the C ABI (moe_b200.h) on the current stream
// of the operands' device.  A failed check raises the package's MoEError with MOE_ERR_ARG.
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <initializer_list>
#include <optional>
#include <string>

#include "moe_b200.h"

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace {

py::handle g_error;         // MoEError(code, what); lives as long as the module

[[noreturn]] void raise(int code, const std::string &what) {
    py::object e = g_error(code, what);
    PyErr_SetObject(g_error.ptr(), e.ptr());
    throw py::error_already_set();
}

[[noreturn]] void bad(const std::string &what) { raise(MOE_ERR_ARG, what); }

std::string shown(const Tensor &t) {
    std::string s = "[";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + "] " + c10::toString(t.scalar_type()) + " on " + t.device().str();
}

int64_t blocks(int64_t n) { return (n + 127) / 128; }

int type_code(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return MOE_BF16;
        case at::kHalf: return MOE_FP16;
        case at::kFloat: return MOE_FP32;
        default: return -1;
    }
}

bool is_codes(const Tensor &t) { return t.scalar_type() == at::kFloat8_e4m3fn || t.scalar_type() == at::kByte; }

struct Call {
    int device;
    const char *op;

    void here(const Tensor &t, const char *name) const {
        if (!t.is_cuda() || t.get_device() != device)
            bad(std::string(op) + ": " + name + " is not on cuda:" + std::to_string(device) + ": " + shown(t));
    }
    // A matrix of contiguous rows; its row distance (any, where there are not two rows).
    int64_t rows(const Tensor &t, const char *name, bool type_ok, int64_t r = -1, int64_t c = -1) const {
        here(t, name);
        if (t.dim() != 2 || !type_ok || (r >= 0 && t.size(0) != r) || (c >= 0 && t.size(1) != c))
            bad(std::string(op) + ": " + name + " has another shape or type than wanted: " + shown(t));
        if (t.size(1) > 1 && t.stride(1) != 1) bad(std::string(op) + ": the rows of " + name + " are not contiguous");
        return t.size(0) > 1 ? t.stride(0) : (t.size(1) + 15) / 16 * 16;
    }
    void whole(const Tensor &t, const char *name, bool type_ok, std::initializer_list<int64_t> shape) const {
        here(t, name);
        if (!type_ok || t.sizes() != at::IntArrayRef(shape) || !t.is_contiguous())
            bad(std::string(op) + ": " + name + " has another shape or type than wanted, or is not contiguous: " + shown(t));
    }
    int size(int64_t n, const char *name) const {
        if (n > INT32_MAX) bad(std::string(op) + ": too many " + name);
        return (int)n;
    }
    Tensor empty(at::IntArrayRef shape, at::ScalarType t) const {
        return at::detail::empty_cuda(shape, t, at::Device(at::kCUDA, (c10::DeviceIndex)device), std::nullopt);
    }
    void *stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }
    void done(int rc) const {
        if (rc) raise(rc, op);
    }
};

// Whether the byte ranges of two tensors meet.
bool overlap(const Tensor &a, const Tensor &b) {
    auto last = [](const Tensor &t) {
        int64_t n = 1;
        for (int64_t i = 0; i < t.dim(); ++i) n += (t.size(i) - 1) * t.stride(i);
        return static_cast<const char *>(t.const_data_ptr()) + n * t.itemsize();
    };
    if (!a.numel() || !b.numel()) return false;
    return static_cast<const char *>(a.const_data_ptr()) < last(b) && static_cast<const char *>(b.const_data_ptr()) < last(a);
}

// Of two matrices of one shape and contiguous rows; one row may have any nominal distance to the next.
bool same_place(const Tensor &a, const Tensor &b) {
    return a.const_data_ptr() == b.const_data_ptr() && (a.size(0) < 2 || a.stride(0) == b.stride(0));
}

template <typename T>
T *ptr(const Tensor &t) { return static_cast<T *>(const_cast<void *>(t.const_data_ptr())); }
template <typename T>
T *ptr_to_write(const Tensor &t) { return static_cast<T *>(t.mutable_data_ptr()); }
template <typename T>
T *ptr(const OptTensor &t) { return t ? ptr<T>(*t) : nullptr; }

moe_fp8_ctx_t *ctx_of(uintptr_t c) { return reinterpret_cast<moe_fp8_ctx_t *>(c); }

py::tuple add_rmsnorm(uintptr_t ctx, int device, const Tensor &x, const Tensor &norm_scale, const OptTensor &residual,
                      double eps, const OptTensor &sum_out) {
    const Call c{device, "add_rmsnorm"};
    const at::ScalarType t = x.scalar_type();
    const int code = type_code(t);
    const int64_t ldx = c.rows(x, "x", code >= 0), T = x.size(0), d = x.size(1);
    c.whole(norm_scale, "norm_scale", norm_scale.scalar_type() == at::kBFloat16, {d});
    int64_t ldr = 0, lds = 0;
    if (residual) ldr = c.rows(*residual, "residual", residual->scalar_type() == t, T, d);
    Tensor sum;
    if (sum_out) {
        if (!residual) bad("add_rmsnorm: there is no sum without a residual");
        sum = *sum_out;
        lds = c.rows(sum, "sum_out", sum.scalar_type() == t, T, d);
        if ((overlap(sum, x) && !same_place(sum, x)) || (overlap(sum, *residual) && !same_place(sum, *residual)))
            bad("add_rmsnorm: sum_out overlaps an input without being it");
        if (overlap(sum, norm_scale)) bad("add_rmsnorm: sum_out overlaps norm_scale");
    } else if (residual) {
        sum = c.empty({T, d}, t);
        lds = d;
    }
    Tensor q = c.empty({T, d}, at::kFloat8_e4m3fn), s = c.empty({T, blocks(d)}, at::kFloat);
    c.done(moe_add_rmsnorm_fp8(ctx_of(ctx), c.size(T, "rows"), c.size(d, "columns"), code, x.const_data_ptr(), ldx,
                               ptr<void>(residual), ldr, ptr<uint16_t>(norm_scale), (float)eps,
                               residual ? ptr_to_write<void>(sum) : nullptr, lds, ptr_to_write<uint8_t>(q), ptr_to_write<float>(s),
                               c.stream()));
    return residual ? py::make_tuple(q, s, sum) : py::make_tuple(q, s);
}

Tensor matmul(uintptr_t ctx, int device, const Tensor &a, const Tensor &a_scale, const Tensor &b, const Tensor &b_scale,
              const OptTensor &bias, const OptTensor &residual, const OptTensor &out,
              const std::optional<at::ScalarType> &out_dtype) {
    const Call c{device, "matmul"};
    const int64_t lda = c.rows(a, "a", is_codes(a)), M = a.size(0), K = a.size(1);
    const int64_t N = b.dim() == 2 ? b.size(0) : 0;
    c.whole(b, "b", is_codes(b), {N, K});
    c.whole(a_scale, "a_scale", a_scale.scalar_type() == at::kFloat, {M, blocks(K)});
    c.whole(b_scale, "b_scale", b_scale.scalar_type() == at::kFloat, {blocks(N), blocks(K)});
    if (bias) c.whole(*bias, "bias", bias->scalar_type() == at::kBFloat16, {N});
    const at::ScalarType t = out_dtype ? *out_dtype : out ? out->scalar_type() : residual ? residual->scalar_type() : at::kBFloat16;
    const int code = type_code(t);
    if (code < 0) bad("matmul: outputs are bf16, fp16 or fp32");
    const int64_t ldr = residual ? c.rows(*residual, "residual", residual->scalar_type() == t, M, N) : 0;
    int64_t ldc = N;
    if (out) {
        ldc = c.rows(*out, "out", out->scalar_type() == t, M, N);
        if (overlap(*out, a) || overlap(*out, a_scale) || overlap(*out, b) || overlap(*out, b_scale) || (bias && overlap(*out, *bias)))
            bad("matmul: out overlaps an operand");
        if (residual && overlap(*out, *residual) && !same_place(*out, *residual))
            bad("matmul: out overlaps residual without being it");
    }
    Tensor y = out ? *out : c.empty({M, N}, t);
    c.done(moe_fp8_matmul(ctx_of(ctx), c.size(M, "rows"), c.size(N, "columns"), c.size(K, "elements"), ptr<uint8_t>(a), lda,
                          ptr<float>(a_scale), ptr<uint8_t>(b), ptr<float>(b_scale), ptr<uint16_t>(bias),
                          ptr<void>(residual), ldr, ptr_to_write<void>(y), ldc, code, c.stream()));
    return y;
}

py::tuple gated_matmul(uintptr_t ctx, int device, const Tensor &a, const Tensor &a_scale, const Tensor &w13,
                       const Tensor &w13_scale, const OptTensor &bias, double alpha, double limit, double shift) {
    const Call c{device, "gated_matmul"};
    const int64_t lda = c.rows(a, "a", is_codes(a)), M = a.size(0), K = a.size(1);
    const int64_t F = w13.dim() == 3 ? w13.size(1) : w13.dim() == 2 ? w13.size(0) / 2 : 0;
    if (w13.dim() == 3) c.whole(w13, "w13", is_codes(w13), {2, F, K});
    else c.whole(w13, "w13", is_codes(w13), {2 * F, K});
    c.whole(a_scale, "a_scale", a_scale.scalar_type() == at::kFloat, {M, blocks(K)});
    c.whole(w13_scale, "w13_scale", w13_scale.scalar_type() == at::kFloat, {2, blocks(F), blocks(K)});
    if (bias) c.whole(*bias, "bias", bias->scalar_type() == at::kBFloat16, {2 * F});
    Tensor h = c.empty({M, F}, at::kFloat8_e4m3fn), s = c.empty({M, blocks(F)}, at::kFloat);
    c.done(moe_fp8_gated_matmul(ctx_of(ctx), c.size(M, "rows"), c.size(F, "columns"), c.size(K, "elements"),
                                ptr<uint8_t>(a), lda, ptr<float>(a_scale), ptr<uint8_t>(w13), ptr<float>(w13_scale),
                                ptr<uint16_t>(bias), (float)alpha, (float)limit, (float)shift,
                                ptr_to_write<uint8_t>(h), ptr_to_write<float>(s), c.stream()));
    return py::make_tuple(h, s);
}

}  // namespace

PYBIND11_MODULE(_binding, m) {
    m.attr("built_for") = MOE_BINDING_BUILT_FOR;        // (the build looks for it in the file)
    m.def("set_error", [](py::object cls) { g_error = cls.release(); });
    m.def("add_rmsnorm", &add_rmsnorm);
    m.def("matmul", &matmul);
    m.def("gated_matmul", &gated_matmul);
}

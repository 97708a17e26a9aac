// rc_op_api.cpp -- the C ABI of the operators around the codec (declared in
// include/rcodec.h): argument validation, then the kernels on the caller's
// stream.  Validation never touches HIP.
#include "rcodec.h"
#include "rc_op_launch.hpp"

namespace {

constexpr size_t kMaxElems = (size_t)1 << 40;    // as for the codec

bool dtype_ok(int d) { return d == RC_DT_FP32 || d == RC_DT_FP16 || d == RC_DT_BF16; }
size_t dtype_size(int d) { return d == RC_DT_FP32 ? 4 : 2; }
bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool aligned16(const void* p) { return aligned(p, 16); }

rc_status from_hip(hipError_t e) { return e == hipSuccess ? RC_OK : RC_ERR_HIP; }

// Sizes of a grouped product; RC_OK when the kernels can address them.
rc_status grouped_sizes(size_t experts, size_t n, size_t k, size_t rows)
{
    if (experts < 1 || experts > RC_MAX_EXPERTS) return RC_ERR_RANGE;
    if (n == 0 || n % 8 != 0 || n > RC_MAX_WIDTH || k == 0 || k % RC_BLOCK_ELEMS != 0 || k > RC_MAX_WIDTH) return RC_ERR_RANGE;
    if (n * k > kMaxElems / experts) return RC_ERR_RANGE;
    if (rows > 0x7FFFFFFF) return RC_ERR_RANGE;      // offsets are 32-bit
    return RC_OK;
}

}  // namespace

extern "C" {

rc_status rc_mxfp4_grouped_matmul(const void* w, size_t experts, size_t n, size_t k, const int32_t* offsets,
                                  rc_dtype x_t, const void* x, size_t rows, rc_dtype y_t, void* y, void* stream)
{
    if (!dtype_ok(x_t) || !dtype_ok(y_t)) return RC_ERR_UNSUPPORTED;
    const rc_status s = grouped_sizes(experts, n, k, rows);
    if (s != RC_OK || rows == 0) return s;
    if (!w || !offsets || !x || !y) return RC_ERR_NULL;
    if (!aligned16(w) || !aligned16(offsets) || !aligned16(x) || !aligned16(y)) return RC_ERR_ALIGN;
    const rc::Grouped g = {x, nullptr, static_cast<const uint8_t*>(w), offsets, y, rows, (int64_t)n, (int64_t)k, (int)experts, y_t};
    return from_hip(rc::launch_grouped_forward(x_t, g, static_cast<hipStream_t>(stream)));
}

rc_status rc_mxfp4_grouped_matmul_dx(const void* w, size_t experts, size_t n, size_t k, const int32_t* offsets,
                                     rc_dtype dy_t, const void* dy, size_t rows, rc_dtype dx_t, void* dx, void* stream)
{
    if (!dtype_ok(dy_t) || !dtype_ok(dx_t)) return RC_ERR_UNSUPPORTED;
    const rc_status s = grouped_sizes(experts, n, k, rows);
    if (s != RC_OK || rows == 0) return s;
    if (!w || !offsets || !dy || !dx) return RC_ERR_NULL;
    if (!aligned16(w) || !aligned16(offsets) || !aligned16(dy) || !aligned16(dx)) return RC_ERR_ALIGN;
    const rc::Grouped g = {dy, nullptr, static_cast<const uint8_t*>(w), offsets, dx, rows, (int64_t)n, (int64_t)k, (int)experts, dx_t};
    return from_hip(rc::launch_grouped_dx(dy_t, g, static_cast<hipStream_t>(stream)));
}

rc_status rc_grouped_matmul_dw(size_t experts, size_t n, size_t k, const int32_t* offsets, rc_dtype t,
                               const void* dy, const void* x, size_t rows, rc_dtype dw_t, void* dw, void* stream)
{
    if (!dtype_ok(t) || !dtype_ok(dw_t)) return RC_ERR_UNSUPPORTED;
    const rc_status s = grouped_sizes(experts, n, k, rows);
    if (s != RC_OK) return s;
    if (!offsets || !dw || (rows != 0 && (!dy || !x))) return RC_ERR_NULL;
    if (!aligned16(offsets) || !aligned16(dw) || !aligned16(dy) || !aligned16(x)) return RC_ERR_ALIGN;
    const rc::Grouped g = {dy, x, nullptr, offsets, dw, rows, (int64_t)n, (int64_t)k, (int)experts, dw_t};
    return from_hip(rc::launch_grouped_dw(t, g, static_cast<hipStream_t>(stream)));
}

rc_status rc_block_norm(rc_dtype t, size_t rows, size_t d, const void* y, const void* r, rc_dtype w_t,
                        const void* post_w, rc_gate gate_mode, const void* gate, const void* pre_w, float alpha,
                        float eps, void* h, void* z, float* stats, void* stream)
{
    if (!dtype_ok(t) || !dtype_ok(w_t)) return RC_ERR_UNSUPPORTED;
    if (gate_mode != RC_GATE_NONE && gate_mode != RC_GATE_CHANNEL && gate_mode != RC_GATE_FULL) return RC_ERR_UNSUPPORTED;
    if (d == 0 || d > rc::kNormMaxDim || rows > kMaxElems / d) return RC_ERR_RANGE;
    if (rows == 0) return RC_OK;
    if (!y || !r || !pre_w || !h || !z || (gate_mode != RC_GATE_NONE && !gate)) return RC_ERR_NULL;
    if (!aligned16(y) || !aligned16(r) || !aligned16(post_w) || !aligned16(gate) || !aligned16(pre_w) ||
        !aligned16(h) || !aligned16(z) || !aligned16(stats)) return RC_ERR_ALIGN;
    const rc::BlockNorm a = {y, r, post_w, gate, pre_w, h, z, stats, rows, (uint32_t)d, gate_mode, w_t, alpha, eps};
    return from_hip(rc::launch_block_norm(t, a, static_cast<hipStream_t>(stream)));
}

size_t rc_block_norm_backward_workspace(size_t rows, size_t d)
{
    if (d == 0 || d > rc::kNormMaxDim) return 0;
    return (size_t)rc::block_norm_groups(rows, (uint32_t)d) * 2 * d * sizeof(float);
}

rc_status rc_block_norm_backward(rc_dtype t, size_t rows, size_t d, const void* dz, const void* dh, const void* h,
                                 const float* stats, const void* y, rc_dtype w_t, const void* post_w,
                                 rc_gate gate_mode, const void* gate, const void* pre_w, float alpha, void* dy,
                                 void* dr, float* dpre, float* dpost, void* dgate, void* workspace, void* stream)
{
    if (!dtype_ok(t) || !dtype_ok(w_t)) return RC_ERR_UNSUPPORTED;
    if (gate_mode != RC_GATE_NONE && gate_mode != RC_GATE_CHANNEL && gate_mode != RC_GATE_FULL) return RC_ERR_UNSUPPORTED;
    if (d == 0 || d > rc::kNormMaxDim || rows > kMaxElems / d) return RC_ERR_RANGE;
    if (!pre_w || !dpre || (post_w && !dpost) || (gate_mode == RC_GATE_CHANNEL && (!gate || !dgate))) return RC_ERR_NULL;
    if (rows != 0 && (!dz || !h || !stats || !y || !dy || !dr || !workspace ||
                      (gate_mode == RC_GATE_FULL && (!gate || !dgate)))) return RC_ERR_NULL;
    if (!aligned16(dz) || !aligned16(dh) || !aligned16(h) || !aligned16(stats) || !aligned16(y) || !aligned16(post_w) ||
        !aligned16(gate) || !aligned16(pre_w) || !aligned16(dy) || !aligned16(dr) || !aligned16(dpre) ||
        !aligned16(dpost) || !aligned16(dgate) || !aligned16(workspace)) return RC_ERR_ALIGN;
    const rc::BlockNormBackward a = {dz, dh, h, y, post_w, gate, pre_w, stats, dy, dr, dgate, dpre,
                                     post_w ? dpost : nullptr, static_cast<float*>(workspace), rows, (uint32_t)d,
                                     gate_mode, w_t, alpha};
    return from_hip(rc::launch_block_norm_backward(t, a, static_cast<hipStream_t>(stream)));
}

size_t rc_grad_norm_clip_workspace(void) { return rc::kClipGroups * sizeof(double); }

rc_status rc_grad_norm_clip(const rc_grad* grads, size_t count, float scale, float max_norm, float eps,
                            void* workspace, float* norm, void* stream)
{
    if (!(max_norm >= 0.0f) || !(eps >= 0.0f)) return RC_ERR_RANGE;
    if (!workspace || !norm || (count != 0 && !grads)) return RC_ERR_NULL;
    if (!aligned16(workspace) || !aligned(norm, 4)) return RC_ERR_ALIGN;
    for (size_t i = 0; i < count; ++i) {
        const rc_grad& g = grads[i];
        if (!dtype_ok(g.in_t) || !dtype_ok(g.out_t)) return RC_ERR_UNSUPPORTED;
        if (g.n == 0) continue;
        if (g.n > kMaxElems) return RC_ERR_RANGE;
        if (!g.in || !g.out) return RC_ERR_NULL;
        if (!aligned(g.in, dtype_size(g.in_t)) || !aligned(g.out, dtype_size(g.out_t))) return RC_ERR_ALIGN;
        if (g.in == g.out && g.in_t != g.out_t) return RC_ERR_UNSUPPORTED;
    }
    static_assert(sizeof(rc_grad) == sizeof(rc::GradTensor), "one layout");
    return from_hip(rc::launch_grad_norm_clip(reinterpret_cast<const rc::GradTensor*>(grads), count, scale, max_norm,
                                              eps, workspace, norm, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

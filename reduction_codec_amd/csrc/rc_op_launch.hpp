// rc_op_launch.hpp -- host-side declarations of the operators around the
// codec (gradient clipping, the norms around a block, products grouped by
// expert), shared by the C-ABI layer and the kernel units.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace rc {

// Compute units of the current device (256 when it cannot be asked).
inline int compute_units()
{
    int dev = 0, cus = 256;
    if (hipGetDevice(&dev) == hipSuccess) (void)hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
    return cus > 0 ? cus : 256;
}

// ---- gradient norm and clipping (rc_op_grad_clip.hip)
constexpr unsigned kClipGroups = 1024;           // most workgroups of a launch, one partial sum each
struct GradTensor { const void* in; void* out; uint64_t n; int32_t in_t, out_t; };
hipError_t launch_grad_norm_clip(const GradTensor* grads, size_t count, float scale, float max_norm, float eps,
                                 void* workspace, float* norm, hipStream_t st);

// ---- norms around a block (rc_op_block_norm.hip)
enum : int { kGateNone = 0, kGateChannel = 1, kGateFull = 2 };   // rc_gate values
constexpr uint32_t kNormMaxDim = 32768;          // 1024 lanes of 32 elements
struct BlockNorm {
    const void *y, *r, *post_w, *gate, *pre_w;   // post_w may be null
    void *h, *z;
    float* stats;                                // [2][rows] or null
    size_t rows;
    uint32_t d;
    int gate_mode, w_t;
    float alpha, eps;
};
struct BlockNormBackward {
    const void *dz, *dh, *h, *y, *post_w, *gate, *pre_w;   // dh, post_w may be null
    const float* stats;
    void *dy, *dr, *dgate;
    float *dpre, *dpost, *partial;
    size_t rows;
    uint32_t d;
    int gate_mode, w_t;
    float alpha;
};
// Workgroups of the backward kernel, rows of its workspace: by sizes alone, so
// the workspace can be sized without a GPU.  T lanes of eight elements hold a
// row; 1024 lanes per unit of 256 for wide rows, 512 for narrow ones, whose
// many small workgroups fill the units less evenly (measured at 256 .. 2048
// workgroups: d = 8192 161, 174, 198 us; 4096 100, 90, 100; 2048 71, 52, 62;
// 1024 117, 71, 54, 66; every workgroup costs 8 d bytes written and read).
inline unsigned block_norm_groups(size_t rows, uint32_t d)
{
    unsigned t = 64;
    while (t < 1024 && t * 8 < d) t *= 2;
    const unsigned most = t >= 512 ? 256 * 1024 / t : 256 * 512 / t;
    return (unsigned)(rows < most ? rows : most);
}
hipError_t launch_block_norm(int dt, const BlockNorm& a, hipStream_t st);
hipError_t launch_block_norm_backward(int dt, const BlockNormBackward& a, hipStream_t st);

// ---- products grouped by expert (rc_op_experts.hip)
// a: x (forward) or dy, of type dt; b: x (weight gradient only); w: packed
// weights (not for the weight gradient); out of type out_t.
struct Grouped {
    const void *a, *b;
    const uint8_t* w;
    const int32_t* offsets;
    void* out;
    size_t rows;
    int64_t n, k;
    int experts, out_t;
};
hipError_t launch_grouped_forward(int dt, const Grouped& a, hipStream_t st);
hipError_t launch_grouped_dx(int dt, const Grouped& a, hipStream_t st);
hipError_t launch_grouped_dw(int dt, const Grouped& a, hipStream_t st);

}  // namespace rc

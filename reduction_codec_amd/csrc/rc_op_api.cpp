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

// A cache's sizes; RC_OK when the kernels can address it.
rc_status cache_sizes(const rc_cache& c, size_t tokens)
{
    const uint64_t d = c.d, p = c.page;
    if (d != 64 && d != 96 && d != 128 && d != 192 && d != 256) return RC_ERR_RANGE;
    if (p < 16 || p > 65536 || (p & (p - 1)) != 0 || p * d % RC_TILE_ELEMS != 0) return RC_ERR_RANGE;
    if (c.kv_heads < 1 || c.kv_heads > 65535 || c.seqs > RC_MAX_SEQS || c.pages > 0x7FFFFFFF || tokens > 0x7FFFFFFF ||
        c.max_pages > ((uint64_t)1 << 30) / p) return RC_ERR_RANGE;
    if (p * d > kMaxElems / c.kv_heads || (c.pages != 0 && p * d * c.kv_heads > kMaxElems / c.pages)) return RC_ERR_RANGE;
    return RC_OK;
}

rc_status cache_pointers(const rc_cache& c)
{
    if (!c.offsets || !c.lengths || (c.max_pages != 0 && !c.table) || (c.pages != 0 && (!c.k || !c.v))) return RC_ERR_NULL;
    if (!aligned16(c.k) || !aligned16(c.v) || !aligned(c.table, 4) || !aligned(c.lengths, 4) || !aligned(c.offsets, 4)) return RC_ERR_ALIGN;
    return RC_OK;
}

rc::Cache cache_args(const rc_cache& c, size_t tokens)
{
    int shift = 0;
    while ((1u << shift) < c.page) ++shift;
    return {static_cast<uint8_t*>(c.k), static_cast<uint8_t*>(c.v), c.table, c.lengths, c.offsets, (int)c.pages, shift,
            (int)c.kv_heads, (int)c.seqs, (int)c.max_pages, (int)tokens, (uint32_t)(c.page * c.d / RC_TILE_ELEMS * 1088)};
}

// Rows of `width` elements, `stride` apart.
bool stride_ok(size_t stride, size_t width, int t)
{
    return stride >= width && stride <= ((size_t)1 << 31) / dtype_size(t) && stride * dtype_size(t) % 16 == 0;
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

rc_status rc_mxfp4_cache_append(const rc_cache* cache, rc_dtype t, size_t tokens, const void* k, size_t k_stride,
                                const void* v, size_t v_stride, size_t heads, const void* q, size_t q_stride,
                                void* q_out, const float* rotation, size_t positions, size_t rot, int interleaved,
                                void* stream)
{
    if (!cache) return RC_ERR_NULL;
    if (!dtype_ok(t)) return RC_ERR_UNSUPPORTED;
    const rc_status s = cache_sizes(*cache, tokens);
    if (s != RC_OK) return s;
    const size_t d = cache->d, kv = cache->kv_heads;
    if (heads > 65535 || heads % kv != 0 || rot % 16 != 0 || rot > d) return RC_ERR_RANGE;
    // (rows before the first position take the first angles, which a table without columns needs too)
    if (rotation && rot != 0 && (positions == 0 || positions < cache->max_pages * cache->page)) return RC_ERR_RANGE;
    if (tokens == 0 || cache->seqs == 0) return RC_OK;
    if (!stride_ok(k_stride, kv * d, t) || !stride_ok(v_stride, kv * d, t) || (heads != 0 && !stride_ok(q_stride, heads * d, t))) return RC_ERR_RANGE;
    if (q_out == q && q != nullptr && heads != 0) return RC_ERR_UNSUPPORTED;
    if (!k || !v || (heads != 0 && (!q || !q_out))) return RC_ERR_NULL;
    const rc_status ps = cache_pointers(*cache);
    if (ps != RC_OK) return ps;
    if (!aligned16(k) || !aligned16(v) || !aligned16(q) || !aligned16(q_out) || !aligned16(rotation)) return RC_ERR_ALIGN;
    const rc::CacheAppend a = {cache_args(*cache, tokens), k, v, q, q_out, rot != 0 ? rotation : nullptr, k_stride,
                               v_stride, q_stride, (int)heads, rotation ? (int)rot : 0, interleaved != 0};
    return from_hip(rc::launch_cache_append(t, (int)d, a, static_cast<hipStream_t>(stream)));
}

rc_status rc_mxfp4_cache_read(const rc_cache* cache, size_t tokens, rc_dtype t, void* k, void* v, void* stream)
{
    if (!cache) return RC_ERR_NULL;
    if (!dtype_ok(t)) return RC_ERR_UNSUPPORTED;
    rc_status s = cache_sizes(*cache, tokens);
    if (s != RC_OK || tokens == 0 || cache->seqs == 0) return s;
    if (!k || !v) return RC_ERR_NULL;
    s = cache_pointers(*cache);
    if (s != RC_OK) return s;
    if (!aligned16(k) || !aligned16(v)) return RC_ERR_ALIGN;
    return from_hip(rc::launch_cache_read(t, (int)cache->d, cache_args(*cache, tokens), k, v, static_cast<hipStream_t>(stream)));
}

size_t rc_mxfp4_cache_attention_workspace(size_t tokens, size_t heads, size_t kv_heads, size_t d)
{
    if (kv_heads == 0 || heads == 0 || heads > 65535 || heads % kv_heads != 0 || d > 256) return 0;
    return rc::cache_attention_work(tokens, heads, kv_heads, d);
}

rc_status rc_mxfp4_cache_attention(const rc_cache* cache, rc_dtype t, size_t tokens, size_t heads, const void* q,
                                   size_t q_stride, float scale, int causal, size_t window, size_t max_query,
                                   void* out, float* lse, void* workspace, void* stream)
{
    if (!cache) return RC_ERR_NULL;
    if (!dtype_ok(t) || (window != 0 && !causal)) return RC_ERR_UNSUPPORTED;
    rc_status s = cache_sizes(*cache, tokens);
    if (s != RC_OK) return s;
    if (heads == 0 || heads > 65535 || heads % cache->kv_heads != 0 || tokens > 0x7FFFFFFF / heads) return RC_ERR_RANGE;
    if (tokens == 0 || cache->seqs == 0) return RC_OK;
    if (!stride_ok(q_stride, heads * cache->d, t)) return RC_ERR_RANGE;
    if (!q || !out || !workspace) return RC_ERR_NULL;
    // in place: a tile's rows are read by the workgroup that writes them, or all before the joining kernel does;
    // rows of another stride would be written over others' that are yet to be read
    if (out == q && tokens > 1 && q_stride != heads * cache->d) return RC_ERR_UNSUPPORTED;
    s = cache_pointers(*cache);
    if (s != RC_OK) return s;
    if (!aligned16(q) || !aligned16(out) || !aligned(lse, 4) || !aligned16(workspace)) return RC_ERR_ALIGN;
    const rc::CacheAttention a = {cache_args(*cache, tokens), q, out, lse, static_cast<float*>(workspace), q_stride,
                                  (int)heads, window > 0x7FFFFFFF ? 0 : (int)window, causal != 0, scale};
    return from_hip(rc::launch_cache_attention(t, (int)cache->d, a, max_query, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// libkda C ABI of linear attention with a decay per head and of paged decode attention:
// argument validation, dispatch to the kernels.  The contract of every entry point is
// documented in include/kda.h.
#include <math.h>
#include <stdint.h>

#include "kda_la.cuh"
#include "kda_paged.cuh"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool head_dim_ok(int d) { return d == 64 || d == 128; }
float scale_or_default(float scale, int d) { return scale == 0.0f ? 1.0f / sqrtf((float)d) : scale; }

// What every linear-attention call checks of its sizes, in the order of its statuses.
kda_status check_sizes(int B, int T, int H, int dk, int dv, kda_dtype dtype, float scale)
{
    if (B <= 0 || H <= 0 || T < 0 || dk <= 0 || dv <= 0) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_INVALID_ARG;
    if (!isfinite(scale)) return KDA_ERR_INVALID_ARG;
    // the grids have up to passes x segments (or column slices) CTAs per head
    if ((int64_t)B * H > (int64_t)INT32_MAX / 256) return KDA_ERR_INVALID_ARG;
    if ((int64_t)T > (int64_t)INT32_MAX - 256) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

kda::LaArgs la_args(const float *log_decay, int B, int T, int H, int dk, int dv, kda_dtype dtype, int npass)
{
    kda::LaArgs a = {};
    a.npass = npass;
    a.log_decay = log_decay;
    a.B = B; a.T = T; a.H = H; a.dk = dk; a.dv = dv; a.dtype = dtype;
    kda::la_choose_segments(a);
    return a;
}

// The gradients are three passes: with dk = dv one launch, else dv alone and (dq, dk),
// whose states are the transposed ones.  The launches follow one another on the stream and
// share the workspace.
size_t backward_bytes(int B, int T, int H, int dk, int dv, kda_dtype dtype)
{
    if (dk == dv) return kda::la_workspace_bytes(la_args(nullptr, B, T, H, dk, dv, dtype, 3));
    const size_t x = kda::la_workspace_bytes(la_args(nullptr, B, T, H, dk, dv, dtype, 1));
    const size_t y = kda::la_workspace_bytes(la_args(nullptr, B, T, H, dv, dk, dtype, 2));
    return x > y ? x : y;
}

}  // namespace

extern "C" {

size_t kda_la_forward_workspace_bytes(int B, int T, int H, int dk, int dv, kda_dtype dtype)
{
    if (check_sizes(B, T, H, dk, dv, dtype, 0.f) != KDA_OK || !head_dim_ok(dk) || !head_dim_ok(dv)) return 0;
    return kda::la_workspace_bytes(la_args(nullptr, B, T, H, dk, dv, dtype, 1));
}

size_t kda_la_backward_workspace_bytes(int B, int T, int H, int dk, int dv, kda_dtype dtype)
{
    if (check_sizes(B, T, H, dk, dv, dtype, 0.f) != KDA_OK || !head_dim_ok(dk) || !head_dim_ok(dv)) return 0;
    return backward_bytes(B, T, H, dk, dv, dtype);
}

kda_status kda_la_forward(const void *q, const void *k, const void *v, const float *log_decay,
                          const float *initial_state, void *out, float *final_state,
                          int B, int T, int H, int dk, int dv, kda_dtype dtype, float scale,
                          void *workspace, size_t workspace_bytes, void *stream)
{
    kda::clear_cuda_error();
    const kda_status cs = check_sizes(B, T, H, dk, dv, dtype, scale);
    if (cs != KDA_OK) return cs;
    if (T > 0 && (!q || !k || !v || !out)) return KDA_ERR_INVALID_ARG;
    if (!head_dim_ok(dk) || !head_dim_ok(dv)) return KDA_ERR_UNSUPPORTED;
    if (T > 0 && (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))) return KDA_ERR_MISALIGNED;
    if (!aligned4(log_decay) || !aligned16(initial_state) || !aligned16(final_state) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return KDA_ERR_MISALIGNED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        // no tokens: the final state is the initial state (or zeros)
        if (!final_state || final_state == initial_state) return KDA_OK;
        const size_t bytes = sizeof(float) * (size_t)B * H * dk * dv;
        const cudaError_t e = initial_state
            ? cudaMemcpyAsync(final_state, initial_state, bytes, cudaMemcpyDeviceToDevice, st)
            : cudaMemsetAsync(final_state, 0, bytes, st);
        return e == cudaSuccess ? KDA_OK : kda::record_cuda_error(e);
    }
    kda::LaArgs a = la_args(log_decay, B, T, H, dk, dv, dtype, 1);
    const size_t need = kda::la_workspace_bytes(a);
    if (need && (!workspace || workspace_bytes < need)) return KDA_ERR_INVALID_ARG;
    a.ws = static_cast<float *>(workspace);
    const float sc = scale_or_default(scale, dk);
    a.pass[0] = {q, k, v, out, initial_state, final_state, 0, 0, sc, sc, 1.f};
    const cudaError_t e = kda::launch_la(a, st);
    return e == cudaSuccess ? KDA_OK : kda::record_cuda_error(e);
}

kda_status kda_la_backward(const void *q, const void *k, const void *v, const float *log_decay,
                           const float *initial_state, const void *grad_out, const float *grad_final_state,
                           void *grad_q, void *grad_k, void *grad_v, float *grad_initial_state,
                           int B, int T, int H, int dk, int dv, kda_dtype dtype, float scale,
                           void *workspace, size_t workspace_bytes, void *stream)
{
    kda::clear_cuda_error();
    const kda_status cs = check_sizes(B, T, H, dk, dv, dtype, scale);
    if (cs != KDA_OK) return cs;
    if (T > 0 && (!q || !k || !v || !grad_out || !grad_q || !grad_k || !grad_v)) return KDA_ERR_INVALID_ARG;
    if (!head_dim_ok(dk) || !head_dim_ok(dv)) return KDA_ERR_UNSUPPORTED;
    if (T > 0 && (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(grad_out) || !aligned16(grad_q) ||
                  !aligned16(grad_k) || !aligned16(grad_v)))
        return KDA_ERR_MISALIGNED;
    if (!aligned4(log_decay) || !aligned16(initial_state) || !aligned16(grad_final_state) ||
        !aligned16(grad_initial_state) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return KDA_ERR_MISALIGNED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        // no tokens: final_state is initial_state, so its gradient passes through
        if (!grad_initial_state || grad_initial_state == grad_final_state) return KDA_OK;
        const size_t bytes = sizeof(float) * (size_t)B * H * dk * dv;
        const cudaError_t e = grad_final_state
            ? cudaMemcpyAsync(grad_initial_state, grad_final_state, bytes, cudaMemcpyDeviceToDevice, st)
            : cudaMemsetAsync(grad_initial_state, 0, bytes, st);
        return e == cudaSuccess ? KDA_OK : kda::record_cuda_error(e);
    }
    const size_t need = backward_bytes(B, T, H, dk, dv, dtype);
    if (need && (!workspace || workspace_bytes < need)) return KDA_ERR_INVALID_ARG;
    const float sc = scale_or_default(scale, dk);
    const kda::LaPass dv_pass = {k, q, grad_out, grad_v, grad_final_state, grad_initial_state, 0, 1, sc, 1.f, sc};
    const kda::LaPass dk_pass = {v, grad_out, q, grad_k, grad_final_state, nullptr, 1, 1, sc, 1.f, sc};
    const kda::LaPass dq_pass = {grad_out, v, k, grad_q, initial_state, nullptr, 1, 0, sc, sc, 1.f};
    cudaError_t e;
    if (dk == dv) {
        kda::LaArgs a = la_args(log_decay, B, T, H, dk, dv, dtype, 3);
        a.ws = static_cast<float *>(workspace);
        a.pass[0] = dv_pass; a.pass[1] = dk_pass; a.pass[2] = dq_pass;
        e = kda::launch_la(a, st);
    } else {
        kda::LaArgs a = la_args(log_decay, B, T, H, dv, dk, dtype, 2);
        a.ws = static_cast<float *>(workspace);
        a.pass[0] = dk_pass; a.pass[1] = dq_pass;
        e = kda::launch_la(a, st);
        if (e == cudaSuccess) {
            a = la_args(log_decay, B, T, H, dk, dv, dtype, 1);
            a.ws = static_cast<float *>(workspace);
            a.pass[0] = dv_pass;
            e = kda::launch_la(a, st);
        }
    }
    return e == cudaSuccess ? KDA_OK : kda::record_cuda_error(e);
}

kda_status kda_la_decode_step(const void *q, const void *k, const void *v, const float *log_decay,
                              float *state_inout, void *out, int B, int H, int dk, int dv,
                              kda_dtype dtype, float scale, void *stream)
{
    kda::clear_cuda_error();
    const kda_status cs = check_sizes(B, 1, H, dk, dv, dtype, scale);
    if (cs != KDA_OK) return cs;
    if (!q || !k || !v || !state_inout || !out) return KDA_ERR_INVALID_ARG;
    if (!head_dim_ok(dk) || !head_dim_ok(dv)) return KDA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(state_inout) || !aligned16(out) ||
        !aligned4(log_decay))
        return KDA_ERR_MISALIGNED;
    const kda::LaDecodeArgs a = {q, k, v, log_decay, state_inout, out, B, H, dk, dv, dtype, scale_or_default(scale, dk)};
    const cudaError_t e = kda::launch_la_decode(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KDA_OK : kda::record_cuda_error(e);
}

size_t kda_paged_decode_workspace_bytes(int H, int Hkv, int D, kda_dtype dtype)
{
    if (H <= 0 || Hkv <= 0 || H % Hkv || !head_dim_ok(D) || (dtype != KDA_BF16 && dtype != KDA_F32)) return 0;
    return kda::paged_workspace_bytes(H, Hkv, D, dtype);
}

kda_status kda_paged_decode_step(const void *q, const void *k, const void *v, void *k_cache, void *v_cache,
                                 const int *block_table, const int *lengths, void *out,
                                 int B, int H, int Hkv, int D, int num_pages, int page_size, int max_pages,
                                 kda_dtype dtype, float scale, void *workspace, size_t workspace_bytes,
                                 void *stream)
{
    kda::clear_cuda_error();
    if (B <= 0 || H <= 0 || Hkv <= 0 || D <= 0 || num_pages <= 0 || page_size <= 0 || max_pages <= 0)
        return KDA_ERR_INVALID_ARG;
    if (H % Hkv) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_INVALID_ARG;
    if (!isfinite(scale)) return KDA_ERR_INVALID_ARG;
    // the joining grid has one CTA per row and query head
    if ((int64_t)B * H > (int64_t)INT32_MAX / 4) return KDA_ERR_INVALID_ARG;
    // a key's position and the tile behind the last one are 32-bit numbers
    if ((int64_t)max_pages * page_size > (int64_t)INT32_MAX - 1024) return KDA_ERR_INVALID_ARG;
    if (!q || !k_cache || !v_cache || !block_table || !lengths || !out || !workspace) return KDA_ERR_INVALID_ARG;
    if ((k == nullptr) != (v == nullptr)) return KDA_ERR_INVALID_ARG;
    if (!head_dim_ok(D)) return KDA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
        !aligned16(out) || !aligned4(block_table) || !aligned4(lengths) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return KDA_ERR_MISALIGNED;
    if (workspace_bytes < kda::paged_workspace_bytes(H, Hkv, D, dtype)) return KDA_ERR_INVALID_ARG;
    const kda::PagedArgs a = {q, k, v, k_cache, v_cache, block_table, lengths, out, B, H, Hkv, D, num_pages,
                              page_size, max_pages, dtype, scale_or_default(scale, D), static_cast<float *>(workspace)};
    const cudaError_t e = kda::launch_paged_decode(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KDA_OK : kda::record_cuda_error(e);
}

}  // extern "C"

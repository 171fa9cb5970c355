// Linear attention with one constant decay per head: declarations shared by its kernels
// (internal header).
//
// Forward, per head with lambda = exp(log_decay) (Lambda^n below is lambda to the n):
//     S_t = lambda S_{t-1} + k_t v_t^T,    o_t = scale S_t^T q_t,
// and over a chunk of c tokens entered with the state S0
//     o_i = scale (sum_{j <= i} lambda^(i-j) (q_i . k_j) v_j + lambda^(i+1) S0^T q_i),
//     S   = lambda^c S0 + sum_j lambda^(c-1-j) k_j v_j^T.
//
// Its gradients are linear attentions too.  With D_t the adjoint of S_t,
//     D_t = scale q_t do_t^T + lambda D_{t+1},   D_T = scale q_T do_T^T + dS_T,
//     dq_t = scale S_t do_t,  dk_t = D_t v_t,  dv_t = D_t^T k_t,  dS_0 = lambda D_1,
// so dq reads the forward state with (q, k, v) -> (do, v, k) and the state transposed,
// dv and dk read the adjoint state in reversed time with (q, k, v) -> (k, q, do) and
// (v, do, q).  One kernel therefore does the forward and all gradients: a LaPass names
// its tensors, its direction and its factors.  In reversed time the state decays after
// the write instead of before it, which moves two exponents by one.
#pragma once

#include "kda_internal.cuh"

namespace kda {

struct LaPass {
    const void *q, *k, *v;      // [B, T, H, dk], [B, T, H, dk], [B, T, H, dv]
    void *out;                  // [B, T, H, dv]
    const float *s0;            // state the pass starts from, or null (zeros)
    float *sT;                  // state behind the last token, or null
    int s0_transposed;          // s0 is stored [dv, dk]
    int rev;                    // walk the sequence from its end
    float f_intra, f_inter;     // factors of the two terms of the output
    float f_write;              // factor of k_t v_t^T
};
constexpr int kLaMaxPasses = 3;

struct LaArgs {
    LaPass pass[kLaMaxPasses];  // passes of one launch: the same dk and dv
    int npass;
    const float *log_decay;     // [H] or null (lambda = 1)
    int B, T, H, dk, dv;
    kda_dtype dtype;
    // Split of the sequence: nseg segments of seg_tokens (the last in time shorter), and the
    // workspace that they need where there is more than one.
    int nseg, seg_tokens;
    float *ws;
};

// Chooses a.nseg and a.seg_tokens (a.npass, sizes and dtype are set).
void la_choose_segments(LaArgs &a);
size_t la_workspace_bytes(const LaArgs &a);
// All passes of a.
cudaError_t launch_la(const LaArgs &a, cudaStream_t stream);

// Tensor cores (tcgen05): bf16 with dk = dv = 128.  One launch, segments included.
bool la_tc_supported(int dk, int dv, kda_dtype dtype);
size_t la_tc_workspace_bytes(const LaArgs &a);
cudaError_t launch_la_tc(const LaArgs &a, cudaStream_t stream);
// Reads and clears the status word that the kernel sets when a bounded wait gives up.  Synchronous.
cudaError_t take_la_device_status(unsigned int *status);

struct LaDecodeArgs {
    const void *q, *k, *v;
    const float *log_decay;     // [H] or null
    float *state;
    void *out;
    int B, H, dk, dv;
    kda_dtype dtype;
    float scale;
};
cudaError_t launch_la_decode(const LaDecodeArgs &a, cudaStream_t stream);

// Segment s of a pass, counted in the order the pass walks: its tokens in time.
__device__ __forceinline__ void la_segment(int s, int nseg, int seg_tokens, int T, int rev, int &t0, int &t1)
{
    const int at = rev ? nseg - 1 - s : s;
    t0 = at * seg_tokens;
    t1 = min(T, t0 + seg_tokens);
}

// lambda^n of head h in 64 bits; lambda = 0 (log_decay = -inf) has 0^0 = 1.
__device__ __forceinline__ double la_power(const float *log_decay, int h, double n)
{
    return (!log_decay || n == 0.0) ? 1.0 : exp((double)log_decay[h] * n);
}

template <typename T> __device__ __forceinline__ T la_round(float x);
template <> __device__ __forceinline__ float la_round<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 la_round<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Four consecutive elements as fp32, and back (16-byte aligned for fp32, 8 for bf16).
__device__ __forceinline__ float4 la_load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 la_load4(const __nv_bfloat16 *p)
{
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void la_store4(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }
__device__ __forceinline__ void la_store4(__nv_bfloat16 *p, float4 x)
{
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

}  // namespace kda

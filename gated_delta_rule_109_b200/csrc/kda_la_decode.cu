// Single-token step of linear attention with one decay per head, state updated in place:
//     S <- lambda S + k v^T,    o = scale S^T q        (the mathematics is in kda_la.cuh)
//
// The state, read once and written once (8 dk dv bytes per head), is all the traffic that
// matters.  A CTA owns DV / NS value columns of one head (columns never mix): every thread
// keeps its float4 column group of DK / RS rows in registers from the load to the store, and
// only the read o needs a reduction over rows.
#include "kda_la.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;

// lambda as the sum of two floats.  The state of a slowly decaying head holds thousands of steps,
// and each would repeat the rounding of a single one: 2^-25 of the state and step.  1 + expm1(g)
// is off by 2^-23 of |g| instead, and a head remembers 1 / |g| steps.  A head that decays faster
// than that holds a few, for which expf does.
__device__ __forceinline__ float2 decay_of(const float *__restrict__ log_decay, int h)
{
    const float g = log_decay ? log_decay[h] : 0.f;
    if (!(fabsf(g) < 0.5f)) return make_float2(expf(g), 0.f);
    const float e = expm1f(g), hi = 1.f + e;
    return make_float2(hi, e - (hi - 1.f));
}

template <int DK, int DV, typename InT, int NS>
__global__ void __launch_bounds__(kThreads, 3)
la_decode_kernel(const InT *__restrict__ q, const InT *__restrict__ k, const InT *__restrict__ v,
                 const float *__restrict__ log_decay, float *__restrict__ state, InT *__restrict__ out, int H,
                 float scale)
{
    constexpr int CGH = DV / 4;                // float4 column groups of a head
    constexpr int CG = CGH / NS;               // ... of this CTA
    constexpr int RS = kThreads / CG;          // rows apart that a thread's rows are
    constexpr int RPT = DK / RS;               // rows of a thread
    static_assert(RPT * RS == DK && CG * RS == kThreads, "shape");
    __shared__ float4 red[RS][CG];

    // As kda_decode_step: the next launch on the stream may start its CTAs once all of these
    // have started; nothing is read before the kernel ahead has completed.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const int bh = blockIdx.x / NS, tid = threadIdx.x;
    const int x = tid % CG, cg = (blockIdx.x % NS) * CG + x, r0 = tid / CG;
    float4 *S = reinterpret_cast<float4 *>(state) + (size_t)bh * DK * CGH;
    float4 s[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) s[i] = __ldcs(&S[(r0 + i * RS) * CGH + cg]);
    const float2 a = decay_of(log_decay, bh % H);
    const float4 vv = la_load4(v + (size_t)bh * DV + 4 * cg);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = r0 + i * RS;
        const float kc = to_f32(k[(size_t)bh * DK + r]), qc = to_f32(q[(size_t)bh * DK + r]);
        s[i].x = fmaf(a.x, s[i].x, fmaf(a.y, s[i].x, kc * vv.x)); s[i].y = fmaf(a.x, s[i].y, fmaf(a.y, s[i].y, kc * vv.y));
        s[i].z = fmaf(a.x, s[i].z, fmaf(a.y, s[i].z, kc * vv.z)); s[i].w = fmaf(a.x, s[i].w, fmaf(a.y, s[i].w, kc * vv.w));
        __stcs(&S[r * CGH + cg], s[i]);
        o.x += qc * s[i].x; o.y += qc * s[i].y; o.z += qc * s[i].z; o.w += qc * s[i].w;
    }
    red[r0][x] = o;
    __syncthreads();
    if (tid < CG * 4) {                        // one thread per column: sum over the row groups
        const int c = tid / 4, e = tid % 4;
        float acc = 0.f;
#pragma unroll 8
        for (int j = 0; j < RS; ++j) acc += reinterpret_cast<const float *>(&red[j][c])[e];
        out[(size_t)bh * DV + 4 * ((blockIdx.x % NS) * CG + c) + e] = la_round<InT>(scale * acc);
    }
}

template <int DK, int DV, typename InT, int NS>
cudaError_t launch_split(const LaDecodeArgs &a, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((size_t)a.B * a.H * NS));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, la_decode_kernel<DK, DV, InT, NS>, static_cast<const InT *>(a.q),
                                       static_cast<const InT *>(a.k), static_cast<const InT *>(a.v), a.log_decay,
                                       a.state, static_cast<InT *>(a.out), a.H, a.scale);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e == cudaSuccess) note_launch();
    return e;
}

template <int DK, int DV, typename InT>
cudaError_t launch_typed(const LaDecodeArgs &a, cudaStream_t stream)
{
    // Many heads: 64 columns per CTA keep whole 256-byte rows together.  Few heads (at that
    // split not even one CTA per SM): 16 columns per CTA, so that the state is spread over
    // four times as many SMs.
    constexpr int kWide = DV / 64, kNarrow = DV / 16;
    if ((long long)a.B * a.H * kWide <= 148) return launch_split<DK, DV, InT, kNarrow>(a, stream);
    return launch_split<DK, DV, InT, kWide>(a, stream);
}

template <typename InT>
cudaError_t launch_dims(const LaDecodeArgs &a, cudaStream_t stream)
{
    if (a.dk == 128 && a.dv == 128) return launch_typed<128, 128, InT>(a, stream);
    if (a.dk == 64 && a.dv == 64) return launch_typed<64, 64, InT>(a, stream);
    if (a.dk == 128 && a.dv == 64) return launch_typed<128, 64, InT>(a, stream);
    if (a.dk == 64 && a.dv == 128) return launch_typed<64, 128, InT>(a, stream);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_la_decode(const LaDecodeArgs &a, cudaStream_t stream)
{
    if (a.dtype == KDA_BF16) return launch_dims<__nv_bfloat16>(a, stream);
    return launch_dims<float>(a, stream);
}

}  // namespace kda

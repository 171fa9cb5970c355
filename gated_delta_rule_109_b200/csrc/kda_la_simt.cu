// Linear attention with one decay per head on CUDA cores, fp32 arithmetic throughout
// (the mathematics is in kda_la.cuh).
//
// One CTA walks the chunks of 64 tokens of one (pass, b, h, segment) with the state
// resident in shared memory.  A chunk is four small products of register tiles:
// 64 x 64 scores (4 x 4 a thread), the outputs P V + Q S (4 rows x DV/16 columns a
// thread) and the state K'^T V (DK/16 x DV/16 a thread), operands read as 16-byte
// vectors of padded rows.  A chunk's 8 dk dv + .. multiply-adds are what bounds it (4.3 us a
// chunk of 64-channel heads at the SM's full rate), so the tile loads of a chunk are all under
// way together and two CTAs share an SM where they fit.  Powers of lambda are computed in 64
// bits once per CTA, so their rounding does not grow along the sequence.
#include "kda_la.cuh"

namespace kda {
namespace {

constexpr int kC = 64;
constexpr int kThreads = 256;

template <int DK, int DV>
struct LaSmem {
    static constexpr int PK = DK + 4, PV = DV + 4, PP = kC + 4;   // row pitches: 16-byte aligned, 4 banks apart
    static constexpr int off_q = 0;
    static constexpr int off_k = off_q + kC * PK;
    static constexpr int off_v = off_k + kC * PK;
    static constexpr int off_p = off_v + kC * PV;
    static constexpr int off_s = off_p + kC * PP;
    static constexpr int off_w = off_s + DK * PV;                 // lambda^n, n = 0..64
    static constexpr int off_l = off_w + kC + 4;                  // lambda^c of a whole and of the ragged chunk, two floats each
    static constexpr int total = off_l + 4;
    static constexpr size_t bytes = sizeof(float) * (size_t)total;
};

__device__ __forceinline__ void fma4(float4 &acc, float a, float4 b)
{
    acc.x += a * b.x; acc.y += a * b.y; acc.z += a * b.z; acc.w += a * b.w;
}
__device__ __forceinline__ float dot4(float4 a, float4 b, float acc)
{
    acc += a.x * b.x; acc += a.y * b.y; acc += a.z * b.z; acc += a.w * b.w;
    return acc;
}

// A chunk's rows of D channels to shared memory as fp32, in the order of the walk: row t is
// token t (forward) or c - 1 - t (reversed), rows from c on are zeros.  `src` is row 0's, `step`
// leads to the next.  The loads are all issued before the first is needed.
template <int D>
__device__ __forceinline__ void stage(float *dst, const float *src, ptrdiff_t step, int c, int tid)
{
#pragma unroll
    for (int e = 0; e < kC * D / 4 / kThreads; ++e) {
        const int id = e * kThreads + tid, t = id / (D / 4), x = 4 * (id % (D / 4));
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst + t * (D + 4) + x);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                     :: "r"(to), "l"(src + (t < c ? t * step + x : 0)), "r"(t < c ? 16 : 0) : "memory");
    }
}
template <int D>
__device__ __forceinline__ void stage(float *dst, const __nv_bfloat16 *src, ptrdiff_t step, int c, int tid)
{
    float4 v[kC * D / 4 / kThreads];
#pragma unroll
    for (int e = 0; e < kC * D / 4 / kThreads; ++e) {
        const int id = e * kThreads + tid, t = id / (D / 4), x = 4 * (id % (D / 4));
        v[e] = t < c ? la_load4(src + t * step + x) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int e = 0; e < kC * D / 4 / kThreads; ++e) {
        const int id = e * kThreads + tid;
        la_store4(dst + (id / (D / 4)) * (D + 4) + 4 * (id % (D / 4)), v[e]);
    }
}

// CTAs of an SM: two where the shared memory of both fits
template <int DK, int DV> constexpr int simt_resident() { return LaSmem<DK, DV>::bytes <= 112 * 1024 ? 2 : 1; }

template <int DK, int DV, typename InT, bool STATES_ONLY>
__global__ void __launch_bounds__(kThreads, simt_resident<DK, DV>())
la_simt_kernel(const __grid_constant__ LaArgs a)
{
    using L = LaSmem<DK, DV>;
    constexpr int PK = L::PK, PV = L::PV, PP = L::PP;
    constexpr int RK = DK / 16, CV = DV / 64;   // state rows, float4 column groups per thread
    extern __shared__ __align__(16) float sm[];
    float *sQ = sm + L::off_q, *sK = sm + L::off_k, *sV = sm + L::off_v, *sP = sm + L::off_p, *sS = sm + L::off_s;
    float *sW = sm + L::off_w;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // A product's 64 x 64 tile: warp w has rows 16 wr .. and columns 32 wc .., a lane 4 rows and 4
    // columns of them, so that a warp's 16-byte reads of an operand are 64 or 128 bytes of different
    // banks.  Warps w and w + 4 share a scheduler: together they have as many causal pairs as any two.
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wr = warp < 4 ? warp : 7 - warp, wc = warp >> 2, ry = lane >> 3, cx = lane & 7;
    const int row0 = 16 * wr + ry, col4 = 32 * wc + 4 * cx;     // rows row0 + 4 i; channels col4 + 64 m ..
    const int nwork = STATES_ONLY ? a.nseg - 1 : a.nseg;
    const int seg = blockIdx.x % nwork;
    const int bh = (blockIdx.x / nwork) % (a.B * a.H);
    const int ip = blockIdx.x / nwork / (a.B * a.H);
    const LaPass &ps = a.pass[ip];
    const int b = bh / a.H, h = bh % a.H, rev = ps.rev;
    int t_lo, t_hi;
    la_segment(seg, a.nseg, a.seg_tokens, a.T, rev, t_lo, t_hi);
    float *slots = a.nseg > 1 ? a.ws + ((size_t)ip * a.B * a.H + bh) * a.nseg * DK * DV : nullptr;

    asm volatile("griddepcontrol.wait;" ::: "memory");   // nothing is read before what is ahead has completed
    if (tid <= kC) sW[tid] = (float)la_power(a.log_decay, h, tid);
    else if (tid >= 96 && tid < 98) {
        const double l = la_power(a.log_decay, h, tid == 96 ? kC : (t_hi - 1) % kC + 1);
        sm[L::off_l + 2 * (tid - 96)] = (float)l;
        sm[L::off_l + 2 * (tid - 96) + 1] = (float)(l - (double)(float)l);
    }
    const InT *q = static_cast<const InT *>(ps.q), *k = static_cast<const InT *>(ps.k), *v = static_cast<const InT *>(ps.v);
    const int n0 = t_lo / kC, n1 = (t_hi + kC - 1) / kC;
    auto tokens_of = [&](int it, int &t0, int &c) {             // the walk's chunk `it`: first token, tokens
        t0 = (rev ? n1 - 1 - (it - n0) : it) * kC;
        c = min(kC, t_hi - t0);
    };
    // token of row t of chunk `it`, counted over [B, T, H]
    auto token_at = [&](int t0, int c, int t) { return ((size_t)b * a.T + t0 + (rev ? c - 1 - t : t)) * a.H + h; };
    auto load = [&](int it) {
        int t0, c;
        tokens_of(it, t0, c);
        const size_t at = token_at(t0, c, 0);
        const ptrdiff_t step = rev ? -(ptrdiff_t)a.H : (ptrdiff_t)a.H;
        if (!STATES_ONLY) stage<DK>(sQ, q + at * DK, step * DK, c, tid);
        stage<DK>(sK, k + at * DK, step * DK, c, tid);
        stage<DV>(sV, v + at * DV, step * DV, c, tid);
    };
    load(n0);                               // under way while the entering state is made
    // ---- entering state.  One segment, and segment 0 of the walk without outputs: the initial
    // state (kept in slot nseg - 1 for the outputs of segment 0: final_state may be the same
    // buffer).  Otherwise the earlier segments' contributions, each faded by the tokens between.
    if (slots && !STATES_ONLY) {
        __syncthreads();
        float *weight = sP;                                     // [seg] pairs
        if (tid < seg) {
            int x0, x1;
            la_segment(tid, a.nseg, a.seg_tokens, a.T, rev, x0, x1);
            const double l = la_power(a.log_decay, h, rev ? x0 - t_hi : t_lo - x1);
            weight[2 * tid] = (float)l;
            weight[2 * tid + 1] = (float)(l - (double)(float)l);
        }
        __syncthreads();
#pragma unroll 1
        for (int e0 = 4 * tid; e0 < DK * DV; e0 += 16 * kThreads) {
            float4 s[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s[i] = seg == 0 ? la_load4(slots + (size_t)(a.nseg - 1) * DK * DV + e0 + 4 * i * kThreads)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int g = 0; g < seg; ++g)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 u = la_load4(slots + (size_t)g * DK * DV + e0 + 4 * i * kThreads);
                    fma4(s[i], weight[2 * g + 1], u);
                    fma4(s[i], weight[2 * g], u);
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = e0 + 4 * i * kThreads;
                la_store4(sS + (e / DV) * PV + e % DV, s[i]);
            }
        }
    } else {
        const float *s0 = ps.s0 && (!STATES_ONLY || seg == 0) ? ps.s0 + (size_t)bh * DK * DV : nullptr;
#pragma unroll 4
        for (int e = 4 * tid; e < DK * DV; e += 4 * kThreads) {
            const int r = e / DV, c = e % DV;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            if (s0) {
                const float *p = s0 + (ps.s0_transposed ? c * DK + r : e);
                s = ps.s0_transposed ? make_float4(p[0], p[DK], p[2 * DK], p[3 * DK]) : la_load4(p);
            }
            la_store4(sS + r * PV + c, s);
            if (STATES_ONLY && seg == 0) la_store4(slots + (size_t)(a.nseg - 1) * DK * DV + e, s);
        }
    }

    for (int it = n0; it < n1; ++it) {
        int t0, c;
        tokens_of(it, t0, c);
        if (it > n0) {
            __syncthreads();                    // the chunk before is consumed
            load(it);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();

        if (!STATES_ONLY) {
            // ---- P_ij = f_intra lambda^(i-j) (q_i . k_j), j <= i; columns 32 wc + cx + 8 b.  Tiles
            // that no pair j <= i falls into are left out, here and in P V.
            if (2 * wc <= wr) {
                float s[4][4] = {};
#pragma unroll 4
                for (int d = 0; d < DK; d += 4) {
                    float4 x[4], y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = la_load4(sQ + (row0 + 4 * i) * PK + d);
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[j] = la_load4(sK + (32 * wc + cx + 8 * j) * PK + d);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) s[i][j] = dot4(x[i], y[j], s[i][j]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = row0 + 4 * i, m = 32 * wc + cx + 8 * j;
                        sP[r * PP + m] = r >= m ? s[i][j] * (sW[max(r - m, 0)] * ps.f_intra) : 0.f;
                    }
            }
            __syncthreads();
            // ---- out: P V + lambda^(.) Q S
            float4 o[4][CV], x[4][CV];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int m = 0; m < CV; ++m) o[i][m] = x[i][m] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int j = 0; j < 16 * wr + 16; j += 4) {
                float4 p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = la_load4(sP + (row0 + 4 * i) * PP + j);
#pragma unroll
                for (int m = 0; m < CV; ++m)
#pragma unroll
                    for (int jj = 0; jj < 4; ++jj) {
                        const float4 y = la_load4(sV + (j + jj) * PV + col4 + 64 * m);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            fma4(o[i][m], jj == 0 ? p[i].x : jj == 1 ? p[i].y : jj == 2 ? p[i].z : p[i].w, y);
                    }
            }
#pragma unroll 2
            for (int d = 0; d < DK; d += 4) {
                float4 p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = la_load4(sQ + (row0 + 4 * i) * PK + d);
#pragma unroll
                for (int m = 0; m < CV; ++m)
#pragma unroll
                    for (int jj = 0; jj < 4; ++jj) {
                        const float4 y = la_load4(sS + (d + jj) * PV + col4 + 64 * m);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            fma4(x[i][m], jj == 0 ? p[i].x : jj == 1 ? p[i].y : jj == 2 ? p[i].z : p[i].w, y);
                    }
            }
            InT *out = static_cast<InT *>(ps.out);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = row0 + 4 * i;
                if (r >= c) continue;
                const float f = ps.f_inter * sW[rev ? r : r + 1];
                const size_t g = token_at(t0, c, r) * DV + col4;
#pragma unroll
                for (int m = 0; m < CV; ++m) {
                    fma4(o[i][m], f, x[i][m]);
                    la_store4(out + g + 64 * m, o[i][m]);
                }
            }
            __syncthreads();                    // every reader of the state and of k is done
        }
        // ---- k_j <- f_write lambda^(.) k_j, then S <- lambda^c S + K'^T V
#pragma unroll
        for (int e = 0; e < kC * DK / 4 / kThreads; ++e) {
            const int id = e * kThreads + tid, t = id / (DK / 4);
            float *p = sK + t * PK + 4 * (id % (DK / 4));
            const float w = ps.f_write * sW[max(rev ? c - t : c - 1 - t, 0)];
            float4 x = la_load4(p);
            x.x *= w; x.y *= w; x.z *= w; x.w *= w;
            la_store4(p, x);
        }
        __syncthreads();
        float4 u[RK][CV];
#pragma unroll
        for (int r = 0; r < RK; ++r)
#pragma unroll
            for (int m = 0; m < CV; ++m) u[r][m] = make_float4(0.f, 0.f, 0.f, 0.f);
        // rows 4 (4 wr + ry) + 64 g + {0..3}: RK = 4 or 8 rows in RK / 4 groups
        const int srow = 16 * wr + 4 * ry;
#pragma unroll (RK * CV > 8 ? 2 : 8)
        for (int j = 0; j < kC; ++j) {
            float4 y[CV];
#pragma unroll
            for (int m = 0; m < CV; ++m) y[m] = la_load4(sV + j * PV + col4 + 64 * m);
#pragma unroll
            for (int g = 0; g < RK / 4; ++g) {
                const float4 x = la_load4(sK + j * PK + srow + 64 * g);
#pragma unroll
                for (int m = 0; m < CV; ++m) {
                    fma4(u[4 * g][m], x.x, y[m]);
                    fma4(u[4 * g + 1][m], x.y, y[m]);
                    fma4(u[4 * g + 2][m], x.z, y[m]);
                    fma4(u[4 * g + 3][m], x.w, y[m]);
                }
            }
        }
        const float hi = sm[L::off_l + (c == kC ? 0 : 2)], lo = sm[L::off_l + (c == kC ? 1 : 3)];
#pragma unroll
        for (int r = 0; r < RK; ++r)
#pragma unroll
            for (int m = 0; m < CV; ++m) {
                float *p = sS + (srow + 64 * (r / 4) + r % 4) * PV + col4 + 64 * m;
                const float4 s = la_load4(p);
                fma4(u[r][m], lo, s);
                fma4(u[r][m], hi, s);
                la_store4(p, u[r][m]);
            }
    }
    __syncthreads();
    // ---- leaving state
    float *dst = STATES_ONLY ? slots + (size_t)seg * DK * DV
                 : (seg == a.nseg - 1 && ps.sT) ? ps.sT + (size_t)bh * DK * DV : nullptr;
    if (dst)
#pragma unroll 8
        for (int e = 4 * tid; e < DK * DV; e += 4 * kThreads) la_store4(dst + e, la_load4(sS + (e / DV) * PV + e % DV));
}

// A launch that may begin while the kernel ahead of it ends (it waits for that one's results).
template <typename Kernel>
cudaError_t launch_behind(Kernel kernel, size_t grid, size_t smem, const LaArgs &a, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e == cudaSuccess) note_launch();
    return e;
}

template <int DK, int DV, typename InT, bool STATES_ONLY>
cudaError_t launch_typed(const LaArgs &a, cudaStream_t stream)
{
    auto kernel = la_simt_kernel<DK, DV, InT, STATES_ONLY>;
    constexpr size_t bytes = LaSmem<DK, DV>::bytes;
    static OncePerDevice once;
    cudaError_t e = set_shared_memory(kernel, (int)bytes, once);
    if (e != cudaSuccess) return e;
    const int nwork = STATES_ONLY ? a.nseg - 1 : a.nseg;
    return launch_behind(kernel, (size_t)a.npass * a.B * a.H * nwork, bytes, a, stream);
}

template <typename InT, bool STATES_ONLY>
cudaError_t launch_dims(const LaArgs &a, cudaStream_t stream)
{
    if constexpr (sizeof(InT) == 4)             // bf16 runs on the tensor cores there
        if (a.dk == 128 && a.dv == 128) return launch_typed<128, 128, InT, STATES_ONLY>(a, stream);
    if (a.dk == 64 && a.dv == 64) return launch_typed<64, 64, InT, STATES_ONLY>(a, stream);
    if (a.dk == 128 && a.dv == 64) return launch_typed<128, 64, InT, STATES_ONLY>(a, stream);
    if (a.dk == 64 && a.dv == 128) return launch_typed<64, 128, InT, STATES_ONLY>(a, stream);
    return cudaErrorInvalidValue;
}

// fp32 arithmetic on CUDA cores.  states_only: each segment's own contribution to the state
// (all but the last's) goes to its slot of a.ws, [npass][B * H][nseg][dk][dv] fp32, no outputs.
cudaError_t launch_la_simt(const LaArgs &a, bool states_only, cudaStream_t stream)
{
    if (a.dtype == KDA_BF16)
        return states_only ? launch_dims<__nv_bfloat16, true>(a, stream) : launch_dims<__nv_bfloat16, false>(a, stream);
    return states_only ? launch_dims<float, true>(a, stream) : launch_dims<float, false>(a, stream);
}

}  // namespace

// Segments: with one per head a launch has npass B H CTAs that walk all chunks; with n of them
// the walk is n times shorter, but every segment's own state has to be known first (a second
// walk over k and v) and joined.  The number with the least modelled time is taken: waves of
// CTAs x (chunks of a walk x the cost of both walks + a fixed cost of the join), in chunks of
// the walk with outputs.
void la_choose_segments(LaArgs &a)
{
    constexpr int kMaxSegments = 32;        // a warp's lanes look at them
    const bool tc = la_tc_supported(a.dk, a.dv, a.dtype);
    const int C = tc ? 128 : kC;
    const int places = 148 * (!tc && a.dk == 64 && a.dv == 64 ? simt_resident<64, 64>() : 1);
    const double state_cost = tc ? 0.6 : 0.5, join_cost = tc ? 3.0 : 1.0, per_segment = tc ? 0.5 : 0.05;
    const int chunks = (a.T + C - 1) / C;
    const long long heads = (long long)a.npass * a.B * a.H;
    a.nseg = 1;
    a.seg_tokens = a.T > 0 ? chunks * C : C;
    double best = 0.0;
    for (int want = 1; want <= kMaxSegments && want <= chunks; ++want) {
        const int len = (chunks + want - 1) / want, n = (chunks + len - 1) / len;
        const long long waves = (heads * n + places - 1) / places;
        const double t = (double)waves * (n > 1 ? len * (1.0 + state_cost) + join_cost + per_segment * n : len);
        if (want == 1 || t < best) {
            best = t;
            a.nseg = n;
            a.seg_tokens = len * C;
        }
    }
}

size_t la_workspace_bytes(const LaArgs &a)
{
    if (la_tc_supported(a.dk, a.dv, a.dtype)) return la_tc_workspace_bytes(a);
    return a.nseg > 1 ? sizeof(float) * (size_t)a.npass * a.B * a.H * a.nseg * a.dk * a.dv : 0;
}

// CUDA cores with nseg > 1: every segment's own contribution, then the outputs.
cudaError_t launch_la(const LaArgs &a, cudaStream_t stream)
{
    if (la_tc_supported(a.dk, a.dv, a.dtype)) return launch_la_tc(a, stream);
    if (a.nseg > 1) {
        const cudaError_t e = launch_la_simt(a, true, stream);
        if (e != cudaSuccess) return e;
    }
    return launch_la_simt(a, false, stream);
}

}  // namespace kda

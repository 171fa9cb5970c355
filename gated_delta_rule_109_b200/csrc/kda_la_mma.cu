// Linear attention with one decay per head on warp matrix instructions: fp32 for all head
// dimensions, bf16 where one is 64 (the mathematics is in kda_la.cuh).
//
// One CTA walks the chunks of 64 tokens of one (pass, b, h, segment) with the state
// resident in shared memory as fp32.  A chunk is four products of 64-wide tiles, Q K^T, P V,
// Q S and K'^T V; of each tile a warp has 16 rows and 32 columns.  Operands are fp32 in shared
// memory and go in as two tf32 parts, so the sums keep fp32's accuracy.  Multiply-adds on CUDA
// cores with 4 x 4 register tiles were bound by shared memory, 3 wavefronts to 4 x 32
// multiply-adds of a 16-byte read (B4 T2048 H32 d128 fp32 695 us, B8 T2048 H32 d64 bf16 468):
// here they are 504 and 266, the tensor pipe is half busy and the waits are its own and the
// barriers'.  A chunk's loads are all under way together, ahead of the state's update, and
// two CTAs share an SM where they fit.  Powers of lambda are computed in 64 bits once per CTA,
// so their rounding does not grow along the sequence.
#include <type_traits>

#include "kda_la.cuh"

namespace kda {
namespace {

constexpr int kC = 64;
constexpr int kThreads = 256;

template <int DK, int DV>
struct LaSmem {
    static constexpr int PK = DK + 8, PV = DV + 4, PP = kC + 8;   // row pitches; see mma_split
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

// ---- products on warp matrix instructions (m16n8k8, tf32 operands, fp32 accumulators).  An fp32
// operand goes in as two tf32 parts of 11 bits: hi is the nearest, lo the rest with its last bits
// cut off, 2^-22 of x at most and of either sign.  Of the four products of parts lo lo is left
// out, 2^-22 of a term.  A NaN stays one: where the sum that rounds hi runs over, lo is the NaN.
// (Rounding lo as well, by conversion instructions, left the same errors: 4 % more time at
// B2 T1023 H8 d64.)  What is bf16 is its own hi.
//
// Lane (g, t) = (lane / 4, lane % 4) holds rows g, g + 8 of A, column g of B, and of both the
// depths 2 t, 2 t + 1 of a step's 8 (the order of the depths is free as long as A and B agree).
// Operands that lie [row][depth] are read as pairs: pitches of 8 banks a row spread them over all
// banks.  [depth][column] ones are read as words from rows 2 t and 2 t + 1: there it is 4 banks.
struct Parts { uint32_t hi, lo; };
template <bool EXACT> __device__ __forceinline__ Parts parts_of(float x)
{
    if (EXACT) return {__float_as_uint(x), 0u};
    const uint32_t hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    return {hi, __float_as_uint(x - __uint_as_float(hi)) & 0xffffe000u};
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c[n] += A B_n over 8 depths.  The matrix instruction cuts what it adds to its accumulator off
// instead of rounding it, so each step's sum starts from zero, with the small products, and is
// added to c by an fp32 addition: one accumulator over all depths left 1.7e-6 of an output's
// norm where this leaves 1.8e-7, for 3 to 9 % of the time.  COARSE: one accumulator (an output
// that is rounded to bf16).  x0, x1: A's rows g and g + 8 at the lane's two depths; y[n]: B_n's
// column at them.
template <bool A_EXACT, bool B_EXACT, bool COARSE, int N>
__device__ __forceinline__ void mma_split(float (*c)[4], float2 x0, float2 x1, const float2 (&y)[N])
{
    const Parts p[4] = {parts_of<A_EXACT>(x0.x), parts_of<A_EXACT>(x1.x), parts_of<A_EXACT>(x0.y), parts_of<A_EXACT>(x1.y)};
    const uint32_t hi[4] = {p[0].hi, p[1].hi, p[2].hi, p[3].hi}, lo[4] = {p[0].lo, p[1].lo, p[2].lo, p[3].lo};
    Parts q[N][2];
#pragma unroll
    for (int n = 0; n < N; ++n) { q[n][0] = parts_of<B_EXACT>(y[n].x); q[n][1] = parts_of<B_EXACT>(y[n].y); }
    float fresh[N][4] = {};
    float (*sum)[4] = COARSE ? c : fresh;
    if (!B_EXACT)
#pragma unroll
        for (int n = 0; n < N; ++n) mma_tf32(sum[n], hi, q[n][0].lo, q[n][1].lo);
    if (!A_EXACT)
#pragma unroll
        for (int n = 0; n < N; ++n) mma_tf32(sum[n], lo, q[n][0].hi, q[n][1].hi);
#pragma unroll
    for (int n = 0; n < N; ++n) mma_tf32(sum[n], hi, q[n][0].hi, q[n][1].hi);
    if (!COARSE)
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) c[n][i] += fresh[n][i];
}
__device__ __forceinline__ float2 load2(const float *p) { return *reinterpret_cast<const float2 *>(p); }
template <typename T> __device__ __forceinline__ void store_pair(T *p, float x, float y);
template <> __device__ __forceinline__ void store_pair<float>(float *p, float x, float y) { *reinterpret_cast<float2 *>(p) = make_float2(x, y); }
template <> __device__ __forceinline__ void store_pair<__nv_bfloat16>(__nv_bfloat16 *p, float x, float y)
{
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(x, y);
}

// A chunk's rows of D channels to shared memory as fp32, in the order of the walk: row t is
// token t (forward) or c - 1 - t (reversed), rows from c on are zeros.  `src` is row 0's, `step`
// leads to the next.  The loads are all issued before the first is needed.
template <int D, int PITCH>
__device__ __forceinline__ void stage(float *dst, const float *src, ptrdiff_t step, int c, int tid)
{
#pragma unroll
    for (int e = 0; e < kC * D / 4 / kThreads; ++e) {
        const int id = e * kThreads + tid, t = id / (D / 4), x = 4 * (id % (D / 4));
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst + t * PITCH + x);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                     :: "r"(to), "l"(src + (t < c ? t * step + x : 0)), "r"(t < c ? 16 : 0) : "memory");
    }
}
template <int D, int PITCH>
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
        la_store4(dst + (id / (D / 4)) * PITCH + 4 * (id % (D / 4)), v[e]);
    }
}

// CTAs of an SM: two where the shared memory of both fits
template <int DK, int DV> constexpr int mma_resident() { return LaSmem<DK, DV>::bytes <= 112 * 1024 ? 2 : 1; }

template <int DK, int DV, typename InT, bool STATES_ONLY>
__global__ void __launch_bounds__(kThreads, mma_resident<DK, DV>())
la_mma_kernel(const __grid_constant__ LaArgs a)
{
    using L = LaSmem<DK, DV>;
    constexpr int PK = L::PK, PV = L::PV, PP = L::PP;
    constexpr bool EX = sizeof(InT) == 2;       // q, k, v are exact in one part
    constexpr int GK = DK / 64, CV = DV / 64;   // groups of 64 state rows and of 64 columns
    extern __shared__ __align__(16) float sm[];
    float *sQ = sm + L::off_q, *sK = sm + L::off_k, *sV = sm + L::off_v, *sP = sm + L::off_p, *sS = sm + L::off_s;
    float *sW = sm + L::off_w;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // Of a product's 64 x 64 tile warp w has rows 16 wr .. and columns 32 wc ..  Warps w and w + 4
    // share a scheduler: together they have as many causal pairs as any two.
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t2 = 2 * (lane & 3);
    const int wr = warp < 4 ? warp : 7 - warp, wc = warp >> 2, row = 16 * wr + g, col = 32 * wc;
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
        if (!STATES_ONLY) stage<DK, PK>(sQ, q + at * DK, step * DK, c, tid);
        stage<DK, PK>(sK, k + at * DK, step * DK, c, tid);
        stage<DV, PV>(sV, v + at * DV, step * DV, c, tid);
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
            for (int x = 0; x < seg; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 u = la_load4(slots + (size_t)x * DK * DV + e0 + 4 * i * kThreads);
                    fma4(s[i], weight[2 * x + 1], u);
                    fma4(s[i], weight[2 * x], u);
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
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();                        // the chunk's rows and the state are there

        if (!STATES_ONLY) {
            // ---- P_ij = f_intra lambda^(i-j) (q_i . k_j), j <= i: of the 2 (wr + 1) tiles of 8 columns
            // that hold such pairs each of a row's two warps makes half
            auto scores = [&](auto tiles) {
                constexpr int N = decltype(tiles)::value;
                const int first = 8 * N * wc;
                float s[N][4] = {};
#pragma unroll 2
                for (int d = t2; d < DK; d += 8) {
                    float2 y[N];
#pragma unroll
                    for (int n = 0; n < N; ++n) y[n] = load2(sK + (first + 8 * n + g) * PK + d);
                    mma_split<EX, EX, EX>(s, load2(sQ + row * PK + d), load2(sQ + (row + 8) * PK + d), y);
                }
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = row + 8 * i, m = first + 8 * n + t2, apart = r - m;
                        *reinterpret_cast<float2 *>(sP + r * PP + m) =
                            make_float2(apart >= 0 ? s[n][2 * i] * (sW[max(apart, 0)] * ps.f_intra) : 0.f,
                                        apart >= 1 ? s[n][2 * i + 1] * (sW[max(apart - 1, 0)] * ps.f_intra) : 0.f);
                    }
            };
            if (wr == 0) scores(std::integral_constant<int, 1>{});
            else if (wr == 1) scores(std::integral_constant<int, 2>{});
            else if (wr == 2) scores(std::integral_constant<int, 3>{});
            else scores(std::integral_constant<int, 4>{});
            // ---- out: (f_inter lambda^(.) Q) S, and with all scores there P V
            float o[4 * CV][4] = {};
            const float f0 = ps.f_inter * sW[rev ? row : row + 1], f1 = ps.f_inter * sW[rev ? row + 8 : row + 9];
#pragma unroll (CV > 1 ? 1 : 2)
            for (int d = t2; d < DK; d += 8) {
                float2 x0 = load2(sQ + row * PK + d), x1 = load2(sQ + (row + 8) * PK + d);
                x0.x *= f0; x0.y *= f0; x1.x *= f1; x1.y *= f1;
#pragma unroll
                for (int m = 0; m < CV; ++m) {
                    float2 y[4];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const float *p = sS + d * PV + col + 64 * m + 8 * n + g;
                        y[n] = make_float2(p[0], p[PV]);
                    }
                    mma_split<false, false, EX>(o + 4 * m, x0, x1, y);
                }
            }
            __syncthreads();
#pragma unroll 2
            for (int j = t2; j < 16 * wr + 16; j += 8) {
                const float2 x0 = load2(sP + row * PP + j), x1 = load2(sP + (row + 8) * PP + j);
#pragma unroll
                for (int m = 0; m < CV; ++m) {
                    float2 y[4];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const float *p = sV + j * PV + col + 64 * m + 8 * n + g;
                        y[n] = make_float2(p[0], p[PV]);
                    }
                    mma_split<false, EX, EX>(o + 4 * m, x0, x1, y);
                }
            }
            InT *out = static_cast<InT *>(ps.out);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (row + 8 * i < c) {
                    InT *p = out + token_at(t0, c, row + 8 * i) * DV + col + t2;
#pragma unroll
                    for (int n = 0; n < 4 * CV; ++n) store_pair(p + 64 * (n / 4) + 8 * (n % 4), o[n][2 * i], o[n][2 * i + 1]);
                }
        }
        // ---- U = K'^T V with k'_j = f_write lambda^(.) k_j
        float u[GK * CV * 4][4] = {};
        const int fade = rev ? c : c - 1;
#pragma unroll 2
        for (int j = t2; j < kC; j += 8) {
            const float w0 = ps.f_write * sW[max(fade - j, 0)], w1 = ps.f_write * sW[max(fade - j - 1, 0)];
            float2 y[4 * CV];
#pragma unroll
            for (int n = 0; n < 4 * CV; ++n) {
                const float *p = sV + j * PV + col + 64 * (n / 4) + 8 * (n % 4) + g;
                y[n] = make_float2(p[0], p[PV]);
            }
#pragma unroll
            for (int k = 0; k < GK; ++k) {
                const float *p = sK + j * PK + row + 64 * k;
                mma_split<false, EX, false>(u + 4 * CV * k, make_float2(w0 * p[0], w1 * p[PK]), make_float2(w0 * p[8], w1 * p[PK + 8]), y);
            }
        }
        __syncthreads();                        // every reader of the rows and of the state is done
        if (it + 1 < n1) load(it + 1);
        // ---- S <- lambda^c S + U
        const float hi = sm[L::off_l + (c == kC ? 0 : 2)], lo = sm[L::off_l + (c == kC ? 1 : 3)];
#pragma unroll
        for (int k = 0; k < GK; ++k)
#pragma unroll
            for (int n = 0; n < 4 * CV; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float2 *p = reinterpret_cast<float2 *>(sS + (row + 8 * i + 64 * k) * PV + col + 64 * (n / 4) + 8 * (n % 4) + t2);
                    float2 x = make_float2(u[4 * CV * k + n][2 * i], u[4 * CV * k + n][2 * i + 1]);
                    const float2 s = *p;
                    x.x += lo * s.x; x.y += lo * s.y;
                    x.x += hi * s.x; x.y += hi * s.y;
                    *p = x;
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
    auto kernel = la_mma_kernel<DK, DV, InT, STATES_ONLY>;
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

// states_only: each segment's own contribution to the state
// (all but the last's) goes to its slot of a.ws, [npass][B * H][nseg][dk][dv] fp32, no outputs.
cudaError_t launch_la_mma(const LaArgs &a, bool states_only, cudaStream_t stream)
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
// the walk with outputs.  The four costs were fitted to times in a graph; us, the number taken /
// the best of 1 to 32 / one, forward:
// bf16 128 x 128: B1 T1023 H8 30 / 27 / 30, B1 T4096 H16 43 / 43 / 93, B1 T8192 H4 49 / 47 / 169,
// B1 T30000 H32 294 / 294 / 626, B1 T16384 H60 342 / 323 / 356, B4 T2047 H32 60 / 60 / 60;
// fp32 128 x 128: B1 T1023 H8 45 / 43 / 264, B1 T30000 H32 2369 / 2369 / 7240; 64 x 64: B2 T1023 H8
// 23 / 23 / 99, B1 T16384 H60 871 / 800 / 1649, B2 T5003 H90 863 / 712 / 862;
// bf16 64 x 64: B1 T4096 H16 53 / 53 / 303; 128 x 64: B1 T16384 H60 1561 / 1560 / 2281.
// Of 100 shapes, gradients among them, 4 are more than 1.1 off the best: the one of 712, the same in
// bf16 (656 / 557), B1 T1023 H8 above, and the gradients of B1 T16384 H60 bf16 128 x 128 (959 / 775).
void la_choose_segments(LaArgs &a)
{
    constexpr int kMaxSegments = 32;        // a warp's lanes look at them
    const bool tc = la_tc_supported(a.dk, a.dv, a.dtype);
    const int C = tc ? 128 : kC;
    const int places = 148 * (!tc && a.dk == 64 && a.dv == 64 ? mma_resident<64, 64>() : 1);
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

// Warp matrix instructions with nseg > 1: every segment's own contribution, then the outputs.
cudaError_t launch_la(const LaArgs &a, cudaStream_t stream)
{
    if (la_tc_supported(a.dk, a.dv, a.dtype)) return launch_la_tc(a, stream);
    if (a.nseg > 1) {
        const cudaError_t e = launch_la_mma(a, true, stream);
        if (e != cudaSuccess) return e;
    }
    return launch_la_mma(a, false, stream);
}

}  // namespace kda

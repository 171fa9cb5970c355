// Paged decode attention on CUDA cores (the split of the work is in kda_paged.cuh).
//
// A CTA is four warps; of every unit of 64 keys a warp takes 16 and keeps its own running
// maximum, sum and output, so that the warps meet only at the end of a stretch.  Each warp
// moves its keys and values through its own ring of shared-memory slots with 16-byte
// asynchronous copies, kStages - 1 units ahead.  Scores: lane = (key, half of the
// channels), the query broadcast from shared memory.  Output: lane = D / 32 channels, the
// probabilities broadcast.  Sums and statistics are fp32.
#include <math.h>

#include "kda_la.cuh"
#include "kda_paged.cuh"

namespace kda {

__device__ unsigned int g_paged_status = 0;

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps, kWarpKeys = kPagedTile / kWarps, kStages = 3;
constexpr int kSms = 148;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool real)
{
    const uint32_t n = real ? 16u : 0u;         // 0: the slot is zeroed and src is not read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

// Keys that row b attends to; -1 for a row that is left alone (idle, or longer than its table).
__device__ __forceinline__ int row_keys(const PagedArgs &a, int b)
{
    const int len = a.lengths[b];
    if (len < 0) return -1;
    if ((long long)len + (a.k ? 1 : 0) > (long long)a.max_pages * a.page_size) {
        atomicOr(&g_paged_status, 1u);
        return -1;
    }
    return len + (a.k ? 1 : 0);
}
__device__ __forceinline__ int row_tiles(const PagedArgs &a, int b) { return (max(row_keys(a, b), 0) + kPagedTile - 1) / kPagedTile; }

// CTAs of a grid that own units: each of them has at least one.
__device__ __forceinline__ unsigned long long owners_of(unsigned long long total, unsigned long long grid)
{
    return total < grid ? total : grid;
}

// Block-wide: the units of all rows, and row b with its first unit: the row asked for
// (row >= 0), or else the one that the first unit of CTA `part` of `parts` belongs to (b = B
// if there is none).  `per` units stand beside each other for every tile of a row (heads).
struct RowAt { int b; unsigned long long first, total; };
__device__ __forceinline__ RowAt find_row(const PagedArgs &a, unsigned long long per, unsigned long long part,
                                          unsigned long long parts, int row)
{
    __shared__ unsigned long long s_sum[kThreads / 32], s_first;
    __shared__ int s_b;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = (a.B + kThreads - 1) / kThreads, b0 = min(tid * n, a.B), b1 = min(b0 + n, a.B);
    unsigned long long sum = 0;
    for (int b = b0; b < b1; ++b) sum += per * (unsigned long long)row_tiles(a, b);
    unsigned long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    if (tid == 0) s_b = a.B;
    if (lane == 31) s_sum[warp] = inc;
    __syncthreads();
    unsigned long long before = inc - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += s_sum[w];
        total += s_sum[w];
    }
    // by row (row >= 0), or by the first unit of part `part` of `parts`
    const unsigned long long at = total ? part * total / owners_of(total, parts) : 0;
    for (int b = b0; b < b1; ++b) {
        const unsigned long long u = per * (unsigned long long)row_tiles(a, b);
        if (row >= 0 ? b == row : (at >= before && at < before + u)) { s_b = b; s_first = before; }
        before += u;
    }
    __syncthreads();
    RowAt r;
    r.b = s_b;
    r.first = s_first;
    r.total = total;
    return r;
}

template <int D, typename InT, int HG>
struct PagedSmem {
    static constexpr int row = D * (int)sizeof(InT) + 16;                 // bytes; rows 4 banks apart
    static constexpr int slot = 2 * kWarpKeys * row;                      // K rows, then V rows
    static constexpr int ring = kWarps * kStages * slot;
    static constexpr int off_q = ring;                                    // [HG][D] fp32, scaled by scale log2 e
    static constexpr int off_p = off_q + HG * D * 4;                      // [warp][HG][16]
    static constexpr int off_ml = off_p + kWarps * HG * kWarpKeys * 4;    // [warp][HG] maximum, sum
    static constexpr int total = off_ml + kWarps * HG * 8;
    static_assert(kWarps * HG * D * 4 <= ring, "the warps' outputs meet in the ring");
};

template <int D, typename InT, int HG>
__global__ void __launch_bounds__(kThreads)
paged_decode_kernel(const __grid_constant__ PagedArgs a)
{
    using L = PagedSmem<D, InT, HG>;
    constexpr int CPR = D * (int)sizeof(InT) / 16;      // 16-byte pieces of a row
    constexpr int DL = D / 32;                          // output channels of a lane
    extern __shared__ __align__(16) uint8_t smem[];
    const uint32_t sbase = (uint32_t)__cvta_generic_to_shared(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float *sQ = reinterpret_cast<float *>(smem + L::off_q);
    float *sP = reinterpret_cast<float *>(smem + L::off_p) + warp * HG * kWarpKeys;
    float *sML = reinterpret_cast<float *>(smem + L::off_ml);
    float *sO = reinterpret_cast<float *>(smem);

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const int group = a.H / a.Hkv, blocks = (group + HG - 1) / HG;
    const unsigned long long per = (unsigned long long)a.Hkv * blocks;
    const RowAt at = find_row(a, per, blockIdx.x, gridDim.x, -1);
    const unsigned long long owners = owners_of(at.total, gridDim.x);
    if (blockIdx.x >= owners) return;
    unsigned long long u = (unsigned long long)blockIdx.x * at.total / owners;
    const unsigned long long u1 = ((unsigned long long)blockIdx.x + 1) * at.total / owners;

    int b = at.b, part = 0;
    unsigned long long row_first = at.first;
    const InT *kc = static_cast<const InT *>(a.k_cache), *vc = static_cast<const InT *>(a.v_cache);
    while (u < u1) {
        int n = row_keys(a, b), tiles = (max(n, 0) + kPagedTile - 1) / kPagedTile;
        while (u >= row_first + per * tiles) {          // next row that has units
            row_first += per * tiles;
            n = row_keys(a, ++b);
            tiles = (max(n, 0) + kPagedTile - 1) / kPagedTile;
        }
        const int hb = (int)((u - row_first) / tiles);          // (key-value head, block) of the stretch
        const int hk = hb / blocks, h0 = hk * group + (hb % blocks) * HG, nh = min(HG, group - (hb % blocks) * HG);
        const int tile0 = (int)((u - row_first) % tiles);
        const int tile1 = (int)min((unsigned long long)tiles, (unsigned long long)tile0 + (u1 - u));
        const bool whole = tile0 == 0 && tile1 == tiles;
        const int new_at = a.k ? n - 1 : -1;

        __syncthreads();                                // the stretch before is written out
        for (int e = tid; e < HG * D; e += kThreads)
            sQ[e] = e / D < nh ? to_f32(static_cast<const InT *>(a.q)[((size_t)b * a.H + h0) * D + e]) * (a.scale * kLog2e)
                               : 0.f;
        __syncthreads();

        // One slot of this warp's ring: 16 keys and values from key t on; masked rows are zeros.
        auto fetch = [&](int tile) {
            const int t = tile * kPagedTile + warp * kWarpKeys + (lane & 15);
            const InT *kp = kc, *vp = vc;
            bool real = tile < tile1 && t < n;
            if (real) {
                const int page = a.block_table[(size_t)b * a.max_pages + t / a.page_size];
                const bool good = page >= 0 && page < a.num_pages;
                if (!good) atomicOr(&g_paged_status, 1u);
                const size_t at_cache = (((size_t)(good ? page : 0) * a.page_size + t % a.page_size) * a.Hkv + hk) * D;
                if (t == new_at) {
                    kp = static_cast<const InT *>(a.k) + ((size_t)b * a.Hkv + hk) * D;
                    vp = static_cast<const InT *>(a.v) + ((size_t)b * a.Hkv + hk) * D;
                } else {
                    kp += at_cache;
                    vp += at_cache;
                    real = good;
                }
            }
            const uint32_t dst = sbase + (uint32_t)((warp * kStages + tile % kStages) * L::slot);
            const unsigned long long kpi = reinterpret_cast<unsigned long long>(kp), vpi = reinterpret_cast<unsigned long long>(vp);
#pragma unroll
            for (int e = 0; e < kWarpKeys * CPR / 32; ++e) {
                const int id = e * 32 + lane, r = id / CPR, c = id % CPR;
                const bool ok = __shfl_sync(0xffffffffu, real, r);
                const uint8_t *ks = reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, kpi, r)) + 16 * c;
                const uint8_t *vs = reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, vpi, r)) + 16 * c;
                cp16(dst + (uint32_t)(r * L::row + 16 * c), ok ? ks : reinterpret_cast<const uint8_t *>(kc), ok);
                cp16(dst + (uint32_t)((kWarpKeys + r) * L::row + 16 * c), ok ? vs : reinterpret_cast<const uint8_t *>(vc), ok);
            }
        };
        // a key counts if it is one of the row's and its page is in the cache
        auto counts = [&](int t) {
            if (t >= n) return false;
            if (t == new_at) return true;
            const int page = a.block_table[(size_t)b * a.max_pages + t / a.page_size];
            return page >= 0 && page < a.num_pages;
        };

        float m[HG], l[HG], o[HG][DL];
#pragma unroll
        for (int g = 0; g < HG; ++g) {
            m[g] = -INFINITY;
            l[g] = 0.f;
#pragma unroll
            for (int x = 0; x < DL; ++x) o[g][x] = 0.f;
        }
#pragma unroll
        for (int st = 0; st < kStages - 1; ++st) {
            fetch(tile0 + st);
            cp_commit();
        }
        for (int tile = tile0; tile < tile1; ++tile) {
            fetch(tile + kStages - 1);
            cp_commit();
            cp_wait<kStages - 1>();
            __syncwarp();
            const uint8_t *slot = smem + (warp * kStages + tile % kStages) * L::slot;
            const int t = tile * kPagedTile + warp * kWarpKeys + (lane & 15);
            // ---- scores of key lane & 15, channels split between the half-warps
            float s[HG];
#pragma unroll
            for (int g = 0; g < HG; ++g) s[g] = 0.f;
            const InT *kr = reinterpret_cast<const InT *>(slot + (lane & 15) * L::row) + (lane >> 4) * (D / 2);
            const float *qh = sQ + (lane >> 4) * (D / 2);
#pragma unroll 4
            for (int d = 0; d < D / 2; d += 4) {
                const float4 kk = la_load4(kr + d);
#pragma unroll
                for (int g = 0; g < HG; ++g) {
                    const float4 qq = la_load4(qh + g * D + d);
                    s[g] += kk.x * qq.x; s[g] += kk.y * qq.y; s[g] += kk.z * qq.z; s[g] += kk.w * qq.w;
                }
            }
            const bool seen = counts(t);
#pragma unroll
            for (int g = 0; g < HG; ++g) {
                s[g] += __shfl_xor_sync(0xffffffffu, s[g], 16);
                if (!seen) s[g] = -INFINITY;
                if (__any_sync(0xffffffffu, s[g] > m[g])) {     // the running maximum rises
                    float top = s[g];
#pragma unroll
                    for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                    top = fmaxf(top, m[g]);
                    const float f = exp2f(m[g] - top);          // exp2(-inf) = 0 the first time
                    l[g] *= f;
#pragma unroll
                    for (int x = 0; x < DL; ++x) o[g][x] *= f;
                    m[g] = top;
                }
                // a maximum of -inf: every score so far is -inf, each weighs nothing
                const float p = seen ? exp2f(s[g] - (m[g] == -INFINITY ? 0.f : m[g])) : 0.f;
                if (lane < 16) {
                    l[g] += p;
                    sP[g * kWarpKeys + lane] = p;
                }
            }
            __syncwarp();
            // ---- output channels DL lane .. of all 16 keys
            const InT *vr = reinterpret_cast<const InT *>(slot + kWarpKeys * L::row) + DL * lane;
#pragma unroll
            for (int j = 0; j < kWarpKeys; j += 4) {
                float x[4][DL];
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) {
                    const InT *p = reinterpret_cast<const InT *>(reinterpret_cast<const uint8_t *>(vr) + (j + jj) * L::row);
#pragma unroll
                    for (int y = 0; y < DL; ++y) x[jj][y] = to_f32(p[y]);
                }
#pragma unroll
                for (int g = 0; g < HG; ++g) {
                    const float4 p = la_load4(sP + g * kWarpKeys + j);
#pragma unroll
                    for (int y = 0; y < DL; ++y) {
                        o[g][y] += p.x * x[0][y]; o[g][y] += p.y * x[1][y];
                        o[g][y] += p.z * x[2][y]; o[g][y] += p.w * x[3][y];
                    }
                }
            }
            __syncwarp();                               // the slot and sP are free again
        }
        cp_wait<0>();
        // ---- the new token's key and value go to their place in the cache (one owner per head)
        if (new_at >= 0 && hb % blocks == 0 && new_at / kPagedTile >= tile0 && new_at / kPagedTile < tile1) {
            const int page = a.block_table[(size_t)b * a.max_pages + new_at / a.page_size];
            if (page >= 0 && page < a.num_pages) {
                const size_t dst = (((size_t)page * a.page_size + new_at % a.page_size) * a.Hkv + hk) * D;
                const size_t src = ((size_t)b * a.Hkv + hk) * D;
                for (int e = tid; e < CPR; e += kThreads) {
                    reinterpret_cast<uint4 *>(static_cast<InT *>(a.k_cache) + dst)[e] =
                        reinterpret_cast<const uint4 *>(static_cast<const InT *>(a.k) + src)[e];
                    reinterpret_cast<uint4 *>(static_cast<InT *>(a.v_cache) + dst)[e] =
                        reinterpret_cast<const uint4 *>(static_cast<const InT *>(a.v) + src)[e];
                }
            }
        }
        // ---- the four warps meet
        __syncthreads();
#pragma unroll
        for (int g = 0; g < HG; ++g) {
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) l[g] += __shfl_xor_sync(0xffffffffu, l[g], x);
            if (lane == 0) {
                sML[(warp * HG + g) * 2] = m[g];
                sML[(warp * HG + g) * 2 + 1] = l[g];
            }
#pragma unroll
            for (int x = 0; x < DL; ++x) sO[(warp * HG + g) * D + DL * lane + x] = o[g][x];
        }
        __syncthreads();
        float *slot = a.ws + ((size_t)blockIdx.x * 2 + (part > 0 ? 1 : 0)) * HG * (D + 2);
        for (int e = tid; e < nh * D; e += kThreads) {
            const int g = e / D, d = e % D;
            float top = -INFINITY, sum = 0.f, acc = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sML[(w * HG + g) * 2]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw = sML[(w * HG + g) * 2], f = mw == -INFINITY ? 0.f : exp2f(mw - top);
                sum += f * sML[(w * HG + g) * 2 + 1];
                acc += f * sO[(w * HG + g) * D + d];
            }
            if (whole) {
                static_cast<InT *>(a.out)[((size_t)b * a.H + h0 + g) * D + d] = la_round<InT>(sum > 0.f ? acc / sum : 0.f);
            } else {
                slot[e] = acc;
                if (d == 0) { slot[HG * D + 2 * g] = top; slot[HG * D + 2 * g + 1] = sum; }
            }
        }
        u += (unsigned long long)(tile1 - tile0);
        ++part;
    }
}

// One CTA per (row, key-value head, block of query heads): rows without keys get zeros, and
// stretches that several CTAs share are joined in the order of the keys.
template <int D, typename InT, int HG>
__global__ void __launch_bounds__(kThreads)
paged_join_kernel(const __grid_constant__ PagedArgs a, unsigned int grid)
{
    const int group = a.H / a.Hkv, blocks = (group + HG - 1) / HG;
    const unsigned long long per = (unsigned long long)a.Hkv * blocks;
    const int b = blockIdx.x / (int)per, hb = blockIdx.x % (int)per;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int n = row_keys(a, b);
    if (n < 0) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int hk = hb / blocks, h0 = hk * group + (hb % blocks) * HG, nh = min(HG, group - (hb % blocks) * HG);
    InT *out = static_cast<InT *>(a.out) + ((size_t)b * a.H + h0) * D;
    if (n == 0) {
        for (int e = tid; e < nh * D; e += kThreads) out[e] = la_round<InT>(0.f);
        return;
    }
    const RowAt at = find_row(a, per, 0, 1, b);
    const unsigned long long tiles = (unsigned long long)(n + kPagedTile - 1) / kPagedTile;
    const unsigned long long x0 = at.first + hb * tiles, x1 = x0 + tiles - 1;
    // the CTA that has unit x: the largest c with c U / G <= x (G here: the owners)
    const unsigned long long owners = owners_of(at.total, grid);
    const unsigned int c0 = (unsigned int)(((x0 + 1) * owners - 1) / at.total), c1 = (unsigned int)(((x1 + 1) * owners - 1) / at.total);
    if (c0 == c1) return;                               // written by its only owner
    // the first owner's stretch is its second part if it began with another one
    const unsigned int first_part = (unsigned long long)c0 * at.total / owners < x0 ? 1u : 0u;
    constexpr int DL = D / 32;
    for (int g = warp; g < nh; g += kWarps) {
        float top = -INFINITY;
        for (unsigned int c = c0 + lane; c <= c1; c += 32) {
            const float *slot = a.ws + ((size_t)c * 2 + (c == c0 ? first_part : 0u)) * HG * (D + 2);
            top = fmaxf(top, slot[HG * D + 2 * g]);
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        float sum = 0.f, acc[DL];
#pragma unroll
        for (int x = 0; x < DL; ++x) acc[x] = 0.f;
#pragma unroll 4
        for (unsigned int c = c0; c <= c1; ++c) {
            const float *slot = a.ws + ((size_t)c * 2 + (c == c0 ? first_part : 0u)) * HG * (D + 2);
            const float mw = slot[HG * D + 2 * g], f = mw == -INFINITY ? 0.f : exp2f(mw - top);
            sum += f * slot[HG * D + 2 * g + 1];
#pragma unroll
            for (int x = 0; x < DL; ++x) acc[x] += f * slot[g * D + DL * lane + x];
        }
#pragma unroll
        for (int x = 0; x < DL; ++x) out[g * D + DL * lane + x] = la_round<InT>(sum > 0.f ? acc[x] / sum : 0.f);
    }
}

// CTAs that fit an SM by their shared memory
template <int D, typename InT, int HG>
constexpr int resident() { return 226 * 1024 / (PagedSmem<D, InT, HG>::total + 1024); }

int heads_per_block(int group) { return group >= 8 ? 8 : group > 4 ? 8 : group > 2 ? 4 : group; }

template <int D, typename InT, int HG>
cudaError_t launch_typed(const PagedArgs &a, cudaStream_t stream)
{
    using L = PagedSmem<D, InT, HG>;
    auto kernel = paged_decode_kernel<D, InT, HG>;
    static OncePerDevice once;
    cudaError_t e = set_shared_memory(kernel, L::total, once);
    if (e != cudaSuccess) return e;
    const unsigned int grid = kSms * resident<D, InT, HG>();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = L::total;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, kernel, a)) != cudaSuccess) return e;
    note_launch();
    const int group = a.H / a.Hkv, blocks = (group + HG - 1) / HG;
    cfg.gridDim = dim3((unsigned)((size_t)a.B * a.Hkv * blocks));
    cfg.dynamicSmemBytes = 0;
    if ((e = cudaLaunchKernelEx(&cfg, paged_join_kernel<D, InT, HG>, a, grid)) != cudaSuccess) return e;
    note_launch();
    return cudaGetLastError();
}

template <int D, typename InT>
cudaError_t launch_group(const PagedArgs &a, cudaStream_t stream)
{
    switch (heads_per_block(a.H / a.Hkv)) {
    case 1: return launch_typed<D, InT, 1>(a, stream);
    case 2: return launch_typed<D, InT, 2>(a, stream);
    case 4: return launch_typed<D, InT, 4>(a, stream);
    default: return launch_typed<D, InT, 8>(a, stream);
    }
}

}  // namespace

size_t paged_workspace_bytes(int H, int Hkv, int D, kda_dtype dtype)
{
    (void)dtype;
    // two stretches per CTA of a grid of at most 5 CTAs per SM
    return sizeof(float) * (size_t)kSms * 5 * 2 * heads_per_block(H / Hkv) * (D + 2);
}

cudaError_t launch_paged_decode(const PagedArgs &a, cudaStream_t stream)
{
    if (a.D == 128) {
        if (a.dtype == KDA_BF16) return launch_group<128, __nv_bfloat16>(a, stream);
        return launch_group<128, float>(a, stream);
    }
    if (a.dtype == KDA_BF16) return launch_group<64, __nv_bfloat16>(a, stream);
    return launch_group<64, float>(a, stream);
}

cudaError_t take_paged_device_status(unsigned int *status)
{
    cudaError_t e = cudaMemcpyFromSymbol(status, g_paged_status, sizeof(*status));
    if (e == cudaSuccess && *status) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_paged_status, &zero, sizeof(zero));
    }
    return e;
}

}  // namespace kda

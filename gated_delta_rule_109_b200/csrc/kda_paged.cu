// Paged decode attention (the split of the work is in kda_paged.cuh).
//
// A CTA is four warps; of every unit a warp takes 16 keys of one key-value head and keeps its
// own running maximum, sum and output, so that the warps of a head meet only at the end of a
// stretch.  Each warp
// moves its keys and values through its own ring of shared-memory slots with 16-byte
// asynchronous copies, kStages - 1 units ahead, and looks the page of its next unit up one
// unit before that.  Reading the cache is what bounds it: every key and value is read once
// for the query heads of a block, which are all of its group's up to 16 (bf16) or 8 (fp32).  A
// larger group has several blocks, and each reads the row again.
//
// bf16: the products are warp matrix instructions with the keys as rows, S^T = K q^T and
// O^T = V^T P^T, so that the 8 columns are query heads and a group of fewer than 8 wastes
// little (with the heads as rows it would be 16).  There is one query per sequence: at most
// some 40 flops per byte, far from what tcgen05's 128-row tiles are for.  P is split into two
// bf16 parts, which leaves the rounding of the output as the only one of that size.  Both parts of
// a weight are positive (the first is the largest bf16 below it, together they are off by at most
// 2^-16 of it), so that an infinite value stays one: rounded to nearest, the second part would be
// zero or negative for half of all weights, and 0 or -1 times infinity a NaN.
// fp32: CUDA cores.  Scores: lane = (key, half of the channels), the query broadcast from
// shared memory.  Output: lane = D / 32 channels, the probabilities broadcast.
// Sums and statistics are fp32 in both.
#include <math.h>

#include "kda_la.cuh"
#include "kda_paged.cuh"

namespace kda {

__device__ unsigned int g_paged_status = 0;

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps, kWarpKeys = 16, kStages = 3;
constexpr int kSms = 148, kMaxResident = 4;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool real)
{
    const uint32_t n = real ? 16u : 0u;         // 0: the slot is zeroed and src is not read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

// t / d and t % d for 0 <= t < 2^31 by multiplication: with 2^l >= d > 2^(l-1) and
// m = floor(2^32 (2^l - d) / d) + 1 the quotient is (m t / 2^32 + t) / 2^l.
struct Divider { unsigned int m, l, d; };
Divider divider(unsigned int d)
{
    unsigned int l = 0;
    while ((1ull << l) < d) ++l;
    return {(unsigned int)(((1ull << 32) * ((1ull << l) - d)) / d + 1), l, d};
}
__device__ __forceinline__ unsigned int quotient(unsigned int t, const Divider &x) { return (__umulhi(x.m, t) + t) >> x.l; }

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
// Positions of a unit of HW heads, and units of a row for one group of heads and one block.
template <int HW> constexpr int unit_keys() { return kWarps * kWarpKeys / HW; }
template <int HW> __device__ __forceinline__ int tiles_of(int keys) { return (max(keys, 0) + unit_keys<HW>() - 1) / unit_keys<HW>(); }

// CTAs of a grid that own units: each of them has at least one.  (Two to six times as many
// CTAs, for the hardware to even out, gained nothing and made more shares to join: 131071 keys
// 108 -> 122 .. 230 us.)
__device__ __forceinline__ unsigned long long owners_of(unsigned long long total, unsigned long long grid)
{
    return total < grid ? total : grid;
}

// Block-wide: the units of all rows, the most tiles of any (for one `per`), and row b with its first unit: the row asked for
// (row >= 0), or else the one that the first unit of CTA `part` of `parts` belongs to (b = B
// if there is none).  `per` units stand beside each other for every tile of a row (heads).
struct RowAt { int b, keys, most; unsigned long long first, total; };
template <int HW>
__device__ __forceinline__ RowAt find_row(const PagedArgs &a, unsigned long long per, unsigned long long part,
                                          unsigned long long parts, int row)
{
    __shared__ unsigned long long s_sum[kThreads / 32], s_first;
    __shared__ int s_b, s_keys, s_most[kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = (a.B + kThreads - 1) / kThreads, b0 = min(tid * n, a.B), b1 = min(b0 + n, a.B);
    unsigned long long sum = 0;
    int most = 0;
    for (int b = b0; b < b1; ++b) {
        const int tiles = tiles_of<HW>(row_keys(a, b));
        sum += per * (unsigned long long)tiles;
        most = max(most, tiles);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    unsigned long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    if (tid == 0) s_b = a.B;
    if (lane == 31) { s_sum[warp] = inc; s_most[warp] = most; }
    __syncthreads();
    unsigned long long before = inc - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += s_sum[w];
        total += s_sum[w];
        most = max(most, s_most[w]);
    }
    // by row (row >= 0), or by the first unit of part `part` of `parts`
    const unsigned long long at = total ? part * total / owners_of(total, parts) : 0;
    for (int b = b0; b < b1; ++b) {
        const int keys = row_keys(a, b);
        const unsigned long long u = per * (unsigned long long)tiles_of<HW>(keys);
        if (row >= 0 ? b == row : (at >= before && at < before + u)) { s_b = b; s_keys = keys; s_first = before; }
        before += u;
    }
    __syncthreads();
    RowAt r;
    r.b = s_b;
    r.keys = s_keys;
    r.first = s_first;
    r.total = total;
    r.most = most;
    return r;
}

// ---- warp matrix instructions (bf16, fp32 accumulators)
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t saddr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(saddr) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t saddr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(saddr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int D, typename InT, int HG>
struct PagedSmem {
    static constexpr bool mma = sizeof(InT) == 2;
    static constexpr int row = D * (int)sizeof(InT) + 16;                 // bytes; rows 4 banks apart
    static constexpr int slot = 2 * kWarpKeys * row;                      // K rows, then V rows
    static constexpr int ring = kWarps * kStages * slot;
    static constexpr int off_q = ring;                                    // fp32: [warp][HG][D], scaled by scale log2 e
    static constexpr int off_p = off_q + (mma ? 0 : kWarps * HG * D * 4);          // fp32: [warp][HG][16]
    static constexpr int off_ml = off_p + (mma ? 0 : kWarps * HG * kWarpKeys * 4);    // [warp][HG] maximum, sum
    static constexpr int total = off_ml + kWarps * HG * 8;
    static_assert(kWarps * HG * D * 4 <= ring, "the warps' outputs meet in the ring");
};

// CTAs that fit an SM by their shared memory
template <int D, typename InT, int HG>
constexpr int resident() { return 226 * 1024 / (PagedSmem<D, InT, HG>::total + 1024); }

// Whether it pays that CTAs take stretches of whole rows: nothing is left to join then, and no CTA
// empties its pipeline at a row's end inside its share.  It does for many rows and for short ones; for
// few long ones the CTAs share the keys.  With `most` units in the longest row and `units` in
// all, the first form takes about 6 us and a unit's time for every unit of every wave of CTAs, the
// second 12 us, its share of the units, and 14 us for every row that begins in a CTA's share.
// In a graph, us, shared / whole (rows up to L keys, drawn): 32 / 8 heads of 128 bf16: 40 rows, L 200
// 21 / 13; 64 rows, L 1000 56 / 36; 128 rows, L 450 69 / 36, L 3000 173 / 166; 16 rows, L 450 19 / 17, L 2500
// 38 / 56; one row, L 500 12 / 17.  32 / 1 heads of 64 bf16: 16 rows, L 450 15 / 12, L 2500 24 / 33.
// 16 / 16 heads of 64 fp32: 24 rows, L 500 28 / 19; 16 rows, L 2500 57 / 70.  64 / 2 heads of 128
// bf16, where the model is farthest off: 24 rows, L 500 35 / 29 (takes the first).  Over 97 such
// shapes what the host picks is within 1.1 of the better form but for 5 (1.25 at most); with a wide
// table, both forms with the second launch, the device's pick is within 1.1 but for 7 (1.28 at most).
// (In hundredths of a us.)  `launched`: the kernel that joins has been launched, and costs 3 us even
// if it finds nothing to do.
template <int D, typename InT, int HG>
__host__ __device__ __forceinline__ bool whole_rows_pay(unsigned long long stretches, unsigned long long units,
                                                        unsigned long long most, bool launched)
{
    constexpr int R = resident<D, InT, HG>();
    constexpr unsigned long long unit = R == 1 ? 160 : R == 2 ? 62 : 42, places = kSms * R;
    return 600 + (launched ? 300 : 0) + unit * most * ((stretches + places - 1) / places) <=
           1200 + (unit * units + 1400 * stretches) / places;
}

// The running maximum, sum and output of HG query heads over a warp's keys.  Lane's share:
// bf16: heads 2 (lane % 4) + {0, 1} + 8 n of n-tile n; output channels lane / 4 + 8 x;
// fp32: all heads; the sum of key lane (of the first 16), output channels DL lane ...
template <int D, int HG>
struct MmaState {
    static constexpr int NT = HG / 8, KS = D / 16;
    uint32_t q[NT][KS][2];
    float m[NT][2], l[NT][2], o[NT][KS][4];

    __device__ __forceinline__ void start(const __nv_bfloat16 *qh, int nh, int lane)
    {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int head = 8 * n + (lane >> 2);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    q[n][ks][x] = head < nh ? *reinterpret_cast<const uint32_t *>(qh + head * D + 16 * ks + 8 * x + 2 * (lane & 3)) : 0u;
                    o[n][ks][2 * x] = o[n][ks][2 * x + 1] = 0.f;
                }
#pragma unroll
            for (int x = 0; x < 2; ++x) { m[n][x] = -INFINITY; l[n][x] = 0.f; }
        }
    }
    // 16 keys of which `seen` (one bit a key) count; scores in units of log 2 after `scale`
    __device__ __forceinline__ void step(uint32_t k, uint32_t v, int row, unsigned int seen, float scale, int lane)
    {
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) s[n][x] = 0.f;
        const uint32_t ka = k + (uint32_t)(((lane & 7) + 8 * ((lane >> 3) & 1)) * row + 16 * (lane >> 4));
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint32_t a[4];
            ldsm4(ka + 32 * ks, a);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(s[n], a, q[n][ks][0], q[n][ks][1]);
        }
        const bool on0 = (seen >> (lane >> 2)) & 1u, on1 = (seen >> ((lane >> 2) + 8)) & 1u;
        uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float p[4];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float s0 = on0 ? s[n][x] * scale : -INFINITY, s1 = on1 ? s[n][2 + x] * scale : -INFINITY;
                float top = fmaxf(s0, s1);
                if (__any_sync(0xffffffffu, top > m[n][x])) {           // a running maximum rises
#pragma unroll
                    for (int y = 4; y < 32; y <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, y));
                    top = fmaxf(top, m[n][x]);
                    // -inf before and after: no key yet, nothing to rescale
                    const float f = m[n][x] == -INFINITY ? 0.f : exp2f(m[n][x] - top);
                    m[n][x] = top;
                    l[n][x] *= f;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) { o[n][ks][x] *= f; o[n][ks][2 + x] *= f; }
                }
                const float base = m[n][x] == -INFINITY ? 0.f : m[n][x];
                p[x] = on0 ? exp2f(s0 - base) : 0.f;
                p[2 + x] = on1 ? exp2f(s1 - base) : 0.f;
                l[n][x] += p[x] + p[2 + x];
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float p0 = p[2 * x], p1 = p[2 * x + 1];
                const uint32_t h0 = (__float_as_uint(p0) - (p0 > 0.f ? 1u : 0u)) & 0xffff0000u;
                const uint32_t h1 = (__float_as_uint(p1) - (p1 > 0.f ? 1u : 0u)) & 0xffff0000u;
                const __nv_bfloat162 r = __floats2bfloat162_rn(p0 - __uint_as_float(h0), p1 - __uint_as_float(h1));
                hi[n][x] = transpose8x8(__byte_perm(h0, h1, 0x7632));
                lo[n][x] = transpose8x8(*reinterpret_cast<const uint32_t *>(&r));
            }
        }
        const uint32_t va = v + (uint32_t)(((lane & 7) + 8 * (lane >> 4)) * row + 16 * ((lane >> 3) & 1));
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint32_t a[4];
            ldsm4_trans(va + 32 * ks, a);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma16816(o[n][ks], a, hi[n][0], hi[n][1]);
                mma16816(o[n][ks], a, lo[n][0], lo[n][1]);
            }
        }
    }
    __device__ __forceinline__ void finish(float *sO, float *sML, int lane)
    {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int head = 8 * n + 2 * (lane & 3) + x;
#pragma unroll
                for (int y = 4; y < 32; y <<= 1) l[n][x] += __shfl_xor_sync(0xffffffffu, l[n][x], y);
                if (lane < 4) {
                    sML[2 * head] = m[n][x];
                    sML[2 * head + 1] = l[n][x];
                }
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    sO[head * D + 16 * ks + (lane >> 2)] = o[n][ks][x];
                    sO[head * D + 16 * ks + 8 + (lane >> 2)] = o[n][ks][2 + x];
                }
            }
    }
};

template <int D, int HG>
struct SimtState {
    static constexpr int DL = D / 32;
    float m[HG], l[HG], o[HG][DL];

    __device__ __forceinline__ void start()
    {
#pragma unroll
        for (int g = 0; g < HG; ++g) {
            m[g] = -INFINITY;
            l[g] = 0.f;
#pragma unroll
            for (int x = 0; x < DL; ++x) o[g][x] = 0.f;
        }
    }
    __device__ __forceinline__ void step(const uint8_t *k, const uint8_t *v, int row, unsigned int seen, const float *sQ,
                                         float *sP, int lane)
    {
        float s[HG];
#pragma unroll
        for (int g = 0; g < HG; ++g) s[g] = 0.f;
        const float *kr = reinterpret_cast<const float *>(k + (lane & 15) * row) + (lane >> 4) * (D / 2);
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
        const bool on = (seen >> (lane & 15)) & 1u;
#pragma unroll
        for (int g = 0; g < HG; ++g) {
            s[g] += __shfl_xor_sync(0xffffffffu, s[g], 16);
            if (!on) s[g] = -INFINITY;
            if (__any_sync(0xffffffffu, s[g] > m[g])) {         // the running maximum rises
                float top = s[g];
#pragma unroll
                for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                top = fmaxf(top, m[g]);
                const float f = exp2f(m[g] - top);              // exp2(-inf) = 0 the first time
                l[g] *= f;
#pragma unroll
                for (int x = 0; x < DL; ++x) o[g][x] *= f;
                m[g] = top;
            }
            // a maximum of -inf: every score so far is -inf, each weighs nothing
            const float p = on ? exp2f(s[g] - (m[g] == -INFINITY ? 0.f : m[g])) : 0.f;
            if (lane < 16) {
                l[g] += p;
                sP[g * kWarpKeys + lane] = p;
            }
        }
        __syncwarp();
        const uint8_t *vr = v + 4 * DL * lane;
#pragma unroll
        for (int j = 0; j < kWarpKeys; j += 4) {
            float x[4][DL];
#pragma unroll
            for (int jj = 0; jj < 4; ++jj)
#pragma unroll
                for (int y = 0; y < DL; ++y) x[jj][y] = reinterpret_cast<const float *>(vr + (j + jj) * row)[y];
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
    }
    __device__ __forceinline__ void finish(float *sO, float *sML, int lane)
    {
#pragma unroll
        for (int g = 0; g < HG; ++g) {
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) l[g] += __shfl_xor_sync(0xffffffffu, l[g], x);
            if (lane == 0) {
                sML[2 * g] = m[g];
                sML[2 * g + 1] = l[g];
            }
#pragma unroll
            for (int x = 0; x < DL; ++x) sO[g * D + DL * lane + x] = o[g][x];
        }
    }
};

// What the first kernel tells the second, behind the CTAs' slots in the workspace
template <int D, int HG, int HW>
__device__ __forceinline__ int *whole_flag(const PagedArgs &a)
{
    return reinterpret_cast<int *>(a.ws + (size_t)kSms * kMaxResident * 2 * HW * HG * (D + 2));
}

template <int D, typename InT, int HG, int HW>
__global__ void __launch_bounds__(kThreads)
paged_decode_kernel(const __grid_constant__ PagedArgs a, const Divider by_page, const bool all_whole)
{
    using L = PagedSmem<D, InT, HG>;
    constexpr int CPR = D * (int)sizeof(InT) / 16;      // 16-byte pieces of a row
    constexpr int RPI = 32 / CPR;                       // rows that a warp's copy instruction covers
    static_assert(CPR <= 32 && 32 % CPR == 0, "pieces");
    constexpr int TW = kWarps / HW, kTile = unit_keys<HW>();     // warps of a head, positions of a unit
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + (uint32_t)(warp * kStages * L::slot);
    float *sML = reinterpret_cast<float *>(smem + L::off_ml);
    float *sO = reinterpret_cast<float *>(smem);

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const int group = a.H / a.Hkv, blocks = (group + HG - 1) / HG;
    const unsigned long long per = (unsigned long long)(a.Hkv / HW) * blocks;
    // this CTA's units [u, u1), the first of them in row b, whose own begin at row_first
    unsigned long long u = 0, u1 = 0, row_first = 0;
    int b = 0, n = 0, part = 0, tiles = 0;
    const unsigned int stretches = (unsigned int)(a.B * per);
    unsigned int next = blockIdx.x;                     // the stretch to take whole
    bool whole_rows = all_whole;
    if (!all_whole) {
        const RowAt at = find_row<HW>(a, per, blockIdx.x, gridDim.x, -1);
        whole_rows = whole_rows_pay<D, InT, HG>(stretches, at.total, at.most, true);
        if (blockIdx.x == 0 && tid == 0) *whole_flag<D, HG, HW>(a) = whole_rows;
        const unsigned long long owners = owners_of(at.total, gridDim.x);
        if (!whole_rows && blockIdx.x < owners) {
            u = (unsigned long long)blockIdx.x * at.total / owners;
            u1 = ((unsigned long long)blockIdx.x + 1) * at.total / owners;
            b = at.b;
            n = at.keys;
            tiles = tiles_of<HW>(n);
            row_first = at.first;
        }
    }
    do {
        if (whole_rows && next < stretches) {
            const unsigned int hb = next % (unsigned int)per;
            b = next / (unsigned int)per;
            n = row_keys(a, b);
            tiles = tiles_of<HW>(n);
            u = (unsigned long long)hb * tiles;
            u1 = u + tiles;
            if (n == 0) {                                   // no keys: zeros
                const int blk0 = (int)(hb % blocks) * HG, nh = min(HG, group - blk0);
                for (int e = tid; e < HW * nh * D; e += kThreads) {
                    const size_t head = (size_t)b * a.H + (hb / blocks * HW + e / (nh * D)) * group + blk0 + e / D % nh;
                    static_cast<InT *>(a.out)[head * D + e % D] = la_round<InT>(0.f);
                }
            }
            next += gridDim.x;
        }
        while (u < u1) {
            while (u >= row_first + per * tiles) {          // next row that has units
                row_first += per * tiles;
                n = row_keys(a, ++b);
                tiles = tiles_of<HW>(n);
            }
            const int hb = (int)((u - row_first) / tiles);          // (key-value heads, block) of the stretch
            const int hk0 = hb / blocks * HW, blk0 = (hb % blocks) * HG, nh = min(HG, group - blk0);
            const int hk = hk0 + warp / TW;                         // this warp's
            const int tile0 = (int)((u - row_first) % tiles);
            const int tile1 = (int)min((unsigned long long)tiles, (unsigned long long)tile0 + (u1 - u));
            const bool whole = tile0 == 0 && tile1 == tiles;
            const int new_at = a.k ? n - 1 : -1;
            const int *table = a.block_table + (size_t)b * a.max_pages;

            // Page of this lane's key of a unit: key lane % 16 of the warp's 16 (-1: none).
            auto key_of = [&](int tile) { return tile * kTile + (warp % TW) * kWarpKeys + (lane & 15); };
            auto page_of = [&](int tile) {
                const int t = key_of(tile);
                return tile < tile1 && t < n ? table[quotient((unsigned int)t, by_page)] : -1;
            };
            // One slot of this warp's ring; rows that do not count are zeros and nothing is read for
            // them.  Returns a bit for each key that counts.
            auto fetch = [&](int tile, int page) {
                const int t = key_of(tile);
                const bool mine = tile < tile1 && t < n, is_new = mine && t == new_at;
                const bool good = page >= 0 && page < a.num_pages;
                if (mine && !good) atomicOr(&g_paged_status, 1u);
                const bool real = is_new || (mine && good);
                const InT *kp = static_cast<const InT *>(a.k_cache), *vp = static_cast<const InT *>(a.v_cache);
                if (is_new) {
                    kp = static_cast<const InT *>(a.k) + ((size_t)b * a.Hkv + hk) * D;
                    vp = static_cast<const InT *>(a.v) + ((size_t)b * a.Hkv + hk) * D;
                } else if (real) {
                    const size_t off = (((size_t)page * a.page_size + ((unsigned int)t - quotient((unsigned int)t, by_page) * by_page.d)) *
                                            a.Hkv + hk) * D;
                    kp += off;
                    vp += off;
                }
                const unsigned int seen = __ballot_sync(0xffffffffu, real) & 0xffffu;
                const uint32_t dst = ring + (uint32_t)((tile % kStages) * L::slot + (lane / CPR) * L::row + 16 * (lane % CPR));
                const unsigned long long kpi = reinterpret_cast<unsigned long long>(kp) , vpi = reinterpret_cast<unsigned long long>(vp);
#pragma unroll
                for (int e = 0; e < kWarpKeys / RPI; ++e) {
                    const int r = e * RPI + lane / CPR;
                    const bool ok = (seen >> r) & 1u;
                    const unsigned long long ks = __shfl_sync(0xffffffffu, kpi, r), vs = __shfl_sync(0xffffffffu, vpi, r);
                    cp16(dst + (uint32_t)(e * RPI * L::row), reinterpret_cast<const uint8_t *>(ks) + 16 * (lane % CPR), ok);
                    cp16(dst + (uint32_t)((kWarpKeys + e * RPI) * L::row), reinterpret_cast<const uint8_t *>(vs) + 16 * (lane % CPR), ok);
                }
                cp_commit();
                return seen;
            };

            static_assert(kStages == 3, "two units ahead");
            unsigned int seen0 = fetch(tile0, page_of(tile0)), seen1 = fetch(tile0 + 1, page_of(tile0 + 1)), seen2;
            int page2 = page_of(tile0 + 2);
            const InT *qh = static_cast<const InT *>(a.q) + ((size_t)b * a.H + hk * group + blk0) * D;
            if constexpr (L::mma) {
                MmaState<D, HG> st;
                st.start(qh, nh, lane);
                for (int tile = tile0; tile < tile1; ++tile) {
                    seen2 = fetch(tile + 2, page2);
                    page2 = page_of(tile + 3);
                    cp_wait<2>();
                    __syncwarp();
                    const uint32_t k = ring + (uint32_t)((tile % kStages) * L::slot);
                    st.step(k, k + kWarpKeys * L::row, L::row, seen0, a.scale * kLog2e, lane);
                    seen0 = seen1;
                    seen1 = seen2;
                    __syncwarp();                           // the slot is free again
                }
                cp_wait<0>();
                __syncthreads();
                st.finish(sO + warp * HG * D, sML + warp * HG * 2, lane);
            } else {
                float *sQ = reinterpret_cast<float *>(smem + L::off_q) + warp * HG * D;
                float *sP = reinterpret_cast<float *>(smem + L::off_p) + warp * HG * kWarpKeys;
                for (int e = lane; e < HG * D; e += 32) sQ[e] = e / D < nh ? to_f32(qh[e]) * (a.scale * kLog2e) : 0.f;
                __syncwarp();
                SimtState<D, HG> st;
                st.start();
                for (int tile = tile0; tile < tile1; ++tile) {
                    seen2 = fetch(tile + 2, page2);
                    page2 = page_of(tile + 3);
                    cp_wait<2>();
                    __syncwarp();
                    const uint8_t *k = smem + (warp * kStages + tile % kStages) * L::slot;
                    st.step(k, k + kWarpKeys * L::row, L::row, seen0, sQ, sP, lane);
                    seen0 = seen1;
                    seen1 = seen2;
                    __syncwarp();                           // the slot and sP are free again
                }
                cp_wait<0>();
                __syncthreads();
                st.finish(sO + warp * HG * D, sML + warp * HG * 2, lane);
            }
            // ---- the new token's keys and values go to their place in the cache (one owner per head)
            if (new_at >= 0 && blk0 == 0 && new_at / kTile >= tile0 && new_at / kTile < tile1) {
                const unsigned int pi = quotient((unsigned int)new_at, by_page);
                const int page = table[pi];
                if (page >= 0 && page < a.num_pages) {
                    const size_t dst = (((size_t)page * a.page_size + ((unsigned int)new_at - pi * by_page.d)) * a.Hkv + hk0) * D;
                    const size_t src = ((size_t)b * a.Hkv + hk0) * D;
                    for (int e = tid; e < HW * CPR; e += kThreads) {
                        reinterpret_cast<uint4 *>(static_cast<InT *>(a.k_cache) + dst)[e] =
                            reinterpret_cast<const uint4 *>(static_cast<const InT *>(a.k) + src)[e];
                        reinterpret_cast<uint4 *>(static_cast<InT *>(a.v_cache) + dst)[e] =
                            reinterpret_cast<const uint4 *>(static_cast<const InT *>(a.v) + src)[e];
                    }
                }
            }
            // ---- the warps of a head meet
            __syncthreads();
            float *slot = a.ws + ((size_t)blockIdx.x * 2 + (part > 0 ? 1 : 0)) * HW * HG * (D + 2);
            for (int e = tid; e < HW * nh * D; e += kThreads) {
                const int hw = e / (nh * D), g = e / D % nh, d = e % D;
                float top = -INFINITY, sum = 0.f, acc = 0.f;
#pragma unroll
                for (int w = 0; w < TW; ++w) top = fmaxf(top, sML[((hw * TW + w) * HG + g) * 2]);
#pragma unroll
                for (int w = 0; w < TW; ++w) {
                    const int x = (hw * TW + w) * HG + g;
                    const float mw = sML[x * 2], f = mw == -INFINITY ? 0.f : exp2f(mw - top);
                    sum += f * sML[x * 2 + 1];
                    acc += f * sO[x * D + d];
                }
                if (whole) {
                    static_cast<InT *>(a.out)[((size_t)b * a.H + (hk0 + hw) * group + blk0 + g) * D + d] =
                        la_round<InT>(sum == 0.f ? 0.f : acc / sum);     // no weight: zeros; a NaN stays one
                } else {
                    float *mine = slot + hw * HG * (D + 2);
                    mine[g * D + d] = acc;
                    if (d == 0) { mine[HG * D + 2 * g] = top; mine[HG * D + 2 * g + 1] = sum; }
                }
            }
            __syncthreads();                                // sO and sML lie where the next stretch's copies go
            u += (unsigned long long)(tile1 - tile0);
            ++part;
        }
    } while (whole_rows && next < stretches);
}

// One CTA per (row, query head): rows without keys get zeros, and stretches that several CTAs
// share are joined, every fourth share by one warp, in the order of the keys.
template <int D, typename InT, int HG, int HW>
__global__ void __launch_bounds__(kThreads)
paged_join_kernel(const __grid_constant__ PagedArgs a, unsigned int grid)
{
    constexpr int kShares = kSms * kMaxResident;        // owners there can be
    __shared__ float s_acc[kWarps][D], s_sum[kWarps], s_top[kWarps], s_weight[kShares];
    const int group = a.H / a.Hkv, blocks = (group + HG - 1) / HG;
    const unsigned long long per = (unsigned long long)(a.Hkv / HW) * blocks;
    const int b = blockIdx.x / a.H, h = blockIdx.x % a.H;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (*whole_flag<D, HG, HW>(a)) return;              // every row has been written out
    const int n = row_keys(a, b);
    if (n < 0) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    InT *out = static_cast<InT *>(a.out) + (size_t)blockIdx.x * D;
    if (n == 0) {
        if (tid < D) out[tid] = la_round<InT>(0.f);
        return;
    }
    const RowAt at = find_row<HW>(a, per, 0, 1, b);
    const int hk = h / group, g = h % group % HG, hw = hk % HW, hb = hk / HW * blocks + h % group / HG;
    const unsigned long long tiles = (unsigned long long)tiles_of<HW>(n);
    const unsigned long long x0 = at.first + hb * tiles, x1 = x0 + tiles - 1;
    // the CTA that has unit x: the largest c with c U / G <= x (G here: the owners)
    const unsigned long long owners = owners_of(at.total, grid);
    const unsigned int c0 = (unsigned int)(((x0 + 1) * owners - 1) / at.total), c1 = (unsigned int)(((x1 + 1) * owners - 1) / at.total);
    if (c0 == c1) return;                               // written by its only owner
    // the first owner's stretch is its second part if it began with another one
    const unsigned int first_part = (unsigned long long)c0 * at.total / owners < x0 ? 1u : 0u;
    constexpr int DL = D / 32;
    auto share = [&](unsigned int c) {
        return a.ws + (((size_t)c * 2 + (c == c0 ? first_part : 0u)) * HW + hw) * HG * (D + 2);
    };
    // the shares' weights 2^(m_c - m), and the sum
    const int count = (int)(c1 - c0) + 1;
    float top = -INFINITY, sum = 0.f;
    for (int c = tid; c < count; c += kThreads) {
        const float m = share(c0 + c)[HG * D + 2 * g];
        s_weight[c] = m;
        top = fmaxf(top, m);
    }
#pragma unroll
    for (int y = 16; y > 0; y >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, y));
    if (lane == 0) s_top[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_top[w]);
    for (int c = tid; c < count; c += kThreads) {
        const float m = s_weight[c], f = m == -INFINITY ? 0.f : exp2f(m - top);
        s_weight[c] = f;
        sum += f * share(c0 + c)[HG * D + 2 * g + 1];
    }
#pragma unroll
    for (int y = 16; y > 0; y >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, y);
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    // eight shares at a time, so that their loads are under way together
    float acc[DL];
#pragma unroll
    for (int y = 0; y < DL; ++y) acc[y] = 0.f;
    for (int c = warp; c < count; c += 8 * kWarps) {
        float x[8][DL];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float *slot = share(c0 + min(c + i * kWarps, count - 1)) + g * D + lane;
#pragma unroll
            for (int y = 0; y < DL; ++y) x[i][y] = slot[32 * y];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool in = c + i * kWarps < count;     // else the last share's, which may be infinite
            const float f = in ? s_weight[c + i * kWarps] : 0.f;
#pragma unroll
            for (int y = 0; y < DL; ++y) acc[y] += f * (in ? x[i][y] : 0.f);
        }
    }
#pragma unroll
    for (int y = 0; y < DL; ++y) s_acc[warp][lane + 32 * y] = acc[y];
    __syncthreads();
    if (tid < D) {
        float s = 0.f, o = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            s += s_sum[w];
            o += s_acc[w][tid];
        }
        out[tid] = la_round<InT>(s == 0.f ? 0.f : o / s);     // as above
    }
}

// Query heads that share one reading of the cache.  bf16: 8 columns of a product, or two
// times 8 for larger groups (a third would no longer fit the registers); fp32: as many as the
// group has, up to 8.
int heads_per_block(int group, kda_dtype dtype)
{
    if (dtype == KDA_BF16) return group > 8 ? 16 : 8;
    return group > 4 ? 8 : group > 2 ? 4 : group;
}

// Neighbouring key-value heads of a unit.
// Two read 64 ragged rows (8 heads of 128 bf16) in 225 us, one in 228, four in 228; 128 rows of
// 8 heads of 64: 215, 277, 221 us; 131071 keys of one row, where the shares of a head to be
// joined grow with them: 101, 98, 108 us.
int heads_per_unit(int Hkv) { return Hkv % 2 == 0 ? 2 : 1; }

template <int D, typename InT, int HG, int HW>
cudaError_t launch_typed(const PagedArgs &a, cudaStream_t stream)
{
    using L = PagedSmem<D, InT, HG>;
    auto kernel = paged_decode_kernel<D, InT, HG, HW>;
    static OncePerDevice once;
    cudaError_t e = set_shared_memory(kernel, L::total, once);
    if (e != cudaSuccess) return e;
    static_assert(resident<D, InT, HG>() <= kMaxResident, "the workspace holds two stretches per CTA");
    unsigned int grid = kSms * resident<D, InT, HG>();
    // by the table's bounds, which are what the host knows; otherwise the device decides by the lengths
    const unsigned long long stretches = (unsigned long long)a.B * (a.Hkv / HW) * ((a.H / a.Hkv + HG - 1) / HG);
    const unsigned long long most = ((unsigned long long)a.max_pages * a.page_size + unit_keys<HW>() - 1) / unit_keys<HW>();
    const bool whole_rows = whole_rows_pay<D, InT, HG>(stretches, stretches * most, most, false);
    if (whole_rows) grid = (unsigned int)stretches;
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
    if ((e = cudaLaunchKernelEx(&cfg, kernel, a, divider((unsigned int)a.page_size), whole_rows)) != cudaSuccess) return e;
    note_launch();
    if (whole_rows) return cudaGetLastError();
    cfg.gridDim = dim3((unsigned)((size_t)a.B * a.H));
    cfg.dynamicSmemBytes = 0;
    if ((e = cudaLaunchKernelEx(&cfg, paged_join_kernel<D, InT, HG, HW>, a, grid)) != cudaSuccess) return e;
    note_launch();
    return cudaGetLastError();
}

template <int D, typename InT, int HG>
cudaError_t launch_heads(const PagedArgs &a, cudaStream_t stream)
{
    return heads_per_unit(a.Hkv) == 2 ? launch_typed<D, InT, HG, 2>(a, stream) : launch_typed<D, InT, HG, 1>(a, stream);
}

template <int D>
cudaError_t launch_group(const PagedArgs &a, cudaStream_t stream)
{
    const int hg = heads_per_block(a.H / a.Hkv, a.dtype);
    if (a.dtype == KDA_BF16)
        return hg == 16 ? launch_heads<D, __nv_bfloat16, 16>(a, stream) : launch_heads<D, __nv_bfloat16, 8>(a, stream);
    switch (hg) {
    case 1: return launch_heads<D, float, 1>(a, stream);
    case 2: return launch_heads<D, float, 2>(a, stream);
    case 4: return launch_heads<D, float, 4>(a, stream);
    default: return launch_heads<D, float, 8>(a, stream);
    }
}

}  // namespace

size_t paged_workspace_bytes(int H, int Hkv, int D, kda_dtype dtype)
{
    return sizeof(float) * (size_t)kSms * kMaxResident * 2 * heads_per_unit(Hkv) * heads_per_block(H / Hkv, dtype) * (D + 2) + 256;
}

cudaError_t launch_paged_decode(const PagedArgs &a, cudaStream_t stream)
{
    return a.D == 128 ? launch_group<128>(a, stream) : launch_group<64>(a, stream);
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

// Linear attention with one decay per head on the tensor cores (tcgen05): bf16 inputs,
// dk = dv = 128 (the mathematics is in kda_la.cuh).
//
// One CTA walks the chunks of 128 tokens of one (pass, b, h, segment).  Per chunk, with
// accumulators in tensor memory:
//     S = Q K^T                 P = f_intra lambda^|i-j| S on the causal side, as bf16, in place
//     O = Q S0                  rescaled by rows with f_inter lambda^(i+1), then  O += P V
//     U = K'^T V                K' = f_write lambda^(c-1-j) K;  S0 <- lambda^c S0 + U in registers
// Roundings.  Q, K, V enter exactly.  P and the entering state S0 are rounded to bf16 for
// their products: each output is a sum of such terms, so their errors together are of the
// size of the output's own rounding to bf16.  The state that is carried is fp32: K' is
// written as three bf16 parts that hold all 24 bits of the fp32 product, U starts afresh
// every chunk (the tensor core's accumulation is short) and is added in registers, and
// lambda^c is a pair of floats, because its rounding would grow with the number of chunks.
//
// Warps: 0-3 turn S into P, rescale O and write the outputs (a thread is a token); 4-11 make
// K'^T in tensor memory, the two groups of four by turns (ldmatrix transposes the K tile);
// 12-19 carry the state (a thread is a key channel and half of the value columns); 20 moves
// tiles by TMA; 21 issues the products.  Their order, half of U, Q K^T, Q S0, the other half of
// U, P V, gives every hand-over between warps the time of another product.
// Shared memory holds two stages of q, k, v (192 KB) and the state as an operand (32 KB); the
// outputs of a chunk leave through its q tile.  Tiles are two boxes of 64 channels x 128
// tokens in the 128-byte swizzle, which serves as K-major operand (channels contracted) and
// as MN-major operand (tokens contracted) alike.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <mutex>

#include "kda_la.cuh"
#include "kda_tc_ptx.cuh"

namespace kda {

__device__ unsigned int g_la_device_status = 0;

namespace {

using namespace tcx;

constexpr int kC = 128, kD = 128;
constexpr int kRowWarps = 4, kKeyWarps = 8, kStateWarps = 8;
constexpr int kStateWarp0 = kRowWarps + kKeyWarps, kTmaWarp = kStateWarp0 + kStateWarps, kMmaWarp = kTmaWarp + 1;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int kLaunchRegs = 80, kKeyRegs = 64, kStateRegs = 96;
static_assert(kKeyWarps * (kLaunchRegs - kKeyRegs) >= kStateWarps * (kStateRegs - kLaunchRegs), "registers moved");

// shared memory
constexpr uint32_t kHalf = 64 * kC * 2, kTile = 2 * kHalf;        // 16 KB box, 32 KB tile
constexpr uint32_t SM_Q = 0, SM_K = SM_Q + 2 * kTile, SM_V = SM_K + 2 * kTile, SM_S0 = SM_V + 2 * kTile;
constexpr uint32_t SM_WP = SM_S0 + kTile;             // [256] f_intra lambda^(i-j) at i - j + 127, zeros beyond
constexpr uint32_t SM_WK = SM_WP + 256 * 4;           // [2][128] f_write lambda^(.) of a whole and of the ragged chunk
constexpr uint32_t SM_PW = SM_WK + 2 * 128 * 4;       // [129] lambda^n
constexpr uint32_t SM_BAR = SM_PW + 132 * 4;
enum Bar {
    FULL_Q = 0, FULL_K = 2, FULL_V = 4, FREE_K = 6, FREE_V = 8, OUT_READY = 10, KP_READY = 12, KP_FREE = 17,
    S_READY = 22, QS_READY, PV_GO, PV_DONE, O_FREE, U_READY, U_FREE, S0_READY, kBars
};
constexpr uint32_t SM_TMEM = SM_BAR + 8 * kBars;
constexpr uint32_t SM_TOTAL = SM_TMEM + 16;
static_assert(SM_TOTAL <= 227 * 1024, "shared memory of a CTA");

// tensor memory columns
constexpr uint32_t TM_S = 0, TM_P = 0, TM_O = 128, TM_U = 256, TM_KP = 384;
constexpr uint32_t kKpPart = 8, kKpSlot = 3 * kKpPart;         // a slot: 16 tokens x 3 parts
constexpr int kKpSlots = 5;
static_assert(TM_KP + kKpSlots * kKpSlot <= 512 && KP_FREE == KP_READY + kKpSlots && S_READY == KP_FREE + kKpSlots, "slots");

struct LaMaps {
    CUtensorMap q[kLaMaxPasses], k[kLaMaxPasses], v[kLaMaxPasses], out[kLaMaxPasses];
};

__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t lbo)
{
    return smem_desc(saddr, lbo, 1024u) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void *tmap, uint32_t mbar, int c0, int c1, int c2, int c3)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%3, %4, %5, %6}], [%2];"
                 :: "r"(dst), "l"(tmap), "r"(mbar), "r"(c0), "r"(c1), "r"(c2), "r"(c3) : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32])
{
    uint32_t r[32];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                   "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
                   "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr) : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&x);
}

__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// Registers move from the key warps to the state warps, within what the block was launched with.
template <int N> __device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N)); }
template <int N> __device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N)); }

// Four 8 x 8 matrices of 16-bit elements, transposed: thread t gets rows 2 (t % 4) and + 1 of
// column t / 4 of each.
__device__ __forceinline__ void ldmatrix4_trans(uint32_t saddr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(saddr) : "memory");
}
// Sixteen lanes x eight columns: thread t's registers are (lane t / 4, column t % 4), (lane
// t / 4 + 8, same column), then the same four columns on.
__device__ __forceinline__ void tmem_st_16x8(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};"
                 :: "r"(taddr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Two products k w (k a packed pair of bf16) as sums of three bf16 each: the 24 bits of the
// fp32 product cut into 8 + 8 + 8.
__device__ __forceinline__ void cut3(uint32_t k, float2 w, uint32_t &hi, uint32_t &mid, uint32_t &lo)
{
    const float2 x = mul2(make_float2(__uint_as_float(k << 16), __uint_as_float(k & 0xffff0000u)), w);
    const uint32_t x0 = __float_as_uint(x.x), x1 = __float_as_uint(x.y);
    hi = __byte_perm(x0, x1, 0x7632);
    const float2 r = sub2(x, make_float2(__uint_as_float(x0 & 0xffff0000u), __uint_as_float(x1 & 0xffff0000u)));
    const uint32_t r0 = __float_as_uint(r.x), r1 = __float_as_uint(r.y);
    mid = __byte_perm(r0, r1, 0x7632);
    const float2 q = sub2(r, make_float2(__uint_as_float(r0 & 0xffff0000u), __uint_as_float(r1 & 0xffff0000u)));
    lo = __byte_perm(__float_as_uint(q.x), __float_as_uint(q.y), 0x7632);
}

// STATES_ONLY: the segment's own state from zero goes to slot seg + 1 of the workspace; no
// outputs (warps 0-3 idle, no q).
template <bool STATES_ONLY>
__global__ void __launch_bounds__(kThreads, 1)
la_tc_kernel(const __grid_constant__ LaArgs a, const __grid_constant__ LaMaps maps)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sb = (uint32_t)__cvta_generic_to_shared(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nwork = STATES_ONLY ? a.nseg - 1 : a.nseg;
    const int seg = blockIdx.x % nwork;
    const int bh = (blockIdx.x / nwork) % (a.B * a.H);
    const int ip = blockIdx.x / nwork / (a.B * a.H);
    const LaPass &ps = a.pass[ip];
    const int b = bh / a.H, h = bh % a.H, rev = ps.rev;
    int t_lo, t_hi;
    la_segment(seg, a.nseg, a.seg_tokens, a.T, rev, t_lo, t_hi);
    const int n0 = t_lo / kC, nchunks = (t_hi + kC - 1) / kC - n0;
    const int c_last = t_hi - (n0 + nchunks - 1) * kC;          // tokens of the chunk at the segment's end in time
    auto chunk_at = [&](int it) { return n0 + (rev ? nchunks - 1 - it : it); };
    auto tokens_of = [&](int n) { return n == n0 + nchunks - 1 ? c_last : kC; };
    auto bar = [&](int i) { return sb + SM_BAR + 8u * (uint32_t)i; };
    float *slots = a.nseg > 1 ? a.ws + ((size_t)ip * a.B * a.H + bh) * a.nseg * kD * kD : nullptr;

    // ---- set up: barriers, tensor memory, powers of lambda
    float *sWP = reinterpret_cast<float *>(smem + SM_WP), *sWK = reinterpret_cast<float *>(smem + SM_WK);
    float *sPW = reinterpret_cast<float *>(smem + SM_PW);
    if (tid == 0) {
        for (int i = 0; i < kBars; ++i) {
            const int count = (i >= FREE_K && i < FREE_V) ? (STATES_ONLY ? kKeyWarps : kKeyWarps + 1)
                              : (i >= OUT_READY && i < KP_READY) || i == PV_GO || i == O_FREE ? kRowWarps
                              : (i >= KP_READY && i < KP_FREE) ? kKeyWarps / 2
                              : i == U_FREE || i == S0_READY ? kStateWarps : 1;
            mbar_init(bar(i), (uint32_t)count);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(sb + SM_TMEM) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid <= kC) {
        const float p = (float)la_power(a.log_decay, h, tid);
        sPW[tid] = p;
        if (tid < kC) {
            const int up = 127 + tid, down = 127 - tid;         // i - j = tid, and -tid
            sWP[up] = (!rev || tid == 0) ? p * ps.f_intra : 0.f;
            if (tid > 0) sWP[down] = rev ? p * ps.f_intra : 0.f;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid < 2 * kC) {
        const int j = tid & (kC - 1), c = tid < kC ? kC : c_last;
        sWK[tid] = ps.f_write * sPW[rev ? j + 1 : max(c - 1 - j, 0)];
    }
    __syncthreads();
    constexpr uint32_t tm = 0;              // all 512 columns: they begin at 0

    bool ok = true;                         // false: a wait of this role ran out
    auto wait = [&](int i, uint32_t parity) {           // by one thread
        if (ok && !mbar_wait(bar(i), parity & 1u)) {
            ok = false;
            atomicOr(&g_la_device_status, 1u);
        }
        return ok;
    };
    auto wait_warp = [&](int i, uint32_t parity) {      // by a whole warp, with one answer
        return ok = __all_sync(0xffffffffu, wait(i, parity));
    };
    auto arrive_warp = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(i));
    };

    if (warp < kRowWarps) {
        if (!STATES_ONLY) {
            const int i = 32 * warp + lane;
            const uint32_t row = tm + ((uint32_t)(32 * warp) << 16);
            for (int it = 0; it < nchunks; ++it) {
                const int c = tokens_of(chunk_at(it)), st = it & 1;
                // ---- P from S
                if (!wait_warp(S_READY, it)) break;
                tc_fence_after();
#pragma unroll
                for (int cb = 0; cb < 4; ++cb) {
                    uint32_t p[16];
                    if (rev ? cb >= warp : cb <= warp) {
                        float s[32];
                        tmem_ld32(row + TM_S + 32 * cb, s);
                        const float *w = sWP + 127 + i - 32 * cb;
#pragma unroll
                        for (int j = 0; j < 16; ++j) p[j] = pack_bf16(s[2 * j] * w[-2 * j], s[2 * j + 1] * w[-2 * j - 1]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) p[j] = 0u;
                    }
                    tmem_st16u(row + TM_P + 16 * cb, p);
                }
                // ---- O <- f_inter lambda^(.) O
                if (!wait_warp(QS_READY, it)) break;
                tc_fence_after();
                const float f = ps.f_inter * sPW[rev ? max(c - 1 - i, 0) : i + 1];
#pragma unroll
                for (int cb = 0; cb < 8; ++cb) {
                    float o[16];
                    tmem_ld16(row + TM_O + 16 * cb, o);
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] *= f;
                    tmem_st16(row + TM_O + 16 * cb, o);
                }
                tmem_wait_st();
                tc_fence_before();
                arrive_warp(PV_GO);
                // ---- outputs through the q tile
                if (!wait_warp(PV_DONE, it)) break;
                tc_fence_after();
                uint8_t *dst = smem + SM_Q + st * kTile + i * 128;
#pragma unroll
                for (int cb = 0; cb < 4; ++cb) {
                    float o[32];
                    tmem_ld32(row + TM_O + 32 * cb, o);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint4 u = make_uint4(pack_bf16(o[8 * x], o[8 * x + 1]), pack_bf16(o[8 * x + 2], o[8 * x + 3]),
                                                   pack_bf16(o[8 * x + 4], o[8 * x + 5]), pack_bf16(o[8 * x + 6], o[8 * x + 7]));
                        *reinterpret_cast<uint4 *>(dst + (cb >> 1) * kHalf + (((4 * (cb & 1) + x) ^ (i & 7)) << 4)) = u;
                    }
                }
                tc_fence_before();
                proxy_fence();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(O_FREE));
                    mbar_arrive(bar(OUT_READY + st));
                }
            }
        }
    } else if (warp < kStateWarp0) {
        // ---- K'^T: slots of 16 tokens, this group's every second one; 32 key channels a warp
        const int quad = warp & 3, group = (warp - kRowWarps) >> 2;
        const uint32_t row = tm + ((uint32_t)(32 * quad) << 16) + TM_KP;
        int slot = group, use = 0;                              // of the ring: every second one
        reg_dec<kKeyRegs>();
        // ldmatrix: lanes 8 m .. 8 m + 7 name the rows (tokens) of matrix m: tokens 8 (m / 2) ..,
        // channels 8 (m % 2) .. of the 16 of a half-warp; 16-byte pieces swizzled by token % 8
        const int jr = lane & 7, m = lane >> 3, piece = 4 * (quad & 1) + (m & 1);
        const uint32_t kt = sb + SM_K + (quad >> 1) * kHalf + (uint32_t)((16 * group + 8 * (m >> 1) + jr) * 128);
        const uint32_t off0 = (uint32_t)((piece ^ jr) << 4), off1 = (uint32_t)(((piece + 2) ^ jr) << 4);
        for (int it = 0; it < nchunks; ++it) {
            const int st = it & 1;
            const float *wk = sWK + (tokens_of(chunk_at(it)) != kC ? kC : 0) + 16 * group + 2 * (lane & 3);
            if (!wait_warp(FULL_K + st, it >> 1)) break;
#pragma unroll 1
            for (int s4 = 0; s4 < 4; ++s4) {
                const float2 w0 = *reinterpret_cast<const float2 *>(wk + 32 * s4);
                const float2 w1 = *reinterpret_cast<const float2 *>(wk + 32 * s4 + 8);
                const uint32_t src = kt + st * kTile + s4 * (32 * 128);
                uint32_t k0[4], k1[4], hi[8], mid[8], lo[8];
                ldmatrix4_trans(src + off0, k0);
                ldmatrix4_trans(src + off1, k1);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    cut3(k0[e], e < 2 ? w0 : w1, hi[e], mid[e], lo[e]);
                    cut3(k1[e], e < 2 ? w0 : w1, hi[4 + e], mid[4 + e], lo[4 + e]);
                }
                if (use > 0 && !wait_warp(KP_FREE + slot, use - 1)) break;
                tc_fence_after();
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const uint32_t dst = row + ((uint32_t)(4 * e) << 16) + slot * kKpSlot;
                    tmem_st_16x8(dst, hi[e], hi[e + 1], hi[e + 2], hi[e + 3]);
                    tmem_st_16x8(dst + kKpPart, mid[e], mid[e + 1], mid[e + 2], mid[e + 3]);
                    tmem_st_16x8(dst + 2 * kKpPart, lo[e], lo[e + 1], lo[e + 2], lo[e + 3]);
                }
                tmem_wait_st();
                tc_fence_before();
                arrive_warp(KP_READY + slot);
                slot += 2;
                if (slot >= kKpSlots) { slot -= kKpSlots; ++use; }
            }
            if (!ok) break;
            arrive_warp(FREE_K + st);
        }
    } else if (warp < kTmaWarp) {
        // ---- the state: key channel r, value columns 64 part ..
        const int quad = warp & 3, part = (warp - kStateWarp0) >> 2;
        const int r = 32 * quad + lane;
        const uint32_t row = tm + ((uint32_t)(32 * quad) << 16) + TM_U + 64 * part;
        reg_inc<kStateRegs>();
        float S[64];
        {
            const float *s0 = STATES_ONLY ? nullptr : slots ? slots + (size_t)seg * kD * kD
                              : ps.s0 ? ps.s0 + (size_t)bh * kD * kD : nullptr;
            if (!s0) {
#pragma unroll
                for (int x = 0; x < 64; ++x) S[x] = 0.f;
            } else if (!slots && ps.s0_transposed) {
#pragma unroll
                for (int x = 0; x < 64; ++x) S[x] = s0[(64 * part + x) * kD + r];
            } else {
#pragma unroll
                for (int x = 0; x < 64; x += 4)
                    *reinterpret_cast<float4 *>(&S[x]) = *reinterpret_cast<const float4 *>(s0 + r * kD + 64 * part + x);
            }
        }
        uint8_t *sS0 = smem + SM_S0 + part * kHalf + r * 128;
        auto publish = [&] {                                    // the state as the operand of Q S0
#pragma unroll
            for (int x = 0; x < 8; ++x)
                *reinterpret_cast<uint4 *>(sS0 + ((x ^ (r & 7)) << 4)) =
                    make_uint4(pack_bf16(S[8 * x], S[8 * x + 1]), pack_bf16(S[8 * x + 2], S[8 * x + 3]),
                               pack_bf16(S[8 * x + 4], S[8 * x + 5]), pack_bf16(S[8 * x + 6], S[8 * x + 7]));
            proxy_fence();
            arrive_warp(S0_READY);
        };
        if (!STATES_ONLY) publish();
        const double whole = la_power(a.log_decay, h, kC), ragged = la_power(a.log_decay, h, c_last);
        const float2 l_whole = make_float2((float)whole, (float)(whole - (double)(float)whole));
        const float2 l_ragged = make_float2((float)ragged, (float)(ragged - (double)(float)ragged));
        for (int it = 0; it < nchunks; ++it) {
            // S <- lambda^c S + U
            if (!wait_warp(U_READY, it)) break;
            tc_fence_after();
            const float2 l = tokens_of(chunk_at(it)) != kC ? l_ragged : l_whole;
            const float2 lh = make_float2(l.x, l.x), ll = make_float2(l.y, l.y);
#pragma unroll
            for (int x = 0; x < 64; x += 16) {
                float u[16];
                tmem_ld16(row + x, u);
#pragma unroll
                for (int y = 0; y < 16; y += 2) {
                    const float2 s = make_float2(S[x + y], S[x + y + 1]);
                    const float2 n = fma2(lh, s, fma2(ll, s, make_float2(u[y], u[y + 1])));
                    S[x + y] = n.x;
                    S[x + y + 1] = n.y;
                }
            }
            tc_fence_before();
            arrive_warp(U_FREE);
            if (!STATES_ONLY && it + 1 < nchunks) {
                if (!wait_warp(QS_READY, it)) break;            // the operand of this chunk has been read
                publish();
            }
        }
        float *dst = STATES_ONLY ? slots + (size_t)(seg + 1) * kD * kD
                     : (seg == a.nseg - 1 && ps.sT) ? ps.sT + (size_t)bh * kD * kD : nullptr;
        if (dst && ok)
#pragma unroll
            for (int x = 0; x < 64; x += 4)
                *reinterpret_cast<float4 *>(dst + r * kD + 64 * part + x) = *reinterpret_cast<const float4 *>(&S[x]);
    } else if (warp == kTmaWarp) {
        if (lane == 0) {
            auto load = [&](const CUtensorMap *m, uint32_t dst, int full, int n) {
                mbar_expect_tx(bar(full), kTile);
                tma_load_4d(dst, m, bar(full), 0, h, n * kC, b);
                tma_load_4d(dst + kHalf, m, bar(full), 64, h, n * kC, b);
            };
            int issued = 0;
            for (int it = 0; it < nchunks; ++it) {
                const int n = chunk_at(it), st = it & 1;
                if (it >= 2 && !wait(FREE_K + st, (it >> 1) - 1)) break;
                load(&maps.k[ip], sb + SM_K + st * kTile, FULL_K + st, n);
                if (!STATES_ONLY && it < 2) load(&maps.q[ip], sb + SM_Q + st * kTile, FULL_Q + st, n);
                if (it >= 2 && !wait(FREE_V + st, (it >> 1) - 1)) break;
                load(&maps.v[ip], sb + SM_V + st * kTile, FULL_V + st, n);
                issued = it + 1;
                if (!STATES_ONLY && it >= 2) {
                    // the outputs of chunk it - 2 leave the q tile, then it is loaded again
                    if (!wait(OUT_READY + st, (it >> 1) - 1)) break;
                    const int t = chunk_at(it - 2) * kC;
                    tma_store_4d(&maps.out[ip], sb + SM_Q + st * kTile, 0, h, t, b);
                    tma_store_4d(&maps.out[ip], sb + SM_Q + st * kTile + kHalf, 64, h, t, b);
                    bulk_commit();
                    bulk_wait_read();
                    load(&maps.q[ip], sb + SM_Q + st * kTile, FULL_Q + st, n);
                }
            }
            if (!STATES_ONLY)
                for (int it = max(nchunks - 2, 0); it < nchunks && ok; ++it) {
                    const int st = it & 1, t = chunk_at(it) * kC;
                    if (!wait(OUT_READY + st, it >> 1)) break;
                    tma_store_4d(&maps.out[ip], sb + SM_Q + st * kTile, 0, h, t, b);
                    tma_store_4d(&maps.out[ip], sb + SM_Q + st * kTile + kHalf, 64, h, t, b);
                    bulk_commit();
                }
            bulk_wait_read();
            if (!ok)                        // no copy may land after the CTA has left
                for (int it = max(issued - 2, 0); it < issued; ++it) {
                    mbar_wait(bar(FULL_K + (it & 1)), (it >> 1) & 1);
                    mbar_wait(bar(FULL_V + (it & 1)), (it >> 1) & 1);
                    if (!STATES_ONLY) mbar_wait(bar(FULL_Q + (it & 1)), (it >> 1) & 1);
                }
        }
    } else {
        // The whole warp walks the loop and one elected lane issues, so that descriptors stay in
        // uniform registers: under `lane == 0` each product took 100 cycles to issue, against
        // the 64 it runs.
        constexpr uint32_t id_nt = idesc_bf16(128, 128, 0, 0), id_nn = idesc_bf16(128, 128, 0, 1);
        const uint64_t dq = desc_sw128(sb + SM_Q, 16), dk = desc_sw128(sb + SM_K, 16), dv = desc_sw128(sb + SM_V, kHalf);
        const uint64_t ds = desc_sw128(sb + SM_S0, kHalf);
        // A K step of 16 channels is 32 bytes inside the swizzled rows of a K-major tile, 16 rows
        // of an MN-major one (addresses in 16 bytes).
        auto k_major = [](int ks) { return (uint64_t)((ks >> 2) * (kHalf >> 4) + (ks & 3) * 2); };
        int slot = 0, use = 0;
        // U (+)= K'^T V over 64 tokens: a K step of three parts per slot
        auto update = [&](uint64_t v, int half) {
#pragma unroll
            for (int ks = 4 * half; ks < 4 * half + 4; ++ks) {
                if (!wait_warp(KP_READY + slot, use)) return false;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int p = 0; p < 3; ++p)
                        umma_bf16_ta(tm + TM_U, tm + TM_KP + slot * kKpSlot + p * kKpPart, v + (uint64_t)(ks * 128), id_nn,
                                     ks > 0 || p > 0);
                    umma_commit(bar(KP_FREE + slot));
                    if (ks == 7) umma_commit(bar(U_READY));
                }
                if (++slot == kKpSlots) { slot = 0; ++use; }
            }
            return true;
        };
        for (int it = 0; it < nchunks; ++it) {
            const int st = it & 1;
            const uint64_t q = dq + (uint64_t)(st * (kTile >> 4)), k = dk + (uint64_t)(st * (kTile >> 4));
            const uint64_t v = dv + (uint64_t)(st * (kTile >> 4));
            if (!wait_warp(FULL_V + st, it >> 1)) break;
            if (it > 0 && !wait_warp(U_FREE, it - 1)) break;
            if (!update(v, 0)) break;
            if (!STATES_ONLY) {
                // S = Q K^T
                if (!wait_warp(FULL_Q + st, it >> 1) || !wait_warp(FULL_K + st, it >> 1)) break;
                if (it > 0 && !wait_warp(PV_DONE, it - 1)) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) umma_bf16(tm + TM_S, q + k_major(ks), k + k_major(ks), id_nt, ks > 0);
                    umma_commit(bar(S_READY));
                    umma_commit(bar(FREE_K + st));
                }
                // O = Q S0
                if (!wait_warp(S0_READY, it) || (it > 0 && !wait_warp(O_FREE, it - 1))) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) umma_bf16(tm + TM_O, q + k_major(ks), ds + (uint64_t)(ks * 128), id_nn, ks > 0);
                    umma_commit(bar(QS_READY));
                }
            }
            if (!update(v, 1)) break;
            if (!STATES_ONLY) {
                // O += P V
                if (!wait_warp(PV_GO, it)) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        umma_bf16_ta(tm + TM_O, tm + TM_P + 8 * ks, v + (uint64_t)(ks * 128), id_nn, 1);
                    umma_commit(bar(PV_DONE));
                    umma_commit(bar(FREE_V + st));
                }
            } else if (elect_one()) umma_commit(bar(FREE_V + st));
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" :: "r"(tm));
}

// cuTensorMapEncodeTiled from the driver, looked up once (the library links the CUDA
// runtime statically and not the driver library)
PFN_cuTensorMapEncodeTiled_v12000 map_encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        else
            cudaGetLastError();
    });
    return fn;
}

// A [B, T, H, 128] bf16 tensor as (channel, head, token, batch), boxes of one head's 64
// channels x 128 tokens.  The token axis has its own bound: rows behind a sequence's end are
// read as zeros and not written.
cudaError_t token_map(const LaArgs &a, const void *p, CUtensorMap *m)
{
    const PFN_cuTensorMapEncodeTiled_v12000 enc = map_encoder();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t row = (cuuint64_t)a.H * kD * 2u;
    const cuuint64_t dims[4] = {(cuuint64_t)kD, (cuuint64_t)a.H, (cuuint64_t)a.T, (cuuint64_t)a.B};
    const cuuint64_t strides[3] = {(cuuint64_t)kD * 2u, row, row * (cuuint64_t)a.T};
    const cuuint32_t box[4] = {64u, 1u, (cuuint32_t)kC, 1u};
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

bool la_tc_supported(int dk, int dv, kda_dtype dtype) { return dtype == KDA_BF16 && dk == kD && dv == kD; }

cudaError_t launch_la_tc(const LaArgs &a, bool states_only, cudaStream_t stream)
{
    LaMaps maps;
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < a.npass && e == cudaSuccess; ++i) {
        e = token_map(a, a.pass[i].k, &maps.k[i]);
        if (e == cudaSuccess) e = token_map(a, a.pass[i].v, &maps.v[i]);
        if (e == cudaSuccess && !states_only) e = token_map(a, a.pass[i].q, &maps.q[i]);
        if (e == cudaSuccess && !states_only) e = token_map(a, a.pass[i].out, &maps.out[i]);
    }
    if (e != cudaSuccess) return e;
    auto kernel = states_only ? la_tc_kernel<true> : la_tc_kernel<false>;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SM_TOTAL)) != cudaSuccess)
        return e;
    // the move of registers between warps is sized for this many: with fewer it would wait for ever
    cudaFuncAttributes attr;
    if ((e = cudaFuncGetAttributes(&attr, kernel)) != cudaSuccess) return e;
    if (attr.numRegs != kLaunchRegs) return cudaErrorInvalidKernelImage;
    const size_t grid = (size_t)a.npass * a.B * a.H * (states_only ? a.nseg - 1 : a.nseg);
    kernel<<<(unsigned)grid, kThreads, SM_TOTAL, stream>>>(a, maps);
    e = cudaGetLastError();
    if (e == cudaSuccess) note_launch();
    return e;
}

cudaError_t take_la_device_status(unsigned int *status)
{
    cudaError_t e = cudaMemcpyFromSymbol(status, g_la_device_status, sizeof(*status));
    if (e == cudaSuccess && *status) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_la_device_status, &zero, sizeof(zero));
    }
    return e;
}

}  // namespace kda

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
// The third part is left out where it cannot be seen: two parts are off by at most 2^-17 of a
// term, so they do for a state that only enters bf16 products, and for terms that fade to
// less than 2^-6 of their size before the state is written out (their errors to 2^-23).  The
// kernel runs into the power limit (1.5 of 1.97 GHz at B4 H32 T16384, 980 W), and U is half
// of its products.
//
// Warps: 0-3 turn S into P, rescale O and write the outputs (a thread is a token); 4-11 make
// K'^T in tensor memory, the two groups of four by turns (ldmatrix transposes the K tile);
// 12-19 carry the state (a thread is a key channel and half of the value columns); 20 moves
// tiles by TMA; 21 issues Q K^T, Q S0 and P V, 22 the steps of U: a wait and an issue take a
// warp about as long as the tensor core takes for a step, so one warp for all of them would
// leave it idle half of the time (B4 H32 T16384: 452 us with one, LAT2 us with two).
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
constexpr int kStateWarp0 = kRowWarps + kKeyWarps, kTmaWarp = kStateWarp0 + kStateWarps, kMmaWarp = kTmaWarp + 1, kUpdateWarp = kMmaWarp + 1;
constexpr int kThreads = 32 * (kUpdateWarp + 1);
constexpr int kLaunchRegs = 80, kKeyRegs = 56, kStateRegs = 104;
static_assert(kKeyWarps * (kLaunchRegs - kKeyRegs) >= kStateWarps * (kStateRegs - kLaunchRegs), "registers moved");

// shared memory
constexpr uint32_t kHalf = 64 * kC * 2, kTile = 2 * kHalf;        // 16 KB box, 32 KB tile
constexpr uint32_t SM_Q = 0, SM_K = SM_Q + 2 * kTile, SM_V = SM_K + 2 * kTile, SM_S0 = SM_V + 2 * kTile;
constexpr uint32_t SM_WP = SM_S0 + kTile;             // [256] f_intra lambda^(i-j) at i - j + 127, zeros beyond
constexpr uint32_t SM_WK = SM_WP + 256 * 4;           // [2][128] f_write lambda^(.) of a whole and of the ragged chunk
constexpr uint32_t SM_PW = SM_WK + 2 * 128 * 4;       // [129] lambda^n
constexpr uint32_t SM_LC = SM_PW + 132 * 4;           // [2] lambda^c of a whole and of the ragged chunk, two floats each
constexpr uint32_t SM_BAR = SM_LC + 16;
constexpr int kKpSlots = 5, kKpSlotsStates = 10;       // slots of K', of the two kernels
enum Bar {
    FULL_Q = 0, FULL_K = 2, FULL_V = 4, FREE_K = 6, FREE_V = 8, OUT_READY = 10, U_READY = 12, U_FREE = 14,
    KP_READY = 16, KP_FREE = KP_READY + kKpSlotsStates, S_READY = KP_FREE + kKpSlotsStates, QS_READY, PV_GO, PV_DONE,
    O_FREE, S0_READY, kBars
};
constexpr uint32_t SM_TMEM = SM_BAR + 8 * kBars;
constexpr uint32_t SM_TOTAL = SM_TMEM + 16;
static_assert(SM_TOTAL <= 227 * 1024, "shared memory of a CTA");

// Tensor memory columns.  Without outputs, S and O make room for five more slots of K' and a
// second U, so that a chunk's U is computed while the one before is added to the state.
constexpr uint32_t TM_S = 0, TM_P = 0, TM_O = 128, TM_U = 256, TM_KP = 384;
constexpr uint32_t kKpPart = 8, kKpSlot = 3 * kKpPart;         // a slot: 16 tokens x 3 parts
static_assert(TM_KP + kKpSlots * kKpSlot <= 512 && (kKpSlotsStates - kKpSlots) * kKpSlot <= TM_O, "slots");
__device__ __forceinline__ uint32_t kp_column(int slot)
{
    return slot < kKpSlots ? TM_KP + kKpSlot * (uint32_t)slot : TM_S + kKpSlot * (uint32_t)(slot - kKpSlots);
}

struct LaMaps {
    CUtensorMap q[kLaMaxPasses], k[kLaMaxPasses], v[kLaMaxPasses], out[kLaMaxPasses];
};

// Descriptors of 128-byte-swizzled tiles whose 8-row groups are 1024 bytes apart, in two
// words: the lower one holds the address (in 16 bytes, so that steps are added to it) and the
// leading stride, the upper one is the same for all of them.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | ((lbo >> 4) << 16); }
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool acc)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0;\n\t"
                 "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}\n"
                 :: "r"(d), "r"(a_lo), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"((uint32_t)acc) : "memory");
}
// A in tensor memory
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, bool acc)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\t"
                 "mov.b64 b, {%2, %3};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}\n"
                 :: "r"(d), "r"(a_tmem), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"((uint32_t)acc) : "memory");
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

__device__ __forceinline__ void st_shared16(uint32_t saddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" :: "r"(saddr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8])
{
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr) : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
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

// Two products k w (k a packed pair of bf16) in fp32.
__device__ __forceinline__ float2 scale_pair(uint32_t k, float2 w)
{
    return mul2(make_float2(__uint_as_float(k << 16), __uint_as_float(k & 0xffff0000u)), w);
}
// x as the sum of three bf16: its 24 bits cut into 8 + 8 + 8.
__device__ __forceinline__ void cut3(float2 x, uint32_t &hi, uint32_t &mid, uint32_t &lo)
{
    const uint32_t x0 = __float_as_uint(x.x), x1 = __float_as_uint(x.y);
    hi = __byte_perm(x0, x1, 0x7632);
    const float2 r = sub2(x, make_float2(__uint_as_float(x0 & 0xffff0000u), __uint_as_float(x1 & 0xffff0000u)));
    const uint32_t r0 = __float_as_uint(r.x), r1 = __float_as_uint(r.y);
    mid = __byte_perm(r0, r1, 0x7632);
    const float2 q = sub2(r, make_float2(__uint_as_float(r0 & 0xffff0000u), __uint_as_float(r1 & 0xffff0000u)));
    lo = __byte_perm(__float_as_uint(q.x), __float_as_uint(q.y), 0x7632);
}

// What a CTA works on.
struct Item { int seg, bh, ip; };
__device__ __forceinline__ Item item_at(const LaArgs &a, bool states_only, unsigned int id)
{
    const unsigned int nwork = states_only ? a.nseg - 1 : a.nseg, heads = a.B * a.H;
    return {(int)(id % nwork), (int)((id / nwork) % heads), (int)(id / nwork / heads)};
}
__device__ __forceinline__ float *state_slot(const LaArgs &a, const Item &x, int seg)
{
    return a.ws + (((size_t)x.ip * a.B * a.H + x.bh) * a.nseg + seg) * kD * kD;
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
    const Item item = item_at(a, STATES_ONLY, blockIdx.x);
    const int seg = item.seg, bh = item.bh, ip = item.ip;
    const LaPass &ps = a.pass[ip];
    const int b = bh / a.H, h = bh % a.H, rev = ps.rev;
    int t_lo, t_hi;
    la_segment(seg, a.nseg, a.seg_tokens, a.T, rev, t_lo, t_hi);
    const int n0 = t_lo / kC, nchunks = (t_hi + kC - 1) / kC - n0;
    const int c_last = t_hi - (n0 + nchunks - 1) * kC;          // tokens of the chunk at the segment's end in time
    auto chunk_at = [&](int it) { return n0 + (rev ? nchunks - 1 - it : it); };
    auto bar = [&](int i) { return sb + SM_BAR + 8u * (uint32_t)i; };
    // steps of the walk from three_at on keep all three parts of K'
    int three_at = 0;
    if (a.log_decay) {
        const float fade = 6.f / (-1.4426950408889634f * a.log_decay[h]);       // tokens to 2^-6 (inf: never)
        three_at = fade >= 0.f && fade < (float)(nchunks * kC) ? max(0, nchunks - 1 - (int)(fade / kC) - 1) : 0;
    }
    if (!STATES_ONLY && (seg != a.nseg - 1 || !ps.sT)) three_at = nchunks;
    const int tail_at = c_last == kC ? -1 : rev ? 0 : nchunks - 1;      // the walk's step that is the ragged chunk

    // ---- set up: barriers, tensor memory, powers of lambda
    float *sWP = reinterpret_cast<float *>(smem + SM_WP), *sWK = reinterpret_cast<float *>(smem + SM_WK);
    float *sPW = reinterpret_cast<float *>(smem + SM_PW);
    if (tid == 0) {
        for (int i = 0; i < kBars; ++i) {
            const int count = (i >= FREE_K && i < FREE_V) ? (STATES_ONLY ? kKeyWarps : kKeyWarps + 1)
                              : (i >= FREE_V && i < OUT_READY) ? (STATES_ONLY ? 1 : 2)
                              : (i >= OUT_READY && i < U_READY) || i == PV_GO || i == O_FREE ? kRowWarps
                              : (i >= KP_READY && i < KP_FREE) ? kKeyWarps / 2
                              : (i >= U_FREE && i < KP_READY) || i == S0_READY ? kStateWarps : 1;
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
    if (tid >= 2 * kC && tid < 2 * kC + 2) {
        const double l = la_power(a.log_decay, h, tid == 2 * kC ? kC : c_last);
        reinterpret_cast<float2 *>(smem + SM_LC)[tid - 2 * kC] = make_float2((float)l, (float)(l - (double)(float)l));
    }
    if (tid < 2 * kC) {
        const int j = tid & (kC - 1), c = tid < kC ? kC : c_last;
        sWK[tid] = ps.f_write * sPW[rev ? j + 1 : max(c - 1 - j, 0)];
    }
    __syncthreads();
    constexpr int kSlots = STATES_ONLY ? kKpSlotsStates : kKpSlots;
    constexpr uint32_t tm = 0;              // all 512 columns: they begin at 0
    constexpr uint32_t id_nt = idesc_bf16(128, 128, 0, 0), id_nn = idesc_bf16(128, 128, 0, 1);

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
                const int c = it == tail_at ? c_last : kC, st = it & 1;
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
                const uint32_t dst = sb + SM_Q + (uint32_t)(st * kTile + i * 128);
#pragma unroll
                for (int cb = 0; cb < 4; ++cb) {
                    float o[32];
                    tmem_ld32(row + TM_O + 32 * cb, o);
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        st_shared16(dst + (cb >> 1) * kHalf + (uint32_t)(((4 * (cb & 1) + x) ^ (i & 7)) << 4),
                                    pack_bf16(o[8 * x], o[8 * x + 1]), pack_bf16(o[8 * x + 2], o[8 * x + 3]),
                                    pack_bf16(o[8 * x + 4], o[8 * x + 5]), pack_bf16(o[8 * x + 6], o[8 * x + 7]));
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
        const uint32_t row = tm + ((uint32_t)(32 * quad) << 16);
        int slot = group, use = 0;                              // of the ring: every second one
        reg_dec<kKeyRegs>();
        // ldmatrix: lanes 8 m .. 8 m + 7 name the rows (tokens) of matrix m: tokens 8 (m / 2) ..,
        // channels 8 (m % 2) .. of the 16 of a half-warp; 16-byte pieces swizzled by token % 8
        const int jr = lane & 7, m = lane >> 3, piece = 4 * (quad & 1) + (m & 1);
        const uint32_t kt = sb + SM_K + (quad >> 1) * kHalf + (uint32_t)((16 * group + 8 * (m >> 1) + jr) * 128);
        const uint32_t off0 = (uint32_t)((piece ^ jr) << 4), off1 = (uint32_t)(((piece + 2) ^ jr) << 4);
        for (int it = 0; it < nchunks; ++it) {
            const int st = it & 1;
            const float *wk = sWK + (it == tail_at ? kC : 0) + 16 * group + 2 * (lane & 3);
            if (!wait_warp(FULL_K + st, it >> 1)) break;
#pragma unroll 1
            for (int s4 = 0; s4 < 4; ++s4) {
                const float2 w0 = *reinterpret_cast<const float2 *>(wk + 32 * s4);
                const float2 w1 = *reinterpret_cast<const float2 *>(wk + 32 * s4 + 8);
                const uint32_t src = kt + st * kTile + s4 * (32 * 128);
                uint32_t k0[4], k1[4], hi[8], mid[8], lo[8];
                ldmatrix4_trans(src + off0, k0);
                ldmatrix4_trans(src + off1, k1);
                const bool three = it >= three_at;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 x = scale_pair(e < 4 ? k0[e & 3] : k1[e & 3], (e & 2) ? w1 : w0);
                    if (three) cut3(x, hi[e], mid[e], lo[e]);
                    else split_pair2(x, hi[e], mid[e]);
                }
                if (use > 0 && !wait_warp(KP_FREE + slot, use - 1)) break;
                tc_fence_after();
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const uint32_t dst = row + ((uint32_t)(4 * e) << 16) + kp_column(slot);
                    tmem_st_16x8(dst, hi[e], hi[e + 1], hi[e + 2], hi[e + 3]);
                    tmem_st_16x8(dst + kKpPart, mid[e], mid[e + 1], mid[e + 2], mid[e + 3]);
                    if (three) tmem_st_16x8(dst + 2 * kKpPart, lo[e], lo[e + 1], lo[e + 2], lo[e + 3]);
                }
                tmem_wait_st();
                tc_fence_before();
                arrive_warp(KP_READY + slot);
                slot += 2;
                if (slot >= kSlots) { slot -= kSlots; ++use; }
            }
            if (!ok) break;
            arrive_warp(FREE_K + st);
        }
    } else if (warp < kTmaWarp) {
        // ---- the state: key channel r, value columns 64 part ..
        const int quad = warp & 3, part = (warp - kStateWarp0) >> 2;
        const int r = 32 * quad + lane;
        const uint32_t row = tm + ((uint32_t)(32 * quad) << 16) + 64 * part;
        reg_inc<kStateRegs>();
        float S[64];
        {
            const float *s0 = STATES_ONLY ? nullptr : a.nseg > 1 ? state_slot(a, item, seg)
                              : ps.s0 ? ps.s0 + (size_t)bh * kD * kD : nullptr;
            if (!s0) {
#pragma unroll
                for (int x = 0; x < 64; ++x) S[x] = 0.f;
            } else if (a.nseg == 1 && ps.s0_transposed) {
#pragma unroll
                for (int x = 0; x < 64; ++x) S[x] = s0[(64 * part + x) * kD + r];
            } else {
#pragma unroll
                for (int x = 0; x < 64; x += 4) {
                    const float4 u = *reinterpret_cast<const float4 *>(s0 + r * kD + 64 * part + x);
                    S[x] = u.x; S[x + 1] = u.y; S[x + 2] = u.z; S[x + 3] = u.w;
                }
            }
        }
        const uint32_t s0_row = sb + SM_S0 + part * kHalf + (uint32_t)(r * 128), s0_swz = (uint32_t)(r & 7) << 4;
        auto publish = [&] {                                    // the state as the operand of Q S0
#pragma unroll
            for (int x = 0; x < 8; ++x)
                st_shared16(s0_row + ((16u * (uint32_t)x) ^ s0_swz), pack_bf16(S[8 * x], S[8 * x + 1]),
                            pack_bf16(S[8 * x + 2], S[8 * x + 3]), pack_bf16(S[8 * x + 4], S[8 * x + 5]),
                            pack_bf16(S[8 * x + 6], S[8 * x + 7]));
            proxy_fence();
            arrive_warp(S0_READY);
        };
        if (!STATES_ONLY) publish();
        for (int it = 0; it < nchunks; ++it) {
            // S <- lambda^c S + U
            const int ub = STATES_ONLY ? it & 1 : 0;
            if (!wait_warp(U_READY + ub, STATES_ONLY ? it >> 1 : it)) break;
            tc_fence_after();
            const float2 l = reinterpret_cast<const float2 *>(smem + SM_LC)[it == tail_at];
#pragma unroll
            for (int x = 0; x < 64; x += 8) {
                float u[8];
                tmem_ld8(row + (ub ? TM_O : TM_U) + x, u);
#pragma unroll
                for (int y = 0; y < 8; ++y) S[x + y] = fmaf(l.x, S[x + y], fmaf(l.y, S[x + y], u[y]));
            }
            tc_fence_before();
            arrive_warp(U_FREE + ub);
            if (!STATES_ONLY && it + 1 < nchunks) {
                if (!wait_warp(QS_READY, it)) break;            // the operand of this chunk has been read
                publish();
            }
        }
        unsigned int id;                        // read again: the loop has no register for what follows from it
        asm volatile("mov.u32 %0, %%ctaid.x;" : "=r"(id));
        const Item end = item_at(a, STATES_ONLY, id);
        float *dst = STATES_ONLY ? state_slot(a, end, end.seg + 1)
                     : (end.seg == a.nseg - 1 && a.pass[end.ip].sT) ? a.pass[end.ip].sT + (size_t)end.bh * kD * kD : nullptr;
        if (dst && ok)
#pragma unroll
            for (int x = 0; x < 64; x += 4)
                *reinterpret_cast<float4 *>(dst + r * kD + 64 * part + x) = make_float4(S[x], S[x + 1], S[x + 2], S[x + 3]);
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
    } else if (warp == kMmaWarp) {
        // Whole warps walk the loops and one elected lane issues, so that descriptors stay in
        // uniform registers: under `lane == 0` each product took 100 cycles to issue, against
        // the 64 it runs.
        if (!STATES_ONLY) {
            const uint32_t dq = desc_lo(sb + SM_Q, 16), dk = desc_lo(sb + SM_K, 16);
            const uint32_t dv = desc_lo(sb + SM_V, kHalf), ds = desc_lo(sb + SM_S0, kHalf);
            // A K step of 16 channels is 32 bytes inside the swizzled rows of a K-major tile, 16
            // rows of an MN-major one (addresses in 16 bytes).
            auto k_major = [](int ks) { return (uint32_t)((ks >> 2) * (kHalf >> 4) + (ks & 3) * 2); };
            for (int it = 0; it < nchunks; ++it) {
                const int st = it & 1;
                const uint32_t stage = (uint32_t)st * (kTile >> 4);
                // S = Q K^T
                if (!wait_warp(FULL_Q + st, it >> 1) || !wait_warp(FULL_K + st, it >> 1)) break;
                if (it > 0 && !wait_warp(PV_DONE, it - 1)) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        umma_ss(tm + TM_S, dq + stage + k_major(ks), dk + stage + k_major(ks), id_nt, ks > 0);
                    umma_commit(bar(S_READY));
                    umma_commit(bar(FREE_K + st));
                }
                // O = Q S0
                if (!wait_warp(S0_READY, it) || (it > 0 && !wait_warp(O_FREE, it - 1))) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        umma_ss(tm + TM_O, dq + stage + k_major(ks), ds + (uint32_t)(ks * 128), id_nn, ks > 0);
                    umma_commit(bar(QS_READY));
                }
                // O += P V
                if (!wait_warp(FULL_V + st, it >> 1) || !wait_warp(PV_GO, it)) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        umma_ts(tm + TM_O, tm + TM_P + 8 * ks, dv + stage + (uint32_t)(ks * 128), id_nn, true);
                    umma_commit(bar(PV_DONE));
                    umma_commit(bar(FREE_V + st));
                }
            }
        }
    } else {
        // U = K'^T V: a K step of three parts per slot
        const uint32_t dv = desc_lo(sb + SM_V, kHalf);
        int slot = 0, use = 0;
        for (int it = 0; it < nchunks; ++it) {
            const int st = it & 1;
            const uint32_t v = dv + (uint32_t)st * (kTile >> 4);
            if (!wait_warp(FULL_V + st, it >> 1)) break;
            const int ub = STATES_ONLY ? it & 1 : 0;
            const uint32_t u = tm + (ub ? TM_O : TM_U);
            if (STATES_ONLY ? it >= 2 && !wait_warp(U_FREE + ub, (it >> 1) - 1) : it > 0 && !wait_warp(U_FREE, it - 1)) break;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                if (!wait_warp(KP_READY + slot, use)) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int p = 0; p < 3; ++p)
                        if (p < 2 || it >= three_at)
                            umma_ts(u, tm + kp_column(slot) + p * kKpPart, v + (uint32_t)(ks * 128), id_nn,
                                    ks > 0 || p > 0);
                    umma_commit(bar(KP_FREE + slot));
                    if (ks == 7) {
                        umma_commit(bar(U_READY + ub));
                        umma_commit(bar(FREE_V + st));
                    }
                }
                if (++slot == kSlots) { slot = 0; ++use; }
            }
            if (!ok) break;
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

template <typename Kernel>
int launch_registers(Kernel kernel)
{
    cudaFuncAttributes attr;
    return cudaFuncGetAttributes(&attr, kernel) == cudaSuccess ? attr.numRegs : -1;
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
    // the move of registers between warps is sized for this many: with fewer it would wait for ever
    static const int regs[2] = {launch_registers(la_tc_kernel<false>), launch_registers(la_tc_kernel<true>)};
    if (regs[states_only] != kLaunchRegs) return cudaErrorInvalidKernelImage;
    static OncePerDevice once[2];
    if ((e = set_shared_memory(kernel, (int)SM_TOTAL, once[states_only])) != cudaSuccess) return e;
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

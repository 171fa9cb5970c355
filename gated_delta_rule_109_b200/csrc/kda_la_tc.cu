// Linear attention with one decay per head on the tensor cores (tcgen05): bf16 inputs,
// dk = dv = 128 (the mathematics is in kda_la.cuh).
//
// One CTA has one (pass, b, h, segment) and walks its chunks of 128 tokens.  Per chunk, with
// accumulators in tensor memory:
//     S = Q K^T                 P = f_intra lambda^|i-j| S on the causal side, as bf16, in place
//     O = Q S0                  rescaled by rows with f_inter lambda^(i+1), then  O += P V
//     U = K'^T V                K' = f_write lambda^(c-1-j) K;  S0 <- lambda^c S0 + U in registers
// Where the heads alone do not fill the device the sequence is cut into segments.  A segment is
// then walked twice: first over k and v alone for its own contribution to the state, which it
// leaves in the workspace, then, with the contributions of all earlier segments added up to its
// entering state, for the outputs.  Both walks are in one launch: a CTA waits (with a limit) for
// the earlier segments' contributions.  CTAs take their work by a counter, earlier segments
// first, so that whatever a CTA waits for has been taken by one that runs.
// Roundings.  Q, K, V enter exactly.  P and the entering state S0 are rounded to bf16 for
// their products: each output is a sum of such terms, so their errors together are of the
// size of the output's own rounding to bf16.  The state that is carried is fp32: K' is
// written as three bf16 parts that hold all 24 bits of the fp32 product, U starts afresh
// every chunk (the tensor core's accumulation is short) and is added in registers, and
// lambda^c is a pair of floats, because its rounding would grow with the number of chunks.
// The third part is left out where it is not seen: two parts are off by at most 2^-14.7 of a
// term and 2^-17.7 in the root mean square (cut2), so they do for a state that only enters bf16
// products, and for terms that fade to less than 2^-6 of their size before the state is written
// out (their errors to 2^-20.7 and 2^-23.7; states measure 1e-7 to 6e-7 off, most of it what the
// tensor core cuts off when it adds, towards zero).  An output's last bit may so depend on whether
// a final state is asked for.  The kernel runs into the power limit (1.5 of 1.97 GHz at
// B4 H32 T16384, 980 W), and U is half of its products.
//
// Warps: 0-3 turn S into P and 4-7 rescale O and write the outputs (a thread is a token); 8-15
// make K'^T in tensor memory, groups of four by turns (ldmatrix transposes the K tile; while
// there are no outputs, warps 0-7 help);
// 16-23 carry the state (a thread is a key channel and half of the value columns); 24 moves
// tiles by TMA; 25 issues Q K^T, Q S0 and P V, 26 the steps of U: a wait and an issue take a
// warp about as long as the tensor core takes for a step.
// Shared memory holds two stages of q, k, v (192 KB) and the state as an operand (32 KB); the
// outputs of a chunk leave through its q tile.  Tiles are two boxes of 64 channels x 128
// tokens in the 128-byte swizzle, which serves as K-major operand (channels contracted) and
// as MN-major operand (tokens contracted) alike.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <atomic>

#include "kda_la.cuh"
#include "kda_tc_ptx.cuh"

namespace kda {

__device__ unsigned int g_la_device_status = 0;

namespace {

using namespace tcx;

constexpr int kC = 128, kD = 128;
constexpr int kRowWarps = 4, kKeyWarps = 8, kStateWarps = 8;
constexpr int kKeyWarp0 = 2 * kRowWarps, kStateWarp0 = kKeyWarp0 + kKeyWarps, kTmaWarp = kStateWarp0 + kStateWarps, kMmaWarp = kTmaWarp + 1, kUpdateWarp = kMmaWarp + 1;
constexpr int kThreads = 32 * (kUpdateWarp + 1);
constexpr int kLaunchRegs = 72, kWorkRegs = 56, kStateRegs = 104;      // the first kStateWarp0 warps, the state's
static_assert(kStateWarp0 * (kLaunchRegs - kWorkRegs) >= kStateWarps * (kStateRegs - kLaunchRegs), "registers moved");

// shared memory
constexpr uint32_t kHalf = 64 * kC * 2, kTile = 2 * kHalf;        // 16 KB box, 32 KB tile
constexpr uint32_t SM_Q = 0, SM_K = SM_Q + 2 * kTile, SM_V = SM_K + 2 * kTile, SM_S0 = SM_V + 2 * kTile;
constexpr uint32_t SM_WP = SM_S0 + kTile;             // [256] f_intra lambda^(i-j) at i - j + 127, zeros beyond
constexpr uint32_t SM_WK = SM_WP + 256 * 4;           // [2][128] f_write lambda^(.) of a whole and of the ragged chunk
constexpr uint32_t SM_PW = SM_WK + 2 * 128 * 4;       // [129] lambda^n
constexpr uint32_t SM_LC = SM_PW + 132 * 4;           // [2] lambda^c of a whole and of the ragged chunk, two floats each
constexpr uint32_t SM_BAR = SM_LC + 16;
constexpr int kKpSlots = 5;
enum Bar {
    FULL_Q = 0, FULL_K = 2, FULL_V = 4, FREE_K = 6, FREE_V = 8, OUT_READY = 10, U_READY = 12, U_FREE = 14,
    X_FULL = 16, X_FREE = 18, KP_READY = 20, KP_FREE = KP_READY + kKpSlots, S_READY = KP_FREE + kKpSlots, QS_READY,
    PV_GO, PV_DONE, O_FREE, S0_READY, kBars
};
constexpr uint32_t SM_TMEM = SM_BAR + 8 * kBars;      // address of the tensor memory, work item
constexpr uint32_t SM_TOTAL = SM_TMEM + 16;
static_assert(SM_TOTAL <= 227 * 1024, "shared memory of a CTA");

// Tensor memory columns.  The walk without outputs has O's columns for a second U, so that a
// chunk's U is computed while the one before is added to the state.
constexpr uint32_t TM_S = 0, TM_P = 0, TM_O = 128, TM_U = 256, TM_KP = 384;
constexpr uint32_t kKpPart = 8, kKpSlot = 3 * kKpPart;         // a slot: 16 tokens x 3 parts
static_assert(TM_KP + kKpSlots * kKpSlot <= 512, "slots");

// The workspace: a counter of work items, for each contribution the number of warps that have
// left their part, and [npass][B H][nseg] states of 64 KB in the order in which the state's
// threads hold them: the contributions, and at nseg - 1 what segment 0 started from (it needs
// that again for its outputs, when final_state, which may be initial_state, may be written).
constexpr size_t kSlotFloats = (size_t)kD * kD;
size_t flag_bytes(const LaArgs &a)
{
    return (sizeof(int) * (1 + (size_t)a.npass * a.B * a.H * a.nseg) + 255) & ~size_t(255);
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

// One head's 128 tokens from t on, both halves.
__device__ __forceinline__ void load_tile(const void *tmap, uint32_t dst, uint32_t mbar, int h, int t, int b)
{
    mbar_expect_tx(mbar, 64 * 128 * 2 * 2);
    tma_load_4d(dst, tmap, mbar, 0, h, t, b);
    tma_load_4d(dst + 64 * 128 * 2, tmap, mbar, 64, h, t, b);
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

__device__ __forceinline__ void mbar_arrive_n(uint32_t mbar, uint32_t n)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" :: "r"(mbar), "r"(n) : "memory");
}

__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// Registers move to the state warps from the others, within what the block was launched with.
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
// k w as the sum of two bf16, k a pair of bf16 and w = wh + wl in two parts, in packed bf16
// arithmetic: hi = k wh rounded, whose error k wh - hi has at most 8 bits and is exact, and
// mid = k wl + that error, rounded.  mid is below 2^-6 of hi's power of two, so its rounding
// costs up to 2^-15 of k w and the rest of w that wl does not hold 2^-17: off by at most 2^-14.7,
// 2^-17.7 in the root mean square (over 2 10^7 random pairs: 2^-14.9 and 2^-17.75).  Half the
// instructions of the same in fp32.
__device__ __forceinline__ void cut2(uint32_t k, uint32_t wh, uint32_t wl, uint32_t &hi, uint32_t &mid)
{
    asm("{\n\t.reg .b32 n;\n\tmul.rn.bf16x2 %0, %2, %3;\n\tneg.bf16x2 n, %0;\n\tfma.rn.bf16x2 n, %2, %3, n;\n\t"
        "fma.rn.bf16x2 %1, %2, %4, n;\n\t}" : "=&r"(hi), "=r"(mid) : "r"(k), "r"(wh), "r"(wl));
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

__device__ __forceinline__ int load_acquire(const int *p)
{
    int v;
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
// ---- the state of work item x, 64 floats a thread: key channel r, value columns 64 part ..
__device__ __forceinline__ int reread(uint32_t saddr)
{
    int v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(saddr) : "memory");
    return v;
}
// Work items: segments outermost, then heads, then passes, so that the passes of a head, which
// read the same four tensors, run beside each other and find them in L2.
__device__ __forceinline__ const LaPass &pass_of(const LaArgs &a, int x, int &bh)
{
    const int chain = x % (a.npass * a.B * a.H);
    bh = chain / a.npass;
    return a.pass[chain % a.npass];
}
// The pass's initial state, or zeros (`zero`, or none given).  32 rows x 32 columns at a time go
// through 4 KB of shared memory of the warp's own, so that global memory is read by whole
// sectors and a thread still gets its row; one way for all cases, so that S has one definition.
__device__ __forceinline__ void load_initial(const LaArgs &a, int x, bool zero, int quad, int part, int lane, uint32_t buf,
                                             float (&S)[64])
{
    int bh;
    const LaPass &ps = pass_of(a, x, bh);
    const float *s0 = ps.s0 && !zero ? ps.s0 + (size_t)bh * kSlotFloats : nullptr;
    const uint32_t mine = buf + (uint32_t)lane * 128u, swz = (uint32_t)(lane & 7) << 4;
#pragma unroll
    for (int c0 = 0; c0 < 64; c0 += 32) {
        __syncwarp();
        if (!s0) {
            if (c0 == 0)
#pragma unroll
                for (int i = 0; i < 8; ++i) st_shared16(mine + 16u * (uint32_t)i, 0u, 0u, 0u, 0u);
        } else if (ps.s0_transposed) {                      // lane = row, four columns of it
#pragma unroll 4
            for (int i = 0; i < 8; ++i) {
                const float *p = s0 + (64 * part + c0 + 4 * i) * kD + 32 * quad + lane;
                st_shared16(mine + ((16u * (uint32_t)i) ^ swz), __float_as_uint(p[0]), __float_as_uint(p[kD]),
                            __float_as_uint(p[2 * kD]), __float_as_uint(p[3 * kD]));
            }
        } else {                                            // eight lanes = 128 bytes of a row
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int row = 4 * i + (lane >> 3), piece = lane & 7;
                const uint4 u = *reinterpret_cast<const uint4 *>(s0 + (32 * quad + row) * kD + 64 * part + c0 + 4 * piece);
                st_shared16(buf + (uint32_t)(row * 128) + ((16u * (uint32_t)piece) ^ ((uint32_t)(row & 7) << 4)), u.x, u.y,
                            u.z, u.w);
            }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t src = mine + ((16u * (uint32_t)i) ^ swz);
            asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                         : "=f"(S[c0 + 4 * i]), "=f"(S[c0 + 4 * i + 1]), "=f"(S[c0 + 4 * i + 2]), "=f"(S[c0 + 4 * i + 3])
                         : "r"(src) : "memory");
        }
    }
    __syncwarp();
}
__device__ __forceinline__ void store_final(const LaArgs &a, int x, int r, int part, const float (&S)[64])
{
    int bh;
    const LaPass &ps = pass_of(a, x, bh);
    if (!ps.sT || x / (a.B * a.H) / a.npass != a.nseg - 1) return;
    float *dst = ps.sT + (size_t)bh * kSlotFloats + r * kD + 64 * part;
#pragma unroll
    for (int i = 0; i < 64; i += 4) *reinterpret_cast<float4 *>(dst + i) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
}
// S to state `g` of the workspace's chain of item x, 16 x float4 of thread `me`, a warp's 512
// bytes beside each other, and counted for those that wait for it.
__device__ __forceinline__ void leave_state(const LaArgs &a, int x, int g, int me, int *flags, float *slots,
                                            const float (&S)[64])
{
    const size_t at = (size_t)(x % (a.npass * a.B * a.H)) * a.nseg + g;
    float4 *dst = reinterpret_cast<float4 *>(slots + at * kSlotFloats) + me;
#pragma unroll
    for (int i = 0; i < 16; ++i) dst[256 * i] = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
    __threadfence();
    __syncwarp();
    if ((me & 31) == 0) atomicAdd(flags + 1 + at, 1);
}
__global__ void __launch_bounds__(kThreads, 1)
la_tc_kernel(const __grid_constant__ LaArgs a, const __grid_constant__ LaMaps maps, int *flags, float *slots)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sb = (uint32_t)__cvta_generic_to_shared(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int heads = a.npass * a.B * a.H;
    auto bar = [&](int i) { return sb + SM_BAR + 8u * (uint32_t)i; };

    // ---- barriers, tensor memory, the work item
    if (warp == kTmaWarp && lane == 0) {
        for (int i = 0; i < kBars; ++i) {
            const int count = (i >= FREE_K && i < FREE_V) ? kStateWarp0
                              : (i >= FREE_V && i < OUT_READY) ? 2
                              : (i >= OUT_READY && i < U_READY) || i == O_FREE ? kRowWarps
                              : i == PV_GO ? 2 * kRowWarps
                              : (i >= KP_READY && i < KP_FREE) ? kKeyWarps / 2
                              : (i >= U_FREE && i < X_FULL) || (i >= X_FREE && i < KP_READY) || i == S0_READY ? kStateWarps : 1;
            mbar_init(bar(i), (uint32_t)count);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        *reinterpret_cast<int *>(smem + SM_TMEM + 4) = a.nseg > 1 ? atomicAdd(flags, 1) : (int)blockIdx.x;
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(sb + SM_TMEM) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int item = *reinterpret_cast<const int *>(smem + SM_TMEM + 4);
    const int seg = item / heads, ip = item % heads % a.npass, bh = item % heads / a.npass;
    const LaPass &ps = a.pass[ip];
    const int b = bh / a.H, h = bh % a.H, rev = ps.rev;
    int t_lo, t_hi;
    la_segment(seg, a.nseg, a.seg_tokens, a.T, rev, t_lo, t_hi);
    const int n0 = t_lo / kC, nchunks = (t_hi + kC - 1) / kC - n0;
    const int c_last = t_hi - (n0 + nchunks - 1) * kC;          // tokens of the chunk at the segment's end in time
    const int tail_at = c_last == kC ? -1 : rev ? 0 : nchunks - 1;      // the walk's step that is the ragged chunk
    // steps 0 .. nown - 1: the segment's own contribution; nown .. nown + nchunks - 1: the outputs
    const int nown = seg < a.nseg - 1 ? nchunks : 0, nsteps = nown + nchunks;
    auto chunk_at = [&](int j) { return n0 + (rev ? nchunks - 1 - j : j); };

    if (warp == kTmaWarp) {
        // the first tiles are on their way while the others set up
        if (lane == 0)
            for (int it = 0; it < 2 && it < nsteps; ++it) {
                const int t = chunk_at(it < nown ? it : it - nown) * kC;
                load_tile(&maps.k[ip], sb + SM_K + it * kTile, bar(FULL_K + it), h, t, b);
                load_tile(&maps.v[ip], sb + SM_V + it * kTile, bar(FULL_V + it), h, t, b);
                if (a.nseg == 1) load_tile(&maps.q[ip], sb + SM_Q + it * kTile, bar(FULL_Q + it), h, t, b);
            }
        __syncwarp();
    } else if (tid < 256) {
        // powers of lambda in 64 bits
        float *sWP = reinterpret_cast<float *>(smem + SM_WP), *sWK = reinterpret_cast<float *>(smem + SM_WK);
        const int j = tid & (kC - 1), c = tid < kC ? kC : c_last;
        sWK[tid] = ps.f_write * (float)la_power(a.log_decay, h, rev ? j + 1 : max(c - 1 - j, 0));
        const int apart = tid - 127;                            // i - j
        sWP[tid] = (rev ? apart <= 0 : apart >= 0) ? ps.f_intra * (float)la_power(a.log_decay, h, abs(apart)) : 0.f;
    } else if (tid < 256 + kC + 1) {
        reinterpret_cast<float *>(smem + SM_PW)[tid - 256] = (float)la_power(a.log_decay, h, tid - 256);
    } else if (tid < 256 + kC + 3) {
        const int ragged = tid - (256 + kC + 1);
        const double l = la_power(a.log_decay, h, ragged ? c_last : kC);
        reinterpret_cast<float2 *>(smem + SM_LC)[ragged] = make_float2((float)l, (float)(l - (double)(float)l));
    }
    __syncthreads();
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
    // Steps of a walk whose K' has all three parts: from this one on.  `tokens` come behind
    // the segment; counted one chunk short, so that a ragged chunk leaves no step out.
    auto three_from = [&](bool wanted) {
        if (!wanted) return nchunks;
        if (!a.log_decay) return 0;
        const float fade = 6.f / (-1.4426950408889634f * a.log_decay[h]);       // tokens to 2^-6
        if (!(fade >= 0.f && fade < 1e9f)) return 0;                            // it does not fade
        const float behind = rev ? (float)t_lo : (float)(a.T - t_hi);
        return min(max(nchunks - 2 - (int)floorf((fade - behind) * (1.f / kC)), 0), nchunks);
    };

    if (warp < kStateWarp0) {
        reg_dec<kWorkRegs>();
        // ---- K'^T: 16 tokens a slot of the ring, 32 key channels a warp.  Of a step's eight slots
        // group g of n makes g, g + n, ..
        const int quad = warp & 3;
        // ldmatrix: lanes 8 m .. 8 m + 7 name the rows (tokens) of matrix m: tokens 8 (m / 2) ..,
        // channels 8 (m % 2) .. of the 16 of a half-warp; 16-byte pieces swizzled by token % 8
        const int jr = lane & 7, m = lane >> 3, piece = 4 * (quad & 1) + (m & 1);
        const uint32_t kt = sb + SM_K + (quad >> 1) * kHalf + (uint32_t)((8 * (m >> 1) + jr) * 128);
        const uint32_t off0 = (uint32_t)((piece ^ jr) << 4), off1 = (uint32_t)(((piece + 2) ^ jr) << 4);
        auto make_keys = [&](int it, int j, bool three, int group, int ngroups) {
            const float *wk = reinterpret_cast<const float *>(smem + SM_WK) + (j == tail_at ? kC : 0) + 2 * (lane & 3);
            const int st = it & 1;
            if (!wait_warp(FULL_K + st, it >> 1)) return false;
#pragma unroll 1
            for (int ks = group; ks < 8; ks += ngroups) {
                const uint32_t src = kt + st * kTile + ks * (16 * 128);
                const int use = (8 * it + ks) / kKpSlots, slot = 8 * it + ks - use * kKpSlots;
                uint32_t k0[4], k1[4], hi[8], mid[8], lo[8];
                ldmatrix4_trans(src + off0, k0);
                ldmatrix4_trans(src + off1, k1);
                const float2 w0 = *reinterpret_cast<const float2 *>(wk + 16 * ks);
                const float2 w1 = *reinterpret_cast<const float2 *>(wk + 16 * ks + 8);
                if (three) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        cut3(scale_pair(e < 4 ? k0[e & 3] : k1[e & 3], (e & 2) ? w1 : w0), hi[e], mid[e], lo[e]);
                } else {
                    uint32_t wh[2], wl[2];
                    split_pair2(w0, wh[0], wl[0]);
                    split_pair2(w1, wh[1], wl[1]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) cut2(e < 4 ? k0[e & 3] : k1[e & 3], wh[(e >> 1) & 1], wl[(e >> 1) & 1], hi[e], mid[e]);
                }
                if (use > 0 && !wait_warp(KP_FREE + slot, use - 1)) return false;
                tc_fence_after();
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const uint32_t dst = tm + ((uint32_t)(32 * quad + 4 * e) << 16) + TM_KP + slot * kKpSlot;
                    tmem_st_16x8(dst, hi[e], hi[e + 1], hi[e + 2], hi[e + 3]);
                    tmem_st_16x8(dst + kKpPart, mid[e], mid[e + 1], mid[e + 2], mid[e + 3]);
                    if (three) tmem_st_16x8(dst + 2 * kKpPart, lo[e], lo[e + 1], lo[e + 2], lo[e + 3]);
                }
                tmem_wait_st();
                tc_fence_before();
                arrive_warp(KP_READY + slot);
            }
            return true;
        };
        const int three_own = three_from(ps.sT);
        for (int it = 0; it < nown; ++it) {
            if (!make_keys(it, it, it >= three_own, warp >> 2, kStateWarp0 / 4)) break;
            arrive_warp(FREE_K + (it & 1));
        }
        if (warp >= kKeyWarp0) {
            const int three_out = three_from(ps.sT && seg == a.nseg - 1), group = (warp - kKeyWarp0) >> 2;
            for (int j = 0; j < nchunks && ok; ++j) {
                const int it = nown + j;
                if (!make_keys(it, j, j >= three_out, group, kKeyWarps / 4)) break;
                __syncwarp();
                // the eight of these warps, Q K^T's commit, and one for the warps that do not read K here
                if (lane == 0) mbar_arrive_n(bar(FREE_K + (it & 1)), warp == kKeyWarp0 ? kStateWarp0 - kKeyWarps : 1);
            }
        } else if (warp < kRowWarps) {
            // ---- P from S: token i
            const int i = 32 * warp + lane;
            const uint32_t row = tm + ((uint32_t)(32 * warp) << 16);
            const float *w = reinterpret_cast<const float *>(smem + SM_WP) + 127 + i;
            for (int j = 0; j < nchunks && ok; ++j) {
                if (!wait_warp(S_READY, j)) break;
                tc_fence_after();
#pragma unroll 1
                for (int cb = 0; cb < 4; ++cb) {
                    uint32_t p[16];
                    if (rev ? cb >= warp : cb <= warp) {
                        float s[32];
                        tmem_ld32(row + TM_S + 32 * cb, s);
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            p[x] = pack_bf16(s[2 * x] * w[-32 * cb - 2 * x], s[2 * x + 1] * w[-32 * cb - 2 * x - 1]);
                    } else {
#pragma unroll
                        for (int x = 0; x < 16; ++x) p[x] = 0u;
                    }
                    tmem_st16u(row + TM_P + 16 * cb, p);
                }
                tmem_wait_st();
                tc_fence_before();
                arrive_warp(PV_GO);
            }
        } else {
            // ---- O <- f_inter lambda^(.) O for P V to add to, then the outputs: token i
            const int i = 32 * (warp - kRowWarps) + lane;
            const uint32_t row = tm + ((uint32_t)(32 * (warp - kRowWarps)) << 16);
            const float *sPW = reinterpret_cast<const float *>(smem + SM_PW);
            for (int j = 0; j < nchunks && ok; ++j) {
                const int c = j == tail_at ? c_last : kC, st = j & 1;
                const float f = ps.f_inter * sPW[rev ? max(c - 1 - i, 0) : i + 1];
                if (!wait_warp(QS_READY, j)) break;
                tc_fence_after();
#pragma unroll 1
                for (int cb = 0; cb < 8; ++cb) {
                    float o[16];
                    tmem_ld16(row + TM_O + 16 * cb, o);
#pragma unroll
                    for (int x = 0; x < 16; ++x) o[x] *= f;
                    tmem_st16(row + TM_O + 16 * cb, o);
                }
                tmem_wait_st();
                tc_fence_before();
                arrive_warp(PV_GO);
                if (!wait_warp(PV_DONE, j)) break;
                tc_fence_after();
                const uint32_t dst = sb + SM_Q + (uint32_t)(st * kTile + i * 128);
#pragma unroll 1
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
                arrive_warp(O_FREE);                                // Q S0 of the next chunk may begin
                proxy_fence();
                arrive_warp(OUT_READY + st);
            }
        }
    } else if (warp < kTmaWarp) {
        // ---- the state: key channel r, value columns 64 part ..  (The walk leaves no registers for
        // what is needed before and after it: that is read from the work item again.)
        const int quad = warp & 3, part = (warp - kStateWarp0) >> 2;
        const int r = 32 * quad + lane;
        const uint32_t row = tm + ((uint32_t)(32 * quad) << 16) + 64 * part;
        reg_inc<kStateRegs>();
        float S[64];
        // segment 0's own contribution includes the initial state
        const uint32_t buf = sb + SM_S0 + (uint32_t)(4096 * (4 * part + quad));     // until the state is published
        load_initial(a, reread(sb + SM_TMEM + 4), seg != 0, quad, part, lane, buf, S);
        // S <- lambda^c S + U; the second float of lambda^c goes with the third part of K'
        auto absorb = [&](int ub, int use, int j, bool exact) {
            if (!wait_warp(U_READY + ub, use)) return false;
            tc_fence_after();
            const float2 l = reinterpret_cast<const float2 *>(smem + SM_LC)[j == tail_at];
            const uint32_t src = row + (ub ? TM_O : TM_U);
#pragma unroll
            for (int x = 0; x < 64; x += 8) {
                float u[8];
                tmem_ld8(src + x, u);
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    if (exact) u[y] = fmaf(l.y, S[x + y], u[y]);
                    S[x + y] = fmaf(l.x, S[x + y], u[y]);
                }
            }
            tc_fence_before();
            arrive_warp(U_FREE + ub);
            return true;
        };
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
        if (a.nseg > 1) {
            const int me = tid - 32 * kStateWarp0;
            if (seg == 0) leave_state(a, reread(sb + SM_TMEM + 4), a.nseg - 1, me, flags, slots, S);
            const int three_own = three_from(ps.sT);
            for (int j = 0; j < nown; ++j)
                if (!absorb(j & 1, j >> 1, j, j >= three_own)) break;
            if (ok) {
                const int x0 = reread(sb + SM_TMEM + 4);
                if (nown > 0) leave_state(a, x0, x0 / heads, me, flags, slots, S);
                // The state that enters the segment: the contributions of all segments before it, or
                // what segment 0 started from, one after the other through the q tiles, summed up from
                // zero: the segment's own, which comes behind all of its outputs, may not be finite.
                // Lane g holds how much fades over segment g.
#pragma unroll
                for (int i = 0; i < 64; ++i) S[i] = 0.f;
                float wh = 0.f, wl = 0.f;
                if (lane > 0 && lane < x0 / heads) {
                    int bh0, t0, t1;
                    const LaPass &p0 = pass_of(a, x0, bh0);
                    la_segment(lane, a.nseg, a.seg_tokens, a.T, p0.rev, t0, t1);
                    const double l = la_power(a.log_decay, bh0 % a.H, t1 - t0);
                    wh = (float)l;
                    wl = (float)(l - (double)wh);
                }
                for (int g = 0; ok && g < max(x0 / heads, 1); ++g) {
                    const float lh = __shfl_sync(0xffffffffu, wh, g), ll = __shfl_sync(0xffffffffu, wl, g);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        if (!wait_warp(X_FULL + half, g)) break;
                        const uint32_t src = sb + SM_Q + (uint32_t)(half * kTile + 16 * me);
#pragma unroll
                        for (int i = 32 * half; i < 32 * half + 32; i += 4) {
                            float u[4];
                            asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(u[0]), "=f"(u[1]), "=f"(u[2]), "=f"(u[3])
                                         : "r"(src + (uint32_t)(1024 * (i - 32 * half))) : "memory");
#pragma unroll
                            for (int y = 0; y < 4; ++y) S[i + y] = fmaf(lh, S[i + y], fmaf(ll, S[i + y], u[y]));
                        }
                        arrive_warp(X_FREE + half);
                    }
                }
            }
        }
        if (ok) publish();
        const int three_out = three_from(ps.sT && seg == a.nseg - 1);
        for (int j = 0; j < nchunks && ok; ++j) {
            if (!absorb(0, ((nown + 1) >> 1) + j, j, j >= three_out)) break;
            if (j + 1 < nchunks) {
                if (!wait_warp(QS_READY, j)) break;             // the operand of this chunk has been read
                publish();
            }
        }
        if (ok) store_final(a, reread(sb + SM_TMEM + 4), r, part, S);
    } else if (warp == kTmaWarp) {
        if (lane == 0) {
            auto store = [&](int j) {
                const uint32_t src = sb + SM_Q + (j & 1) * kTile;
                const int t = chunk_at(j) * kC;
                tma_store_4d(&maps.out[ip], src, 0, h, t, b);
                tma_store_4d(&maps.out[ip], src + kHalf, 64, h, t, b);
                bulk_commit();
            };
            auto load_q = [&](int j) {
                load_tile(&maps.q[ip], sb + SM_Q + (j & 1) * kTile, bar(FULL_Q + (j & 1)), h, chunk_at(j) * kC, b);
            };
            // the states that enter the segment's outputs, in halves of 32 KB through the q tiles
            int halves = 0;
            auto load_states = [&] {
                const size_t chain = (size_t)(item % heads) * a.nseg;
                for (int g = 0; g < max(seg, 1); ++g) {
                    const size_t at = chain + (seg == 0 ? a.nseg - 1 : g);
                    const long long t0 = clock64();
                    while (load_acquire(flags + 1 + at) != kStateWarps)
                        if (clock64() - t0 > kWaitCycles) {
                            ok = false;
                            atomicOr(&g_la_device_status, 1u);
                            return;
                        }
                    asm volatile("fence.proxy.async;" ::: "memory");        // plain stores there, bulk copies here
                    for (int half = 0; half < 2; ++half) {
                        if (g > 0 && !wait(X_FREE + half, g - 1)) return;
                        mbar_expect_tx(bar(X_FULL + half), kTile);
                        bulk_g2s(sb + SM_Q + half * kTile, reinterpret_cast<const uint8_t *>(slots + at * kSlotFloats) + half * kTile,
                                 kTile, bar(X_FULL + half));
                        ++halves;
                    }
                }
                for (int half = 0; half < 2; ++half) wait(X_FREE + half, max(seg, 1) - 1);
            };
            int it = 0;
            for (; it < nsteps; ++it) {
                const int st = it & 1, j = it < nown ? it : it - nown, t = chunk_at(j) * kC;
                if (it >= 2) {                                  // the first two are under way
                    if (!wait(FREE_K + st, (it >> 1) - 1)) break;
                    load_tile(&maps.k[ip], sb + SM_K + st * kTile, bar(FULL_K + st), h, t, b);
                    if (!wait(FREE_V + st, (it >> 1) - 1)) break;
                    load_tile(&maps.v[ip], sb + SM_V + st * kTile, bar(FULL_V + st), h, t, b);
                }
                if (it < nown) continue;
                if (j >= 2) {
                    // the outputs of chunk j - 2 leave the q tile, then it is loaded again
                    if (!wait(OUT_READY + (j & 1), (j >> 1) - 1)) break;
                    store(j - 2);
                    bulk_wait_read();
                    load_q(j);
                } else if (a.nseg > 1 && (j == 1 || nchunks == 1)) {
                    load_states();
                    if (!ok) break;
                    for (int x = 0; x <= j; ++x) load_q(x);
                }
            }
            for (int j = max(nchunks - 2, 0); j < nchunks && ok; ++j) {
                if (!wait(OUT_READY + (j & 1), j >> 1)) break;
                store(j);
            }
            bulk_wait_read();
            if (!ok)                        // no copy may land after the CTA has left
                for (int i = max(it - 2, 0); i <= it && i < nsteps; ++i) {
                    mbar_wait(bar(FULL_K + (i & 1)), (i >> 1) & 1);
                    mbar_wait(bar(FULL_V + (i & 1)), (i >> 1) & 1);
                    if (i >= nown) mbar_wait(bar(FULL_Q + ((i - nown) & 1)), ((i - nown) >> 1) & 1);
                }
            if (!ok)
                for (int x = max(halves - 2, 0); x < halves; ++x) mbar_wait(bar(X_FULL + (x & 1)), (x >> 1) & 1);
        }
    } else if (warp == kMmaWarp) {
        // Whole warps walk the loops and one elected lane issues, so that descriptors stay in
        // uniform registers: under `lane == 0` each product took 100 cycles to issue, against
        // the 64 it runs.
        const uint32_t dq = desc_lo(sb + SM_Q, 16), dk = desc_lo(sb + SM_K, 16);
        const uint32_t dv = desc_lo(sb + SM_V, kHalf), ds = desc_lo(sb + SM_S0, kHalf);
        // A K step of 16 channels is 32 bytes inside the swizzled rows of a K-major tile, 16
        // rows of an MN-major one (addresses in 16 bytes).
        auto k_major = [](int ks) { return (uint32_t)((ks >> 2) * (kHalf >> 4) + (ks & 3) * 2); };
        for (int j = 0; j < nchunks; ++j) {
            const int it = nown + j, st = it & 1;
            const uint32_t qs = (uint32_t)(j & 1) * (kTile >> 4), stage = (uint32_t)st * (kTile >> 4);
            // S = Q K^T
            if (!wait_warp(FULL_Q + (j & 1), j >> 1) || !wait_warp(FULL_K + st, it >> 1)) break;
            if (j > 0 && !wait_warp(PV_DONE, j - 1)) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    umma_ss(tm + TM_S, dq + qs + k_major(ks), dk + stage + k_major(ks), id_nt, ks > 0);
                umma_commit(bar(S_READY));
                umma_commit(bar(FREE_K + st));
            }
            // O = Q S0 (its columns were U's before: the state is published after the last of those)
            if (!wait_warp(S0_READY, j) || (j > 0 && !wait_warp(O_FREE, j - 1))) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    umma_ss(tm + TM_O, dq + qs + k_major(ks), ds + (uint32_t)(ks * 128), id_nn, ks > 0);
                umma_commit(bar(QS_READY));
            }
            // O += P V
            if (!wait_warp(FULL_V + st, it >> 1) || !wait_warp(PV_GO, j)) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    umma_ts(tm + TM_O, tm + TM_P + 8 * ks, dv + stage + (uint32_t)(ks * 128), id_nn, true);
                umma_commit(bar(PV_DONE));
                umma_commit(bar(FREE_V + st));
            }
        }
    } else {
        // U = K'^T V: a K step of three (or two) parts per slot
        const uint32_t dv = desc_lo(sb + SM_V, kHalf);
        const int three_own = three_from(ps.sT), three_out = nown + three_from(ps.sT && seg == a.nseg - 1);
        int slot = 0, use = 0;
        for (int it = 0; it < nsteps; ++it) {
            const bool own = it < nown;
            const int st = it & 1, ub = own ? it & 1 : 0, uuse = own ? it >> 1 : ((nown + 1) >> 1) + it - nown;
            const uint32_t v = dv + (uint32_t)st * (kTile >> 4), u = tm + (ub ? TM_O : TM_U);
            const bool three = it >= (own ? three_own : three_out);
            if (!wait_warp(FULL_V + st, it >> 1)) break;
            if (uuse > 0 && !wait_warp(U_FREE + ub, uuse - 1)) break;
#pragma unroll 1
            for (int ks = 0; ks < 8; ++ks) {
                if (!wait_warp(KP_READY + slot, use)) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int p = 0; p < 3; ++p)
                        if (p < 2 || three)
                            umma_ts(u, tm + TM_KP + slot * kKpSlot + p * kKpPart, v + (uint32_t)(ks * 128), id_nn,
                                    ks > 0 || p > 0);
                    umma_commit(bar(KP_FREE + slot));
                    if (ks == 7) {
                        umma_commit(bar(U_READY + ub));
                        umma_commit(bar(FREE_V + st));
                        if (own) mbar_arrive(bar(FREE_V + st));         // no other product reads the tile
                    }
                }
                if (++slot == kKpSlots) { slot = 0; ++use; }
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

// cuTensorMapEncodeTiled from the driver (the library links the CUDA runtime statically and not
// the driver library), looked up until it has been found once
cudaError_t map_encoder(PFN_cuTensorMapEncodeTiled_v12000 &fn)
{
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> found{nullptr};
    if ((fn = found.load(std::memory_order_acquire))) return cudaSuccess;
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || !p) return cudaErrorNotSupported;
    fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    found.store(fn, std::memory_order_release);
    return cudaSuccess;
}

// A [B, T, H, 128] bf16 tensor as (channel, head, token, batch), boxes of one head's 64
// channels x 128 tokens.  The token axis has its own bound: rows behind a sequence's end are
// read as zeros and not written.
cudaError_t token_map(PFN_cuTensorMapEncodeTiled_v12000 enc, const LaArgs &a, const void *p, CUtensorMap *m)
{
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

size_t la_tc_workspace_bytes(const LaArgs &a)
{
    return a.nseg > 1 ? flag_bytes(a) + sizeof(float) * kSlotFloats * a.npass * a.B * a.H * a.nseg : 0;
}

cudaError_t launch_la_tc(const LaArgs &a, cudaStream_t stream)
{
    static OncePerDevice once;
    // the move of registers between warps is sized for this many: with fewer it would wait for ever
    cudaError_t e = set_shared_memory(la_tc_kernel, (int)SM_TOTAL, once, kLaunchRegs);
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    if (e == cudaSuccess) e = map_encoder(enc);
    LaMaps maps;
    for (int i = 0; i < a.npass && e == cudaSuccess; ++i) {
        e = token_map(enc, a, a.pass[i].q, &maps.q[i]);
        if (e == cudaSuccess) e = token_map(enc, a, a.pass[i].k, &maps.k[i]);
        if (e == cudaSuccess) e = token_map(enc, a, a.pass[i].v, &maps.v[i]);
        if (e == cudaSuccess) e = token_map(enc, a, a.pass[i].out, &maps.out[i]);
    }
    if (e != cudaSuccess) return e;
    int *flags = reinterpret_cast<int *>(a.ws);
    float *slots = nullptr;
    if (a.nseg > 1) {
        if ((e = cudaMemsetAsync(flags, 0, flag_bytes(a), stream)) != cudaSuccess) return e;
        slots = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(a.ws) + flag_bytes(a));
    }
    const size_t grid = (size_t)a.npass * a.B * a.H * a.nseg;
    la_tc_kernel<<<(unsigned)grid, kThreads, SM_TOTAL, stream>>>(a, maps, flags, slots);
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

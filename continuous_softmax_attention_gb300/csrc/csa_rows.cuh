// Many rows over a paged cache: the stretch before the draft of a tree of drafted
// tokens (csa_tree.cu) where a cached head has more than 16 rows, on tcgen05.  Rows,
// ranges and parts as in csa_paged.cuh; a block of up to 128 rows is a segment.
//
// A CTA is a worker: a contiguous range of tiles of KT cached rows over all segments in
// a row.  Over bf16 pools two CTAs per SM with tiles of 64 rows, whose phases fall where
// they may (one CTA with two halves of 128 rows in step: 64 sequences of 300 rows with 8
// drafted tokens 61 us, so 51); 8-bit pools, which need more warps, and d = 256, whose
// sums fill half of the tensor memory, have one.  Warps:
//   softmax   a thread has one lane of tensor memory and one half of the tile's columns
//             (with bf16 pools and at d = 256 there is one half)
//   then      the tensor core (one lane), the copies of keys, those of values, and with
//             8-bit pools the cached rows' scales and four that turn codes into fp16 numbers
// Tensor memory: S (KT + 16 columns), P of each half (packed 16-bit weights), the sums O
// of each half.  Each half has its own maximum, weight sum and sums per row.
//
// Intervals.  A tile's columns are its KT rows and, for the interval to the row behind,
// the next one (a copy of 8 rows, of which the first is used); the interval from the row
// before comes from the tile before (its last logit, kept in a register), or for the first
// tile of a part from a copy of the 8 rows before, or is the sink's.  So a thread has all
// logits of its columns' intervals in its own lane, and no exchange.
//
// Fewer than 128 rows: the 128 lanes hold `reps` copies of R = 32 or 64 rows, and copy i
// weighs the i-th share of each half's columns: the threads always have 128 / reps columns
// of a tile, none idles, and the tensor core does the copies' products, which it has time
// for (a quarter of it at 64 rows).  The columns of the other shares in P are next to zero
// from the start.
//
// Weights over bf16 pools are two bf16 numbers (2^-16); tensor memory has room for one, so
// the low parts take the high ones' place and have a product of their own, while the next
// tile's logits are read.  One bf16 number (2^-9 off, where the output is rounded by as
// much) left o up to 2.7e-3 of its norm off, and two 1.7e-3, which is the output's rounding;
// it took 88 us where two took 100 (16 drafted tokens, 16 sequences of 4096 to 8192 rows, before
// the parts' cost was set).  Over 8-bit pools a weight times its row's scale is one fp16 number
// (2^-12), in a unit that follows the largest, and o is 1.6e-3 off.  All carry the factor
// (ln 2)^2, removed where parts are written.
//
// What bounds it: the weights, 24 instructions each of which 16 are the formula's; with two
// softmax warps per scheduler the issue slots are half busy (50%, e4m3 57%), the warps waiting
// for tensor memory and for one another's results.  16 sequences of 4096 to 8192 rows, 32 heads
// on 8, d = 128 (400 MB, 60 us at the copy bandwidth), with the join: 5 drafted tokens 81 us, 8
// 82 us, 16 98 us, 32 151 us, 64 293 us; e4m3 (210 MB) 5 97 us, 16 112 us, 32 166 us, int8 16
// 123 us; d = 64 16 84 us; d = 256 16 180 us, e4m3 205 us.  Where every tile's scales are far
// apart (2^-20 to 2^20), e4m3 16 118 us, 32 186 us.
#pragma once

#include <atomic>
#include <type_traits>

#include "csa_paged.cuh"

namespace {

// TMEM: consecutive columns of a thread's lane
__device__ __forceinline__ void tm_ld16(uint32_t at, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tm_ld1(uint32_t at, uint32_t &r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(at) : "memory");
}
__device__ __forceinline__ void tm_st8(uint32_t at, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// tcgen05.wait::ld that names the registers it waits for, so that no use is scheduled before it
__device__ __forceinline__ void tm_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
__device__ __forceinline__ void tm_wait(uint32_t &a) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(a)::"memory");
}
__device__ __forceinline__ void tm_wait(uint32_t &a, uint32_t &b, uint32_t &c) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(a), "+r"(b), "+r"(c)::"memory");
}

// Waits of the warps beside the softmax: a thread whose phase is not complete sleeps (up to 100 us at a time) and takes
// no issue slots from the others.
__device__ __forceinline__ bool wait_asleep(uint32_t bar, uint32_t parity, volatile int *abort_flag, int *status) {
    uint64_t t0 = 0;  // the timer is slow to read: not where the phase is complete
    while (true) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity), "r"(100000u)
            : "memory");
        if (done) return true;
        if (*abort_flag) return false;
        if (t0 == 0) t0 = globaltimer_ns();
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            *abort_flag = 1;
            *(volatile int *)status = kStatusTimeout;
            __threadfence();
            return false;
        }
    }
}

// The tensor core's lane asks again and again: woken from a wait with a time hint it would begin 200 cycles later, three
// times a tile.
__device__ __forceinline__ bool wait_awake(uint32_t bar, uint32_t parity, volatile int *abort_flag, int *status) {
    uint64_t t0 = 0;
    for (int i = 0;; ++i) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
        if (done) return true;
        if ((i & 63) != 63) continue;
        if (*abort_flag) return false;
        if (t0 == 0) t0 = globaltimer_ns();
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            *abort_flag = 1;
            *(volatile int *)status = kStatusTimeout;
            __threadfence();
            return false;
        }
    }
}

template <int D, int KIND>
struct RowsCfg {
    static constexpr bool Eight = KIND != CSA_BF16;
    static constexpr int Halves = D == 256 || !Eight ? 1 : 2;
    static constexpr int Blocks = Eight || D == 256 ? 1 : 2;  // per SM
    static constexpr int KT = 64 * Halves;   // cached rows per tile
    // What beginning and ending a part costs, in tiles.  64 ragged sequences of 1 to 8192 rows, 32 heads on 8, 8 drafted
    // tokens, d = 128: 104 us with 2, 84 with 4, 80 with 6, 85 with 12; e4m3 (tiles of 128 rows) 134 with 2, 118 with 3, 110
    // with 4, 116 with 6, 119 with 8, int8 135, 120, 112, 121 and 126; 16 drafted, d = 256 (one block per SM) 207 with 4, 185
    // with 6, 178 with 8, 196 with 12, e4m3 244 with 4, 234 with 6, 222 with 8, 226 with 10, 238 with 13.
    static constexpr int PartCost = D == 256 ? 8 : Eight ? 4 : 6;
    static constexpr int KR = KT + 16;       // and those of K: 8 behind, 8 before
    // warps: the softmax, the tensor core, the copies of keys and of values (which wait for different products, so each
    // has a warp), with 8 bits the cached rows' scales (else a spare one), and the four that turn codes into fp16 numbers
    static constexpr int SoftWarps = 4 * Halves, MmaWarp = SoftWarps, CopyWarp = SoftWarps + 1, ScaleWarp = SoftWarps + 3,
                         TurnWarp = SoftWarps + 4;
    static constexpr int TurnWarps = Eight ? 4 : 0;
    static constexpr int Threads = 32 * (SoftWarps + 4 + TurnWarps);
    // registers of the softmax warps and of the others; at launch every thread has 65536 / Threads, in eights
    static constexpr int SoftRegs = D == 256 ? 248 : Eight ? 152 : 160;
    static constexpr int OtherRegs = D == 256 && Eight ? 120 : Eight || D == 256 ? 104 : 96;
    static constexpr int LaunchRegs = 65536 / (Threads * Blocks) / 8 * 8 > 248 ? 248 : 65536 / (Threads * Blocks) / 8 * 8;
    static_assert(32 * SoftWarps * SoftRegs + (Threads - 32 * SoftWarps) * OtherRegs <= Threads * LaunchRegs, "the block's own registers");
    static constexpr int Boxes = D / 64;
    // operands of 16 bits: boxes of 64 columns, 128-byte swizzle
    static constexpr int QBox = 128 * 128, KBox = KR * 128, VBox = KT * 128;
    static constexpr int QBytes = Boxes * QBox, KBytes = Boxes * KBox, VBytes = Boxes * VBox;
    // 8 bits: the ring holds codes and scales, one pair of operand buffers the fp16 numbers
    static constexpr int Stages = D == 64 ? 4 : 2;
    static constexpr int RawK = KR * D, RawV = KT * D, RawS = KR * 8;
    static constexpr int StageBytes = Eight ? RawK + RawV + (RawS + 1023) / 1024 * 1024 : KBytes + VBytes;
    static constexpr int NV = Eight && D < 256 ? 2 : 1;  // buffers of turned values
    static constexpr int OffQ = 0, OffK = QBytes, OffV = OffK + KBytes;  // the operand buffers of 8-bit pools
    static constexpr int OffRing = Eight ? OffV + NV * VBytes : QBytes;
    // the sums of a part are joined on its queries, XC columns at a time
    static constexpr int XC = 128 * Halves * 32 * 4 <= QBytes ? 32 : 16, XBytes = 128 * Halves * XC * 4, OffX = OffQ;
    static_assert(XBytes <= QBytes, "the sums fit");
    static constexpr int OffScales = OffRing + Stages * StageBytes;  // [4 tiles][3][KR]
    static constexpr int Smem = OffScales + (Eight ? 4 * KR * 12 : 0) + 1024;
    static_assert(Blocks * (Smem + 4096) <= 227 * 1024, "shared memory");
    // tensor memory columns
    static constexpr int ColP = KR, ColO = KR + 32 * Halves;
    static constexpr int Columns = 512 / Blocks;
    static_assert(ColO + D * Halves <= Columns, "tensor memory");
};

__host__ __device__ constexpr uint32_t rows_idesc(bool bf16, int N, bool b_mn_major) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
           ((128u >> 4) << 24);
}

// What 16 columns weigh, times (ln 2)^2.  u: their logits and the one behind (log2 units less the maximum); Lc: the share
// that the interval before gives to the first, then that of the interval behind to the column behind.  first: columns
// below it end intervals that exist.  W: pairs of columns.
//
// An interval from u0 to u1, X = u1 - u0, p = 2^u, has the integral S and gives R to its left and S - R to its right column:
//   |X| >= 0.11   S ln 2 = (p1 - p0) / X,   R = ((p1 - p0) / X - p0 ln 2) / X
//   else          S ln 2 = (p0 + p1) (ln 2) / 2 * (1 - (X ln 2)^2 / 12),   R = (ln 2)^2 (2 p0 + p1) / 6 + its share of the rest
// as one sequence of operations with other coefficients.  The quotients make the exponentials' 2^-22 as much larger as X is
// small, twice over in R; the series leaves out (X ln 2)^2 / 72 of 1/2 in R, always towards the left, and less than 2^-21 of
// S.  Just above the border R is off by 2.1e-4 of itself and S by 8e-6 (2^-16.9) at most, just below it R by 1.7e-4; with the
// border at 1/16 these were 6.4e-4, 1.4e-5 (2^-16.2) and 5e-5, at 0.14 1.3e-4, 6e-6 and 2.7e-4.  The exponentials are mostly
// better than 2^-22: equal intervals of values -1 and 1 move o by up to 8e-5 above 1/16, by 5e-5 above 0.11.  What R gives too
// much to one row the other gets too little.
constexpr float kSeries = 0.11f;
template <bool MASKED>
__device__ __forceinline__ void weights16(const float (&u)[17], float &Lc, int columns, Two (&W)[8]) {
    constexpr float l1 = kLn2, l2 = l1 * l1;
    float p[17];
#pragma unroll
    for (int e = 0; e < 17; ++e) p[e] = ex2_approx(u[e]);
    float before = Lc;
#pragma unroll
    for (int e = 0; e < 16; e += 2) {  // intervals e and e + 1
        const float x0 = u[e] - u[e + 1], x1 = u[e + 1] - u[e + 2];  // -X
        const float i0 = rcp_approx(x0), i1 = rcp_approx(x1);
        const bool s0 = fabsf(x0) < kSeries, s1 = fabsf(x1) < kSeries;
        const Two x = two(x0, x1), P0 = two(p[e], p[e + 1]);
        const float g0 = s0 ? 1.0f : -1.0f, g1 = s1 ? 1.0f : -1.0f;
        float k0, k1;
        apart(fma2(x * x, both(-l1 * l2 / 24.0f), both(0.5f * l1)), k0, k1);
        const Two f1 = two(s0 ? k0 : i0, s1 ? k1 : i1), f2 = two(s0 ? -l1 / 3.0f : i0, s1 ? -l1 / 3.0f : i1);
        const Two a2 = fma2(two(g0, g1), both(0.75f * l1), both(-0.25f * l1));  // (ln 2) / 2 or -ln 2
        const Two S = two(fmaf(p[e + 1], g0, p[e]), fmaf(p[e + 2], g1, p[e + 1])) * f1;
        const Two R = fma2(P0, a2, S) * f2, L = fma2(S, both(l1), R);  // R: what the left gets, times -1
        float r0, r1, q0, q1;
        apart(R, r0, r1);
        apart(L, q0, q1);
        if (MASKED) {
            if (e + 1 >= columns) r0 = q0 = 0.0f;
            if (e + 2 >= columns) r1 = q1 = 0.0f;
        }
        W[e / 2] = two(before - r0, q0 - r1);
        before = q1;
    }
    Lc = before;
}

// Two weights as bf16 numbers hi + lo, right within 2^-16 of each.  The high part is cut off, so that neither is negative
// and the low one is at least 2^-23 of the weight: an infinite value stays one.
__device__ __forceinline__ void split(Two w, uint32_t &hi, uint32_t &lo) {
    float a, c, la, lc;
    apart(w, a, c);
    const uint32_t ua = __float_as_uint(a), uc = __float_as_uint(c);
    hi = __byte_perm(ua, uc, 0x7632);
    apart(fma2(w, both(1.00000011920928955f), two(-__uint_as_float(ua & 0xffff0000u), -__uint_as_float(uc & 0xffff0000u))), la, lc);
    lo = pack_bf16x2(la, lc);
}

// CW: a thread's columns of a half: 64 for 128 rows, 32 for two copies of 64, 16 for four of 32.
template <int D, int KIND, int CW>
__global__ void __launch_bounds__(RowsCfg<D, KIND>::Threads, RowsCfg<D, KIND>::Blocks)
rows_kernel(const __grid_constant__ PagedParams p, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
            const __grid_constant__ CUtensorMap map_k8) {
    using C = RowsCfg<D, KIND>;
    constexpr bool EIGHT = C::Eight, E4M3 = KIND == CSA_E4M3;
    constexpr int KT = C::KT, KR = C::KR, NS = C::Stages, H = C::Halves, R = 2 * CW;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t s_bars[4 * NS + 15];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_bad[8];
    __shared__ float s_lift[4], s_m[2 * 128], s_l[2 * 128];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t base = (smem_u32(raw) + 1023) / 1024 * 1024;
    uint8_t *smem = raw + (base - smem_u32(raw));
    long long *s_cut = reinterpret_cast<long long *>(smem + C::OffX);  // at the start only
    static_assert((C::Threads + 1) * 8 <= C::XBytes, "the cut fits");
    volatile int *abort_flag = &s_abort;
    // barriers: stages of the ring, full and empty, keys and values; then one each
    const uint32_t bars = smem_u32(s_bars);
    auto k_full = [&](int s) { return bars + 8 * s; };
    auto v_full = [&](int s) { return bars + 8 * (NS + s); };
    auto k_empty = [&](int s) { return bars + 8 * (2 * NS + s); };
    auto v_empty = [&](int s) { return bars + 8 * (3 * NS + s); };
    const uint32_t one = bars + 8 * 4 * NS;
    const uint32_t s_full = one, s_empty = one + 8, q_full = one + 16, k_ready = one + 24, k_free = one + 40,
                   drain = one + 56, joint = one + 96;
    auto v_ready = [&](int s) { return s == 0 ? one + 32 : one + 104; };
    auto v_free = [&](int s) { return s == 0 ? one + 48 : one + 112; };
    auto p_full = [&](int h) { return one + 64 + 8 * h; };
    auto o_done = [&](int h) { return one + 80 + 8 * h; };
    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(k_full(s), 1);
            mbar_init(v_full(s), 1);
            mbar_init(k_empty(s), EIGHT ? C::TurnWarps + 1 : 1);
            mbar_init(v_empty(s), EIGHT ? C::TurnWarps : 1);
        }
        mbar_init(s_full, 1);
        mbar_init(s_empty, C::SoftWarps);
        mbar_init(q_full, C::SoftWarps);
        mbar_init(k_ready, EIGHT ? C::TurnWarps + 1 : 1);
        mbar_init(k_free, 1);
        mbar_init(drain, 1);
        mbar_init(joint, C::SoftWarps);
        for (int h = 0; h < 2; ++h) {
            mbar_init(p_full(h), 4);
            mbar_init(o_done(h), 1);
            mbar_init(v_ready(h), EIGHT ? C::TurnWarps : 1);
            mbar_init(v_free(h), 1);
        }
        s_abort = 0;
        fence_mbar_init();
    }
    if (warp == C::MmaWarp) {
        csa_dev::tmem_alloc(smem_u32(&s_tmem), C::Columns);
        csa_dev::tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    after_previous();

    const int heads = p.Hkv * p.GB;
    const long long most = (long long)p.M * p.S;
    const Lengths lens = {p.seqlens, p.counts, p.T, most};
    auto wait = [&](uint32_t bar, int phase) {
        return mbar_wait_bounded(bar, phase & 1, abort_flag, &g_paged_status, kWaitLimitNs);
    };
    auto awake = [&](uint32_t bar, int phase) { return wait_awake(bar, phase & 1, abort_flag, &g_paged_status); };
    auto idle = [&](uint32_t bar, int phase) { return wait_asleep(bar, phase & 1, abort_flag, &g_paged_status); };
    // the range of this CTA, by every warp for itself
    Part now;
    Cut cut;
    long long u0 = 0, u1 = 0;
    const long long worker = blockIdx.x;
    bool some;
    {
        const bool few = p.B <= 32;
        const int lane_n = few && lane < p.B ? lens[lane] : 0;
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        long long lane_before = 0;
        cut = few ? form_cut_warp(lane_n, KT, most, heads, gridDim.x, C::PartCost, lane_before)
                  : form_cut(lens, p.B, KT, most, heads, gridDim.x, C::PartCost, s_cut);
        for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
            const int n = lens[b];
            if (n > 0 && n <= most) continue;
            for (int h = tid; h < heads; h += blockDim.x) p.joins[b * heads + h] = make_int4(-1, 0, 0, 0);
        }
        some = worker < cut.in_use;
        if (some) {
            u0 = quot(worker * cut.U, cut.in_use);
            u1 = quot((worker + 1) * cut.U, cut.in_use);
            some = u0 < u1;
        }
        if (some) {
            if (few) {
                now.b = __popc(__ballot_sync(0xffffffffu, lane < p.B && lane_before * heads <= u0)) - 1;
                now.s0 = __shfl_sync(0xffffffffu, lane_before, now.b) * heads;
                now.n = __shfl_sync(0xffffffffu, lane_n, now.b);
            } else {
                now.b = find_sequence(u0, cut, s_cut, lens, p.B, KT, most, heads, now.s0);
                now.n = lens[now.b];
            }
            now.tiles = tiles_of(now.n, KT, most);
            now.head = (int)quot(u0 - now.s0, cut.units(now.tiles));
            now.s0 += (long long)now.head * cut.units(now.tiles);
            clip(now, cut, u0, u1);
            if (now.tile >= now.last) some = next_part(now, cut, u0, u1, lens, KT, most, heads);
        }
    }
    if (p.B > 32) __syncthreads();  // the cut is read; what it lies on can be written
    auto next = [&]() { return next_part(now, cut, u0, u1, lens, KT, most, heads); };
    auto cached_head = [&](int head) { return p.GB == 1 ? head : head / p.GB; };

    if (warp < C::SoftWarps)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::SoftRegs));
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OtherRegs));
    if (some && warp < C::SoftWarps) {
        // ---------------------------------------------------------------- softmax
        const int h = warp >> 2, i = (warp & 3) * 32 + lane;  // half, lane of tensor memory
        const uint32_t at_lane = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + at_lane, tP = tmem + at_lane + C::ColP + 32 * h, tO = tmem + at_lane + C::ColO + D * h;
        const int rep = i / R, row = i - rep * R;  // a warp has one copy
        const int c0 = 64 * h + rep * CW;          // this thread's columns
        const float *ring = reinterpret_cast<const float *>(smem + C::OffScales);  // [4 tiles][of keys, of values, bounds][KR]
        {  // the other copies' columns of P stay as good as zero: 2^-126 over bf16 pools, as 0 times infinity is not infinity
            constexpr uint32_t z = EIGHT ? 0u : 0x00800080u;
            const uint32_t zero[8] = {z, z, z, z, z, z, z, z};
            for (int j = 0; j < 4; ++j) tm_st8(tP + 8 * j, zero);
            tmem_wait_st();
        }
        int tiles = 0, joints = 0;  // of this CTA so far
        bool ok = true;
        // barrier of the softmax warps, bounded as every wait; false: give up
        auto soft_sync = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(joint);
            return ok = __all_sync(0xffffffffu, wait(joint, joints++));
        };
        do {
            const int b = now.b, n = now.n, hk = cached_head(now.head), hb = now.head - hk * p.GB;
            const int rows_h = min(p.HB, p.G - hb * p.HB);
            const long long first = (long long)b * p.Hq + hk * p.G + hb * p.HB;
            const bool mine = row < rows_h;
            // the queries, copies side by side: this thread's half of row `row`; of a negative scale their opposites, so
            // that the largest product is the largest logit
            float unit = fabsf(p.qscale);
            const uint32_t flip = p.qscale < 0.0f ? 0x80008000u : 0u;
            {
                constexpr int N = D / 8 / H;  // chunks of 8
                const uint4 *qg = reinterpret_cast<const uint4 *>(p.q + (first + row) * D);
                uint4 x[N];
#pragma unroll
                for (int c = 0; c < N; ++c) x[c] = mine ? qg[h * N + c] : make_uint4(0u, 0u, 0u, 0u);
                if constexpr (EIGHT) {  // fp16 numbers, a row by the power of two that takes its largest to [2^14, 2^15)
                    uint32_t big = 0;
                    auto most = [&](const uint4 &y) {
                        for (uint32_t w : {y.x, y.y, y.z, y.w}) big = max(big, max(w & 0x7fffu, (w >> 16) & 0x7fffu));
                    };
#pragma unroll
                    for (int c = 0; c < N; ++c) most(x[c]);
                    if (mine && H > 1)
#pragma unroll
                        for (int c = 0; c < N; ++c) most(qg[(1 - h) * N + c]);
                    const uint32_t e2 = min(max(big >> 7, 16u), 254u);
                    const float up = __uint_as_float((268u - e2) << 23);
                    unit *= __uint_as_float((e2 - 14u) << 23);
                    auto turn = [&](uint32_t w) { return pack_f16x2(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up); };
#pragma unroll
                    for (int c = 0; c < N; ++c) x[c] = make_uint4(turn(x[c].x), turn(x[c].y), turn(x[c].z), turn(x[c].w));
                }
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const int c = h * N + k;
                    *reinterpret_cast<uint4 *>(smem + C::OffQ + (c >> 3) * C::QBox + i * 128 + (((c & 7) ^ (i & 7)) << 4)) =
                        make_uint4(x[k].x ^ flip, x[k].y ^ flip, x[k].z ^ flip, x[k].w ^ flip);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
            }
            const int r0 = now.tile * KT;
            float m = -INFINITY, l = 0.0f, w_sink = 0.0f, lift = 0.0f;
            float highest = -INFINITY;  // 8 bits: the largest logit, where m may be below it
            float carry = 0.0f;  // the logit before column 0, log2 units
            if (c0 == 0 && r0 == 0 && p.mode == CSA_K0_GIVEN && mine) {
                const uint4 *qg = reinterpret_cast<const uint4 *>(p.q + (first + row) * D), *kg = reinterpret_cast<const uint4 *>(p.k0 + (long long)hk * D);
                float sum = 0.0f;
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 x = qg[c], y = kg[c];
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sum = fmaf(__uint_as_float(xs[e] << 16), __uint_as_float(ys[e] << 16), sum);
                        sum = fmaf(__uint_as_float(xs[e] & 0xffff0000u), __uint_as_float(ys[e] & 0xffff0000u), sum);
                    }
                }
                carry = sum * p.qscale;
            }
            bool bad = false;
            // bf16: the low parts of the tile before's weights, for the second of its two products
            uint32_t low[EIGHT ? 1 : CW / 2];
            auto second = [&]() {  // false: give up
                if (!(ok = __all_sync(0xffffffffu, wait(o_done(h), 2 * tiles - 2)))) return false;
                tc_fence_after();
                if constexpr (!EIGHT) {
#pragma unroll
                    for (int e = 0; e < CW / 2; e += 8) {
                        const uint32_t part[8] = {low[e], low[e + 1], low[e + 2], low[e + 3], low[e + 4], low[e + 5], low[e + 6], low[e + 7]};
                        tm_st8(tP + rep * CW / 2 + e, part);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(h));
                return true;
            };
            // a tile; false: give up.  MASKED: not all of its intervals exist.
            auto tile = [&](int j, auto masked) -> bool {
                constexpr bool MASKED = decltype(masked)::value;
                if (!(ok = __all_sync(0xffffffffu, wait(s_full, tiles)))) return false;
                tc_fence_after();
                bad |= *(volatile int *)&s_bad[tiles & 7] != 0;
                const int own = n - j * KT;  // rows of this tile and behind it
                const float *sk = ring + (tiles & 3) * 3 * KR, *sv = sk + KR, *sb = sv + KR;
                const bool sink = j == 0 && c0 == 0, copied = sink && p.mode == CSA_K0_COPY_FIRST;
                // this thread's columns, up to 32 at a time, and their neighbours: all loads at once
                uint32_t xa[16], xb[16], behind, edge, tail;
                auto load = [&]() {
                    tm_ld16(tS + c0, xa);
                    if (CW >= 32) tm_ld16(tS + c0 + 16, xb);
                    tm_ld1(tS + c0 + (CW < 32 ? CW : 32), behind);
                    tm_ld1(tS + (c0 > 0 ? c0 - 1 : KR - 1), edge);
                    tm_ld1(tS + KT - 1, tail);
                };
                if (!(EIGHT && CW == 64)) load();  // those have no registers for 64 columns
                float high = -INFINITY;  // of products
                auto scaled = [&](uint32_t (&x)[16], int col) {  // 8 bits: times the cached rows' scales
                    if constexpr (EIGHT) {
                        const float4 *at = reinterpret_cast<const float4 *>(sk + col);
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            const float4 y = at[e / 4];
                            x[e] = __float_as_uint(__uint_as_float(x[e]) * y.x);
                            x[e + 1] = __float_as_uint(__uint_as_float(x[e + 1]) * y.y);
                            x[e + 2] = __float_as_uint(__uint_as_float(x[e + 2]) * y.z);
                            x[e + 3] = __float_as_uint(__uint_as_float(x[e + 3]) * y.w);
                        }
                    }
                };
                auto largest = [&](const uint32_t (&x)[16], int col) {
                    if (!MASKED || col + 16 <= own) {
                        float t[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            t[e] = fmaxf(__uint_as_float(x[4 * e]), __uint_as_float(x[4 * e + 1]));
                            t[e] = csa_tc::fmax3f(t[e], __uint_as_float(x[4 * e + 2]), __uint_as_float(x[4 * e + 3]));
                        }
                        high = csa_tc::fmax3f(high, csa_tc::fmax3f(t[0], t[1], t[2]), t[3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (col + e < own) high = fmaxf(high, __uint_as_float(x[e]));
                    }
                };
                if constexpr (CW == 64) {  // the other 32: their maximum only
                    uint32_t ya[16], yb[16], yn;
                    tm_ld16(tS + c0 + 32, ya);
                    tm_ld16(tS + c0 + 48, yb);
                    tm_ld1(tS + c0 + 64, yn);
                    tm_wait(ya);
                    tm_wait(yb);
                    tm_wait(yn);
                    scaled(ya, c0 + 32);
                    scaled(yb, c0 + 48);
                    largest(ya, c0 + 32);
                    largest(yb, c0 + 48);
                    if (EIGHT) yn = __float_as_uint(__uint_as_float(yn) * sk[c0 + 64]);
                    if (!MASKED || c0 + CW < own) high = fmaxf(high, __uint_as_float(yn));
                }
                if (EIGHT && CW == 64) load();
                tm_wait(xa);
                if (CW >= 32) tm_wait(xb);
                tm_wait(behind, edge, tail);
                auto all_read = [&]() {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_empty);
                };
                if (CW < 64) all_read();
                scaled(xa, c0);
                largest(xa, c0);
                if (CW >= 32) {
                    scaled(xb, c0 + 16);
                    largest(xb, c0 + 16);
                }
                if (EIGHT) {
                    behind = __float_as_uint(__uint_as_float(behind) * sk[c0 + (CW < 32 ? CW : 32)]);
                    edge = __float_as_uint(__uint_as_float(edge) * sk[c0 > 0 ? c0 - 1 : KR - 1]);
                    tail = __float_as_uint(__uint_as_float(tail) * sk[KT - 1]);
                }
                if (CW < 64 && (!MASKED || c0 + CW < own)) high = fmaxf(high, __uint_as_float(behind));
                // the logit before the first column; the tile's last one is the next tile's
                float before = carry;
                if (copied)
                    before = __uint_as_float(xa[0]) * unit;
                else if (c0 > 0 || (j == now.tile && r0 > 0))
                    before = __uint_as_float(edge) * unit;
                carry = __uint_as_float(tail) * unit;
                float top = high == -INFINITY ? high : high * unit;
                if (!MASKED || c0 < own) top = fmaxf(top, before);
                // A raised maximum, or another unit of the values: the sums of the tiles before follow.  8 bits: weights are
                // relative to 2^m such that the largest product with a scale is an fp16 number with all its bits.  Where scales
                // are far apart that is not the largest weight's, and in another unit what the rows before may have had counts
                // for less: m can be below the largest logit, by 2^80 at most, that the weights' sum stays finite.
                float f_lift = 1.0f, down = 0.0f;  // down: log2 of it
                bool uneven = false;
                if (EIGHT) {
                    const float its = s_lift[tiles & 3], to = fabsf(its);
                    uneven = its < 0.0f;
                    if (to != lift) {
                        if (j > now.tile) {
                            f_lift = to / lift;
                            down = (float)(((int)__float_as_uint(to) - (int)__float_as_uint(lift)) >> 23);
                        }
                        lift = to;
                    }
                }
                bool over = top > m + (EIGHT ? kRaise8 : kRaise);
                // The low parts of the tile before, when its first product is done: with 64 columns after the interval
                // before them (152 us for 32 drafted tokens as above, 164 here), else here (two places spill registers:
                // 112 us for 16 drafted, so 100)
                bool given = EIGHT || j == now.tile;
                auto give = [&]() { return given || (given = second()); };
                if (CW < 64 && !give()) return false;
                bool free = j == now.tile;  // PV of the tile before is done: P can be written, and O can change
                auto wait_free = [&]() {
                    if (!free) {
                        ok = __all_sync(0xffffffffu, wait(o_done(h), EIGHT ? tiles - 1 : 2 * tiles - 1));
                        tc_fence_after();
                        free = true;
                    }
                    return ok;
                };
                bool change = __any_sync(0xffffffffu, over || f_lift != 1.0f || uneven);
                if (EIGHT && change && (uneven || f_lift != 1.0f)) {
                    highest = fmaxf(highest, fmaxf(m, top));
                    if (uneven) {  // the logits with their rows' bounds, this thread's and the next; -infinity behind the end
                        top = before + sb[c0 > 0 ? c0 - 1 : KR - 1];
                        auto bound = [&](const uint32_t (&x)[16], int col) {
                            const float4 *at = reinterpret_cast<const float4 *>(sb + col);
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                const float4 y = at[e / 4];
                                float a = __uint_as_float(x[e]), b = __uint_as_float(x[e + 1]), c = __uint_as_float(x[e + 2]), d = __uint_as_float(x[e + 3]);
                                if constexpr (CW == 16) {
                                    apart(fma2(two(a, b), both(unit), two(y.x, y.y)), a, b);
                                    apart(fma2(two(c, d), both(unit), two(y.z, y.w)), c, d);
                                } else {
                                    a = fmaf(a, unit, y.x), b = fmaf(b, unit, y.y), c = fmaf(c, unit, y.z), d = fmaf(d, unit, y.w);
                                }
                                top = csa_tc::fmax3f(csa_tc::fmax3f(top, a, b), c, d);
                            }
                        };
                        if constexpr (CW == 64) {
                            uint32_t x[16], next;
                            tm_ld1(tS + c0 + 64, next);
                            tm_wait(next);
                            top = fmaxf(top, fmaf(__uint_as_float(next) * sk[c0 + 64], unit, sb[c0 + 64]));
#pragma unroll 1
                            for (int c = c0; c < c0 + CW; c += 16) {
                                tm_ld16(tS + c, x);
                                tm_wait(x);
                                scaled(x, c);
                                bound(x, c);
                            }
                        } else {
                            bound(xa, c0);
                            if (CW == 32) bound(xb, c0 + 16);
                            top = fmaxf(top, fmaf(__uint_as_float(behind), unit, sb[c0 + CW]));
                        }
                        over = top > m + kRaise8;
                        change = __any_sync(0xffffffffu, over || f_lift != 1.0f);
                    }
                }
                if (change) {
                    if ((CW == 64 && !give()) || !wait_free()) return false;
                    float to = over ? top : m;
                    if (EIGHT && f_lift != 1.0f) to = fmaxf(fmaxf(top, m + down), highest - 80.0f);
                    const float f = m == -INFINITY ? 0.0f : ex2_approx(m - to);
                    m = to;
                    l *= f;
                    w_sink *= f;
                    if (j > now.tile) {
                        const float fo = f * f_lift;
                        for (int c = 0; c < D; c += 16) {
                            uint32_t x[16];
                            tm_ld16(tO + c, x);
                            tm_wait(x);
                            uint32_t y[8], z[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                y[e] = __float_as_uint(__uint_as_float(x[e]) * fo);
                                z[e] = __float_as_uint(__uint_as_float(x[8 + e]) * fo);
                            }
                            tm_st8(tO + c, y);
                            tm_st8(tO + c + 8, z);
                        }
                        tmem_wait_st();
                    }
                }
                const float nm = m == -INFINITY ? 0.0f : -m;
                // the interval from the row before
                float Lc;
                {
                    float u[17];
                    u[0] = before + nm;
                    u[1] = fmaf(__uint_as_float(xa[0]), unit, nm);
                    const float x = u[1] - u[0], inv = rcp_approx(x), p0 = ex2_approx(u[0]), p1 = ex2_approx(u[1]);
                    const bool small = fabsf(x) < kSeries;
                    const float g = small ? 1.0f : -1.0f, a2 = small ? 0.5f * kLn2 : -kLn2;
                    const float S = fmaf(p0, g, p1) * (small ? 0.5f * kLn2 * fmaf(-kLn2 * kLn2 / 12.0f, x * x, 1.0f) : inv);
                    float left = fmaf(p0, a2, S) * (small ? kLn2 / 3.0f : inv);
                    Lc = fmaf(S, kLn2, -left);
                    if (MASKED && c0 >= own) Lc = left = 0.0f;
                    if (sink) {
                        if (copied) {
                            Lc += left;  // the sink's value is the first row's
                        } else {
                            w_sink = left;
                            l += left;
                        }
                    }
                }
                if (CW == 64 && !give()) return false;
                Two sum = both(0.0f);
                // `at`: of `low`
                auto chunk = [&](const uint32_t (&x)[16], uint32_t xn, int col, int at, uint32_t (&pk)[8]) {
                    float u[17];
#pragma unroll
                    for (int e = 0; e < 16; e += 2) apart(fma2(two(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), both(unit), both(nm)), u[e], u[e + 1]);
                    u[16] = fmaf(__uint_as_float(xn), unit, nm);
                    Two W[8];
                    weights16<MASKED>(u, Lc, own - col, W);
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum = sum + W[e];
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        if constexpr (EIGHT) {
                            const float4 y = *reinterpret_cast<const float4 *>(sv + col + 2 * e);
                            W[e] = W[e] * two(y.x, y.y);
                            W[e + 1] = W[e + 1] * two(y.z, y.w);
                        }
                        float a, c, d, f;
                        apart(W[e], a, c);
                        apart(W[e + 1], d, f);
                        if constexpr (EIGHT) {
                            pk[e] = pack_f16x2(a, c);
                            pk[e + 1] = pack_f16x2(d, f);
                        } else {
                            split(W[e], pk[e], low[at + e]);
                            split(W[e + 1], pk[e + 1], low[at + e + 1]);
                        }
                    }
                };
#pragma unroll 1
                for (int c = 0; c < CW; c += 32) {
                    if (c > 0) {
                        tm_ld16(tS + c0 + c, xa);
                        tm_ld16(tS + c0 + c + 16, xb);
                        tm_ld1(tS + c0 + c + 32, behind);
                        tm_wait(xa);
                        tm_wait(xb);
                        tm_wait(behind);
                        all_read();
                        scaled(xa, c0 + c);
                        scaled(xb, c0 + c + 16);
                        if (EIGHT) behind = __float_as_uint(__uint_as_float(behind) * sk[c0 + c + 32]);
                    }
                    auto store = [&](const uint32_t (&pk)[8], int col) {
                        if (!wait_free()) return false;
                        tm_st8(tP + (rep * CW + col) / 2, pk);
                        return true;
                    };
                    if constexpr (CW == 16) {
                        uint32_t pk[8];
                        chunk(xa, behind, c0, 0, pk);
                        if (!store(pk, 0)) return false;
                    } else if constexpr (EIGHT) {
                        // the second 16 by the first's instructions: with the turning and the scales two copies of them
                        // miss the instruction caches (16 sequences of 4096 to 8192 rows, 64 rows each: 156 us, so 131;
                        // bf16 pools have room for both, 89 us instead of 94)
#pragma unroll 1
                        for (int e = 0; e < 32; e += 16) {
                            uint32_t pk[8];
                            chunk(xa, e == 0 ? xb[0] : behind, c0 + c + e, 0, pk);
                            if (!store(pk, c + e)) return false;
#pragma unroll
                            for (int k = 0; k < 16; ++k) xa[k] = xb[k];
                        }
                    } else {
                        uint32_t pk[8], pl[8];
                        chunk(xa, xb[0], c0 + c, c / 2, pk);
                        chunk(xb, behind, c0 + c + 16, c / 2 + 8, pl);
                        if (!store(pk, c) || !store(pl, c + 16)) return false;
                    }
                }
                float sx, sy;
                apart(sum, sx, sy);
                l += sx + sy;
                if (!EIGHT && MASKED && own < KT) {  // rows behind the end: their weights are 0, and 0 * NaN is not
                    const int stage = tiles % NS;
                    if (!(ok = __all_sync(0xffffffffu, wait(v_full(stage), tiles / NS)))) return false;
                    uint8_t *vt = smem + C::OffRing + stage * C::StageBytes + C::KBytes;
                    const int t0 = tid & 127;
                    for (int k = t0; k < 64 * (D / 8); k += 128) {
                        const int r = 64 * h + k / (D / 8), c = k % (D / 8);
                        if (r >= own)
                            *reinterpret_cast<uint4 *>(vt + (c >> 3) * C::VBox + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(h));
                return true;
            };
            for (int j = now.tile; ok && j < now.last; ++j, ++tiles)
                if (!(n - j * KT > KT ? tile(j, std::false_type{}) : tile(j, std::true_type{}))) ok = false;
            if (!ok || (!EIGHT && !second())) break;
            if (!(ok = __all_sync(0xffffffffu, wait(o_done(h), EIGHT ? tiles - 1 : 2 * tiles - 1)))) break;
            tc_fence_after();
            // ---- the copies and halves of a row joined: maxima, then sums, XC columns at a time
            const bool all_rows = r0 == 0 && min(n, now.last * KT) == n;
            s_m[h * 128 + i] = m;
            s_l[h * 128 + i] = bad ? NAN : l;
            if (!soft_sync()) break;
            // the sources of a row: half s / reps, copy s mod reps
            constexpr int reps = 128 / R, sources = H * reps;
            auto source = [&](int s, int r) { return (s / reps) * 128 + (s % reps) * R + r; };
            float high = -INFINITY;
#pragma unroll
            for (int s = 0; s < sources; ++s) high = fmaxf(high, s_m[source(s, row)]);
            constexpr float kUnit = 1.0f / (kLn2 * kLn2);
            const float f = (high == -INFINITY ? 0.0f : ex2_approx(m - high)) * kUnit, fo = EIGHT ? f / lift : f;
            const long long slot = (all_rows ? 2 * row_workers(D) + (long long)b * heads + now.head : worker * 2 + (u0 < now.s0 ? 1 : 0)) * p.HB;
            if (tid < rows_h) {  // half 0, copy 0
                float total = 0.0f;
#pragma unroll
                for (int s = 0; s < sources; ++s) {
                    const float mm = s_m[source(s, row)], ll = s_l[source(s, row)];
                    // without a column: 0 or NaN
                    total += mm == -INFINITY ? ll : ll * ex2_approx(mm - high);
                }
                *reinterpret_cast<float2 *>(p.part_ml + 2 * (slot + row)) = make_float2(high, total * kUnit);
            }
            // X: rows of XC columns, their chunks of 16 bytes permuted by the row: eight lanes meet no bank twice
            float4 *X = reinterpret_cast<float4 *>(smem + C::OffX);
            constexpr int E = C::XC / 4;
            auto place = [&](int at, int e) { return at * E + (e ^ (E == 8 ? at & 7 : (at >> 1) & 3)); };
            const bool given = c0 == 0 && r0 == 0 && p.mode == CSA_K0_GIVEN;
            for (int c = 0; ok && c < D; c += C::XC) {
                uint32_t xa[16], xb[16];
                tm_ld16(tO + c, xa);
                if (E == 8) tm_ld16(tO + c + 16, xb);
                tm_wait(xa);
                if (E == 8) tm_wait(xb);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    float y[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        y[k] = fo == 0.0f ? 0.0f : __uint_as_float(e < 4 ? xa[(4 * e + k) & 15] : xb[(4 * e + k) & 15]) * fo;
                        if (given) y[k] = fmaf(w_sink * f, __bfloat162float(p.v0[(long long)hk * D + c + 4 * e + k]), y[k]);
                    }
                    X[place(h * 128 + i, e)] = make_float4(y[0], y[1], y[2], y[3]);
                }
                if (!soft_sync()) break;
                for (int k = tid; k < rows_h * E; k += 128 * H) {
                    const int r = k / E, e = k % E;
                    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int s = 0; s < sources; ++s) {
                        const float4 x = X[place(source(s, r), e)];
                        y.x += x.x;
                        y.y += x.y;
                        y.z += x.z;
                        y.w += x.w;
                    }
                    *reinterpret_cast<float4 *>(p.part_o + (slot + r) * D + c + 4 * e) = y;
                }
                soft_sync();  // read, before the next columns are written
            }
            if (!ok) break;
            if (bad && tid == 0) atomicCAS(&g_paged_status, 0, CSA_ERR_INVALID_ARG);
            if (r0 == 0 && tid == 0) {
                const long long end = now.s0 + cut.units(now.tiles);
                const int segment = b * heads + now.head;
                p.joins[segment] = make_int4(segment, all_rows ? -1 : (int)worker, (int)cut.worker_of(end - 1), u0 < now.s0 ? 1 : 0);
            }
            tc_fence_before();
        } while (next());
    } else if (some && warp == C::MmaWarp) {
        // ------------------------------------------------------------ tensor core
        constexpr uint32_t idesc_s = rows_idesc(!EIGHT, KR, false), idesc_o = rows_idesc(!EIGHT, D, true);
        int tiles_s = 0, tiles_o = 0, parts = 0;  // products issued, parts begun
        bool ok = true;
        // descriptors: an offset of n bytes is n / 16 more
        const uint64_t q_desc = csa_tc::make_sdesc(base + C::OffQ, 16, 1024);
        const uint64_t k_desc = csa_tc::make_sdesc(EIGHT ? base + C::OffK : base + C::OffRing, 16, 1024);
        const uint64_t v_desc = csa_tc::make_sdesc(EIGHT ? base + C::OffV : base + C::OffRing + C::KBytes, C::VBox, 1024);
        auto issue_s = [&]() {
            const int stage = tiles_s % NS;
            if (!awake(EIGHT ? k_ready : k_full(stage), EIGHT ? tiles_s : tiles_s / NS)) return false;
            if (!awake(s_empty, tiles_s + 1)) return false;
            tc_fence_after();
            const uint64_t kd = k_desc + (EIGHT ? 0 : stage * (C::StageBytes >> 4));
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
                tc_mma_ss(tmem, q_desc + (((k >> 2) * C::QBox + (k & 3) * 32) >> 4), kd + (((k >> 2) * C::KBox + (k & 3) * 32) >> 4),
                          idesc_s, k > 0 ? 1u : 0u);
            tc_commit(s_full);
            tc_commit(EIGHT ? k_free : k_empty(stage));
            ++tiles_s;
            return true;
        };
        do {
            if (lane == 0) {
                // the product of half h's weights with the values at vd, onto sums that there are already or not
                auto product = [&](int h, uint64_t vd, bool onto) {
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc_mma_ts(tmem + C::ColO + D * h, tmem + C::ColP + 32 * h + 8 * k, vd + (((64 * h + 16 * k) * 128) >> 4), idesc_o,
                                  onto || k > 0 ? 1u : 0u);
                    tc_commit(o_done(h));
                };
                ok = awake(q_full, parts) && issue_s();
                if constexpr (EIGHT) {
                    for (int j = now.tile; ok && j < now.last; ++j) {
                        if (j + 1 < now.last && !(ok = issue_s())) break;
                        const int buf = tiles_o % C::NV;
                        if (!(ok = awake(v_ready(buf), tiles_o / C::NV))) break;
                        for (int h = 0; h < H && ok; ++h)
                            if ((ok = awake(p_full(h), tiles_o))) product(h, v_desc + buf * (C::VBytes >> 4), j > now.tile);
                        if (!ok) break;
                        tc_commit(v_free(buf));
                        ++tiles_o;
                    }
                } else {  // the low parts of a tile's weights follow while the next one's logits are read
                    auto values = [&](int t) { return v_desc + t % NS * (C::StageBytes >> 4); };
                    auto second = [&]() {
                        if (!(ok = awake(p_full(0), 2 * tiles_o - 1))) return;
                        product(0, values(tiles_o - 1), true);
                        tc_commit(v_empty((tiles_o - 1) % NS));
                    };
                    for (int j = now.tile; ok && j < now.last; ++j) {
                        if (j > now.tile) second();
                        if (!ok || (j + 1 < now.last && !(ok = issue_s()))) break;
                        if (!(ok = awake(v_full(tiles_o % NS), tiles_o / NS) && awake(p_full(0), 2 * tiles_o))) break;
                        product(0, values(tiles_o), j > now.tile);
                        ++tiles_o;
                    }
                    if (ok) second();
                }
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            ++parts;
        } while (ok && next());
        if (lane == 0) {  // every product is done before the block can end
            tc_commit(drain);
            const uint64_t began = globaltimer_ns();
            while (!mbar_try_wait(drain, 0) && globaltimer_ns() - began < kWaitLimitNs) {
            }
        }
        __syncwarp();
    } else if (some && (warp == C::CopyWarp || warp == C::CopyWarp + 1)) {
        // ----------------------------------------------------------------- copies
        const bool values = warp != C::CopyWarp;  // else keys
        const int RP = p.R, pieces = KT / RP;     // rows per copy
        auto full = [&](int s) { return values ? v_full(s) : k_full(s); };
        auto empty = [&](int s) { return values ? v_empty(s) : k_empty(s); };
        // lane i < pieces: rows of the tile; of keys lane `pieces`: the 8 behind, and, for a part's first tile, the next: the 8 before
        const bool inside = lane < pieces;
        const int rows = inside ? RP : 8, to = inside ? lane * RP : lane == pieces ? KT : KT + 8;
        const int of_row = EIGHT ? D + (values ? 0 : 8) : 2 * D;
        // a lane's rows of a tile: where they begin in the pool, -1 for none, -2 on a page out of range
        auto look_up = [&](bool first) {
            const int j = now.tile, row = inside ? j * KT + lane * RP : lane == pieces ? (j + 1) * KT : j * KT - 8;
            const bool wanted = inside ? row < now.n : !values && (lane == pieces ? row < now.n : lane == pieces + 1 && first && row >= 0);
            if (!wanted) return -1;
            const int index = (int)__umul64hi((unsigned long long)row, p.s_inv), page = p.table[(long long)now.b * p.M + index];
            return page >= 0 && page < p.P ? (page * p.Hkv + cached_head(now.head)) * p.S + (row - index * p.S) : -2;
        };
        int copied = 0;
        bool ok = true, more = true;
        int from = look_up(true);
        while (more) {
            const int stage = copied % NS, here = from;
            const uint32_t at = base + C::OffRing + stage * C::StageBytes;
            // the next tile's pages are asked for before this one's stage is waited for
            const bool ends = ++now.tile == now.last;
            if (ends) more = next();
            if (more) from = look_up(ends);
            if (!(ok = __all_sync(0xffffffffu, idle(empty(stage), copied / NS + 1)))) break;
            const int bytes = __reduce_add_sync(0xffffffffu, here >= 0 ? rows * of_row : 0);
            const bool lost = __any_sync(0xffffffffu, here == -2);
            if (lane == 0) {
                if (!values) *(volatile int *)&s_bad[copied & 7] = lost;
                mbar_arrive_expect_tx(full(stage), bytes);
            }
            __syncwarp();
            if (here >= 0) {
                if constexpr (EIGHT) {
                    const uint8_t *src = static_cast<const uint8_t *>(values ? p.v : p.k) + (long long)here * D;
                    bulk_load(at + (values ? C::RawK : 0) + to * D, src, rows * D, full(stage));
                    if (!values) bulk_load(at + C::RawK + C::RawV + to * 8, p.scales + 2ll * here, rows * 8, full(stage));
                } else {
#pragma unroll
                    for (int c = 0; c < C::Boxes; ++c) {
                        if (values)
                            tma_load_3d(at + C::KBytes + c * C::VBox + to * 128, &map_v, 0, here, c, full(stage));
                        else
                            tma_load_3d(at + c * C::KBox + to * 128, inside ? &map_k : &map_k8, 0, here, c, full(stage));
                    }
                }
            }
            ++copied;
        }
        // the copies land before the block can end, whatever the others do
        __syncwarp();
        if (lane == 0)
            for (int t = max(0, copied - NS); t < copied; ++t) {
                const uint64_t began = globaltimer_ns();
                while (!mbar_try_wait(full(t % NS), (t / NS) & 1) && globaltimer_ns() - began < kWaitLimitNs) {
                }
            }
        __syncwarp();
    } else if (EIGHT && some && warp >= C::TurnWarp) {
        // ------------------------------------------- codes become fp16 numbers
        // (before the scales' warp: behind its instructions these miss the caches more often, 115 us instead of 111 for 16
        // drafted tokens as above, d = 256 217 instead of 206)
        if constexpr (EIGHT) {
            const int t = tid - 32 * C::TurnWarp;
            constexpr int T = 32 * C::TurnWarps, PerRow = D / 16, Step = T / PerRow;
            static_assert(Step % 8 == 0 && KT % Step == 0, "a thread has every Step-th row, alike in the swizzle");
            // 16 codes of row r, columns 16 c ..: two swizzled chunks of 16 bytes.  Of each pair of rows the odd boxes' lanes
            // have the other one, so that eight lanes meet no bank twice, neither reading nor writing.
            const int c = t % PerRow, t0 = (t / PerRow) ^ ((c >> 2) & 1);
            const uint32_t low = ((2 * (c & 3)) ^ (t0 & 7)) << 4;
            auto turn = [&](const uint4 &x, uint8_t *row) {
                uint4 y;
                halves_of<E4M3>(x.x, y.x, y.y);
                halves_of<E4M3>(x.y, y.z, y.w);
                *reinterpret_cast<uint4 *>(row + low) = y;
                halves_of<E4M3>(x.z, y.x, y.y);
                halves_of<E4M3>(x.w, y.z, y.w);
                *reinterpret_cast<uint4 *>(row + (low ^ 16)) = y;
            };
            // `rows` rows, the ones from `own` on as zeros; two of a thread's at a time
            auto turn_rows = [&](const uint8_t *src, uint8_t *box, int rows, int own) {
                src += t0 * D + c * 16;
                box += t0 * 128;
#pragma unroll 1
                for (int r = t0; r < rows; r += 2 * Step, src += 2 * T * 16, box += 2 * Step * 128) {
                    uint4 x[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        x[e] = r + e * Step < min(rows, own) ? *reinterpret_cast<const uint4 *>(src + e * T * 16) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (r + e * Step < rows) turn(x[e], box + e * Step * 128);
                }
            };
            bool ok = true;
            // Keys up to two tiles ahead of the values: the keys' buffer is free once the tile before has its logits, a
            // buffer of the values not before the sums of the tile that it held.  One loop for both, that their
            // instructions are in the caches once.
            Part ahead = now;
            int keys = 0, values = 0;
            bool more = true;
#pragma unroll 1
            while (true) {
                const bool k = more && keys <= values + 1;
                const int of = k ? keys : values, stage = of % NS, buf = of % C::NV;
                if (!(ok = __all_sync(0xffffffffu, idle(k ? k_full(stage) : v_full(stage), of / NS) &&
                                                       idle(k ? k_free : v_free(buf), (k ? of : of / C::NV) + 1))))
                    break;
                turn_rows(smem + C::OffRing + stage * C::StageBytes + (k ? 0 : C::RawK),
                          smem + (k ? C::OffK + (c >> 2) * C::KBox : C::OffV + buf * C::VBytes + (c >> 2) * C::VBox), k ? KR : KT,
                          k ? 1 << 30 : now.n - now.tile * KT);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(k ? k_ready : v_ready(buf));
                    mbar_arrive(k ? k_empty(stage) : v_empty(stage));
                }
                Part at = k ? ahead : now;
                const bool goes_on = ++at.tile < at.last || next_part(at, cut, u0, u1, lens, KT, most, heads);
                if (k) {
                    ++keys;
                    ahead = at;
                    more = goes_on;
                } else {
                    ++values;
                    now = at;
                    if (!goes_on) break;
                }
            }
        }
    } else if (EIGHT && some && warp == C::ScaleWarp) {
        // ------------------------------------------------- the cached rows' scales
        if constexpr (EIGHT) {
            float *ring = reinterpret_cast<float *>(smem + C::OffScales);
            int tiles = 0;
            float lift = 0.0f;
            bool ok = true;
            do {
                for (int j = now.tile; j < now.last; ++j, ++tiles) {
                    const int stage = tiles % NS, own = now.n - j * KT;
                    const float2 *rs = reinterpret_cast<const float2 *>(smem + C::OffRing + stage * C::StageBytes + C::RawK + C::RawV);
                    if (!(ok = __all_sync(0xffffffffu, idle(k_full(stage), tiles / NS) && idle(k_free, tiles + 1)))) break;
                    float2 x[(KR + 31) / 32];
                    float big = 0.0f, least = INFINITY;
#pragma unroll
                    for (int i = 0; i < (KR + 31) / 32; ++i) {
                        const int r = 32 * i + lane;
                        x[i] = r < KR ? rs[r] : make_float2(0.0f, 0.0f);
                        if (r < own && r < KT) {
                            big = fmaxf(big, fabsf(x[i].y));
                            least = fminf(least, fabsf(x[i].y));
                        }
                    }
                    // the unit of the values: see csa_paged.cuh; a new part, a new unit
                    big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));
                    least = __uint_as_float(__reduce_min_sync(0xffffffffu, __float_as_uint(least)));
                    if (j == now.tile || big * lift > kMostScale) {
                        // 2^kLift2 by the power of two at or above the largest
                        const uint32_t e2 = min(max((__float_as_uint(big) + 0x7fffffu) >> 23, 8u), 253u);
                        lift = __uint_as_float((254u + kLift2 - e2) << 23);
                    }
                    float *to = ring + (tiles & 3) * 3 * KR;
#pragma unroll
                    for (int i = 0; i < (KR + 31) / 32; ++i) {
                        const int r = 32 * i + lane;
                        if (r < KR) {
                            to[r] = x[i].x;
                            to[KR + r] = r < own && r < KT ? x[i].y * lift : 0.0f;
                        }
                    }
                    const bool uneven = least * lift < kLeastScale;
                    if (lane == 0) s_lift[tiles & 3] = uneven ? -lift : lift;
                    __syncwarp();
                    if (uneven) {
                        // what a logit's power may bring to its row's product and its neighbours', log2 over 2^kLift2; the
                        // last column is the row before the tile, whose power the first row's weight has
                        const float *sv = to + KR;
#pragma unroll 1
                        for (int r = lane; r < KR; r += 32) {
                            float y = fabsf(sv[r < KR - 1 ? r : 0]);
                            if (r < KR - 1) y = fmaxf(y, fmaxf(r > 0 ? fabsf(sv[r - 1]) : 0.0f, fabsf(sv[r + 1])));
                            to[2 * KR + r] = r < own || r == KR - 1 ? fmaxf(__log2f(y) - (float)kLift2, -80.0f) : -INFINITY;
                        }
                        __syncwarp();
                    }
                    if (lane == 0) {
                        mbar_arrive(k_ready);
                        mbar_arrive(k_empty(stage));
                    }
                }
            } while (ok && next());
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == C::MmaWarp) csa_dev::tmem_dealloc(tmem, C::Columns);
}

// [P * Hkv * S, D] bf16 as {64, rows, D / 64}, boxes of 64 columns and R rows.
inline bool encode_boxes(CUtensorMap *map, const void *ptr, long long rows, int D, int R) {
    auto fn = csa_tc::get_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)(D / 64)};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, 128};
    const cuuint32_t box[3] = {64, (cuuint32_t)R, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int KIND, int CW>
int launch_rows(PagedParams &p, cudaStream_t stream) {
    using C = RowsCfg<D, KIND>;
    p.R = C::KT;
    while (p.S % p.R != 0) p.R /= 2;  // S is a multiple of 8
    p.s_inv = ~0ull / p.S + 1;
    CUtensorMap maps[3] = {};
    if (!C::Eight) {
        const long long rows = (long long)p.P * p.Hkv * p.S;
        const void *some = p.q;  // no pool: no sequence has a valid page, and the maps are never used
        for (int i = 0; i < 3; ++i)
            if (!encode_boxes(&maps[i], rows ? i == 1 ? p.v : p.k : some, rows ? rows : 8, D, i == 2 ? 8 : p.R)) return CSA_ERR_CUDA;
    }
    const long long tiles = (long long)p.B * p.Hkv * p.GB * (((long long)p.M * p.S + C::KT - 1) / C::KT);
    const int most = C::Blocks * kGrid, grid = (int)(tiles < most ? (tiles < 1 ? 1 : tiles) : most);
    auto kern = rows_kernel<D, KIND, CW>;
    // the shares of the registers come out of those that the block is launched with; a query that fails is asked again by
    // the next call
    static std::atomic<bool> fits{false};
    cudaFuncAttributes attr;
    bool ready = fits.load(std::memory_order_relaxed);
    if (!ready && cudaFuncGetAttributes(&attr, kern) == cudaSuccess) {
        ready = 32 * C::SoftWarps * C::SoftRegs + (C::Threads - 32 * C::SoftWarps) * C::OtherRegs <= C::Threads * attr.numRegs;
        fits.store(ready, std::memory_order_relaxed);
    }
    if (!ready || cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::Smem) != cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) != cudaSuccess) {
        (void)cudaGetLastError();  // taken, or the next launch would report it too
        return CSA_ERR_CUDA;
    }
    if (launch_after_previous(kern, grid, C::Threads, C::Smem, stream, p, maps[0], maps[1], maps[2]) != cudaSuccess)
        return CSA_ERR_CUDA;
    return CSA_OK;
}

// Blocks of a group's rows, at most 128 each, as equal as can be.
inline int row_blocks(int rows) { return (rows + 127) / 128; }

template <int D, int KIND>
int launch_rows_of(PagedParams &p, cudaStream_t stream) {
    if (p.HB <= 32) return launch_rows<D, KIND, 16>(p, stream);
    if (p.HB <= 64) return launch_rows<D, KIND, 32>(p, stream);
    return launch_rows<D, KIND, 64>(p, stream);
}

template <int KIND>
int run_rows(const csa_paged_args &a, void *scratch, int d, cudaStream_t stream) {
    PagedParams p = paged_params(a);
    p.G = p.Hq / p.Hkv;
    p.GB = row_blocks(p.G);
    p.HB = (p.G + p.GB - 1) / p.GB;
    const long long segments = (long long)p.B * p.Hkv * p.GB;
    p.joins = static_cast<int4 *>(scratch);
    p.part_o = reinterpret_cast<float *>(p.joins + std::max(row_workers(d), segments));  // 16-byte aligned
    p.part_ml = p.part_o + (2 * row_workers(d) + segments) * p.HB * d;
    if (d == 64) return launch_rows_of<64, KIND>(p, stream);
    if (d == 128) return launch_rows_of<128, KIND>(p, stream);
    return launch_rows_of<256, KIND>(p, stream);
}

}  // namespace

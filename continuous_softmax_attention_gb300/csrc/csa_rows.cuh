// Many rows over a paged cache: the stretch before the draft of a tree of drafted
// tokens (csa_tree.cu) where a cached head has more than 16 rows, on tcgen05.  Rows,
// ranges and parts as in csa_paged.cuh; a block of up to 128 rows is a segment.
//
// A CTA per SM is a worker: a contiguous range of tiles of KT cached rows over all
// segments in a row.  Warps:
//   0-3, 4-7  softmax: a thread has one lane of tensor memory, and one half of the tile's
//             columns (at d = 256 there is one half: the sums of two do not fit)
//   then      the copies (one warp), the tensor core (one lane), and with 8-bit pools two
//             warps that turn codes into fp16 numbers
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
// for (5 of 11 parts of it at 64 rows).  The columns of the other shares in P are zeros
// from the start.
//
// What bounds it.  64 rows over bf16 rows of d = 128: HBM bandwidth and the softmax about
// alike (a tile of 128 rows is 64 KiB, 2.8 kcycles of an SM's share; its 8192 weights about
// 18 instructions each).  More rows: the weights.
//
// Weights are single 16-bit numbers, as csa_forward's: bf16 (2^-8) over bf16 pools, fp16
// (2^-11) over 8-bit ones.  All carry the factor (ln 2)^2, removed where parts are written.
#pragma once

#include "csa_paged.cuh"

namespace {

// TMEM: N consecutive columns of a thread's lane
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

template <int D, int KIND>
struct RowsCfg {
    static constexpr bool Eight = KIND != CSA_BF16;
    static constexpr int Halves = D == 256 ? 1 : 2;
    static constexpr int KT = 64 * Halves;   // cached rows per tile
    static constexpr int KR = KT + 16;       // and those of K: 8 behind, 8 before
    static constexpr int SoftWarps = 4 * Halves, CopyWarp = SoftWarps, MmaWarp = SoftWarps + 1;
    static constexpr int TurnWarps = Eight ? 2 : 0;
    static constexpr int Threads = 32 * (SoftWarps + 2 + TurnWarps);
    static constexpr int Boxes = D / 64;
    // operands of 16 bits: boxes of 64 columns, 128-byte swizzle
    static constexpr int QBox = 128 * 128, KBox = KR * 128, VBox = KT * 128;
    static constexpr int QBytes = Boxes * QBox, KBytes = Boxes * KBox, VBytes = Boxes * VBox;
    // 8 bits: the ring holds codes and scales, one pair of operand buffers the fp16 numbers
    static constexpr int Stages = Eight ? (D == 64 ? 4 : 2) : D == 64 ? 3 : 2;
    static constexpr int RawK = KR * D, RawV = KT * D, RawS = KR * 8;
    static constexpr int StageBytes = Eight ? RawK + RawV + (RawS + 1023) / 1024 * 1024 : KBytes + VBytes;
    static constexpr int OffQ = 0, OffK = QBytes, OffV = OffK + KBytes;  // the operand buffers of 8-bit pools
    static constexpr int OffRing = Eight ? OffV + VBytes : QBytes;
    static constexpr int XC = D == 256 ? 16 : 32;  // columns of the sums joined at a time
    static constexpr int OffX = OffRing + Stages * StageBytes;
    static constexpr int OffScales = OffX + 128 * Halves * (XC + 1) * 4;  // [4 tiles][KR] pairs
    static constexpr int Smem = OffScales + (Eight ? 4 * KR * 8 : 0) + 1024;
    static_assert(Smem <= 227 * 1024 - 4096, "one block per SM");
    // tensor memory columns
    static constexpr int ColP = KR, ColO = KR + 32 * Halves;
    static_assert(ColO + D * Halves <= 512, "tensor memory");
};

struct RowsParams {
    PagedParams p;
    int R;     // rows of a copy: 32, 64 or 128
};

__host__ __device__ constexpr uint32_t rows_idesc(bool bf16, int N, bool b_mn_major) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
           ((128u >> 4) << 24);
}

// Shares of two intervals, times (ln 2)^2: between u0 and u1 (log2 units less the maximum) with p = 2^u.
// |X| < 1.44 (a natural step of 1): the power series of phi2, below 6e-7 relative; its even and odd parts serve both ends.
__device__ __forceinline__ void shares(Two u0, Two u1, Two p0, Two p1, Two &left, Two &right) {
    constexpr float l1 = kLn2, l2 = l1 * l1, l3 = l2 * l1, l4 = l2 * l2, l5 = l4 * l1, l6 = l4 * l2, l7 = l6 * l1, l8 = l4 * l4, l9 = l8 * l1;
    const Two minus = both(-1.0f);
    const Two X = fma2(u0, minus, u1), y = X * X;
    Two even = fma2(both(l8 / 40320.0f), y, both(l6 / 720.0f));
    even = fma2(even, y, both(l4 / 24.0f));
    even = fma2(even, y, both(l2 / 2.0f));
    Two odd = fma2(both(l9 / 362880.0f), y, both(l7 / 5040.0f));
    odd = fma2(odd, y, both(l5 / 120.0f));
    odd = fma2(odd, y, both(l3 / 6.0f)) * X;
    float x0, x1;
    apart(X, x0, x1);
    const Two inv = two(rcp_approx(x0), rcp_approx(x1));
    const Two sig = fma2(p0, minus, p1) * inv;
    const Two lf = fma2(p0, both(-l1), sig) * inv, rf = fma2(sig, minus, p1 * both(l1)) * inv;
    const Two ln = p0 * (even + odd), rn = p1 * fma2(odd, minus, even);
    float a0, a1, b0, b1, c0, c1, d0, d1;
    apart(lf, a0, a1);
    apart(rf, b0, b1);
    apart(ln, c0, c1);
    apart(rn, d0, d1);
    const bool near0 = fabsf(x0) < kLog2e, near1 = fabsf(x1) < kLog2e;
    left = two(near0 ? c0 : a0, near1 ? c1 : a1);
    right = two(near0 ? d0 : b0, near1 ? d1 : b1);
}

template <int D, int KIND>
__global__ void __launch_bounds__(RowsCfg<D, KIND>::Threads, 1)
rows_kernel(const __grid_constant__ RowsParams rp, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
            const __grid_constant__ CUtensorMap map_k8) {
    using C = RowsCfg<D, KIND>;
    constexpr bool EIGHT = C::Eight, E4M3 = KIND == CSA_E4M3;
    constexpr int KT = C::KT, KR = C::KR, NS = C::Stages, H = C::Halves;
    const PagedParams &p = rp.p;
    extern __shared__ uint8_t raw[];
    __shared__ long long s_cut[C::Threads + 1];
    __shared__ __align__(8) uint64_t s_bars[4 * NS + 13];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_bad[8];
    __shared__ float s_lift[4], s_m[2 * 128], s_l[2 * 128];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t base = (smem_u32(raw) + 1023) / 1024 * 1024;
    uint8_t *smem = raw + (base - smem_u32(raw));
    volatile int *abort_flag = &s_abort;
    // barriers: stages of the ring, full and empty, keys and values; then one each
    const uint32_t bars = smem_u32(s_bars);
    auto k_full = [&](int s) { return bars + 8 * s; };
    auto v_full = [&](int s) { return bars + 8 * (NS + s); };
    auto k_empty = [&](int s) { return bars + 8 * (2 * NS + s); };
    auto v_empty = [&](int s) { return bars + 8 * (3 * NS + s); };
    const uint32_t one = bars + 8 * 4 * NS;
    const uint32_t s_full = one, s_empty = one + 8, q_full = one + 16, k_ready = one + 24, v_ready = one + 32, k_free = one + 40,
                   v_free = one + 48, drain = one + 56, joint = one + 96;
    auto p_full = [&](int h) { return one + 64 + 8 * h; };
    auto o_done = [&](int h) { return one + 80 + 8 * h; };
    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(k_full(s), 1);
            mbar_init(v_full(s), 1);
            mbar_init(k_empty(s), EIGHT ? C::TurnWarps : 1);
            mbar_init(v_empty(s), EIGHT ? C::TurnWarps : 1);
        }
        mbar_init(s_full, 1);
        mbar_init(s_empty, C::SoftWarps);
        mbar_init(q_full, C::SoftWarps);
        mbar_init(k_ready, C::TurnWarps > 0 ? C::TurnWarps : 1);
        mbar_init(v_ready, C::TurnWarps > 0 ? C::TurnWarps : 1);
        mbar_init(k_free, 1);
        mbar_init(v_free, 1);
        mbar_init(drain, 1);
        mbar_init(joint, C::SoftWarps);
        for (int h = 0; h < 2; ++h) {
            mbar_init(p_full(h), 4);
            mbar_init(o_done(h), 1);
        }
        s_abort = 0;
        fence_mbar_init();
    }
    if (warp == C::MmaWarp) {
        csa_dev::tmem_alloc(smem_u32(&s_tmem), 512);
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
        cut = few ? form_cut_warp(lane_n, KT, most, heads, gridDim.x, lane_before)
                  : form_cut(lens, p.B, KT, most, heads, gridDim.x, s_cut);
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
    auto next = [&]() { return next_part(now, cut, u0, u1, lens, KT, most, heads); };
    auto cached_head = [&](int head) { return p.GB == 1 ? head : head / p.GB; };

    if (some && warp < C::SoftWarps) {
        // ---------------------------------------------------------------- softmax
        const int h = warp >> 2, i = (warp & 3) * 32 + lane;  // half, lane of tensor memory
        const uint32_t at_lane = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + at_lane, tP = tmem + at_lane + C::ColP + 32 * h, tO = tmem + at_lane + C::ColO + D * h;
        const int R = rp.R, rep = i / R, row = i - rep * R;  // a warp has one copy
        const int CW = 64 * R / 128, c0 = 64 * h + rep * CW;  // this thread's columns
        const float2 *ring = reinterpret_cast<const float2 *>(smem + C::OffScales);
        {  // the other copies' columns of P stay zero
            const uint32_t zero[8] = {};
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
            // the queries, copies side by side: this thread's half of row `row`
            float unit = p.qscale;
            {
                const uint4 *qg = reinterpret_cast<const uint4 *>(p.q + (first + row) * D);
                float up = 1.0f;
                if constexpr (EIGHT) {  // fp16 numbers, a row by the power of two that takes its largest to [2^14, 2^15)
                    uint32_t big = 0;
                    if (mine)
                        for (int c = 0; c < D / 8; ++c) {
                            const uint4 x = qg[c];
                            for (uint32_t w : {x.x, x.y, x.z, x.w}) big = max(big, max(w & 0x7fffu, (w >> 16) & 0x7fffu));
                        }
                    const uint32_t e2 = min(max(big >> 7, 16u), 254u);
                    up = __uint_as_float((268u - e2) << 23);
                    unit *= __uint_as_float((e2 - 14u) << 23);
                }
#pragma unroll 4
                for (int c = h * (D / 8 / H); c < (h + 1) * (D / 8 / H); ++c) {
                    uint4 x = mine ? qg[c] : make_uint4(0u, 0u, 0u, 0u);
                    if constexpr (EIGHT) {
                        auto turn = [&](uint32_t w) { return pack_f16x2(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up); };
                        x = make_uint4(turn(x.x), turn(x.y), turn(x.z), turn(x.w));
                    }
                    *reinterpret_cast<uint4 *>(smem + C::OffQ + (c >> 3) * C::QBox + i * 128 + (((c & 7) ^ (i & 7)) << 4)) = x;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
            }
            const int r0 = now.tile * KT;
            float m = -INFINITY, l = 0.0f, w_sink = 0.0f, lift = 0.0f;
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
            for (int j = now.tile; j < now.last; ++j, ++tiles) {
                if (!(ok = __all_sync(0xffffffffu, wait(s_full, tiles)))) break;
                tc_fence_after();
                bad |= *(volatile int *)&s_bad[tiles & 7] != 0;
                const int own = n - j * KT;  // rows of this tile and behind it
                const float2 *sc = ring + (tiles & 3) * KR;
                // a logit in log2 units
                auto logit = [&](uint32_t x, int col) {
                    return EIGHT ? __uint_as_float(x) * sc[col].x * unit : __uint_as_float(x) * unit;
                };
                // the maximum over this thread's columns and their neighbours
                uint32_t edge;
                float before = carry, top;
                if (c0 > 0) {
                    tm_ld1(tS + c0 - 1, edge);
                    tm_wait(edge);
                    before = logit(edge, c0 - 1);
                } else if (j == now.tile && r0 > 0) {
                    tm_ld1(tS + KR - 1, edge);
                    tm_wait(edge);
                    before = logit(edge, KR - 1);
                }
                const bool sink = j == 0 && c0 == 0, copied = sink && p.mode == CSA_K0_COPY_FIRST;
                top = copied || (c0 > 0 && c0 - 1 >= own) ? -INFINITY : before;
                for (int c = 0; c < CW; c += 16) {
                    uint32_t x[16];
                    tm_ld16(tS + c0 + c, x);
                    tm_wait(x);
                    float t = -INFINITY;
                    if (c0 + CW <= own) {
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float a = logit(x[e], c0 + c + e), a1 = logit(x[e + 1], c0 + c + e + 1);
                            t = csa_tc::fmax3f(t, a, a1);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (c0 + c + e < own) t = fmaxf(t, logit(x[e], c0 + c + e));
                    }
                    top = fmaxf(top, t);
                    if (copied && c == 0) before = logit(x[0], 0);
                }
                uint32_t behind;
                tm_ld1(tS + c0 + CW, behind);
                tm_wait(behind);
                const float last_a = logit(behind, c0 + CW);
                if (c0 + CW < own) top = fmaxf(top, last_a);
                // a raised maximum: the sums of the tiles before follow it
                float f_lift = 1.0f;
                if (EIGHT) {
                    const float to = s_lift[tiles & 3];
                    if (to != lift) {
                        f_lift = j > now.tile ? to / lift : 1.0f;
                        lift = to;
                    }
                }
                const bool over = top > m + (EIGHT ? kRaise8 : kRaise);
                if (j > now.tile) {  // PV of the tile before is done: P is free, and O can change
                    if (!(ok = __all_sync(0xffffffffu, wait(o_done(h), tiles - 1)))) break;
                    tc_fence_after();
                }
                if (__any_sync(0xffffffffu, over || f_lift != 1.0f)) {
                    const float to = over ? top : m, f = m == -INFINITY ? 0.0f : ex2_approx(m - to);
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
                // the interval from the row before: its right share
                float Lc;
                {
                    uint32_t x0;
                    tm_ld1(tS + c0, x0);
                    tm_wait(x0);
                    const float a = logit(x0, c0) + nm, bf = before + nm, pa = ex2_approx(a), pb = ex2_approx(bf);
                    Two left, right;
                    shares(both(bf), both(a), both(pb), both(pa), left, right);
                    float lft, none;
                    apart(left, lft, none);
                    apart(right, Lc, none);
                    if (c0 >= own) Lc = lft = 0.0f;
                    if (sink) {
                        if (copied)
                            Lc += lft;  // the sink's value is the first row's
                        else
                            w_sink = lft, l += lft;
                    }
                }
                Two sum = both(0.0f);
#pragma unroll 1
                for (int c = 0; c < CW; c += 16) {
                    uint32_t x[16], xn;
                    tm_ld16(tS + c0 + c, x);
                    tm_ld1(tS + c0 + c + 16, xn);
                    tm_wait(x);
                    tm_wait(xn);
                    if (c + 16 == CW) {  // all of S is read
                        if (c0 == 0) {  // the tile's last logit is the next tile's row before
                            uint32_t y;
                            tm_ld1(tS + KT - 1, y);
                            tm_wait(y);
                            carry = logit(y, KT - 1);
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(s_empty);
                    }
                    float u[17], pw[17], sv[16];
                    if constexpr (EIGHT) {
                        const float4 *sp = reinterpret_cast<const float4 *>(sc + c0 + c);
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float4 y = sp[e / 2];
                            u[e] = fmaf(__uint_as_float(x[e]) * y.x, unit, nm);
                            u[e + 1] = fmaf(__uint_as_float(x[e + 1]) * y.z, unit, nm);
                            sv[e] = y.y;
                            sv[e + 1] = y.w;
                        }
                        u[16] = fmaf(__uint_as_float(xn) * sc[c0 + c + 16].x, unit, nm);
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) u[e] = fmaf(__uint_as_float(x[e]), unit, nm);
                        u[16] = fmaf(__uint_as_float(xn), unit, nm);
                    }
#pragma unroll
                    for (int e = 0; e < 17; ++e) pw[e] = ex2_approx(u[e]);
                    const bool masked = own <= c0 + c + 16;
                    Two W[8];
                    float to_next = 0.0f, held_y = 0.0f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {  // intervals e and e + 8
                        Two left, right;
                        shares(two(u[e], u[e + 8]), two(u[e + 1], u[e + 9]), two(pw[e], pw[e + 8]), two(pw[e + 1], pw[e + 9]), left, right);
                        if (masked) {
                            float a, d, f, g;
                            apart(left, a, d);
                            apart(right, f, g);
                            if (c0 + c + e + 1 >= own) a = f = 0.0f;
                            if (c0 + c + e + 9 >= own) d = g = 0.0f;
                            left = two(a, d);
                            right = two(f, g);
                        }
                        if (e == 0)
                            W[0] = left;
                        else
                            W[e] = left + W[e];
                        if (e < 7) {
                            W[e + 1] = right;
                        } else {
                            apart(right, held_y, to_next);
                        }
                    }
                    W[0] = W[0] + two(Lc, held_y);
                    Lc = to_next;
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum = sum + W[e];
                    if constexpr (EIGHT) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) W[e] = W[e] * two(sv[e], sv[e + 8]);
                    }
                    float wx[8], wy[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) apart(W[e], wx[e], wy[e]);
                    uint32_t pk[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        pk[e] = EIGHT ? pack_f16x2(wx[2 * e], wx[2 * e + 1]) : pack_bf16x2(wx[2 * e], wx[2 * e + 1]);
                        pk[4 + e] = EIGHT ? pack_f16x2(wy[2 * e], wy[2 * e + 1]) : pack_bf16x2(wy[2 * e], wy[2 * e + 1]);
                    }
                    tm_st8(tP + (rep * CW + c) / 2, pk);
                }
                float sx, sy;
                apart(sum, sx, sy);
                l += sx + sy;
                if (!EIGHT && own < KT) {  // rows behind the end: their weights are 0, and 0 * NaN is not
                    const int stage = tiles % NS;
                    if (!(ok = __all_sync(0xffffffffu, wait(v_full(stage), tiles / NS)))) break;
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
            }
            if (!ok) break;
            if (!(ok = __all_sync(0xffffffffu, wait(o_done(h), tiles - 1)))) break;
            tc_fence_after();
            // ---- the copies and halves of a row joined: maxima, then sums, XC columns at a time
            const bool all_rows = r0 == 0 && min(n, now.last * KT) == n;
            s_m[h * 128 + i] = m;
            s_l[h * 128 + i] = bad ? NAN : l;
            if (!soft_sync()) break;
            float high = -INFINITY;
            for (int k = 0; k < H; ++k)
                for (int c = row; c < 128; c += R) high = fmaxf(high, s_m[k * 128 + c]);
            constexpr float kUnit = 1.0f / (kLn2 * kLn2);
            const float f = (high == -INFINITY ? 0.0f : ex2_approx(m - high)) * kUnit, fo = EIGHT ? f / lift : f;
            const long long slot = (all_rows ? 2 * kGrid + (long long)b * heads + now.head : worker * 2 + (u0 < now.s0 ? 1 : 0)) * p.HB;
            if (tid < rows_h) {  // half 0, copy 0
                float total = 0.0f;
                for (int k = 0; k < H; ++k)
                    for (int c = row; c < 128; c += R) {
                        const float mm = s_m[k * 128 + c];
                        total += s_l[k * 128 + c] * (mm == -INFINITY ? (isnan(s_l[k * 128 + c]) ? 1.0f : 0.0f) : ex2_approx(mm - high));
                    }
                *reinterpret_cast<float2 *>(p.part_ml + 2 * (slot + row)) = make_float2(high, total * kUnit);
            }
            float *X = reinterpret_cast<float *>(smem + C::OffX);
            const bool given = c0 == 0 && r0 == 0 && p.mode == CSA_K0_GIVEN;
            for (int c = 0; ok && c < D; c += C::XC) {
#pragma unroll
                for (int k = 0; k < C::XC; k += 16) {
                    uint32_t x[16];
                    tm_ld16(tO + c + k, x);
                    tm_wait(x);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float y = __uint_as_float(x[e]) * fo;
                        if (given) y = fmaf(w_sink * f, __bfloat162float(p.v0[(long long)hk * D + c + k + e]), y);
                        X[(h * 128 + i) * (C::XC + 1) + k + e] = y;
                    }
                }
                if (!soft_sync()) break;
                for (int k = tid; k < rows_h * C::XC; k += 128 * H) {
                    const int r = k / C::XC, e = k - r * C::XC;
                    float y = 0.0f;
                    for (int s = 0; s < H; ++s)
                        for (int t = r; t < 128; t += R) y += X[(s * 128 + t) * (C::XC + 1) + e];
                    p.part_o[(slot + r) * D + c + e] = y;
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
    } else if (some && warp == C::CopyWarp) {
        // ----------------------------------------------------------------- copies
        const int RP = p.R, pieces = KT / RP;  // rows per copy
        auto page_of = [&](int b, int row) {
            const int index = row / p.S, page = p.table[(long long)b * p.M + index];
            return page >= 0 && page < p.P ? (long long)page * p.Hkv * p.S + (row - index * p.S) : -1ll;
        };
        int tiles = 0;
        bool ok = true;
        do {
            const int hk = cached_head(now.head);
            for (int j = now.tile; j < now.last; ++j, ++tiles) {
                const int stage = tiles % NS, round = tiles / NS;
                const uint32_t at = base + C::OffRing + stage * C::StageBytes;
                // lane i < pieces: rows of the tile; lane `pieces`: the 8 behind; the next: the 8 before
                const int row = lane < pieces ? j * KT + lane * RP : lane == pieces ? (j + 1) * KT : j * KT - 8;
                const bool wanted = lane < pieces + 1 ? row < now.n : lane == pieces + 1 && j == now.tile && row >= 0;
                long long from = wanted ? page_of(now.b, row) : -1;
                const bool lost = wanted && from < 0;
                if (from >= 0) from += (long long)hk * p.S;
                const bool inside = lane < pieces;
                const int rows = inside ? RP : 8, to = inside ? lane * RP : lane == pieces ? KT : KT + 8;
                int bytes = from >= 0 ? rows * D * (EIGHT ? 1 : 2) : 0;
                int kb = bytes + (EIGHT && from >= 0 ? 8 * rows : 0), vb = inside ? bytes : 0;
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) {
                    kb += __shfl_xor_sync(0xffffffffu, kb, off);
                    vb += __shfl_xor_sync(0xffffffffu, vb, off);
                }
                const bool any_lost = __any_sync(0xffffffffu, lost);
                if (!(ok = __all_sync(0xffffffffu, wait(k_empty(stage), round + 1)))) break;
                if (lane == 0) {
                    *(volatile int *)&s_bad[tiles & 7] = any_lost;
                    mbar_arrive_expect_tx(k_full(stage), kb);
                }
                __syncwarp();
                if (from >= 0) {
                    if constexpr (EIGHT) {
                        bulk_load(at + to * D, static_cast<const uint8_t *>(p.k) + from * D, rows * D, k_full(stage));
                        bulk_load(at + C::RawK + C::RawV + to * 8, p.scales + 2 * from, rows * 8, k_full(stage));
                    } else {
#pragma unroll
                        for (int c = 0; c < C::Boxes; ++c)
                            tma_load_3d(at + c * C::KBox + to * 128, inside ? &map_k : &map_k8, 0, (int)from, c, k_full(stage));
                    }
                }
                if (!(ok = __all_sync(0xffffffffu, wait(v_empty(stage), round + 1)))) {
                    ++tiles;  // its keys are on their way
                    break;
                }
                if (lane == 0) mbar_arrive_expect_tx(v_full(stage), vb);
                __syncwarp();
                if (inside && from >= 0) {
                    if constexpr (EIGHT) {
                        bulk_load(at + C::RawK + to * D, static_cast<const uint8_t *>(p.v) + from * D, rows * D, v_full(stage));
                    } else {
#pragma unroll
                        for (int c = 0; c < C::Boxes; ++c)
                            tma_load_3d(at + C::KBytes + c * C::VBox + to * 128, &map_v, 0, (int)from, c, v_full(stage));
                    }
                }
            }
        } while (ok && next());
        // the copies land before the block can end, whatever the others do
        __syncwarp();
        if (lane == 0)
            for (int t = max(0, tiles - NS); t < tiles; ++t) {
                const uint64_t began = globaltimer_ns();
                while (!(mbar_try_wait(k_full(t % NS), (t / NS) & 1) && mbar_try_wait(v_full(t % NS), (t / NS) & 1)) &&
                       globaltimer_ns() - began < kWaitLimitNs) {
                }
            }
        __syncwarp();
    } else if (some && warp == C::MmaWarp) {
        // ------------------------------------------------------------ tensor core
        constexpr uint32_t idesc_s = rows_idesc(!EIGHT, KR, false), idesc_o = rows_idesc(!EIGHT, D, true);
        int tiles_s = 0, tiles_o = 0, parts = 0;  // products issued, parts begun
        bool ok = true;
        const uint32_t sQ = base + C::OffQ;
        auto issue_s = [&]() {
            const int stage = tiles_s % NS;
            if (!wait(EIGHT ? k_ready : k_full(stage), EIGHT ? tiles_s : tiles_s / NS)) return false;
            if (!wait(s_empty, tiles_s + 1)) return false;
            tc_fence_after();
            const uint32_t kb = EIGHT ? base + C::OffK : base + C::OffRing + stage * C::StageBytes;
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
                tc_mma_ss(tmem, csa_tc::make_sdesc(sQ + (k >> 2) * C::QBox + (k & 3) * 32, 16, 1024),
                          csa_tc::make_sdesc(kb + (k >> 2) * C::KBox + (k & 3) * 32, 16, 1024), idesc_s, k > 0 ? 1u : 0u);
            tc_commit(s_full);
            tc_commit(EIGHT ? k_free : k_empty(stage));
            ++tiles_s;
            return true;
        };
        do {
            if (lane == 0) {
                ok = wait(q_full, parts) && issue_s();
                for (int j = now.tile; ok && j < now.last; ++j) {
                    if (j + 1 < now.last && !(ok = issue_s())) break;
                    const int stage = tiles_o % NS;
                    if (!(ok = wait(EIGHT ? v_ready : v_full(stage), EIGHT ? tiles_o : tiles_o / NS))) break;
                    const uint32_t vb = EIGHT ? base + C::OffV : base + C::OffRing + stage * C::StageBytes + C::KBytes;
                    for (int h = 0; h < H && ok; ++h) {
                        if (!(ok = wait(p_full(h), tiles_o))) break;
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc_mma_ts(tmem + C::ColO + D * h, tmem + C::ColP + 32 * h + 8 * k,
                                      csa_tc::make_sdesc(vb + (64 * h + 16 * k) * 128, C::VBox, 1024), idesc_o,
                                      j > now.tile || k > 0 ? 1u : 0u);
                        tc_commit(o_done(h));
                    }
                    if (!ok) break;
                    tc_commit(EIGHT ? v_free : v_empty(stage));
                    ++tiles_o;
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
    } else if (EIGHT && some) {
        // ------------------------------------------- codes become fp16 numbers
        if constexpr (EIGHT) {
            const int t = tid - 32 * (C::SoftWarps + 2);
            constexpr int T = 32 * C::TurnWarps, PerRow = D / 16;
            float2 *ring = reinterpret_cast<float2 *>(smem + C::OffScales);
            int tiles = 0;
            float lift = 0.0f;
            bool ok = true;
            // 16 codes of row r, columns 16 c ..: two swizzled chunks of 16 bytes.  The odd boxes' second chunk goes
            // first, so that eight lanes meet no bank twice.
            auto turn = [&](const uint8_t *src, uint8_t *dst, int box_bytes, int r, int c) {
                const uint4 x = *reinterpret_cast<const uint4 *>(src);
                uint4 y[2];
                halves_of<E4M3>(x.x, y[0].x, y[0].y);
                halves_of<E4M3>(x.y, y[0].z, y[0].w);
                halves_of<E4M3>(x.z, y[1].x, y[1].y);
                halves_of<E4M3>(x.w, y[1].z, y[1].w);
                uint8_t *box = dst + (c >> 2) * box_bytes + r * 128;
                const int k = (c >> 2) & 1;
                *reinterpret_cast<uint4 *>(box + (((2 * (c & 3) + k) ^ (r & 7)) << 4)) = k ? y[1] : y[0];
                *reinterpret_cast<uint4 *>(box + (((2 * (c & 3) + 1 - k) ^ (r & 7)) << 4)) = k ? y[0] : y[1];
            };
            do {
                for (int j = now.tile; j < now.last; ++j, ++tiles) {
                    const int stage = tiles % NS, round = tiles / NS, own = now.n - j * KT;
                    const uint8_t *rk = smem + C::OffRing + stage * C::StageBytes, *rv = rk + C::RawK;
                    const float2 *rs = reinterpret_cast<const float2 *>(rv + C::RawV);
                    if (!(ok = __all_sync(0xffffffffu, wait(k_full(stage), round) && wait(k_free, tiles + 1)))) break;
                    // the unit of the values: see csa_paged.cuh
                    float big = 0.0f;
                    for (int r = lane; r < KT; r += 32)
                        if (r < own) big = fmaxf(big, rs[r].y);
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
                    if (j == now.tile || big * lift > 2.0f * kLift) {
                        const uint32_t e2 = min(max((__float_as_uint(big) + 0x7fffffu) >> 23, 12u), 253u);
                        lift = __uint_as_float((265u - e2) << 23);
                    }
                    for (int r = t; r < KR; r += T) {
                        const float2 s = rs[r];
                        ring[(tiles & 3) * KR + r] = make_float2(s.x, r < own && r < KT ? s.y * lift : 0.0f);
                    }
                    if (t == 0) s_lift[tiles & 3] = lift;
                    for (int k = t; k < KR * PerRow; k += T) {
                        const int r = k / PerRow, c = k - r * PerRow;
                        turn(rk + r * D + 16 * c, smem + C::OffK, C::KBox, r, c);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(k_ready);
                        mbar_arrive(k_empty(stage));
                    }
                    if (!(ok = __all_sync(0xffffffffu, wait(v_full(stage), round) && wait(v_free, tiles + 1)))) break;
                    for (int k = t; k < KT * PerRow; k += T) {
                        const int r = k / PerRow, c = k - r * PerRow;
                        if (r < own) {
                            turn(rv + r * D + 16 * c, smem + C::OffV, C::VBox, r, c);
                        } else {
                            uint8_t *box = smem + C::OffV + (c >> 2) * C::VBox + r * 128;
                            *reinterpret_cast<uint4 *>(box + (((2 * (c & 3)) ^ (r & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                            *reinterpret_cast<uint4 *>(box + (((2 * (c & 3) + 1) ^ (r & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(v_ready);
                        mbar_arrive(v_empty(stage));
                    }
                }
            } while (ok && next());
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == C::MmaWarp) csa_dev::tmem_dealloc(tmem, 512);
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

template <int D, int KIND>
int launch_rows(RowsParams &rp, cudaStream_t stream) {
    using C = RowsCfg<D, KIND>;
    PagedParams &p = rp.p;
    p.R = C::KT;
    while (p.S % p.R != 0) p.R /= 2;  // S is a multiple of 8
    CUtensorMap maps[3] = {};
    if (!C::Eight) {
        const long long rows = (long long)p.P * p.Hkv * p.S;
        const void *some = p.q;  // no pool: no sequence has a valid page, and the maps are never used
        for (int i = 0; i < 3; ++i)
            if (!encode_boxes(&maps[i], rows ? i == 1 ? p.v : p.k : some, rows ? rows : 8, D, i == 2 ? 8 : p.R)) return CSA_ERR_CUDA;
    }
    const long long tiles = (long long)p.B * p.Hkv * p.GB * (((long long)p.M * p.S + C::KT - 1) / C::KT);
    const int grid = (int)(tiles < kGrid ? (tiles < 1 ? 1 : tiles) : kGrid);
    auto kern = rows_kernel<D, KIND>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::Smem) != cudaSuccess ||
        launch_after_previous(kern, grid, C::Threads, C::Smem, stream, rp, maps[0], maps[1], maps[2]) != cudaSuccess)
        return CSA_ERR_CUDA;
    return CSA_OK;
}

// Blocks of a group's rows, at most 128 each, as equal as can be.
inline int row_blocks(int rows) { return (rows + 127) / 128; }

template <int KIND>
int run_rows(const csa_paged_args &a, void *scratch, int d, cudaStream_t stream) {
    RowsParams rp = {};
    PagedParams &p = rp.p;
    p = paged_params(a);
    p.G = p.Hq / p.Hkv;
    p.GB = row_blocks(p.G);
    p.HB = (p.G + p.GB - 1) / p.GB;
    rp.R = p.HB <= 32 ? 32 : p.HB <= 64 ? 64 : 128;
    const long long segments = (long long)p.B * p.Hkv * p.GB;
    p.joins = static_cast<int4 *>(scratch);
    p.part_ml = reinterpret_cast<float *>(p.joins + std::max((long long)kGrid, segments));
    p.part_o = p.part_ml + (2 * kGrid + segments) * p.HB * 2;
    if (d == 64) return launch_rows<64, KIND>(rp, stream);
    if (d == 128) return launch_rows<128, KIND>(rp, stream);
    return launch_rows<256, KIND>(rp, stream);
}

}  // namespace

// Decode step of causal continuous softmax attention over a paged cache: for
// every sequence b and query head, the newest token's query against the sink
// and the n_b cached rows of the head's group (eq. (10)/(11) of "Continuous
// Softmax Attention", the single row t = n_b).
//
// Between neighbouring logits a and a' = a + x the interval gives the key at a
// the weight e^{a-m} phi2(x) and the key at a' the weight e^{a'-m} phi2(-x)
// (eq. (9)); with p = e^{a-m} and p' = e^{a'-m} these are ((p'-p)/x - p)/x and
// (p' - (p'-p)/x)/x.  A key's weight is the sum over its two intervals, so a
// row's weight is complete once the next row's logit is known.
//
// What bounds it: the cached rows are read once, HBM bandwidth.  What follows
// from that:
//  - A warp (at d = 256 two, in step) is a worker of its own.  It has a ring of
//    tiles in shared memory that it fills itself by TMA (one lane), runs over a
//    contiguous range of tiles and never waits for another worker, so some
//    worker's copies are always in flight: 192 KiB of rings per SM.
//  - The tiles of all (sequence, cached head, block of query heads) in a row
//    are cut into equal ranges, one per worker, whatever the lengths.  The
//    lengths are on the device, so every block forms the cut itself.
//  - The query heads of a group are the rows of the matrix instruction (16, of
//    which 8 are used for up to 8 heads), the cached rows its columns, so one
//    read of a cached row serves up to 16 heads of the group.  A larger group is
//    cut into equal blocks of heads, each a segment with copies of the rows of
//    its own: 537 MB of 8 cached heads at d = 128 take 97 us with 16 query heads
//    each, 167 with 20 and 169 with 32.  mma.sync rather than
//    tcgen05: with 16 rows at most the products take a few percent of the time
//    either way, and mma.sync leaves logits and sums in the registers of the
//    warp that needs them.
//  - The weights enter the second product as a sum of two bf16 numbers, right
//    within 2^-16 of the weight, the high part cut off so that neither is
//    negative and the low one at least 2^-23 of the weight: an infinite value
//    stays one.  For up to 8 heads both halves fit one instruction: rows 0..7
//    hold the high parts and rows 8..15 the low ones.  Their sum, the
//    denominator, is that of the fp32 weights.  Two numbers put o off by 5e-6 of
//    its norm before it is rounded to bf16, and that rounding by 1.6e-3.  A third
//    number makes the weights exact: o is then off by 2e-7 to 4e-7 before the
//    rounding and by the same 1.6e-3 after it, one output in 250 being a bf16
//    step away from what two numbers give.  It takes 122.8 us in place of 118.5
//    (537 MB, 16 heads per group, d = 64), 98.2 of 97.2 (d = 128), 113.9 of 107.6
//    (d = 256), 60.4 of 59.8 (64 ragged sequences), 5.8 of 5.7 (one short one):
//    two numbers are kept.
//  - Few short sequences are bound by latency: a cluster of blocks then does one
//    cached head of one sequence in a single launch and joins its parts through
//    distributed shared memory (8.7 -> 5.8 us for 32 heads of 333 tokens).
//  - Otherwise a part of a sequence leaves its unnormalised sums, maximum and
//    weight sum in the workspace; a second kernel, launched early, joins the
//    parts in order.  A sequence that one worker had whole is written at once.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "csa.h"
#include "csa_device.cuh"
#include "csa_internal.h"
#include "csa_launch.cuh"
#include "csa_tc_common.cuh"

namespace {

using namespace csa_dev;

constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s
// One block per SM.  Workers do not wait for one another: a part with fewer SMs
// gives the same results, its last blocks in a second wave.
constexpr int kGrid = 152;
// Tiles per worker up to which latency counts: a worker per tile and no cost of
// a part.  1024 sequences of 17 tokens x 4 heads (3.4 tiles a worker) take 21 us
// with 2 here and 25 us with 4 or 8.
constexpr int kFew = 2;
// What beginning and ending a part costs, in tiles: with it a range of many
// short sequences takes as long as one of a long sequence.  64 ragged sequences
// of 1 to 8192 tokens take 63.1 us with 1, 59.7 with 2, 59.5 with 3, 32 of 333
// tokens 14.4, 13.4 and 14.2 us.
constexpr int kPartCost = 2;
// The one-kernel form: clusters of 1, 2, 4 and 8 blocks that run at a time ...
constexpr int kOneAtATime[4] = {152, 76, 36, 15};
// ... and tiles per warp that the longest sequence may have in it, where it
// keeps at least 3/4 of the SMs busy and where it does not.  Measured, this
// form and the other, equal lengths: 32 heads of 2048 tokens (4 tiles per warp,
// 128 SMs) 9.3 and 14 us, of 8192 (16) 26 and 30 us; 8 heads of 4096 (4, 64
// SMs) 9.6 and 9.6 us, of 8192 (8) 13.5 and 12.8 us; one head of 16384 (16, 8
// SMs) 22.5 and 15.8 us.  A batch of one long sequence among short ones waits
// for the long one's cluster, 0.5 us a tile, where the other form would spread
// it: hence no more than 16.
constexpr int kOneTiles = 16, kOneTilesLess = 4;
constexpr float kRaise = 16.0f;   // log2 units a logit may pass the running maximum by

__device__ int g_paged_status;  // sticky status word of this file's kernels

// RH: query heads per block / 8, rounded up (1 or 2).
template <int D, int RH>
struct Cfg {
    static constexpr int KT = 16;                      // rows per tile
    // Workers per block.  At d = 64 twelve: 16 of 128 registers spill with 16 heads (92 us for 268
    // MB, 75 us with 12), and with 8 there are more parts to join (2 x 131072 tokens 33.4 us, 31.4
    // with 12).
    static constexpr int Workers = D == 64 ? 12 : 1024 / D;
    // Warps of a worker: at d = 256 two, each for half of the output's columns and both for all
    // logits: the sums of one warp alone would be 128 registers, and it would spill.  537 MB of 128
    // cached heads with 8 and 16 query heads each take 92 and 108 us, 97 and 139 with one warp, 32
    // heads of 333 tokens 7.8 and 8.6.  At d = 128 (6 workers of two) it is slower: 103 and 143 us, 89
    // and 98 with one.
    static constexpr int Pair = D == 256 ? 2 : 1;
    static constexpr int Warps = Workers * Pair;
    static constexpr int Stages = D == 64 ? 4 : 3;     // tiles in a worker's ring
    static constexpr int Tile = KT * D * 2;            // bytes of a tile of keys, or of values
    static constexpr int Stage = 2 * Tile;
    static constexpr int Smem = Workers * Stages * Stage + 1024;  // + alignment
    static_assert(Smem <= 227 * 1024 - 6144, "one block per SM");
};

// Workers of a full grid, at most.
__host__ __device__ constexpr long long workers(int d) { return (d == 64 ? 12 : 1024 / d) * kGrid; }

struct PagedParams {
    const __nv_bfloat16 *q, *k, *v, *k0, *v0;
    const int *table, *seqlens;
    __nv_bfloat16 *out;
    float *lse;
    float *part_o;    // [2 * workers][HB][D]: unnormalised sums of a part
    float *part_ml;   // [2 * workers][HB][2]: its maximum (log2 units) and weight sum
    // the segments (heads of sequences) that several workers share: {segment or -1, first worker,
    // last worker, the first one's slot}, by segment or by the worker that begins one
    int4 *joins;      // [workers]
    int by_segment;
    int cluster;      // blocks per segment of the one-kernel form
    unsigned long long s_inv;  // 2^64 / S rounded up: row / S is the high word of row * s_inv
    int B, Hq, Hkv, P, S, M;
    int G, GB, HB;    // query heads of a group, blocks of them, heads per block
    int R;            // rows per copy: divides S and the tile
    float qscale;     // scale * log2(e): logits come out in log2 units
    int mode;
};

// Two fp32 numbers that one instruction works on.
struct Two {
    uint64_t v;
};
__device__ __forceinline__ Two two(float a, float b) {
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ Two both(float a) { return two(a, a); }
__device__ __forceinline__ void apart(Two x, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v));
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// The weights that two intervals, between logits a0 and b0 and between a1 and
// b1 (log2 units), give their two keys each, with p = 2^{a-m} and r = 2^{b-m}.
// |x| < 1 (natural units): the power series sum x^j/(j+2)!, j = 0..9, truncated
// below 5.3e-9 relative (at x = -1), split into its even and odd terms, which the two keys
// share.
__device__ __forceinline__ void intervals(float a0, float b0, float a1, float b1, float p0, float r0, float p1,
                                          float r1, float &left0, float &right0, float &left1, float &right1) {
    const Two minus = both(-1.0f), p = two(p0, p1), r = two(r0, r1);
    const Two x = fma2(two(a0, a1), minus, two(b0, b1)) * both(kLn2), y = x * x;
    Two even = both(2.755731922398589e-07f);                    // 1/10!
    even = fma2(even, y, both(2.48015873015873e-05f));          // 1/8!
    even = fma2(even, y, both(1.388888888888889e-03f));         // 1/6!
    even = fma2(even, y, both(4.166666666666667e-02f));         // 1/4!
    even = fma2(even, y, both(0.5f));                           // 1/2!
    Two odd = both(2.505210838544172e-08f);                     // 1/11!
    odd = fma2(odd, y, both(2.755731922398589e-06f));           // 1/9!
    odd = fma2(odd, y, both(1.984126984126984e-04f));           // 1/7!
    odd = fma2(odd, y, both(8.333333333333333e-03f));           // 1/5!
    odd = fma2(odd, y, both(1.666666666666667e-01f)) * x;       // 1/3!
    float x0, x1;
    apart(x, x0, x1);
    const Two inv = two(rcp_approx(x0), rcp_approx(x1));
    const Two s = fma2(p, minus, r) * inv;
    float ln0, ln1, rn0, rn1, lf0, lf1, rf0, rf1;
    apart(p * (even + odd), ln0, ln1);
    apart(r * fma2(odd, minus, even), rn0, rn1);
    apart(fma2(p, minus, s) * inv, lf0, lf1);
    apart(fma2(s, minus, r) * inv, rf0, rf1);
    const bool near0 = fabsf(x0) < 1.0f, near1 = fabsf(x1) < 1.0f;
    left0 = near0 ? ln0 : lf0;
    right0 = near0 ? rn0 : rf0;
    left1 = near1 ? ln1 : lf1;
    right1 = near1 ? rn1 : rf1;
}

// D (+)= A B, 16 x 8 x 16, bf16 in, fp32 out.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ int tiles_of(int n, int KT, long long most) {
    return n < 0 || n > most ? 0 : (int)(((long long)n + KT - 1) / KT);
}

// a / b for a >= 0, b > 0, mostly of 32 bits.
__device__ __forceinline__ long long quot(long long a, long long b) {
    return (a | b) >> 32 ? a / b : (long long)((unsigned)a / (unsigned)b);
}

// The cut of the work into ranges.  A unit is a tile of one cached head or, in
// a large batch, a share of a part's cost: each (sequence, head) then counts
// for its tiles and `cost` units in front of them.
struct Cut {
    long long U, in_use;  // units of all heads, workers in use
    int cost;
    __device__ __forceinline__ int units(int tiles) const { return tiles > 0 ? tiles + cost : 0; }
    // the worker that has unit u
    __device__ __forceinline__ long long worker_of(long long u) const { return quot((u + 1) * in_use - 1, U); }
};

// at[0 .. blockDim.x] gets the units (per head) of the sequences before each
// thread's chunk of sequences, the last entry the total.  Whole block.
__device__ Cut form_cut(const int *seqlens, int B, int KT, long long most, int heads, long long all, long long *at) {
    const int tid = threadIdx.x, per = (B + blockDim.x - 1) / blockDim.x;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    long long tiles = 0;
    int some = 0;  // sequences with tiles
    for (int b = b0; b < b1; ++b) {
        const int t = tiles_of(seqlens[b], KT, most);
        tiles += t;
        some += t > 0;
    }
    __shared__ long long tile_sums[32];
    __shared__ int some_sums[32];
    long long s = tiles;
    int c = some;
    const int lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, s, off);
        const int oc = __shfl_up_sync(0xffffffffu, c, off);
        if (lane >= off) {
            s += o;
            c += oc;
        }
    }
    if (lane == 31) {
        tile_sums[warp] = s;
        some_sums[warp] = c;
    }
    __syncthreads();
    long long before = 0, total = 0;
    int some_before = 0, some_total = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp) {
            before += tile_sums[w];
            some_before += some_sums[w];
        }
        total += tile_sums[w];
        some_total += some_sums[w];
    }
    Cut cut;
    cut.cost = total * heads > kFew * all ? kPartCost : 0;
    at[tid] = before + s - tiles + (long long)cut.cost * (some_before + c - some);
    if (tid == (int)blockDim.x - 1) at[blockDim.x] = total + (long long)cut.cost * some_total;
    __syncthreads();
    cut.U = at[blockDim.x] * heads;
    cut.in_use = cut.U < all ? cut.U : all;  // few tiles: a worker each
    return cut;
}

// The sequence that holds unit u, and the units before it.  Whole warp.
__device__ __forceinline__ int find_sequence(long long u, const Cut &cut, const long long *at, const int *seqlens,
                                             int B, int KT, long long most, int heads, long long &before) {
    // the last chunk that begins at or before u (chunks without units begin where the next one does)
    int begun = 0;
    for (int i = threadIdx.x & 31; i < (int)blockDim.x; i += 32) begun += __popc(__ballot_sync(0xffffffffu, at[i] * heads <= u));
    int b = (begun - 1) * ((B + blockDim.x - 1) / blockDim.x);
    before = at[begun - 1] * heads;
    while (true) {
        const long long mine = (long long)cut.units(tiles_of(seqlens[b], KT, most)) * heads;
        if (u < before + mine) return b;
        before += mine;
        ++b;
    }
}

// The cut of up to 32 sequences by a warp on its own, without a barrier of the
// block: lane b holds the units (per head) before sequence b.
__device__ __forceinline__ Cut form_cut_warp(int n, int KT, long long most, int heads, long long all,
                                             long long &before) {
    const int lane = threadIdx.x & 31, tiles = tiles_of(n, KT, most);
    const unsigned some = __ballot_sync(0xffffffffu, tiles > 0);
    long long s = tiles;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += o;
    }
    const long long total = __shfl_sync(0xffffffffu, s, 31);
    Cut cut;
    cut.cost = total * heads > kFew * all ? kPartCost : 0;
    before = s - tiles + cut.cost * __popc(some & ((1u << lane) - 1));
    cut.U = (total + cut.cost * __popc(some)) * heads;
    cut.in_use = cut.U < all ? cut.U : all;
    return cut;
}

// A worker's units [u0, u1) as parts: tiles [tile, last) of one head of one
// sequence each.
struct Part {
    int b, head, n, tiles, tile, last;
    long long s0;  // the segment's first unit
};

__device__ __forceinline__ void clip(Part &t, const Cut &cut, long long u0, long long u1) {
    t.tile = (int)max(0LL, u0 - t.s0 - cut.cost);
    t.last = (int)min((long long)t.tiles, max(0LL, u1 - t.s0 - cut.cost));
}

// The next part with tiles; false behind the last.
__device__ __forceinline__ bool next_part(Part &t, const Cut &cut, long long u0, long long u1, const int *seqlens,
                                          int KT, long long most, int heads) {
    do {
        t.s0 += cut.units(t.tiles);
        if (t.s0 >= u1) return false;
        if (++t.head == heads) {
            t.head = 0;
            do {
                t.n = seqlens[++t.b];
                t.tiles = tiles_of(t.n, KT, most);
            } while (t.tiles == 0);
        }
        clip(t, cut, u0, u1);
    } while (t.tile >= t.last);
    return true;
}

// Barrier over the blocks of a cluster.
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float2 cluster_load(uint32_t addr, int rank) {  // 8 bytes of another block's shared memory
    float2 v;
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
}

// ONE: a cluster of p.cluster blocks does one segment (a cached head of one
// sequence and a block of its query heads), cut over its warps, and joins the
// parts itself through shared memory: one launch, for few segments of bounded
// length.  Otherwise the cut over all workers described above.
template <int D, int RH, bool ONE>
__global__ void __launch_bounds__(Cfg<D, RH>::Warps * 32, 1)
paged_kernel(const __grid_constant__ PagedParams p, const __grid_constant__ CUtensorMap map_k,
             const __grid_constant__ CUtensorMap map_v) {
    using C = Cfg<D, RH>;
    constexpr int KT = C::KT, NT = KT / 8, KS = D / 16, kStages = C::Stages;
    constexpr int DW = D / C::Pair, ON = DW / 8;  // columns of the output that a warp forms
    extern __shared__ uint8_t raw[];
    __shared__ long long s_cut[ONE ? 1 : C::Warps * 32 + 1];
    __shared__ __align__(8) uint64_t bars[C::Workers][kStages];
    __shared__ int s_abort[C::Workers];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    const int heads = p.Hkv * p.GB;
    const long long most = (long long)p.M * p.S;
    const int mine = warp / C::Pair, half_of = warp % C::Pair;  // worker in the block, warp of the worker
    volatile int *abort_flag = &s_abort[mine];
    // the warps of a worker
    auto sync_worker = [&]() {
        if (C::Pair == 1)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(1 + mine), "n"(32 * C::Pair) : "memory");
    };

    if (lane == 0 && half_of == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(smem_u32(&bars[mine][s]), 1);
        fence_mbar_init();
        s_abort[mine] = 0;
    }
    sync_worker();
    after_previous();
    Part now;
    Cut cut = {};
    long long worker = 0, u0 = 0, u1 = 0;
    int parts = 1;           // of this segment (ONE)
    bool working = true;     // whether this warp has one (ONE)
    const int rank = ONE ? (int)(blockIdx.x % p.cluster) : 0;
    if constexpr (ONE) {
        const int segment = blockIdx.x / p.cluster;
        now.b = segment / heads;
        now.head = segment - now.b * heads;
        now.n = p.seqlens[now.b];
        now.tiles = tiles_of(now.n, KT, most);
        now.s0 = 0;
        if (now.tiles == 0) {  // no rows, or a length out of range: all blocks of the cluster leave
            const int hk = p.GB == 1 ? now.head : now.head / p.GB, hb = now.head - hk * p.GB;
            const long long first = (long long)now.b * p.Hq + hk * p.G + hb * p.HB;
            const int rows_h = min(p.HB, p.G - hb * p.HB);
            if (rank == 0) {
                for (int i = threadIdx.x; i < rows_h * D; i += blockDim.x)
                    p.out[first * D + i] = __float2bfloat16_rn(now.n == 0 ? 0.0f : NAN);
                if (p.lse)
                    for (int h = threadIdx.x; h < rows_h; h += blockDim.x)
                        p.lse[first + h] = now.n == 0 ? -INFINITY : NAN;
                if (threadIdx.x == 0 && now.n != 0) atomicCAS(&g_paged_status, 0, CSA_ERR_INVALID_ARG);
            }
            return;
        }
        // parts across blocks first
        parts = min(C::Workers * p.cluster, now.tiles);
        const int part = mine * p.cluster + rank;
        working = part < parts;
        now.tile = working ? (int)quot((long long)part * now.tiles, parts) : 0;
        now.last = working ? (int)quot((long long)(part + 1) * now.tiles, parts) : 1;
    } else {
        const bool few = p.B <= 32;  // sequences: every warp forms the cut
        const int lane_n = few && lane < p.B ? p.seqlens[lane] : 0;
        // the join's blocks may take their places as this kernel's blocks end
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        const long long all = (long long)C::Workers * gridDim.x;
        long long lane_before = 0;
        cut = few ? form_cut_warp(lane_n, KT, most, heads, all, lane_before)
                  : form_cut(p.seqlens, p.B, KT, most, heads, all, s_cut);
        // sequences without rows, and lengths out of range
        for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
            const int n = p.seqlens[b];
            if (n > 0 && n <= most) continue;
            const float v = n == 0 ? 0.0f : NAN;
            for (int i = threadIdx.x; i < p.Hq * D; i += blockDim.x)
                p.out[(long long)b * p.Hq * D + i] = __float2bfloat16_rn(v);
            if (p.lse)
                for (int h = threadIdx.x; h < p.Hq; h += blockDim.x)
                    p.lse[(long long)b * p.Hq + h] = n == 0 ? -INFINITY : NAN;
            if (p.by_segment)
                for (int h = threadIdx.x; h < heads; h += blockDim.x) p.joins[b * heads + h] = make_int4(-1, 0, 0, 0);
            if (threadIdx.x == 0 && n != 0) atomicCAS(&g_paged_status, 0, CSA_ERR_INVALID_ARG);
        }

        // workers are numbered across blocks first, so that few of them spread over all SMs
        worker = (long long)mine * gridDim.x + blockIdx.x;
        if (lane == 0 && half_of == 0 && !p.by_segment) p.joins[worker] = make_int4(-1, 0, 0, 0);
        if (worker >= cut.in_use) return;
        u0 = quot(worker * cut.U, cut.in_use);
        u1 = quot((worker + 1) * cut.U, cut.in_use);
        if (u0 >= u1) return;

        // ---- position in the range: what is copied next, and what is consumed
        if (few) {  // the last sequence that begins at or before u0
            now.b = __popc(__ballot_sync(0xffffffffu, lane < p.B && lane_before * heads <= u0)) - 1;
            now.s0 = __shfl_sync(0xffffffffu, lane_before, now.b) * heads;
            now.n = __shfl_sync(0xffffffffu, lane_n, now.b);
        } else {
            now.b = find_sequence(u0, cut, s_cut, p.seqlens, p.B, KT, most, heads, now.s0);
            now.n = p.seqlens[now.b];
        }
        now.tiles = tiles_of(now.n, KT, most);
        now.head = (int)quot(u0 - now.s0, cut.units(now.tiles));  // hk * GB + block of query heads
        now.s0 += (long long)now.head * cut.units(now.tiles);
        clip(now, cut, u0, u1);
        if (now.tile >= now.last && !next_part(now, cut, u0, u1, p.seqlens, KT, most, heads)) return;
    }
    auto page_index = [&](int row) { return (int)__umul64hi((unsigned long long)row, p.s_inv); };  // row / S
    auto cached_head = [&](int head) { return p.GB == 1 ? head : head / p.GB; };

    const uint32_t ring = (smem_u32(raw) + 1023) / 1024 * 1024 + mine * (kStages * C::Stage);
    const int R = p.R, pieces = KT / R;
    const uint32_t half = (uint32_t)R * 128;  // bytes of one 64-column box of a copy

    // What a part needs from memory besides its tiles, asked for before the copies are waited for.
    // Plain loads here and below: __ldg says that nothing writes during the kernel, which begins
    // while the one before still may.
    // Queries: A operand, rows g (and g + 8).  The rows before and behind the range: their pages.
    uint32_t qa[KS][4];
    int edge_row = 0, edge_page = 0;
    auto ask = [&]() {
        const int hk = cached_head(now.head), hb = now.head - hk * p.GB;
        const int rows_h = min(p.HB, p.G - hb * p.HB);
        const uint32_t *qg = reinterpret_cast<const uint32_t *>(
            p.q + ((long long)now.b * p.Hq + hk * p.G + hb * p.HB + g) * D);
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            qa[i][0] = g < rows_h ? qg[i * 8 + q] : 0u;
            qa[i][2] = g < rows_h ? qg[i * 8 + 4 + q] : 0u;
            qa[i][1] = RH == 2 && g + 8 < rows_h ? qg[4 * D + i * 8 + q] : 0u;
            qa[i][3] = RH == 2 && g + 8 < rows_h ? qg[4 * D + i * 8 + 4 + q] : 0u;
        }
        edge_row = g == 0 ? now.tile * KT - 1 : g == 1 && now.last * KT < now.n ? now.last * KT : -1;
        edge_page = edge_row >= 0 ? p.table[(long long)now.b * p.M + page_index(edge_row)] : -1;
    };
    auto next = [&](Part &t) { return !ONE && next_part(t, cut, u0, u1, p.seqlens, KT, most, heads); };
    ask();

    Part ahead = now;
    bool more = working;  // something is left to copy
    // one piece per lane: its row of the pool for cached head 0, -1 on a page out of range, -2 behind the end
    int held_b = -1, held_at = -1, held = 0;
    unsigned copied = 0, used = 0, bad_stages = 0;
    int copy_stage = 0;
    auto copy_next = [&]() {
        if (!more) return;
        const int first = ahead.tile * pieces;
        if (ahead.b != held_b || (first & ~31) != held_at) {
            held_b = ahead.b;
            held_at = first & ~31;
            const long long row = (long long)(held_at + lane) * R;
            held = -2;
            if (row < ahead.n) {
                const int index = page_index((int)row), page = p.table[(long long)ahead.b * p.M + index];
                held = page >= 0 && page < p.P ? page * p.Hkv * p.S + (int)row - index * p.S : -1;
            }
        }
        const uint32_t bar = smem_u32(&bars[mine][copy_stage]), at = ring + copy_stage * C::Stage;
        int bytes = 0, place[KT / 8];
#pragma unroll
        for (int i = 0; i < KT / 8; ++i) {
            place[i] = -1;
            if (i < pieces) {
                const int at = __shfl_sync(0xffffffffu, held, (first + i) & 31);
                if (at >= 0) {
                    place[i] = at + cached_head(ahead.head) * p.S;
                    bytes += 2 * R * D * 2;
                } else if (at == -1) {
                    bad_stages |= 1u << copy_stage;
                }
            }
        }
        if (lane == 0 && half_of == 0) {
            mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
            for (int i = 0; i < KT / 8; ++i)
                if (place[i] >= 0) {
                    tma_load_3d(at + i * R * D * 2, &map_k, 0, place[i], 0, bar);
                    tma_load_3d(at + C::Tile + i * R * D * 2, &map_v, 0, place[i], 0, bar);
                }
        }
        copy_stage = copy_stage + 1 == kStages ? 0 : copy_stage + 1;
        ++copied;
        if (++ahead.tile == ahead.last) more = next(ahead);
    };
    for (int s = 0; s < kStages; ++s) copy_next();

    // ldmatrix addresses: keys, lane -> row (lane & 7) + 8 * (lane >> 4) of a pair of column
    // tiles, chunk (lane >> 3) & 1; values, lane -> row (lane & 15), chunk lane >> 4.  Row r of a
    // tile lies in copy r / R; its 16-byte chunks are permuted by r & 7: tiles begin on 1024 bytes, so
    // chunk c of a lane's row is its chunk 0 with bits 4 to 6 of the address flipped by c & 7.
    auto row_at = [&](int r) { return (uint32_t)((r / R) * (R * D * 2) + (r % R) * 128); };
    uint32_t k_row[NT / 2], v_row[KT / 16];
    const uint32_t x7 = lane & 7;
#pragma unroll
    for (int i = 0; i < NT / 2; ++i) k_row[i] = row_at(16 * i + (lane & 7) + 8 * (lane >> 4)) + ((x7 ^ ((lane >> 3) & 1)) << 4);
#pragma unroll
    for (int i = 0; i < KT / 16; ++i) v_row[i] = row_at(16 * i + (lane & 15)) + ((x7 ^ (lane >> 4)) << 4);
    const uint32_t to_half = half_of * (DW / 64) * half;
    auto chunk = [&](uint32_t row, uint32_t c) { return (row ^ ((c & 7) << 4)) + (c >> 3) * half; };

    int stage = 0;
    uint32_t parity = 0;
    bool lost = false;  // a wait has run out
    while (working) {
        const int b = now.b, n = now.n, tile = now.tile, last = now.last;
        const int hk = cached_head(now.head), hb = now.head - hk * p.GB;
        const int rows_h = min(p.HB, p.G - hb * p.HB);  // query heads of this block
        const int q0 = hk * p.G + hb * p.HB;            // the first of them
        const int r0 = tile * KT, r1 = min(n, last * KT);
        bool bad = false;

        // logits of the row before the range, the row behind it and a given sink: one more column
        // tile whose "keys" 0, 1, 2 are read straight from memory
        const bool given = r0 == 0 && p.mode == CSA_K0_GIVEN, copied_sink = r0 == 0 && p.mode == CSA_K0_COPY_FIRST;
        float edge[4] = {0.f, 0.f, 0.f, 0.f};
        if (r0 > 0 || r1 < n || given) {
            const __nv_bfloat16 *at = nullptr;
            if (edge_row >= 0) {
                if (edge_page >= 0 && edge_page < p.P)
                    at = p.k + (((long long)edge_page * p.Hkv + hk) * p.S + edge_row -
                                page_index(edge_row) * p.S) * D;
                else
                    bad = true;
            } else if (g == 2 && given) {
                at = p.k0 + (long long)hk * D;
            }
            const uint32_t *kg = reinterpret_cast<const uint32_t *>(at);
#pragma unroll
            for (int i = 0; i < KS; ++i)
                mma(edge, qa[i], at ? kg[i * 8 + q] : 0u, at ? kg[i * 8 + 4 + q] : 0u);
        }
        // prev, and pm = 2^{prev - m}, are those of the row before (used by q = 3)
        float prev[RH], behind[RH], m[RH], pm[RH], l[RH], w0[RH];
#pragma unroll
        for (int h = 0; h < RH; ++h) {
            const float before_a = __shfl_sync(0xffffffffu, edge[2 * h], lane & ~3);
            const float sink_a = __shfl_sync(0xffffffffu, edge[2 * h], (lane & ~3) | 1);
            behind[h] = __shfl_sync(0xffffffffu, edge[2 * h + 1], lane & ~3) * p.qscale;
            prev[h] = (r0 > 0 ? before_a : sink_a) * p.qscale;
            // a copied sink has the first row's logit, which the first tile brings
            m[h] = copied_sink ? -INFINITY : prev[h];
            pm[h] = 1.0f;  // 2^{prev - m}
            l[h] = w0[h] = 0.f;
        }
        float o[ON][4];
#pragma unroll
        for (int i = 0; i < ON; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float w[RH][NT][2];  // weights of the tile before, its last one without the next interval
        uint32_t v_at = 0;   // that tile's values

        // all weights relative to a raised maximum
        auto raise = [&](const float (&top)[RH]) {
            float f[RH];
#pragma unroll
            for (int h = 0; h < RH; ++h) {
                float t = top[h];
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
                t = fmaxf(t, m[h]);
                f[h] = ex2_approx(m[h] - t);
                m[h] = t;
                l[h] *= f[h];
                w0[h] *= f[h];
                pm[h] *= f[h];
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    w[h][i][0] *= f[h];
                    w[h][i][1] *= f[h];
                }
            }
#pragma unroll
            for (int i = 0; i < ON; ++i) {
                o[i][0] *= f[0];
                o[i][1] *= f[0];
                o[i][2] *= f[RH - 1];
                o[i][3] *= f[RH - 1];
            }
        };
        // the second product for the tile before
        auto values = [&]() {
#pragma unroll
            for (int h = 0; h < RH; ++h)
#pragma unroll
                for (int i = 0; i < NT; ++i) l[h] += w[h][i][0] + w[h][i][1];
#pragma unroll
            for (int ks = 0; ks < KT / 16; ++ks) {
                uint32_t hi[RH][2], lo[RH][2];
#pragma unroll
                for (int h = 0; h < RH; ++h)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float a = w[h][2 * ks + i][0], c = w[h][2 * ks + i][1];
                        const uint32_t ua = __float_as_uint(a) & 0xffff0000u, uc = __float_as_uint(c) & 0xffff0000u;
                        hi[h][i] = __byte_perm(ua, uc, 0x7632);
                        float la, lc;  // a (1 + 2^-23) - high part: never 0
                        apart(fma2(two(a, c), both(1.00000011920928955f),
                                   two(-__uint_as_float(ua), -__uint_as_float(uc))), la, lc);
                        lo[h][i] = pack_bf16x2(la, lc);
                    }
#pragma unroll
                for (int i = 0; i < ON / 2; ++i) {
                    uint32_t vb[4];
                    ldsm_t(chunk(v_at + v_row[ks], 2 * i) + to_half, vb);
                    if (RH == 1) {
                        const uint32_t a[4] = {hi[0][0], lo[0][0], hi[0][1], lo[0][1]};
                        mma(o[2 * i], a, vb[0], vb[1]);
                        mma(o[2 * i + 1], a, vb[2], vb[3]);
                    } else {
                        const uint32_t a[4] = {hi[0][0], hi[RH - 1][0], hi[0][1], hi[RH - 1][1]};
                        const uint32_t c[4] = {lo[0][0], lo[RH - 1][0], lo[0][1], lo[RH - 1][1]};
                        mma(o[2 * i], a, vb[0], vb[1]);
                        mma(o[2 * i + 1], a, vb[2], vb[3]);
                        mma(o[2 * i], c, vb[0], vb[1]);
                        mma(o[2 * i + 1], c, vb[2], vb[3]);
                    }
                }
            }
        };

        for (int j = tile; j < last; ++j) {
            if (C::Pair == 1 || !lost) {
                const bool arrived = mbar_wait_bounded(smem_u32(&bars[mine][stage]), parity, abort_flag,
                                                       &g_paged_status, kWaitLimitNs);
                if (!__all_sync(0xffffffffu, arrived)) {
                    // keeps the ring alive until its copies have landed, for at most one more limit each
                    if (lane == 0 && half_of == 0)
                        for (unsigned i = used; i < copied; ++i) {
                            const uint32_t bar = smem_u32(&bars[mine][i % kStages]);
                            const uint64_t t0 = globaltimer_ns();
                            while (!mbar_try_wait(bar, (i / kStages) & 1) && globaltimer_ns() - t0 < kWaitLimitNs) {
                            }
                        }
                    __syncwarp();
                    if (C::Pair == 1 && !ONE) return;
                    lost = true;
                    if (C::Pair == 1) break;
                }
            }
            if (C::Pair > 1 && lost) {  // the worker's barriers are still met
                if (j > tile) sync_worker();
                continue;
            }
            if (bad_stages >> stage & 1) {
                bad = true;
                bad_stages &= ~(1u << stage);
            }
            const uint32_t k_at = ring + stage * C::Stage;
            const int own = n - j * KT;  // rows of this tile that exist, if fewer than KT
            if (own < KT) {
                // rows behind the end: their weights are 0, and 0 * NaN is not
                uint8_t *vt = raw + (k_at + C::Tile - smem_u32(raw));
                for (int i = lane; i < (KT - own) * ON; i += 32) {
                    const int r = own + i / ON, c = half_of * ON + i % ON;
                    *reinterpret_cast<uint4 *>(vt + row_at(r) + (c >> 3) * half + ((c & 7) << 4)) =
                        make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            // logits
            float s[NT][4], s2[NT][4];  // two sums of every other product: the chain of dependent ones is half as long
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[i][e] = s2[i][e] = 0.f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int i = 0; i < NT / 2; ++i) {
                    uint32_t kb[4];
                    ldsm(chunk(k_at + k_row[i], 2 * ks), kb);
                    mma(ks & 1 ? s2[2 * i] : s[2 * i], qa[ks], kb[0], kb[1]);
                    mma(ks & 1 ? s2[2 * i + 1] : s[2 * i + 1], qa[ks], kb[2], kb[3]);
                }
            float top[RH];
            bool over = false;
#pragma unroll
            for (int h = 0; h < RH; ++h)
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) s[i][2 * h + e] = (s[i][2 * h + e] + s2[i][2 * h + e]) * p.qscale;
            if (own < KT) {
#pragma unroll
                for (int h = 0; h < RH; ++h)
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (8 * i + 2 * q + e >= own) s[i][2 * h + e] = -INFINITY;
            }
#pragma unroll
            for (int h = 0; h < RH; ++h) {
                top[h] = -INFINITY;
#pragma unroll
                for (int i = 0; i < NT; ++i) top[h] = fmaxf(top[h], fmaxf(s[i][2 * h], s[i][2 * h + 1]));
                over |= top[h] > m[h] + kRaise;
            }
            if (j == tile) {
#pragma unroll
                for (int h = 0; h < RH; ++h)
#pragma unroll
                    for (int i = 0; i < NT; ++i) w[h][i][0] = w[h][i][1] = 0.f;
            }
            if (__any_sync(0xffffffffu, over)) raise(top);
            if (j == tile && copied_sink) {
#pragma unroll
                for (int h = 0; h < RH; ++h) {
                    prev[h] = __shfl_sync(0xffffffffu, s[0][2 * h], lane & ~3);
                    pm[h] = ex2_approx(prev[h] - m[h]);
                }
            }

            // this tile's weights, and the share of its first interval that the row before gets (for q = 3,
            // whose w holds that row)
            float nw[RH][NT][2], even_left[RH][NT], to_before[RH];
#pragma unroll
            for (int h = 0; h < RH; ++h) {
                float pe[NT][2];
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    pe[i][0] = ex2_approx(s[i][2 * h] - m[h]);
                    pe[i][1] = ex2_approx(s[i][2 * h + 1] - m[h]);
                }
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    // the logit and power before this lane's first row: from the lane to the left, for
                    // q = 0 from q = 3 of the column tile before
                    const float a_src = q == 3 ? (i == 0 ? prev[h] : s[i > 0 ? i - 1 : 0][2 * h + 1]) : s[i][2 * h + 1];
                    const float p_src = q == 3 ? (i == 0 ? pm[h] : pe[i > 0 ? i - 1 : 0][1]) : pe[i][1];
                    const float a_b = __shfl_sync(0xffffffffu, a_src, (lane & ~3) | ((q + 3) & 3));
                    const float p_b = __shfl_sync(0xffffffffu, p_src, (lane & ~3) | ((q + 3) & 3));
                    float r_even, l_odd, r_odd;
                    intervals(a_b, s[i][2 * h], s[i][2 * h], s[i][2 * h + 1], p_b, pe[i][0], pe[i][0], pe[i][1],
                              even_left[h][i], r_even, l_odd, r_odd);
                    nw[h][i][0] = r_even + l_odd;
                    nw[h][i][1] = r_odd;
                    if (own < KT) {  // nothing from intervals that end behind the last row
                        if (8 * i + 2 * q + 1 >= own) {
                            nw[h][i][0] = r_even;
                            nw[h][i][1] = 0.f;
                        }
                        if (8 * i + 2 * q >= own) nw[h][i][0] = even_left[h][i] = 0.f;
                    }
                }
                // for the next tile, and for q = 3 only
                prev[h] = s[NT - 1][2 * h + 1];
                pm[h] = pe[NT - 1][1];
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const float src = q == 0 ? even_left[h][i + 1 < NT ? i + 1 : 0] : even_left[h][i];
                    const float from = __shfl_sync(0xffffffffu, src, (lane & ~3) | ((q + 1) & 3));
                    if (i + 1 < NT || q < 3) nw[h][i][1] += from;
                    if (i + 1 == NT) to_before[h] = from;
                }
            }
            if (j > tile) {
#pragma unroll
                for (int h = 0; h < RH; ++h)
                    if (q == 3) w[h][NT - 1][1] += to_before[h];
                values();
                sync_worker();  // every lane has read the tile before: its stage is free
                ++used;
                copy_next();
            } else if (copied_sink) {  // its value is the first row's too
#pragma unroll
                for (int h = 0; h < RH; ++h)
                    if (q == 0) nw[h][0][0] += even_left[h][0];
            } else if (r0 == 0) {
#pragma unroll
                for (int h = 0; h < RH; ++h) w0[h] = __shfl_sync(0xffffffffu, even_left[h][0], lane & ~3);
            }
#pragma unroll
            for (int h = 0; h < RH; ++h)
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    w[h][i][0] = nw[h][i][0];
                    w[h][i][1] = nw[h][i][1];
                }
            v_at = k_at + C::Tile;
            if (++stage == kStages) {
                stage = 0;
                parity ^= 1;
            }
        }
        if (!lost && r1 < n) {  // the range's last row has a neighbour behind it
            bool over = false;
#pragma unroll
            for (int h = 0; h < RH; ++h) over |= behind[h] > m[h] + kRaise;
            if (__any_sync(0xffffffffu, over)) raise(behind);
#pragma unroll
            for (int h = 0; h < RH; ++h) {
                float left, right, none0, none1;
                const float pb = ex2_approx(behind[h] - m[h]);
                intervals(prev[h], behind[h], prev[h], behind[h], pm[h], pb, pm[h], pb, left, right, none0, none1);
                if (q == 3) w[h][NT - 1][1] += left;
            }
        }
        if (!lost) values();
        sync_worker();
        if (!lost) {
            ++used;
            copy_next();
        }

        bad = __any_sync(0xffffffffu, bad || lost);
        const bool whole = r0 == 0 && r1 == n;
        float sum[RH];
#pragma unroll
        for (int h = 0; h < RH; ++h) {
            float t = l[h];
            t += __shfl_xor_sync(0xffffffffu, t, 1);
            t += __shfl_xor_sync(0xffffffffu, t, 2);
            sum[h] = bad ? NAN : t + w0[h];
        }
        // a worker's part that does not begin a segment is its first
        const long long slot = (worker * 2 + (u0 < now.s0 ? 1 : 0)) * p.HB;
        // ONE: this warp's ring, whose copies have all been read
        float *kept = reinterpret_cast<float *>(raw + (ring - smem_u32(raw)));
        const uint32_t *sink_v = given ? reinterpret_cast<const uint32_t *>(p.v0 + (long long)hk * D + half_of * DW) : nullptr;
#pragma unroll
        for (int h = 0; h < RH; ++h) {
            const int row = g + 8 * h;
            if (row < rows_h) {
                const float inv = 1.0f / sum[h];
                const long long oh = (long long)b * p.Hq + q0 + row;
                __nv_bfloat16 *og = p.out + oh * D + half_of * DW;
                float *po = (ONE ? kept + row * D : p.part_o + (slot + row) * D) + half_of * DW;
#pragma unroll
                for (int i = 0; i < ON; ++i) {
                    float a = o[i][2 * h], c = o[i][2 * h + 1];
                    if (RH == 1) {  // the low parts of the weights
                        a += o[i][2];
                        c += o[i][3];
                    }
                    if (sink_v) {
                        const uint32_t v2 = sink_v[i * 4 + q];
                        a = fmaf(w0[h], __uint_as_float(v2 << 16), a);
                        c = fmaf(w0[h], __uint_as_float(v2 & 0xffff0000u), c);
                    }
                    if (!ONE && whole)
                        *reinterpret_cast<uint32_t *>(og + 8 * i + 2 * q) = pack_bf16x2(a * inv, c * inv);
                    else
                        *reinterpret_cast<float2 *>(po + 8 * i + 2 * q) = make_float2(a, c);
                }
                if (q == 0 && half_of == 0) {
                    if (ONE) {
                        *reinterpret_cast<float2 *>(kept + p.HB * D + 2 * row) = make_float2(m[h], sum[h]);
                    } else if (!whole) {
                        p.part_ml[2 * (slot + row)] = m[h];
                        p.part_ml[2 * (slot + row) + 1] = sum[h];
                    } else if (p.lse) {
                        p.lse[oh] = (m[h] + log2f(sum[h])) * kLn2;
                    }
                }
            }
        }
        if (bad && lane == 0) atomicCAS(&g_paged_status, 0, CSA_ERR_INVALID_ARG);
        if (!ONE && r0 == 0 && lane == 0 && half_of == 0 && (p.by_segment || !whole)) {
            const long long end = now.s0 + cut.units(now.tiles);
            const int segment = b * heads + now.head;
            p.joins[p.by_segment ? segment : worker] =
                make_int4(whole ? -1 : segment, (int)worker, (int)cut.worker_of(end - 1), u0 < now.s0 ? 1 : 0);
        }
        if (!next(now)) break;
        ask();
    }
    if constexpr (ONE) {
        // Joins the parts: those of the block's warps through its shared memory, a warp per query
        // head, then those of the cluster's blocks, each block a share of the columns.
        const int hk = cached_head(now.head), hb = now.head - hk * p.GB, rows_h = min(p.HB, p.G - hb * p.HB);
        const long long first = (long long)now.b * p.Hq + hk * p.G + hb * p.HB;
        const int blocks = min(p.cluster, parts);                                       // with parts
        const int count = rank < parts ? (parts - rank - 1) / p.cluster + 1 : 0;        // warps of this block with parts
        uint8_t *rings = raw + ((smem_u32(raw) + 1023) / 1024 * 1024 - smem_u32(raw));
        constexpr int kRing = kStages * C::Stage;
        float *sums = reinterpret_cast<float *>(rings + kRing / 2);  // behind the first ring's part
        static_assert(16 * (D + 2) * 4 <= kRing / 2 || RH == 1, "two sets of sums fit a ring");
        static_assert(8 * (D + 2) * 4 <= kRing / 2, "two sets of sums fit a ring");
        __syncthreads();
        for (int row = warp; row < rows_h && count > 0; row += C::Warps) {
            auto of = [&](int i) { return reinterpret_cast<const float *>(rings + i * kRing); };
            float2 ml = make_float2(-INFINITY, 0.f);
            if (lane < count) ml = *reinterpret_cast<const float2 *>(of(lane) + p.HB * D + 2 * row);
            float top = ml.x;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float f = ex2_approx(ml.x - top);
            float total = f * ml.y;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
            const float inv = 1.0f / total;
#pragma unroll
            for (int c = 0; c < D; c += 64) {
                float2 v = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < C::Workers; ++i) {
                    const float fi = __shfl_sync(0xffffffffu, f, i);
                    if (i < count) {
                        const float2 x = *reinterpret_cast<const float2 *>(of(i) + row * D + c + 2 * lane);
                        v.x = fmaf(fi, x.x, v.x);
                        v.y = fmaf(fi, x.y, v.y);
                    }
                }
                if (blocks == 1)
                    *reinterpret_cast<uint32_t *>(p.out + (first + row) * D + c + 2 * lane) =
                        pack_bf16x2(v.x * inv, v.y * inv);
                else
                    *reinterpret_cast<float2 *>(sums + row * D + c + 2 * lane) = v;
            }
            if (lane == 0) {
                if (blocks > 1)
                    *reinterpret_cast<float2 *>(sums + p.HB * D + 2 * row) = make_float2(top, total);
                else if (p.lse)
                    p.lse[first + row] = (top + log2f(total)) * kLn2;
            }
        }
        if (blocks > 1) {  // the same for every block of the cluster
            cluster_sync();
            const uint32_t at = smem_u32(sums);
            for (int u = rank * blockDim.x + threadIdx.x; u < rows_h * (D / 2); u += p.cluster * blockDim.x) {
                const int row = u / (D / 2), c = 2 * (u - row * (D / 2));
                float2 ml[8], x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < blocks) {
                        ml[i] = cluster_load(at + (p.HB * D + 2 * row) * 4, i);
                        x[i] = cluster_load(at + (row * D + c) * 4, i);
                    }
                float top = ml[0].x;
#pragma unroll
                for (int i = 1; i < 8; ++i)
                    if (i < blocks) top = fmaxf(top, ml[i].x);
                float total = 0.f, a = 0.f, b = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < blocks) {
                        const float f = ex2_approx(ml[i].x - top);
                        total = fmaf(f, ml[i].y, total);
                        a = fmaf(f, x[i].x, a);
                        b = fmaf(f, x[i].y, b);
                    }
                const float inv = 1.0f / total;
                *reinterpret_cast<uint32_t *>(p.out + (first + row) * D + c) = pack_bf16x2(a * inv, b * inv);
                if (c == 0 && p.lse) p.lse[first + row] = (top + log2f(total)) * kLn2;
            }
            cluster_sync();  // no block leaves while its sums are read
        }
    }
}

// Joins the parts of a segment (a cached head of a sequence and a block of its
// query heads) that several workers share.  With M the largest m_c:
// o = sum 2^{m_c-M} o_c / sum 2^{m_c-M} l_c, lse = (M + log2 sum) ln 2.
// The parts are the first worker's and the first ones of the workers behind it.
constexpr int kJoinWarps = 8, kJoinWarpsMost = 32;

// Adds the parts first, first + step, ... of one query head into (M, L, o),
// V = D / 32 columns per lane, a batch of loads at a time.
template <int D>
__device__ __forceinline__ void add_parts(const PagedParams &p, int c0, int c1, int first_slot, int row,
                                          int first, int step, float &M, float &L, float (&o)[D / 32]) {
    constexpr int V = D / 32, kBatch = D == 256 ? 4 : 8;
    const int lane = threadIdx.x & 31;
    for (int base = first; base <= c1; base += kBatch * step) {
        float2 ml[kBatch], v[kBatch][V / 2];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int c = base + k * step;
            ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) v[k][i] = make_float2(0.f, 0.f);
            if (c <= c1) {
                const long long slot = ((long long)c * 2 + (c == c0 ? first_slot : 0)) * p.HB + row;
                ml[k] = *reinterpret_cast<const float2 *>(p.part_ml + 2 * slot);
#pragma unroll
                for (int i = 0; i < V / 2; ++i)
                    v[k][i] = *reinterpret_cast<const float2 *>(p.part_o + slot * D + 64 * i + 2 * lane);
            }
        }
        float top = M;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) top = fmaxf(top, ml[k].x);
        const float f = ex2_approx(M - top);
        M = top;
        L *= f;
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] *= f;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const float fk = ex2_approx(ml[k].x - top);
            L = fmaf(fk, ml[k].y, L);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                o[2 * i] = fmaf(fk, v[k][i].x, o[2 * i]);
                o[2 * i + 1] = fmaf(fk, v[k][i].y, o[2 * i + 1]);
            }
        }
    }
}

// By segment (few of them, so many parts): a block per segment and query head,
// its warps taking every gridDim-th part each.  By worker: a block per worker,
// for the segment that begins there, a warp per query head (few parts).
template <int D>
__global__ void __launch_bounds__(kJoinWarpsMost * 32) join_kernel(const PagedParams p) {
    __shared__ float s_o[kJoinWarpsMost][D], s_m[kJoinWarpsMost], s_l[kJoinWarpsMost];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int heads = p.Hkv * p.GB;
    // every block waits: this kernel must not end before the one that forms the parts
    after_previous();
    const int4 seg = p.joins[blockIdx.x];
    // none; or left over, where a wait ran out and the parts are undefined anyway
    if (seg.x < 0 || seg.x >= p.B * heads || seg.y < 0 || seg.z < seg.y || seg.z >= workers(D)) return;
    const int b = seg.x / heads, head = seg.x - b * heads, c0 = seg.y;
    const int hk = head / p.GB, hb = head - hk * p.GB, rows = min(p.HB, p.G - hb * p.HB);
    const long long out0 = (long long)b * p.Hq + hk * p.G + hb * p.HB;
    float o[D / 32];
    if (!p.by_segment) {
        for (int row = warp; row < rows; row += warps) {
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
            add_parts<D>(p, c0, seg.z, seg.w, row, c0, 1, M, L, o);
            const float inv = 1.0f / L;
#pragma unroll
            for (int i = 0; i < D / 32; i += 2)
                *reinterpret_cast<uint32_t *>(p.out + (out0 + row) * D + 32 * i + 2 * lane) =
                    pack_bf16x2(o[i] * inv, o[i + 1] * inv);
            if (lane == 0 && p.lse) p.lse[out0 + row] = (M + log2f(L)) * kLn2;
        }
        return;
    }
    const int row = blockIdx.y;
    if (row >= rows) return;
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
    add_parts<D>(p, c0, seg.z, seg.w, row, c0 + warp, warps, M, L, o);
#pragma unroll
    for (int i = 0; i < D / 32; i += 2)
        *reinterpret_cast<float2 *>(&s_o[warp][32 * i + 2 * lane]) = make_float2(o[i], o[i + 1]);
    if (lane == 0) {
        s_m[warp] = M;
        s_l[warp] = L;
    }
    __syncthreads();
    // each warp for itself: lane i has warp i's factor, 0 where it had no parts
    const float m = lane < warps ? s_m[lane] : -INFINITY;
    float top = m;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float f = ex2_approx(m - top);
    float total = lane < warps ? f * s_l[lane] : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    const float inv = 1.0f / total;
    for (int col = threadIdx.x; col < D; col += blockDim.x) {  // D is a multiple of 32: whole warps
        float v = 0.f;
#pragma unroll 8
        for (int i = 0; i < warps; ++i) v = fmaf(__shfl_sync(0xffffffffu, f, i), s_o[i][col], v);
        p.out[(out0 + row) * D + col] = __float2bfloat16_rn(v * inv);
    }
    if (threadIdx.x == 0 && p.lse) p.lse[out0 + row] = (top + log2f(total)) * kLn2;
}

// [P * Hkv * S, D] bf16 as {64, rows, D / 64}, boxes of R rows.
bool encode_pool(CUtensorMap *map, const void *ptr, long long rows, int D, int R) {
    auto fn = csa_tc::get_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)(D / 64)};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, 128};
    const cuuint32_t box[3] = {64, (cuuint32_t)R, (cuuint32_t)(D / 64)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Blocks per segment of the one-kernel form, 0 where the other form is used.
// The lengths are not known here, only the tiles that a row of the table can
// hold.
int cluster_for(long long segments, long long tiles, int warps) {
    if (segments > kOneAtATime[0]) return 0;
    int c = 8;
    for (int i = 3; i > 0 && (segments > kOneAtATime[i] || (long long)(c / 2) * warps >= tiles); --i) c /= 2;
    const long long most = 4 * segments * c >= 3 * kGrid ? kOneTiles : kOneTilesLess;
    return tiles <= most * c * warps ? c : 0;
}

template <int D, int RH>
int launch(PagedParams &p, cudaStream_t stream) {
    using C = Cfg<D, RH>;
    p.R = C::KT;
    while (p.S % p.R != 0) p.R /= 2;  // S is a multiple of 8
    CUtensorMap map_k, map_v;
    const long long rows = (long long)p.P * p.Hkv * p.S;
    // no pool: no sequence has a valid page, and the maps are never used
    const void *some = p.q;
    if (!encode_pool(&map_k, rows ? (const void *)p.k : some, rows ? rows : 8, D, p.R) ||
        !encode_pool(&map_v, rows ? (const void *)p.v : some, rows ? rows : 8, D, p.R))
        return CSA_ERR_CUDA;
    const int heads = p.Hkv * p.GB;
    p.s_inv = ~0ull / p.S + 1;
    const long long segments = (long long)p.B * heads, tiles = ((long long)p.M * p.S + C::KT - 1) / C::KT;
    p.cluster = cluster_for(segments, tiles, C::Workers);
    if (p.cluster > 0) {
        auto kern = paged_kernel<D, RH, true>;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::Smem) != cudaSuccess ||
            launch_clusters_after_previous(kern, (unsigned)segments * p.cluster, C::Warps * 32, C::Smem, stream,
                                           p.cluster, p, map_k, map_v) != cudaSuccess)
            return CSA_ERR_CUDA;
        return CSA_OK;
    }
    // blocks that the largest possible lengths can keep busy
    const long long most = segments * tiles;
    const int grid = (int)(most < kGrid ? (most < 1 ? 1 : most) : kGrid);
    auto kern = paged_kernel<D, RH, false>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::Smem) != cudaSuccess)
        return CSA_ERR_CUDA;
    const long long all = (long long)grid * C::Workers;
    p.by_segment = segments <= kGrid;
    if (launch_after_previous(kern, grid, C::Warps * 32, C::Smem, stream, p, map_k, map_v) != cudaSuccess)
        return CSA_ERR_CUDA;
    // parts of a segment, at most about
    const long long parts = all / segments;
    const dim3 blocks = p.by_segment ? dim3((unsigned)segments, (unsigned)p.HB) : dim3((unsigned)all);
    const int threads = 32 * (p.by_segment && parts > 64 ? kJoinWarpsMost : kJoinWarps);
    return launch_after_previous(join_kernel<D>, blocks, threads, 0, stream, p) == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

// Blocks of the query heads of a group, at most 16 each, as equal as can be.
int head_blocks(int G) { return (G + 15) / 16; }


}  // namespace

long long csa_decode_paged_scratch_bytes(int B, int Hq, int Hkv, int d) {
    if (B < 0 || Hq < 0 || Hkv < 1 || Hq % Hkv != 0 || !(d == 64 || d == 128 || d == 256)) return -1;
    const int G = Hq / Hkv;
    const int GB = head_blocks(G), HB = GB ? (G + GB - 1) / GB : 0;
    return workers(d) * (2 * HB * (d + 2) * (long long)sizeof(float) + (long long)sizeof(int4));
}

int csa_decode_paged_run(const void *q, const void *k_pages, const void *v_pages, const void *k0,
                         const void *v0, const int *block_table, const int *seqlens, void *out,
                         float *lse, void *scratch, int B, int Hq, int Hkv, int P, int S, int M,
                         int d, float scale, int mode, cudaStream_t stream) {
    PagedParams p = {};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k_pages);
    p.v = static_cast<const __nv_bfloat16 *>(v_pages);
    p.k0 = static_cast<const __nv_bfloat16 *>(k0);
    p.v0 = static_cast<const __nv_bfloat16 *>(v0);
    p.table = block_table;
    p.seqlens = seqlens;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.lse = lse;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.P = P;
    p.S = S;
    p.M = M;
    p.G = Hq / Hkv;
    p.GB = head_blocks(p.G);
    p.HB = (p.G + p.GB - 1) / p.GB;
    p.qscale = scale * kLog2e;
    p.mode = mode;
    p.joins = static_cast<int4 *>(scratch);
    p.part_ml = reinterpret_cast<float *>(p.joins + workers(d));
    p.part_o = p.part_ml + 2 * workers(d) * p.HB * 2;
    if (p.HB <= 8) {
        if (d == 64) return launch<64, 1>(p, stream);
        if (d == 128) return launch<128, 1>(p, stream);
        return launch<256, 1>(p, stream);
    }
    if (d == 64) return launch<64, 2>(p, stream);
    if (d == 128) return launch<128, 2>(p, stream);
    return launch<256, 2>(p, stream);
}

int csa_paged_take_status(void) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_paged_status, sizeof(int)) != cudaSuccess) return CSA_ERR_CUDA;
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_paged_status, &zero, sizeof(int)) != cudaSuccess) return CSA_ERR_CUDA;
    return v;
}

// Attention of a tree of drafted tokens over a paged cache that already holds their
// rows (eq. (10)/(11) of "Continuous Softmax Attention" for each row's own list of
// positions: the sink, the n tokens before the draft, and the drafted tokens on the
// path from a root to the row's node).
//
// In the interval form (csa_paged.cuh) a list is a chain of intervals, and a row's
// sums are those of two stretches of it that share the last position before the
// draft:
//   - the positions up to there are the same for all rows of a cached head. They are
//     the paged decode step's, the T rows of each of the group's query heads taking
//     the place of query heads (T consecutive rows of a head are consecutive in
//     memory), and leave parts: sums, maximum and weight sum per row and range;
//   - behind it, each drafted token on the path ends one interval, which begins at its
//     parent (at that last position for a root).  With at most 64 drafted tokens this
//     is a product of the rows with T + 1 cached rows, weights by the tree, and a
//     product with their values: tree_kernel, which then joins all parts of a row.
//
// A token's right share goes to its own weight, its left share to its parent's: a
// path has one child of each of its nodes, so both are stored without a sum over
// rows, and every interval is formed by a lane of its own.
//
// What bounds it: the first stretch (csa_paged.cuh); the second is bound by latency: a
// few dependent trips to memory, two small products, and its own instructions, which
// are executed once a block and come from memory after the first kernel has streamed
// the cache through the L2.  So loops are rolled even where they are short: with the two
// rows of a warp and four parts of a row side by side, 16 drafted tokens over 16
// sequences of 4096 to 8192 rows (32 heads on 8, d = 128) took 96 us instead of 90 and 64
// drafted 255 instead of 250, when a weight was one number.  Now they take 98 and 293; the
// second kernel, taken alone, 15 and 56.
#include "csa_rows.cuh"

namespace {

constexpr int kTreeThreads = 256, kTreeWarps = kTreeThreads / 32;
constexpr int kTreeRows = 16;       // rows of a block's products
// Blocks per SM that the registers allow.
template <int D>
constexpr int kTreeBlocks = D == 256 ? 3 : 4;
constexpr int kDeep = 80;           // T + 1 positions at most, to whole products

struct TreeParams {
    const __nv_bfloat16 *q;
    const void *k, *v;
    const float *scales;
    const __nv_bfloat16 *k0, *v0;
    const int *table, *seqlens, *counts, *parents;
    __nv_bfloat16 *out;
    float *lse;
    const float *part_o, *part_ml;
    const int4 *joins;
    int workers;           // that the parts are of
    int B, Hkv, T, P, S, M;
    int rows, GB, HB;      // rows of a group (G * T), blocks of them, rows per block
    int RB;                // rows per block of this kernel, at most kTreeRows
    float qscale;
    int mode;
};

// Shared memory, by the positions that T asks for: few drafted tokens leave room for more blocks per SM.
template <int D>
struct TreeSmem {
    static constexpr int Row = 2 * D + 16;  // bytes of a cached row: 16 more, so that eight rows meet no bank twice
    int deep, pitch, Q, S, Right, Left, Parts, bytes;  // positions; pitch of the weights in elements; offsets
    __host__ __device__ explicit TreeSmem(int T) {
        deep = (T + 16) / 16 * 16;
        pitch = deep + 4;
        Q = 2 * deep * Row;  // behind the keys and the values
        S = Q + kTreeRows * Row;
        Right = S + kTreeRows * pitch * 4;
        Left = Right + kTreeRows * pitch * 4;
        Parts = Left + kTreeRows * pitch * 4;  // [warps][D] of a row's parts
        // where a row has many parts, the sums over the drafted tokens take the place of the queries and weights
        if (Parts < Q + kTreeRows * D * 4) Parts = Q + kTreeRows * D * 4;
        bytes = Parts + kTreeWarps * D * 4;
    }
};

// Eight values as bf16 numbers, exact for the codes of either 8-bit kind.
template <int KIND>
__device__ __forceinline__ uint4 as_bf16(const void *row, int c) {
    if constexpr (KIND == CSA_BF16) {
        return *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(row) + c);
    } else {
        const uint2 raw = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(row) + c);
        float x[8];
        values_of<KIND == CSA_E4M3, false, 8>(raw, 1.0f, x);
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
}

__device__ __forceinline__ bool any_not_finite(const uint4 &x) {
    auto bad = [](uint32_t w) { return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u; };
    return bad(x.x) || bad(x.y) || bad(x.z) || bad(x.w);
}

__device__ __forceinline__ void copy16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void ldsm_t2(uint32_t addr, uint32_t &r0, uint32_t &r1) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(addr) : "memory");
}

// A block: a segment's drafted tokens, once into shared memory, and one or several of its groups of RB rows.
template <int D, int KIND>
__global__ void __launch_bounds__(kTreeThreads, kTreeBlocks<D>) tree_kernel(const __grid_constant__ TreeParams p) {
    constexpr int Row = TreeSmem<D>::Row, C = D / 8;  // bytes; chunks of 8 values
    constexpr bool EIGHT = KIND != CSA_BF16;
    const TreeSmem<D> L(p.T);
    const int deep = L.deep, pitch = L.pitch;
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ unsigned long long s_path[64];
    __shared__ int s_jump[64], s_up[64];
    __shared__ unsigned long long s_bad;  // nodes whose parent is out of range
    __shared__ __align__(8) uint8_t s_flags[8];  // of the warps: 1 where a page is out of range, 2 where values are not finite
    __shared__ long long s_row[kDeep];    // a position's row of the pool, -1 for none, -2 for a given sink
    __shared__ float s_sk[kDeep], s_sv[kDeep], s_m[kTreeRows], s_l[kTreeRows], s_pm[kTreeWarps], s_pl[kTreeWarps];
    uint8_t *Ks = raw, *Vs = raw + deep * Row, *Qs = raw + L.Q;
    float *S = reinterpret_cast<float *>(raw + L.S), *Rt = reinterpret_cast<float *>(raw + L.Right),
          *Lf = reinterpret_cast<float *>(raw + L.Left), *sums = reinterpret_cast<float *>(raw + L.Parts);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
    const int segment = blockIdx.x, heads = p.Hkv * p.GB;
    const int b = segment / heads, head = segment - b * heads, hk = head / p.GB, hb = head - hk * p.GB;
    const int last_row = min((hb + 1) * p.HB, p.rows);
    const long long rows0 = ((long long)b * p.Hkv + hk) * p.rows;  // row of q, out and lse of the group's first
    auto ask_queries = [&](int first, int rows) {
        for (int i = tid; i < kTreeRows * C; i += kTreeThreads) {
            const int r = i / C, c = i % C;
            uint8_t *to = Qs + r * Row + c * 16;
            if (r < rows)
                copy16(smem_u32(to), p.q + (rows0 + first + r) * D + c * 8);
            else
                *reinterpret_cast<uint4 *>(to) = make_uint4(0u, 0u, 0u, 0u);
        }
    };
    int first = hb * p.HB + blockIdx.y * p.RB;  // row of the group of query heads
    if (first >= last_row) return;
    // What the draft needs was written before the kernel that forms the parts began, and this one begins
    // after it did; its parts are waited for below.
    ask_queries(first, min(p.RB, last_row - first));
    const int len = p.seqlens[b], c = p.counts ? p.counts[b] : p.T, n = len - c;
    const bool sound = c >= 0 && c <= p.T && n >= 0 && len <= (long long)p.M * p.S;
    const int have = sound && c > 0 ? c + 1 : 0;  // position 0 is the last one before the draft, 1 + u is drafted token u
    bool lost = false, wild = false;     // a page out of range; values that are not finite
    if (warp < 2) {
        int up = tid >= p.T ? -1 : p.parents ? p.parents[(long long)b * p.T + tid] : tid - 1;
        if (tid >= c || !sound) up = -1;
        const bool bad = up < -1 || up >= tid;
        s_up[tid] = s_jump[tid] = bad ? -1 : up;
        s_path[tid] = 1ull << tid;
        const unsigned at = __ballot_sync(0xffffffffu, bad);
        if (lane == 0) reinterpret_cast<unsigned *>(&s_bad)[warp] = at;
        asm volatile("bar.sync 1, 64;" ::: "memory");
        // ancestors, twice as far each time
#pragma unroll 1
        for (int i = 0; i < 6; ++i) {
            const int jump = s_jump[tid];
            const unsigned long long more = jump >= 0 ? s_path[jump] : 0;
            const int next = jump >= 0 ? s_jump[jump] : -1;
            asm volatile("bar.sync 1, 64;" ::: "memory");
            s_path[tid] |= more;
            s_jump[tid] = next;
            asm volatile("bar.sync 1, 64;" ::: "memory");
        }
    } else {  // meanwhile, the cached rows: where they are, then themselves as bf16 numbers
        constexpr int Threads = kTreeThreads - 64;
        const int t0 = tid - 64;
        if (t0 < deep) {
            const int at = n - 1 + t0;
            long long row = -1;
            float2 s = make_float2(0.0f, 0.0f);
            if (t0 < have) {
                s = make_float2(1.0f, 1.0f);
                if (at >= 0) {
                    const int page = p.table[(long long)b * p.M + at / p.S];
                    if (page >= 0 && page < p.P) {
                        row = ((long long)page * p.Hkv + hk) * p.S + at % p.S;
                        if (EIGHT) s = *reinterpret_cast<const float2 *>(p.scales + 2 * row);
                    } else {
                        lost = true;
                    }
                } else if (p.mode == CSA_K0_GIVEN) {
                    row = -2;
                }
            }
            s_row[t0] = row;
            s_sk[t0] = s.x;
            s_sv[t0] = s.y;
        }
        asm volatile("bar.sync 2, %0;" ::"n"(Threads) : "memory");
        constexpr int E = EIGHT ? 1 : 2;
        const uint8_t *kp = static_cast<const uint8_t *>(p.k), *vp = static_cast<const uint8_t *>(p.v);
#pragma unroll 1
        for (int i = t0; i < deep * C; i += Threads) {
            const int j = i / C, col = i % C * 8;
            const long long row = s_row[j], at = (row * D + col) * E;
            uint8_t *to = Ks + j * Row + col * 2;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (row >= 0) {
                if constexpr (EIGHT)
                    *reinterpret_cast<uint4 *>(to) = as_bf16<KIND>(kp + at, 0);
                else
                    copy16(smem_u32(to), kp + at);
                v = as_bf16<KIND>(vp + at, 0);
            } else if (row == -2) {
                copy16(smem_u32(to), p.k0 + (long long)hk * D + col);
                v = *reinterpret_cast<const uint4 *>(p.v0 + (long long)hk * D + col);
            } else {
                *reinterpret_cast<uint4 *>(to) = v;
            }
            wild |= any_not_finite(v);
            *reinterpret_cast<uint4 *>(Vs + j * Row + col * 2) = v;
        }
    }
    lost = __any_sync(0xffffffffu, lost);
    wild = __any_sync(0xffffffffu, wild);
    if (lane == 0) s_flags[warp] = (uint8_t)(lost | 2 * wild);
    for (;; ask_queries(first, min(p.RB, last_row - first))) {
        const int rows = min(p.RB, last_row - first);
        const long long out0 = rows0 + first;
        copies_done();
        __syncthreads();
        const unsigned long long flags = *reinterpret_cast<const unsigned long long *>(s_flags);
        if (!sound || (flags & 0x0101010101010101ull)) {
            after_previous();  // this kernel must not end before the one that forms the parts
            for (int i = tid; i < rows * D; i += kTreeThreads) p.out[out0 * D + i] = __float2bfloat16_rn(NAN);
            if (p.lse && tid < rows) p.lse[out0 + tid] = NAN;
            if (tid == 0) atomicCAS(&g_paged_status, 0, CSA_ERR_INVALID_ARG);
        } else {
            // logits, in log2 units: a warp has eight positions
            for (int t = warp; t < (have + 7) / 8; t += kTreeWarps) {
                float acc[4] = {0.f, 0.f, 0.f, 0.f}, acc2[4] = {0.f, 0.f, 0.f, 0.f};
                const uint32_t qa = smem_u32(Qs) + (lane & 15) * Row + (lane >> 4) * 16,
                               ka = smem_u32(Ks) + (8 * t + (lane & 7)) * Row + (lane >> 3) * 16;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    uint32_t a0[4], a1[4], k[4];
                    ldsm(qa + 64 * i, a0);
                    ldsm(qa + 64 * i + 32, a1);
                    ldsm(ka + 64 * i, k);
                    mma(acc, a0, k[0], k[1]);
                    mma(acc2, a1, k[2], k[3]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = 8 * t + 2 * q + (e & 1);
                    S[(g + 8 * (e >> 1)) * pitch + j] = (acc[e] + acc2[e]) * (p.qscale * s_sk[j]);
                }
            }
            __syncthreads();
            // Weights: a warp has a row, a lane the intervals that end at nodes lane and lane + 32.  A weight is two bf16
            // numbers, right within 2^-16; a row's take the place of its logits, `deep` high parts and `deep` low ones.
            const bool copied = n == 0 && p.mode == CSA_K0_COPY_FIRST;  // the sink is a copy of the row's own first token
#pragma unroll 1
            for (int r = warp; r < kTreeRows; r += kTreeWarps) {
                const int t = (first + r) % p.T;
                const unsigned long long path = r < rows && t < c ? s_path[t] : 0;
                const bool in0 = path >> lane & 1, in1 = path >> (lane + 32) & 1;
                const int root = copied ? __ffsll((long long)path) : 0;
                float *s = S + r * pitch, *right = Rt + r * pitch, *left = Lf + r * pitch, l = 0.0f;
                if (copied && path) {
                    if (lane == 0) s[0] = s[root];
                    __syncwarp();
                }
                float m = path ? s[0] : -INFINITY;
                if (in0) m = fmaxf(m, s[lane + 1]);
                if (in1) m = fmaxf(m, s[lane + 33]);
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
                for (int j = lane; j < deep; j += 32) right[j] = left[j] = 0.0f;
                __syncwarp();
#pragma unroll 1
                for (int u = lane; u < c; u += 32) {
                    if (!(u < 32 ? in0 : in1)) continue;
                    const int up = s_up[u] + 1;
                    const float before = s[up], own = s[u + 1], pb = ex2_approx(before - m), po = ex2_approx(own - m);
                    float lf, rt, none0, none1;
                    intervals(before, own, before, own, pb, po, pb, po, lf, rt, none0, none1);
                    right[u + 1] = rt;
                    left[up] = lf;
                }
                __syncwarp();
                __nv_bfloat16 *hi = reinterpret_cast<__nv_bfloat16 *>(s), *lo = hi + deep;
#pragma unroll 1
                for (int j = lane; j < deep; j += 32) {
                    const bool in = j == 0 ? path != 0 : j <= 64 && (path >> (j - 1) & 1);
                    float w = 0.0f;
                    if (in) {
                        w = right[j] + left[j];
                        l += w;
                        if (copied) w = j == 0 ? 0.0f : j == root ? w + left[0] : w;
                        w *= s_sv[j];
                    }
                    right[j] = w;
                    hi[j] = __float2bfloat16_rn(w);
                    lo[j] = __float2bfloat16_rn(w - __bfloat162float(hi[j]));
                }
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
                if (lane == 0) {
                    s_m[r] = m;
                    s_l[r] = path & s_bad ? NAN : l;
                }
            }
            if (tid == 0 && s_bad) atomicCAS(&g_paged_status, 0, CSA_ERR_INVALID_ARG);
            __syncthreads();
            // Sums over the drafted tokens: a warp has D / 8 of the columns, a lane columns col0 + 8 i + 2 q (+ 1) of rows
            // g and g + 8.
            constexpr int CW = D / kTreeWarps;
            const int col0 = warp * CW;
            float o[CW / 8][4] = {};
            if (!(flags & 0x0202020202020202ull)) {
                const uint32_t wa = smem_u32(S) + (lane & 15) * pitch * 4 + (lane >> 4) * 16,
                               va = smem_u32(Vs) + (lane & 15) * Row + (col0 + (CW > 8 ? 8 * (lane >> 4) : 0)) * 2;
#pragma unroll 1
                for (int ks = 0; ks < (have + 15) / 16; ++ks) {
                    uint32_t hi[4], lo[4];
                    ldsm(wa + 32 * ks, hi);
                    ldsm(wa + 32 * ks + 2 * deep, lo);
                    if constexpr (CW == 8) {
                        uint32_t b0, b1;
                        ldsm_t2(va + 16 * ks * Row, b0, b1);
                        mma(o[0], hi, b0, b1);
                        mma(o[0], lo, b0, b1);
                    } else {
#pragma unroll
                        for (int i = 0; i < CW / 16; ++i) {
                            uint32_t v[4];
                            ldsm_t(va + 16 * ks * Row + 32 * i, v);
                            mma(o[2 * i], hi, v[0], v[1]);
                            mma(o[2 * i + 1], hi, v[2], v[3]);
                            mma(o[2 * i], lo, v[0], v[1]);
                            mma(o[2 * i + 1], lo, v[2], v[3]);
                        }
                    }
                }
            } else {  // a row must not see what is not finite in the others' tokens
#pragma unroll 1
                for (int k = 0; k < 2; ++k) {
                    const int r = g + 8 * k, t = (first + r) % p.T;
                    const unsigned long long on = r < rows && t < c ? s_path[t] : 0;
#pragma unroll 1
                    for (int j = 0; j < have; ++j) {
                        const float w = Rt[r * pitch + j];
                        if (!(j == 0 ? w != 0.0f : on >> (j - 1) & 1)) continue;
#pragma unroll
                        for (int i = 0; i < CW / 8; ++i) {
                            const uint32_t x = *reinterpret_cast<const uint32_t *>(Vs + j * Row + (col0 + 8 * i + 2 * q) * 2);
                            const float x0 = __uint_as_float(x << 16), x1 = __uint_as_float(x & 0xffff0000u);
                            if (k == 0) {
                                o[i][0] = fmaf(w, x0, o[i][0]);
                                o[i][1] = fmaf(w, x1, o[i][1]);
                            } else {
                                o[i][2] = fmaf(w, x0, o[i][2]);
                                o[i][3] = fmaf(w, x1, o[i][3]);
                            }
                        }
                    }
                }
            }
            __syncthreads();  // the weights are read: their place and the queries' are the sums'
            float *Od = reinterpret_cast<float *>(Qs);
#pragma unroll
            for (int i = 0; i < CW / 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; e += 2)
                    *reinterpret_cast<float2 *>(Od + (g + 4 * e) * D + col0 + 8 * i + 2 * q) = make_float2(o[i][e], o[i][e + 1]);
            __syncthreads();
            after_previous();
            // the parts of the tokens before the draft
            const int4 seg = p.joins[segment];
            const bool any = n > 0 && c > 0;
            if (any && (seg.x != segment || seg.y < -1 || (seg.y >= 0 && (seg.z < seg.y || seg.z >= p.workers))))
                return;  // left over, where a wait has run out and the parts are undefined
            auto slot_of = [&](int cc) {
                return seg.y < 0 ? (2 * (long long)p.workers + segment) * p.HB : ((long long)cc * 2 + (cc == seg.y ? seg.w : 0)) * p.HB;
            };
            const int c0 = seg.y < 0 ? 0 : seg.y, c1 = seg.y < 0 ? 0 : seg.z;
            const int in_block = first - hb * p.HB;  // row of the parts
            if (!any || c1 - c0 < 16) {  // few parts: D / 8 lanes have a row, eight columns each
                constexpr int Lanes = D / 8, Batch = 2;
#pragma unroll 1
                for (int r = tid / Lanes; r < rows; r += kTreeThreads / Lanes) {
                    const int col = tid % Lanes * 8, t = (first + r) % p.T;
                    float M = -INFINITY, sum = 0.0f, acc[8] = {};
                    if (any && t < c) {
                        // a part's slot is two behind the one before, the first one's by seg.w less
                        long long slot = slot_of(c0) + in_block + r;
                        const long long step = 2 * p.HB - (seg.y < 0 ? 0 : seg.w * p.HB);
#pragma unroll 1
                        for (int cc = c0; cc <= c1; cc += Batch) {
                            float2 ml[Batch], x[Batch][4];  // parts lie on 8 bytes
#pragma unroll
                            for (int e = 0; e < Batch; ++e) {
                                const bool there = cc + e <= c1;
                                ml[e] = make_float2(-INFINITY, 0.f);
                                if (there) ml[e] = *reinterpret_cast<const float2 *>(p.part_ml + 2 * slot);
                                const float2 *at = reinterpret_cast<const float2 *>(p.part_o + slot * D + col);
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    x[e][i] = make_float2(0.f, 0.f);
                                    if (there) x[e][i] = at[i];
                                }
                                slot += cc + e == c0 ? step : 2 * p.HB;
                            }
                            float top = M;
#pragma unroll
                            for (int e = 0; e < Batch; ++e) top = fmaxf(top, ml[e].x);
                            const float f = ex2_approx(M - top);
                            M = top;
                            sum *= f;
#pragma unroll
                            for (int i = 0; i < 8; ++i) acc[i] *= f;
#pragma unroll
                            for (int e = 0; e < Batch; ++e) {
                                const float fe = ex2_approx(ml[e].x - top);
                                sum = fmaf(fe, ml[e].y, sum);
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    acc[2 * i] = fmaf(fe, x[e][i].x, acc[2 * i]);
                                    acc[2 * i + 1] = fmaf(fe, x[e][i].y, acc[2 * i + 1]);
                                }
                            }
                        }
                    }
                    uint4 out = make_uint4(0u, 0u, 0u, 0u);
                    float lse = -INFINITY;
                    if (t < c) {  // else no such token
                        const float top = fmaxf(M, s_m[r]), f0 = any ? ex2_approx(M - top) : 0.0f, f1 = ex2_approx(s_m[r] - top);
                        const float total = fmaf(f0, sum, f1 * s_l[r]), inv = 1.0f / total;
                        const float4 *od = reinterpret_cast<const float4 *>(Od + r * D + col);
                        const float4 y = od[0], z = od[1];
                        lse = (top + log2f(total)) * kLn2;
                        out.x = pack_bf16x2(fmaf(f0, acc[0], f1 * y.x) * inv, fmaf(f0, acc[1], f1 * y.y) * inv);
                        out.y = pack_bf16x2(fmaf(f0, acc[2], f1 * y.z) * inv, fmaf(f0, acc[3], f1 * y.w) * inv);
                        out.z = pack_bf16x2(fmaf(f0, acc[4], f1 * z.x) * inv, fmaf(f0, acc[5], f1 * z.y) * inv);
                        out.w = pack_bf16x2(fmaf(f0, acc[6], f1 * z.z) * inv, fmaf(f0, acc[7], f1 * z.w) * inv);
                    }
                    *reinterpret_cast<uint4 *>(p.out + (out0 + r) * D + col) = out;
                    if (p.lse && col == 0) p.lse[out0 + r] = lse;
                }
            } else {  // the block's warps share a row's parts
                constexpr int V = D / 32, Batch = D == 256 ? 2 : 4;
                for (int r = 0; r < rows; ++r) {
                    const int t = (first + r) % p.T;
                    float M = -INFINITY, sum = 0.0f, acc[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
                    if (t < c)
                        for (int base = c0 + warp; base <= c1; base += Batch * kTreeWarps) {
                            float2 ml[Batch], x[Batch][V / 2];
#pragma unroll
                            for (int k = 0; k < Batch; ++k) {
                                const int cc = base + k * kTreeWarps;
                                ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
                                for (int i = 0; i < V / 2; ++i) x[k][i] = make_float2(0.f, 0.f);
                                if (cc <= c1) {
                                    const long long slot = slot_of(cc) + in_block + r;
                                    ml[k] = *reinterpret_cast<const float2 *>(p.part_ml + 2 * slot);
#pragma unroll
                                    for (int i = 0; i < V / 2; ++i)
                                        x[k][i] = *reinterpret_cast<const float2 *>(p.part_o + slot * D + 64 * i + 2 * lane);
                                }
                            }
                            float top = M;
#pragma unroll
                            for (int k = 0; k < Batch; ++k) top = fmaxf(top, ml[k].x);
                            const float f = ex2_approx(M - top);
                            M = top;
                            sum *= f;
#pragma unroll
                            for (int i = 0; i < V; ++i) acc[i] *= f;
#pragma unroll
                            for (int k = 0; k < Batch; ++k) {
                                const float fk = ex2_approx(ml[k].x - top);
                                sum = fmaf(fk, ml[k].y, sum);
#pragma unroll
                                for (int i = 0; i < V / 2; ++i) {
                                    acc[2 * i] = fmaf(fk, x[k][i].x, acc[2 * i]);
                                    acc[2 * i + 1] = fmaf(fk, x[k][i].y, acc[2 * i + 1]);
                                }
                            }
                        }
                    __syncthreads();  // sums may still be read for the row before
#pragma unroll
                    for (int i = 0; i < V / 2; ++i)
                        *reinterpret_cast<float2 *>(sums + warp * D + 64 * i + 2 * lane) = make_float2(acc[2 * i], acc[2 * i + 1]);
                    if (lane == 0) {
                        s_pm[warp] = M;
                        s_pl[warp] = sum;
                    }
                    __syncthreads();
                    if (warp > 0) continue;
                    float top = t < c ? s_m[r] : 0.0f;
#pragma unroll
                    for (int k = 0; k < kTreeWarps; ++k) top = fmaxf(top, s_pm[k]);
                    const float f1 = t < c ? ex2_approx(s_m[r] - top) : 0.0f;
                    float total = t < c ? f1 * s_l[r] : 0.0f;
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[i] = f1 * Od[r * D + 64 * (i / 2) + 2 * lane + (i & 1)];
#pragma unroll
                    for (int k = 0; k < kTreeWarps; ++k) {
                        const float f = ex2_approx(s_pm[k] - top);
                        total = fmaf(f, s_pl[k], total);
#pragma unroll
                        for (int i = 0; i < V; ++i) acc[i] = fmaf(f, sums[k * D + 64 * (i / 2) + 2 * lane + (i & 1)], acc[i]);
                    }
                    const float inv = 1.0f / total;
#pragma unroll
                    for (int i = 0; i < V / 2; ++i)
                        *reinterpret_cast<uint32_t *>(p.out + (out0 + r) * D + 64 * i + 2 * lane) =
                            t >= c ? 0u : pack_bf16x2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
                    if (lane == 0 && p.lse) p.lse[out0 + r] = t >= c ? -INFINITY : (top + log2f(total)) * kLn2;
                }
            }
        }
        first += gridDim.y * p.RB;
        if (first >= last_row) break;
        __syncthreads();  // the queries and the weights are read
    }
}

template <int D, int KIND>
int launch_tree(TreeParams &p, cudaStream_t stream) {
    auto kern = tree_kernel<D, KIND>;
    const int smem = TreeSmem<D>(p.T).bytes;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TreeSmem<D>(64).bytes) != cudaSuccess)
        return CSA_ERR_CUDA;
    // fewer rows per block where a segment has many parts
    const long long segments = (long long)p.B * p.Hkv * p.GB;
    p.RB = kTreeRows;
    while (p.RB > 1 && segments * ((p.HB + p.RB - 1) / p.RB) < kGrid) p.RB /= 2;
    // beyond four rounds of blocks several groups each, that the drafted tokens are copied once for them (64 drafted over
    // 16 sequences of 4096 to 8192 rows, 32 heads on 8, d = 256: 520 us, 549 with a group each)
    unsigned groups = (unsigned)((p.HB + p.RB - 1) / p.RB);
    while (groups > 1 && segments * groups > 4ll * kTreeBlocks<D> * kGrid) groups = (groups + 1) / 2;
    const dim3 grid((unsigned)segments, groups);
    return launch_after_previous(kern, grid, kTreeThreads, smem, stream, p) == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

template <int KIND>
int launch_tree_of(TreeParams &p, int d, cudaStream_t stream) {
    if (d == 64) return launch_tree<64, KIND>(p, stream);
    if (d == 128) return launch_tree<128, KIND>(p, stream);
    return launch_tree<256, KIND>(p, stream);
}

// Rows of a cached head above which they go to the kernel of csa_rows.cuh: at 17 the other one reads the cache twice.
// 16 sequences of 4096 to 8192 rows, 8 cached heads, d = 128, 17 rows: 81 us there and 125 here (e4m3 97 and 115, int8
// 109 and 121), 48 rows 97 and 178 (e4m3 110 and 164); d = 64, 32 rows 65 and 96; d = 256 161 and 283 (e4m3 183 and 251);
// one sequence of 333 rows 12.3 and 14.6, of 2000 18.8 and 17.5; 64 ragged ones of 1 to 8192, e4m3, 32 rows 109 and 98.
constexpr int kMany = 16;

// Where the parts lie: notes, maxima and sums, unnormalised outputs.
struct TreeScratch {
    bool many;
    int GB, HB, parts_of;  // workers that leave parts
    long long segments, slots, notes;
    TreeScratch(int B, int Hq, int Hkv, int T, int d) {
        const int rows = Hq / Hkv * T;
        many = rows > kMany;
        GB = many ? row_blocks(rows) : head_blocks(rows);
        HB = GB ? (rows + GB - 1) / GB : 0;
        parts_of = (int)(many ? row_workers(d) : workers(d));
        segments = (long long)B * Hkv * GB;
        slots = 2 * parts_of + segments;
        notes = std::max((long long)parts_of, segments);
    }
    long long bytes(int d) const { return notes * (long long)sizeof(int4) + slots * HB * (d + 2) * (long long)sizeof(float); }
};

}  // namespace

long long csa_decode_tree_scratch_bytes(int B, int Hq, int Hkv, int T, int d) {
    return TreeScratch(B, Hq, Hkv, T, d).bytes(d);
}

int csa_decode_tree_run(const csa_paged_args &args, const int *parents, const int *counts, int T, int d, int kind,
                        void *scratch, cudaStream_t stream) {
    const TreeScratch at(args.B, args.Hq, args.Hkv, T, d);
    csa_paged_args a = args;
    a.Hq = args.Hq * T;
    a.counts = counts;
    a.T = T;
    auto run = kind == CSA_BF16   ? (at.many ? csa_rows_bf16_run : csa_decode_paged_run)
               : kind == CSA_E4M3 ? (at.many ? csa_rows_e4m3_run : csa_decode_paged_e4m3_run)
                                  : (at.many ? csa_rows_int8_run : csa_decode_paged_int8_run);
    const int rc = run(a, scratch, d, stream);
    if (rc != CSA_OK) return rc;
    TreeParams p = {};
    p.q = static_cast<const __nv_bfloat16 *>(args.q);
    p.k = args.k_pages;
    p.v = args.v_pages;
    p.scales = args.row_scales;
    p.k0 = static_cast<const __nv_bfloat16 *>(args.k0);
    p.v0 = static_cast<const __nv_bfloat16 *>(args.v0);
    p.table = args.block_table;
    p.seqlens = args.seqlens;
    p.counts = counts;
    p.parents = parents;
    p.out = static_cast<__nv_bfloat16 *>(args.out);
    p.lse = args.lse;
    p.joins = static_cast<const int4 *>(scratch);
    const float *parts = reinterpret_cast<const float *>(p.joins + at.notes);
    p.part_o = at.many ? parts : parts + at.slots * at.HB * 2;
    p.part_ml = at.many ? parts + at.slots * at.HB * d : parts;
    p.workers = at.parts_of;
    p.B = args.B;
    p.Hkv = args.Hkv;
    p.T = T;
    p.P = args.P;
    p.S = args.S;
    p.M = args.M;
    p.rows = args.Hq / args.Hkv * T;
    p.GB = at.GB;
    p.HB = at.HB;
    p.qscale = args.scale * kLog2e;
    p.mode = args.mode;
    if (kind == CSA_BF16) return launch_tree_of<CSA_BF16>(p, d, stream);
    if (kind == CSA_E4M3) return launch_tree_of<CSA_E4M3>(p, d, stream);
    return launch_tree_of<CSA_INT8>(p, d, stream);
}

int *csa_tree_status_word(void) { return status_word(); }

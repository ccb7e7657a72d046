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
// What bounds it: the first stretch (csa_paged.cuh); the second is bound by latency, a
// few dependent trips to memory and two small products.
#include "csa_rows.cuh"

namespace {

constexpr int kTreeThreads = 256, kTreeWarps = kTreeThreads / 32;
constexpr int kTreeRows = 16;       // rows of a block's products
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
    int B, Hkv, G, T, P, S, M;
    int rows, GB, HB;      // rows of a group (G * T), blocks of them, rows per block
    int RB;                // rows per block of this kernel, at most kTreeRows
    float qscale;
    int mode;
};

// Shared memory, by the positions that T asks for: few drafted tokens leave room for more blocks per SM.
template <int D>
struct TreeSmem {
    static constexpr int Row = 2 * D + 16;  // bytes of a cached row: 16 more, so that eight rows meet no bank twice
    int deep, pitch, S, W, Left, Parts, bytes;  // positions; pitch of the weights in elements; offsets
    __host__ __device__ explicit TreeSmem(int T) {
        deep = (T + 16) / 16 * 16;
        pitch = deep + 4;
        S = 2 * deep * Row;  // behind the keys and the values
        W = S + kTreeRows * pitch * 4;
        Left = W + kTreeRows * pitch * 4;
        Parts = Left + kTreeRows * pitch * 4;  // [warps][D + 2] of a row's parts
        bytes = Parts + kTreeWarps * (D + 2) * 4;
        // the sums over the drafted tokens take the keys' place, if they fit
        if (deep * Row < kTreeRows * D * 4) bytes += kTreeRows * D * 4;
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
        values_of<KIND == CSA_E4M3, 8>(raw, 1.0f, x);
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
}

__device__ __forceinline__ bool any_not_finite(const uint4 &x) {
    auto bad = [](uint32_t w) { return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u; };
    return bad(x.x) || bad(x.y) || bad(x.z) || bad(x.w);
}

template <int D, int KIND>
__global__ void __launch_bounds__(kTreeThreads, 4) tree_kernel(const __grid_constant__ TreeParams p) {
    constexpr int Row = TreeSmem<D>::Row;
    const TreeSmem<D> L(p.T);
    const int deep = L.deep, kPitch = L.pitch, kV = deep * Row;  // the values behind the keys
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ unsigned long long s_path[64];
    __shared__ int s_jump[64], s_up[64];
    __shared__ unsigned long long s_bad;  // nodes whose parent is out of range
    __shared__ int s_page, s_wild;        // a page out of range; values that are not finite
    __shared__ float s_sk[kDeep], s_sv[kDeep], s_m[kTreeRows], s_l[kTreeRows], s_pm[kTreeWarps], s_pl[kTreeWarps];
    float *S = reinterpret_cast<float *>(raw + L.S), *W = reinterpret_cast<float *>(raw + L.W),
          *Lf = reinterpret_cast<float *>(raw + L.Left), *sums = reinterpret_cast<float *>(raw + L.Parts);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
    const int segment = blockIdx.x, heads = p.Hkv * p.GB;
    const int b = segment / heads, head = segment - b * heads, hk = head / p.GB, hb = head - hk * p.GB;
    const int first = hb * p.HB + blockIdx.y * p.RB;  // row of the group
    const int rows = min(p.RB, min((hb + 1) * p.HB, p.rows) - first);
    if (rows <= 0) return;
    // What the draft needs was written before the kernel that forms the parts began, and this one begins
    // after it did; its parts are waited for below.
    const int len = p.seqlens[b], c = p.counts ? p.counts[b] : p.T, n = len - c;
    const bool sound = c >= 0 && c <= p.T && n >= 0 && len <= (long long)p.M * p.S;
    const long long out0 = ((long long)b * p.Hkv + hk) * p.rows + first;  // row of out and of lse
    if (tid < 64) {
        const int up = sound && tid < c ? (p.parents ? p.parents[(long long)b * p.T + tid] : tid - 1) : -1;
        const bool bad = sound && tid < c && (up < -1 || up >= tid);
        s_up[tid] = s_jump[tid] = bad ? -1 : up;
        s_path[tid] = 1ull << tid;
        const unsigned at = __ballot_sync(0xffffffffu, bad);
        if (lane == 0) reinterpret_cast<unsigned *>(&s_bad)[warp] = at;
    }
    if (tid == 0) s_page = s_wild = 0;
    __syncthreads();
    // ancestors, twice as far each time
    if (warp < 2) {
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
    }
    // the cached rows: position 0 is the last one before the draft, 1 + u is drafted token u
    const int have = sound ? c + 1 : 0;
    for (int i = tid; i < deep * (D / 8); i += kTreeThreads) {
        const int j = i / (D / 8), col = (i - j * (D / 8)) * 8;
        uint4 xk = make_uint4(0u, 0u, 0u, 0u), xv = xk;
        if (j < have) {
            const int at = n - 1 + j;
            float2 s = make_float2(1.0f, 1.0f);
            if (at >= 0) {
                const int page = p.table[(long long)b * p.M + at / p.S];
                if (page >= 0 && page < p.P) {
                    const long long row = ((long long)page * p.Hkv + hk) * p.S + at % p.S;
                    constexpr int E = KIND == CSA_BF16 ? 2 : 1;
                    xk = as_bf16<KIND>(static_cast<const uint8_t *>(p.k) + row * D * E, col);
                    xv = as_bf16<KIND>(static_cast<const uint8_t *>(p.v) + row * D * E, col);
                    if (KIND != CSA_BF16) s = *reinterpret_cast<const float2 *>(p.scales + 2 * row);
                } else {
                    s_page = 1;
                }
            } else if (p.mode == CSA_K0_GIVEN) {
                xk = *reinterpret_cast<const uint4 *>(p.k0 + (long long)hk * D + col);
                xv = *reinterpret_cast<const uint4 *>(p.v0 + (long long)hk * D + col);
            }
            if (col == 0) {
                s_sk[j] = s.x;
                s_sv[j] = s.y;
            }
            if (any_not_finite(xv)) s_wild = 1;
        } else if (col == 0) {
            s_sk[j] = s_sv[j] = 0.0f;
        }
        *reinterpret_cast<uint4 *>(raw + j * Row + col * 2) = xk;
        *reinterpret_cast<uint4 *>(raw + kV + j * Row + col * 2) = xv;
    }
    __syncthreads();
    if (!sound || s_page) {
        after_previous();  // this kernel must not end before the one that forms the parts
        for (int i = tid; i < rows * D; i += kTreeThreads) p.out[out0 * D + i] = __float2bfloat16_rn(NAN);
        if (p.lse && tid < rows) p.lse[out0 + tid] = NAN;
        if (tid == 0) atomicCAS(&g_paged_status, 0, CSA_ERR_INVALID_ARG);
        return;
    }
    // logits, in log2 units: a warp has eight positions
    for (int t = warp; t < (have + 7) / 8; t += kTreeWarps) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f}, acc2[4] = {0.f, 0.f, 0.f, 0.f};
        const uint32_t *q0 = reinterpret_cast<const uint32_t *>(p.q + (out0 + g) * D), *q1 = q0 + 4 * D;
        const uint32_t *kr = reinterpret_cast<const uint32_t *>(raw + (8 * t + g) * Row);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const uint32_t a[4] = {g < rows ? q0[i * 8 + q] : 0u, g + 8 < rows ? q1[i * 8 + q] : 0u,
                                   g < rows ? q0[i * 8 + 4 + q] : 0u, g + 8 < rows ? q1[i * 8 + 4 + q] : 0u};
            mma(i & 1 ? acc2 : acc, a, kr[i * 8 + q], kr[i * 8 + 4 + q]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = 8 * t + 2 * q + (e & 1);
            S[(g + 8 * (e >> 1)) * kPitch + j] = (acc[e] + acc2[e]) * (p.qscale * s_sk[j]);
        }
    }
    __syncthreads();
    // weights: a warp has a row, a lane positions lane, lane + 32 and, lane 0, 64
    for (int r = warp; r < kTreeRows; r += kTreeWarps) {
        float *s = S + r * kPitch, *w = W + r * kPitch, *lf = Lf + r * kPitch;
        const int t = (first + r) % p.T;
        if (r >= rows || t >= c) {
            for (int j = lane; j < deep; j += 32) w[j] = 0.0f;
            continue;
        }
        const unsigned long long path = s_path[t];
        if (n == 0 && p.mode == CSA_K0_COPY_FIRST) {  // the sink is a copy of the row's own first token
            if (lane == 0) s[0] = s[__ffsll((long long)path)];
            __syncwarp();
        }
        float a[3], m = -INFINITY;
        bool in[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int j = lane + 32 * i;
            in[i] = j == 0 || (j <= c && (path >> (j - 1) & 1));
            if (j > 64) in[i] = false;
            a[i] = in[i] ? s[j] : -INFINITY;
            m = fmaxf(m, a[i]);
            if (j < deep) w[j] = lf[j] = 0.0f;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        __syncwarp();
        float right[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int j = lane + 32 * i;
            right[i] = 0.0f;
            if (!in[i] || j == 0) continue;
            const int up = s_up[j - 1] + 1;
            const float before = s[up], pb = ex2_approx(before - m), pa = ex2_approx(a[i] - m);
            float left, none0, none1;
            intervals(before, a[i], before, a[i], pb, pa, pb, pa, left, right[i], none0, none1);
            lf[up] = left;
        }
        __syncwarp();
        float l = 0.0f;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int j = lane + 32 * i;
            if (!in[i]) continue;
            const float x = right[i] + lf[j];
            l += x;
            w[j] = x * s_sv[j];
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        if (n == 0 && p.mode == CSA_K0_COPY_FIRST) {
            __syncwarp();
            if (lane == 0) {
                const int root = __ffsll((long long)path);
                w[root] += lf[0] * s_sv[root];
                w[0] = 0.0f;
            }
        }
        if (lane == 0) {
            s_m[r] = m;
            s_l[r] = path & s_bad ? NAN : l;
        }
    }
    if (tid == 0 && s_bad) atomicCAS(&g_paged_status, 0, CSA_ERR_INVALID_ARG);
    __syncthreads();
    // sums over the drafted tokens, into S: a warp has D / 8 of the columns.  A weight is two bf16 numbers, right
    // within 2^-16.
    constexpr int CW = D / kTreeWarps;
    float o[CW / 8][4] = {};
    if (!s_wild) {
        const int col0 = warp * CW;
#pragma unroll 1
        for (int ks = 0; ks < (have + 15) / 16; ++ks) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 x = *reinterpret_cast<const float2 *>(W + (g + 8 * (i & 1)) * kPitch + 16 * ks + 8 * (i >> 1) + 2 * q);
                hi[i] = pack_bf16x2(x.x, x.y);
                lo[i] = pack_bf16x2(x.x - __uint_as_float(hi[i] << 16), x.y - __uint_as_float(hi[i] & 0xffff0000u));
            }
#pragma unroll
            for (int i = 0; i < CW / 8; ++i) {
                // rows 16 ks + 2 q (+ 1, + 8, + 9) of column col0 + 8 i + g
                const uint16_t *at = reinterpret_cast<const uint16_t *>(raw + kV + (16 * ks + 2 * q) * Row) + col0 + 8 * i + g;
                const uint32_t b0 = at[0] | (uint32_t)at[Row / 2] << 16, b1 = at[8 * (Row / 2)] | (uint32_t)at[9 * (Row / 2)] << 16;
                mma(o[i], hi, b0, b1);
                mma(o[i], lo, b0, b1);
            }
        }
    }
    __syncthreads();
    // [kTreeRows][D]: over the keys, or behind everything where they are fewer
    float *Od = reinterpret_cast<float *>(raw + (deep * Row < kTreeRows * D * 4 ? L.bytes - kTreeRows * D * 4 : 0));
    if (!s_wild) {
#pragma unroll
        for (int i = 0; i < CW / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) Od[(g + 8 * (e >> 1)) * D + warp * CW + 8 * i + 2 * q + (e & 1)] = o[i][e];
    } else {  // a row must not see what is not finite in the others' tokens
        for (int i = tid; i < rows * D; i += kTreeThreads) {
            const int r = i / D, col = i - r * D, t = (first + r) % p.T;
            const unsigned long long path = t < c ? s_path[t] : 0;
            float sum = 0.0f;
            for (int j = 0; j < have; ++j)
                if (j == 0 ? W[r * kPitch] != 0.0f : path >> (j - 1) & 1)
                    sum = fmaf(W[r * kPitch + j], __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(raw + kV + j * Row + col * 2) << 16), sum);
            Od[r * D + col] = sum;
        }
    }
    __syncthreads();
    after_previous();
    // the parts of the tokens before the draft
    const int4 seg = p.joins[segment];
    const bool any = n > 0;
    if (any && (seg.x != segment || seg.y < -1 || (seg.y >= 0 && (seg.z < seg.y || seg.z >= p.workers))))
        return;  // left over, where a wait has run out and the parts are undefined
    constexpr int V = D / 32, kBatch = D == 256 ? 2 : 4;
    auto slot_of = [&](int cc) {
        return seg.y < 0 ? (2 * (long long)p.workers + segment) * p.HB : ((long long)cc * 2 + (cc == seg.y ? seg.w : 0)) * p.HB;
    };
    const int c0 = seg.y < 0 ? 0 : seg.y, c1 = seg.y < 0 ? 0 : seg.z;
    const int in_block = first - hb * p.HB;  // row of the parts
    // A warp per row where the parts are few; else the block's warps share a row's parts.
    const bool few = !any || c1 - c0 < 16;
    for (int r = few ? warp : 0; r < rows; r += few ? kTreeWarps : 1) {
        const int t = (first + r) % p.T;
        float M = -INFINITY, sum = 0.0f, acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.0f;
        if (any && t < c) {
            const int step = few ? 1 : kTreeWarps;
            for (int base = c0 + (few ? 0 : warp); base <= c1; base += kBatch * step) {
                float2 ml[kBatch], x[kBatch][V / 2];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int cc = base + k * step;
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
                for (int k = 0; k < kBatch; ++k) top = fmaxf(top, ml[k].x);
                const float f = ex2_approx(M - top);
                M = top;
                sum *= f;
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] *= f;
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const float fk = ex2_approx(ml[k].x - top);
                    sum = fmaf(fk, ml[k].y, sum);
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        acc[2 * i] = fmaf(fk, x[k][i].x, acc[2 * i]);
                        acc[2 * i + 1] = fmaf(fk, x[k][i].y, acc[2 * i + 1]);
                    }
                }
            }
        }
        if (!few) {
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
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < kTreeWarps; ++k) top = fmaxf(top, s_pm[k]);
            M = top;
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = 0.0f;
#pragma unroll
            for (int k = 0; k < kTreeWarps; ++k) {
                const float f = ex2_approx(s_pm[k] - top);
                sum = fmaf(f, s_pl[k], sum);
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] = fmaf(f, sums[k * D + 64 * (i / 2) + 2 * lane + (i & 1)], acc[i]);
            }
        }
        if (t >= c) {  // no such token
#pragma unroll
            for (int i = 0; i < V / 2; ++i) *reinterpret_cast<uint32_t *>(p.out + (out0 + r) * D + 64 * i + 2 * lane) = 0u;
            if (lane == 0 && p.lse) p.lse[out0 + r] = -INFINITY;
            continue;
        }
        const float top = fmaxf(M, s_m[r]), f0 = any ? ex2_approx(M - top) : 0.0f, f1 = ex2_approx(s_m[r] - top);
        const float total = fmaf(f0, sum, f1 * s_l[r]), inv = 1.0f / total;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 x = *reinterpret_cast<const float2 *>(Od + r * D + 64 * i + 2 * lane);
            *reinterpret_cast<uint32_t *>(p.out + (out0 + r) * D + 64 * i + 2 * lane) =
                pack_bf16x2(fmaf(f0, acc[2 * i], f1 * x.x) * inv, fmaf(f0, acc[2 * i + 1], f1 * x.y) * inv);
        }
        if (lane == 0 && p.lse) p.lse[out0 + r] = (top + log2f(total)) * kLn2;
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
    const dim3 grid((unsigned)segments, (unsigned)((p.HB + p.RB - 1) / p.RB));
    return launch_after_previous(kern, grid, kTreeThreads, smem, stream, p) == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

template <int KIND>
int launch_tree_of(TreeParams &p, int d, cudaStream_t stream) {
    if (d == 64) return launch_tree<64, KIND>(p, stream);
    if (d == 128) return launch_tree<128, KIND>(p, stream);
    return launch_tree<256, KIND>(p, stream);
}

// Rows of a cached head above which they go to the kernel of csa_rows.cuh.
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
    p.G = args.Hq / args.Hkv;
    p.T = T;
    p.P = args.P;
    p.S = args.S;
    p.M = args.M;
    p.rows = p.G * T;
    p.GB = at.GB;
    p.HB = at.HB;
    p.qscale = args.scale * kLog2e;
    p.mode = args.mode;
    if (kind == CSA_BF16) return launch_tree_of<CSA_BF16>(p, d, stream);
    if (kind == CSA_E4M3) return launch_tree_of<CSA_E4M3>(p, d, stream);
    return launch_tree_of<CSA_INT8>(p, d, stream);
}

int csa_tree_take_status(void) { return take_status(); }

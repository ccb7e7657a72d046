// Rows of a key-value cache held in 8 bits: quantised as they are written into
// their pages (keys turned on the way, queries turned beside), and rows read back
// in order as 16- or 32-bit values.
//
// A row x of d values is held as d codes and a scale s, x ~ code * s:
//   e4m3  s = the smallest power of two with max|x| / s <= 448.  x / s is then
//         exact, so that a code is the nearest number of the format (ties to even)
//         and not the nearest to a rounded quotient; the format's relative step is
//         the same at every power of two, so nothing is lost against s = max / 448
//         but an octave of its subnormal range, 2^-9 s at the bottom.
//   int8  s = max|x| / 127, code = the integer nearest to x * (127 / max|x|), both
//         factors rounded to fp32, the product not: one fma adds 1.5 * 2^23 to it and
//         rounds once.
// Rows with max|x| < 2^-100 are zeros; a row with an infinity or NaN gets the scale
// NaN and codes 0, so that what reads it shows it.
//
// What bounds it.  Each value is read once and each code written once: HBM bandwidth, and
// the instructions of the rotation (issue slots 60% busy).  8 x up to 2048 tokens, 32 heads
// on 8, d = 128 (330 MB) take 58 us, 85% of the copy bandwidth; 64 single tokens 3.2 us.
// Reading back is a copy: 754 MB of int8 rows as bf16 take 117 us, 96%; 25 MB 6.4 us.
// A power of two of lanes owns a row, 16 bytes twice per lane as in csa_rope.cu (the
// two members of 8 bf16 or 4 fp32 pairs), holds it in registers between the maximum
// and the codes, and walks over a range of heads with the token's sines and cosines.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "csa.h"
#include "csa_internal.h"
#include "csa_launch.cuh"
#include "csa_quant.cuh"
#include "csa_rotate.cuh"

namespace {

using namespace csa_dev;

constexpr int kThreads = 128;

__device__ int g_quant_status;  // sticky status word of this file's kernels

__device__ __forceinline__ void complain() { atomicCAS(&g_quant_status, 0, CSA_ERR_INVALID_ARG); }

struct Rows {
    const void *in;
    void *out;                  // of queries
    long long ib, ih, it;       // strides of in over batch, head, time, in elements
    long long ob, oh, ot;
    int H;
};

struct FillParams {
    csa_rope_plan plan;
    Rows x[3];  // queries, keys, values
    const int *positions;
    long long pa, pb, pt;  // strides over axes, batch, time
    int B, T, d;
    int lanes;             // per row, a power of two
    int heads_per_block;
    int blocks[2];         // blocks of heads of the queries, and of the keys
    uint8_t *k_pages, *v_pages;
    float *scales;
    const int *table, *seqlens, *counts;
    int P, S, M;
};

// Codes of N values by the row's factor; 4 to a word.
template <bool E4M3, int N>
__device__ __forceinline__ void store_codes(uint8_t *to, const float (&x)[N], float factor, bool zero) {
    uint32_t word[(N + 3) / 4];
#pragma unroll
    for (int i = 0; i < (N + 3) / 4; ++i) {
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = 4 * i + j < N ? x[4 * i + j < N ? 4 * i + j : 0] : 0.0f;
        word[i] = zero ? 0u : E4M3 ? to_e4m3x4(y, factor) : to_int8x4(y, factor);
    }
    if constexpr (N == 8)
        *reinterpret_cast<uint2 *>(to) = make_uint2(word[0], word[1]);
    else if constexpr (N == 4)
        *reinterpret_cast<uint32_t *>(to) = word[0];
    else
        *to = (uint8_t)word[0];
}

// A block: a range of tokens (rows of B x T) and a range of heads of one tensor.
// V elements of type T per chunk; a unit of a row is two chunks, at columns c0 and
// c1; a lane has U units.  Units [0, n/V) turn, the ones behind copy the columns
// from 2n on.
template <typename T, int V, int U, bool ADJ, bool E4M3>
__global__ void __launch_bounds__(kThreads, 8) fill_kernel(const __grid_constant__ FillParams p) {
    using C = typename Chunk<V * sizeof(T)>::type;
    __shared__ unsigned long long turn[CSA_ROPE_MAX_PAIRS];
    __shared__ unsigned char axis[CSA_ROPE_MAX_PAIRS];
    const int n = p.plan.pairs;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        turn[i] = p.plan.turn[i];
        axis[i] = p.plan.axis[i];
    }
    after_previous();
    __syncthreads();
    const int rest = (p.d - 2 * n) / V;  // chunks that do not turn
    const int units = n / V + (rest + 1) / 2;
    const int r = threadIdx.x / p.lanes, lane = threadIdx.x & (p.lanes - 1);
    const unsigned token = blockIdx.x * (kThreads / p.lanes) + r;  // B * T fits 31 bits
    bool live = token < (unsigned)p.B * p.T;
    const int b = live ? token / (unsigned)p.T : 0, t = live ? token - (unsigned)b * p.T : 0;
    int y = blockIdx.y, which = 0;
    if (y >= p.blocks[0]) {
        y -= p.blocks[0];
        which = 1;
        if (y >= p.blocks[1]) {
            y -= p.blocks[1];
            which = 2;
        }
    }
    const Rows &x = p.x[which];
    const int h0 = y * p.heads_per_block, count = min(p.heads_per_block, x.H - h0);
    const T *in = static_cast<const T *>(x.in) + b * x.ib + h0 * x.ih + t * x.it;
    T *out = static_cast<T *>(x.out) + (which == 0 ? b * x.ob + h0 * x.oh + t * x.ot : 0);
    const int len = live ? p.seqlens[b] : 0, held = !live ? 0 : p.counts ? p.counts[b] : p.T;
    const int cache_row = len - held + t;
    uint8_t *codes = nullptr;
    float *scale = nullptr;
    if (which > 0 && live) {
        if (held < 0 || held > p.T || len < held || len > (long long)p.M * p.S) {
            if (t == 0 && lane == 0) complain();
            live = false;
        } else if (t >= held) {
            live = false;
        } else {
            const int page = p.table[(long long)b * p.M + cache_row / p.S];
            if (page < 0 || page >= p.P) {
                if (lane == 0) complain();
                live = false;
            } else {
                const long long row = ((long long)page * x.H + h0) * p.S + cache_row % p.S;
                codes = (which == 1 ? p.k_pages : p.v_pages) + row * p.d;
                scale = p.scales + 2 * row + (which - 1);
            }
        }
    }
    int c0[U], c1[U];
    bool one[U], two[U], turns[U];
    float cs[U][V], sn[U][V];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int u = lane + i * p.lanes;
        const bool turned = u < n / V;
        turns[i] = turned && which < 2;
        c0[i] = turned ? (ADJ ? 2 * V * u : V * u) : 2 * n + 2 * V * (u - n / V);
        c1[i] = turned ? (ADJ ? c0[i] + V : c0[i] + n) : c0[i] + V;
        one[i] = live && u < units;
        two[i] = one[i] && c1[i] < p.d;
        if (one[i] && turns[i]) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int at = V * u + j;
                const int pos = p.positions ? p.positions[axis[at] * p.pa + b * p.pb + t * p.pt] : cache_row;
                turn_by((unsigned long long)(long long)pos * turn[at], sn[i][j], cs[i][j]);
            }
        }
    }
    union Pack {
        __device__ Pack() {}
        C raw;
        T e[V];
        __nv_bfloat162 two[V > 1 ? V * sizeof(T) / 4 : 1];
    };
    // the next head's values are asked for before this one's are used
    Pack ahead[U][2];
    auto load = [&]() {
#pragma unroll
        for (int i = 0; i < U; ++i) {
#pragma unroll
            for (int j = 0; j < V; ++j) ahead[i][0].e[j] = ahead[i][1].e[j] = narrow<T>(0.0f);
            if (one[i]) ahead[i][0].raw = *reinterpret_cast<const C *>(in + c0[i]);
            if (two[i]) ahead[i][1].raw = *reinterpret_cast<const C *>(in + c1[i]);
        }
        in += x.ih;
    };
    load();
#pragma unroll 1
    for (int h = 0; h < count; ++h) {
        float val[U][2][V];
        unsigned most = 0;  // the bits of the largest magnitude, infinities and NaN above all
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) val[i][k][j] = widen(ahead[i][k].e[j]);
        if (h + 1 < count) load();
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (one[i] && turns[i]) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    // pair j: adjacent, elements 2j and 2j + 1 of the two chunks; else element j of each
                    float &eu = !ADJ ? val[i][0][j] : val[i][2 * j / V][(2 * j) % V];
                    float &ew = !ADJ ? val[i][1][j] : val[i][(2 * j + 1) / V][(2 * j + 1) % V];
                    const float xu = eu, xw = ew;
                    eu = xu * cs[i][j] - xw * sn[i][j];
                    ew = xu * sn[i][j] + xw * cs[i][j];
                }
            }
        }
        if (which == 0) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                Pack a, c;
                if constexpr (sizeof(T) == 2 && V > 1) {  // two values by one instruction
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        a.two[j / 2] = __floats2bfloat162_rn(val[i][0][j], val[i][0][j + 1]);
                        c.two[j / 2] = __floats2bfloat162_rn(val[i][1][j], val[i][1][j + 1]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        a.e[j] = narrow<T>(val[i][0][j]);
                        c.e[j] = narrow<T>(val[i][1][j]);
                    }
                }
                if (one[i]) *reinterpret_cast<C *>(out + c0[i]) = a.raw;
                if (two[i]) *reinterpret_cast<C *>(out + c1[i]) = c.raw;
            }
        } else {
#pragma unroll
            for (int i = 0; i < U; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    most = max(most, max(__float_as_uint(val[i][0][j]) & 0x7fffffffu,
                                         __float_as_uint(val[i][1][j]) & 0x7fffffffu));
            for (int off = p.lanes / 2; off > 0; off >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, off));
            float s, factor;
            const bool zero = row_scale<E4M3>(most, s, factor);
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (one[i]) store_codes<E4M3, V>(codes + c0[i], val[i][0], factor, zero);
                if (two[i]) store_codes<E4M3, V>(codes + c1[i], val[i][1], factor, zero);
            }
            if (live && lane == 0) *scale = s;
        }
        out += x.oh;
        codes += (long long)p.S * p.d;
        scale += 2 * p.S;
    }
}

template <typename T, int V, int U, bool E4M3>
int launch_fill(FillParams &p, cudaStream_t stream) {
    const int n = p.plan.pairs, rest = (p.d - 2 * n) / V;
    const int units = n / V + (rest + 1) / 2;
    p.lanes = 1;
    while (p.lanes * U < units) p.lanes *= 2;
    const int rows = kThreads / p.lanes;
    const long long tokens = (long long)p.B * p.T, bx = (tokens + rows - 1) / rows;
    // A token's sines serve the block's heads: 32, fewer where that leaves less than three full blocks per SM.  32
    // heads on 8, d = 128: 16 x 3000 tokens take 161 us with 32, 167 with 16, 196 with 4; 8 x 512 22, 14.4 and 17.9
    // us; 8 x 128 9.0, 6.6 and 6.5.
    const long long heads = p.x[0].H + 2 * p.x[1].H;
    p.heads_per_block = 32;
    while (p.heads_per_block > 1 && bx * heads < 3 * 152 * p.heads_per_block) p.heads_per_block /= 2;
    auto blocks = [&](int H) { return (H + p.heads_per_block - 1) / p.heads_per_block; };
    auto all = [&] { return blocks(p.x[0].H) + blocks(p.x[1].H) + blocks(p.x[2].H); };
    p.blocks[0] = blocks(p.x[0].H);
    p.blocks[1] = blocks(p.x[1].H);
    auto kernel = p.plan.adjacent ? fill_kernel<T, V, U, true, E4M3> : fill_kernel<T, V, U, false, E4M3>;
    const dim3 grid((unsigned)bx, (unsigned)all());
    return launch_after_previous(kernel, grid, kThreads, 0, stream, p) == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

bool on(const void *q, uintptr_t bytes) { return reinterpret_cast<uintptr_t>(q) % bytes == 0; }

template <typename T, bool E4M3>
int run_fill(FillParams &p, cudaStream_t stream) {
    constexpr int V = 16 / (int)sizeof(T);
    bool wide = p.d % V == 0 && p.plan.pairs % V == 0 && on(p.k_pages, 8) && on(p.v_pages, 8);
    for (int i = 0; i < 3; ++i) {
        const Rows &x = p.x[i];
        if (x.H == 0) continue;
        wide = wide && on(x.in, 16) && x.ib % V == 0 && x.ih % V == 0 && x.it % V == 0;
        if (i == 0) wide = wide && on(x.out, 16) && x.ob % V == 0 && x.oh % V == 0 && x.ot % V == 0;
    }
    return wide ? launch_fill<T, V, 1, E4M3>(p, stream) : launch_fill<T, 1, 4, E4M3>(p, stream);
}

Rows rows_of(const void *in, const long long *is, void *out, const long long *os, int H, int T, int d) {
    Rows x;
    x.in = in;
    x.out = out;
    x.H = H;
    x.ib = is ? is[0] : (long long)H * T * d;
    x.ih = is ? is[1] : (long long)T * d;
    x.it = is ? is[2] : d;
    x.ob = os ? os[0] : (long long)H * T * d;
    x.oh = os ? os[1] : (long long)T * d;
    x.ot = os ? os[2] : d;
    return x;
}

// ------------------------------------------------------------------ read back
constexpr int kReadThreads = 256, kReadDeep = 4;

struct ReadParams {
    const void *k, *v;
    const float *scales;
    const int *table, *seqlens, *starts;
    void *out[2];             // keys, values
    long long ob[2], oh[2], ot[2];
    int B, H, T, d, P, S, M;
    int chunks;               // per row
    unsigned chunks_inv;      // 2^32 / chunks rounded up
    int tokens, blocks;       // per block, and blocks per (sequence, head)
};

template <int KIND>
struct Stored;
template <>
struct Stored<CSA_BF16> {
    using type = __nv_bfloat16;
};
template <>
struct Stored<CSA_F32> {
    using type = float;
};
template <>
struct Stored<CSA_E4M3> {
    using type = uint8_t;
};
template <>
struct Stored<CSA_INT8> {
    using type = uint8_t;
};

// Items are (token, chunk of V elements), keys and values each; a thread asks for all
// of its kReadDeep items before it writes the first.
template <int KIND, typename O, int V>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ ReadParams p) {
    using E = typename Stored<KIND>::type;
    constexpr bool EIGHT = KIND == CSA_E4M3 || KIND == CSA_INT8;
    using C = typename Chunk<V * sizeof(E)>::type;
    using CO = typename Chunk<V * sizeof(O)>::type;
    after_previous();
    const unsigned bh = blockIdx.x / (unsigned)p.blocks;
    const int b = bh / (unsigned)p.H, h = bh - (unsigned)b * p.H;
    const int t0 = (int)(blockIdx.x - bh * p.blocks) * p.tokens;
    const int n = p.seqlens[b], start = p.starts ? p.starts[b] : 0;
    const bool sound = n >= 0 && n <= (long long)p.M * p.S && start >= 0 && start <= n;
    if (!sound && t0 == 0 && h == 0 && threadIdx.x == 0) complain();
    const int items = min(p.tokens, p.T - t0) * p.chunks;
    // i / chunks; i is below 2^11
    auto row_of = [&](int i) { return p.chunks == 1 ? i : (int)__umulhi((unsigned)i, p.chunks_inv); };
    for (int i0 = threadIdx.x; i0 < items; i0 += kReadThreads * kReadDeep) {
        C raw[kReadDeep][2];
        float2 scale[kReadDeep];
        int state[kReadDeep];  // 0 behind the end, 1 a row, 2 no row where one should be
#pragma unroll
        for (int j = 0; j < kReadDeep; ++j) {
            const int i = i0 + j * kReadThreads;
            const int r = row_of(i), c = (i - r * p.chunks) * V;
            state[j] = 0;
            if (i >= items) continue;
            const long long row = (long long)start + t0 + r;
            state[j] = !sound ? 2 : row < n ? 1 : 0;
            if (state[j] != 1) continue;
            const int page = p.table[(long long)b * p.M + (int)row / p.S];
            if (page < 0 || page >= p.P) {
                complain();
                state[j] = 2;
                continue;
            }
            const long long at = ((long long)page * p.H + h) * p.S + (int)row % p.S;
            raw[j][0] = *reinterpret_cast<const C *>(static_cast<const E *>(p.k) + at * p.d + c);
            raw[j][1] = *reinterpret_cast<const C *>(static_cast<const E *>(p.v) + at * p.d + c);
            if (EIGHT) scale[j] = *reinterpret_cast<const float2 *>(p.scales + 2 * at);
        }
#pragma unroll
        for (int j = 0; j < kReadDeep; ++j) {
            const int i = i0 + j * kReadThreads;
            if (i >= items) continue;
            const int r = row_of(i), c = (i - r * p.chunks) * V;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                union {
                    CO raw;
                    O e[V];
                } to;
                if (state[j] == 1) {
                    if constexpr (EIGHT) {
                        float x[V];
                        values_of<KIND == CSA_E4M3, sizeof(O) == 2, V>(raw[j][w], w ? scale[j].y : scale[j].x, x);
#pragma unroll
                        for (int e = 0; e < V; ++e) to.e[e] = narrow<O>(x[e]);
                    } else {
                        to.raw = raw[j][w];
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) to.e[e] = narrow<O>(state[j] ? NAN : 0.0f);
                }
                O *out = static_cast<O *>(p.out[w]) + b * p.ob[w] + h * p.oh[w] + (t0 + r) * p.ot[w] + c;
                *reinterpret_cast<CO *>(out) = to.raw;
            }
        }
    }
}

template <int KIND, typename O, int V>
int launch_read(ReadParams &p, cudaStream_t stream) {
    p.chunks = p.d / V;
    p.chunks_inv = (unsigned)((0x100000000ull + p.chunks - 1) / p.chunks);
    p.tokens = kReadThreads * kReadDeep / p.chunks;
    if (p.tokens < 1) p.tokens = 1;
    if (p.tokens > p.T) p.tokens = p.T;
    p.blocks = (p.T + p.tokens - 1) / p.tokens;
    const long long grid = (long long)p.B * p.H * p.blocks;
    if (grid > 0x7fffffffLL) return CSA_ERR_UNSUPPORTED;
    return launch_after_previous(read_kernel<KIND, O, V>, (unsigned)grid, kReadThreads, 0, stream, p) == cudaSuccess
               ? CSA_OK
               : CSA_ERR_CUDA;
}

// V elements per chunk where every row allows it, else one.
template <int KIND, typename O, int V>
int run_read(ReadParams &p, cudaStream_t stream) {
    constexpr uintptr_t in = V * sizeof(typename Stored<KIND>::type), out = V * sizeof(O) > 16 ? 16 : V * sizeof(O);
    constexpr int E = (int)(out / sizeof(O));
    bool wide = p.d % V == 0 && on(p.k, in) && on(p.v, in);
    for (int w = 0; w < 2; ++w)
        wide = wide && on(p.out[w], out) && p.ob[w] % E == 0 && p.oh[w] % E == 0 && p.ot[w] % E == 0;
    return wide ? launch_read<KIND, O, V>(p, stream) : launch_read<KIND, O, 1>(p, stream);
}

}  // namespace

int csa_cache_append_q8_run(const csa_rope_plan *plan, const void *q, const long long *q_strides, void *q_out,
                            const long long *q_out_strides, const void *k, const long long *k_strides, const void *v,
                            const long long *v_strides, void *k_pages, void *v_pages, float *row_scales,
                            const int *block_table, const int *seqlens, const int *counts, const int *positions,
                            const long long *pos_strides, int B, int Hq, int Hkv, int T, int d, int P, int S, int M,
                            bool bf16, bool e4m3, cudaStream_t stream) {
    FillParams p = {};
    if (plan) p.plan = *plan;  // no plan: no pair turns
    p.x[0] = rows_of(q, q_strides, q_out, q_out_strides, Hq, T, d);
    p.x[1] = rows_of(k, k_strides, nullptr, nullptr, Hkv, T, d);
    p.x[2] = rows_of(v, v_strides, nullptr, nullptr, Hkv, T, d);
    p.positions = positions;
    p.pa = pos_strides ? pos_strides[0] : (long long)B * T;
    p.pb = pos_strides ? pos_strides[1] : T;
    p.pt = pos_strides ? pos_strides[2] : 1;
    p.B = B;
    p.T = T;
    p.d = d;
    p.k_pages = static_cast<uint8_t *>(k_pages);
    p.v_pages = static_cast<uint8_t *>(v_pages);
    p.scales = row_scales;
    p.table = block_table;
    p.seqlens = seqlens;
    p.counts = counts;
    p.P = P;
    p.S = S;
    p.M = M;
    if (bf16) return e4m3 ? run_fill<__nv_bfloat16, true>(p, stream) : run_fill<__nv_bfloat16, false>(p, stream);
    return e4m3 ? run_fill<float, true>(p, stream) : run_fill<float, false>(p, stream);
}

int csa_cache_read_run(const void *k_pages, const void *v_pages, const float *row_scales, const int *block_table,
                       const int *seqlens, const int *starts, void *k, const long long *k_strides, void *v,
                       const long long *v_strides, int B, int Hkv, int T, int d, int P, int S, int M, int kind,
                       int out_type, cudaStream_t stream) {
    ReadParams p = {};
    p.k = k_pages;
    p.v = v_pages;
    p.scales = row_scales;
    p.table = block_table;
    p.seqlens = seqlens;
    p.starts = starts;
    const long long *strides[2] = {k_strides, v_strides};
    p.out[0] = k;
    p.out[1] = v;
    for (int w = 0; w < 2; ++w) {
        p.ob[w] = strides[w] ? strides[w][0] : (long long)Hkv * T * d;
        p.oh[w] = strides[w] ? strides[w][1] : (long long)T * d;
        p.ot[w] = strides[w] ? strides[w][2] : d;
    }
    p.B = B;
    p.H = Hkv;
    p.T = T;
    p.d = d;
    p.P = P;
    p.S = S;
    p.M = M;
    const bool bf = out_type == CSA_BF16;
    if (kind == CSA_E4M3)
        return bf ? run_read<CSA_E4M3, __nv_bfloat16, 8>(p, stream) : run_read<CSA_E4M3, float, 4>(p, stream);
    if (kind == CSA_INT8)
        return bf ? run_read<CSA_INT8, __nv_bfloat16, 8>(p, stream) : run_read<CSA_INT8, float, 4>(p, stream);
    return bf ? run_read<CSA_BF16, __nv_bfloat16, 8>(p, stream) : run_read<CSA_F32, float, 4>(p, stream);
}

int *csa_quant_status_word(void) {
    void *at = nullptr;
    return cudaGetSymbolAddress(&at, g_quant_status) == cudaSuccess ? static_cast<int *>(at) : nullptr;
}

// Rotary positions with several axes, on queries and keys of any strides, and
// the rows of new tokens written into the pages of a cache.
//
// The first 2n columns of a row are n pairs; pair i of a token at position
// p = positions[axis(i)] turns by the angle p * base^(-i/n):
//     (u, w) -> (u cos - w sin, u sin + w cos),
// and the backward pass is the same turn by the negative angle (a rotation's
// transpose).  Pairs are (i, i + n), or (2i, 2i + 1) when adjacent.
//
// Angles.  Far positions lose an angle formed in fp32 (at 2^20 radians a step
// of fp32 is 1/16), so the angle is formed in turns, in integers: the plan
// holds base^(-i/n) / 2 pi as a 64-bit fraction F of a turn, and p * F modulo
// 2^64 is the angle's fraction of a turn, off by |p| times what F is off by
// (2^-65 turns for its rounding).
//
// What bounds it.  Each element is read once and written once: HBM bandwidth.
// A thread owns 16 bytes twice (the two members of 8 bf16 or 4 fp32 pairs) of
// one token and walks over a range of heads, so that the sines and cosines of
// a token are formed once for those heads.  What hides the latency is threads,
// not loads in flight per thread: queries and keys of 8192 tokens (32 + 8 heads
// of 128, bf16, 168 MB) take 29.5 us, 5.7 TB/s, with 1536 threads per SM and one
// head at a time, 31.3 us with 1280 and 8 heads per block, 36 to 57 us with 2 to
// 4 heads loaded ahead (94 registers); 4 x 2048 tokens of 16 + 16 heads in fp32
// (268 MB) 42.1 us, 6.4 TB/s.  The launch, the ramp and the tail are 4 us of it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "csa.h"
#include "csa_internal.h"
#include "csa_launch.cuh"
#include "csa_rotate.cuh"

namespace {

using namespace csa_dev;

constexpr int kThreads = 128, kBlocks = 12;  // 40 registers a thread: 1536 threads per SM

__device__ int g_rope_status;  // sticky status word of this file's kernels

struct RopeTensor {
    const void *in;
    void *out;
    long long ib, ih, it;  // strides of in over batch, head, time, in elements
    long long ob, oh, ot;
    int H;
};

struct RopeParams {
    csa_rope_plan plan;
    RopeTensor x[3];  // queries, keys, values
    const int *positions;
    long long pa, pb, pt;  // strides over axes, batch, time
    int B, T, d;
    float sign;
    int heads_per_block;
    int blocks[2];  // blocks of heads of the queries, and of the keys
    bool paged;  // keys (x[1]) and values (x[2]) go to pages; else every tensor to its out
    void *k_pages, *v_pages;
    const int *table, *seqlens, *counts;
    int P, S, M;
};

// One block: a range of tokens (rows of B x T) and a range of heads of one
// tensor.  V elements of type T per chunk; a thread's unit of a row is two
// chunks, at columns c0 and c1.  Units [0, n/V) are rotated, the ones behind
// copy the columns from 2n on.
template <typename T, int V, bool ADJ, bool PAGED>
__global__ void __launch_bounds__(kThreads, kBlocks) rope_kernel(const __grid_constant__ RopeParams p) {
    using C = typename Chunk<V * sizeof(T)>::type;
    __shared__ unsigned long long turn[CSA_ROPE_MAX_PAIRS];
    __shared__ unsigned char axis[CSA_ROPE_MAX_PAIRS];
    const int n = p.plan.pairs;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        turn[i] = p.plan.turn[i];
        axis[i] = p.plan.axis[i];
    }
    csa_dev::after_previous();
    __syncthreads();
    const int rest = (p.d - 2 * n) / V;  // chunks that are not rotated
    const int units = n / V + (rest + 1) / 2, rows = kThreads / units;
    const int r = threadIdx.x / units, u = threadIdx.x - r * units;
    const unsigned token = blockIdx.x * rows + r;  // B * T fits 31 bits
    if (r >= rows || token >= (unsigned)p.B * p.T) return;
    const int b = token / (unsigned)p.T, t = token - (unsigned)b * p.T;
    const bool turned = u < n / V;
    int c0, c1;
    bool two = true;
    if (turned) {
        c0 = ADJ ? 2 * V * u : V * u;
        c1 = ADJ ? c0 + V : c0 + n;
    } else {
        c0 = 2 * n + 2 * V * (u - n / V);
        c1 = c0 + V;
        two = c1 < p.d;
    }
    int y = blockIdx.y, which = 0;
    if (y >= p.blocks[0]) {
        y -= p.blocks[0];
        which = 1;
        if (y >= p.blocks[1]) {
            y -= p.blocks[1];
            which = 2;
        }
    }
    const RopeTensor &x = p.x[which];
    const int h0 = y * p.heads_per_block, count = min(p.heads_per_block, x.H - h0);
    const T *in = static_cast<const T *>(x.in) + b * x.ib + h0 * x.ih + t * x.it;
    T *out = static_cast<T *>(x.out);
    long long step = x.oh;
    int cache_row = 0;
    if (PAGED) {
        const int len = p.seqlens[b], held = p.counts ? p.counts[b] : p.T;
        cache_row = len - held + t;
        if (which > 0) {
            if (held < 0 || held > p.T || len < held || len > (long long)p.M * p.S) {
                if (t == 0 && u == 0) atomicCAS(&g_rope_status, 0, CSA_ERR_INVALID_ARG);
                return;
            }
            if (t >= held) return;
            const int page = p.table[(long long)b * p.M + cache_row / p.S];
            if (page < 0 || page >= p.P) {
                if (u == 0) atomicCAS(&g_rope_status, 0, CSA_ERR_INVALID_ARG);
                return;
            }
            out = static_cast<T *>(which == 1 ? p.k_pages : p.v_pages) +
                  (((long long)page * x.H + h0) * p.S + cache_row % p.S) * p.d;
            step = (long long)p.S * p.d;
        }
    }
    if (!PAGED || which == 0) out += b * x.ob + h0 * x.oh + t * x.ot;
    const bool turns = turned && which < 2;
    float cs[V], sn[V];
    if (turns) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = V * u + j;
            const int pos = PAGED && !p.positions ? cache_row
                                                  : p.positions[axis[i] * p.pa + b * p.pb + t * p.pt];
            turn_by((unsigned long long)(long long)pos * turn[i], sn[j], cs[j]);
            sn[j] *= p.sign;
        }
    }
    union Pack {
        C raw;
        T e[V];
    } a, c;
#pragma unroll 1
    for (int h = 0; h < count; ++h) {
        a.raw = *reinterpret_cast<const C *>(in + c0);
        if (two) c.raw = *reinterpret_cast<const C *>(in + c1);
        if (turns) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                // pair j: adjacent, elements 2j and 2j + 1 of the two chunks; else element j of each
                T &eu = !ADJ ? a.e[j] : 2 * j < V ? a.e[(2 * j) % V] : c.e[(2 * j) % V];
                T &ew = !ADJ ? c.e[j] : 2 * j + 1 < V ? a.e[(2 * j + 1) % V] : c.e[(2 * j + 1) % V];
                const float xu = widen(eu), xw = widen(ew);
                eu = narrow<T>(xu * cs[j] - xw * sn[j]);
                ew = narrow<T>(xu * sn[j] + xw * cs[j]);
            }
        }
        *reinterpret_cast<C *>(out + c0) = a.raw;
        if (two) *reinterpret_cast<C *>(out + c1) = c.raw;
        in += x.ih;
        out += step;
    }
}

template <typename T, int V>
int launch(RopeParams &p, cudaStream_t stream) {
    const int n = p.plan.pairs, rest = (p.d - 2 * n) / V;
    const int units = n / V + (rest + 1) / 2, rows = kThreads / units;
    const long long tokens = (long long)p.B * p.T, bx = (tokens + rows - 1) / rows;
    // a token's sines serve the block's heads: 4, fewer where that leaves SMs without work
    auto blocks = [&](int H) { return (H + p.heads_per_block - 1) / p.heads_per_block; };
    auto all = [&] { return blocks(p.x[0].H) + blocks(p.x[1].H) + blocks(p.x[2].H); };
    p.heads_per_block = 4;
    while (p.heads_per_block > 1 && bx * all() < 4 * 152) p.heads_per_block /= 2;
    p.blocks[0] = blocks(p.x[0].H);
    p.blocks[1] = blocks(p.x[1].H);
    const int by = all();
    const dim3 grid((unsigned)bx, (unsigned)by);
    const bool adj = p.plan.adjacent != 0;
    auto kernel = p.paged ? adj ? rope_kernel<T, V, true, true> : rope_kernel<T, V, false, true>
                  : adj   ? rope_kernel<T, V, true, false>
                          : rope_kernel<T, V, false, false>;
    return csa_dev::launch_after_previous(kernel, grid, kThreads, 0, stream, p) == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

bool on16(const void *q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; }

// Whether rows of x can be moved in 16-byte chunks of V elements.
bool wide(const RopeTensor &x, int V, bool has_out) {
    if (x.H == 0) return true;
    return on16(x.in) && x.ib % V == 0 && x.ih % V == 0 && x.it % V == 0 &&
           (!has_out || (on16(x.out) && x.ob % V == 0 && x.oh % V == 0 && x.ot % V == 0));
}

template <typename T>
int run(RopeParams &p, cudaStream_t stream) {
    constexpr int V = 16 / (int)sizeof(T);
    const bool ok = p.d % V == 0 && p.plan.pairs % V == 0 && wide(p.x[0], V, true) &&
                    wide(p.x[1], V, !p.paged) && wide(p.x[2], V, !p.paged) &&
                    (!p.paged || (on16(p.k_pages) && on16(p.v_pages)));
    return ok ? launch<T, V>(p, stream) : launch<T, 1>(p, stream);
}

RopeTensor tensor(const void *in, const long long *is, void *out, const long long *os, int H, int T,
                  int d) {
    RopeTensor x;
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

}  // namespace

int csa_rope_plan_make(csa_rope_plan *plan, const int *sections, int axes, double base, int flags) {
    int left[CSA_ROPE_MAX_AXES], total = 0, most = 0;
    for (int a = 0; a < axes; ++a) {
        left[a] = sections[a];
        if (left[a] < 0 || left[a] > CSA_ROPE_MAX_PAIRS) return CSA_ERR_INVALID_ARG;
        total += left[a];
        if (left[a] > most) most = left[a];
    }
    if (total < 1) return CSA_ERR_INVALID_ARG;
    if (total > CSA_ROPE_MAX_PAIRS) return CSA_ERR_UNSUPPORTED;
    *plan = csa_rope_plan{};
    plan->pairs = total;
    plan->axes = axes;
    plan->adjacent = (flags & CSA_ROPE_ADJACENT) ? 1 : 0;
    int i = 0;
    if (flags & CSA_ROPE_DEALT) {
        for (int turn = 0; turn < most; ++turn)
            for (int a = 0; a < axes; ++a)
                if (turn < left[a]) plan->axis[i++] = (unsigned char)a;
    } else {
        for (int a = 0; a < axes; ++a)
            for (int j = 0; j < left[a]; ++j) plan->axis[i++] = (unsigned char)a;
    }
    // The frequencies in turns per position, base^(-i/n) / 2 pi, as fractions of a turn times 2^64.
    // A power each where a long double has 64 bits: (|ln base| + 4) 2^-64 relative.  Where it has 113
    // a power is computed in software (2 us), so one power and n products: n 2^-111 relative.
    const long double whole = 0.159154943091895335768883763372514362L, step = powl((long double)base, -1.0L / total);
    long double f = whole;
    for (i = 0; i < total; ++i) {
        const long double units = ldexpl(f - floorl(f), 64);
        const unsigned long long down = (unsigned long long)units;
        plan->turn[i] = down + (units - (long double)down >= 0.5L ? 1 : 0);  // to nearest; 2^64 is 0, a whole turn
        f = LDBL_MANT_DIG > 64 ? f * step : whole * powl((long double)base, -(long double)(i + 1) / total);
    }
    return CSA_OK;
}

int csa_rope_run(const csa_rope_plan *plan, const void *q, const long long *q_strides, void *q_out,
                 const long long *q_out_strides, const void *k, const long long *k_strides,
                 void *k_out, const long long *k_out_strides, const int *positions,
                 const long long *pos_strides, int B, int Hq, int Hkv, int T, int d, bool inverse,
                 bool bf16, cudaStream_t stream) {
    RopeParams p = {};
    p.plan = *plan;
    p.x[0] = tensor(q, q_strides, q_out, q_out_strides, Hq, T, d);
    p.x[1] = tensor(k, k_strides, k_out, k_out_strides, Hkv, T, d);
    p.x[2] = tensor(nullptr, nullptr, nullptr, nullptr, 0, T, d);
    p.positions = positions;
    p.pa = pos_strides ? pos_strides[0] : (long long)B * T;
    p.pb = pos_strides ? pos_strides[1] : T;
    p.pt = pos_strides ? pos_strides[2] : 1;
    p.B = B;
    p.T = T;
    p.d = d;
    p.sign = inverse ? -1.0f : 1.0f;
    return bf16 ? run<__nv_bfloat16>(p, stream) : run<float>(p, stream);
}

int csa_cache_append_run(const csa_rope_plan *plan, const void *q, const long long *q_strides,
                         void *q_out, const long long *q_out_strides, const void *k,
                         const long long *k_strides, const void *v, const long long *v_strides,
                         void *k_pages, void *v_pages, const int *block_table, const int *seqlens,
                         const int *counts, const int *positions, const long long *pos_strides,
                         int B, int Hq, int Hkv, int T, int d, int P, int S, int M, bool bf16,
                         cudaStream_t stream) {
    RopeParams p = {};
    if (plan) p.plan = *plan;  // no plan: no pair turns, every column is copied
    p.x[0] = tensor(q, q_strides, q_out, q_out_strides, Hq, T, d);
    p.x[1] = tensor(k, k_strides, nullptr, nullptr, Hkv, T, d);
    p.x[2] = tensor(v, v_strides, nullptr, nullptr, Hkv, T, d);
    p.positions = positions;
    p.pa = pos_strides ? pos_strides[0] : (long long)B * T;
    p.pb = pos_strides ? pos_strides[1] : T;
    p.pt = pos_strides ? pos_strides[2] : 1;
    p.B = B;
    p.T = T;
    p.d = d;
    p.sign = 1.0f;
    p.paged = true;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.table = block_table;
    p.seqlens = seqlens;
    p.counts = counts;
    p.P = P;
    p.S = S;
    p.M = M;
    return bf16 ? run<__nv_bfloat16>(p, stream) : run<float>(p, stream);
}

int *csa_rope_status_word(void) {
    void *at = nullptr;
    return cudaGetSymbolAddress(&at, g_rope_status) == cudaSuccess ? static_cast<int *>(at) : nullptr;
}

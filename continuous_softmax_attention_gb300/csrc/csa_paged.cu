// Decode step of causal continuous softmax attention over a paged cache: for
// every sequence b and query head, the newest token's query against the sink
// and the n_b cached rows of the head's group (eq. (10)/(11) of "Continuous
// Softmax Attention", the single row t = n_b).
//
// Between neighbouring logits a and a' = a + x the interval gives the key at a
// the weight e^{a-m} phi2(x) and the key at a' the weight e^{a'-m} phi2(-x)
// (eq. (9)); with p = e^{a-m} and p' = e^{a'-m} these are ((p'-p)/x - p)/x and
// (p' - (p'-p)/x)/x.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "csa.h"
#include "csa_device.cuh"
#include "csa_internal.h"

namespace {

using namespace csa_dev;

constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ int g_paged_status;  // sticky status word of this file's kernels

struct PagedParams {
    const __nv_bfloat16 *q, *k, *v, *k0, *v0;
    const int *table, *seqlens;
    __nv_bfloat16 *out;
    float *lse;
    int B, Hq, Hkv, P, S, M, d;
    float qscale;  // scale * log2(e): logits come out in log2 units
    int mode;
};

// The weights that the interval between logits a and a1 (log2 units, both at
// most about m) gives its two keys.  |x| < 1 (natural units): the power series
// sum x^j/(j+2)!, j = 0..9, truncated below 3e-9 relative, split into its even
// and odd terms, which the two keys share.
__device__ __forceinline__ void interval(float a, float a1, float m, float &left, float &right) {
    const float x = (a1 - a) * kLn2, p = ex2_approx(a - m), p1 = ex2_approx(a1 - m), y = x * x;
    float even = 2.755731922398589e-07f;             // 1/10!
    even = fmaf(even, y, 2.48015873015873e-05f);     // 1/8!
    even = fmaf(even, y, 1.388888888888889e-03f);    // 1/6!
    even = fmaf(even, y, 4.166666666666667e-02f);    // 1/4!
    even = fmaf(even, y, 0.5f);                      // 1/2!
    float odd = 2.505210838544172e-08f;              // 1/11!
    odd = fmaf(odd, y, 2.755731922398589e-06f);      // 1/9!
    odd = fmaf(odd, y, 1.984126984126984e-04f);      // 1/7!
    odd = fmaf(odd, y, 8.333333333333333e-03f);      // 1/5!
    odd = fmaf(odd, y, 1.666666666666667e-01f);      // 1/3!
    const float r = rcp_approx(x), s = (p1 - p) * r;
    const bool near = fabsf(x) < 1.0f;
    left = near ? p * fmaf(odd, x, even) : (s - p) * r;
    right = near ? p1 * fmaf(-odd, x, even) : (p1 - s) * r;
}

constexpr int kThreads = 128;

// One block per (sequence, query head), the whole sequence in tiles of
// kThreads - 1 rows: a thread forms one row's logit (the last one the logit of
// the row behind the tile), then one weight, then sums columns.
__global__ void __launch_bounds__(kThreads) paged_kernel(const PagedParams p) {
    __shared__ float qs[256], a[kThreads + 1], w[kThreads], red[8];
    __shared__ int pg[kThreads];
    const int b = blockIdx.x / p.Hq, hq = blockIdx.x - b * p.Hq, tid = threadIdx.x;
    const int hk = hq / (p.Hq / p.Hkv), n = p.seqlens[b], d = p.d;
    __nv_bfloat16 *out = p.out + (long long)blockIdx.x * d;
    bool bad = n < 0 || n > (long long)p.M * p.S;
    const int held = bad ? 0 : (int)(((long long)n + p.S - 1) / p.S);
    for (int j = tid; j < held; j += kThreads) {
        const int page = p.table[(long long)b * p.M + j];
        bad |= page < 0 || page >= p.P;
    }
    bad = __syncthreads_or(bad);
    if (bad || n == 0) {
        for (int c = tid; c < d; c += kThreads) out[c] = __float2bfloat16_rn(bad ? NAN : 0.0f);
        if (tid == 0 && p.lse) p.lse[blockIdx.x] = bad ? NAN : -INFINITY;
        if (tid == 0 && bad) atomicCAS(&g_paged_status, 0, CSA_ERR_INVALID_ARG);
        return;
    }
    for (int c = tid; c < d; c += kThreads)
        qs[c] = __bfloat162float(p.q[(long long)blockIdx.x * d + c]) * p.qscale;
    __syncthreads();
    auto row_of = [&](const __nv_bfloat16 *pages, int r) {
        const int page = p.table[(long long)b * p.M + r / p.S];
        return pages + (((long long)page * p.Hkv + hk) * p.S + r % p.S) * d;
    };
    auto dot = [&](const __nv_bfloat16 *row) {
        float s = 0.f;
        for (int c = 0; c < d; ++c) s = fmaf(qs[c], __bfloat162float(row[c]), s);
        return s;
    };
    const __nv_bfloat16 *k0 = p.mode == CSA_K0_GIVEN ? p.k0 + (long long)hk * d : row_of(p.k, 0);
    const __nv_bfloat16 *v0 = p.mode == CSA_K0_GIVEN ? p.v0 + (long long)hk * d : row_of(p.v, 0);
    float prev = p.mode == CSA_K0_ZERO ? 0.f : dot(k0);  // logit of the position before the tile
    float m = prev, l = 0.f, o[2] = {0.f, 0.f};
    constexpr int kTile = kThreads - 1;
    for (int r0 = 0; r0 < n; r0 += kTile) {
        const int have = min(kTile + 1, n - r0), own = min(kTile, n - r0);
        if (tid < have) {
            a[tid + 1] = dot(row_of(p.k, r0 + tid));
            pg[tid] = p.table[(long long)b * p.M + (r0 + tid) / p.S];
        }
        if (tid == 0) a[0] = prev;
        float mx = tid < have ? a[tid + 1] : -INFINITY;
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, off));
        if ((tid & 31) == 0) red[tid >> 5] = mx;
        __syncthreads();
        const float m1 = fmaxf(fmaxf(fmaxf(m, red[0]), fmaxf(red[1], red[2])), red[3]);
        const float f = ex2_approx(m - m1);
        m = m1;
        l *= f;
        o[0] *= f;
        o[1] *= f;
        float left = 0.f, right = 0.f, from_left = 0.f, sink = 0.f;
        if (tid < own) {
            interval(a[tid], a[tid + 1], m, sink, from_left);
            if (tid + 1 < have) interval(a[tid + 1], a[tid + 2], m, left, right);
            w[tid] = from_left + left;
        }
        if (tid == 0 && r0 == 0) red[4] = sink;
        __syncthreads();
        if (r0 == 0) {
            l += red[4];
            if (p.mode != CSA_K0_ZERO)
                for (int i = 0; i < 2; ++i)
                    if (tid + i * kThreads < d) o[i] = red[4] * __bfloat162float(v0[tid + i * kThreads]);
        }
        for (int r = 0; r < own; ++r) {
            l += w[r];
            const __nv_bfloat16 *row =
                p.v + (((long long)pg[r] * p.Hkv + hk) * p.S + (r0 + r) % p.S) * d;
            for (int i = 0; i < 2; ++i)
                if (tid + i * kThreads < d) o[i] = fmaf(w[r], __bfloat162float(row[tid + i * kThreads]), o[i]);
        }
        prev = a[own];
        __syncthreads();
    }
    for (int i = 0; i < 2; ++i)
        if (tid + i * kThreads < d) out[tid + i * kThreads] = __float2bfloat16_rn(o[i] / l);
    if (tid == 0 && p.lse) p.lse[blockIdx.x] = (m + log2f(l)) * kLn2;
}

}  // namespace

long long csa_decode_paged_scratch_bytes(int B, int Hq, int Hkv, int d) {
    if (B < 0 || Hq < 0 || Hkv < 0 || !(d == 64 || d == 128 || d == 256)) return -1;
    return 16;
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
    p.d = d;
    p.qscale = scale * kLog2e;
    p.mode = mode;
    paged_kernel<<<(unsigned)(B * Hq), kThreads, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

int csa_paged_take_status(void) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_paged_status, sizeof(int)) != cudaSuccess) return CSA_ERR_CUDA;
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_paged_status, &zero, sizeof(int)) != cudaSuccess) return CSA_ERR_CUDA;
    return v;
}

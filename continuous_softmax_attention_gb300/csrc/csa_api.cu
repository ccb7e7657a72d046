// C ABI of libcsa.so (declared in include/csa.h): argument validation and
// dispatch to the CUDA-core and tensor-core kernels.  No allocation, no
// host synchronisation on the compute entry points.
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <mutex>

#include "csa.h"
#include "csa_internal.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Common checks of the attention entry points.  Returns CSA_OK, or the
// error code; *empty is set when there is nothing to compute.
int check_common(const void *q, const void *k, const void *v, const void *k0, const void *v0,
                 const void *out, int B, int H, int T, int d, float scale, int mode, bool use_sink,
                 bool *empty) {
    *empty = false;
    if (B < 0 || H < 0 || T < 0 || d < 1) return CSA_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return CSA_ERR_INVALID_ARG;
    if (use_sink && (mode < CSA_K0_ZERO || mode > CSA_K0_GIVEN)) return CSA_ERR_INVALID_ARG;
    if ((long long)B * H * T == 0) {
        *empty = true;
        return CSA_OK;
    }
    if (!q || !k || !v || !out) return CSA_ERR_INVALID_ARG;
    if (use_sink && mode == CSA_K0_GIVEN && (!k0 || !v0)) return CSA_ERR_INVALID_ARG;
    if ((long long)B * H > 0x7fffffffLL || (long long)B * H * T > (1LL << 40))
        return CSA_ERR_UNSUPPORTED;
    return CSA_OK;
}

int device_ok() {
    static std::atomic<unsigned long long> good{0};  // devices 0..63 found usable: what they are does not change
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return CSA_ERR_NO_DEVICE;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (good.load(std::memory_order_relaxed) & bit) return CSA_OK;
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
        return CSA_ERR_NO_DEVICE;
    // The binary carries sm_103a code only.
    if (major != 10 || minor != 3) return CSA_ERR_NO_DEVICE;
    good.fetch_or(bit, std::memory_order_relaxed);
    return CSA_OK;
}

// The status words of the paged cache's and rotary kernels, of which each translation unit has one, taken by one launch and
// one copy: csa_device_status takes 73 us, 187 with two copies for each of the words.
constexpr int kWords = 10;
struct Words {
    int *at[kWords];
};
__device__ int g_taken;
__global__ void take_kernel(Words w) {
    int first = CSA_OK;
    for (int i = 0; i < kWords; ++i) {
        const int word = atomicExch(w.at[i], CSA_OK);
        if (first == CSA_OK) first = word;
    }
    g_taken = first;
}
int take_words() {
    static std::mutex one_at_a_time;  // g_taken is a call's from its launch to its copy
    Words w = {{csa_paged_status_word(), csa_rope_status_word(), csa_cache_status_word(), csa_quant_status_word(),
                csa_paged_e4m3_status_word(), csa_paged_int8_status_word(), csa_tree_status_word(),
                csa_rows_bf16_status_word(), csa_rows_e4m3_status_word(), csa_rows_int8_status_word()}};
    for (const int *at : w.at)
        if (!at) return CSA_ERR_CUDA;
    const std::lock_guard<std::mutex> held(one_at_a_time);
    void *args[] = {&w};
    if (cudaLaunchKernel((const void *)take_kernel, dim3(1), dim3(1), args, 0, nullptr) != cudaSuccess) {
        (void)cudaGetLastError();  // and taken, or the next launch would report it too
        return CSA_ERR_CUDA;
    }
    int v = 0;
    return cudaMemcpyFromSymbol(&v, g_taken, sizeof(int)) == cudaSuccess ? v : CSA_ERR_CUDA;
}

int from_cuda(cudaError_t e) { return e == cudaSuccess ? CSA_OK : CSA_ERR_CUDA; }

int forward_bf16(const void *q, const void *k, const void *v, const void *k0, const void *v0,
                 void *out, float *lse, int B, int H, int T, int d, float scale, int mode,
                 int form, csa_stream_t stream) {
    const bool continuous = form != kFormStd;
    bool empty;
    int rc = check_common(q, k, v, k0, v0, out, B, H, T, d, scale, mode, continuous, &empty);
    if (rc != CSA_OK || empty) return rc;
    if (d > 256) return CSA_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
        (lse && !aligned(lse, 4)))
        return CSA_ERR_ALIGNMENT;
    if (continuous && mode == CSA_K0_GIVEN && (!aligned(k0, 2) || !aligned(v0, 2)))
        return CSA_ERR_ALIGNMENT;
    if ((rc = device_ok()) != CSA_OK) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (d == 64 || d == 128) {
        if (continuous)
            return csa_tc_forward(q, k, v, k0, v0, out, lse, B, H, T, d, scale, mode, form, s);
        return csa_tc_std_forward(q, k, v, out, lse, B, H, T, d, scale, s);
    }
    // the CUDA-core kernel forms b in the log domain in its exact form
    return from_cuda(csa_simt_forward_bf16(q, k, v, k0, v0, out, lse, B, H, T, d, scale, mode,
                                           form == kFormLogDomain ? kFormExact : form, s));
}

int forward_f32(const float *q, const float *k, const float *v, const float *k0, const float *v0,
                float *out, float *lse, int B, int H, int T, int d, float scale, int mode,
                int form, csa_stream_t stream) {
    const bool continuous = form != kFormStd;
    bool empty;
    int rc = check_common(q, k, v, k0, v0, out, B, H, T, d, scale, mode, continuous, &empty);
    if (rc != CSA_OK || empty) return rc;
    if (d > 256) return CSA_ERR_UNSUPPORTED;
    if (!aligned(q, 4) || !aligned(k, 4) || !aligned(v, 4) || !aligned(out, 4) ||
        (lse && !aligned(lse, 4)))
        return CSA_ERR_ALIGNMENT;
    if ((rc = device_ok()) != CSA_OK) return rc;
    return from_cuda(csa_simt_forward_f32(q, k, v, k0, v0, out, lse, B, H, T, d, scale, mode,
                                          form, reinterpret_cast<cudaStream_t>(stream)));
}

// The checks of the decode step's arguments other than its workspace, in
// csa_decode's order.  Returns CSA_OK, or the error code; *empty is set when
// there is nothing to compute (B*H == 0).  On CSA_OK, *need holds the scratch
// bytes the sizes take.
int decode_check(const void *q, const void *k_cache, const void *v_cache, const void *k0,
                 const void *v0, const int *seqlens, const void *out, const float *lse, int B,
                 int H, int T, int d, float scale, int mode, bool *empty, long long *need) {
    *empty = false;
    if (B < 0 || H < 0 || T < 0 || d < 1) return CSA_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return CSA_ERR_INVALID_ARG;
    if (mode < CSA_K0_ZERO || mode > CSA_K0_GIVEN) return CSA_ERR_INVALID_ARG;
    if (!(d == 64 || d == 128 || d == 256)) return CSA_ERR_UNSUPPORTED;
    if ((long long)B * H == 0) {
        *empty = true;
        return CSA_OK;
    }
    if (T == 0) return CSA_ERR_INVALID_ARG;  // the newest token's own key is in the cache
    if (T == INT_MAX) return CSA_ERR_UNSUPPORTED;  // positions 0..T must fit an int
    if (!q || !k_cache || !v_cache || !out) return CSA_ERR_INVALID_ARG;
    if (mode == CSA_K0_GIVEN && (!k0 || !v0)) return CSA_ERR_INVALID_ARG;
    if ((long long)B * H * T > (1LL << 40)) return CSA_ERR_UNSUPPORTED;
    *need = csa_decode_scratch_bytes(B, H, T, d);
    if (*need < 0) return CSA_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        (lse && !aligned(lse, 4)) || (seqlens && !aligned(seqlens, 4)))
        return CSA_ERR_ALIGNMENT;
    if (mode == CSA_K0_GIVEN && (!aligned(k0, 16) || !aligned(v0, 16))) return CSA_ERR_ALIGNMENT;
    return CSA_OK;
}

int decode_bf16(const void *q, const void *k_cache, const void *v_cache, const void *k0,
                const void *v0, const int *seqlens, void *out, float *lse, void *workspace,
                long long workspace_bytes, int B, int H, int T, int d, float scale, int mode,
                csa_stream_t stream) {
    bool empty;
    long long need = 0;
    int rc = decode_check(q, k_cache, v_cache, k0, v0, seqlens, out, lse, B, H, T, d, scale, mode,
                          &empty, &need);
    if (rc != CSA_OK || empty) return rc;
    if (!workspace || workspace_bytes < need) return CSA_ERR_INVALID_ARG;
    if (!aligned(workspace, 16)) return CSA_ERR_ALIGNMENT;
    if ((rc = device_ok()) != CSA_OK) return rc;
    return csa_decode_run(q, k_cache, v_cache, k0, v0, seqlens, out, lse, workspace, B, H, T, d,
                          scale, mode, reinterpret_cast<cudaStream_t>(stream));
}

int decode_range_bf16(const void *q, const void *k_shard, const void *v_shard, const void *k0,
                      const void *v0, const int *seqlens, float *out, float *lse,
                      void *workspace, long long workspace_bytes, int B, int H, int T, int d,
                      float scale, int mode, int pos_lo, int pos_hi, csa_stream_t stream) {
    if (B < 0 || H < 0 || T < 0 || d < 1) return CSA_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return CSA_ERR_INVALID_ARG;
    if (mode < CSA_K0_ZERO || mode > CSA_K0_GIVEN) return CSA_ERR_INVALID_ARG;
    if (!(d == 64 || d == 128 || d == 256)) return CSA_ERR_UNSUPPORTED;
    // positions 0..T exist; a range may not start right after the sink
    if (pos_lo < 0 || pos_lo == 1 || pos_hi <= pos_lo || (long long)pos_hi > (long long)T + 1)
        return CSA_ERR_INVALID_ARG;
    if ((long long)B * H == 0) return CSA_OK;
    if (T == 0) return CSA_ERR_INVALID_ARG;
    if (!q || !k_shard || !v_shard || !out || !lse || !workspace) return CSA_ERR_INVALID_ARG;
    if (mode == CSA_K0_GIVEN && (!k0 || !v0)) return CSA_ERR_INVALID_ARG;
    if ((long long)B * H * T > (1LL << 40)) return CSA_ERR_UNSUPPORTED;
    const long long need = csa_decode_range_scratch_bytes(B, H, pos_lo, pos_hi, d);
    if (need < 0) return CSA_ERR_UNSUPPORTED;
    if (workspace_bytes < need) return CSA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_shard, 16) || !aligned(v_shard, 16) || !aligned(out, 16) ||
        !aligned(workspace, 16) || !aligned(lse, 4) || (seqlens && !aligned(seqlens, 4)))
        return CSA_ERR_ALIGNMENT;
    if (mode == CSA_K0_GIVEN && (!aligned(k0, 16) || !aligned(v0, 16))) return CSA_ERR_ALIGNMENT;
    int rc = device_ok();
    if (rc != CSA_OK) return rc;
    return csa_decode_range_run(q, k_shard, v_shard, k0, v0, seqlens, out, lse, workspace, B, H, T,
                                d, scale, mode, pos_lo, pos_hi,
                                reinterpret_cast<cudaStream_t>(stream));
}

long long backward_scratch_bytes(int B, int H, int T, int d) {
    if (B < 0 || H < 0 || T < 0 || d < 1 || d > 256) return -1;
    const long long a = csa_simt_backward_scratch_bytes(B, H, T, d);
    const long long b = csa_tc_backward_scratch_bytes(B, H, T, d);
    return a > b ? a : b;
}

int backward_any(const void *q, const void *k, const void *v, const void *k0, const void *v0,
                 const void *out, const float *lse, const void *dout, void *dq, void *dk,
                 void *dv, float *dk0, float *dv0, void *workspace, long long workspace_bytes,
                 int B, int H, int T, int d, float scale, int mode, bool bf16,
                 csa_stream_t stream) {
    bool empty;
    int rc = check_common(q, k, v, k0, v0, out, B, H, T, d, scale, mode, true, &empty);
    if (rc != CSA_OK) return rc;
    if (empty) {
        // nothing to differentiate; the sink gradients are zero
        if (mode == CSA_K0_GIVEN && (long long)H * d > 0) {
            if (!dk0 || !dv0) return CSA_ERR_INVALID_ARG;
            if ((rc = device_ok()) != CSA_OK) return rc;
            cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
            if (cudaMemsetAsync(dk0, 0, sizeof(float) * (size_t)H * d, s) != cudaSuccess ||
                cudaMemsetAsync(dv0, 0, sizeof(float) * (size_t)H * d, s) != cudaSuccess)
                return CSA_ERR_CUDA;
        }
        return CSA_OK;
    }
    if (!lse || !dout || !dq || !dk || !dv || !workspace) return CSA_ERR_INVALID_ARG;
    if (mode == CSA_K0_GIVEN && (!dk0 || !dv0)) return CSA_ERR_INVALID_ARG;
    if (d > 256) return CSA_ERR_UNSUPPORTED;
    const long long need = backward_scratch_bytes(B, H, T, d);
    if (need < 0) return CSA_ERR_UNSUPPORTED;
    if (workspace_bytes < need) return CSA_ERR_INVALID_ARG;
    const uintptr_t al = bf16 ? 2 : 4;
    if (!aligned(q, al) || !aligned(k, al) || !aligned(v, al) || !aligned(out, al) ||
        !aligned(dout, al) || !aligned(dq, al) || !aligned(dk, al) || !aligned(dv, al) ||
        !aligned(lse, 4) || !aligned(workspace, 16) ||
        (mode == CSA_K0_GIVEN && (!aligned(k0, al) || !aligned(v0, al) || !aligned(dk0, 4) ||
                                  !aligned(dv0, 4))))
        return CSA_ERR_ALIGNMENT;
    if ((rc = device_ok()) != CSA_OK) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool tc_aligned = aligned(q, 16) && aligned(k, 16) && aligned(v, 16) &&
                            aligned(out, 16) && aligned(dout, 16) && aligned(dq, 16) &&
                            aligned(dk, 16) && aligned(dv, 16) &&
                            (mode != CSA_K0_GIVEN || (aligned(k0, 16) && aligned(v0, 16)));
    if (bf16 && (d == 64 || d == 128) && tc_aligned)
        return csa_tc_backward(q, k, v, k0, v0, out, lse, dout, dq, dk, dv, dk0, dv0, workspace,
                               B, H, T, d, scale, mode, s);
    if (bf16)
        return from_cuda(csa_simt_backward_bf16(q, k, v, k0, v0, out, lse, dout, dq, dk, dv, dk0,
                                                dv0, workspace, B, H, T, d, scale, mode, s));
    return from_cuda(csa_simt_backward_f32(
        static_cast<const float *>(q), static_cast<const float *>(k),
        static_cast<const float *>(v), static_cast<const float *>(k0),
        static_cast<const float *>(v0), static_cast<const float *>(out), lse,
        static_cast<const float *>(dout), static_cast<float *>(dq), static_cast<float *>(dk),
        static_cast<float *>(dv), dk0, dv0, workspace, B, H, T, d, scale, mode, s));
}

// ------------------------------------------------------ paged cache and rope
constexpr long long kIntMax = 0x7fffffffLL;

// Sizes of a paged cache's tables.
int check_tables(int B, int P, int S, int M) {
    if (B < 0 || P < 0 || S < 1 || M < 1) return CSA_ERR_INVALID_ARG;
    // rows are counted in ints, rounded up to tiles of 16
    if ((long long)B * M > kIntMax || (long long)M * S > kIntMax - 15) return CSA_ERR_UNSUPPORTED;
    return CSA_OK;
}

int check_books(const int *refs, const int *table, const int *seqlens, int B, int P, int S, int M) {
    int rc = check_tables(B, P, S, M);
    if (rc != CSA_OK) return rc;
    if ((!refs && P > 0) || ((!table || !seqlens) && B > 0)) return CSA_ERR_INVALID_ARG;
    if (!aligned(refs, 4) || !aligned(table, 4) || !aligned(seqlens, 4)) return CSA_ERR_ALIGNMENT;
    return CSA_OK;
}

// A plan that csa_rope_plan_init can have made: the kernels index by its fields.
bool sound_plan(const csa_rope_plan *plan) {
    if (plan->pairs < 1 || plan->pairs > CSA_ROPE_MAX_PAIRS || plan->axes < 1 ||
        plan->axes > CSA_ROPE_MAX_AXES)
        return false;
    for (int i = 0; i < plan->pairs; ++i)
        if (plan->axis[i] >= plan->axes) return false;
    return true;
}

int rope_any(const csa_rope_plan *plan, const void *q, const long long *q_strides, void *q_out,
             const long long *q_out_strides, const void *k, const long long *k_strides,
             void *k_out, const long long *k_out_strides, const int *positions,
             const long long *pos_strides, int B, int Hq, int Hkv, int T, int d, int inverse,
             bool bf16, csa_stream_t stream) {
    if (!plan || !sound_plan(plan)) return CSA_ERR_INVALID_ARG;
    if (B < 0 || Hq < 0 || Hkv < 0 || T < 0 || d < 1 || 2 * plan->pairs > d) return CSA_ERR_INVALID_ARG;
    if (d > 256 || (long long)B * T > kIntMax || (long long)Hq + Hkv > 65535) return CSA_ERR_UNSUPPORTED;
    if ((long long)B * T == 0 || (long long)Hq + Hkv == 0) return CSA_OK;
    if ((Hq > 0 && (!q || !q_out)) || (Hkv > 0 && (!k || !k_out)) || !positions)
        return CSA_ERR_INVALID_ARG;
    const uintptr_t al = bf16 ? 2 : 4;
    if (!aligned(q, al) || !aligned(q_out, al) || !aligned(k, al) || !aligned(k_out, al) ||
        !aligned(positions, 4))
        return CSA_ERR_ALIGNMENT;
    int rc = device_ok();
    if (rc != CSA_OK) return rc;
    return csa_rope_run(plan, q, q_strides, q_out, q_out_strides, k, k_strides, k_out,
                        k_out_strides, positions, pos_strides, B, Hq, Hkv, T, d, inverse != 0, bf16,
                        reinterpret_cast<cudaStream_t>(stream));
}

// What every append checks; the tensors' elements have `in` bytes, the pools' `held`.
int append_check(const csa_rope_plan *plan, const void *q, const void *q_out, const void *k, const void *v,
                 const void *k_pages, const void *v_pages, const int *block_table, const int *seqlens,
                 const int *counts, const int *positions, int B, int Hq, int Hkv, int T, int d, int P, int S, int M,
                 uintptr_t in, uintptr_t held, bool *empty) {
    *empty = false;
    if (plan && !sound_plan(plan)) return CSA_ERR_INVALID_ARG;
    if (B < 0 || Hq < 0 || Hkv < 1 || T < 0 || d < 1) return CSA_ERR_INVALID_ARG;
    if (plan ? 2 * plan->pairs > d : Hq > 0) return CSA_ERR_INVALID_ARG;
    int rc = check_tables(B, P, S, M);
    if (rc != CSA_OK) return rc;
    if (d > 256 || (long long)B * T > kIntMax || (long long)Hq + 2LL * Hkv > 65535)
        return CSA_ERR_UNSUPPORTED;
    *empty = (long long)B * T == 0;
    if (*empty) return CSA_OK;
    if (!k || !v || (P > 0 && (!k_pages || !v_pages)) || !block_table || !seqlens || (Hq > 0 && (!q || !q_out)))
        return CSA_ERR_INVALID_ARG;
    if (!aligned(q, in) || !aligned(q_out, in) || !aligned(k, in) || !aligned(v, in) ||
        !aligned(k_pages, held) || !aligned(v_pages, held) || !aligned(block_table, 4) ||
        !aligned(seqlens, 4) || !aligned(counts, 4) || !aligned(positions, 4))
        return CSA_ERR_ALIGNMENT;
    return CSA_OK;
}

int append_any(const csa_rope_plan *plan, const void *q, const long long *q_strides, void *q_out,
               const long long *q_out_strides, const void *k, const long long *k_strides,
               const void *v, const long long *v_strides, void *k_pages, void *v_pages,
               const int *block_table, const int *seqlens, const int *counts, const int *positions,
               const long long *pos_strides, int B, int Hq, int Hkv, int T, int d, int P, int S,
               int M, bool bf16, csa_stream_t stream) {
    const uintptr_t al = bf16 ? 2 : 4;
    bool empty;
    int rc = append_check(plan, q, q_out, k, v, k_pages, v_pages, block_table, seqlens, counts, positions, B, Hq, Hkv, T,
                          d, P, S, M, al, al, &empty);
    if (rc != CSA_OK || empty) return rc;
    if ((rc = device_ok()) != CSA_OK) return rc;
    return csa_cache_append_run(plan, q, q_strides, q_out, q_out_strides, k, k_strides, v, v_strides,
                                k_pages, v_pages, block_table, seqlens, counts, positions,
                                pos_strides, B, Hq, Hkv, T, d, P, S, M, bf16,
                                reinterpret_cast<cudaStream_t>(stream));
}

bool eight_bits(int kind) { return kind == CSA_E4M3 || kind == CSA_INT8; }

// The decode step's arguments; T >= 0: those of its form for T drafted tokens.
int paged_check(const csa_paged_args &a, const void *workspace, long long workspace_bytes, int d, int kind, int T,
                bool *empty) {
    *empty = false;
    if (a.Hq < 0 || a.Hkv < 1 || a.Hq % a.Hkv != 0 || d < 1) return CSA_ERR_INVALID_ARG;
    if (!std::isfinite(a.scale)) return CSA_ERR_INVALID_ARG;
    if (a.mode < CSA_K0_ZERO || a.mode > CSA_K0_GIVEN) return CSA_ERR_INVALID_ARG;
    int rc = check_tables(a.B, a.P, a.S, a.M);
    if (rc != CSA_OK) return rc;
    if (!(d == 64 || d == 128 || d == 256) || a.S % 8 != 0) return CSA_ERR_UNSUPPORTED;
    // tiles of 32 rows of 8 bits, and for drafted tokens of 128 rows and their neighbours
    if (eight_bits(kind) && (long long)a.M * a.S > kIntMax - 31) return CSA_ERR_UNSUPPORTED;
    if (T >= 0 && (long long)a.M * a.S > kIntMax - 255) return CSA_ERR_UNSUPPORTED;
    if ((long double)a.P * a.Hkv * a.S > kIntMax) return CSA_ERR_UNSUPPORTED;
    if ((long double)a.B * a.Hq * (T > 0 ? T : 1) > kIntMax) return CSA_ERR_UNSUPPORTED;
    *empty = (long long)a.B * a.Hq == 0 || T == 0;
    if (*empty) return CSA_OK;
    if (!a.q || (a.P > 0 && (!a.k_pages || !a.v_pages)) || !a.block_table || !a.seqlens || !a.out) return CSA_ERR_INVALID_ARG;
    if (eight_bits(kind) && a.P > 0 && !a.row_scales) return CSA_ERR_INVALID_ARG;
    if (a.mode == CSA_K0_GIVEN && (!a.k0 || !a.v0)) return CSA_ERR_INVALID_ARG;
    const long long need = T > 0 ? csa_decode_tree_scratch_bytes(a.B, a.Hq, a.Hkv, T, d)
                                 : csa_decode_paged_scratch_bytes(a.B, a.Hq, a.Hkv, d);
    if (need < 0) return CSA_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < need) return CSA_ERR_INVALID_ARG;
    if (!aligned(a.q, 16) || !aligned(a.k_pages, 16) || !aligned(a.v_pages, 16) || !aligned(a.out, 16) ||
        !aligned(workspace, 16) || !aligned(a.lse, 4) || !aligned(a.seqlens, 4) || !aligned(a.block_table, 4) ||
        !aligned(a.row_scales, 16))
        return CSA_ERR_ALIGNMENT;
    if (a.mode == CSA_K0_GIVEN && (!aligned(a.k0, 16) || !aligned(a.v0, 16))) return CSA_ERR_ALIGNMENT;
    return device_ok();
}

}  // namespace

extern "C" {

long long csa_decode_paged_workspace_bytes(int B, int Hq, int Hkv, int d) {
    if (B < 0 || Hq < 0 || Hkv < 1 || Hq % Hkv != 0) return -1;
    return csa_decode_paged_scratch_bytes(B, Hq, Hkv, d);
}

int csa_decode_paged(const void *q, const void *k_pages, const void *v_pages, const void *k0,
                     const void *v0, const int *block_table, const int *seqlens, void *out,
                     float *lse, void *workspace, long long workspace_bytes, int B, int Hq,
                     int Hkv, int P, int S, int M, int d, float scale, int k0_mode,
                     csa_stream_t stream) {
    const csa_paged_args a = {q, k_pages, v_pages, nullptr, k0, v0, block_table, seqlens, out, lse, B, Hq, Hkv, P, S, M,
                              scale, k0_mode};
    bool empty;
    int rc = paged_check(a, workspace, workspace_bytes, d, CSA_BF16, -1, &empty);
    if (rc != CSA_OK || empty) return rc;
    return csa_decode_paged_run(a, workspace, d, reinterpret_cast<cudaStream_t>(stream));
}

int csa_decode_paged_q8(const void *q, const void *k_pages, const void *v_pages, const float *row_scales,
                        const void *k0, const void *v0, const int *block_table, const int *seqlens, void *out,
                        float *lse, void *workspace, long long workspace_bytes, int B, int Hq, int Hkv, int P,
                        int S, int M, int d, float scale, int k0_mode, int kind, csa_stream_t stream) {
    if (!eight_bits(kind)) return CSA_ERR_INVALID_ARG;
    const csa_paged_args a = {q, k_pages, v_pages, row_scales, k0, v0, block_table, seqlens, out, lse, B, Hq, Hkv, P, S,
                              M, scale, k0_mode};
    bool empty;
    int rc = paged_check(a, workspace, workspace_bytes, d, kind, -1, &empty);
    if (rc != CSA_OK || empty) return rc;
    return (kind == CSA_E4M3 ? csa_decode_paged_e4m3_run : csa_decode_paged_int8_run)(
        a, workspace, d, reinterpret_cast<cudaStream_t>(stream));
}

long long csa_decode_tree_workspace_bytes(int B, int Hq, int Hkv, int T, int d) {
    if (B < 0 || Hq < 0 || Hkv < 1 || Hq % Hkv != 0 || T < 0 || T > CSA_TREE_MAX) return -1;
    if (!(d == 64 || d == 128 || d == 256) || (long double)B * Hq * (T > 0 ? T : 1) > kIntMax) return -1;
    return (long long)B * Hq * T == 0 ? 0 : csa_decode_tree_scratch_bytes(B, Hq, Hkv, T, d);
}

int csa_decode_tree(const void *q, const void *k_pages, const void *v_pages, const float *row_scales, const void *k0,
                    const void *v0, const int *block_table, const int *seqlens, const int *parents, const int *counts,
                    void *out, float *lse, void *workspace, long long workspace_bytes, int B, int Hq, int Hkv, int T,
                    int P, int S, int M, int d, float scale, int k0_mode, int kind, csa_stream_t stream) {
    if (T < 0 || (kind != CSA_BF16 && !eight_bits(kind))) return CSA_ERR_INVALID_ARG;
    if (T > CSA_TREE_MAX) return CSA_ERR_UNSUPPORTED;
    if (kind == CSA_BF16 && row_scales) return CSA_ERR_INVALID_ARG;
    const csa_paged_args a = {q, k_pages, v_pages, row_scales, k0, v0, block_table, seqlens, out, lse, B, Hq, Hkv, P, S,
                              M, scale, k0_mode};
    bool empty;
    int rc = paged_check(a, workspace, workspace_bytes, d, kind, T, &empty);
    if (empty || (rc != CSA_OK && rc != CSA_ERR_NO_DEVICE)) return rc;
    if (!aligned(parents, 4) || !aligned(counts, 4)) return CSA_ERR_ALIGNMENT;
    if (rc != CSA_OK) return rc;
    return csa_decode_tree_run(a, parents, counts, T, d, kind, workspace, reinterpret_cast<cudaStream_t>(stream));
}

int csa_rope_plan_init(csa_rope_plan *plan, const int *sections, int axes, double base, int flags) {
    if (!plan || !sections || axes < 1 || axes > CSA_ROPE_MAX_AXES) return CSA_ERR_INVALID_ARG;
    if (!std::isfinite(base) || base <= 0.0 || (flags & ~(CSA_ROPE_ADJACENT | CSA_ROPE_DEALT)))
        return CSA_ERR_INVALID_ARG;
    return csa_rope_plan_make(plan, sections, axes, base, flags);
}

int csa_rope(const csa_rope_plan *plan, const void *q, const long long *q_strides, void *q_out,
             const long long *q_out_strides, const void *k, const long long *k_strides,
             void *k_out, const long long *k_out_strides, const int *positions,
             const long long *pos_strides, int B, int Hq, int Hkv, int T, int d, int inverse,
             csa_stream_t stream) {
    return rope_any(plan, q, q_strides, q_out, q_out_strides, k, k_strides, k_out, k_out_strides,
                    positions, pos_strides, B, Hq, Hkv, T, d, inverse, true, stream);
}

int csa_rope_f32(const csa_rope_plan *plan, const float *q, const long long *q_strides,
                 float *q_out, const long long *q_out_strides, const float *k,
                 const long long *k_strides, float *k_out, const long long *k_out_strides,
                 const int *positions, const long long *pos_strides, int B, int Hq, int Hkv, int T,
                 int d, int inverse, csa_stream_t stream) {
    return rope_any(plan, q, q_strides, q_out, q_out_strides, k, k_strides, k_out, k_out_strides,
                    positions, pos_strides, B, Hq, Hkv, T, d, inverse, false, stream);
}

int csa_cache_append(const csa_rope_plan *plan, const void *q, const long long *q_strides,
                     void *q_out, const long long *q_out_strides, const void *k,
                     const long long *k_strides, const void *v, const long long *v_strides,
                     void *k_pages, void *v_pages, const int *block_table, const int *seqlens,
                     const int *counts, const int *positions, const long long *pos_strides, int B,
                     int Hq, int Hkv, int T, int d, int P, int S, int M, csa_stream_t stream) {
    return append_any(plan, q, q_strides, q_out, q_out_strides, k, k_strides, v, v_strides, k_pages,
                      v_pages, block_table, seqlens, counts, positions, pos_strides, B, Hq, Hkv, T,
                      d, P, S, M, true, stream);
}

int csa_cache_append_f32(const csa_rope_plan *plan, const float *q, const long long *q_strides,
                         float *q_out, const long long *q_out_strides, const float *k,
                         const long long *k_strides, const float *v, const long long *v_strides,
                         float *k_pages, float *v_pages, const int *block_table,
                         const int *seqlens, const int *counts, const int *positions,
                         const long long *pos_strides, int B, int Hq, int Hkv, int T, int d, int P,
                         int S, int M, csa_stream_t stream) {
    return append_any(plan, q, q_strides, q_out, q_out_strides, k, k_strides, v, v_strides, k_pages,
                      v_pages, block_table, seqlens, counts, positions, pos_strides, B, Hq, Hkv, T,
                      d, P, S, M, false, stream);
}

int csa_cache_append_q8(const csa_rope_plan *plan, const void *q, const long long *q_strides,
                        void *q_out, const long long *q_out_strides, const void *k,
                        const long long *k_strides, const void *v, const long long *v_strides,
                        void *k_pages, void *v_pages, float *row_scales, const int *block_table,
                        const int *seqlens, const int *counts, const int *positions,
                        const long long *pos_strides, int B, int Hq, int Hkv, int T, int d, int P,
                        int S, int M, int in_type, int kind, csa_stream_t stream) {
    if ((in_type != CSA_BF16 && in_type != CSA_F32) || !eight_bits(kind)) return CSA_ERR_INVALID_ARG;
    bool empty;
    int rc = append_check(plan, q, q_out, k, v, k_pages, v_pages, block_table, seqlens, counts, positions, B, Hq, Hkv, T,
                          d, P, S, M, in_type == CSA_BF16 ? 2 : 4, 1, &empty);
    if (rc != CSA_OK || empty) return rc;
    if (P > 0 && !row_scales) return CSA_ERR_INVALID_ARG;
    if (!aligned(row_scales, 8)) return CSA_ERR_ALIGNMENT;
    if ((rc = device_ok()) != CSA_OK) return rc;
    return csa_cache_append_q8_run(plan, q, q_strides, q_out, q_out_strides, k, k_strides, v, v_strides,
                                   k_pages, v_pages, row_scales, block_table, seqlens, counts, positions,
                                   pos_strides, B, Hq, Hkv, T, d, P, S, M, in_type == CSA_BF16,
                                   kind == CSA_E4M3, reinterpret_cast<cudaStream_t>(stream));
}

int csa_cache_read(const void *k_pages, const void *v_pages, const float *row_scales,
                   const int *block_table, const int *seqlens, const int *starts, void *k,
                   const long long *k_strides, void *v, const long long *v_strides, int B, int Hkv,
                   int T, int d, int P, int S, int M, int kind, int out_type, csa_stream_t stream) {
    if (kind < CSA_BF16 || kind > CSA_INT8 || (out_type != CSA_BF16 && out_type != CSA_F32)) return CSA_ERR_INVALID_ARG;
    if (!eight_bits(kind) && out_type != kind) return CSA_ERR_INVALID_ARG;
    if (B < 0 || Hkv < 1 || T < 0 || d < 1) return CSA_ERR_INVALID_ARG;
    int rc = check_tables(B, P, S, M);
    if (rc != CSA_OK) return rc;
    if (d > 256 || (long double)B * Hkv * T > kIntMax) return CSA_ERR_UNSUPPORTED;
    if ((long long)B * T == 0) return CSA_OK;
    if (!k || !v || (P > 0 && (!k_pages || !v_pages)) || !block_table || !seqlens) return CSA_ERR_INVALID_ARG;
    if (eight_bits(kind) ? P > 0 && !row_scales : row_scales != nullptr) return CSA_ERR_INVALID_ARG;
    const uintptr_t in = kind == CSA_BF16 ? 2 : kind == CSA_F32 ? 4 : 1, out = out_type == CSA_BF16 ? 2 : 4;
    if (!aligned(k_pages, in) || !aligned(v_pages, in) || !aligned(k, out) || !aligned(v, out) || !aligned(row_scales, 8) ||
        !aligned(block_table, 4) || !aligned(seqlens, 4) || !aligned(starts, 4))
        return CSA_ERR_ALIGNMENT;
    if ((rc = device_ok()) != CSA_OK) return rc;
    return csa_cache_read_run(k_pages, v_pages, row_scales, block_table, seqlens, starts, k, k_strides, v, v_strides, B,
                              Hkv, T, d, P, S, M, kind, out_type, reinterpret_cast<cudaStream_t>(stream));
}

int csa_cache_accept(int *page_refs, int *block_table, int *seqlens, const int *parents,
                     const int *counts, const int *last, int *src, int *dst, int T, int B, int P,
                     int S, int M, csa_stream_t stream) {
    int rc = check_books(page_refs, block_table, seqlens, B, P, S, M);
    if (rc != CSA_OK) return rc;
    if (T < 0) return CSA_ERR_INVALID_ARG;
    if (T > CSA_TREE_MAX || (long long)P * S > kIntMax) return CSA_ERR_UNSUPPORTED;
    if (B == 0 || T == 0) return CSA_OK;
    if (!last || !src || !dst) return CSA_ERR_INVALID_ARG;
    if (!aligned(parents, 4) || !aligned(counts, 4) || !aligned(last, 4) || !aligned(src, 4) || !aligned(dst, 4))
        return CSA_ERR_ALIGNMENT;
    if ((rc = device_ok()) != CSA_OK) return rc;
    return csa_cache_accept_run(page_refs, block_table, seqlens, parents, counts, last, src, dst, T, B, P, S, M,
                                reinterpret_cast<cudaStream_t>(stream));
}

int csa_cache_copy_rows(void *k_pages, void *v_pages, long long row_bytes, void *row_scales,
                        long long scale_bytes, int layers, int P, int H, int S, const int *src,
                        const int *dst, int groups, int T, csa_stream_t stream) {
    if (row_bytes < 0 || scale_bytes < 0 || layers < 0 || P < 0 || H < 0 || S < 1 || groups < 0 || T < 0)
        return CSA_ERR_INVALID_ARG;
    if (row_bytes > 1 << 20 || scale_bytes > 1 << 20) return CSA_ERR_UNSUPPORTED;
    if (T > CSA_TREE_MAX || layers > 65535 || 3LL * H > 65535 || (long long)P * S > kIntMax) return CSA_ERR_UNSUPPORTED;
    if (layers == 0 || P == 0 || H == 0 || groups == 0 || T == 0) return CSA_OK;
    if ((!k_pages && !v_pages && !row_scales) || !src || !dst) return CSA_ERR_INVALID_ARG;
    if (!aligned(src, 4) || !aligned(dst, 4)) return CSA_ERR_ALIGNMENT;
    int rc = device_ok();
    if (rc != CSA_OK) return rc;
    return csa_cache_copy_rows_run(k_pages, v_pages, row_bytes, row_scales, scale_bytes, layers, P, H, S, src, dst,
                                   groups, T, reinterpret_cast<cudaStream_t>(stream));
}

int csa_cache_reserve(int *page_refs, int *block_table, int *seqlens, const int *counts,
                      int *shortfall, int B, int P, int S, int M, csa_stream_t stream) {
    int rc = check_books(page_refs, block_table, seqlens, B, P, S, M);
    if (rc != CSA_OK) return rc;
    if ((!counts && B > 0) || !shortfall) return CSA_ERR_INVALID_ARG;
    if (!aligned(counts, 4) || !aligned(shortfall, 4)) return CSA_ERR_ALIGNMENT;
    if ((rc = device_ok()) != CSA_OK) return rc;
    return csa_cache_reserve_run(page_refs, block_table, seqlens, counts, shortfall, B, P, S, M,
                                 reinterpret_cast<cudaStream_t>(stream));
}

int csa_cache_free(int *page_refs, int *block_table, int *seqlens, const int *rows, int R, int B,
                   int P, int S, int M, csa_stream_t stream) {
    int rc = check_books(page_refs, block_table, seqlens, B, P, S, M);
    if (rc != CSA_OK) return rc;
    if (R < 0 || (R > 0 && !rows)) return CSA_ERR_INVALID_ARG;
    if (!aligned(rows, 4)) return CSA_ERR_ALIGNMENT;
    if (R == 0) return CSA_OK;
    if ((rc = device_ok()) != CSA_OK) return rc;
    return csa_cache_free_run(page_refs, block_table, seqlens, rows, R, B, P, S, M,
                              reinterpret_cast<cudaStream_t>(stream));
}

int csa_cache_fork(int *page_refs, int *block_table, int *seqlens, const int *parents,
                   const int *children, int n, int *src, int *dst, int *shortfall, int B, int P,
                   int S, int M, csa_stream_t stream) {
    int rc = check_books(page_refs, block_table, seqlens, B, P, S, M);
    if (rc != CSA_OK) return rc;
    if (n > CSA_CACHE_MAX_FORKS) return CSA_ERR_UNSUPPORTED;
    if (n < 0 || !shortfall || (n > 0 && (!parents || !children || !src || !dst)))
        return CSA_ERR_INVALID_ARG;
    if (!aligned(parents, 4) || !aligned(children, 4) || !aligned(src, 4) || !aligned(dst, 4) ||
        !aligned(shortfall, 4))
        return CSA_ERR_ALIGNMENT;
    if ((rc = device_ok()) != CSA_OK) return rc;
    return csa_cache_fork_run(page_refs, block_table, seqlens, parents, children, n, src, dst,
                              shortfall, B, P, S, M, reinterpret_cast<cudaStream_t>(stream));
}

int csa_cache_compact(int *page_refs, int *block_table, const int *seqlens, int *src, int *dst,
                      int *moved, int B, int P, int S, int M, csa_stream_t stream) {
    int rc = check_books(page_refs, block_table, seqlens, B, P, S, M);
    if (rc != CSA_OK) return rc;
    if (!moved || (P > 1 && (!src || !dst))) return CSA_ERR_INVALID_ARG;
    if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(moved, 4)) return CSA_ERR_ALIGNMENT;
    if ((rc = device_ok()) != CSA_OK) return rc;
    return csa_cache_compact_run(page_refs, block_table, seqlens, src, dst, moved, B, P, S, M,
                                 reinterpret_cast<cudaStream_t>(stream));
}

int csa_cache_copy_pages(void *k_pages, void *v_pages, long long page_bytes, int layers, int P,
                         const int *src, const int *dst, int n, const int *count,
                         csa_stream_t stream) {
    if (page_bytes < 0 || layers < 0 || P < 0 || n < 0) return CSA_ERR_INVALID_ARG;
    if (page_bytes == 0 || layers == 0 || P == 0 || n == 0) return CSA_OK;
    if (!k_pages || !src || !dst) return CSA_ERR_INVALID_ARG;
    if ((long double)page_bytes * layers * P > 9.0e18L) return CSA_ERR_UNSUPPORTED;
    if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(count, 4)) return CSA_ERR_ALIGNMENT;
    int rc = device_ok();
    if (rc != CSA_OK) return rc;
    return csa_cache_copy_pages_run(k_pages, v_pages, page_bytes, layers, P, src, dst, n, count,
                                    reinterpret_cast<cudaStream_t>(stream));
}

long long csa_backward_workspace_bytes(int B, int H, int T, int d) {
    return backward_scratch_bytes(B, H, T, d);
}

int csa_backward(const void *q, const void *k, const void *v, const void *k0, const void *v0,
                 const void *out, const float *lse, const void *dout, void *dq, void *dk,
                 void *dv, float *dk0, float *dv0, void *workspace, long long workspace_bytes,
                 int B, int H, int T, int d, float scale, int k0_mode, csa_stream_t stream) {
    return backward_any(q, k, v, k0, v0, out, lse, dout, dq, dk, dv, dk0, dv0, workspace,
                        workspace_bytes, B, H, T, d, scale, k0_mode, true, stream);
}

int csa_backward_f32(const float *q, const float *k, const float *v, const float *k0,
                     const float *v0, const float *out, const float *lse, const float *dout,
                     float *dq, float *dk, float *dv, float *dk0, float *dv0, void *workspace,
                     long long workspace_bytes, int B, int H, int T, int d, float scale,
                     int k0_mode, csa_stream_t stream) {
    return backward_any(q, k, v, k0, v0, out, lse, dout, dq, dk, dv, dk0, dv0, workspace,
                        workspace_bytes, B, H, T, d, scale, k0_mode, false, stream);
}

long long csa_forward_host_workspace_bytes(int B, int H, int T, int d) {
    if (d > 256) return -1;
    return csa_host_scratch_bytes(B, H, T, d);
}

int csa_forward_host_ex(const void *q, const void *k, const void *v, const void *k0,
                        const void *v0, void *out, float *lse, void *workspace,
                        long long workspace_bytes, int B, int H, int T, int d, float scale,
                        int k0_mode, int heads_per_chunk, unsigned flags, csa_stream_t stream,
                        csa_stream_t stream_h2d, csa_stream_t stream_d2h) {
    if (flags & ~CSA_HOST_NO_ENTRY_WAIT) return CSA_ERR_INVALID_ARG;
    bool empty;
    int rc = check_common(q, k, v, k0, v0, out, B, H, T, d, scale, k0_mode, true, &empty);
    if (rc != CSA_OK || empty) return rc;
    if (d > 256) return CSA_ERR_UNSUPPORTED;
    if (heads_per_chunk < 1 || heads_per_chunk > H || H % heads_per_chunk != 0)
        return CSA_ERR_INVALID_ARG;
    if (!workspace) return CSA_ERR_INVALID_ARG;
    const long long need = csa_host_scratch_bytes(B, H, T, d);
    if (need < 0 || workspace_bytes < need) return CSA_ERR_INVALID_ARG;
    if (!aligned(workspace, 256) || (lse && !aligned(lse, 4))) return CSA_ERR_ALIGNMENT;
    if (k0_mode == CSA_K0_GIVEN && (!aligned(k0, 2) || !aligned(v0, 2))) return CSA_ERR_ALIGNMENT;
    if ((rc = device_ok()) != CSA_OK) return rc;
    return csa_host_forward(q, k, v, k0, v0, out, lse, workspace, B, H, T, d, scale, k0_mode,
                            heads_per_chunk, !(flags & CSA_HOST_NO_ENTRY_WAIT),
                            reinterpret_cast<cudaStream_t>(stream),
                            reinterpret_cast<cudaStream_t>(stream_h2d),
                            reinterpret_cast<cudaStream_t>(stream_d2h));
}

int csa_forward_host(const void *q, const void *k, const void *v, const void *k0, const void *v0,
                     void *out, float *lse, void *workspace, long long workspace_bytes, int B,
                     int H, int T, int d, float scale, int k0_mode, int heads_per_chunk,
                     csa_stream_t stream, csa_stream_t stream_h2d, csa_stream_t stream_d2h) {
    return csa_forward_host_ex(q, k, v, k0, v0, out, lse, workspace, workspace_bytes, B, H, T, d,
                               scale, k0_mode, heads_per_chunk, 0u, stream, stream_h2d,
                               stream_d2h);
}

long long csa_decode_range_workspace_bytes(int B, int H, int pos_lo, int pos_hi, int d) {
    return csa_decode_range_scratch_bytes(B, H, pos_lo, pos_hi, d);
}

int csa_decode_range(const void *q, const void *k_shard, const void *v_shard, const void *k0,
                     const void *v0, const int *seqlens, float *out, float *lse, void *workspace,
                     long long workspace_bytes, int B, int H, int T, int d, float scale,
                     int k0_mode, int pos_lo, int pos_hi, csa_stream_t stream) {
    return decode_range_bf16(q, k_shard, v_shard, k0, v0, seqlens, out, lse, workspace,
                             workspace_bytes, B, H, T, d, scale, k0_mode, pos_lo, pos_hi, stream);
}

int csa_decode_merge_ranges(const float *o_parts, const float *lse_parts, int R, int B, int H,
                            int d, void *out, float *lse, csa_stream_t stream) {
    if (R < 1 || B < 0 || H < 0 || d < 1 || d > 256) return CSA_ERR_INVALID_ARG;
    if ((long long)B * H == 0) return CSA_OK;
    if (!o_parts || !lse_parts || !out) return CSA_ERR_INVALID_ARG;
    if ((long long)R * B * H * d > (1LL << 40)) return CSA_ERR_UNSUPPORTED;
    if (!aligned(o_parts, 4) || !aligned(lse_parts, 4) || !aligned(out, 2) || (lse && !aligned(lse, 4)))
        return CSA_ERR_ALIGNMENT;
    int rc = device_ok();
    if (rc != CSA_OK) return rc;
    return csa_decode_merge_ranges_run(o_parts, lse_parts, R, B, H, d, out, lse,
                                       reinterpret_cast<cudaStream_t>(stream));
}

long long csa_decode_workspace_bytes(int B, int H, int T, int d) {
    return csa_decode_scratch_bytes(B, H, T, d);
}

int csa_decode(const void *q, const void *k_cache, const void *v_cache, const void *k0,
               const void *v0, const int *seqlens, void *out, float *lse, void *workspace,
               long long workspace_bytes, int B, int H, int T, int d, float scale, int k0_mode,
               csa_stream_t stream) {
    return decode_bf16(q, k_cache, v_cache, k0, v0, seqlens, out, lse, workspace,
                       workspace_bytes, B, H, T, d, scale, k0_mode, stream);
}

int csa_forward(const void *q, const void *k, const void *v, const void *k0, const void *v0,
                void *out, float *lse, int B, int H, int T, int d, float scale, int k0_mode,
                csa_stream_t stream) {
    return forward_bf16(q, k, v, k0, v0, out, lse, B, H, T, d, scale, k0_mode, kFormExact, stream);
}

int csa_forward_short_conv(const void *q, const void *k, const void *v, const void *k0,
                           const void *v0, void *out, float *lse, int B, int H, int T, int d,
                           float scale, int k0_mode, csa_stream_t stream) {
    return forward_bf16(q, k, v, k0, v0, out, lse, B, H, T, d, scale, k0_mode, kFormShortConv,
                        stream);
}

int csa_forward_logdomain(const void *q, const void *k, const void *v, const void *k0,
                          const void *v0, void *out, float *lse, int B, int H, int T, int d,
                          float scale, int k0_mode, csa_stream_t stream) {
    return forward_bf16(q, k, v, k0, v0, out, lse, B, H, T, d, scale, k0_mode, kFormLogDomain,
                        stream);
}

int csa_forward_symmetric(const void *q, const void *k, const void *v, void *out, float *lse,
                          int B, int H, int T, int d, float scale, csa_stream_t stream) {
    return forward_bf16(q, k, v, nullptr, nullptr, out, lse, B, H, T, d, scale, CSA_K0_ZERO,
                        kFormSymmetric, stream);
}

int csa_forward_symmetric_f32(const float *q, const float *k, const float *v, float *out,
                              float *lse, int B, int H, int T, int d, float scale,
                              csa_stream_t stream) {
    return forward_f32(q, k, v, nullptr, nullptr, out, lse, B, H, T, d, scale, CSA_K0_ZERO,
                       kFormSymmetric, stream);
}

int csa_forward_short_conv_f32(const float *q, const float *k, const float *v, const float *k0,
                               const float *v0, float *out, float *lse, int B, int H, int T,
                               int d, float scale, int k0_mode, csa_stream_t stream) {
    return forward_f32(q, k, v, k0, v0, out, lse, B, H, T, d, scale, k0_mode, kFormShortConv,
                       stream);
}

int csa_forward_f32(const float *q, const float *k, const float *v, const float *k0,
                    const float *v0, float *out, float *lse, int B, int H, int T, int d,
                    float scale, int k0_mode, csa_stream_t stream) {
    return forward_f32(q, k, v, k0, v0, out, lse, B, H, T, d, scale, k0_mode, kFormExact, stream);
}

int csa_std_forward(const void *q, const void *k, const void *v, void *out, float *lse, int B,
                    int H, int T, int d, float scale, csa_stream_t stream) {
    return forward_bf16(q, k, v, nullptr, nullptr, out, lse, B, H, T, d, scale, CSA_K0_ZERO,
                        kFormStd, stream);
}

int csa_std_forward_f32(const float *q, const float *k, const float *v, float *out, float *lse,
                        int B, int H, int T, int d, float scale, csa_stream_t stream) {
    return forward_f32(q, k, v, nullptr, nullptr, out, lse, B, H, T, d, scale, CSA_K0_ZERO,
                       kFormStd, stream);
}

int csa_logphi2_eval(const float *x, float *y, int n, csa_stream_t stream) {
    if (n < 0) return CSA_ERR_INVALID_ARG;
    if (n == 0) return CSA_OK;
    if (!x || !y) return CSA_ERR_INVALID_ARG;
    int rc = device_ok();
    if (rc != CSA_OK) return rc;
    return from_cuda(csa_simt_logphi2_eval(x, y, n, reinterpret_cast<cudaStream_t>(stream)));
}

int csa_segment_weights_eval(const float *u0, const float *u1, float *right, float *left, int n,
                             csa_stream_t stream) {
    if (n < 0) return CSA_ERR_INVALID_ARG;
    if (n == 0) return CSA_OK;
    if (!u0 || !u1 || !right || !left) return CSA_ERR_INVALID_ARG;
    int rc = device_ok();
    if (rc != CSA_OK) return rc;
    return from_cuda(csa_tc_segment_weights_eval(u0, u1, right, left, n,
                                                 reinterpret_cast<cudaStream_t>(stream)));
}

int csa_device_status(void) {
    int rc = device_ok();
    if (rc != CSA_OK) return rc;
    const int a = csa_tc_take_status();  // synchronises the device
    const int b = csa_tc_std_take_status();
    const int c = csa_decode_take_status();
    const int d = csa_tc_backward_take_status();
    const int e = take_words();
    for (const int word : {a, b, c, d, e})
        if (word != CSA_OK) return word;
    return CSA_OK;
}

int csa_selftest_wait_timeout(unsigned timeout_us, csa_stream_t stream) {
    if (timeout_us < 1 || timeout_us > 1000000u) return CSA_ERR_INVALID_ARG;
    int rc = device_ok();
    if (rc != CSA_OK) return rc;
    return from_cuda(csa_tc_selftest_wait_timeout(timeout_us, reinterpret_cast<cudaStream_t>(stream)));
}

int csa_selftest_forward_delay(const void *q, const void *k, const void *v, const void *k0,
                               const void *v0, void *out, float *lse, int B, int H, int T, int d,
                               float scale, int k0_mode, unsigned delay_ns, int delay_half,
                               csa_stream_t stream) {
    if (delay_ns > 1000000u || (delay_half != 0 && delay_half != 1)) return CSA_ERR_INVALID_ARG;
    bool empty;
    int rc = check_common(q, k, v, k0, v0, out, B, H, T, d, scale, k0_mode, true, &empty);
    if (rc != CSA_OK || empty) return rc;
    if (d != 64 && d != 128) return CSA_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
        (lse && !aligned(lse, 4)))
        return CSA_ERR_ALIGNMENT;
    if (k0_mode == CSA_K0_GIVEN && (!aligned(k0, 2) || !aligned(v0, 2))) return CSA_ERR_ALIGNMENT;
    if ((rc = device_ok()) != CSA_OK) return rc;
    return csa_tc_forward_delayed(q, k, v, k0, v0, out, lse, B, H, T, d, scale, k0_mode, delay_ns,
                                  delay_half, reinterpret_cast<cudaStream_t>(stream));
}

int csa_decode_noalloc(const void *q, const void *k_cache, const void *v_cache, const void *k0,
                       const void *v0, const int *seqlens, void *out, float *lse, int B, int H,
                       int T, int d, float scale, int k0_mode, csa_stream_t stream) {
    // csa_decode's checks first, in its order; then the scratch capacity
    bool empty;
    long long need = 0;
    int rc = decode_check(q, k_cache, v_cache, k0, v0, seqlens, out, lse, B, H, T, d, scale,
                          k0_mode, &empty, &need);
    if (rc != CSA_OK || empty) return rc;
    if (need > (long long)CSA_DECODE_NOALLOC_SCRATCH_BYTES) return CSA_ERR_UNSUPPORTED;
    if ((rc = device_ok()) != CSA_OK) return rc;
    void *scratch = nullptr;
    if ((rc = csa_decode_noalloc_scratch(&scratch)) != CSA_OK) return rc;
    return csa_decode_run(q, k_cache, v_cache, k0, v0, seqlens, out, lse, scratch, B, H, T, d,
                          scale, k0_mode, reinterpret_cast<cudaStream_t>(stream));
}

const char *csa_status_string(int status) {
    switch (status) {
        case CSA_OK: return "ok";
        case CSA_ERR_INVALID_ARG: return "invalid argument";
        case CSA_ERR_UNSUPPORTED: return "unsupported shape or value";
        case CSA_ERR_ALIGNMENT: return "misaligned pointer";
        case CSA_ERR_CUDA: return "CUDA runtime error";
        case CSA_ERR_TIMEOUT: return "device-side wait timed out";
        case CSA_ERR_NO_DEVICE: return "no sm_103 device is current";
        default: return "unknown status";
    }
}

int csa_abi_version(void) { return CSA_ABI_VERSION; }

}  // extern "C"

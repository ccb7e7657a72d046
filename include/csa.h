/*
 * csa.h - C ABI of libcsa.so: forward pass of causal Continuous Softmax
 * Attention on one NVIDIA GB300 (sm_103a).
 *
 * The method: Jianlin Su, "Continuous Softmax Attention" (Scientific Spaces
 * #11980).  Attention over the causal prefix is made continuous by linear
 * interpolation of keys and values between integer positions (eq. (2), (3));
 * the integrals close (eq. (4)-(7)) and reduce to a softmax over corrected
 * logits (eq. (10), (11)):
 *
 *     a_{t,i} = scale * q_t . k_i                       i = 0..t
 *     e^{b_{t,0}} = phi2(a_{t,1} - a_{t,0})
 *     e^{b_{t,i}} = phi2(a_{t,i-1} - a_{t,i}) + phi2(a_{t,i+1} - a_{t,i})
 *     e^{b_{t,t}} = phi2(a_{t,t-1} - a_{t,t})
 *     o_t = sum_i e^{a+b} v_i / sum_i e^{a+b},   phi2(x) = (e^x - 1 - x)/x^2
 *
 * with an extra sink pair k_0, v_0 (section "Analysis of the Result": zero,
 * a copy of the first token, or trainable).
 *
 * Common conventions for every attention entry point below
 * ---------------------------------------------------------
 *  Layout     q, k, v, out: contiguous row-major [B, H, T, d]; token r of the
 *             arrays (0-based) is the page's t = r + 1, array key j is the
 *             page's k_{j+1}.  k0, v0: contiguous [H, d] (one sink pair per
 *             head, shared across the batch).  lse: contiguous float [B, H, T].
 *  Memory     every pointer is DEVICE memory owned by the caller; the library
 *             allocates nothing and keeps no pointer after the call returns.
 *             out and lse must not overlap any input.
 *  Scheduling the tensor-core forward kernels (csa_forward, its short-conv and
 *             symmetric forms, and the kernels csa_forward_host launches)
 *             run one CTA per SM and take query tiles from a counter in the
 *             library's device image: 64 counter slots per device, drawn in
 *             turn.  Each slot has one CUDA event, created on first use and
 *             kept for the life of the process; a launch's stream waits on
 *             its slot's event (the slot's previous launch), so calls on any
 *             streams never share a counter.  Under stream capture the event
 *             is left out: a captured graph keeps the slot it drew, so a
 *             replay must not run at the same time as another replay of the
 *             same graph, nor as a later call that draws the same slot (every
 *             64th forward call on the device).
 *  Stream     the work is enqueued on `stream` (a cudaStream_t; NULL = the
 *             legacy default stream) and the call returns without waiting.
 *             Outputs are valid once the stream reaches that point.
 *  Scale      logits are scale * q.k; the correction b is formed on the
 *             scaled logits.  scale must be finite.
 *  lse        natural-log normaliser: lse_t = log sum_i e^{a_{t,i}+b_{t,i}},
 *             which equals log of eq. (2)'s denominator integral.  May be
 *             NULL when not wanted.
 *  Empty      B, H or T equal to 0 is a valid empty problem: CSA_OK, nothing
 *             is launched.
 *  Errors     the return value is CSA_OK (0) or one of the negative codes
 *             below.  Argument errors are detected on the host before any
 *             launch, and nothing is enqueued.  CSA_ERR_CUDA reports a launch
 *             failure (cudaGetLastError); asynchronous kernel faults surface,
 *             as usual in CUDA, on the next synchronising call.  Device-side
 *             bounded waits that expire set a sticky status word readable
 *             with csa_device_status().
 */
#ifndef CSA_H_
#define CSA_H_

#ifdef __cplusplus
extern "C" {
#endif

/* Same handle type as cudaStream_t / CUstream. */
typedef struct CUstream_st *csa_stream_t;

/* Choice of the extra pair k_0, v_0 ("Analysis of the Result", last
 * paragraph: all zeros; k_0 = k_1, v_0 = v_1; or trainable). */
typedef enum {
    CSA_K0_ZERO = 0,       /* k_0 = v_0 = 0 (the page's experiments)       */
    CSA_K0_COPY_FIRST = 1, /* k_0 = k_1, v_0 = v_1 of the same (b, h)       */
    CSA_K0_GIVEN = 2       /* k0, v0 supplied per head, [H, d]              */
} csa_k0_mode;

enum {
    CSA_OK = 0,
    CSA_ERR_INVALID_ARG = -1, /* NULL pointer, negative size, d < 1,
                                 non-finite scale, bad mode, k0/v0 NULL in
                                 CSA_K0_GIVEN                                 */
    CSA_ERR_UNSUPPORTED = -2, /* shape or value outside what a kernel
                                 supports (see each entry point)              */
    CSA_ERR_ALIGNMENT = -3,   /* a pointer is not aligned as required         */
    CSA_ERR_CUDA = -4,        /* a CUDA runtime call or launch failed         */
    CSA_ERR_TIMEOUT = -5,     /* a device-side bounded wait expired           */
    CSA_ERR_NO_DEVICE = -6    /* no usable sm_103 device is current           */
};

/*
 * csa_forward - continuous attention, bf16 inputs, tensor-core path.
 *   Defines: eq. (10)/(11) of "Continuous Softmax Attention" ("Assembly and
 *   Simplification"), which equals eq. (2) ("Problem Statement").
 *   q, k, v, k0, v0: bf16 (__nv_bfloat16); out: bf16; lse: float.
 *   Accumulation and the correction b are computed in fp32.
 *   d = 64 or 128 runs the tcgen05/TMA kernel; any other 1 <= d <= 256 runs
 *   the CUDA-core kernel.  d > 256: CSA_ERR_UNSUPPORTED.  Any finite scale,
 *   of either sign, on both kernels.
 *   q, k, v, out must be 16-byte aligned (CSA_ERR_ALIGNMENT otherwise).
 *   k0, v0 are read only in CSA_K0_GIVEN mode and may be NULL otherwise.
 */
int csa_forward(const void *q, const void *k, const void *v, const void *k0, const void *v0,
                void *out, float *lse, int B, int H, int T, int d, float scale, int k0_mode,
                csa_stream_t stream);

/*
 * csa_forward_f32 - continuous attention, fp32 inputs and outputs, computed
 *   in fp32 on CUDA cores (no TF32), with b formed in the log domain by a
 *   stable log phi2 (series near 0, logarithmic form for large |x|, combined
 *   by logaddexp).  Same definition and conventions as csa_forward;
 *   1 <= d <= 256.  All pointers 4-byte aligned.
 */
int csa_forward_f32(const float *q, const float *k, const float *v, const float *k0,
                    const float *v0, float *out, float *lse, int B, int H, int T, int d,
                    float scale, int k0_mode, csa_stream_t stream);

/*
 * csa_forward_host - csa_forward from HOST buffers, end to end: copies q, k,
 *   v to the device, runs the forward pass and copies out and lse back,
 *   overlapping the copies of one chunk of heads with the kernel of another
 *   (the (b, h) problems are independent).  Same definition, result and
 *   d rules as csa_forward.
 *   q, k, v, out: HOST bf16 [B, H, T, d]; lse: HOST float [B, H, T] or NULL.
 *   They should be page-locked (cudaHostAlloc / cudaHostRegister): pageable
 *   memory is still correct but the copies then do not overlap.  The host
 *   inputs must stay unchanged, and out/lse must not be read, until the work
 *   completes on `stream`.
 *   k0, v0: DEVICE bf16 [H, d] (CSA_K0_GIVEN only).
 *   workspace: DEVICE scratch of at least csa_forward_host_workspace_bytes
 *   (B, H, T, d) bytes, 256-byte aligned (device copies of q, k, v, out,
 *   lse).
 *   heads_per_chunk: heads per pipeline chunk; must divide H.
 *   stream runs the kernels; stream_h2d and stream_d2h the two copy
 *   directions (they may equal stream, at the cost of the overlap).  All
 *   work of the call is complete once `stream` reaches the point after it.
 *   Errors as csa_forward, plus CSA_ERR_INVALID_ARG for a heads_per_chunk
 *   that does not divide H or a workspace too small.
 */
int csa_forward_host(const void *q, const void *k, const void *v, const void *k0, const void *v0,
                     void *out, float *lse, void *workspace, long long workspace_bytes, int B,
                     int H, int T, int d, float scale, int k0_mode, int heads_per_chunk,
                     csa_stream_t stream, csa_stream_t stream_h2d, csa_stream_t stream_d2h);

/*
 * csa_forward_host_ex - csa_forward_host with flags (the pages have no
 *   counterpart).  flags = 0 is csa_forward_host.  CSA_HOST_NO_ENTRY_WAIT:
 *   the host-to-device copies do not wait for the work already queued on
 *   `stream`, so that a call's copies in can overlap the previous call's
 *   kernels and copies out.  The caller then orders the calls that share a
 *   workspace itself: a call's copies in must not start before the previous
 *   call on the same workspace has completed on `stream` (for instance: two
 *   workspaces used alternately, each call recording an event on `stream`
 *   after it, and stream_h2d waiting for the event of the call before last).
 *   Unknown flag bits: CSA_ERR_INVALID_ARG.  Otherwise as csa_forward_host.
 */
#define CSA_HOST_NO_ENTRY_WAIT 1u
int csa_forward_host_ex(const void *q, const void *k, const void *v, const void *k0,
                        const void *v0, void *out, float *lse, void *workspace,
                        long long workspace_bytes, int B, int H, int T, int d, float scale,
                        int k0_mode, int heads_per_chunk, unsigned flags, csa_stream_t stream,
                        csa_stream_t stream_h2d, csa_stream_t stream_d2h);

/* csa_forward_host_workspace_bytes - device workspace csa_forward_host needs
 * (host only), or -1 for a negative size or d outside 1..256. */
long long csa_forward_host_workspace_bytes(int B, int H, int T, int d);

/*
 * csa_forward_short_conv - the short-conv reading of eq. (13) ("Analysis of
 *   the Result" of "Continuous Softmax Attention"): the correction b is
 *   replaced by its first-order Taylor term, which the page likens to a
 *   short convolution over the attention logits:
 *       b_{t,i} = (a_{t,i-1} + a_{t,i+1} - 2 a_{t,i}) / 6      1 <= i <= t-1
 *       b_{t,0} = -log 2 + (a_{t,1} - a_{t,0}) / 3
 *       b_{t,t} = -log 2 + (a_{t,t-1} - a_{t,t}) / 3
 *   (the ends from log phi2(x) = -log 2 + x/3 + O(x^2)); o and lse as in
 *   eq. (11).  It agrees with csa_forward to second order in the logit
 *   steps and forms no phi2, so it runs faster.  Same arguments, layout,
 *   alignment, d rules, sink modes and errors as csa_forward.
 */
int csa_forward_short_conv(const void *q, const void *k, const void *v, const void *k0,
                           const void *v0, void *out, float *lse, int B, int H, int T, int d,
                           float scale, int k0_mode, csa_stream_t stream);

/*
 * csa_forward_logdomain - csa_forward with the weights formed as eq. (10)
 *   and (11) of "Continuous Softmax Attention" ("Assembly and
 *   Simplification") write them: per key, z = a + b with
 *   b = log(phi2(a_{i-1} - a_i) + phi2(a_{i+1} - a_i)) (one-sided at the
 *   sink and at the row's own key) from log phi2 of each logit step, added
 *   in the log domain, and then e^{z - m}.  The same result as csa_forward
 *   (which forms each key's weight from the two interval shares of eq. (9)
 *   with one exponential and one reciprocal) within the bf16 rounding of
 *   the weights; it takes about nine special-function operations per
 *   (query, key) pair where csa_forward takes two, and is kept as the
 *   reference evaluation of that step.  Same arguments, layout, alignment,
 *   d rules (d other than 64 and 128 runs the CUDA-core kernel, which
 *   forms b this way too), sink modes and errors as csa_forward.
 */
int csa_forward_logdomain(const void *q, const void *k, const void *v, const void *k0,
                          const void *v0, void *out, float *lse, int B, int H, int T, int d,
                          float scale, int k0_mode, csa_stream_t stream);

/* csa_forward_short_conv_f32 - the same in fp32 on CUDA cores, 1 <= d <= 256. */
int csa_forward_short_conv_f32(const float *q, const float *k, const float *v, const float *k0,
                               const float *v0, float *out, float *lse, int B, int H, int T,
                               int d, float scale, int k0_mode, csa_stream_t stream);

/*
 * csa_forward_symmetric - continuous attention over the symmetric interval
 *   [1/2, t + 1/2] that the original Continuum Attention paper uses (cited in
 *   "Problem Statement" of "Continuous Softmax Attention"; eq. (2) with that
 *   interval).  Inside [1, t] keys and values follow eq. (3); the end
 *   half-cells [1/2, 1] and [t, t + 1/2] hold k_1, v_1 and k_t, v_t constant
 *   (a causal row has no k_{t+1}), so there is no sink.  As weights:
 *       e^{b_{t,1}} = 1/2 + phi2(a_{t,2} - a_{t,1}),
 *       e^{b_{t,t}} = phi2(a_{t,t-1} - a_{t,t}) + 1/2,
 *       interior keys as eq. (10); t = 1 gives o_1 = v_1.
 *   lse_t = log of the denominator integral over [1/2, t + 1/2].  bf16; same
 *   layout, alignment and d rules as csa_forward (no k0, v0, mode).
 */
int csa_forward_symmetric(const void *q, const void *k, const void *v, void *out, float *lse,
                          int B, int H, int T, int d, float scale, csa_stream_t stream);

/* csa_forward_symmetric_f32 - the same in fp32 on CUDA cores, 1 <= d <= 256. */
int csa_forward_symmetric_f32(const float *q, const float *k, const float *v, float *out,
                              float *lse, int B, int H, int T, int d, float scale,
                              csa_stream_t stream);

/*
 * csa_std_forward - standard causal softmax attention (b = 0, no sink),
 *   bf16 inputs, tensor-core path.
 *   Defines: eq. (12) of "Continuous Softmax Attention" ("Analysis of the
 *   Result"), the same as softmax(q k^T * scale + M) v with the causal mask M
 *   of "Attention, from the softmax up" ("The one line").
 *   lse_t = log sum_{i=1}^t e^{a_{t,i}}.  Same layout, alignment and d rules
 *   as csa_forward.
 */
int csa_std_forward(const void *q, const void *k, const void *v, void *out, float *lse, int B,
                    int H, int T, int d, float scale, csa_stream_t stream);

/* csa_std_forward_f32 - eq. (12) in fp32 on CUDA cores; 1 <= d <= 256. */
int csa_std_forward_f32(const float *q, const float *k, const float *v, float *out, float *lse,
                        int B, int H, int T, int d, float scale, csa_stream_t stream);

/*
 * csa_backward - gradients of the continuous forward pass (csa_forward) for
 *   an upstream gradient dout = dL/d(out): dq, dk, dv and, in CSA_K0_GIVEN
 *   mode, the gradients of the trainable sink pair.
 *   Defines: the derivative of eq. (10)/(11) of "Continuous Softmax
 *   Attention" ("Assembly and Simplification"); the pages train models with
 *   the method ("Simple Experiments") but do not write this step out.  With
 *   p_i = e^{a_i - lse}, P_i the attention weight e^{a_i + b_i - lse},
 *   dP_i = dout . v_i and D = dout . out, for every row
 *       dL/da_i = P_i (dP_i - D) + F_i - F_{i+1},
 *       F_i = c_i (dP_{i-1} - dP_i),  c_i = p_{i-1} phi2'(a_i - a_{i-1}),
 *   (F = 0 past both ends of the row; phi2' is the derivative of eq. (6)'s
 *   phi2), and dq = scale sum_i dL/da_i k_i, dk_i += scale dL/da_i q,
 *   dv_i += P_i dout.
 *   q, k, v, out, dout: bf16 [B, H, T, d] (out from csa_forward);
 *   lse: float [B, H, T] from csa_forward (required);
 *   dq, dk, dv: bf16 [B, H, T, d], overwritten;
 *   k0, v0: bf16 [H, d] (CSA_K0_GIVEN only); dk0, dv0: float [H, d], the
 *   gradients of the sink pair summed over the batch and the rows
 *   (CSA_K0_GIVEN only; may be NULL otherwise).  In CSA_K0_COPY_FIRST the
 *   sink's gradient is added to key 0's; in CSA_K0_ZERO the sink is a
 *   constant.
 *   workspace: DEVICE scratch of at least csa_backward_workspace_bytes(B, H,
 *   T, d) bytes, 16-byte aligned, contents on entry irrelevant.  Concurrent
 *   calls need distinct workspaces.
 *   1 <= d <= 256 (CSA_ERR_UNSUPPORTED otherwise).  Tensors 2-byte aligned,
 *   lse, dk0, dv0 4-byte aligned.  Empty problems (B, H or T = 0) are
 *   CSA_OK; in CSA_K0_GIVEN mode dk0 and dv0 are then zeroed.  Atomic
 *   accumulation makes the low bits of dk, dv, dk0, dv0 depend on the order
 *   in which the hardware completes them.
 */
int csa_backward(const void *q, const void *k, const void *v, const void *k0, const void *v0,
                 const void *out, const float *lse, const void *dout, void *dq, void *dk,
                 void *dv, float *dk0, float *dv0, void *workspace, long long workspace_bytes,
                 int B, int H, int T, int d, float scale, int k0_mode, csa_stream_t stream);

/* csa_backward_f32 - the same in fp32 throughout (CUDA cores, no TF32); all
 * tensors 4-byte aligned. */
int csa_backward_f32(const float *q, const float *k, const float *v, const float *k0,
                     const float *v0, const float *out, const float *lse, const float *dout,
                     float *dq, float *dk, float *dv, float *dk0, float *dv0, void *workspace,
                     long long workspace_bytes, int B, int H, int T, int d, float scale,
                     int k0_mode, csa_stream_t stream);

/* csa_backward_workspace_bytes - workspace bytes csa_backward and
 * csa_backward_f32 need (host only), or -1 for a negative size or d outside
 * 1..256. */
long long csa_backward_workspace_bytes(int B, int H, int T, int d);

/*
 * csa_decode - one decode step: for every sequence b and head h, the output
 *   of the newest token, position t = n_b, against the sink and the n_b
 *   cached keys and values.
 *   Defines: eq. (10)/(11) of "Continuous Softmax Attention" ("Assembly and
 *   Simplification") for the single row t = n_b; the result equals row
 *   n_b - 1 of csa_forward run on the first n_b tokens, except that the
 *   weights stay in fp32 (they are not rounded to bf16 for a tensor core).
 *   q:         bf16 [B, H, d], the newest token's query of each sequence.
 *   k_cache, v_cache: bf16 [B, H, T, d]; T is the capacity.  Sequence b uses
 *              rows 0 .. n_b - 1, the last being the newest token's own key
 *              and value.
 *   k0, v0:    bf16 [H, d], read in CSA_K0_GIVEN mode only.  In
 *              CSA_K0_COPY_FIRST the sink is row 0 of the cache.
 *   seqlens:   DEVICE int32 [B] with n_b, or NULL for n_b = T for every b.
 *              A length outside [1, T] is not detectable on the host: that
 *              sequence's out and lse are set to NaN and the sticky status
 *              word (csa_device_status) records CSA_ERR_INVALID_ARG.
 *   out:       bf16 [B, H, d]; lse: float [B, H] natural log, or NULL.
 *   workspace: DEVICE scratch of at least csa_decode_workspace_bytes(B, H,
 *              T, d) bytes owned by the caller (16-byte aligned); its
 *              contents on entry do not matter and are overwritten.  Calls
 *              that run concurrently must use distinct workspaces.
 *   d must be 64, 128 or 256 (CSA_ERR_UNSUPPORTED otherwise).  q, k_cache,
 *   v_cache, out, workspace (and k0, v0 in GIVEN mode) must be 16-byte
 *   aligned.  B * H == 0: CSA_OK, nothing launched.  T == 0 with B * H > 0:
 *   CSA_ERR_INVALID_ARG (the newest token's key must be in the cache).
 *   workspace_bytes smaller than needed: CSA_ERR_INVALID_ARG.
 *   Computed on CUDA cores in fp32 (the step is bound by reading the cache):
 *   the positions 0..n_b are split into chunks, each chunk's partial sums
 *   are formed against its own maximum and merged by log-sum-exp.
 */
int csa_decode(const void *q, const void *k_cache, const void *v_cache, const void *k0,
               const void *v0, const int *seqlens, void *out, float *lse, void *workspace,
               long long workspace_bytes, int B, int H, int T, int d, float scale, int k0_mode,
               csa_stream_t stream);

/*
 * csa_decode_noalloc - csa_decode without a caller workspace.  The method's
 *   pages have no counterpart to this entry point: it is a convenience of
 *   this library for callers that cannot hand over scratch memory.
 *   Same arguments and result as csa_decode, minus workspace and
 *   workspace_bytes.  The chunk partials go to a fixed scratch array of
 *   CSA_DECODE_NOALLOC_SCRATCH_BYTES bytes that lives in the library's device
 *   image (one per device); the call allocates no memory of any kind.  Each
 *   call writes every partial it reads, so nothing in the array needs to
 *   start at zero.
 *   Memory: the array is CSA_DECODE_NOALLOC_SCRATCH_BYTES (64 MiB) of device
 *   memory on each device that loads it, held until the process exits.  It
 *   sits in a module of its own: with lazy module loading (the CUDA
 *   default) only processes that call csa_decode_noalloc hold it.
 *   Set-up: the first call on a device, and the first call after a device
 *   reset (a new context), looks the scratch address up with
 *   cudaGetSymbolAddress (that device must be current): make that call
 *   before any stream capture begins.
 *   Checks: csa_decode's argument checks run first, in its order and with
 *   its error codes; a size that passes them but whose scratch need exceeds
 *   the capacity then gives CSA_ERR_UNSUPPORTED, before anything is
 *   launched.
 *   Concurrency: every call on a device shares that one scratch array, so
 *   calls that can overlap on the device (different streams, or several host
 *   threads) race and corrupt each other's results.  Serialise them, e.g. on
 *   one stream, or use csa_decode with distinct workspaces.
 */
#define CSA_DECODE_NOALLOC_SCRATCH_BYTES (64u << 20)
int csa_decode_noalloc(const void *q, const void *k_cache, const void *v_cache, const void *k0,
                       const void *v0, const int *seqlens, void *out, float *lse, int B, int H,
                       int T, int d, float scale, int k0_mode, csa_stream_t stream);

/*
 * csa_decode_workspace_bytes - bytes of workspace csa_decode needs for these
 *   sizes (host only, no device needed), or -1 for a negative size, a d
 *   other than 64, 128, 256, or a size beyond 2^62 bytes.
 */
long long csa_decode_workspace_bytes(int B, int H, int T, int d);

/*
 * csa_decode_range - the decode step restricted to the positions [pos_lo,
 *   pos_hi) of every row (position 0 is the sink, position i >= 1 is cache
 *   row i - 1), for a KV cache whose time axis is split across devices
 *   (context parallelism).  The pages have no counterpart; it is eq. (11)
 *   ("Assembly and Simplification" of "Continuous Softmax Attention")
 *   summed over the owned positions only, each position's weight e^{a+b}
 *   still taking its correction b from both neighbours (eq. (10)), so that
 *   merging the ranges of a partition of [0, n] with csa_decode_merge_ranges
 *   gives csa_decode's result.
 *   q: DEVICE bf16 [B, H, d]; seqlens, k0, v0, scale, k0_mode, T and d as
 *   csa_decode (T is the capacity of the whole cache, 1 <= n_b <= T).
 *   k_shard, v_shard: DEVICE bf16 [B, H, rows, d] holding the cache rows
 *   [max(pos_lo - 2, 0), min(pos_hi, T)), rows = min(pos_hi, T) -
 *   max(pos_lo - 2, 0): the owned positions and one neighbour on each side.
 *   0 <= pos_lo < pos_hi <= T + 1 and pos_lo != 1 (a range cannot start
 *   right after the sink); otherwise CSA_ERR_INVALID_ARG.
 *   out: DEVICE fp32 [B, H, d], the range's normalised output o_r;
 *   lse: DEVICE fp32 [B, H] (required), log of the range's weight sum.  A
 *   row whose length n_b < pos_lo has no owned position: o_r = 0 and
 *   lse_r = -inf.
 *   workspace: DEVICE scratch of csa_decode_range_workspace_bytes(B, H,
 *   pos_lo, pos_hi, d) bytes, 16-byte aligned.  Tensors 16-byte aligned,
 *   lse and seqlens 4-byte aligned.  Errors as csa_decode.
 */
int csa_decode_range(const void *q, const void *k_shard, const void *v_shard, const void *k0,
                     const void *v0, const int *seqlens, float *out, float *lse, void *workspace,
                     long long workspace_bytes, int B, int H, int T, int d, float scale,
                     int k0_mode, int pos_lo, int pos_hi, csa_stream_t stream);

/* csa_decode_range_workspace_bytes - workspace bytes csa_decode_range needs
 * (host only), or -1 for a negative size, pos_hi < pos_lo or d outside
 * {64, 128, 256}. */
long long csa_decode_range_workspace_bytes(int B, int H, int pos_lo, int pos_hi, int d);

/*
 * csa_decode_merge_ranges - merges R partial results of the same rows (from
 *   csa_decode_range over ranges that partition each row's positions):
 *       o = sum_r e^{lse_r - L} o_r / sum_r e^{lse_r - L},
 *       lse = L + log sum_r e^{lse_r - L},   L = max_r lse_r;
 *   an empty range (lse_r = -inf) weighs nothing.  The pages have no
 *   counterpart: this is the one exchange step of context parallelism.
 *   o_parts: DEVICE fp32 [R, B, H, d]; lse_parts: DEVICE fp32 [R, B, H];
 *   out: DEVICE bf16 [B, H, d]; lse: DEVICE fp32 [B, H] or NULL.
 *   R >= 1, 1 <= d <= 256; CSA_ERR_INVALID_ARG otherwise.
 */
int csa_decode_merge_ranges(const float *o_parts, const float *lse_parts, int R, int B, int H,
                            int d, void *out, float *lse, csa_stream_t stream);

/*
 * Paged key-value caches
 * ----------------------
 *  Pools      k_pages, v_pages: contiguous [P, Hkv, S, d], P pages of S rows
 *             for each of Hkv cached heads (NULL allowed with P = 0).
 *  Tables     block_table: contiguous int32 [B, M]; row b holds the page
 *             numbers of sequence b in order, its token i being row i mod S
 *             of page block_table[b][i / S].  seqlens: int32 [B], tokens held.
 *             Entries behind a sequence's ceil(n / S) pages are not read.
 *  Holders    page_refs: int32 [P], how many sequences hold a page; 0 is
 *             free.  A partly filled page is held by one sequence only: the
 *             calls below keep it so.
 *  All of these are DEVICE memory and are read and written on `stream` only,
 *  so a step of a server (free, reserve, append, decode) can be captured into
 *  a graph.  Values on the device that the host cannot see (lengths, page
 *  numbers, rows) are checked on the device: what each call does with bad
 *  ones is said there, no access goes out of bounds, and the sticky status
 *  word (csa_device_status) records CSA_ERR_INVALID_ARG.
 *  S, M >= 1; B * M at most 2^31 - 1 and M * S at most 2^31 - 16
 *  (CSA_ERR_UNSUPPORTED).  The pages of the method have no counterpart to any of these entry points but
 *  csa_decode_paged.
 */

/*
 * Elements of a pool.  Pools of 8 bits have row_scales: contiguous float
 *  [P, Hkv, S, 2], the scale of each row of k_pages and of v_pages; a row stands
 *  for code * scale.  row_scales is NULL for the other pools.
 */
enum {
    CSA_BF16 = 0,
    CSA_F32 = 1,
    CSA_E4M3 = 2, /* 8-bit floats of 3 fraction bits, largest 448             */
    CSA_INT8 = 3
};

/*
 * csa_decode_paged - csa_decode over a paged cache, with grouped heads: query
 *   head h reads cached head h / (Hq / Hkv).
 *   Defines: eq. (10)/(11) of "Continuous Softmax Attention" ("Assembly and
 *   Simplification") for the single row t = n_b, as csa_decode.
 *   q: bf16 [B, Hq, d]; k_pages, v_pages: bf16 [P, Hkv, S, d]; k0, v0: bf16
 *   [Hkv, d], read in CSA_K0_GIVEN mode only (CSA_K0_COPY_FIRST: token 0 of
 *   the cache); out: bf16 [B, Hq, d]; lse: float [B, Hq] or NULL.
 *   seqlens: int32 [B], the tokens held, the newest one among them.  n_b = 0
 *   is an empty place in the batch: out = 0 and lse = -inf.  A length outside
 *   [0, M * S], or a page number outside [0, P) among the ones held, makes
 *   that sequence's out and lse NaN and sets the status word; other
 *   sequences are not affected.
 *   workspace: DEVICE scratch of at least csa_decode_paged_workspace_bytes(B,
 *   Hq, Hkv, d) bytes, 16-byte aligned, contents on entry irrelevant; calls
 *   that can run at the same time need distinct workspaces.
 *   d must be 64, 128 or 256 and S a multiple of 8 (CSA_ERR_UNSUPPORTED
 *   otherwise, as for P * Hkv * S > 2^31 - 1); Hq a multiple of Hkv
 *   (CSA_ERR_INVALID_ARG).  q, pools, out, workspace (and k0, v0 in GIVEN
 *   mode) 16-byte aligned, the rest 4-byte.  B * Hq == 0: CSA_OK, nothing
 *   launched.  Equal inputs give equal bits, whatever the scheduling; how a
 *   sequence is cut into parts goes by all lengths of the batch, so its last
 *   bits may change with the lengths of the others.
 */
int csa_decode_paged(const void *q, const void *k_pages, const void *v_pages, const void *k0,
                     const void *v0, const int *block_table, const int *seqlens, void *out,
                     float *lse, void *workspace, long long workspace_bytes, int B, int Hq,
                     int Hkv, int P, int S, int M, int d, float scale, int k0_mode,
                     csa_stream_t stream);

/*
 * csa_decode_paged_q8 - csa_decode_paged over pools of 8 bits (kind CSA_E4M3 or
 *   CSA_INT8), whose rows stand for code * scale; q, k0, v0 and out as there.
 *   row_scales 16-byte aligned; M * S at most 2^31 - 32.  A row whose scale is NaN
 *   makes what attends to it NaN.  Logits are formed from the codes in fp32, the
 *   weights times the values' scales are fp16 numbers (with up to 8 query heads per
 *   cached head, or per block of them, sums of two), the sums fp32.  The unit of those
 *   numbers follows a head's largest product of a logit's exponential and the scale of
 *   its row's value or a neighbour's, so that they keep their 11 bits down to 2^-8 of it,
 *   whatever the scales, and are off by 2^-19 of it below.  Everything else as
 *   csa_decode_paged, the workspace too.
 */
int csa_decode_paged_q8(const void *q, const void *k_pages, const void *v_pages,
                        const float *row_scales, const void *k0, const void *v0,
                        const int *block_table, const int *seqlens, void *out, float *lse,
                        void *workspace, long long workspace_bytes, int B, int Hq, int Hkv, int P,
                        int S, int M, int d, float scale, int k0_mode, int kind,
                        csa_stream_t stream);

/* csa_decode_paged_workspace_bytes - workspace bytes csa_decode_paged needs
 * (host only), or -1 for a negative size, Hkv that does not divide Hq, or d
 * outside {64, 128, 256}. */
long long csa_decode_paged_workspace_bytes(int B, int Hq, int Hkv, int d);

/*
 * csa_decode_tree - the attention of drafted tokens that the cache already holds:
 *   the last counts[b] of sequence b's seqlens[b] tokens are nodes of a tree (or of
 *   several, one after the other), node t at place n + t, n = seqlens[b] - counts[b].
 *   Node t's row attends to the sink, the n tokens before the draft and the nodes on
 *   the path from a root to t, in that order.
 *   Defines: eq. (10)/(11) of "Continuous Softmax Attention" ("Assembly and
 *   Simplification") for the last row of that list; with a chain (parents NULL) row t
 *   is csa_decode_paged's of the first n + t + 1 tokens.
 *   q: bf16 [B, Hq, T, d], the nodes' queries; out: bf16 [B, Hq, T, d]; lse: float
 *   [B, Hq, T] or NULL.  parents: int32 [B, T], the parent of node t < counts[b],
 *   -1 (it follows the tokens before the draft) or a node below t; NULL: t - 1 each.
 *   counts: int32 [B], 0 <= counts[b] <= min(T, seqlens[b]); NULL: T each.  Rows
 *   t >= counts[b] get out = 0 and lse = -inf; their q and parents do not matter.  Of a
 *   sequence with counts[b] = 0 no page is read.
 *   n = 0: the sink is followed by a root (CSA_K0_COPY_FIRST: a copy of the row's own
 *   root).  Pools, row_scales, k0, v0, block_table, scale and k0_mode as
 *   csa_decode_paged (kind CSA_BF16, row_scales NULL) and csa_decode_paged_q8.
 *   A count or length out of range, or a page number outside [0, P) among the ones
 *   held, makes that sequence's out and lse NaN; a parent out of range those of the
 *   nodes that have it on their path; both set the status word.
 *   T at most CSA_TREE_MAX and M * S at most 2^31 - 256 (CSA_ERR_UNSUPPORTED).  workspace: at least
 *   csa_decode_tree_workspace_bytes(B, Hq, Hkv, T, d) bytes, 16-byte aligned, contents
 *   on entry irrelevant; calls that can run at the same time need distinct ones.
 *   Alignment, other refusals, and what decides the last bits as csa_decode_paged.
 *   Weights over bf16 pools are sums of two bf16 numbers; over 8-bit ones, with more
 *   than 8 rows per cached head (T times the query heads on it), one fp16 number, its
 *   unit as in csa_decode_paged_q8 (with more than 16 rows for values' scales that lie
 *   within 2^80 of one another).
 *   With more than 16 rows per cached head the interval between two neighbours is divided
 *   between them within 2.2e-4 of the share (else within 2^-16), its whole within 2^-16.8.
 */
#define CSA_TREE_MAX 64
int csa_decode_tree(const void *q, const void *k_pages, const void *v_pages,
                    const float *row_scales, const void *k0, const void *v0,
                    const int *block_table, const int *seqlens, const int *parents,
                    const int *counts, void *out, float *lse, void *workspace,
                    long long workspace_bytes, int B, int Hq, int Hkv, int T, int P, int S, int M,
                    int d, float scale, int k0_mode, int kind, csa_stream_t stream);

/* csa_decode_tree_workspace_bytes - workspace bytes csa_decode_tree needs (host only),
 * or -1 for a negative size, T above CSA_TREE_MAX, Hkv that does not divide Hq, or d
 * outside {64, 128, 256}. */
long long csa_decode_tree_workspace_bytes(int B, int Hq, int Hkv, int T, int d);

/*
 * csa_rope_plan - which pairs of a row turn, by which axis of the positions
 *   and how far per position; filled by csa_rope_plan_init and passed by
 *   value into the kernels (HOST memory, not kept).
 */
#define CSA_ROPE_MAX_PAIRS 128
#define CSA_ROPE_MAX_AXES 8
#define CSA_ROPE_ADJACENT 1 /* pairs (2i, 2i + 1) instead of (i, i + n)        */
#define CSA_ROPE_DEALT 2    /* pairs dealt to the axes in turn, an axis that
                               has its number of pairs being passed over,
                               instead of section after section                */
typedef struct {
    int pairs, axes, adjacent;
    unsigned char axis[CSA_ROPE_MAX_PAIRS];      /* the axis of each pair      */
    unsigned long long turn[CSA_ROPE_MAX_PAIRS]; /* turns per position, * 2^64 */
} csa_rope_plan;

/*
 * csa_rope_plan_init - plan for rotary positions with `axes` axes (1 to 8),
 *   sections[a] pairs turning by axis a (n pairs in all, 1 <= n <= 128); pair i
 *   turns by positions[axis(i)] * base^(-i / n).  base finite and > 0 (below 1
 *   the turns per position grow, and their fraction loses as many bits); flags:
 *   CSA_ROPE_ADJACENT, CSA_ROPE_DEALT.  Host only.
 *   CSA_ERR_INVALID_ARG, or CSA_ERR_UNSUPPORTED for more than 128 pairs.
 */
int csa_rope_plan_init(csa_rope_plan *plan, const int *sections, int axes, double base, int flags);

/*
 * csa_rope - turns the first 2n columns of every row of q and k by the plan,
 *   the other columns copied: (u, w) -> (u cos - w sin, u sin + w cos) per
 *   pair, by the negative angle if `inverse` (the backward pass: the gradient
 *   of the input from the gradient of the output).  fp32 arithmetic, one
 *   rounding.  Turns per position are right within 2^-65 and, on hosts with
 *   64-bit long doubles, (ln base + 4) 2^-64 relative (base >= 1); the angle's
 *   distance to the nearest quarter of a turn is then rounded by 2^-23
 *   relative, and opposite positions turn by exactly opposite angles.
 *   q, q_out: bf16 [B, Hq, T, d]; k, k_out: bf16 [B, Hkv, T, d], not read
 *   where the head count is 0.  *_strides: HOST long long[3], the strides over
 *   batch, head and time in elements (the last dimension is contiguous); NULL
 *   for contiguous tensors.  An output may be its input with the same strides;
 *   otherwise outputs overlap neither inputs nor themselves.
 *   positions: DEVICE int32, strides pos_strides (HOST long long[3]) over axis,
 *   batch and time, NULL for contiguous [axes, B, T]; stride 0 broadcasts.
 *   1 <= d <= 256 and 2n <= d; B * T at most 2^31 - 1.  2-byte aligned; the
 *   fast path wants 16-byte alignment of every row and d and n multiples of 8.
 */
int csa_rope(const csa_rope_plan *plan, const void *q, const long long *q_strides, void *q_out,
             const long long *q_out_strides, const void *k, const long long *k_strides,
             void *k_out, const long long *k_out_strides, const int *positions,
             const long long *pos_strides, int B, int Hq, int Hkv, int T, int d, int inverse,
             csa_stream_t stream);

/* csa_rope_f32 - the same on fp32 tensors (4-byte aligned; fast path: d and n
 * multiples of 4). */
int csa_rope_f32(const csa_rope_plan *plan, const float *q, const long long *q_strides,
                 float *q_out, const long long *q_out_strides, const float *k,
                 const long long *k_strides, float *k_out, const long long *k_out_strides,
                 const int *positions, const long long *pos_strides, int B, int Hq, int Hkv, int T,
                 int d, int inverse, csa_stream_t stream);

/*
 * csa_cache_append - writes the rows of new tokens into their pages: row t of
 *   k and v (t < counts[b]) becomes token seqlens[b] - counts[b] + t of
 *   sequence b, so seqlens already counts the new tokens (csa_cache_reserve
 *   sets it).  With a plan the keys are turned on the way, and q, if given, is
 *   turned into q_out by the same positions (all T rows).
 *   k, v: bf16 [B, Hkv, T, d]; q, q_out: bf16 [B, Hq, T, d] or Hq = 0; strides
 *   as csa_rope.  counts: int32 [B], or NULL for T each.  positions, strides as
 *   csa_rope, or NULL: a token's place in the cache, on every axis.  plan NULL:
 *   nothing turns (then Hq must be 0).  Pages may have any S >= 1.
 *   A sequence whose count is outside [0, T] or whose length is outside
 *   [count, M * S], and a row whose page number is outside [0, P), is not
 *   written and sets the status word.
 */
int csa_cache_append(const csa_rope_plan *plan, const void *q, const long long *q_strides,
                     void *q_out, const long long *q_out_strides, const void *k,
                     const long long *k_strides, const void *v, const long long *v_strides,
                     void *k_pages, void *v_pages, const int *block_table, const int *seqlens,
                     const int *counts, const int *positions, const long long *pos_strides, int B,
                     int Hq, int Hkv, int T, int d, int P, int S, int M, csa_stream_t stream);

/* csa_cache_append_f32 - the same on fp32 tensors and pools, for a caller's own
 * attention: csa_decode_paged reads bf16 pools only. */
int csa_cache_append_f32(const csa_rope_plan *plan, const float *q, const long long *q_strides,
                         float *q_out, const long long *q_out_strides, const float *k,
                         const long long *k_strides, const float *v, const long long *v_strides,
                         float *k_pages, float *v_pages, const int *block_table,
                         const int *seqlens, const int *counts, const int *positions,
                         const long long *pos_strides, int B, int Hq, int Hkv, int T, int d, int P,
                         int S, int M, csa_stream_t stream);

/*
 * csa_cache_append_q8 - csa_cache_append into pools of 8 bits: the rows of the
 *   new tokens are quantised as they are written, after the keys have turned and
 *   without a rounding between.  For a row x, max the largest |x_c| (fp32):
 *     CSA_E4M3  scale = the smallest power of two with max / scale <= 448, codes
 *               the nearest e4m3 numbers to x / scale, ties to even;
 *     CSA_INT8  scale = max / 127 and codes the integers nearest to
 *               x * (127 / max), ties to even, both quotients rounded to fp32.
 *   max < 2^-100: scale 0 and codes 0.  A row with an infinity or NaN: scale NaN
 *   and codes 0, so that it reads as NaN.
 *   in_type: CSA_BF16 or CSA_F32, of q, k, v and q_out; kind: CSA_E4M3 or CSA_INT8.
 *   k_pages, v_pages: 1 byte per element; row_scales as above, 8-byte aligned.
 *   Everything else as csa_cache_append.
 */
int csa_cache_append_q8(const csa_rope_plan *plan, const void *q, const long long *q_strides,
                        void *q_out, const long long *q_out_strides, const void *k,
                        const long long *k_strides, const void *v, const long long *v_strides,
                        void *k_pages, void *v_pages, float *row_scales, const int *block_table,
                        const int *seqlens, const int *counts, const int *positions,
                        const long long *pos_strides, int B, int Hq, int Hkv, int T, int d, int P,
                        int S, int M, int in_type, int kind, csa_stream_t stream);

/*
 * csa_cache_read - rows of the cache in order: row t < T of k and v gets token
 *   starts[b] + t of sequence b, as a value of out_type (code * scale, rounded
 *   once), or 0 where the sequence has no such token.
 *   k_pages, v_pages: pools of `kind`; row_scales NULL unless kind is CSA_E4M3 or
 *   CSA_INT8; out_type: CSA_BF16 or CSA_F32 for those, else equal to kind.
 *   starts: int32 [B], or NULL for 0.  k, v: [B, Hkv, T, d], strides as csa_rope;
 *   outputs overlap neither inputs nor themselves.  Pages may have any S >= 1.
 *   1 <= d <= 256; B * Hkv * T at most 2^31 - 1.
 *   A sequence with a length outside [0, M * S] or a start outside [0, length],
 *   and a row whose page number is outside [0, P), reads as NaN and sets the
 *   status word.
 */
int csa_cache_read(const void *k_pages, const void *v_pages, const float *row_scales,
                   const int *block_table, const int *seqlens, const int *starts, void *k,
                   const long long *k_strides, void *v, const long long *v_strides, int B, int Hkv,
                   int T, int d, int P, int S, int M, int kind, int out_type, csa_stream_t stream);

/*
 * csa_cache_reserve - room for counts[b] >= 0 more tokens of every sequence:
 *   the pages that are missing are the lowest-numbered free ones, given out in
 *   the order of the sequences; their refs become 1, the table gets them, and
 *   seqlens[b] += counts[b].
 *   shortfall: DEVICE int32 [1]: 0 if it was done; the number of pages missing
 *   if the pool has too few, or -1 for a negative count or length or one that
 *   does not fit a row of the table (which also sets the status word).  Where
 *   it is not 0, nothing has changed.
 */
int csa_cache_reserve(int *page_refs, int *block_table, int *seqlens, const int *counts,
                      int *shortfall, int B, int P, int S, int M, csa_stream_t stream);

/*
 * csa_cache_free - the listed sequences give their pages back: their refs fall
 *   by one each, the entries become -1 and the lengths 0.  rows: int32 [R];
 *   -1 is padding, a row listed twice is freed once.  A row outside [-1, B),
 *   or with a length outside [0, M * S], sets the status word and nothing
 *   changes; a page number outside [0, P), or of a page that nobody holds, is
 *   passed over and sets the status word.
 */
int csa_cache_free(int *page_refs, int *block_table, int *seqlens, const int *rows, int R, int B,
                   int P, int S, int M, csa_stream_t stream);

/*
 * csa_cache_fork - children[i] becomes a copy of parents[i]: full pages are
 *   shared (refs + 1), a partly filled last page gets a page of its own, the
 *   lowest-numbered free ones in the order of the pairs.  src[i], dst[i] are
 *   the pages to copy then (csa_cache_copy_pages, once per pool), or -1, -1.
 *   parents, children: int32 [n]; a pair with a negative entry is padding.
 *   A parent may have several children; a child must be empty (length 0) and
 *   listed once.  The child's row of the table is -1 behind its pages.
 *   shortfall as csa_cache_reserve (-1: a row out of range, a bad length, a
 *   last page to copy outside [0, P), a child that is not empty or listed
 *   twice); where it is not 0, nothing has changed and src, dst are -1.  A
 *   number outside [0, P) among the shared pages is copied as it is and sets
 *   the status word.
 *   n at most CSA_CACHE_MAX_FORKS (CSA_ERR_UNSUPPORTED).
 */
#define CSA_CACHE_MAX_FORKS 4096
int csa_cache_fork(int *page_refs, int *block_table, int *seqlens, const int *parents,
                   const int *children, int n, int *src, int *dst, int *shortfall, int B, int P,
                   int S, int M, csa_stream_t stream);

/*
 * csa_cache_compact - moves the held pages together: with U pages held, those
 *   numbered U or more take the free numbers below U, both in ascending order.
 *   src, dst: int32 [P / 2], the moves, then -1; moved: int32 [1], how many.
 *   page_refs and the held entries of the table are already renamed; the
 *   caller moves the data (csa_cache_copy_pages with count = moved, once per
 *   pool) before anything reads the pools.
 */
int csa_cache_compact(int *page_refs, int *block_table, const int *seqlens, int *src, int *dst,
                      int *moved, int B, int P, int S, int M, csa_stream_t stream);

/*
 * csa_cache_copy_pages - copies page src[i] onto page dst[i] for i < min(n,
 *   *count) (count: DEVICE int32 [1], or NULL for n), in k_pages and, unless
 *   it is NULL, v_pages: pools of `layers` times P pages of page_bytes bytes.
 *   A pair with a negative entry is padding; one with a number >= P is passed
 *   over and sets the status word.  Pairs are copied in no particular order:
 *   a page that is a dst must not be the src or dst of another pair.
 */
int csa_cache_copy_pages(void *k_pages, void *v_pages, long long page_bytes, int layers, int P,
                         const int *src, const int *dst, int n, const int *count,
                         csa_stream_t stream);

/*
 * csa_cache_accept - keeps the accepted branch of a tree of drafted tokens (the
 *   last counts[b] tokens of sequence b, csa_decode_tree) and gives the others up:
 *   with n tokens before the draft and m nodes on the path from a root to node
 *   last[b], the sequence holds n + m tokens afterwards, the path's in order; pages
 *   behind them are given back (refs fall by one, entries become -1).
 *   parents: int32 [B, T] as csa_decode_tree, or NULL for a chain; counts: int32 [B],
 *   or NULL for T each; last: int32 [B], the last accepted node, -1 for none.
 *   src, dst: int32 [B, T], the rows to move: entry i < m has the pool's rows
 *   (page * S + slot) where the path's i-th token is and where it goes, or -1, -1
 *   where it is there already; -1 behind.  The caller moves the data
 *   (csa_cache_copy_rows, once per pool) before anything reads the pools or takes
 *   pages.  A sequence must not be forked between its draft and this call.
 *   A count outside [0, T], a length outside [count, M * S], a last node outside
 *   [-1, count), a parent on the path outside [-1, node) or a page number outside
 *   [0, P) of a row to move leaves that sequence as it is (src, dst -1) and sets the
 *   status word; a page to give back that is outside [0, P) or held by nobody is
 *   passed over and sets it.
 *   T at most CSA_TREE_MAX and P * S at most 2^31 - 1 (CSA_ERR_UNSUPPORTED).
 */
int csa_cache_accept(int *page_refs, int *block_table, int *seqlens, const int *parents,
                     const int *counts, const int *last, int *src, int *dst, int T, int B, int P,
                     int S, int M, csa_stream_t stream);

/*
 * csa_cache_copy_rows - copies row src[g][i] of every head onto row dst[g][i] in
 *   k_pages and, unless they are NULL, v_pages and row_scales (any of the three may
 *   be NULL): pools of `layers` times [P, H, S] rows of row_bytes bytes
 *   (scale_bytes for row_scales).  src, dst: int32 [groups, T], rows page * S +
 *   slot; a pair with a negative entry is padding, one with a row >= P * S is
 *   passed over and sets the status word.  All rows of a group are read before any
 *   is written; a row that is a dst must not be in another group, nor a dst twice.
 *   T at most CSA_TREE_MAX; layers and 3 * H at most 65535 (CSA_ERR_UNSUPPORTED).
 */
int csa_cache_copy_rows(void *k_pages, void *v_pages, long long row_bytes, void *row_scales,
                        long long scale_bytes, int layers, int P, int H, int S, const int *src,
                        const int *dst, int groups, int T, csa_stream_t stream);

/*
 * csa_logphi2_eval - y[i] = log phi2(x[i]) with the library's fp32 device
 *   function (phi2 of eq. (6), "Preliminaries").  x, y: device float arrays
 *   of n elements (n >= 0).  A test hook for the numerics of b.
 */
int csa_logphi2_eval(const float *x, float *y, int n, csa_stream_t stream);

/*
 * csa_segment_weights_eval - the tensor-core kernel's fp32 evaluation of
 *   one interval's two end weights, for tests.  For each i, with
 *   x = u1[i] - u0[i] in natural-log units and p = e^{u}:
 *       right[i] = p0 * phi2(x)    (the share of interval (u0,u1) that eq. (9)
 *       left[i]  = p1 * phi2(-x)    moves onto its left and right key)
 *   u0, u1: device float arrays (u <= 0 expected, as after subtracting a
 *   running max); right, left: device float outputs; n >= 0.
 */
int csa_segment_weights_eval(const float *u0, const float *u1, float *right, float *left, int n,
                             csa_stream_t stream);

/*
 * csa_device_status - reads and clears the library's sticky device status
 *   words of the current device: CSA_OK; CSA_ERR_TIMEOUT if a kernel's
 *   bounded wait expired since the last read (that kernel then skipped the
 *   rest of its work and its outputs are undefined); CSA_ERR_INVALID_ARG if
 *   csa_decode met a sequence length outside [1, T], or one of the paged
 *   cache's calls a length, row or page number out of range.  Synchronises
 *   the device.  Returns CSA_ERR_CUDA if the read itself fails.
 */
int csa_device_status(void);

/*
 * csa_selftest_wait_timeout - launches one block whose thread waits on an
 *   mbarrier that nothing ever completes, with a time limit of timeout_us
 *   microseconds (1..10^6).  The wait gives up, the kernel records
 *   CSA_ERR_TIMEOUT in the status word and returns normally; the context
 *   stays usable.  Exercises the bounded-wait path of the kernels without
 *   any fault.
 */
int csa_selftest_wait_timeout(unsigned timeout_us, csa_stream_t stream);

/*
 * csa_selftest_forward_delay - csa_forward's exact form (the tensor-core
 *   kernel, bf16, d in {64, 128}; arguments, layout, ownership and checks as
 *   csa_forward) with a delay planted in every epilogue: the softmax threads
 *   of column half delay_half (0 or 1) sleep delay_ns nanoseconds (at most
 *   10^6) after the item's last PV product is done and before they read the
 *   two accumulators O_0 and O_1.  Meanwhile the other half's threads run
 *   ahead into the CTA's next query tile, whose first PV product overwrites
 *   O_0 and O_1 ("Assembly and Simplification", eq. (10): the numerator and
 *   denominator sums per query row).  The kernel orders that product after
 *   every thread's reads, so the output and lse must equal csa_forward's bit
 *   for bit whatever the delay.  CSA_ERR_INVALID_ARG for a delay or half out
 *   of range.  A test hook: it only slows the kernel down.
 */
int csa_selftest_forward_delay(const void *q, const void *k, const void *v, const void *k0,
                               const void *v0, void *out, float *lse, int B, int H, int T, int d,
                               float scale, int k0_mode, unsigned delay_ns, int delay_half,
                               csa_stream_t stream);

/* Human-readable text for a status code (never NULL, static storage). */
const char *csa_status_string(int status);

/* ABI version of this header (bumped on incompatible change). */
int csa_abi_version(void);
#define CSA_ABI_VERSION 1

#ifdef __cplusplus
}
#endif
#endif /* CSA_H_ */

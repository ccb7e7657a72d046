// The decode step over a paged cache of bf16 rows: the kernels of csa_paged.cuh.
#include "csa_paged.cuh"

long long csa_decode_paged_scratch_bytes(int B, int Hq, int Hkv, int d) {
    if (B < 0 || Hq < 0 || Hkv < 1 || Hq % Hkv != 0 || !(d == 64 || d == 128 || d == 256)) return -1;
    const int G = Hq / Hkv;
    const int GB = head_blocks(G), HB = GB ? (G + GB - 1) / GB : 0;
    return workers(d) * (2 * HB * (d + 2) * (long long)sizeof(float) + (long long)sizeof(int4));
}

int csa_decode_paged_run(const csa_paged_args &a, void *scratch, int d, cudaStream_t stream) {
    PagedParams p = paged_params(a);
    return run_paged<CSA_BF16>(p, scratch, d, stream);
}

int *csa_paged_status_word(void) { return status_word(); }

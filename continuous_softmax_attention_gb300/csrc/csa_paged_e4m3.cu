// The decode step over a paged cache of e4m3 rows: the kernels of csa_paged.cuh.
#include "csa_paged.cuh"

int csa_decode_paged_e4m3_run(const csa_paged_args &a, void *scratch, int d, cudaStream_t stream) {
    PagedParams p = paged_params(a);
    return run_paged<CSA_E4M3>(p, scratch, d, stream);
}

int *csa_paged_e4m3_status_word(void) { return status_word(); }

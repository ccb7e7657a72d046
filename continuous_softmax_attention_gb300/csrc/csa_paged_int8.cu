// The decode step over a paged cache of int8 rows: the kernels of csa_paged.cuh.
#include "csa_paged.cuh"

int csa_decode_paged_int8_run(const csa_paged_args &a, void *scratch, int d, cudaStream_t stream) {
    PagedParams p = paged_params(a);
    return run_paged<CSA_INT8>(p, scratch, d, stream);
}

int *csa_paged_int8_status_word(void) { return status_word(); }

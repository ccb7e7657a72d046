// Many rows over a paged cache of int8 rows: the kernel of csa_rows.cuh.
#include "csa_rows.cuh"

int csa_rows_int8_run(const csa_paged_args &a, void *scratch, int d, cudaStream_t stream) {
    return run_rows<CSA_INT8>(a, scratch, d, stream);
}

int *csa_rows_int8_status_word(void) { return status_word(); }

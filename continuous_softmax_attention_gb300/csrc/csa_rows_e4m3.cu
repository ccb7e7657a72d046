// Many rows over a paged cache of e4m3 rows: the kernel of csa_rows.cuh.
#include "csa_rows.cuh"

int csa_rows_e4m3_run(const csa_paged_args &a, void *scratch, int d, cudaStream_t stream) {
    return run_rows<CSA_E4M3>(a, scratch, d, stream);
}

int *csa_rows_e4m3_status_word(void) { return status_word(); }

// Many rows over a paged cache of bf16 rows: the kernel of csa_rows.cuh.
#include "csa_rows.cuh"

int csa_rows_bf16_run(const csa_paged_args &a, void *scratch, int d, cudaStream_t stream) {
    return run_rows<CSA_BF16>(a, scratch, d, stream);
}

int *csa_rows_bf16_status_word(void) { return status_word(); }

// Pages of a key-value cache: which are free, which sequences hold them, and
// the movement of whole pages.
//
// State, all of it int32 device memory of the caller: refs[P], how many
// sequences hold a page (0: free); table[B][M], the pages of each sequence in
// order; seqlens[B].  A sequence of n tokens holds ceil(n / S) pages, and the
// page it is writing to (n not a multiple of S) is held by no other sequence.
// Pages are given out lowest number first, in the order of the sequences and
// of each sequence's pages, so every result is a function of the state alone.
//
// What bounds it.  The bookkeeping reads refs once (4 bytes a page) and is
// bound by latency: one block keeps the order by a scan over the whole pool
// without any exchange between blocks.  The copies are bound by HBM bandwidth.
#include <cuda_runtime.h>

#include <cstdint>

#include "csa.h"
#include "csa_internal.h"

namespace {

constexpr int kBookThreads = 1024;
constexpr int kBookWarps = kBookThreads / 32;
constexpr int kSub = 8;  // pages per thread and step of a walk over refs

__device__ int g_cache_status;  // sticky status word of this file's kernels

__device__ __forceinline__ void complain() { atomicCAS(&g_cache_status, 0, CSA_ERR_INVALID_ARG); }

// Exclusive prefix sum over the block's threads; *total gets the block's sum.
__device__ __forceinline__ int block_scan(int v, int *warp_sums, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += o;
    }
    __syncthreads();  // warp_sums may still be read from an earlier scan
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    const int w = lane < (int)(blockDim.x >> 5) ? warp_sums[lane] : 0;
    int ws = w;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, ws, off);
        if (lane >= off) ws += o;
    }
    *total = __shfl_sync(0xffffffffu, ws, 31);
    const int before = __shfl_sync(0xffffffffu, ws - w, warp);
    return before + s - v;
}

// Walks over the pages [lo, hi) in ascending order, calling hit(page, rank)
// for those of which pick(refs[page], page) holds; ranks count from 0.  Stops
// once `most` have been found.  Returns how many were found (at least `most`
// if it stopped early).  Called by the whole block.
template <typename Pick, typename Hit>
__device__ int walk(const int *refs, int lo, int hi, int most, int *warp_sums, Pick pick, Hit hit) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int found = 0;
    for (long long base = lo; base < hi && found < most; base += kBookThreads * kSub) {
        // a warp takes 32 * kSub consecutive pages, 32 at a time
        const long long first = base + (long long)warp * (32 * kSub) + lane;
        int val[kSub];
#pragma unroll
        for (int i = 0; i < kSub; ++i) val[i] = first + 32 * i < hi ? refs[first + 32 * i] : 0;
        unsigned mask[kSub];
        int mine = 0;  // of the whole warp
#pragma unroll
        for (int i = 0; i < kSub; ++i) {
            const long long page = first + 32 * i;
            mask[i] = __ballot_sync(0xffffffffu, page < hi && pick(val[i], (int)page));
            mine += __popc(mask[i]);
        }
        int total;
        // one count per warp, on its first lane
        int rank = found + __shfl_sync(0xffffffffu, block_scan(lane == 0 ? mine : 0, warp_sums, &total), 0);
#pragma unroll
        for (int i = 0; i < kSub; ++i) {
            if (mask[i] >> lane & 1)
                hit((int)(first + 32 * i), rank + __popc(mask[i] & ((1u << lane) - 1)));
            rank += __popc(mask[i]);
        }
        found += total;
    }
    return found;
}

__device__ __forceinline__ int pages_of(int n, int S) { return (int)(((long long)n + S - 1) / S); }

// ------------------------------------------------------------------ reserve
// list: [P] ints, prefix: [B] ints of the workspace.
__global__ void __launch_bounds__(kBookThreads)
reserve_kernel(int *refs, int *table, int *seqlens, const int *counts, int *shortfall, int B, int P,
               int S, int M, int *list, int *prefix) {
    __shared__ int warp_sums[32];
    const int tid = threadIdx.x, per = (B + kBookThreads - 1) / kBookThreads;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    long long need = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
        const int n = seqlens[b], c = counts[b];
        if (n < 0 || c < 0 || (long long)n + c > (long long)M * S) {
            bad = true;
            break;
        }
        need += pages_of(n + c, S) - pages_of(n, S);
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) {
            *shortfall = -1;
            complain();
        }
        return;
    }
    int wanted;  // at most B * M, which fits an int
    int at = block_scan((int)need, warp_sums, &wanted);
    for (int b = b0; b < b1; ++b) {
        prefix[b] = at;
        at += pages_of(seqlens[b] + counts[b], S) - pages_of(seqlens[b], S);
    }
    const int found = walk(refs, 0, P, wanted, warp_sums, [](int v, int) { return v == 0; },
                           [&](int page, int rank) { list[rank] = page; });
    if (found < wanted) {
        if (tid == 0) *shortfall = wanted - found;
        return;
    }
    __syncthreads();  // list and prefix complete
    for (int i = tid; i < wanted; i += kBookThreads) {
        int lo = 0, hi = B - 1;  // the last b with prefix[b] <= i
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (prefix[mid] <= i)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int page = list[i];
        table[(long long)lo * M + pages_of(seqlens[lo], S) + i - prefix[lo]] = page;
        refs[page] = 1;
    }
    __syncthreads();  // the old lengths have been read
    for (int b = b0; b < b1; ++b) seqlens[b] += counts[b];
    if (tid == 0) *shortfall = 0;
}

// --------------------------------------------------------------------- free
// One block per listed row.  A call with a row that does not exist, or whose
// length does not fit the table, changes nothing: every block looks at all
// rows first (a length that another block has already set to 0 is sound).
__global__ void __launch_bounds__(256)
free_kernel(int *refs, int *table, int *seqlens, const int *rows, int R, int B, int P, int S, int M) {
    const int me = blockIdx.x, row = rows[me];
    bool bad = false, earlier = false;
    for (int i = threadIdx.x; i < R; i += blockDim.x) {
        const int r = rows[i];
        if (r >= B || r < -1) {
            bad = true;
        } else if (r >= 0) {
            const int n = *(volatile int *)(seqlens + r);
            bad |= n < 0 || n > (long long)M * S;
            earlier |= i < me && r == row;
        }
    }
    bad = __syncthreads_or(bad);
    earlier = __syncthreads_or(earlier);
    if (bad) {
        if (threadIdx.x == 0 && me == 0) complain();
        return;
    }
    if (row < 0 || earlier) return;  // padding, or listed before
    const int held = pages_of(seqlens[row], S);
    for (int j = threadIdx.x; j < held; j += blockDim.x) {
        int *entry = table + (long long)row * M + j;
        const int page = *entry;
        *entry = -1;
        if (page < 0 || page >= P) {
            complain();
        } else if (atomicSub(refs + page, 1) <= 0) {  // held by nobody: left at what it was
            atomicAdd(refs + page, 1);
            complain();
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) seqlens[row] = 0;
}

// --------------------------------------------------------------------- fork
// Checks every pair, takes a page for each child whose parent's last page is
// partly filled, and notes the lengths; all or nothing.  mark: [B] ints, lens:
// [n] ints (-1: nothing to do), list: [P] ints of the workspace.
__global__ void __launch_bounds__(kBookThreads)
fork_plan_kernel(int *refs, const int *table, const int *seqlens, const int *parents,
                 const int *children, int n, int *src, int *dst, int *shortfall, int B, int P, int S,
                 int M, int *mark, int *lens, int *list) {
    __shared__ int warp_sums[32];
    const int tid = threadIdx.x, per = (n + kBookThreads - 1) / kBookThreads;
    for (int b = tid; b < B; b += kBookThreads) mark[b] = 0;
    __syncthreads();
    const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
    bool bad = false;
    int need = 0;
    for (int i = i0; i < i1; ++i) {
        const int p = parents[i], c = children[i];
        lens[i] = -1;
        src[i] = dst[i] = -1;
        if (p < 0 || c < 0) continue;  // padding
        if (p >= B || c >= B) {
            bad = true;
            continue;
        }
        const int len = seqlens[p];
        bad |= len < 0 || len > (long long)M * S || seqlens[c] != 0 || atomicAdd(mark + c, 1) != 0;
        lens[i] = len;
        if (!bad && len % S != 0) {
            const int page = table[(long long)p * M + len / S];
            bad |= page < 0 || page >= P;
            src[i] = page;
            ++need;
        }
    }
    if (__syncthreads_or(bad)) {
        for (int i = i0; i < i1; ++i) {
            lens[i] = -1;
            src[i] = -1;
        }
        if (tid == 0) {
            *shortfall = -1;
            complain();
        }
        return;
    }
    int wanted;
    int at = block_scan(need, warp_sums, &wanted);
    const int found = walk(refs, 0, P, wanted, warp_sums, [](int v, int) { return v == 0; },
                           [&](int page, int rank) { list[rank] = page; });
    const bool enough = found >= wanted;
    __syncthreads();
    for (int i = i0; i < i1; ++i) {
        if (!enough) {
            lens[i] = -1;
            src[i] = -1;
        } else if (src[i] >= 0) {
            dst[i] = list[at++];
            refs[dst[i]] = 1;
        }
    }
    if (tid == 0) *shortfall = enough ? 0 : wanted - found;
}

// One block per pair: the child's row of the table, its length, and one more
// holder for each page that it shares.
__global__ void __launch_bounds__(256)
fork_rows_kernel(int *refs, int *table, int *seqlens, const int *parents, const int *children,
                 const int *dst, const int *lens, int P, int S, int M) {
    const int i = blockIdx.x, len = lens[i];
    if (len < 0) return;
    const int p = parents[i], c = children[i], whole = len / S;
    for (int j = threadIdx.x; j < M; j += blockDim.x) {
        int page = -1;
        if (j < whole) {
            page = table[(long long)p * M + j];
            if (page >= 0 && page < P)
                atomicAdd(refs + page, 1);
            else
                complain();
        } else if (j == whole) {
            page = dst[i];  // -1 where the last page is full
        }
        table[(long long)c * M + j] = page;
    }
    if (threadIdx.x == 0) seqlens[c] = len;
}

// ------------------------------------------------------------------ compact
// The used pages [U, P) go to the free pages [0, U), both in ascending order;
// U is the number of used pages.  src, dst: [P / 2]; moved: [1]; map: [P] ints
// of the workspace, of which [U, P) is written; used: [1].
__global__ void __launch_bounds__(kBookThreads)
compact_plan_kernel(int *refs, int P, int *src, int *dst, int *moved, int *map, int *used) {
    __shared__ int warp_sums[32];
    const int tid = threadIdx.x;
    const int U = walk(refs, 0, P, 0x7fffffff, warp_sums, [](int v, int) { return v > 0; },
                       [](int, int) {});
    const int K = walk(refs, U, P, 0x7fffffff, warp_sums, [](int v, int) { return v > 0; },
                       [&](int page, int rank) { src[rank] = page; });
    walk(refs, 0, U, K, warp_sums, [](int v, int) { return v <= 0; },
         [&](int page, int rank) { dst[rank] = page; });
    for (int p = U + tid; p < P; p += kBookThreads) map[p] = p;
    __syncthreads();
    for (int i = tid; i < K; i += kBookThreads) {
        const int s = src[i], d = dst[i];
        map[s] = d;
        refs[d] = refs[s];
        refs[s] = 0;
    }
    for (int i = K + tid; i < P / 2; i += kBookThreads) src[i] = dst[i] = -1;
    if (tid == 0) {
        *moved = K;
        *used = U;
    }
}

// The table's entries by the map, every row's held pages.
__global__ void __launch_bounds__(256)
remap_kernel(int *table, const int *seqlens, const int *map, const int *used, int B, int P, int S,
             int M) {
    const int U = *used;
    for (int b = blockIdx.x; b < B; b += gridDim.x) {
        const int n = seqlens[b];
        if (n < 0 || n > (long long)M * S) {
            if (threadIdx.x == 0) complain();
            continue;
        }
        const int held = pages_of(n, S);
        for (int j = threadIdx.x; j < held; j += blockDim.x) {
            const int page = table[(long long)b * M + j];
            if (page >= U && page < P) table[(long long)b * M + j] = map[page];
        }
    }
}

// --------------------------------------------------------------------- copy
// Items are (pair, layer, pool, part of a page); a block takes every
// gridDim.x-th.  C: the widest type that the pages allow.
constexpr int kCopyThreads = 256;
constexpr int kCopyDeep = 4;

template <typename C>
__global__ void __launch_bounds__(kCopyThreads)
copy_pages_kernel(C *k_pages, C *v_pages, long long page, int layers, int P, const int *src,
                  const int *dst, int n, const int *count, int parts) {
    if (count) n = min(n, *count);
    const int pools = v_pages ? 2 : 1;
    const long long per_pair = (long long)layers * pools * parts, items = n * per_pair;
    for (long long item = blockIdx.x; item < items; item += gridDim.x) {
        const int i = (int)(item / per_pair), rest = (int)(item - i * per_pair);
        const int s = src[i], d = dst[i];
        if (s < 0 || d < 0) continue;  // padding
        if (s >= P || d >= P) {
            if (threadIdx.x == 0) complain();
            continue;
        }
        const int which = rest / parts, part = rest - which * parts;  // layer * pools + pool
        const int layer = which / pools;
        C *pool = which - layer * pools ? v_pages : k_pages;
        const C *from = pool + ((long long)layer * P + s) * page;
        C *to = pool + ((long long)layer * P + d) * page;
        const long long lo = (long long)part * kCopyThreads * kCopyDeep + threadIdx.x;
        C val[kCopyDeep];
#pragma unroll
        for (int j = 0; j < kCopyDeep; ++j)
            if (lo + j * kCopyThreads < page) val[j] = from[lo + j * kCopyThreads];
#pragma unroll
        for (int j = 0; j < kCopyDeep; ++j)
            if (lo + j * kCopyThreads < page) to[lo + j * kCopyThreads] = val[j];
    }
}

template <typename C>
int copy_as(void *k, void *v, long long page_bytes, int layers, int P, const int *src,
            const int *dst, int n, const int *count, cudaStream_t stream) {
    const long long page = page_bytes / (long long)sizeof(C);
    const long long part = kCopyThreads * kCopyDeep, parts = (page + part - 1) / part;
    if (parts * layers * 2 > 0x7fffffffLL) return CSA_ERR_UNSUPPORTED;
    const long long items = parts * layers * (v ? 2 : 1) * n;
    const unsigned grid = (unsigned)(items < 152 * 8 ? items : 152 * 8);
    copy_pages_kernel<C><<<grid, kCopyThreads, 0, stream>>>(
        static_cast<C *>(k), static_cast<C *>(v), page, layers, P, src, dst, n, count, (int)parts);
    return cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

int launched() { return cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA; }

}  // namespace

// Workspace: list or map [P], then a table of rows [B] and one of pairs [n],
// then the used count.
long long csa_cache_scratch_bytes(int B, int P, int n) {
    if (B < 0 || P < 0 || n < 0) return -1;
    return 4LL * ((long long)P + B + n + 4);
}

int csa_cache_reserve_run(int *refs, int *table, int *seqlens, const int *counts, int *shortfall,
                          void *scratch, int B, int P, int S, int M, cudaStream_t stream) {
    int *list = static_cast<int *>(scratch);
    reserve_kernel<<<1, kBookThreads, 0, stream>>>(refs, table, seqlens, counts, shortfall, B, P, S,
                                                   M, list, list + P);
    return launched();
}

int csa_cache_free_run(int *refs, int *table, int *seqlens, const int *rows, int R, int B, int P,
                       int S, int M, cudaStream_t stream) {
    free_kernel<<<R, 256, 0, stream>>>(refs, table, seqlens, rows, R, B, P, S, M);
    return launched();
}

int csa_cache_fork_run(int *refs, int *table, int *seqlens, const int *parents, const int *children,
                       int n, int *src, int *dst, int *shortfall, void *scratch, int B, int P,
                       int S, int M, cudaStream_t stream) {
    int *list = static_cast<int *>(scratch), *mark = list + P, *lens = mark + B;
    fork_plan_kernel<<<1, kBookThreads, 0, stream>>>(refs, table, seqlens, parents, children, n, src,
                                                     dst, shortfall, B, P, S, M, mark, lens, list);
    if (launched() != CSA_OK) return CSA_ERR_CUDA;
    if (n == 0) return CSA_OK;
    fork_rows_kernel<<<n, 256, 0, stream>>>(refs, table, seqlens, parents, children, dst, lens, P, S,
                                            M);
    return launched();
}

int csa_cache_compact_run(int *refs, int *table, const int *seqlens, int *src, int *dst, int *moved,
                          void *scratch, int B, int P, int S, int M, cudaStream_t stream) {
    int *map = static_cast<int *>(scratch), *used = map + P;
    compact_plan_kernel<<<1, kBookThreads, 0, stream>>>(refs, P, src, dst, moved, map, used);
    if (launched() != CSA_OK) return CSA_ERR_CUDA;
    if (B > 0 && M > 0)
        remap_kernel<<<B < 152 * 8 ? B : 152 * 8, 256, 0, stream>>>(table, seqlens, map, used, B, P,
                                                                    S, M);
    return launched();
}

int csa_cache_copy_pages_run(void *k_pages, void *v_pages, long long page_bytes, int layers, int P,
                             const int *src, const int *dst, int n, const int *count,
                             cudaStream_t stream) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(k_pages) | reinterpret_cast<uintptr_t>(v_pages) |
                         (uintptr_t)page_bytes;
    if (at % 16 == 0)
        return copy_as<uint4>(k_pages, v_pages, page_bytes, layers, P, src, dst, n, count, stream);
    if (at % 4 == 0)
        return copy_as<uint32_t>(k_pages, v_pages, page_bytes, layers, P, src, dst, n, count, stream);
    return copy_as<uint8_t>(k_pages, v_pages, page_bytes, layers, P, src, dst, n, count, stream);
}

int csa_cache_take_status(void) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_cache_status, sizeof(int)) != cudaSuccess) return CSA_ERR_CUDA;
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_cache_status, &zero, sizeof(int)) != cudaSuccess) return CSA_ERR_CUDA;
    return v;
}

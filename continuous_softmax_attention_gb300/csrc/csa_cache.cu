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

#include <algorithm>
#include <cstdint>

#include "csa.h"
#include "csa_internal.h"
#include "csa_launch.cuh"

namespace {

using namespace csa_dev;

constexpr int kBookThreads = 1024;
constexpr int kBookWarps = kBookThreads / 32;
constexpr int kSub = 16;       // pages per thread and step of a walk over refs
constexpr int kList = 4096;    // pages that a block keeps in shared memory
// Entries of the table up to which the block that plans a fork or a compaction
// also writes them; above, a second kernel does.  A fork of 4096 entries takes
// 8.2 us on the device (14.3 us a call) in one launch and 7.7 us (16.6 us) in
// two, one of 16384 entries 14.2 us (18.4 us) and 10.5 us (16.5 us).
constexpr long long kOneBlock = 4096;

__device__ int g_cache_status;  // sticky status word of this file's kernels

__device__ __forceinline__ void complain() { atomicCAS(&g_cache_status, 0, CSA_ERR_INVALID_ARG); }

// Exclusive prefix sum over the block's kBookWarps warps of one value per warp;
// *total gets the sum.
__device__ __forceinline__ int warps_scan(int v, int *sums, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();  // sums may still be read from an earlier scan
    if (lane == 0) sums[warp] = v;
    __syncthreads();
    const int w = sums[lane];
    int s = w;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += o;
    }
    *total = __shfl_sync(0xffffffffu, s, 31);
    return __shfl_sync(0xffffffffu, s - w, warp);
}

// The same over the block's threads.
__device__ __forceinline__ int block_scan(int v, int *sums, int *total) {
    const int lane = threadIdx.x & 31;
    int s = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += o;
    }
    return warps_scan(__shfl_sync(0xffffffffu, s, 31), sums, total) + s - v;
}

// Walks over the pages [lo, hi) in ascending order, calling hit(page, rank)
// for those of which pick(refs[page]) holds; ranks count from 0.  Stops once
// `most` have been found (hit may be called for a few more).  Returns how many
// were found.  Called by the whole block.
template <typename Pick, typename Hit>
__device__ int walk(const int *refs, int lo, int hi, int most, int *sums, Pick pick, Hit hit) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int found = 0;
    for (long long base = lo; base < hi && found < most; base += kBookThreads * kSub) {
        // a warp takes 32 * kSub consecutive pages, 32 at a time
        const long long first = base + (long long)warp * (32 * kSub) + lane;
        unsigned mask[kSub];
        int val[kSub], mine = 0;  // of the whole warp
#pragma unroll
        for (int i = 0; i < kSub; ++i) val[i] = first + 32 * i < hi ? refs[first + 32 * i] : 0;
#pragma unroll
        for (int i = 0; i < kSub; ++i) {
            mask[i] = __ballot_sync(0xffffffffu, first + 32 * i < hi && pick(val[i]));
            mine += __popc(mask[i]);
        }
        int total, rank = found + warps_scan(mine, sums, &total);
#pragma unroll
        for (int i = 0; i < kSub; ++i) {
            if (mask[i] >> lane & 1) hit((int)(first + 32 * i), rank + __popc(mask[i] & ((1u << lane) - 1)));
            rank += __popc(mask[i]);
        }
        found += total;
    }
    return found;
}

struct Free {
    __device__ bool operator()(int v) const { return v == 0; }
};
struct Held {
    __device__ bool operator()(int v) const { return v > 0; }
};

__device__ __forceinline__ int pages_of(int n, int S) { return (int)(((long long)n + S - 1) / S); }

// ------------------------------------------------------------------ reserve
// The pages are found first and given out once it is known that they suffice:
// up to kList of them wait in shared memory, for more the pool is walked twice.
__global__ void __launch_bounds__(kBookThreads)
reserve_kernel(int *refs, int *table, int *seqlens, const int *counts, int *shortfall, int B, int P,
               int S, int M) {
    after_previous();
    __shared__ int sums[32], list[kList], before[kBookThreads];
    const int tid = threadIdx.x, per = (B + kBookThreads - 1) / kBookThreads;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    auto need_of = [&](int b) { return pages_of(seqlens[b] + counts[b], S) - pages_of(seqlens[b], S); };
    int need = 0;  // at most B * M in all, which fits an int
    bool bad = false;
    for (int b = b0; b < b1 && !bad; ++b) {
        const int n = seqlens[b], c = counts[b];
        bad = n < 0 || c < 0 || (long long)n + c > (long long)M * S;
        if (!bad) need += need_of(b);
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) {
            *shortfall = -1;
            complain();
        }
        return;
    }
    int wanted;
    before[tid] = block_scan(need, sums, &wanted);
    // page `rank` goes to the sequence b with before(b) <= rank < before(b + 1)
    auto give = [&](int page, int rank) {
        if (rank >= wanted) return;
        int lo = 0, hi = kBookThreads - 1;  // the last chunk that begins at or before rank
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (before[mid] <= rank)
                lo = mid;
            else
                hi = mid - 1;
        }
        int b = lo * per, at = before[lo];
        for (int k = need_of(b); rank >= at + k; k = need_of(b)) {
            at += k;
            ++b;
        }
        table[(long long)b * M + pages_of(seqlens[b], S) + rank - at] = page;
        refs[page] = 1;
    };
    const bool keep = wanted <= kList;
    const int found = walk(refs, 0, P, wanted, sums, Free(), [&](int page, int rank) {
        if (keep && rank < wanted) list[rank] = page;
    });
    if (found < wanted) {
        if (tid == 0) *shortfall = wanted - found;
        return;
    }
    __syncthreads();  // list complete
    if (keep) {
        for (int i = tid; i < wanted; i += kBookThreads) give(list[i], i);
    } else {
        // a page given out is written by the thread that has just read it, and not read again
        walk(refs, 0, P, wanted, sums, Free(), give);
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
    after_previous();
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
// A child's row of the table, every step-th entry from the first, and one more
// holder of each page that it shares.
__device__ __forceinline__ void fork_row(int *refs, int *table, int p, int c, int len, int fresh, int P, int S,
                                         int M, int first, int step) {
    const int whole = len / S;
    const int *from = table + (long long)p * M;
    int *to = table + (long long)c * M;
    for (int j = first; j < M; j += step) {
        int page = -1;
        if (j < whole) {
            page = from[j];
            if (page >= 0 && page < P)
                atomicAdd(refs + page, 1);
            else
                complain();
        } else if (j == whole) {
            page = fresh;  // -1 where the last page is full
        }
        to[j] = page;
    }
}

// Checks every pair, takes a page for each child whose parent's last page is
// partly filled, and sets the children's lengths; all or nothing.  A thread
// holds pairs tid, tid + 1024, ... in registers.  A pair marks its child by a
// negative length, which finds one that is listed twice.  rows: the block
// writes the children's rows of the table too, a warp per pair.
constexpr int kPairs = CSA_CACHE_MAX_FORKS / kBookThreads;
static_assert(CSA_CACHE_MAX_FORKS <= kList, "the pages taken wait in shared memory");

__global__ void __launch_bounds__(kBookThreads)
fork_plan_kernel(int *refs, int *table, int *seqlens, const int *parents, const int *children, int n,
                 int *src, int *dst, int *shortfall, int B, int P, int S, int M, bool rows) {
    after_previous();
    __shared__ int sums[32], list[kList];
    const int tid = threadIdx.x;
    int p[kPairs], c[kPairs], len[kPairs], page[kPairs], rank[kPairs];
    bool bad = false;
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
        const int i = k * kBookThreads + tid;
        p[k] = i < n ? parents[i] : -1;
        c[k] = i < n ? children[i] : -1;
    }
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
        len[k] = 0;
        page[k] = -1;
        if (p[k] < 0 || c[k] < 0) {  // padding
            c[k] = -1;
            continue;
        }
        if (p[k] >= B || c[k] >= B) {
            bad = true;
            c[k] = -1;
            continue;
        }
        len[k] = seqlens[p[k]];
        bad |= seqlens[c[k]] != 0 || len[k] < 0 || len[k] > (long long)M * S;
        if (!bad && len[k] % S != 0) {
            page[k] = table[(long long)p[k] * M + len[k] / S];
            bad |= page[k] < 0 || page[k] >= P;
        }
    }
    bad = __syncthreads_or(bad);
    bool twice = false;
    int wanted = 0, found = 0;
    if (!bad) {
#pragma unroll
        for (int k = 0; k < kPairs; ++k)
            if (c[k] >= 0) twice |= atomicCAS(seqlens + c[k], 0, -1) != 0;
        twice = __syncthreads_or(twice);
#pragma unroll
        for (int k = 0; k < kPairs; ++k)
            if (k * kBookThreads < n) {
                int total;
                rank[k] = wanted + block_scan(page[k] >= 0, sums, &total);
                wanted += total;
            }
        if (!twice)
            found = walk(refs, 0, P, wanted, sums, Free(), [&](int free_page, int at) {
                if (at < wanted) list[at] = free_page;
            });
        __syncthreads();
    }
    const bool done = !bad && !twice && found >= wanted;
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
        const int i = k * kBookThreads + tid;
        if (i < n) {
            const int fresh = done && page[k] >= 0 ? list[rank[k]] : -1;
            if (fresh >= 0) refs[fresh] = 1;
            src[i] = done ? page[k] : -1;
            dst[i] = fresh;
            if (c[k] >= 0 && !bad) seqlens[c[k]] = done ? len[k] : 0;  // no mark is left
        }
    }
    if (tid == 0) {
        *shortfall = bad || twice ? -1 : found < wanted ? wanted - found : 0;
        if (bad || twice) complain();
    }
    if (!done || !rows) return;
    __syncthreads();
    for (int i = tid >> 5; i < n; i += kBookWarps) {
        const int from = parents[i], to = children[i];
        if (from >= 0 && to >= 0)
            fork_row(refs, table, from, to, seqlens[to], dst[i], P, S, M, tid & 31, 32);
    }
}

// The children's rows, one block per pair; their lengths are set.
__global__ void __launch_bounds__(256)
fork_rows_kernel(int *refs, int *table, const int *seqlens, const int *parents, const int *children,
                 const int *dst, const int *shortfall, int P, int S, int M) {
    after_previous();
    const int i = blockIdx.x, p = parents[i], c = children[i];
    if (*shortfall != 0 || p < 0 || c < 0) return;
    fork_row(refs, table, p, c, seqlens[c], dst[i], P, S, M, threadIdx.x, blockDim.x);
}

// ------------------------------------------------------------------ compact
// The new number of a held page: dst of its place in src, which ascends, or
// its own.
__device__ __forceinline__ int renamed(int page, const int *src, const int *dst, int moved) {
    int lo = 0, hi = moved;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (src[mid] < page)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo < moved && src[lo] == page ? dst[lo] : page;
}

__device__ __forceinline__ void rename_row(int *table, const int *seqlens, int b, const int *src, const int *dst,
                                           int moved, int S, int M, int first, int step) {
    const int n = seqlens[b];
    if (n < 0 || n > (long long)M * S) {
        if (first == 0) complain();
        return;
    }
    const int held = pages_of(n, S);
    for (int j = first; j < held; j += step) {
        int *entry = table + (long long)b * M + j;
        *entry = renamed(*entry, src, dst, moved);
    }
}

// The held pages [U, P) go to the free pages [0, U), both in ascending order;
// U is the number of held pages.  rows: the block renames the table's entries
// too, a warp per sequence.
__global__ void __launch_bounds__(kBookThreads)
compact_plan_kernel(int *refs, int *table, const int *seqlens, int *src, int *dst, int *moved, int B, int P,
                    int S, int M, bool rows) {
    after_previous();
    __shared__ int sums[32];
    const int tid = threadIdx.x, all = 0x7fffffff;
    const int U = walk(refs, 0, P, all, sums, Held(), [](int, int) {});
    const int K = walk(refs, U, P, all, sums, Held(), [&](int page, int rank) { src[rank] = page; });
    walk(refs, 0, U, K, sums, [](int v) { return v <= 0; }, [&](int page, int rank) { dst[rank] = page; });
    __syncthreads();
    for (int i = tid; i < K; i += kBookThreads) {
        refs[dst[i]] = refs[src[i]];
        refs[src[i]] = 0;
    }
    for (int i = K + tid; i < P / 2; i += kBookThreads) src[i] = dst[i] = -1;
    if (tid == 0) *moved = K;
    if (rows)
        for (int b = tid >> 5; b < B; b += kBookWarps)
            rename_row(table, seqlens, b, src, dst, K, S, M, tid & 31, 32);
}

__global__ void __launch_bounds__(256)
rename_kernel(int *table, const int *seqlens, const int *src, const int *dst, const int *moved, int B, int S,
              int M) {
    after_previous();
    const int K = *moved;
    for (int b = blockIdx.x; b < B; b += gridDim.x)
        rename_row(table, seqlens, b, src, dst, K, S, M, threadIdx.x, blockDim.x);
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
    after_previous();
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

// ------------------------------------------------------------------- accept
// A warp per sequence.  The path from the last accepted node up to its root is a
// mask of 64 nodes, walked by shuffles (lane i has the parents of nodes i and i + 32);
// a node's place on it is the number of nodes below it in the mask.  Latency bounds it:
// three dependent trips to memory, 3 us for 64 sequences of 8 or 64 drafted tokens.
constexpr int kAcceptWarps = 4;

__global__ void __launch_bounds__(32 * kAcceptWarps)
accept_kernel(int *refs, int *table, int *seqlens, const int *parents, const int *counts, const int *last, int *src,
              int *dst, int T, int B, int P, int S, int M) {
    after_previous();
    const int b = blockIdx.x * kAcceptWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (b >= B) return;
    const int len = seqlens[b], count = counts ? counts[b] : T, leaf = last[b];
    int up[2], from[2] = {-1, -1}, to[2] = {-1, -1};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = lane + 32 * i;
        up[i] = t >= T ? -1 : parents ? parents[(long long)b * T + t] : t - 1;
    }
    bool sound = count >= 0 && count <= T && len >= count && len <= (long long)M * S && leaf >= -1 && leaf < count;
    unsigned long long path = 0;
    for (int node = leaf; sound && node >= 0;) {  // the same on every lane
        path |= 1ull << node;
        const int a = __shfl_sync(0xffffffffu, up[0], node & 31), c = __shfl_sync(0xffffffffu, up[1], node & 31);
        const int next = node < 32 ? a : c;
        sound = next >= -1 && next < node;
        node = next;
    }
    const int n = len - count, kept = __popcll(path);
    int *row = table + (long long)b * M;
    auto place = [&](int at) {  // the pool's row of token `at`
        const int page = row[at / S];
        if (page < 0 || page >= P) sound = false;
        return page * S + at % S;
    };
    if (sound)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int node = lane + 32 * i;
            if (path >> node & 1) {
                const int at = __popcll(path & ((1ull << node) - 1));
                if (at != node) {
                    from[i] = place(n + node);
                    to[i] = place(n + at);
                }
            }
        }
    sound = __all_sync(0xffffffffu, sound);
    if (!sound && lane == 0) complain();
    int *s = src + (long long)b * T, *d = dst + (long long)b * T;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int at = lane + 32 * i, below = __popcll(path & ((1ull << at) - 1));
        if (at >= T) continue;
        // a place behind the kept ones, or whose node is there already; the others get theirs below
        if (!sound || at >= kept || (below == at && (path >> at & 1))) s[at] = d[at] = -1;
        if (sound && to[i] >= 0) {
            s[below] = from[i];
            d[below] = to[i];
        }
    }
    if (!sound) return;
    for (int j = pages_of(n + kept, S) + lane; j < pages_of(len, S); j += 32) {
        const int page = row[j];
        if (page < 0 || page >= P) {
            complain();
        } else if (atomicSub(&refs[page], 1) <= 0) {  // nobody held it
            atomicAdd(&refs[page], 1);
            complain();
        }
        row[j] = -1;
    }
    if (lane == 0) seqlens[b] = n + kept;
}

// --------------------------------------------------------------- copied rows
// Row r of a pool of P pages is slot r mod S of page r / S.  A block has one group of
// pairs and a range of the planes (a head of a layer) of one tensor.  Of a plane it
// reads a range of columns of all of the group's rows before it writes the first of
// them, so rows of a group may change places.  The pairs that are rows come first, so
// that a few of many leave no thread idle: as many planes at once as the threads can
// hold.  What bounds it: with few rows, the two trips to memory (4 of 64 drafted tokens
// of 64 sequences, 8 layers of 8 heads, d = 128: 8 us, 21 with a block per plane); with many, HBM.
struct RowTensor {
    uint8_t *at;
    long long bytes;  // of a row
    int unit;         // the widest type that all rows allow: 16, 4 or 1 bytes
};
struct CopyRowsParams {
    RowTensor x[3];
    int planes, per_block;  // of a tensor; H to a layer
    int P, H, S, T;
    const int *src, *dst;
};
constexpr int kRowThreads = 256, kRowDeep = 4, kRowMost = 64;

// Pairs [0, n): rows of the first plane.
template <typename C>
__device__ __forceinline__ void copy_group(const CopyRowsParams &p, const RowTensor &x, const long long (*pair)[2], int n,
                                           int plane, int end) {
    constexpr int kHold = kRowThreads * kRowDeep;
    const int units = (int)(x.bytes / (long long)sizeof(C));
    const bool whole = units <= kHold / n;
    const int width = whole ? units : kHold / n, at_once = whole ? kHold / (n * units) : 1;
    for (; plane < end; plane += at_once)
        for (int c0 = 0; c0 < units; c0 += width) {
            const int w = min(width, units - c0), items = min(at_once, end - plane) * n * w;
            C val[kRowDeep];
            C *to[kRowDeep];
#pragma unroll
            for (int j = 0; j < kRowDeep; ++j) {
                const int i = threadIdx.x + j * kRowThreads;
                if (i >= items) break;
                const int row = i / w, k = row / n, r = row - k * n, layer = (plane + k) / p.H, h = plane + k - layer * p.H;
                const long long first = ((long long)layer * p.P * p.H + h) * p.S;
                val[j] = reinterpret_cast<const C *>(x.at + (first + pair[r][0]) * x.bytes)[c0 + i - row * w];
                to[j] = reinterpret_cast<C *>(x.at + (first + pair[r][1]) * x.bytes) + c0 + i - row * w;
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kRowDeep; ++j)
                if (threadIdx.x + j * kRowThreads < items) *to[j] = val[j];
        }
}

__global__ void __launch_bounds__(kRowThreads) copy_rows_kernel(const __grid_constant__ CopyRowsParams p) {
    __shared__ long long pair[kRowMost][2];
    __shared__ int some[2];
    after_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, T = p.T;
    int s = -1, d = -1;
    bool moves = false;
    unsigned all = 0;
    if (warp < kRowMost / 32) {
        if (threadIdx.x < T) {
            s = p.src[(long long)blockIdx.x * T + threadIdx.x];
            d = p.dst[(long long)blockIdx.x * T + threadIdx.x];
            const long long rows = (long long)p.P * p.S;
            moves = s >= 0 && d >= 0 && s < rows && d < rows;
            if (s >= 0 && d >= 0 && !moves) complain();
        }
        all = __ballot_sync(0xffffffffu, moves);
        if (lane == 0) some[warp] = __popc(all);
    }
    __syncthreads();
    const int n = some[0] + some[1];
    if (n == 0) return;
    if (moves) {
        const int at = (warp > 0 ? some[0] : 0) + __popc(all & ((1u << lane) - 1));
        auto row = [&](int r) { return (long long)(r / p.S) * p.H * p.S + r % p.S; };
        pair[at][0] = row(s);
        pair[at][1] = row(d);
    }
    __syncthreads();
    const RowTensor &x = p.x[blockIdx.y];
    const int plane = blockIdx.z * p.per_block, end = min(plane + p.per_block, p.planes);
    if (x.unit == 16)
        copy_group<uint4>(p, x, pair, n, plane, end);
    else if (x.unit == 4)
        copy_group<uint32_t>(p, x, pair, n, plane, end);
    else
        copy_group<uint8_t>(p, x, pair, n, plane, end);
}

int from(cudaError_t e) { return e == cudaSuccess ? CSA_OK : CSA_ERR_CUDA; }

template <typename C>
int copy_as(void *k, void *v, long long page_bytes, int layers, int P, const int *src,
            const int *dst, int n, const int *count, cudaStream_t stream) {
    const long long page = page_bytes / (long long)sizeof(C);
    const long long part = kCopyThreads * kCopyDeep, parts = (page + part - 1) / part;
    if (parts * layers * 2 > 0x7fffffffLL) return CSA_ERR_UNSUPPORTED;
    const long long items = parts * layers * (v ? 2 : 1) * n;
    const unsigned grid = (unsigned)(items < 152 * 32 ? items : 152 * 32);
    return from(launch_after_previous(copy_pages_kernel<C>, grid, kCopyThreads, 0, stream, static_cast<C *>(k),
                                      static_cast<C *>(v), page, layers, P, src, dst, n, count, (int)parts));
}

}  // namespace

int csa_cache_reserve_run(int *refs, int *table, int *seqlens, const int *counts, int *shortfall, int B,
                          int P, int S, int M, cudaStream_t stream) {
    return from(launch_after_previous(reserve_kernel, 1, kBookThreads, 0, stream, refs, table, seqlens, counts,
                                      shortfall, B, P, S, M));
}

int csa_cache_free_run(int *refs, int *table, int *seqlens, const int *rows, int R, int B, int P,
                       int S, int M, cudaStream_t stream) {
    return from(launch_after_previous(free_kernel, R, 256, 0, stream, refs, table, seqlens, rows, R, B, P, S, M));
}

int csa_cache_fork_run(int *refs, int *table, int *seqlens, const int *parents, const int *children,
                       int n, int *src, int *dst, int *shortfall, int B, int P, int S, int M,
                       cudaStream_t stream) {
    const bool one = (long long)n * M <= kOneBlock;
    if (launch_after_previous(fork_plan_kernel, 1, kBookThreads, 0, stream, refs, table, seqlens, parents, children, n,
                              src, dst, shortfall, B, P, S, M, one) != cudaSuccess)
        return CSA_ERR_CUDA;
    if (one) return CSA_OK;
    return from(launch_after_previous(fork_rows_kernel, n, 256, 0, stream, refs, table, seqlens, parents, children, dst,
                                      shortfall, P, S, M));
}

int csa_cache_compact_run(int *refs, int *table, const int *seqlens, int *src, int *dst, int *moved, int B,
                          int P, int S, int M, cudaStream_t stream) {
    const bool one = (long long)B * M <= kOneBlock;
    if (launch_after_previous(compact_plan_kernel, 1, kBookThreads, 0, stream, refs, table, seqlens, src, dst, moved, B,
                              P, S, M, one) != cudaSuccess)
        return CSA_ERR_CUDA;
    if (one) return CSA_OK;
    return from(launch_after_previous(rename_kernel, B < 152 * 8 ? B : 152 * 8, 256, 0, stream, table, seqlens, src, dst,
                                      moved, B, S, M));
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

int csa_cache_accept_run(int *refs, int *table, int *seqlens, const int *parents, const int *counts, const int *last,
                         int *src, int *dst, int T, int B, int P, int S, int M, cudaStream_t stream) {
    return from(launch_after_previous(accept_kernel, (B + kAcceptWarps - 1) / kAcceptWarps, 32 * kAcceptWarps, 0, stream,
                                      refs, table, seqlens, parents, counts, last, src, dst, T, B, P, S, M));
}

int csa_cache_copy_rows_run(void *k_pages, void *v_pages, long long row_bytes, void *row_scales, long long scale_bytes,
                            int layers, int P, int H, int S, const int *src, const int *dst, int B, int T,
                            cudaStream_t stream) {
    CopyRowsParams p = {};
    int tensors = 0;
    void *at[3] = {k_pages, v_pages, row_scales};
    for (int i = 0; i < 3; ++i) {
        const long long bytes = i < 2 ? row_bytes : scale_bytes;
        if (!at[i] || bytes == 0) continue;
        const uintptr_t bits = reinterpret_cast<uintptr_t>(at[i]) | (uintptr_t)bytes;
        p.x[tensors++] = {static_cast<uint8_t *>(at[i]), bytes, bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 1};
    }
    if (tensors == 0) return CSA_OK;
    p.P = P;
    p.H = H;
    p.S = S;
    p.T = T;
    p.src = src;
    p.dst = dst;
    // about as many blocks as run at a time
    p.planes = layers * H;
    const int places = std::max(1, 8 * 152 / (int)std::min((long long)B * tensors, 8 * 152ll));
    p.per_block = (p.planes + places - 1) / places;
    const dim3 grid((unsigned)B, (unsigned)tensors, (unsigned)((p.planes + p.per_block - 1) / p.per_block));
    return from(launch_after_previous(copy_rows_kernel, grid, kRowThreads, 0, stream, p));
}

int *csa_cache_status_word(void) {
    void *at = nullptr;
    return cudaGetSymbolAddress(&at, g_cache_status) == cudaSuccess ? static_cast<int *>(at) : nullptr;
}

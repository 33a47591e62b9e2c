// kda_mla_common.cuh -- device helpers shared by the latent-attention kernels: the sequences of a
// packed batch and the tokens' places in the paged cache, both checked before use.
#pragma once

#include <stdint.h>

#include "kda.h"
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace mla {

// Waits until the kernels before this one in the stream have ended and their writes are visible.  Every thread of a
// kernel started by launch_early() calls it before its first access to memory that is not its own.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// First row and row count of sequence b of a packed batch of T rows (cu = NULL: equal lengths).  A bad
// entry raises the flag and gives no rows.
__device__ __forceinline__ int seq_rows(const int32_t* cu, int64_t T, int B, int b, int64_t& first,
                                        unsigned int* flags) {
    if (!cu) {
        const int64_t n = T / B;
        first = n * b;
        return static_cast<int>(n);
    }
    const int32_t lo = cu[b], hi = cu[b + 1];
    first = lo;
    if (lo < 0 || hi < lo || hi > T || (b == 0 && lo != 0)) {
        raise_flag(flags, KDA_DEVFLAG_CU_SEQLENS);
        return 0;
    }
    return hi - lo;
}

// Every entry of a packed batch checked by one block's threads, for kernels that work row by row and so need
// not meet a bad entry themselves.
__device__ __forceinline__ void check_cu(const int32_t* cu, int64_t T, int B, unsigned int* flags) {
    if (!cu) return;
    bool bad = threadIdx.x == 0 && cu[0] != 0;
    for (int b = threadIdx.x; b < B; b += blockDim.x) bad = bad || cu[b + 1] < cu[b] || cu[b + 1] > T;
    if (bad) raise_flag(flags, KDA_DEVFLAG_CU_SEQLENS);
}

// The sequence that row t of a packed batch belongs to: the last b with cu[b] <= t; B where t lies behind
// the last sequence.  With a bad (decreasing) cu the answer is some b in [0, B], which seq_rows checks.
__device__ __forceinline__ int seq_of_row(const int32_t* cu, int64_t T, int B, int64_t t) {
    if (!cu) return static_cast<int>(t / (T / B));
    int lo = 0, hi = B;  // cu[lo] <= t < cu[hi + 1] is what is looked for; cu[B] may be <= t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// The pool row of position pos of sequence b; -1 (and the flag) where its page number is out of range.
__device__ __forceinline__ int64_t pool_row(const MlaCache& c, int b, int pos, unsigned int* flags) {
    const int page = c.page_table[static_cast<int64_t>(b) * c.max_pages + (pos >> c.page_shift)];
    if (page < 0 || page >= c.num_pages) {
        raise_flag(flags, KDA_DEVFLAG_PAGE_TABLE);
        return -1;
    }
    return (static_cast<int64_t>(page) << c.page_shift) + (pos & (c.page_size - 1));
}

// Tokens the page table of one sequence reaches.
__device__ __forceinline__ int64_t table_reach(const MlaCache& c) {
    return static_cast<int64_t>(c.max_pages) << c.page_shift;
}

}  // namespace mla
}  // namespace kda

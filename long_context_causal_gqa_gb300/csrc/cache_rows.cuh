// cache_rows.cuh -- which cached token each row of a step stands for: the
// addressing shared by the cache write, cache read and block index kernels.
//
// The rows of a step belong to `batch` sequences, one behind the other:
// sequence b owns rows row_starts[b] .. row_starts[b + 1] - 1 (or tokens /
// batch rows each without row_starts), the last n_b tokens of its context, so
// its row j sits at position ctx_lens[b] - n_b + j.
#pragma once

#include <stdint.h>

#include "internal.h"
#include "sm100.cuh"

namespace gqa {

constexpr int kRowsMaxBatch = 1024;

struct RowMap {
    const int32_t* tables;      // [batch, table_stride] physical page ids
    const int32_t* row_starts;  // [batch + 1], or null: rows_per_seq rows each
    const int32_t* ctx_lens;    // [batch]
    int table_stride;
    int num_pages;
    int log2_page;
    int max_ctx;
    int batch;
    int tokens;
    FastDiv rows_per_seq;
    unsigned* err;
};

// The row starts in shared memory (every thread of the CTA calls this; a
// barrier is needed before the first locate_row).
__device__ __forceinline__ void load_row_starts(const RowMap& m, int* s_starts) {
    if (m.row_starts)
        for (int i = threadIdx.x; i <= m.batch; i += blockDim.x) s_starts[i] = m.row_starts[i];
}

// Row j of the n rows of sequence b: its position and its token row in the
// cache, slot = -1 if the page table's entry is outside the cache (flagged, as
// is a context length outside [n, max_ctx]: pos = -1).
__device__ __forceinline__ void locate_in_sequence(const RowMap& m, int b, int j, int n, int* pos,
                                                   long long* slot) {
    const int ctx = m.ctx_lens[b];
    if (ctx < n || ctx > m.max_ctx) {
        atomicOr(m.err, kErrBadCtxLen);
        return;
    }
    const int p = ctx - n + j;
    *pos = p;
    const int id = m.tables[(long long)b * m.table_stride + (p >> m.log2_page)];
    if (id < 0 || id >= m.num_pages) {
        atomicOr(m.err, kErrBadPageId);
        return;
    }
    *slot = ((long long)id << m.log2_page) + (p & ((1 << m.log2_page) - 1));
}

// Position of `row` in its sequence and its token row in the cache, -1 each for
// a padding row (in front of the first sequence or behind the last).  One
// thread, the starts in shared memory.
__device__ __forceinline__ void locate_row(const RowMap& m, const int* s_starts, int row,
                                           int* pos, long long* slot) {
    *pos = -1;
    *slot = -1;
    if (!m.row_starts) {
        const int b = m.rows_per_seq.div(row), n = m.rows_per_seq.d;
        locate_in_sequence(m, b, row - b * n, n, pos, slot);
        return;
    }
    // The last start <= row (empty sequences share a start with the next).
    int lo = 0, hi = m.batch + 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s_starts[mid] <= row) lo = mid + 1;
        else hi = mid;
    }
    const int b = lo - 1;
    if (b < 0 || b >= m.batch) return;
    const int first = s_starts[b], end = s_starts[b + 1];
    if (first < 0 || end <= row) return;   // starts that do not ascend
    locate_in_sequence(m, b, row - first, end - first, pos, slot);
}

}  // namespace gqa

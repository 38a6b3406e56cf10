// pick.cuh -- the best of one row's blocks by one CTA: the limit of the k largest
// keys by counts over parts of their range, and the taken ids in ascending order.
// The device functions of the block selection's last kernels, in a header of their
// own so that a host compiler can run them too, a thread for each of the CTA's.
#pragma once

#include <stdint.h>

namespace gqa {
namespace select {

// What a row takes: blocks below n_first and from hi on always, `need` of the
// scored blocks [n_first, hi).
struct RowRange {
    int n_vis, take, lo, hi, need;
    // Of a row that does not take all: take again, from what is at hand (take itself,
    // kept in a register for the stores' sake, cost best_kernel a stack frame).
    __device__ __forceinline__ int room() const { return lo + need + n_vis - hi; }
};
__device__ __forceinline__ RowRange row_range(int pos, int max_sel, int n_first, int n_last) {
    RowRange r;
    r.n_vis = (pos >> 2) + 1;
    r.take = min(max_sel, r.n_vis);
    r.lo = n_first;
    r.hi = r.n_vis - n_last;
    r.need = r.take == r.n_vis ? 0 : r.take - n_first - n_last;
    return r;
}

// A float's order as whole numbers above 0; NaN, as 1, below everything.  Adding
// zero makes the two zeros one.
__device__ __forceinline__ uint32_t ordered(float f) {
    if (f != f) return 1;
    const uint32_t u = __float_as_uint(f + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

constexpr int WINDOW = 65536;    // block ids of one pass of the ordered output
__host__ __device__ __forceinline__ int bits_words(int ids) {
    return ((ids < WINDOW ? ids : WINDOW) + 127) / 128 * 4;
}

// A picking CTA's dynamic shared memory, in 32-bit words from its 16-byte aligned
// start: the ids' bits [words, in whole uint4], the candidates' keys and ids [room]
// each, the maxima's keys [room_groups], the groups that reach the limit
// [room_reach].  Launch and kernel take the places and the size from here.
struct PickAreas {
    int words, room, room_groups, room_reach;
    __host__ __device__ __forceinline__ int key() const { return words; }
    __host__ __device__ __forceinline__ int id() const { return key() + room; }
    __host__ __device__ __forceinline__ int groups() const { return id() + room; }
    __host__ __device__ __forceinline__ int reach() const { return groups() + room_groups; }
    __host__ __device__ __forceinline__ int bytes() const { return 4 * (reach() + room_reach); }
};
constexpr int PICK_SMEM = 192 << 10;           // most keys of a CTA, in bytes
constexpr int PICK_MOST_TAKEN = 2048;
constexpr int PICK_MOST_BYTES = PICK_SMEM + (2 * PICK_MOST_TAKEN + 256) * 4 + WINDOW / 8;
constexpr int BEST_MOST_BYTES = PICK_SMEM + WINDOW / 8;

// Of a row that sees n_vis blocks at most, n of them scored: from all its scores, or
// by their maxima.
inline PickAreas pick_areas(int n_vis, int n, int max_sel, bool maxima) {
    const int most = PICK_SMEM / 8;
    if (!maxima) return {bits_words(n_vis), min(n, most), 0, 0};
    // Fewer maxima of more blocks, as long as they are many per block taken: one row
    // of 65470 blocks 17.8 us with 8184 maxima, 17.1 with 4092, and with 512 taken
    // 19.8 and 20.8.
    const int groups = min(min(max(16 * max_sel, 4096), 16384), (n + 7) / 8);
    return {bits_words(n_vis), min(12 * max_sel + 1024, most - (groups + 1) / 2), groups,
            2 * max_sel + 256};
}
// By candidates, `expected` of them.
inline PickAreas best_areas(int n_vis, int expected, int max_sel) {
    return {bits_words(n_vis), min(2 * expected + max_sel + 256, PICK_SMEM / 8), 0, 0};
}

template <int THREADS>
struct BestShared {
    static constexpr int LOG2_BINS = THREADS <= 512 ? 9 : 10;
    static constexpr int BINS = 1 << LOG2_BINS;
    int hist[BINS];
    uint32_t most[32], least[32];
    int sums[32];
    int digit, left, count;
    int total, bad;
};

// Inclusive prefix sum over the CTA's threads; two barriers.
template <int THREADS>
__device__ __forceinline__ int cta_scan(int v, int* sums) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? sums[lane] : 0);
    __syncthreads();
    return v + before;
}

// The smallest and the largest of key[0 .. total), all above 0.
template <int THREADS>
__device__ void range_of(const uint32_t* key, int total, uint32_t* least, uint32_t* most,
                         BestShared<THREADS>& S) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    uint32_t a = ~0u, b = 0;
#pragma unroll 1
    for (int i = threadIdx.x; i < total; i += THREADS) {
        const uint32_t k = key[i];
        a = min(a, k);
        b = max(b, k);
    }
    a = __reduce_min_sync(0xffffffffu, a);
    b = __reduce_max_sync(0xffffffffu, b);
    if (lane == 0) {
        S.least[warp] = a;
        S.most[warp] = b;
    }
    __syncthreads();
    *least = __reduce_min_sync(0xffffffffu, S.least[lane % (THREADS / 32)]);
    *most = __reduce_max_sync(0xffffffffu, S.most[lane % (THREADS / 32)]);
}

// A limit for the `need` largest of key[0 .. total), 1 <= need <= those in
// [least, most] (0: not to be counted; none is above most): those above the
// limit are taken, and `equals` of those equal to it.  Counts over BINS equal
// parts of the keys' range, then of the part that holds the need-th largest,
// until what is in the part is taken whole.  Where fewer than `need` are in
// [least, most] all the same (best_of says when), the limit is any: each part is
// narrower than the last, so it ends as soon.
struct Limit {
    uint32_t key;
    int equals;
};

template <int THREADS>
__device__ __forceinline__ Limit need_th(const uint32_t* key, int total, int need, uint32_t least,
                                         uint32_t most, BestShared<THREADS>& S) {
    constexpr int LOG2_BINS = BestShared<THREADS>::LOG2_BINS, BINS = 1 << LOG2_BINS;
    const int tid = threadIdx.x;
    uint32_t lo = least, width = most - least;   // keys of interest: [lo, lo + width]
#pragma unroll 1
    for (;;) {
        const int shift = width >> LOG2_BINS ? 32 - LOG2_BINS - __clz((int)width) : 0;
        constexpr int PER = BINS / THREADS;
#pragma unroll
        for (int i = 0; i < PER; ++i) S.hist[tid + i * THREADS] = 0;
        __syncthreads();
#pragma unroll 1
        for (int i = tid; i < total; i += THREADS) {
            const uint32_t k = key[i] - lo;      // below lo: wraps to beyond width
            if (k <= width) atomicAdd(&S.hist[k >> shift], 1);
        }
        __syncthreads();
        // Thread t holds bins from the top down.
        int c[PER], sum = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            c[i] = S.hist[BINS - 1 - tid * PER - i];
            sum += c[i];
        }
        int before = cta_scan<THREADS>(sum, S.sums) - sum;
        if (before < need && need <= before + sum) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (before < need && need <= before + c[i]) {
                    S.digit = BINS - 1 - tid * PER - i;
                    S.left = need - before;
                    S.count = c[i];
                }
                before += c[i];
            }
        }
        __syncthreads();
        lo += (uint32_t)S.digit << shift;
        need = S.left;
        if (S.count == need) return {lo - 1, 0};
        if (shift == 0) return {lo, need};
        // (the last part may end beyond `most`: no key is there, but 0 would be)
        width = min((1u << shift) - 1, most - lo);
        __syncthreads();
    }
}

// The same as a function, for a kernel that runs once on one SM and pays more
// for each instruction's first fetch than for executing it.
template <int THREADS>
__device__ __noinline__ Limit need_th_called(const uint32_t* key, int total, int need,
                                             uint32_t least, uint32_t most,
                                             BestShared<THREADS>& S) {
    return need_th<THREADS>(key, total, need, least, most, S);
}

// Writes the taken blocks in ascending order: those below R.lo, those from
// R.hi on, and the R.need best of the candidates (key[i] within [least, most],
// id[i]), i < total, equal keys by the lower id; key[] does not outlast the
// call.  total >= R.need.  bits: room for one per id of a window, in whole uint4.
//
// Keys and limits come from a workspace that a call whose wait ran into its limit
// (an error is flagged), or another call at the same time, leaves in any state.
// Then the ids are not the best, but only the row's own R.take places are written.
template <int THREADS, bool CALLED>
__device__ __forceinline__ void best_of(const RowRange& R, uint32_t* key, const int* id, int total,
                                        uint32_t least, uint32_t most, int32_t* out,
                                        uint32_t* bits, BestShared<THREADS>& S) {
    const int tid = threadIdx.x;
    uint32_t limit = 0;     // keys above it are taken
    if (R.need > 0) {
        Limit l = CALLED ? need_th_called<THREADS>(key, total, R.need, least, most, S)
                         : need_th<THREADS>(key, total, R.need, least, most, S);
        limit = l.key;
        if (l.equals > 0) {
            // Of the equal ones the lowest ids: on with keys that fall with the id,
            // the larger ones above all of them and the smaller ones 0.
            __syncthreads();
#pragma unroll 1
            for (int i = tid; i < total; i += THREADS) {
                const uint32_t k = key[i];
                key[i] = k > limit ? ~0u : k == limit ? ~1u - (uint32_t)id[i] : 0u;
            }
            __syncthreads();
            limit = need_th_called<THREADS>(key, total, l.equals, 1u, ~1u, S).key;
        }
    }
    int done = 0;    // ids written
    for (int w0 = 0; w0 < R.n_vis; w0 += WINDOW) {
        const uint32_t ids = (uint32_t)min(WINDOW, R.n_vis - w0);
        const int quads = (int)(ids + 127) / 128;
        uint4* bits4 = reinterpret_cast<uint4*>(bits);
        for (int i = tid; i < quads; i += THREADS) bits4[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        auto mark = [&](int b) {
            const uint32_t i = (uint32_t)b - (uint32_t)w0;
            if (i < ids) atomicOr(&bits[i / 32], 1u << (i % 32));
        };
        for (int b = tid; b < R.lo; b += THREADS) mark(b);
        for (int b = R.hi + tid; b < R.n_vis; b += THREADS) mark(b);
        if (R.need > 0)
#pragma unroll 1
            for (int i = tid; i < total; i += THREADS)
                if (key[i] > limit) mark(id[i]);
        __syncthreads();
        // Thread t writes the ids of its stretch of words.
        const int per = (quads + THREADS - 1) / THREADS;
        const int a = min(tid * per, quads), b = min(a + per, quads);
        int n = 0;
        for (int i = a; i < b; ++i) {
            const uint4 u = bits4[i];
            n += __popc(u.x) + __popc(u.y) + __popc(u.z) + __popc(u.w);
        }
        const int upto = cta_scan<THREADS>(n, S.sums);
        int at = done + upto - n;
        if (n && at + n <= R.room())
            for (int i = 4 * a; i < 4 * b; ++i)
                for (uint32_t m = bits[i]; m; m &= m - 1)
                    out[at++] = w0 + i * 32 + __ffs(m) - 1;
        if (w0 + WINDOW >= R.n_vis) break;
        if (tid == THREADS - 1) S.count = upto;
        __syncthreads();
        done += S.count;
    }
}

// The best blocks of one row by its scores, one after the other (score(b) for
// lo <= b < hi), whatever their number: the key of the last one taken is found
// eight bits at a time, then one pass over the blocks in order writes those
// above it and the first of those equal to it, R.take at most (as in best_of,
// whatever the scores are from pass to pass).
template <int THREADS, typename Score>
__device__ void scan_best(const RowRange& R, const Score& score, int32_t* out,
                          BestShared<THREADS>& S) {
    const int tid = threadIdx.x;
    uint32_t prefix = 0;
    int need = R.need;
    for (int shift = 24; need > 0 && shift >= 0; shift -= 8) {
        __syncthreads();
        for (int i = tid; i < 256; i += THREADS) S.hist[i] = 0;
        __syncthreads();
        for (int b = R.lo + tid; b < R.hi; b += THREADS) {
            const uint32_t k = ordered(score(b));
            if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
                atomicAdd(&S.hist[(k >> shift) & 255], 1);
        }
        __syncthreads();
        // Thread t holds bins 255 - 2 t and 254 - 2 t.
        const int c0 = tid < 128 ? S.hist[255 - 2 * tid] : 0;
        const int c1 = tid < 128 ? S.hist[254 - 2 * tid] : 0;
        const int before = cta_scan<THREADS>(c0 + c1, S.sums) - c0 - c1;
        if (before < need && need <= before + c0 + c1) {
            const bool second = need > before + c0;
            S.digit = 255 - 2 * tid - second;
            S.left = need - before - (second ? c0 : 0);
        }
        __syncthreads();
        prefix |= (uint32_t)S.digit << shift;
        need = S.left;
    }
    // need = how many of the blocks with key == prefix are taken (lowest ids).
    int done = 0, equals = 0;    // ids written, equal keys met
    for (int b0 = 0; b0 < R.n_vis; b0 += THREADS) {
        const int b = b0 + tid;
        bool above = false, equal = false;
        if (b < R.n_vis) {
            if (b < R.lo || b >= R.hi) above = true;
            else if (R.need > 0) {
                const uint32_t k = ordered(score(b));
                above = k > prefix;
                equal = k == prefix;
            }
        }
        const int e = equals + cta_scan<THREADS>(equal, S.sums);
        const bool take = above || (equal && e <= need);
        const int at = done + cta_scan<THREADS>(take, S.sums);
        if (take && at <= R.room()) out[at - 1] = b;
        if (tid == THREADS - 1) {
            S.left = e;
            S.count = at;
        }
        __syncthreads();
        equals = S.left;
        done = S.count;
    }
}

}  // namespace select
}  // namespace gqa

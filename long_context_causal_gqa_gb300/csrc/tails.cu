// tails.cu -- causal GQA tails of a batch over a 4-bit paged cache (rows as in
// fp4_rows.cuh) or an E4M3 one, with a sliding window and first tokens that stay
// visible ("sinks").
//
//   out = softmax_j(scale * q . k_j) v_j over the keys j of the sequence with
//   j <= p and (no window, or j > p - window, or j < sinks), p the row's position.
//
// One pass over the visible tiles of 128 or 64 keys, with a running maximum and sum.
//
// * Work split.  A KV head's rows of all query heads are packed, up to 48.  The visible
//   tiles of all (KV head, sequence) units, one behind the other in this order, are cut
//   into one equal contiguous range per CTA, from the context lengths on the device.  (Sequences
//   innermost: ranges of two heads then go over the same pages side by side, and what one
//   reads beside its own 128 bytes of an E4M3 row the other finds in L2: 54 us instead of
//   61 for 48 windows of 8192 tokens, two heads of 128.)  A unit that lies in one range is
//   finished there; a unit that is cut leaves (O, m, l) partials, at most two for a CTA,
//   which a second kernel joins in range order.
// * Copies.  Four warps bring the pages of a tile that some row sees into a ring of stages
//   (up to 192 KB: the bytes in flight set the copy rate), 4-bit pages by bulk copies (a
//   page of one head is one contiguous run), E4M3 rows by tensor maps, table entries lots
//   ahead.
// * Products.  Two groups of four warps take a tile each.  A warp decodes its codes from
//   shared memory straight into the fragments of m16n8k16 products, keys (for K) or
//   places of D (for V) along M, packed query rows along N, so eight rows waste nothing.
//   The order of the places within a product is free, so a lane loads whole words of one
//   key: K's pairs are a byte's two nibbles, V's pairs are put together from two keys'.
//   Nothing decoded goes through shared memory.  (For tcgen05.mma V would have to, or be
//   turned: its places of D would lie along M, and codes arrive by key.  Keys along M could
//   be decoded into tensor memory, a key a lane, and the scores taken there; not built.)
// * Softmax.  A reference of a row moves only when a score passes it by more than 8 (log2
//   units), so P <= 256 in fp16.  More than eight packed rows: P goes through shared
//   memory to the warps that hold the sums, computed with the group's reference as it
//   stands, and only where some warp's scores passed it (flagged at the one barrier of a
//   tile) is it moved, and P computed again.  Up to eight: a warp keeps all for itself.
//
// Replays behind one another, with the bytes that have to be read at the copy rate and a
// plain reading kernel's time where it was measured: one row over 261888 4-bit tokens
// 24.1 us (11.3; 18.1 by one call of the reading kernel against 26.8), 64 ragged contexts
// of up to 8192 46.4 us (26.5; 34 against 52), eight rows over 128000 30.8 us (5.6), sixteen
// windows of 2000 11.9 us (1.3), 48 E4M3 windows of 8192 43.6 us (29; 38.5 against 49).
// Small calls are chains of latencies: lengths, table, first page, then the join's
// record and partials (a window of 4096: 7.5 us, 7.2 of it without any product).  The 64
// contexts are bound by decoding (49 us without the copies, 36 without the products),
// windows of E4M3 rows by the copies (40 us without the products), eight packed tails by
// the products (m16n8k16 takes 8.75 cycles of a quarter of an SM: under a third of
// tcgen05's rate): eight rows of six heads over 261888 tokens take 48.4 us in 4 bits and
// 50.4 in E4M3 with a window of all but one, where paged_e4m3.cu's tcgen05 kernel takes
// 38.1 without a window.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <type_traits>

#include "fp4_rows.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace gqa {
namespace tails {

constexpr int MAX_BATCH = 1024;
constexpr float RESCALE_THRESHOLD = 8.0f;

struct Params {
    const __half* q;
    const uint8_t* cache[2];     // K, V
    const float* scale_dev[2];   // their fp32 scales
    const int32_t* tables;
    const int* ctx_lens;
    int table_stride, num_pages, page, log2_page, max_ctx, batch;
    int ltile;                   // log2 of the keys of a tile
    int R, hq, hkv;
    FastDiv grp;                 // query heads of one KV head
    int nq;                      // packed rows of one KV head (R * grp), at most 48
    int window, sinks;           // window 0: none
    float scale;
    int G;                       // ranges (CTAs)
    float* ws_o;                 // [G][2][8 NT][DH]
    float* ws_ml;                // [G][2][8 NT][2]
    int4* tasks;                 // [G]: what the join has to do (Task)
    int by_unit;                 // a task for each unit, not for each range
    __half* out;
    unsigned* err;
};

// The visible tiles of a sequence: `sink_tiles` from the front, then those from
// `first_tile` to the end of the context.
struct Span {
    int ctx;          // context length
    int lo;           // first key some row's window reaches
    int first_tile;
    int sink_tiles;
    int tiles;
};
__device__ __forceinline__ Span span_of(const Params& P, int raw) {
    Span s;
    s.ctx = min(max(raw, 0), P.max_ctx);
    const int first_row = s.ctx - P.R + 1;   // (keys up to the first row's own)
    s.lo = P.window > 0 && first_row > P.window ? first_row - P.window : 0;
    s.first_tile = s.lo >> P.ltile;
    const int sinks = min(P.sinks, s.first_tile << P.ltile);
    s.sink_tiles = sinks > 0 ? ((sinks - 1) >> P.ltile) + 1 : 0;
    s.tiles = s.ctx > 0 ? s.sink_tiles + ((s.ctx - 1) >> P.ltile) + 1 - s.first_tile : 0;
    return s;
}

// A unit cut into several ranges, for the join: its first piece is in slot
// 2 * range + slot0, the others in the first slots of the ranges behind.  Entry
// `range` or (by_unit) `unit` of Params::tasks as {unit, range * 2 + slot0, pieces, 0};
// no pieces: nothing to join.

// Where each sequence's tiles begin among all.  Up to 32 sequences: lane i of every
// warp holds sequence i, nothing is shared.  More: in shared memory.  (All tiles of all
// units and their LEADs are fewer than 2^30: kMaxTailKeys / 64, and three for each of the
// at most 2^16 units.)
//
// Ranges are equal in tiles and what a piece costs besides: LEAD tiles' time in front of
// each unit's.  (Sixteen windows of 17 tiles: 16.4 us without, 12.2 with one or two, 13.1
// with four; 64 contexts of up to 64 tiles 48.5, 47.6 with one, 47.1, 46.6 with four.)
constexpr int LANES = 32;
constexpr int LEAD = 2;
struct Seqs {
    const int* starts;         // [batch + 1], or null
    int start, tiles, ctx;     // of sequence `lane`; tiles with LEAD in front
    int all;                   // of all sequences
};

__device__ __forceinline__ int scan_warp(int x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += t;
    }
    return x;
}

__device__ __forceinline__ Seqs seqs_small(const Params& P) {
    Seqs q;
    const int lane = threadIdx.x & 31;
    q.starts = nullptr;
    q.ctx = q.tiles = 0;
    if (lane < P.batch) {
        const Span s = span_of(P, P.ctx_lens[lane]);
        q.ctx = s.ctx;
        q.tiles = s.tiles ? s.tiles + LEAD : 0;
    }
    const int incl = scan_warp(q.tiles);
    q.start = incl - q.tiles;
    q.all = __shfl_sync(0xffffffffu, incl, 31);
    return q;
}

// starts[b] = tiles of the sequences before b, for b = 0 .. batch.  All threads of the
// CTA (at least 256), with two barriers.
__device__ __forceinline__ void seqs_large(const Params& P, int* starts, int* totals) {
    constexpr int EACH = MAX_BATCH / 256;
    const int tid = threadIdx.x, warp = tid >> 5;
    int n[EACH], sum = 0, incl = 0;
    if (tid < 256) {
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int b = tid * EACH + i;
            n[i] = b < P.batch ? span_of(P, P.ctx_lens[b]).tiles : 0;
            if (n[i]) n[i] += LEAD;
            sum += n[i];
        }
        incl = scan_warp(sum);
        if ((tid & 31) == 31) totals[warp] = incl;
    }
    __syncthreads();
    if (tid < 256) {
        int at = incl - sum;
        for (int w = 0; w < warp; ++w) at += totals[w];
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int b = tid * EACH + i;
            if (b <= P.batch) starts[b] = at;
            at += n[i];
        }
        if (tid == 255 && P.batch == MAX_BATCH) starts[MAX_BATCH] = at;
    }
    __syncthreads();
}

// G equal ranges over all tiles of all units: range c begins at floor(c total / G).
struct Ranges {
    uint32_t each, more;   // total = each G + more
    int G, total;
    __device__ Ranges(const Params& P, const Seqs& q) {
        total = q.all * P.hkv;
        G = min(P.G, total);
        each = G ? (uint32_t)total / (uint32_t)G : 0;
        more = total - each * G;
    }
    __device__ int begin(int c) const { return c * each + c * more / (uint32_t)max(G, 1); }
    __device__ int of(int pos) const {
        int c = (int)((float)pos * ((float)G / (float)total));   // (or one beside it)
        while (begin(c) > pos) --c;
        while (begin(c + 1) <= pos) ++c;
        return c;
    }
};

// Walks the pieces (unit, tiles [jb, je)) of one range.  (All lanes of a warp.)
struct Pieces {
    int pos, end;     // LEADs counted
    int b, h;         // sequence, KV head
    int jb, je, n;    // tiles of the piece, of the unit
    int unit;         // where the unit begins, its LEAD counted
    bool first;       // the range's first piece
    Span s;
    __device__ bool whole() const { return jb == 0 && je == n; }
    // Sets b, h, n, unit and s to the unit that holds position at.
    __device__ void find(const Params& P, const Seqs& q, int at) {
        h = P.hkv == 1 ? 0 : at / q.all;
        const int in_h = at - h * q.all;
        int start, ctx;
        if (!q.starts) {
            b = 31 - __clz(__ballot_sync(0xffffffffu, q.tiles > 0 && q.start <= in_h));
            start = __shfl_sync(0xffffffffu, q.start, b);
            n = __shfl_sync(0xffffffffu, q.tiles, b);
            ctx = __shfl_sync(0xffffffffu, q.ctx, b);
        } else {
            int lo = 0, hi = P.batch;   // starts[lo] <= in_h < starts[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (q.starts[mid] <= in_h) lo = mid;
                else hi = mid;
            }
            b = lo;
            start = q.starts[lo];
            n = q.starts[lo + 1] - start;
            ctx = P.ctx_lens[b];
        }
        s = span_of(P, ctx);
        unit = at - in_h + start;
        n -= LEAD;
    }
    // A boundary in or right behind a LEAD is the unit's beginning.
    __device__ int boundary(const Params& P, const Seqs& q, int at, int total) {
        if (at >= total) return total;
        find(P, q, at);
        return at <= unit + LEAD ? unit : at;
    }
    __device__ bool next(const Params& P, const Seqs& q, int begin) {
        if (pos >= end) return false;
        first = pos == begin;
        find(P, q, pos);
        jb = max(pos - unit - LEAD, 0);
        je = min(end - unit - LEAD, n);
        pos = je == n ? unit + LEAD + n : end;
        return true;
    }
};

// Wait for a barrier's phase; bounded as mbar_wait.  After a wait that ran out all others
// return at once and the warps go on to their end over whatever is there (every address
// comes from the arguments and the tables), so that the barriers between them, which
// know no limit, are met by all.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                     unsigned* err) {
    if (mbar_try_wait(bar, parity)) return true;
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait(bar, parity)) return true;
        if (n & 15) continue;
        if (*abort) return false;
        const uint64_t now = global_timer_ns();
        if (!t0) t0 = now;
        if (now - t0 > kWaitTimeoutNs) {
            *abort = 1;
            atomicOr(err, kErrWaitTimeout);
            return false;
        }
    }
}
// Barrier `id` of `threads` threads.
__device__ __forceinline__ void meet(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ int tile_key(const Params& P, const Span& s, int j) {
    return (j < s.sink_tiles ? j : s.first_tile + j - s.sink_tiles) << P.ltile;
}

// Element offset of packed row r of a KV head in q / out.
__device__ __forceinline__ long long row_offset(const Params& P, int b, int h, int r, int dh) {
    const int pos = P.grp.div(r);
    return (((long long)b * P.R + pos) * P.hq + h * P.grp.d + (r - pos * P.grp.d)) * dh;
}

// This CTA's range of the tiles.  Nothing of global memory is read or written before the
// kernel in front has completed; this kernel's launch overlaps it.
__device__ __forceinline__ Ranges begin_range(const Params& P, int* starts, int* totals, Pieces& it,
                                              Seqs& seqs) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (P.batch <= LANES) {
        seqs = seqs_small(P);
    } else {
        seqs_large(P, starts, totals);
        seqs = Seqs{starts, 0, 0, 0, starts[P.batch]};
    }
    asm volatile("griddepcontrol.launch_dependents;");
    const Ranges ranges(P, seqs);
    it.pos = it.end = 0;
    if ((int)blockIdx.x < ranges.G) {
        const int total = seqs.all * P.hkv;
        it.pos = it.boundary(P, seqs, ranges.begin(blockIdx.x), total);
        it.end = it.boundary(P, seqs, ranges.begin(blockIdx.x + 1), total);
    }
    return ranges;
}

// What has no tiles (one warp): rows of sequences without a key are zeros; no units of
// theirs, and no cut unit for ranges that get no tiles.
__device__ __forceinline__ void finish_empty(const Params& P, bool idle, int dh) {
    const int lane = threadIdx.x & 31, cta = blockIdx.x;
    if (idle && !P.by_unit && lane == 0) P.tasks[cta] = make_int4(0, 0, 0, 0);
#pragma unroll 1
    for (int b = cta; b < P.batch; b += gridDim.x) {
        const int raw = P.ctx_lens[b];
        if ((raw < 0 || raw > P.max_ctx) && lane == 0) atomicOr(P.err, kErrBadCtxLen);
        if (raw > 0) continue;
        uint4* o = reinterpret_cast<uint4*>(P.out + (long long)b * P.R * P.hq * dh);
#pragma unroll 1
        for (int i = lane; i < P.R * P.hq * dh / 8; i += 32) o[i] = make_uint4(0, 0, 0, 0);
        if (P.by_unit)
#pragma unroll 1
            for (int h = lane; h < P.hkv; h += 32)
                P.tasks[b * P.hkv + h] = make_int4(0, 0, 0, 0);
    }
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The 8 x 8 matrix of 16-bit values the warp holds, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t low_nibbles(uint32_t a, uint32_t b) {
    return (a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u);
}
__device__ __forceinline__ uint32_t high_nibbles(uint32_t a, uint32_t b) {
    return ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
}

// What a tile of a cache looks like in shared memory, and how the products' fragments are
// made of it.  A lane (gid, t) of a warp loads, of K, its share of the key gid: places
// that need not be neighbours, as long as Q has the same order; of V, of four keys, the
// places of gid.
//   key_of(k): the key that stands at place k of the sixteen along the second product's K.
//     Any order does if P has the same one.
//   K::load(x), K::decode(i, h): load x of LOADS, then for each GROUPS eight places as four
//     fp16 pairs; q_of(t, x, i): where Q has these eight, q_at(c) where its places 8 c
//     go; q_place(t, x, i): which they are.
//   pairs(a, b, lo, hi): eight places of two keys as (key a, key b) pairs, the even ones
//     and the odd ones.
//
// A tile's keys: 128 (E4M3 rows of 256: 64, stages of 32 KB); from four eights of packed
// rows on 64, whose scores take half the registers.  (4-bit, heads of 256, 128 and 64
// keys: eight rows of six heads over 128000 37.8 us and 31.2, five rows over 200000 34.0
// and 31.9, four rows 28.3 and 28.6, sixteen windows of two 12.3 and 12.9.  Heads of 128,
// two eights: sixteen contexts of four rows of four heads 34 and 39.  Heads of 128 from four
// eights on, where neither is the better one for all: 32 packed rows, 4-bit, sixteen
// windows of 2000 13.6 and 11.9, one context of 128000 18.0 and 18.6, of 261888 26.4 and
// 28.7, sixteen contexts of 8000 18.2 and 19.4; E4M3, a window of 100000 17.2 and 17.0,
// sixteen of 4096 13.9 and 15.4; 48 packed rows, 4-bit, sixteen windows of 2000 18.8 and
// 15.0, one context of 128000 23.9 and 22.1, sixteen of 8000 25.2 and 24.2; E4M3, a window of
// 100000 23.3 and 21.8, sixteen of 4096 19.5 and 21.9.)
template <bool F8, int DH>
__host__ __device__ constexpr int tile_keys(int nt) {
    return (F8 && DH == 256) || nt >= 4 ? 64 : 128;
}
template <bool F8, int DH, int KEYS>
struct Rows;

// 4-bit rows (fp4_rows.cuh), as they are in memory.
template <int DH, int KEYS>
struct Rows<false, DH, KEYS> {
    static constexpr int TILE = KEYS;
    static constexpr int TILE_BYTES = TILE * fp4::row_bytes(DH);   // of K, or of V
    static constexpr int ROWB = fp4::row_bytes(DH);
    static constexpr int LOADS = 2, GROUPS = DH / 64;
    // Queries: a lane's part of a row so that the eight lanes of a load's phase use
    // different banks (DH 256: quarters padded by 16 bytes; 128: rows).
    static constexpr int Q_ROW = DH == 256 ? 4 * 144 : 272;
    // (Spreads the four keys that a quarter of a warp loads words of over the banks:
    // rows are 36 or 18 words apart.)
    static __device__ __forceinline__ int key_of(int k) {
        return DH == 256 ? k : (k & 6) * 2 + (k & 1) + (k >> 3) * 2;
    }
    static __device__ __forceinline__ int q_at(int c) {
        return DH == 256 ? (c / 8) * 144 + (c % 8) * 16 : c * 16;
    }
    static __device__ __forceinline__ int q_of(int t, int x, int i) {
        return DH == 256 ? t * 144 + x * 64 + i * 16 : t * 32 + x * 128 + i * 16;
    }
    static __device__ __forceinline__ int q_place(int t, int x, int i) {
        return DH == 256 ? t * 64 + x * 32 + i * 8 : x * 64 + t * 16 + i * 8;
    }
    struct K {
        uint32_t w[GROUPS], u[GROUPS / 2];
        __device__ __forceinline__ void load(const uint8_t* tile, int key, int t, int x) {
            const uint8_t* row = tile + key * ROWB;
            if constexpr (DH == 256) {
                const uint4 v = *reinterpret_cast<const uint4*>(row + t * 32 + x * 16);
                w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
                const uint32_t c = fp4::scales2(
                    *reinterpret_cast<const uint16_t*>(row + DH / 2 + t * 4 + x * 2));
                u[0] = __byte_perm(c, 0, 0x1010);
                u[1] = __byte_perm(c, 0, 0x3232);
            } else {
                const uint2 v = *reinterpret_cast<const uint2*>(row + t * 8 + x * 32);
                w[0] = v.x, w[1] = v.y;
                u[0] = fp4::scales2(row[DH / 2 + t + x * 4] * 0x101u);
            }
        }
        __device__ __forceinline__ void decode(int i, uint32_t (&h)[4]) const {
            fp4::decode8(w[i], h);
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = fp4::mul2(h[e], u[i / 2]);
        }
    };
    // (with the pair's scales u)
    static __device__ __forceinline__ void pairs(uint32_t a, uint32_t b, uint32_t u,
                                                 uint32_t (&lo)[4], uint32_t (&hi)[4]) {
        fp4::decode8(low_nibbles(a, b), lo);
        fp4::decode8(high_nibbles(a, b), hi);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            lo[e] = fp4::mul2(lo[e], u);
            hi[e] = fp4::mul2(hi[e], u);
        }
    }
};

// E4M3 rows, in halves of 128 bytes with the 128-byte swizzle: unit u (16 bytes) of row r
// at (u ^ r % 8) * 16.
template <int DH, int KEYS>
struct Rows<true, DH, KEYS> {
    static constexpr int TILE = KEYS;
    static constexpr int HALF_BYTES = TILE * 128, TILE_BYTES = TILE * DH;
    static constexpr int LOADS = DH / 64, GROUPS = 2;
    // (a lane's 64 bytes of each half padded by 16, a row by 64)
    static constexpr int Q_ROW = DH / 128 * 4 * 80 + (DH == 256 ? 64 : 0);
    static __device__ __forceinline__ int key_of(int k) { return k; }
    static __device__ __forceinline__ int q_at(int c) { return c / 4 * 80 + c % 4 * 16; }
    static __device__ __forceinline__ int q_of(int t, int x, int i) {
        return ((x >> 1) * 4 + t) * 80 + (x & 1) * 32 + i * 16;
    }
    static __device__ __forceinline__ int q_place(int t, int x, int i) {
        return (x >> 1) * 128 + t * 32 + (x & 1) * 16 + i * 8;
    }
    static __device__ __forceinline__ int at(int key, int half, int unit) {
        return half * HALF_BYTES + key * 128 + ((unit ^ (key & 7)) << 4);
    }
    static __device__ __forceinline__ uint32_t two(uint32_t v) {   // codes of the low 16 bits
        return fp4::scales2(v);
    }
    struct K {
        uint32_t w[4];
        __device__ __forceinline__ void load(const uint8_t* tile, int key, int t, int x) {
            const uint4 v = *reinterpret_cast<const uint4*>(tile + at(key, x >> 1, 2 * t + (x & 1)));
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        }
        __device__ __forceinline__ void decode(int i, uint32_t (&h)[4]) const {
            h[0] = two(w[2 * i]);
            h[1] = two(w[2 * i] >> 16);
            h[2] = two(w[2 * i + 1]);
            h[3] = two(w[2 * i + 1] >> 16);
        }
    };
    // (four places of a word: lo[0], hi[0], lo[1], hi[1])
    static __device__ __forceinline__ void pairs4(uint32_t a, uint32_t b, uint32_t* lo,
                                                  uint32_t* hi) {
        const uint32_t x = __byte_perm(a, b, 0x5140), y = __byte_perm(a, b, 0x7362);
        lo[0] = two(x);
        hi[0] = two(x >> 16);
        lo[1] = two(y);
        hi[1] = two(y >> 16);
    }
};

// Tensor maps of an E4M3 cache, [num_pages * page, Hkv * DH] codes, K and V.
template <bool F8>
struct Maps {
    CUtensorMap kv[2];
};
template <>
struct Maps<false> {};

// Tiles are dealt to the NG groups in turn, tile n to group n % NG as its tile i = n / NG.
// Its data go to stage n % STAGES of the ring, its barriers are number
// (n % NG) STAGES + i % STAGES of NG STAGES "full" and as many "empty" ones: a group's
// own, so that it sees each of their phases (with a barrier for each stage a group would
// skip the others' phases, and could not tell one it waits for from the one before).
//
// Counted on from tile to tile: the remainders' instructions were most of a copying
// warp's time for a tile (sixteen contexts of four rows, heads of 128: 36 us, 34 so).
template <int NG, int STAGES>
struct Turn {
    uint32_t stage = 0, group = 0, slot = 0, phase = 0;
    __device__ __forceinline__ uint32_t bar() const { return 8 * (group * STAGES + slot); }
    __device__ __forceinline__ void next() {
        if (++stage == STAGES) stage = 0;
        if (++group == NG) {
            group = 0;
            if (++slot == STAGES) slot = 0, phase ^= 1;
        }
    }
    // The group's next.
    __device__ __forceinline__ void next_own() {
        stage = stage + NG < STAGES ? stage + NG : stage + NG - STAGES;
        if (++slot == STAGES) slot = 0, phase ^= 1;
    }
};

// The copies (COPY_WARPS warps): the pages of each tile into the ring.  A copy is an
// instruction of one lane at a time, about 70 cycles each: the 16 copies of a tile of
// 16-token pages are shared out among four warps (one warp's took 1100 cycles a tile of
// head size 128, more than the tile's time at the memory's rate; 62 us instead of 50 for
// 64 contexts of up to 8192 tokens).
constexpr int COPY_WARPS = 4;

template <bool F8, int DH, typename W, int NG, int STAGES>
__device__ __forceinline__ void copy_tiles(const Params& P, const Maps<F8>& maps, Pieces& it,
                                           const Seqs& seqs, uint32_t ring, uint32_t bars,
                                           volatile int* abort_flag, int warp) {
    constexpr int HALVES = F8 ? DH / 128 : 1;     // copies of a page's rows of K (or V)
    constexpr int BYTES = W::TILE_BYTES / W::TILE / HALVES;   // of a row in one copy
    const int lane = threadIdx.x & 31;
    // Rows of a copy, pages of a tile; this lane's is of K or V, page p, half of D.
    const int rows = min(P.page, W::TILE), lppt = max(P.ltile - P.log2_page, 0), ppt = 1 << lppt;
    const int kv = warp & 1, number = lane * (COPY_WARPS / 2) + (warp >> 1);
    const int p = number / HALVES, half = number % HALVES;
    const uint32_t to =
        ring + kv * W::TILE_BYTES + half * (W::TILE_BYTES / HALVES) + p * rows * BYTES;
    const int begin = it.pos;
    Turn<NG, STAGES> at, old;   // the next tile, the oldest in the ring
    uint32_t room = STAGES;     // stages that held none yet
    bool ok = true;
    while (ok && it.next(P, seqs, begin)) {
        const int32_t* table = P.tables + (long long)it.b * P.table_stride;
        // A copy's rows from `key` on hold a key that some row sees.  A tile that the
        // sinks end in, or the window begins in, has pages without one, which may have been
        // given back: their entries are not read, and their places in the stage keep what
        // they held.  (The products' masks go by the key.)
        auto seen = [&](int key) {
            return key < it.s.ctx && (key < P.sinks || key + rows > it.s.lo);
        };
        // Table entries 32 at a time, a lane each, three lots ahead of their use.  (Ordinary
        // loads: the kernel in front may write them while this one is resident already, so
        // they are not read-only for its lifetime.)
        auto entries = [&](int lot) {
            const int e = lot * 32 + lane, j = it.jb + (e >> lppt);
            if (j >= it.je) return 0;
            const int key = tile_key(P, it.s, j) + (e & (ppt - 1)) * rows;
            return seen(key) ? table[key >> P.log2_page] : 0;
        };
        int lot = 0, now = entries(0), next = entries(1), after = entries(2);
#pragma unroll 1
        for (int j = it.jb; j < it.je; ++j) {
            const int e = (j - it.jb) << lppt;
            if (e >> 5 != lot) {
                ++lot;
                now = next;
                next = after;
                after = entries(lot + 2);
            }
            // All that can be known before a stage is free.
            int id = __shfl_sync(0xffffffffu, now, (e & 31) + (p & (ppt - 1)));
            const int key0 = tile_key(P, it.s, j), in_page = key0 & (P.page - 1);
            const bool mine = p < ppt && seen(key0 + p * rows);
            if (mine && (id < 0 || id >= P.num_pages)) {
                atomicOr(P.err, kErrBadPageId);
                id = 0;
            }
            const uint32_t bytes =
                __popc(__ballot_sync(0xffffffffu, mine)) * (rows * BYTES);
            const uint8_t* src = nullptr;
            if constexpr (!F8)
                src = (kv ? P.cache[1] : P.cache[0]) +
                      (((long long)id * P.hkv + it.h) * P.page + in_page) * BYTES;
            const uint32_t full = bars + at.bar(), dst = to + at.stage * (2 * W::TILE_BYTES);
            if (room) {
                --room;
            } else {
                ok = wait(bars + 8 * NG * STAGES + old.bar(), old.phase, abort_flag, P.err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                old.next();
            }
            if (lane == 0) mbar_arrive_expect_tx(full, bytes);
            if (mine) {
                if constexpr (F8)
                    tma_load_2d(dst, &maps.kv[kv], full, it.h * DH + half * 128,
                                id * P.page + in_page);
                else
                    bulk_load(dst, src, rows * BYTES, full);
            }
            at.next();
        }
    }
    if (!ok && lane == 0) {
        // Unwind: every copy in flight lands before the CTA exits.
#pragma unroll 1
        for (int i = 0; i < STAGES; ++i) {
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(bars + old.bar(), old.phase))
                if (global_timer_ns() - t0 > 100000000ull) break;
            old.next();
        }
    }
}

// How a unit is joined, from the piece it begins with; a range whose last piece is no
// cut unit's beginning has none to say.
__device__ __forceinline__ void write_task(const Params& P, const Pieces& it, const Ranges& ranges) {
    const int unit = it.b * P.hkv + it.h, cta = blockIdx.x;
    const bool cut = it.jb == 0 && !it.whole();
    if ((threadIdx.x & 31) == 0 && (cut || (P.by_unit ? it.jb == 0 : it.pos >= it.end)))
        P.tasks[P.by_unit ? unit : cta] =
            make_int4(unit, cta * 2 + (it.first ? 0 : 1),
                      cut ? ranges.of(it.unit + LEAD + it.n - 1) - cta + 1 : 0, 0);
}

// What the copy warps do: the first of them also what concerns the join.
template <bool F8, int DH, typename W, int NG, int STAGES>
__device__ __forceinline__ void bring(const Params& P, const Maps<F8>& maps, int* starts,
                                      int* totals, uint32_t ring, uint32_t bars,
                                      volatile int* abort_flag, int warp) {
    Seqs seqs;
    Pieces it;
    const Ranges ranges = begin_range(P, starts, totals, it, seqs);
    const int begin = it.pos;
    copy_tiles<F8, DH, W, NG, STAGES>(P, maps, it, seqs, ring, bars, abort_flag, warp);
    if (warp) return;
    finish_empty(P, begin == it.end, DH);
    it.pos = begin;
    while (it.next(P, seqs, begin)) write_task(P, it, ranges);
}

// Position of packed row r of a KV head, and whether a row there sees a key.
__device__ __forceinline__ int row_pos(const Params& P, const Span& s, int r) {
    return s.ctx - P.R + min(P.grp.div(r), P.R - 1);
}
__device__ __forceinline__ bool sees(const Params& P, int at, int key) {
    return key <= at && (P.window == 0 || key > at - P.window || key < P.sinks);
}
// Some key of [key0, key0 + n) is hidden from some row; no row sees the key.
__device__ __forceinline__ bool has_edge(const Params& P, const Span& s, int key0, int n) {
    return key0 + n - 1 > s.ctx - P.R ||
           (P.window > 0 && key0 <= s.ctx - 1 - P.window && key0 + n - 1 >= P.sinks);
}
__device__ __forceinline__ bool unseen(const Params& P, const Span& s, int key) {
    return key >= s.ctx || (key < s.lo && key >= P.sinks);
}

// F8: the cache is E4M3, else 4-bit; DH: head size; NT: eights of packed rows.
template <bool F8, int DH, int NT>
struct Config {
    using W = Rows<F8, DH, tile_keys<F8, DH>(NT)>;
    static constexpr int TILE = W::TILE;
    // Two groups of four warps, each group on a tile of its own, so that one's products go
    // on while the other's warps meet, each warp with 32 keys (16 of a tile of 64).
    // (Groups of eight warps with 16 keys and half the registers: 28 us instead of 26 for
    // two rows over 200000 4-bit tokens, 35 instead of 29 for four.)  The warpgroup behind
    // them copies.  Registers: what the launch gives (65536 over the threads, by eights)
    // moved from the copies to the products.
    static constexpr int NG = 2;
    static constexpr int GW = 4;
    static constexpr int KZ = TILE / 16 / GW;      // sixteens of keys of a warp
    static constexpr int NW = GW * NG;
    static constexpr int THREADS = 32 * NW + 128;
    static constexpr int REGS_PRODUCTS = 224;
    static constexpr int REGS_COPIES = 56;
    static constexpr int REGS_LAUNCH = 65536 / THREADS / 8 * 8;
    static_assert(32 * NW * REGS_PRODUCTS + 128 * REGS_COPIES <= THREADS * REGS_LAUNCH, "registers");

    static constexpr int STAGE = 2 * W::TILE_BYTES;
    static constexpr int ROWS = 8 * NT;
    // V: slices of 64 places, and the shares of a tile's keys that then occupy a group.
    static constexpr int SLICES = DH / 64, SHARES = GW / SLICES;
    static constexpr int SOURCES = NG * SHARES;    // warps that sum the same places
    static constexpr int P_ROW = TILE * 2 + 16;    // P^T: rows of a tile's keys, padded
    static constexpr int P_BYTES = 2 * NG * ROWS * P_ROW;   // (of two tiles: see below)
    static constexpr int JOIN_ROW = DH / 4 + 4;    // floats of a row in one round of the join

    static constexpr int OFF_Q = 0;
    static constexpr int OFF_P = OFF_Q + ROWS * W::Q_ROW;   // [NG][2][ROWS]
    static constexpr int OFF_JOIN = OFF_P;                  // [SOURCES][ROWS], when P is done with
    static constexpr int JOIN_BYTES = SOURCES * ROWS * JOIN_ROW * 4;
    static constexpr int OFF_MAX = OFF_P + (P_BYTES > JOIN_BYTES ? P_BYTES : JOIN_BYTES);   // [NW][ROWS]
    static constexpr int OFF_REF = OFF_MAX + NW * ROWS * 4;               // [NG][ROWS]
    static constexpr int OFF_STARTS = OFF_REF + NG * ROWS * 4;
    static constexpr int OFF_TOTALS = OFF_STARTS + (MAX_BATCH + 1) * 4;
    static constexpr int MAX_STAGES = 10;
    static constexpr int OFF_BARS = (OFF_TOTALS + 8 * 4 + 7) / 8 * 8;
    static constexpr int OFF_FLAG = OFF_BARS + 2 * NG * MAX_STAGES * 8;   // [NG][2]
    static constexpr int OFF_ABORT = OFF_FLAG + NG * 2 * 4;
    static constexpr int OFF_RING = (OFF_ABORT + 4 + 1023) / 1024 * 1024;
    // The bytes in flight set the copy rate: all that is left, up to 192 KB.
    static constexpr int MOST = 196608 / STAGE < MAX_STAGES ? 196608 / STAGE : MAX_STAGES;
    static constexpr int FIT = (232448 - 1024 - OFF_RING) / STAGE;
    static constexpr int STAGES = FIT < MOST ? FIT : MOST;
    static constexpr int BYTES = 1024 + OFF_RING + STAGES * STAGE;   // (1024: its alignment)
    static_assert(STAGES >= 2 && BYTES <= 232448, "shared memory");
};

// Dynamic shared memory from a multiple of 1024 on (the swizzle goes by the address).
__device__ __forceinline__ uint8_t* aligned_smem(uint8_t* raw) {
    return raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
}

template <bool F8, int DH, int NT>
__global__ void __launch_bounds__(Config<F8, DH, NT>::THREADS, 1)
split_kernel(const __grid_constant__ Maps<F8> maps, const Params P) {
    using C = Config<F8, DH, NT>;
    using W = typename C::W;
    constexpr int TILE = C::TILE;
    constexpr int ROWS = C::ROWS, STAGES = C::STAGES, NG = C::NG, NW = C::NW;
    constexpr int GW = C::GW, KZ = C::KZ;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = aligned_smem(smem_raw);
    int* starts = reinterpret_cast<int*>(smem + C::OFF_STARTS);
    int* totals = reinterpret_cast<int*>(smem + C::OFF_TOTALS);
    const uint32_t bars = smem_u32(smem + C::OFF_BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NG * STAGES; ++i) {
            mbar_init(bars + 8 * i, COPY_WARPS);
            mbar_init(bars + 8 * (NG * STAGES + i), GW);
        }
        for (int i = 0; i < NG * 2; ++i) reinterpret_cast<int*>(smem + C::OFF_FLAG)[i] = 0;
        *abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    const int cta = blockIdx.x;

    if (warp >= NW) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_COPIES));
        bring<F8, DH, W, NG, STAGES>(P, maps, starts, totals, smem_u32(smem) + C::OFF_RING, bars,
                                  abort_flag, warp - NW);
    } else {
        // ------------------------------------------------------------ products
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_PRODUCTS));
        Seqs seqs;
        Pieces it;
        begin_range(P, starts, totals, it, seqs);
        const int begin = it.pos;
        const int group = warp / GW, gwarp = warp % GW;
        const int gid = lane >> 2, t = lane & 3;
        const int slice = gwarp % C::SLICES, share = gwarp / C::SLICES;
        uint8_t* const sq = smem + C::OFF_Q;
        float* const smax = reinterpret_cast<float*>(smem + C::OFF_MAX);   // [NW][ROWS]
        float* const sref = reinterpret_cast<float*>(smem + C::OFF_REF);   // [NG][ROWS]
        float* const join = reinterpret_cast<float*>(smem + C::OFF_JOIN);
        volatile int* const flag = reinterpret_cast<volatile int*>(smem + C::OFF_FLAG) + group * 2;
        auto meet_all = [&]() { meet(1, 32 * NW); };
        auto meet_group = [&]() { meet(2 + group, 32 * GW); };
        const float sl2 = P.scale * *P.scale_dev[0] * 1.4426950408889634f;
        const float vscale = *P.scale_dev[1];
        uint32_t n = 0;     // tiles of the CTA so far
        Turn<NG, STAGES> at;
        at.stage = at.group = group;
        uint32_t mine = 0;  // tiles of the group so far
        while (it.next(P, seqs, begin)) {
            const Span s = it.s;
            // Q, all loads under way together.
            {
                constexpr int EACH = (ROWS * DH / 8 + 32 * NW - 1) / (32 * NW);
                uint4 v[EACH];
#pragma unroll
                for (int x = 0; x < EACH; ++x) {
                    const int i = threadIdx.x + x * 32 * NW, r = i / (DH / 8), c = i % (DH / 8);
                    v[x] = r < P.nq
                               ? *reinterpret_cast<const uint4*>(
                                     P.q + row_offset(P, it.b, it.h, r, DH) + c * 8)
                               : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int x = 0; x < EACH; ++x) {
                    const int i = threadIdx.x + x * 32 * NW, r = i / (DH / 8), c = i % (DH / 8);
                    if (r < ROWS)
                        *reinterpret_cast<uint4*>(sq + r * W::Q_ROW + W::q_at(c)) = v[x];
                }
            }
            meet_all();
            if (gwarp == 0)
                for (int i = lane; i < ROWS; i += 32) sref[group * ROWS + i] = -INFINITY;
            meet_group();
            float o[4][NT][4];              // places 8 gid + 2 i, + 1 of the slice; rows 2 t, 2 t + 1
            float l[NT][2];                 // of rows 2 t, 2 t + 1
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][nt][e] = 0.f;
            }

            const uint32_t n0 = n;   // the piece's first tile
            n += it.je - it.jb;
#pragma unroll 1
            for (int j = it.jb + (int)((group + NG - n0 % NG) % NG); j < it.je; j += NG) {
                const uint32_t full = bars + at.bar();
                wait(full, at.phase, abort_flag, P.err);
                __syncwarp();
                // P of this tile and the last one lie side by side: a warp that is ahead writes
                // beside what others still read, and one barrier a tile is enough.
                uint8_t* const pt =
                    smem + C::OFF_P + (group * 2 + (mine & 1)) * ROWS * C::P_ROW;
                const int key0 = tile_key(P, s, j);
                const bool edge = has_edge(P, s, key0, TILE);
                const uint8_t* kst = smem + C::OFF_RING + at.stage * C::STAGE;
                const uint8_t* vst = kst + W::TILE_BYTES;
                // ---- scores of keys key_of(gid) and key_of(gid + 8) of each sixteen
                float sc[KZ][NT][4];
#pragma unroll
                for (int z = 0; z < KZ; ++z) {
                    const int k0 = (gwarp * KZ + z) * 16;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[z][nt][e] = 0.f;
#pragma unroll
                    for (int x = 0; x < W::LOADS; ++x) {
                        typename W::K key[2];
                        key[0].load(kst, k0 + W::key_of(gid), t, x);
                        key[1].load(kst, k0 + W::key_of(gid + 8), t, x);
#pragma unroll
                        for (int i = 0; i < W::GROUPS; ++i) {
                            uint32_t a[4], b[4];
                            key[0].decode(i, a);
                            key[1].decode(i, b);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                const uint4 qv = *reinterpret_cast<const uint4*>(
                                    sq + (nt * 8 + gid) * W::Q_ROW + W::q_of(t, x, i));
                                mma16816(sc[z][nt], a[0], b[0], a[1], b[1], qv.x, qv.y);
                                mma16816(sc[z][nt], a[2], b[2], a[3], b[3], qv.z, qv.w);
                            }
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[z][nt][e] *= sl2;
                }
                if (edge) {
#pragma unroll
                    for (int z = 0; z < KZ; ++z)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (!sees(P, row_pos(P, s, nt * 8 + 2 * t + (e & 1)),
                                          key0 + (gwarp * KZ + z) * 16 +
                                              W::key_of(gid + (e & 2) * 4)))
                                    sc[z][nt][e] = -INFINITY;
                }
                // ---- P by the references as they stand
                float mref[NT][2];   // the group's references of rows 2 t, 2 t + 1
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float2 m = *reinterpret_cast<const float2*>(sref + group * ROWS +
                                                                      nt * 8 + 2 * t);
                    mref[nt][0] = m.x;
                    mref[nt][1] = m.y;
                }
                bool exceed = false;
#pragma unroll
                for (int z = 0; z < KZ; ++z)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            exceed |= sc[z][nt][e] > mref[nt][e & 1] + RESCALE_THRESHOLD;
                if (__any_sync(0xffffffffu, exceed) && lane == 0) flag[mine & 1] = (int)mine + 1;
                // The P of a strip, transposed: keys 2 t, 2 t + 1 (and 8 more) of packed
                // row gid.  Returns the rows' sums in ls.
                auto put_p = [&](float (&ls)[NT][2]) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float m0 = mref[nt][0] == -INFINITY ? 0.f : mref[nt][0];
                        const float m1 = mref[nt][1] == -INFINITY ? 0.f : mref[nt][1];
                        ls[nt][0] = ls[nt][1] = 0.f;
#pragma unroll
                        for (int z = 0; z < KZ; ++z) {
                            const float p0 = ex2(sc[z][nt][0] - m0), p1 = ex2(sc[z][nt][1] - m1);
                            const float p2 = ex2(sc[z][nt][2] - m0), p3 = ex2(sc[z][nt][3] - m1);
                            ls[nt][0] += p0 + p2;
                            ls[nt][1] += p1 + p3;
                            uint8_t* to = pt + (nt * 8 + gid) * C::P_ROW +
                                          ((gwarp * KZ + z) * 16 + 2 * t) * 2;
                            *reinterpret_cast<uint32_t*>(to) = transpose8(pack_half2(p0, p1));
                            *reinterpret_cast<uint32_t*>(to + 16) = transpose8(pack_half2(p2, p3));
                        }
                    }
                };
                float ls[NT][2];
                put_p(ls);
                meet_group();
                if (flag[mine & 1] == (int)mine + 1) {
                    // A reference moves: the tile's largest scores of all warps.
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float m = fmaxf(sc[0][nt][e], sc[0][nt][e + 2]);
#pragma unroll
                            for (int z = 1; z < KZ; ++z)
                                m = fmaxf(m, fmaxf(sc[z][nt][e], sc[z][nt][e + 2]));
#pragma unroll
                            for (int x = 4; x < 32; x <<= 1)
                                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
                            if (gid == 0) smax[warp * ROWS + nt * 8 + 2 * t + e] = m;
                        }
                    meet_group();
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float f[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float* from = smax + group * GW * ROWS + nt * 8 + 2 * t + e;
                            float m = from[0];
#pragma unroll
                            for (int x = 1; x < GW; ++x) m = fmaxf(m, from[x * ROWS]);
                            f[e] = 1.f;
                            if (m > mref[nt][e] + RESCALE_THRESHOLD) {
                                f[e] = ex2(mref[nt][e] - m);
                                mref[nt][e] = m;
                            }
                            l[nt][e] *= f[e];
                        }
                        if (gwarp == 0 && gid == 0)
                            *reinterpret_cast<float2*>(sref + group * ROWS + nt * 8 + 2 * t) =
                                make_float2(mref[nt][0], mref[nt][1]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            o[i][nt][0] *= f[0];
                            o[i][nt][1] *= f[1];
                            o[i][nt][2] *= f[0];
                            o[i][nt][3] *= f[1];
                        }
                    }
                    put_p(ls);
                    meet_group();   // (also: the maxima have been read)
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    l[nt][0] += ls[nt][0];
                    l[nt][1] += ls[nt][1];
                }
                // ---- O += V^T P^T over the share's keys, 16 at a time
                constexpr int STEPS = TILE / 16 / C::SHARES;
                // 4-bit: scales of a step's pairs of keys.  Keys no row sees may hold anything:
                // scales of zero, and E4M3 codes of zero.  NaN scales of keys that some rows
                // see and others do not are zeros too (0 * NaN), and the rows that see them
                // are made NaN below.
                uint32_t c01[STEPS], c23[STEPS];
                bool apart = false;
                if constexpr (!F8) {
                    const uint32_t pick = (gid >> 1) | ((gid >> 1) + 4) << 4;
#pragma unroll
                    for (int x = 0; x < STEPS; ++x) {
                        uint32_t u[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            u[e] = *reinterpret_cast<const uint32_t*>(
                                vst + ((share * STEPS + x) * 16 +
                                       W::key_of(2 * t + (e & 1) + (e >> 1) * 8)) * W::ROWB +
                                DH / 2 + slice * 4);
                        c01[x] = __byte_perm(u[0], u[1], pick) & 0xffff;
                        c23[x] = __byte_perm(u[2], u[3], pick) & 0xffff;
                    }
                    if (edge) {
#pragma unroll
                        for (int x = 0; x < STEPS; ++x)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int key = key0 + (share * STEPS + x) * 16 +
                                                W::key_of(2 * t + (e & 1) + (e >> 1) * 8);
                                uint32_t& c = e < 2 ? c01[x] : c23[x];
                                const uint32_t in = 0x7fu << (e & 1) * 8;
                                const bool none = unseen(P, s, key), nan = (c & in) == in;
                                if (none || nan) c &= ~(0xffu << (e & 1) * 8);
                                apart |= nan && !none;
                            }
                    }
                }
#pragma unroll
                for (int x = 0; x < STEPS; x += 2) {
                    uint32_t pf[NT][4];   // B operands of two steps
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint32_t from = smem_u32(pt) + (nt * 8 + (lane & 7)) * C::P_ROW +
                                              ((share * STEPS + x) * 16 + (lane >> 3) * 8) * 2;
                        asm volatile(
                            "ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                            : "=r"(pf[nt][0]), "=r"(pf[nt][1]), "=r"(pf[nt][2]), "=r"(pf[nt][3])
                            : "r"(from)
                            : "memory");
                    }
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int k0 = (share * STEPS + x + y) * 16;
                        uint32_t lo0[4], hi0[4], lo1[4], hi1[4];
                        if constexpr (F8) {
                            uint2 w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int key = k0 + 2 * t + (e & 1) + (e >> 1) * 8;
                                w[e] = *reinterpret_cast<const uint2*>(
                                    vst + W::at(key, slice >> 1, (slice & 1) * 4 + (gid >> 1)) +
                                    (gid & 1) * 8);
                                if (edge && unseen(P, s, key0 + key)) w[e] = make_uint2(0, 0);
                            }
                            W::pairs4(w[0].x, w[1].x, lo0, hi0);
                            W::pairs4(w[0].y, w[1].y, lo0 + 2, hi0 + 2);
                            W::pairs4(w[2].x, w[3].x, lo1, hi1);
                            W::pairs4(w[2].y, w[3].y, lo1 + 2, hi1 + 2);
                        } else {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = *reinterpret_cast<const uint32_t*>(
                                    vst + (k0 + W::key_of(2 * t + (e & 1) + (e >> 1) * 8)) * W::ROWB +
                                    slice * 32 + gid * 4);
                            W::pairs(w[0], w[1], fp4::scales2(c01[x + y]), lo0, hi0);
                            W::pairs(w[2], w[3], fp4::scales2(c23[x + y]), lo1, hi1);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816(o[i][nt], lo0[i], hi0[i], lo1[i], hi1[i], pf[nt][2 * y],
                                         pf[nt][2 * y + 1]);
                    }
                }
                if constexpr (!F8) if (__any_sync(0xffffffffu, apart)) {
                    // All places of a lane lie in one block of 16.
                    uint32_t poison = 0;
#pragma unroll 1
                    for (int k = share * STEPS * 16; k < (share + 1) * STEPS * 16; ++k) {
                        const int key = key0 + k;
                        if ((vst[k * W::ROWB + DH / 2 + slice * 4 + (gid >> 1)] & 0x7f) != 0x7f)
                            continue;
#pragma unroll
                        for (int r = 0; r < 2 * NT; ++r)
                            if (sees(P, row_pos(P, s, (r >> 1) * 8 + 2 * t + (r & 1)), key))
                                poison |= 1u << r;
                    }
#pragma unroll
                    for (int r = 0; r < 2 * NT; ++r)
                        if (poison >> r & 1)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                o[i][r >> 1][r & 1] = o[i][r >> 1][(r & 1) + 2] = NAN;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(full + 8 * NG * STAGES);
                at.next_own();
                ++mine;
            }

            // ---------------------------------------------------------- end of the piece
            // Sums of the rows' weights by warp; then, from them and the references, each row's
            // factors for the groups' O and what its sums are to be divided by.
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1)
                        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], x);
                    if (gid == 0) {
                        smax[warp * ROWS + nt * 8 + 2 * t + e] = l[nt][e];
                    }
                }
            const int slot = cta * 2 + (it.first ? 0 : 1);
            const bool whole = it.whole();
            meet_all();
            if (threadIdx.x < ROWS) {
                const int row = threadIdx.x;
                float M = sref[row];
#pragma unroll
                for (int g = 1; g < NG; ++g) M = fmaxf(M, sref[g * ROWS + row]);
                float sum = 0.f, f[NG];
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float mg = sref[g * ROWS + row];
                    f[g] = mg == -INFINITY ? 0.f : ex2(mg - M);
                    float lg = 0.f;
#pragma unroll
                    for (int x = 0; x < GW; ++x) lg += smax[(g * GW + x) * ROWS + row];
                    sum = fmaf(f[g], lg, sum);
                }
                if (!whole && row < P.nq)
                    *reinterpret_cast<float2*>(P.ws_ml + ((long long)slot * ROWS + row) * 2) =
                        make_float2(M, sum);
                // (a NaN sum is a NaN row, a sum of zero a row that sees nothing)
                const float unit = !whole ? 1.f : sum == 0.f ? 0.f : vscale / sum;
#pragma unroll
                for (int g = 0; g < NG; ++g) sref[g * ROWS + row] = f[g] * unit;
            }
            // O in four rounds, a quarter of each lane's places each: the sources' shares
            // go through shared memory and are added in order.
#pragma unroll 1
            for (int r = 0; r < 4; ++r) {
                float* to = join + (group * C::SHARES + share) * ROWS * C::JOIN_ROW + slice * 16 +
                            gid * 2;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<float2*>(to + (nt * 8 + 2 * t + e) * C::JOIN_ROW) =
                            make_float2(o[0][nt][e], o[0][nt][e + 2]);
                meet_all();
#pragma unroll 1
                for (int i = threadIdx.x; i < ROWS * DH / 8; i += 32 * NW) {
                    const int row = i / (DH / 8), at = i % (DH / 8);   // at: slice, gid
                    if (row >= P.nq) break;
                    float2 a = make_float2(0.f, 0.f);
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        float2 v = make_float2(0.f, 0.f);
#pragma unroll
                        for (int x = 0; x < C::SHARES; ++x) {
                            const float2 y = *reinterpret_cast<const float2*>(
                                join + ((g * C::SHARES + x) * ROWS + row) * C::JOIN_ROW + at * 2);
                            v.x += y.x;
                            v.y += y.y;
                        }
                        const float f = sref[g * ROWS + row];
                        a.x = fmaf(f, v.x, a.x);
                        a.y = fmaf(f, v.y, a.y);
                    }
                    const int d = at * 8 + r * 2;
                    if (whole)
                        *reinterpret_cast<uint32_t*>(
                            P.out + row_offset(P, it.b, it.h, row, DH) + d) =
                            pack_half2(a.x, a.y);
                    else
                        *reinterpret_cast<float2*>(
                            P.ws_o + ((long long)slot * ROWS + row) * DH + d) = a;
                }
                meet_all();
#pragma unroll
                for (int i = 0; i < 3; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[i][nt][e] = o[i + 1][nt][e];
            }
        }
    }
    __syncthreads();
}

// Up to eight packed rows: every warp by itself, 32 keys of a tile, all of D, with its own
// references, until the end of a piece.  (P never leaves the warp, and nothing meets in
// a tile; more rows' sums of all of D do not fit a warp's registers.  64 contexts of one
// row, heads of 128: 47 us, 54 with the kernel above; one row over 261888 23.7 and 23.8.)
template <bool F8, int DH>
struct Narrow {
    using W = Rows<F8, DH, tile_keys<F8, DH>(1)>;
    static constexpr int NG = 2;                     // tiles under way
    static constexpr int GW = 4;                     // warps of a tile
    static constexpr int KZ = W::TILE / 16 / GW;     // sixteens of keys of a warp
    static constexpr int NW = NG * GW;
    static constexpr int THREADS = 32 * NW + 128;
    static constexpr int REGS_PRODUCTS = 224, REGS_COPIES = 56;
    static constexpr int REGS_LAUNCH = 65536 / THREADS / 8 * 8;
    static_assert(32 * NW * REGS_PRODUCTS + 128 * REGS_COPIES <= THREADS * REGS_LAUNCH, "registers");
    static constexpr int STAGE = 2 * W::TILE_BYTES;
    static constexpr int STAGES = 196608 / STAGE;    // 180 KB (4-bit) or 192 KB (E4M3)
    // One round of the join: eight places of every gid, of all warps.
    static constexpr int JOIN_ROW = 64 + 4;
    static constexpr int OFF_JOIN = 0;                                   // [NW][8][JOIN_ROW]
    static constexpr int OFF_ML = OFF_JOIN + NW * 8 * JOIN_ROW * 4;       // [NW][8][2]
    static constexpr int OFF_STARTS = OFF_ML + NW * 8 * 8;
    static constexpr int OFF_TOTALS = OFF_STARTS + (MAX_BATCH + 1) * 4;
    static constexpr int OFF_BARS = (OFF_TOTALS + 8 * 4 + 7) / 8 * 8;
    static constexpr int OFF_ABORT = OFF_BARS + 2 * NG * STAGES * 8;
    static constexpr int OFF_RING = (OFF_ABORT + 4 + 1023) / 1024 * 1024;
    static constexpr int BYTES = 1024 + OFF_RING + STAGES * STAGE;   // (1024: its alignment)
    static_assert(BYTES <= 232448, "shared memory");
};

template <bool F8, int DH>
__global__ void __launch_bounds__(Narrow<F8, DH>::THREADS, 1)
narrow_kernel(const __grid_constant__ Maps<F8> maps, const Params P) {
    using C = Narrow<F8, DH>;
    using W = typename C::W;
    constexpr int STAGES = C::STAGES, NG = C::NG, NW = C::NW;
    constexpr int MT = DH / 16, KZ = C::KZ;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = aligned_smem(smem_raw);
    int* starts = reinterpret_cast<int*>(smem + C::OFF_STARTS);
    int* totals = reinterpret_cast<int*>(smem + C::OFF_TOTALS);
    const uint32_t bars = smem_u32(smem + C::OFF_BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NG * STAGES; ++i) {
            mbar_init(bars + 8 * i, COPY_WARPS);
            mbar_init(bars + 8 * (NG * STAGES + i), C::GW);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    if (warp >= NW) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_COPIES));
        bring<F8, DH, W, NG, STAGES>(P, maps, starts, totals, smem_u32(smem) + C::OFF_RING, bars,
                                  abort_flag, warp - NW);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_PRODUCTS));
        Seqs seqs;
        Pieces it;
        begin_range(P, starts, totals, it, seqs);
        const int begin = it.pos;
        const int group = warp / C::GW, gwarp = warp % C::GW;
        const int gid = lane >> 2, t = lane & 3;
        float* const join = reinterpret_cast<float*>(smem + C::OFF_JOIN);
        float* const sml = reinterpret_cast<float*>(smem + C::OFF_ML);
        auto meet_all = [&]() { meet(1, 32 * NW); };
        const float sl2 = P.scale * *P.scale_dev[0] * 1.4426950408889634f;
        const float vscale = *P.scale_dev[1];
        uint32_t n = 0;     // tiles of the CTA so far
        Turn<NG, STAGES> at;
        at.stage = at.group = group;
        while (it.next(P, seqs, begin)) {
            const Span s = it.s;
            // The lane's places of row gid: the products' B operands.
            uint4 q[DH / 32];
            {
                const bool there = gid < P.nq;
                const __half* src = P.q + (there ? row_offset(P, it.b, it.h, gid, DH) : 0);
#pragma unroll
                for (int i = 0; i < DH / 32; ++i)
                    q[i] = there ? *reinterpret_cast<const uint4*>(
                                       src + W::q_place(t, i / W::GROUPS, i % W::GROUPS))
                                 : make_uint4(0, 0, 0, 0);
            }
            float o[MT][4];
            float mref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

            const uint32_t n0 = n;   // the piece's first tile
            n += it.je - it.jb;
#pragma unroll 1
            for (int j = it.jb + (int)((group + NG - n0 % NG) % NG); j < it.je; j += NG) {
                const uint32_t full = bars + at.bar();
                wait(full, at.phase, abort_flag, P.err);
                __syncwarp();
                const int w0 = gwarp * 16 * KZ;   // the warp's first key of the tile
                const int k0 = tile_key(P, s, j) + w0;
                const uint8_t* kst = smem + C::OFF_RING + at.stage * C::STAGE;
                const uint8_t* vst = kst + W::TILE_BYTES;
                const bool edge = has_edge(P, s, k0, 16 * KZ);
                // ---- scores of keys key_of(gid) and key_of(gid + 8) of each sixteen
                float sc[KZ][2][4];
#pragma unroll
                for (int z = 0; z < KZ; ++z)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[z][x][e] = 0.f;
#pragma unroll
                for (int x = 0; x < W::LOADS; ++x) {
                    typename W::K key[KZ][2];
#pragma unroll
                    for (int z = 0; z < KZ; ++z)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            key[z][e].load(kst, w0 + z * 16 + W::key_of(gid + 8 * e), t, x);
#pragma unroll
                    for (int i = 0; i < W::GROUPS; ++i)
#pragma unroll
                        for (int z = 0; z < KZ; ++z) {
                            uint32_t a[4], b[4];
                            key[z][0].decode(i, a);
                            key[z][1].decode(i, b);
                            const uint4 qv = q[x * W::GROUPS + i];
                            mma16816(sc[z][0], a[0], b[0], a[1], b[1], qv.x, qv.y);
                            mma16816(sc[z][1], a[2], b[2], a[3], b[3], qv.z, qv.w);
                        }
                }
                float sv[KZ][4];
#pragma unroll
                for (int z = 0; z < KZ; ++z)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sv[z][e] = (sc[z][0][e] + sc[z][1][e]) * sl2;
                if (edge) {
#pragma unroll
                    for (int z = 0; z < KZ; ++z)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!sees(P, row_pos(P, s, 2 * t + (e & 1)),
                                      k0 + z * 16 + W::key_of(gid + (e & 2) * 4)))
                                sv[z][e] = -INFINITY;
                }
                bool exceed = false;
#pragma unroll
                for (int z = 0; z < KZ; ++z)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        exceed |= sv[z][e] > mref[e & 1] + RESCALE_THRESHOLD;
                if (__any_sync(0xffffffffu, exceed)) {
                    float f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = fmaxf(sv[0][e], sv[0][e + 2]);
#pragma unroll
                        for (int z = 1; z < KZ; ++z) m = fmaxf(m, fmaxf(sv[z][e], sv[z][e + 2]));
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1)
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
                        f[e] = 1.f;
                        if (m > mref[e] + RESCALE_THRESHOLD) {
                            f[e] = ex2(mref[e] - m);
                            mref[e] = m;
                        }
                        l[e] *= f[e];
                    }
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        o[i][0] *= f[0];
                        o[i][1] *= f[1];
                        o[i][2] *= f[0];
                        o[i][3] *= f[1];
                    }
                }
                // ---- P, transposed into the second product's B operand
                uint32_t pf[KZ][2];
                {
                    const float m0 = mref[0] == -INFINITY ? 0.f : mref[0];
                    const float m1 = mref[1] == -INFINITY ? 0.f : mref[1];
#pragma unroll
                    for (int z = 0; z < KZ; ++z) {
                        const float p0 = ex2(sv[z][0] - m0), p1 = ex2(sv[z][1] - m1);
                        const float p2 = ex2(sv[z][2] - m0), p3 = ex2(sv[z][3] - m1);
                        l[0] += p0 + p2;
                        l[1] += p1 + p3;
                        pf[z][0] = transpose8(pack_half2(p0, p1));
                        pf[z][1] = transpose8(pack_half2(p2, p3));
                    }
                }
                // ---- O += V^T P^T
                // Keys no row sees may hold anything: their codes, or 4-bit scales, are zeros.
                // NaN scales of keys that some rows see and others do not are zeros too (0 *
                // NaN), and the rows that see them are made NaN below.
                bool apart = false;
                if constexpr (F8) {
#pragma unroll
                    for (int z = 0; z < KZ; ++z)
#pragma unroll
                        for (int h = 0; h < DH / 128; ++h) {
                            uint4 w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int key = w0 + z * 16 + 2 * t + (e & 1) + (e >> 1) * 8;
                                w[e] = *reinterpret_cast<const uint4*>(vst + W::at(key, h, gid));
                            }
                            if (edge) {
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (unseen(P, s, k0 + z * 16 + 2 * t + (e & 1) + (e >> 1) * 8))
                                        w[e] = make_uint4(0, 0, 0, 0);
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                auto word = [&](const uint4& v) {
                                    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
                                };
                                uint32_t lo0[2], hi0[2], lo1[2], hi1[2];
                                W::pairs4(word(w[0]), word(w[1]), lo0, hi0);
                                W::pairs4(word(w[2]), word(w[3]), lo1, hi1);
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    mma16816(o[h * 8 + 2 * i + e], lo0[e], hi0[e], lo1[e], hi1[e],
                                             pf[z][0], pf[z][1]);
                            }
                        }
                } else {
                    constexpr int VW = DH / 64;   // words of a lane and key
                    uint32_t c[KZ][4];            // a scale for each 16 values
#pragma unroll
                    for (int z = 0; z < KZ; ++z)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint8_t* at =
                                vst +
                                (w0 + z * 16 + W::key_of(2 * t + (e & 1) + (e >> 1) * 8)) * W::ROWB +
                                DH / 2 + gid * (DH / 128);
                            if constexpr (DH == 256)
                                c[z][e] = *reinterpret_cast<const uint16_t*>(at);
                            else
                                c[z][e] = *at;
                        }
                    if (edge) {
#pragma unroll
                        for (int z = 0; z < KZ; ++z)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int k = z * 16 + W::key_of(2 * t + (e & 1) + (e >> 1) * 8);
                                if (unseen(P, s, k0 + k)) c[z][e] = 0;
#pragma unroll
                                for (int y = 0; y < DH / 128; ++y)
                                    if ((c[z][e] >> 8 * y & 0x7f) == 0x7f) {
                                        apart = true;
                                        c[z][e] &= ~(0xffu << 8 * y);
                                    }
                            }
                    }
#pragma unroll
                    for (int z = 0; z < KZ; ++z) {
                        uint32_t w[4][VW];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint8_t* row =
                                vst +
                                (w0 + z * 16 + W::key_of(2 * t + (e & 1) + (e >> 1) * 8)) * W::ROWB;
                            if constexpr (DH == 256) {
                                const uint4 v = *reinterpret_cast<const uint4*>(row + gid * 16);
                                w[e][0] = v.x, w[e][1] = v.y, w[e][2] = v.z, w[e][3] = v.w;
                            } else {
                                const uint2 v = *reinterpret_cast<const uint2*>(row + gid * 8);
                                w[e][0] = v.x, w[e][1] = v.y;
                            }
                        }
                        // (words 2 i and 2 i + 1 share a scale)
                        uint32_t u01[DH / 128], u23[DH / 128];
#pragma unroll
                        for (int y = 0; y < DH / 128; ++y) {
                            u01[y] = fp4::scales2(__byte_perm(c[z][0], c[z][1], y ? 0x0051 : 0x0040));
                            u23[y] = fp4::scales2(__byte_perm(c[z][2], c[z][3], y ? 0x0051 : 0x0040));
                        }
#pragma unroll
                        for (int i = 0; i < VW; ++i) {
                            uint32_t lo0[4], hi0[4], lo1[4], hi1[4];
                            W::pairs(w[0][i], w[1][i], u01[i / 2], lo0, hi0);
                            W::pairs(w[2][i], w[3][i], u23[i / 2], lo1, hi1);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                mma16816(o[4 * i + e], lo0[e], hi0[e], lo1[e], hi1[e], pf[z][0],
                                         pf[z][1]);
                        }
                    }
                }
                if constexpr (!F8) if (__any_sync(0xffffffffu, apart)) {
                    uint32_t poison = 0;   // bits: block * 2 + row
#pragma unroll 1
                    for (int k = 0; k < 16 * KZ; ++k)
#pragma unroll
                        for (int y = 0; y < DH / 128; ++y)
                            if ((vst[(w0 + k) * W::ROWB + DH / 2 + gid * (DH / 128) + y] & 0x7f) == 0x7f)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (sees(P, row_pos(P, s, 2 * t + e), k0 + k))
                                        poison |= 1u << (2 * y + e);
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (poison >> (i / 8 * 2 + e) & 1) o[i][e] = o[i][e + 2] = NAN;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(full + 8 * NG * STAGES);
                at.next_own();
            }

            // ---------------------------------------------------------- end of the piece
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], x);
                if (gid == 0)
                    *reinterpret_cast<float2*>(sml + (warp * 8 + 2 * t + e) * 2) =
                        make_float2(mref[e], l[e]);
            }
            // O in rounds of a word of each lane's places: the warps' sums go through shared
            // memory and are added in order, in units of the largest reference.  A thread
            // has two places of a row.
            const int slot = blockIdx.x * 2 + (it.first ? 0 : 1);
            const bool whole = it.whole();
            const int row = threadIdx.x >> 5, at = threadIdx.x & 31;
            float f[NW];
            __half* out = nullptr;
#pragma unroll 1
            for (int r = 0; r < MT / 4; ++r) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float4* to = reinterpret_cast<float4*>(
                        join + (warp * 8 + 2 * t + e) * C::JOIN_ROW + gid * 8);
                    to[0] = make_float4(o[0][e], o[0][e + 2], o[1][e], o[1][e + 2]);
                    to[1] = make_float4(o[2][e], o[2][e + 2], o[3][e], o[3][e + 2]);
                }
                meet_all();
                if (row < P.nq) {
                    if (r == 0) {
                        float2 ml[NW];
                        float M = -INFINITY;
#pragma unroll
                        for (int x = 0; x < NW; ++x) {
                            ml[x] = *reinterpret_cast<const float2*>(sml + (x * 8 + row) * 2);
                            M = fmaxf(M, ml[x].x);
                        }
                        float sum = 0.f;
#pragma unroll
                        for (int x = 0; x < NW; ++x) {
                            f[x] = ml[x].x == -INFINITY ? 0.f : ex2(ml[x].x - M);
                            sum = fmaf(f[x], ml[x].y, sum);
                        }
                        if (whole) {
                            // (a NaN sum is a NaN row, a sum of zero a row that sees nothing)
                            const float unit = sum == 0.f ? 0.f : vscale / sum;
#pragma unroll
                            for (int x = 0; x < NW; ++x) f[x] *= unit;
                            out = P.out + row_offset(P, it.b, it.h, row, DH);
                        } else if (at == 0) {
                            *reinterpret_cast<float2*>(P.ws_ml + ((long long)slot * 8 + row) * 2) =
                                make_float2(M, sum);
                        }
                    }
                    float2 a = make_float2(0.f, 0.f);
#pragma unroll
                    for (int x = 0; x < NW; ++x) {
                        const float2 v = *reinterpret_cast<const float2*>(
                            join + (x * 8 + row) * C::JOIN_ROW + at * 2);
                        a.x = fmaf(f[x], v.x, a.x);
                        a.y = fmaf(f[x], v.y, a.y);
                    }
                    const int d = (F8 ? (r >> 1) * 128 + (at >> 2) * 16 + (r & 1) * 8
                                      : (at >> 2) * (DH / 8) + r * 8) +
                                  (at & 3) * 2;
                    if (whole)
                        *reinterpret_cast<uint32_t*>(out + d) = pack_half2(a.x, a.y);
                    else
                        *reinterpret_cast<float2*>(P.ws_o + ((long long)slot * 8 + row) * DH + d) = a;
                }
                meet_all();
#pragma unroll
                for (int i = 0; i < MT - 4; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][e] = o[i + 4][e];
            }
        }
    }
    __syncthreads();
}

// Joins the partials of the units that lie in several ranges.  A block of 16 warps
// takes 128 places of D of 16 / WPR packed rows; a row's WPR warps share its pieces out
// and their sums are added in order.  The whole calls with 16, 4 and 2 warps a row: one
// unit in 152 pieces 23.7, 32.0 and 40.9 us; sixteen units in about ten each 15.5, 12.2
// and 12.6; 96 units in two or three 60.4, 45.5 and 44.4.  The choice goes by the batch, for
// the lengths are known on the device alone: among 63 sequences of no tokens one of 128000
// is joined by two warps a row (one 4-bit row 29.5 us, 18.0 alone; eight rows 47.3 and
// 31.4).
constexpr int MERGE_WARPS = 16;

template <int WPR>
__global__ void __launch_bounds__(MERGE_WARPS * 32) merge_kernel(const Params P, int unit_rows,
                                                                 int dh) {
    __shared__ float4 part[MERGE_WARPS][32];
    __shared__ float2 top[MERGE_WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.y * (MERGE_WARPS / WPR) + warp / WPR, w = warp % WPR;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 task = __ldcg(P.tasks + blockIdx.x);
    const int pieces = task.z;
    if (pieces == 0) return;
    // (calls that overlap on one workspace spoil each other's records: nothing is read or
    // written outside of what is this call's)
    if (pieces < 0 || (unsigned)task.x >= (unsigned)(P.batch * P.hkv) || task.y < 0 ||
        task.y / 2 + (long long)pieces > P.G)
        return;
    const int b = task.x / P.hkv, h = task.x - b * P.hkv;
    const bool there = r < P.nq;
    const int d0 = blockIdx.z * 128 + lane * 4;
    const float vscale = *P.scale_dev[1];
    auto row_of = [&](int i) {
        return (i == 0 ? (long long)task.y : (long long)(task.y / 2 + i) * 2) * unit_rows + r;
    };
    const float* from = P.ws_o + d0;
    auto load = [&](int i) {
        return __ldcg(reinterpret_cast<const float4*>(from + row_of(w + i * WPR) * dh));
    };
    // The warp's pieces w, w + WPR, ..., 32 at a time: references and sums, a lane each, and
    // the first O in flight beside them.
    constexpr int AHEAD = WPR == MERGE_WARPS ? 10 : 4;
    const int mine = there && pieces > w ? (pieces - w + WPR - 1) / WPR : 0;
    float m = -INFINITY, sum = 0.f;   // of the pieces so far, in units of the largest reference
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int i0 = 0; i0 < mine; i0 += 32) {
        const int n = min(mine - i0, 32);
        float4 o[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (i < n) o[i] = load(i0 + i);
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < n)
            ml = __ldcg(
                reinterpret_cast<const float2*>(P.ws_ml + row_of(w + (i0 + lane) * WPR) * 2));
        float mx = fmaxf(ml.x, m);
#pragma unroll
        for (int x = 16; x; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - mx);
        const float keep = m == -INFINITY ? 0.f : ex2(m - mx);
        float part_sum = f * ml.y;
#pragma unroll
        for (int x = 16; x; x >>= 1) part_sum += __shfl_xor_sync(0xffffffffu, part_sum, x);
        m = mx;
        sum = fmaf(keep, sum, part_sum);
        acc.x *= keep, acc.y *= keep, acc.z *= keep, acc.w *= keep;
        auto add = [&](int i, const float4& v) {
            const float fi = __shfl_sync(0xffffffffu, f, i);
            acc.x = fmaf(fi, v.x, acc.x);
            acc.y = fmaf(fi, v.y, acc.y);
            acc.z = fmaf(fi, v.z, acc.z);
            acc.w = fmaf(fi, v.w, acc.w);
        };
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (i < n) add(i, o[i]);
#pragma unroll 4
        for (int i = AHEAD; i < n; ++i) add(i, load(i0 + i));
    }
    part[warp][lane] = acc;
    if (lane == 0) top[warp] = make_float2(m, sum);
    __syncthreads();
    if (w || !there) return;
    float M = m;
#pragma unroll
    for (int x = 1; x < WPR; ++x) M = fmaxf(M, top[warp + x].x);
    float total = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int x = 0; x < WPR; ++x) {
        const float2 tx = top[warp + x];
        const float fx = tx.x == -INFINITY ? 0.f : ex2(tx.x - M);
        const float4 v = part[warp + x][lane];
        total += fx * tx.y;
        acc.x = fmaf(fx, v.x, acc.x);
        acc.y = fmaf(fx, v.y, acc.y);
        acc.z = fmaf(fx, v.z, acc.z);
        acc.w = fmaf(fx, v.w, acc.w);
    }
    const float inv = total == 0.f ? 0.f : vscale / total;
    uint2 v;
    v.x = pack_half2(acc.x * inv, acc.y * inv);
    v.y = pack_half2(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(P.out + row_offset(P, b, h, r, dh) + d0) = v;
}

template <bool F8, int DH, int NT>
int launch(const Maps<F8>& maps, const Params& P, cudaStream_t stream) {
    // (one eight of rows, or more)
    using C = typename std::conditional<NT == 1, Narrow<F8, DH>,
                                        Config<F8, DH, NT == 1 ? 2 : NT>>::type;
    void (*kernel)(Maps<F8>, Params);
    if constexpr (NT == 1) kernel = narrow_kernel<F8, DH>;
    else kernel = split_kernel<F8, DH, NT>;
    if (ensure_smem_limit(reinterpret_cast<const void*>(kernel), C::BYTES) != GQA_OK)
        return GQA_ERR_CUDA;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(P.G);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::BYTES;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, maps, P) != cudaSuccess) return GQA_ERR_CUDA;
    if (P.G == 1) return GQA_OK;   // nothing is cut
    // A row's warps, by how many pieces a unit has if all are of one length.
    const int units = P.batch * P.hkv;
    const int wpr = P.G >= 16 * units ? 16 : P.G >= 4 * units ? 4 : 2;
    void (*const merge)(Params, int, int) =
        wpr == 16 ? merge_kernel<16> : wpr == 4 ? merge_kernel<4> : merge_kernel<2>;
    const int a_block = MERGE_WARPS / wpr;
    cfg.gridDim = dim3(P.by_unit ? units : P.G, (P.nq + a_block - 1) / a_block, DH / 128);
    cfg.blockDim = dim3(MERGE_WARPS * 32);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, merge, P, 8 * NT, DH) == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

// Packed rows of a unit: all of a KV head's, by eights.
int unit_rows(int nq) { return nq <= 32 ? (nq + 7) / 8 * 8 : 48; }

template <bool F8, int DH>
int launch_rows(const Maps<F8>& maps, const Params& P, cudaStream_t stream) {
    switch (unit_rows(P.nq)) {
        case 8: return launch<F8, DH, 1>(maps, P, stream);
        case 16: return launch<F8, DH, 2>(maps, P, stream);
        case 24: return launch<F8, DH, 3>(maps, P, stream);
        case 32: return launch<F8, DH, 4>(maps, P, stream);
        default: return launch<F8, DH, 6>(maps, P, stream);
    }
}

template <bool F8>
int launch_tails(const void* q, const uint8_t* kcache, const uint8_t* vcache, const float* kscale,
                 const float* vscale, const int32_t* block_tables, int table_stride, int num_pages,
                 int page, const int* ctx_lens_dev, int max_ctx_len, int batch, int R, int Hq,
                 int Hkv, int Dh, float scale, int window, int sinks, void* out,
                 cudaStream_t stream) {
    const DeviceInfo* di = device_info();
    if (!di) return GQA_ERR_CUDA;
    Params P;
    P.q = static_cast<const __half*>(q);
    P.cache[0] = kcache;
    P.cache[1] = vcache;
    P.scale_dev[0] = kscale;
    P.scale_dev[1] = vscale;
    P.tables = block_tables;
    P.ctx_lens = ctx_lens_dev;
    P.table_stride = table_stride;
    P.num_pages = num_pages;
    P.page = page;
    P.log2_page = __builtin_ctz((unsigned)page);
    P.max_ctx = max_ctx_len;
    P.batch = batch;
    P.R = R;
    P.hq = Hq;
    P.hkv = Hkv;
    P.grp = make_fastdiv(Hq / Hkv);
    P.nq = R * (Hq / Hkv);
    const int rows = unit_rows(P.nq);
    const int tile = Dh == 256 ? tile_keys<F8, 256>(rows / 8) : tile_keys<F8, 128>(rows / 8);
    P.ltile = __builtin_ctz((unsigned)tile);
    // A window that holds every context hides nothing.
    P.window = window >= max_ctx_len ? 0 : window;
    P.sinks = P.window > 0 ? sinks : 0;
    P.scale = scale;
    // No more ranges than tiles.
    const long long tiles = (long long)batch * Hkv * ((max_ctx_len - 1) / tile + 1);
    P.G = (int)(tiles < di->num_sms ? tiles : di->num_sms);
    P.by_unit = (long long)batch * Hkv < P.G;
    P.out = static_cast<__half*>(out);
    P.err = di->err_word;
    void* ws;
    size_t ws_bytes;
    current_workspace(&ws, &ws_bytes);
    if (!ws || ws_bytes < tails_workspace_bytes(P.nq, di->num_sms, Dh)) return GQA_ERR_WORKSPACE;
    P.ws_o = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kWorkspaceCounterBytes);
    P.ws_ml = P.ws_o + (size_t)2 * P.G * rows * Dh;
    P.tasks = reinterpret_cast<int4*>(P.ws_ml + (size_t)2 * P.G * rows * 2);
    Maps<F8> maps;
    if constexpr (F8) {
        const uint64_t keys = (uint64_t)num_pages * page, width = (uint64_t)Hkv * Dh;
        const uint32_t box = page < tile ? page : tile;
        if (!make_map_2d_u8(&maps.kv[0], kcache, keys, width, width, box, 128) ||
            !make_map_2d_u8(&maps.kv[1], vcache, keys, width, width, box, 128))
            return GQA_ERR_CUDA;
    }
    return Dh == 256 ? launch_rows<F8, 256>(maps, P, stream)
                     : launch_rows<F8, 128>(maps, P, stream);
}

}  // namespace tails

size_t tails_workspace_bytes(int nq, int num_sms, int Dh) {
    return kWorkspaceCounterBytes +
           (size_t)num_sms * (2 * tails::unit_rows(nq < 48 ? nq : 48) * (Dh + 2) * sizeof(float) +
                              sizeof(int4));
}

int tails_launch(bool fp4, const void* q, const uint8_t* kcache, const uint8_t* vcache,
                 const float* kscale, const float* vscale, const int32_t* block_tables,
                 int table_stride, int num_pages, int page, const int* ctx_lens_dev,
                 int max_ctx_len, int batch, int R, int Hq, int Hkv, int Dh, float scale, int window,
                 int sinks, void* out, cudaStream_t stream) {
    const auto fn = fp4 ? tails::launch_tails<false> : tails::launch_tails<true>;
    return fn(q, kcache, vcache, kscale, vscale, block_tables, table_stride, num_pages, page,
              ctx_lens_dev, max_ctx_len, batch, R, Hq, Hkv, Dh, scale, window, sinks, out, stream);
}

}  // namespace gqa

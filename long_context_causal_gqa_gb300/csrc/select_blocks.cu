// select_blocks.cu -- the 4-token blocks each query row attends, by a cheap
// score: the dot of the row's summed queries and the block's summed keys, both
// as int8 codes.
//
// The dot is a whole number below 2^24 in magnitude (127^2 * 1024 at most), so
// it is exact in any order of the sum: on the fp16 tensor cores with 32-bit
// accumulators as well as with dp4a.  The score is that number times the
// block's scale, one 32-bit rounding.  Equal scores go to the lower block id.
// The selection is therefore a function of the inputs alone, whatever the
// path, the split or the other rows of the call.
//
// Few rows: every block's scores by dp4a straight from the int8 index.  More
// rows: the tensor cores (dot_kernel).  With many blocks, writing rows x blocks
// scores and reading them back would cost several times the products
// themselves.  So one block's products of every 2^s are taken first, of which only
// maxima over small groups are kept; the k-th best of those is a lower bound
// of the row's k-th best score (k blocks reach it), found by bound_kernel.  The
// products of all blocks are then compared with the bound as they leave the
// tensor memory, and a little over 2^s k of them stay as candidates.  Either way
// one CTA a row takes the best of what is left (best_of).  A row whose candidates
// do not fit (thousands of equal scores) is searched block by block (scan_best).
//
// What bounds it: 4096 rows over 32000 blocks of width 256 are 67 GFLOP, 35 us
// of the tensor cores; the call takes 120 us: query and index codes 11, the
// sample (a block of four) 22, its bounds 11, the candidates 55, the best of
// them 30, overlapping a little.  Of the candidates' 55 the products alone are
// 44 (loads and products without the epilogue's compares).  One row over 65472
// blocks reads 17 MB, 2.5 us; it takes 16.8 us, of which 11 are the pick on one
// SM, a chain of barriers and dependent loads; the call's host side takes 22.
#include <algorithm>
#include <atomic>
#include <cuda_fp16.h>

#include "internal.h"
#include "pair_mma.cuh"
#include "pick.cuh"
#include "sm100.cuh"

namespace gqa {
namespace select {

// Each kernel of a call but the first is a programmatic dependent of the one
// before: it is launched while that runs, and waits for its end (so for the end
// of all before) ahead of its first read or write of global memory.
__device__ __forceinline__ void wait_for_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void let_next_launch() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// What dot_kernel does with its products: keep all scores, keep the maxima of
// groups of the sampled blocks', or keep the candidates.
enum Mode { SCORES = 0, MAXIMA = 1, CANDIDATES = 2 };

// The sample: one block of every 2^skip, at a place that varies without a period
// (every 4th block may be the only good ones, or none of them), in an order that
// puts neighbours in different groups: neighbours score alike, and a group of them
// would count the best of a good neighbourhood once instead of eight times.
struct Sample {
    int skip;
    int count;       // sampled blocks
    int cols;        // columns: count up to a multiple of 8
    uint32_t mask;   // 2^bits - 1 >= cols - 1
    int half;        // half the bits
    // The block sampled as number x < count, of n.
    __device__ int block(int x, int n) const {
        return min((x << skip) + (int)__umulhi((uint32_t)x * 0x9e3779b1u, 1u << skip), n - 1);
    }
    // Column of number x < cols: the numbers of the mask's bits mixed by steps that
    // can each be undone (odd factors, from the golden ratio and the root of two),
    // again and again until the result is below cols.
    __host__ __device__ int column(int x) const {
        uint32_t y = (uint32_t)x;
        do {
            y = y * 0x9e3779b1u & mask;
            y ^= y >> half;
            y = y * 0x6a09e667u & mask;
            y ^= y >> half;
        } while (y >= (uint32_t)cols);
        return (int)y;
    }
};
constexpr int NO_BLOCK = 0x7fffffff;    // behind every row

// A bound that nothing reaches (a comparison with NaN is false).
#define kNoBound __int_as_float(0x7fffffff)

struct IndexView {
    const int8_t* index;
    const float* scale;
    const int32_t* table;
    int num_pages;
    int log2_ppb;                // log2 of the blocks of a page
    int width;
    unsigned* err;
};

// Physical block of logical block b; a table entry outside the cache reads
// page 0 (flagged), as the attention kernels do.
__device__ __forceinline__ long long physical_block(const IndexView& V, int b) {
    int id = V.table[b >> V.log2_ppb];
    if (id < 0 || id >= V.num_pages) {
        atomicOr(V.err, kErrBadPageId);
        id = 0;
    }
    return ((long long)id << V.log2_ppb) + (b & ((1 << V.log2_ppb) - 1));
}

// Four int8 codes to fp16, exactly: 1024 + (code + 128) has the biased code in
// the low bits of its significand.
__device__ __forceinline__ uint2 codes_half4(uint32_t w) {
    w ^= 0x80808080u;
    uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 off = __float2half2_rn(1152.f);
    __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), off);
    __half2 y = __hsub2(*reinterpret_cast<__half2*>(&b), off);
    return make_uint2(*reinterpret_cast<uint32_t*>(&x), *reinterpret_cast<uint32_t*>(&y));
}

// ------------------------------------------------------------ query codes
// codes[row, g * D + d] = rint(S * 127 / max |S|), S = sum of q over the query
// heads of KV head g, exact and rounded to 32 bits once.  A row with an
// infinity or NaN gets codes of zero.  One warp a row, 8 values a lane.
struct CodeParams {
    const __half* q;
    int rows, Hq, D, group, width;
    int8_t* codes;
    __half* codes16;   // the same codes as fp16 (null: not wanted)
};

// Each fp16 value x is split at 2^-6: x + kSplit has a last place of 2^-6 for
// every |x| < 65536, so its bits, as whole numbers, add up the upper parts (at
// most 64 of 2^22), and the lower parts are multiples of 2^-24 of at most 2^-7,
// whose sum stays exact in 32 bits.
constexpr float kSplit = 196608.f;   // 1.5 * 2^17
constexpr int kSplitBits = 0x48400000;

// CHUNKS: 256-wide pieces of a row.
template <int CHUNKS>
__device__ __forceinline__ void query_codes(const CodeParams& P, int row, int lane,
                                            uint2 (&w)[CHUNKS]) {
    float s[CHUNKS][8];
    float most = 0.f;
    bool fine = true;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
        const int e = c * 256 + lane * 8;
        if (c * 256 >= P.width) break;
        if (e >= P.width) {
#pragma unroll
            for (int j = 0; j < 8; ++j) s[c][j] = 0.f;
            continue;
        }
        const int g = e / P.D;
        const __half* src = P.q + ((long long)row * P.Hq + g * P.group) * P.D + (e - g * P.D);
        int upper[8];
        float lower[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            upper[j] = 0;
            lower[j] = 0.f;
        }
#pragma unroll 4
        for (int h = 0; h < P.group; ++h) {
            const uint4 u = *reinterpret_cast<const uint4*>(src + (long long)h * P.D);
            const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[j / 2]));
                const float x = j & 1 ? f.y : f.x;
                fine = fine && fabsf(x) <= 65504.f;
                const float t = __fadd_rn(x, kSplit);
                upper[j] += __float_as_int(t) - kSplitBits;
                lower[j] += __fsub_rn(x, __fsub_rn(t, kSplit));
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // In units of 2^-24, exact; one rounding to 32 bits.
            const long long sum = ((long long)upper[j] << 18) + (int)(lower[j] * 16777216.f);
            s[c][j] = __ll2float_rn(sum) * (1.f / 16777216.f);
            most = fmaxf(most, fabsf(s[c][j]));
        }
    }
    fine = __all_sync(0xffffffffu, fine);
    most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
    fine = fine && most > 0.f;
    const float inv = fine ? 127.f / most : 0.f;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
        if (c * 256 >= P.width) break;
        uint32_t x[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int code = fine ? (int)rintf(__fmul_rn(s[c][j], inv)) : 0;
            x[j / 4] |= (uint32_t)(code & 0xff) << (8 * (j % 4));
        }
        w[c] = make_uint2(x[0], x[1]);
    }
}

template <int CHUNKS>
__device__ __forceinline__ void store_codes(const CodeParams& P, int row, int lane,
                                            const uint2 (&w)[CHUNKS]) {
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
        const int e = c * 256 + lane * 8;
        if (e >= P.width) break;
        const long long at = (long long)row * P.width + e;
        *reinterpret_cast<uint2*>(P.codes + at) = w[c];
        if (P.codes16) {
            const uint2 a = codes_half4(w[c].x), b = codes_half4(w[c].y);
            *reinterpret_cast<uint4*>(P.codes16 + at) = make_uint4(a.x, a.y, b.x, b.y);
        }
    }
}

// The index's blocks in order as the tensor cores read them, fp16 codes and the
// blocks' scales, and the sampled ones again.
struct ExpandParams {
    IndexView V;
    int n;
    __half* cols;
    float* scale;
    // The sample's columns: codes, scales and blocks (null: no sample).
    __half* sample_cols;
    float* sample_scale;
    int* sample_block;
    Sample sample;
    int n_first;           // blocks below are not scored
};

// The first `code_ctas` CTAs make query codes (8 rows each), the others
// expand EXPAND_PASSES x (256 / (width / 16)) blocks, 16 codes a thread and
// pass, all passes' loads in flight together.
constexpr int EXPAND_PASSES = 4;

template <int CHUNKS>
__global__ void __launch_bounds__(256) prepare_kernel(const CodeParams C, const ExpandParams E,
                                                      int code_ctas) {
    let_next_launch();
    if ((int)blockIdx.x < code_ctas) {
        const int row = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x % 32;
        if (row >= C.rows) return;
        uint2 w[CHUNKS];
        query_codes<CHUNKS>(C, row, lane, w);
        store_codes<CHUNKS>(C, row, lane, w);
        return;
    }
    const int per_block = E.V.width / 16, at_once = 256 / per_block;
    const int mine = threadIdx.x / per_block, part = threadIdx.x - mine * per_block;
    if (mine >= at_once) return;
    const int b0 = (blockIdx.x - code_ctas) * at_once * EXPAND_PASSES + mine;
    long long block[EXPAND_PASSES];
    uint4 w[EXPAND_PASSES];
#pragma unroll
    for (int i = 0; i < EXPAND_PASSES; ++i)
        block[i] = physical_block(E.V, min(b0 + i * at_once, E.n - 1));
#pragma unroll
    for (int i = 0; i < EXPAND_PASSES; ++i)
        w[i] = *reinterpret_cast<const uint4*>(E.V.index + block[i] * E.V.width + part * 16);
#pragma unroll
    for (int i = 0; i < EXPAND_PASSES; ++i) {
        const int b = b0 + i * at_once;
        if (b >= E.n) break;
        __half* dst = E.cols + (long long)b * E.V.width + part * 16;
        const uint2 x = codes_half4(w[i].x), y = codes_half4(w[i].y), z = codes_half4(w[i].z),
                    u = codes_half4(w[i].w);
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(x.x, x.y, y.x, y.y);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(z.x, z.y, u.x, u.y);
        const float s = part == 0 ? E.V.scale[block[i]] : 0.f;
        if (part == 0) E.scale[b] = s;
        const Sample& S = E.sample;
        if (!E.sample_cols || b != S.block(b >> S.skip, E.n)) continue;
        const int col = S.column(b >> S.skip);
        dst = E.sample_cols + (long long)col * E.V.width + part * 16;
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(x.x, x.y, y.x, y.y);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(z.x, z.y, u.x, u.y);
        if (part) continue;
        E.sample_scale[col] = s;
        E.sample_block[col] = b < E.n_first ? NO_BLOCK : b;
        if (b >> S.skip == S.count - 1)      // the columns left over
            for (int c = S.count; c < S.cols; ++c) E.sample_block[S.column(c)] = NO_BLOCK;
    }
}

// ------------------------------------------------------------ products
// rows x columns products on CTA pairs: a pair takes 256 rows (128 a CTA) and
// walks 256-column tiles, each CTA holding half of every column tile, one
// M = 256, N = 256 UMMA stream issued by the even CTA into two tensor-memory
// buffers.  Up to width 256 a pair keeps its rows' codes in shared memory for
// all its tiles; beyond, they stream with the columns.  Warp 0 loads, warp 1
// issues, the others take the products: each thread one row and a quarter of a
// tile's columns.  (With two warps a scheduler instead of four, each waiting on
// its own chain of compares and stores, the products waited for them: 63
// instead of 55 us over 4096 x 32000.)
constexpr int CTA_ROWS = 128;
constexpr int PAIR_ROWS = 256;
constexpr int TILE = 256;                    // columns of a tile
constexpr int CHUNK_BYTES = 128 * 128;       // 128 rows x 64 fp16
constexpr int RES_CHUNKS = 4;                // row chunks kept (width 256)
constexpr int PARTS = 4;                     // warpgroups that share a tile's columns
constexpr int PART = TILE / PARTS;
constexpr int EPI_WARPS = 4 * PARTS;
constexpr int DOT_THREADS = 32 * (2 + EPI_WARPS);
constexpr int SCALE_BYTES = EPI_WARPS * PART * 4;   // a warp's columns' scales
constexpr int DUMP_WORDS = 36;                      // 32 products of a row, 16-byte aligned
constexpr int DUMP_BYTES = EPI_WARPS * 32 * DUMP_WORDS * 4;
constexpr uint32_t DOT_TMEM = 512;
constexpr uint32_t IDESC = idesc_f16_f32(256, TILE, false, false);

template <bool RESIDENT>
struct DotCfg {
    static constexpr int SLOTS = RESIDENT ? 5 : 4;
    static constexpr int SLOT_BYTES = RESIDENT ? CHUNK_BYTES : 2 * CHUNK_BYTES;
    static constexpr int ROW_BYTES = RESIDENT ? RES_CHUNKS * CHUNK_BYTES : 0;
    static constexpr int NUM_BARS = 2 * SLOTS + 7;
    static constexpr int SMEM = 1024 + ROW_BYTES + SLOTS * SLOT_BYTES + SCALE_BYTES +
                                DUMP_BYTES + NUM_BARS * 8 + 16;
    static_assert(SMEM <= 232448, "shared memory");
};

struct DotParams {
    int rows;                  // rows of the launch
    int chunks;                // width / 64
    int row_tiles;
    int G;                     // pairs
    long long total;           // (row tile, column tile) products
    int pos0;                  // position of the first row
    int n_first, n_last;
    const float* scale;        // per column, allocated to a multiple of TILE
    float* scores;             // SCORES, MAXIMA: [rows, stride]
    long long stride;
    int cols;                  // MAXIMA: columns
    const int* block;          // MAXIMA: their blocks, allocated like scale
    int log2_group;            // MAXIMA: columns of a group, 2 to 8
    const float* bound;        // CANDIDATES: per row
    // CANDIDATES: (score, block) [runs][tile_rows][PARTS][cap], and their numbers
    // [runs][tile_rows][PARTS], -1: too many.  A run is what a pair computes of a
    // row tile; pair p's of row tile t is number p + t.
    uint2* list;
    int* counts;
    int tile_rows, cap;
    unsigned* err;
    __host__ __device__ int runs() const { return G + row_tiles; }
    __device__ long long list_at(int run, int row) const {
        return ((long long)run * tile_rows + row % PAIR_ROWS) * PARTS;
    }
};

template <int MODE>
__host__ __device__ __forceinline__ int col_tiles(const DotParams& P, int rt) {
    if (MODE == MAXIMA) return (P.cols + TILE - 1) / TILE;
    const int last = min(rt * PAIR_ROWS + PAIR_ROWS, P.rows) - 1;
    const int hi = ((P.pos0 + last) >> 2) + 1 - P.n_last;
    return hi <= 0 ? 0 : (hi + TILE - 1) / TILE;
}
// The pair that computes product x of the row-tile-major order, and the first
// product of pair p.
__host__ __device__ __forceinline__ long long pair_begin(const DotParams& P, int p) {
    return (long long)p * P.total / P.G;
}
__host__ __device__ __forceinline__ int pair_of(const DotParams& P, long long x) {
    return (int)(((x + 1) * P.G - 1) / P.total);
}

// A pair's products as runs of column tiles [jb, je) of one row tile.
template <int MODE>
struct Runs {
    long long pos, end, cum;
    int rt;
    __device__ void init(const DotParams& P, int pair) {
        pos = pair_begin(P, pair);
        end = pair_begin(P, pair + 1);
        cum = 0;
        rt = 0;
        while (rt < P.row_tiles) {
            const int n = col_tiles<MODE>(P, rt);
            if (cum + n > pos) break;
            cum += n;
            ++rt;
        }
    }
    __device__ bool next(const DotParams& P, int& t, int& jb, int& je) {
        if (pos >= end) return false;
        int n = col_tiles<MODE>(P, rt);
        while (n == 0) n = col_tiles<MODE>(P, ++rt);
        t = rt;
        jb = (int)(pos - cum);
        je = (int)min((long long)n, end - cum);
        pos = cum + je;
        if (je == n) {
            cum += n;
            ++rt;
        }
        return true;
    }
};

__device__ __forceinline__ void store8(float* p, const float* v) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]),
                 "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

// max(a, b, c); a NaN gives way to a number.
__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// The scores of 32 columns: products d times scales.
__device__ __forceinline__ void scores_of(const uint32_t (&d)[32], const float4* scale4,
                                          float (&sc)[32]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float4 f = scale4[i];
        sc[4 * i] = __fmul_rn(__uint_as_float(d[4 * i]), f.x);
        sc[4 * i + 1] = __fmul_rn(__uint_as_float(d[4 * i + 1]), f.y);
        sc[4 * i + 2] = __fmul_rn(__uint_as_float(d[4 * i + 2]), f.z);
        sc[4 * i + 3] = __fmul_rn(__uint_as_float(d[4 * i + 3]), f.w);
    }
}

// The maxima of groups of 2^log2_group of 32 columns' scores, for the blocks below hi.
__device__ __forceinline__ void store_maxima(float (&sc)[32], const int4* block4, int hi,
                                             int log2_group, float* dst, bool valid) {
    // Blocks that are not scored count for nothing.
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int4 b = block4[i];
        if (b.x >= hi) sc[4 * i] = -INFINITY;
        if (b.y >= hi) sc[4 * i + 1] = -INFINITY;
        if (b.z >= hi) sc[4 * i + 2] = -INFINITY;
        if (b.w >= hi) sc[4 * i + 3] = -INFINITY;
    }
    if (!valid) return;
    // Maxima drop a NaN; a group of nothing else counts for nothing.
    if (log2_group == 3) {
        float m[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float* x = sc + 8 * i;
            m[i] = fmax3(fmax3(x[0], x[1], x[2]), fmax3(x[3], x[4], x[5]), fmaxf(x[6], x[7]));
        }
        *reinterpret_cast<float4*>(dst) = make_float4(m[0], m[1], m[2], m[3]);
    } else {
        float m[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) m[i] = fmaxf(sc[2 * i], sc[2 * i + 1]);
        if (log2_group == 1) {
            store8(dst, m);
            store8(dst + 8, m + 8);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i] = fmaxf(m[2 * i], m[2 * i + 1]);
            store8(dst, m);
        }
    }
}

template <int MODE, bool RESIDENT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(DOT_THREADS, 1)
dot_kernel(const __grid_constant__ CUtensorMap tm_rows, const __grid_constant__ CUtensorMap tm_cols,
           const DotParams P) {
    using C = DotCfg<RESIDENT>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* base_ptr = smem_raw + (base - smem_u32(smem_raw));
    const uint32_t s_rows = base;
    const uint32_t s_ring = base + C::ROW_BYTES;
    const uint32_t bars = s_ring + C::SLOTS * C::SLOT_BYTES + SCALE_BYTES + DUMP_BYTES;
    auto full = [&](int s) { return bars + 8 * s; };
    auto empty = [&](int s) { return bars + 8 * (C::SLOTS + s); };
    const uint32_t rows_full = bars + 8 * (2 * C::SLOTS), rows_empty = rows_full + 8;
    auto tfull = [&](int i) { return rows_full + 16 + 8 * i; };    // products in buffer i
    auto tempty = [&](int i) { return rows_full + 32 + 8 * i; };   // buffer i read out
    const uint32_t drain = rows_full + 48;
    float* s_scale = reinterpret_cast<float*>(base_ptr + C::ROW_BYTES + C::SLOTS * C::SLOT_BYTES);
    float* s_dump = s_scale + SCALE_BYTES / 4;
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(s_dump + DUMP_BYTES / 4 + C::NUM_BARS * 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_ptr + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = pairs::cluster_rank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::SLOTS; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(rows_full, 1);
        mbar_init(rows_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull(i), 1);
            mbar_init(tempty(i), 2 * EPI_WARPS);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_rows);
        tma_prefetch_desc(&tm_cols);
    }
    if (warp == 1) pairs::tmem_alloc(smem_u32(tmem_ptr), DOT_TMEM);
    tc_fence_before();
    // Both CTAs' barriers are initialised before either uses the other's.
    pairs::cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *tmem_ptr;
    wait_for_previous();

    Runs<MODE> runs;
    runs.init(P, pair);
    int rt, jb, je;
    if (warp == 0) {
        // ------------------------------------------------------------ loads
        // Completions of both CTAs' halves land on the even CTA's barriers.
        if (lane == 0) {
            uint32_t n = 0;     // slots filled
            int run = 0;
            bool ok = true;
            while (ok && runs.next(P, rt, jb, je)) {
                const int row0 = rt * PAIR_ROWS + CTA_ROWS * (int)rank;
                if (RESIDENT) {
                    ok = mbar_wait(rows_empty, (run & 1) ^ 1, abort_flag, P.err);
                    if (!ok) break;
                    if (leader) mbar_arrive_expect_tx(rows_full, 2 * P.chunks * CHUNK_BYTES);
                    for (int c = 0; c < P.chunks; ++c)
                        pairs::tma_load_2d(s_rows + c * CHUNK_BYTES, &tm_rows,
                                           pairs::leader_addr(rows_full), c * 64, row0);
                }
                for (int j = jb; ok && j < je; ++j)
                    for (int c = 0; c < P.chunks; ++c, ++n) {
                        const int s = n % C::SLOTS;
                        ok = mbar_wait(empty(s), ((n / C::SLOTS) & 1) ^ 1, abort_flag, P.err);
                        if (!ok) break;
                        if (leader) mbar_arrive_expect_tx(full(s), 2 * C::SLOT_BYTES);
                        const uint32_t bar = pairs::leader_addr(full(s));
                        const uint32_t dst = s_ring + s * C::SLOT_BYTES;
                        pairs::tma_load_2d(dst, &tm_cols, bar, c * 64,
                                           j * TILE + CTA_ROWS * (int)rank);
                        if (!RESIDENT)
                            pairs::tma_load_2d(dst + CHUNK_BYTES, &tm_rows, bar, c * 64, row0);
                    }
                ++run;
            }
            if (!ok && leader) {
                // Unwind: let every copy still in flight land before the CTA exits.
                for (uint32_t s = 0; s < (uint32_t)C::SLOTS; ++s) {
                    const uint32_t fills = n > s ? (n - s + C::SLOTS - 1) / C::SLOTS : 0;
                    if (fills) pairs::drain_wait(full(s), (fills - 1) & 1u);
                }
                if (RESIDENT && run > 0) pairs::drain_wait(rows_full, (run - 1) & 1);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        if (lane == 0 && leader) {
            uint32_t n = 0, t = 0;
            int run = 0;
            bool ok = true;
            while (ok && runs.next(P, rt, jb, je)) {
                if (RESIDENT) {
                    ok = mbar_wait(rows_full, run & 1, abort_flag, P.err);
                    if (!ok) break;
                }
                for (int j = jb; ok && j < je; ++j, ++t) {
                    ok = mbar_wait(tempty(t & 1), ((t >> 1) & 1) ^ 1, abort_flag, P.err);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + (t & 1) * TILE;
                    for (int c = 0; c < P.chunks; ++c, ++n) {
                        const int s = n % C::SLOTS;
                        ok = mbar_wait(full(s), (n / C::SLOTS) & 1, abort_flag, P.err);
                        if (!ok) break;
                        const uint32_t b = s_ring + s * C::SLOT_BYTES;
                        const uint32_t a = RESIDENT ? s_rows + c * CHUNK_BYTES : b + CHUNK_BYTES;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            pairs::umma_ss(d, sdesc_sw128(a + k * 32, 16, 1024),
                                           sdesc_sw128(b + k * 32, 16, 1024), IDESC,
                                           c > 0 || k > 0);
                        pairs::umma_commit(empty(s));
                    }
                    if (ok) pairs::umma_commit(tfull(t & 1));
                }
                if (RESIDENT) pairs::umma_commit(rows_empty);
                ++run;
            }
            if (!ok) {
                // Unwind: wait for every UMMA issued before TMEM is freed.
                pairs::umma_commit(drain);
                pairs::drain_wait(drain, 0);
            }
        }
    } else {
        // ------------------------------------------------------------ scores
        const int part = (warp - 2) >> 2;      // which columns of a tile
        const int quarter = warp & 3;          // TMEM lanes this warp may read
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16) + part * PART;
        float* const my_scale = s_scale + (warp - 2) * PART;
        float* const my_dump = s_dump + ((warp - 2) * 32 + lane) * DUMP_WORDS;
        int* const my_block = reinterpret_cast<int*>(s_dump) + (warp - 2) * PART;   // MAXIMA
        uint32_t t = 0;
        bool ok = true;
        while (ok && runs.next(P, rt, jb, je)) {
            const int row0 = rt * PAIR_ROWS + CTA_ROWS * (int)rank + quarter * 32;
            const int row = row0 + lane;
            const bool valid = row < P.rows;
            const int hi = ((P.pos0 + row) >> 2) + 1 - P.n_last;     // this row's scored blocks end
            const int hi0 = ((P.pos0 + row0) >> 2) + 1 - P.n_last;   // the warp's smallest
            const float bound = MODE == CANDIDATES && valid ? P.bound[row] : kNoBound;
            // Just below the bound, so that the sign of one fused multiply-add
            // lets every score that reaches the bound through (and few others).
            const float below = nextafterf(bound, -INFINITY);
            uint32_t open = bound == bound ? 0xffffffffu : 0u;
            const long long at = P.list_at(pair + rt, row) + part;
            uint2* const list = MODE == CANDIDATES ? P.list + at * P.cap : nullptr;
            int n = 0;
            // The columns' scales: four a lane of the first half, loaded a tile ahead,
            // then shared by the warp; of the sample the blocks, by the other half.
            // (Ordinary loads: the kernel before writes them while this one may run
            // already, so they are not read-only for its lifetime.)
            static_assert(PART == 64, "half a warp's float4");
            const bool half = MODE == MAXIMA && lane >= 16;
            const void* const cols = half ? static_cast<const void*>(P.block) : P.scale;
            const uint4* src = static_cast<const uint4*>(cols) + (jb * TILE + part * PART) / 4 +
                               lane % 16;
            uint4* const dst4 = reinterpret_cast<uint4*>(half ? my_block : (int*)my_scale) +
                                lane % 16;
            uint4 ahead = *src;
            for (int j = jb; j < je; ++j, ++t) {
                __syncwarp();
                if (lane < 16 || half) *dst4 = ahead;
                if (j + 1 < je) ahead = *(src += TILE / 4);
                __syncwarp();
                ok = mbar_wait(tfull(t & 1), (t >> 1) & 1, abort_flag, P.err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const int col0 = j * TILE + part * PART;
#pragma unroll
                for (int g = 0; g < PART / 32; ++g) {
                    const int c0 = col0 + g * 32;
                    uint32_t d[32];
                    tmem_ld32(t_lane + (t & 1) * TILE + g * 32, d);
                    tmem_ld_wait<32>(d);
                    if (g + 1 == PART / 32) {
                        // The buffer is read out.
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) pairs::remote_arrive(pairs::leader_addr(tempty(t & 1)));
                    }
                    const float4* sc4 = reinterpret_cast<const float4*>(my_scale + g * 32);
                    if constexpr (MODE == CANDIDATES) {
                        // Columns on the rows' own blocks, behind them, or on the first
                        // ones, are not scored.
                        const bool edge = c0 < P.n_first || c0 + 32 > hi0;
                        uint32_t under = 0;    // signs of score - bound, column i in bit i
#pragma unroll
                        for (int i = 7; i >= 0; --i) {
                            const float4 f = sc4[i];
                            const float s[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                            for (int k = 3; k >= 0; --k)
                                under = __funnelshift_l(
                                    __float_as_uint(fmaf(__uint_as_float(d[4 * i + k]), s[k],
                                                         -below)),
                                    under, 1);
                        }
                        uint32_t m = ~under & open;
                        if (edge) {
                            const int a = min(max(P.n_first - c0, 0), 32);
                            const int b = min(max(hi - c0, 0), 32);
                            m &= (b == 32 ? 0xffffffffu : (1u << b) - 1) &
                                 (a == 32 ? 0u : 0xffffffffu << a);
                        }
                        if (!__any_sync(0xffffffffu, m)) continue;
                        if (n + __popc(m) > P.cap) {
                            open = m = 0;    // no room: the row is searched block by block
                            n = -1;
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            reinterpret_cast<uint4*>(my_dump)[i] =
                                make_uint4(d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3]);
                        // Each lane reads its own row's products only.
                        while (m) {
                            const int i = __ffs(m) - 1;
                            m &= m - 1;
                            const float v = __fmul_rn(my_dump[i], my_scale[g * 32 + i]);
                            if (v >= bound) list[n++] = make_uint2(__float_as_uint(v), c0 + i);
                        }
                    } else {
                        float sc[32];
                        scores_of(d, sc4, sc);
                        float* dst = P.scores + row * P.stride + (c0 >> P.log2_group);
                        if constexpr (MODE == MAXIMA) {
                            store_maxima(sc, reinterpret_cast<const int4*>(my_block + g * 32), hi,
                                         P.log2_group, dst, valid);
                        } else if (valid) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) store8(dst + 8 * i, sc + 8 * i);
                        }
                    }
                }
            }
            if (MODE == CANDIDATES && valid) P.counts[at] = n;
        }
    }

    // After an abort, give copies the other CTA of the pair still had in
    // flight into this CTA's shared memory time to land before it exits.
    __syncthreads();
    if (*abort_flag) {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) {
        }
    }
    tc_fence_before();
    // Neither CTA leaves while the other may still signal its barriers.
    pairs::cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        pairs::tmem_dealloc(tmem, DOT_TMEM);
    }
}

// ------------------------------------------------------------ few rows
// Every CTA makes the codes of its rows itself, which costs less than a launch
// of its own, with its first blocks' codes already on their way.  Eight lanes
// read one block's codes, 16 bytes each at a time, 256 codes ahead of the products;
// a warp takes 4 * PER blocks together and keeps the scores and, over each 8 blocks,
// the largest scored one.
constexpr int FEW_TILE = 8;      // most rows of a CTA

struct FewParams {
    CodeParams C;
    IndexView V;
    int n;                       // blocks
    int pos0, n_first, n_last;
    float* scores;               // [rows, stride]
    long long stride;
    float* maxima;               // [rows, stride / 8]
};

// NR: rows of a CTA, 1 or FEW_TILE.
template <int CHUNKS, int NR>
__global__ void __launch_bounds__(256) score_few_kernel(const FewParams P) {
    constexpr int PER = CHUNKS == 1 && NR == 1 ? 4 : 2;
    __shared__ __align__(16) uint2 s_q[NR][CHUNKS * 32];
    let_next_launch();
    const int width = P.V.width, steps = width / 128, chunks = (width + 255) / 256;
    const int r0 = blockIdx.y * NR;
    const int nr = NR == 1 ? 1 : min(NR, P.C.rows - r0);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int sub = lane / 8, part = lane % 8;
    // This lane's blocks: b0 + 4 i + sub; 256 codes of each at a time.
    const uint4* src[PER];
    uint4 ahead[PER][2];
    float scale_ahead[PER];
    auto point = [&](int b0) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const long long block = physical_block(P.V, min(b0 + 4 * i + sub, P.n - 1));
            src[i] = reinterpret_cast<const uint4*>(P.V.index + block * width) + part;
            scale_ahead[i] = P.V.scale[block];
        }
    };
    auto fetch = [&](int c) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if (c * 2 + s < steps) ahead[i][s] = src[i][(c * 2 + s) * 8];
    };
    int b0 = (blockIdx.x * 8 + warp) * (4 * PER);
    if (b0 < P.n) {
        point(b0);
        fetch(0);
    }
    if (warp < nr) {
        uint2 w[CHUNKS];
        query_codes<CHUNKS>(P.C, r0 + warp, lane, w);
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)
            if (c * 256 + lane * 8 < width) s_q[warp][c * 32 + lane] = w[c];
    }
    __syncthreads();
    while (b0 < P.n) {
        const int b_next = b0 + gridDim.x * 8 * (4 * PER);
        int dot[PER][NR] = {};
        float scale[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) scale[i] = scale_ahead[i];
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            uint4 k[PER][2];
#pragma unroll
            for (int i = 0; i < PER; ++i)
#pragma unroll
                for (int s = 0; s < 2; ++s) k[i][s] = ahead[i][s];
            // The next codes are on their way during these products.
            if (c + 1 < chunks) {
                fetch(c + 1);
            } else if (b_next < P.n) {
                point(b_next);
                fetch(0);
            }
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                if (r >= nr) break;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (c * 2 + s >= steps) break;
                    const uint4 x =
                        reinterpret_cast<const uint4*>(s_q[r])[(c * 2 + s) * 8 + part];
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        dot[i][r] = __dp4a((int)k[i][s].x, (int)x.x, dot[i][r]);
                        dot[i][r] = __dp4a((int)k[i][s].y, (int)x.y, dot[i][r]);
                        dot[i][r] = __dp4a((int)k[i][s].z, (int)x.z, dot[i][r]);
                        dot[i][r] = __dp4a((int)k[i][s].w, (int)x.w, dot[i][r]);
                    }
                }
            }
        }
        if constexpr (NR == 1) {
            const int hi = ((P.pos0 + r0) >> 2) + 1 - P.n_last;
#pragma unroll
            for (int i = 0; i < PER; i += 2) {
                float most = -INFINITY;
#pragma unroll
                for (int j = i; j < i + 2; ++j) {
                    int d = dot[j][0];
                    d += __shfl_xor_sync(0xffffffffu, d, 4);
                    d += __shfl_xor_sync(0xffffffffu, d, 2);
                    d += __shfl_xor_sync(0xffffffffu, d, 1);
                    const int b = b0 + 4 * j + sub;
                    const float v = __fmul_rn((float)d, scale[j]);
                    if (part == 0 && b < P.n) P.scores[r0 * P.stride + b] = v;
                    if (b >= P.n_first && b < hi) most = fmaxf(most, v);
                }
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 8));
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 16));
                if (lane == 0) P.maxima[r0 * (P.stride / 8) + b0 / 8 + i / 2] = most;
            }
        } else {
            // The eight lanes exchange halves of the rows, then quarters and single
            // rows: lane `part` ends up with row `part`'s sums.
            static_assert(NR == 8 && PER == 2, "a row a lane, eight blocks");
            const int row = r0 + part;
            const int hi = ((P.pos0 + row) >> 2) + 1 - P.n_last;
            float most = -INFINITY;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
#pragma unroll
                for (int half = NR / 2; half; half /= 2) {
                    const bool upper = part & half;
#pragma unroll
                    for (int r = 0; r < half; ++r) {
                        const int other = upper ? dot[j][r] : dot[j][r + half];
                        dot[j][r] = (upper ? dot[j][r + half] : dot[j][r]) +
                                    __shfl_xor_sync(0xffffffffu, other, half);
                    }
                }
                const int b = b0 + 4 * j + sub;
                const float v = __fmul_rn((float)dot[j][0], scale[j]);
                if (part < nr && b < P.n) P.scores[row * P.stride + b] = v;
                if (b >= P.n_first && b < hi) most = fmaxf(most, v);
            }
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 8));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 16));
            if (sub == 0 && part < nr) P.maxima[row * (P.stride / 8) + b0 / 8] = most;
        }
        b0 = b_next;
    }
}

template <int CHUNKS>
void launch_score_few(const FewParams& F, const DeviceInfo* di, cudaStream_t stream) {
    const bool one = F.C.rows == 1;
    const int a_cta = 8 * 4 * (CHUNKS == 1 && one ? 4 : 2);
    const int tiles = (F.n + a_cta - 1) / a_cta, cap = di->num_sms * 4;
    const dim3 grid(tiles < cap ? tiles : cap, one ? 1 : (F.C.rows + FEW_TILE - 1) / FEW_TILE);
    if (one) score_few_kernel<CHUNKS, 1><<<grid, 256, 0, stream>>>(F);
    else score_few_kernel<CHUNKS, FEW_TILE><<<grid, 256, 0, stream>>>(F);
}

// ------------------------------------------------------------ the best blocks
struct PickParams {
    int pos0;                    // position of the launch's first row
    int max_sel, n_first, n_last;
    int32_t* sel_idx;            // of the launch's first row
    int32_t* sel_cnt;
};

// A row that takes every block it sees, and the padding behind its ids.
// Returns whether the row is done.
__device__ __forceinline__ bool write_plain(const PickParams& P, const RowRange& R, int row,
                                            int32_t* out) {
    if (threadIdx.x == 0) P.sel_cnt[row] = R.take;
    for (int i = R.take + threadIdx.x; i < P.max_sel; i += blockDim.x) out[i] = -1;
    if (R.take < R.n_vis) return false;
    for (int i = threadIdx.x; i < R.take; i += blockDim.x) out[i] = i;
    return true;
}

// One CTA a row, from all its scores: all of them as candidates if they fit;
// else, with the maxima of each 8 (of more together if they are many), the
// scores that reach the need-th best maximum.  For one row this kernel runs once
// on one SM, where fetching its instructions takes longer than executing them:
// its loops stay loops (256 threads with the maxima unrolled into registers took
// 20 us where these take 17.7, with the scores).
struct ScorePick {
    PickParams K;
    const float* scores;
    long long stride;
    const float* maxima;     // [rows, stride / 8], null: none
    PickAreas A;
};

template <int THREADS>
__global__ void __launch_bounds__(THREADS) pick_kernel(const ScorePick P) {
    extern __shared__ __align__(16) uint32_t s_key[];
    __shared__ BestShared<THREADS> S;
    uint32_t* bits = s_key;
    uint32_t* const key = bits + P.A.key();
    int* const id = reinterpret_cast<int*>(bits + P.A.id());
    uint32_t* groups = bits + P.A.groups();
    int* const reach = reinterpret_cast<int*>(bits + P.A.reach());
    const int row = blockIdx.x, tid = threadIdx.x;
    const RowRange R = row_range(P.K.pos0 + row, P.K.max_sel, P.K.n_first, P.K.n_last);
    int32_t* out = P.K.sel_idx + (long long)row * P.K.max_sel;
    wait_for_previous();
    if (write_plain(P.K, R, row, out)) return;
    const float* s = P.scores + row * P.stride;
    const int n = R.hi - R.lo;
    int total = -1;          // candidates
    uint32_t least = 1, most = 1;
    if (R.need == 0 || n <= P.A.room) {
        total = R.need ? n : 0;
#pragma unroll 4
        for (int i = tid; i < total; i += THREADS) {
            key[i] = ordered(s[R.lo + i]);
            id[i] = R.lo + i;
        }
        __syncthreads();
        range_of<THREADS>(key, total, &least, &most, S);
    } else if (P.maxima) {
        const int g8 = (R.hi + 7) / 8;
        const int per = (g8 + P.A.room_groups - 1) / P.A.room_groups;
        const int n_groups = (g8 + per - 1) / per;
        const float* m = P.maxima + row * (P.stride / 8);
        if (per == 1) {
#pragma unroll 8
            for (int g = tid; g < n_groups; g += THREADS) groups[g] = ordered(m[g]);
        } else {
            for (int g = tid; g < n_groups; g += THREADS) {
                float top = -INFINITY;
                for (int i = g * per; i < min(g * per + per, g8); ++i) top = fmaxf(top, m[i]);
                groups[g] = ordered(top);
            }
        }
        if (tid == 0) S.total = S.bad = 0;
        __syncthreads();
        if (n_groups >= R.need) {
            range_of<THREADS>(groups, n_groups, &least, &most, S);
            // A quarter of the largest bounds the need-th largest from below as a
            // rule, and leaves a range of two octaves.  (Over the whole range, in
            // which most keys are those of tiny numbers, nearly all maxima would be
            // counted in a few of the parts, one after the other.)
            const uint32_t cut = ordered(0.25f * from_ordered(most));
            int reach_cut = 0;
#pragma unroll 1
            for (int g = tid; g < n_groups; g += THREADS) reach_cut += groups[g] >= cut;
            reach_cut = cta_scan<THREADS>(reach_cut, S.sums);
            if (tid == THREADS - 1) S.count = reach_cut;
            __syncthreads();
            if (S.count >= R.need && cut > least && cut <= most) least = cut;
            __syncthreads();
            // need groups, so need scores, reach the limit.
            const Limit limit =
                need_th_called<THREADS>(groups, n_groups, R.need, least, most, S);
            const uint32_t bound = limit.equals ? limit.key : limit.key + 1;
            // The groups that reach it, then their scores that do.
#pragma unroll 1
            for (int g = tid; g < n_groups; g += THREADS)
                if (groups[g] >= bound) {
                    const int at = atomicAdd(&S.bad, 1);
                    if (at < P.A.room_reach) reach[at] = g;
                }
            __syncthreads();
            const int n_reach = S.bad, each = per * 8;
            if (n_reach <= P.A.room_reach) {
#pragma unroll 1
                for (int i = tid; i < n_reach * each; i += THREADS) {
                    const int b = reach[i / each] * each + i % each;
                    if (b < R.lo || b >= R.hi) continue;
                    const uint32_t k = ordered(s[b]);
                    if (k >= bound && k > 1) {   // (1: a NaN)
                        const int to = atomicAdd(&S.total, 1);
                        if (to < P.A.room) {
                            key[to] = k;
                            id[to] = b;
                        }
                    }
                }
                __syncthreads();
                total = S.total;
                if (total < R.need || total > P.A.room) total = -1;
                least = bound;   // (no maximum is above `most`, so no score is)
            }
        }
    }
    if (total >= 0) best_of<THREADS, true>(R, key, id, total, least, most, out, bits, S);
    else scan_best<THREADS>(R, [&](int b) { return s[b]; }, out, S);
}

// ------------------------------------------------------------ the bound
struct BoundParams {
    const float* maxima;     // of the sampled blocks' groups [rows, stride]
    long long stride;
    int groups;              // of a row
    int rows;
    int pos0, max_sel, n_first, n_last;
    float* bound;            // per row
};

// Of a histogram's 256 bins the largest with at least *left entries in it and
// above; *left becomes what is left to take from it.  One warp, *left at most
// all entries.
__device__ __forceinline__ int pick_bin(const int* hist, int lane, int* left) {
    // Lane l holds bins 255 - 8 l .. 248 - 8 l, highest first.
    const int4* h = reinterpret_cast<const int4*>(hist + 248 - 8 * lane);
    const int4 low = h[0], high = h[1];
    const int c[8] = {high.w, high.z, high.y, high.x, low.w, low.z, low.y, low.x};
    int sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += c[i];
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    int bin = 255 - 8 * lane, rest = *left - (upto - sum);
    bool open = true;
#pragma unroll
    for (int i = 0; i < 7; ++i) {
        open = open && rest > c[i];
        if (open) {
            rest -= c[i];
            --bin;
        }
    }
    const int who = __ffs(__ballot_sync(0xffffffffu, upto >= *left)) - 1;
    *left = __shfl_sync(0xffffffffu, rest, who);
    return __shfl_sync(0xffffffffu, bin, who);
}

// A number that at least `need` group maxima, so at least `need` of the row's
// scores, reach: the need-th largest maximum to one part in 2^15 (neighbours score
// alike: hundreds more would reach one a percent lower), from below, by counts over
// 256 parts of the keys' range, then of the part it is in.  The smallest finite
// number if there are too few maxima; none for a row that needs none.
//
// WARPS a row: one, eight rows a CTA, up to 1024 maxima, which its lanes hold; a CTA
// of eight for more (2000 maxima of 4096 rows: 39 us, 67 with one warp).
constexpr int BOUND_ONE_WARP = 1024;

template <int WARPS>
__global__ void __launch_bounds__(256) bound_kernel(const BoundParams P) {
    constexpr int T = 32 * WARPS, ROWS = 8 / WARPS;
    constexpr int HELD = WARPS == 1 ? BOUND_ONE_WARP / 32 : 16;    // keys a lane holds
    __shared__ __align__(16) int s_hist[ROWS][256];
    __shared__ uint32_t s_part[3][8];
    const int row = blockIdx.x * ROWS + threadIdx.x / T, tid = threadIdx.x % T;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    auto sync = [] {
        if (WARPS == 1) __syncwarp();
        else __syncthreads();
    };
    // One value from all of the row's threads.
    auto greatest = [&](uint32_t v, int slot) {
        v = __reduce_max_sync(0xffffffffu, v);
        if (WARPS == 1) return v;
        if (lane == 0) s_part[slot][warp] = v;
        __syncthreads();
        return __reduce_max_sync(0xffffffffu, s_part[slot][lane % 8]);
    };
    auto total = [&](int v, int slot) {
        v = (int)__reduce_add_sync(0xffffffffu, v);
        if (WARPS == 1) return v;
        if (lane == 0) s_part[slot][warp] = (uint32_t)v;
        __syncthreads();
        return (int)__reduce_add_sync(0xffffffffu, lane < 8 ? s_part[slot][lane] : 0u);
    };
    wait_for_previous();
    if (row >= P.rows) return;
    const RowRange R = row_range(P.pos0 + row, P.max_sel, P.n_first, P.n_last);
    if (R.need == 0) {
        if (tid == 0) P.bound[row] = kNoBound;
        return;
    }
    const float* m = P.maxima + row * P.stride;
    const int n = P.groups;
    // Maxima that are not numbers above -inf count for nothing (key 0).  (-0 below
    // +0 here: a bound of either lets both through.)
    auto key_of = [&](int i) {
        const float v = m[min(i, n - 1)];
        const uint32_t u = __float_as_uint(v);
        return i < n && v > -INFINITY ? u ^ ((uint32_t)((int)u >> 31) | 0x80000000u) : 0u;
    };
    uint32_t held[HELD];
#pragma unroll
    for (int i = 0; i < HELD; ++i) held[i] = 0;
#pragma unroll
    for (int c = 0; c < HELD; c += 8) {
        if (c * T >= n) break;
#pragma unroll
        for (int i = c; i < c + 8; ++i) held[i] = key_of(i * T + tid);
    }
    auto each = [&](auto f) {
#pragma unroll
        for (int c = 0; c < HELD; c += 8) {
            if (c * T >= n) break;
#pragma unroll
            for (int i = c; i < c + 8; ++i) f(held[i]);
        }
        if constexpr (WARPS > 1) {
#pragma unroll 1
            for (int i0 = HELD * T; i0 < n; i0 += 4 * T) {
                uint32_t k[4];     // loads in flight together
#pragma unroll
                for (int u = 0; u < 4; ++u) k[u] = key_of(i0 + u * T + tid);
#pragma unroll
                for (int u = 0; u < 4; ++u) f(k[u]);
            }
        }
    };
    uint32_t most = 0, least = 0xffffffffu;
    int some = 0;
    each([&](uint32_t k) {
        most = max(most, k);
        least = min(least, k ? k : 0xffffffffu);
        some += k != 0;
    });
    most = greatest(most, 0);
    least = ~greatest(~least, 1);
    some = total(some, 2);
    float bound = -3.402823466e38f;
    if (some >= R.need) {
        int* hist = s_hist[ROWS == 1 ? 0 : warp];
        uint32_t lo = least, width = most - least;
        int left = R.need;
#pragma unroll 1
        for (;;) {
            const int shift = width >> 8 ? 24 - __clz((int)width) : 0;
            sync();
            for (int i = tid; i < 64; i += T)
                reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
            sync();
            each([&](uint32_t k) {
                if (k - lo <= width) atomicAdd(&hist[(k - lo) >> shift], 1);
            });
            sync();
            lo += (uint32_t)pick_bin(hist, lane, &left) << shift;
            if (shift <= 8) break;
            width = min((1u << shift) - 1, most - lo);
        }
        bound = from_ordered(lo);
    }
    if (tid == 0) P.bound[row] = bound;
}

// ------------------------------------------------------------ best of the candidates
constexpr int MAX_ROW_TILES = 256;   // of a launch
struct RunTable {
    uint8_t first[MAX_ROW_TILES], runs[MAX_ROW_TILES];   // pairs of each row tile
};

struct BestParams {
    PickParams K;
    DotParams D;             // the products' lists and schedule
    RunTable T;
    const float* bound;
    PickAreas A;
    IndexView V;             // for rows searched block by block
    const int8_t* codes;
};

constexpr int BEST_THREADS = 128;
constexpr int MAX_PAIRS = 80;
constexpr int MAX_LISTS = PARTS * MAX_PAIRS;   // a row tile's runs are at most the pairs

__global__ void __launch_bounds__(BEST_THREADS) best_kernel(const BestParams P) {
    extern __shared__ __align__(16) uint32_t s_bits[];
    __shared__ BestShared<BEST_THREADS> S;
    __shared__ int s_n[MAX_LISTS], s_at[MAX_LISTS];
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const RowRange R = row_range(P.K.pos0 + row, P.K.max_sel, P.K.n_first, P.K.n_last);
    int32_t* out = P.K.sel_idx + (long long)row * P.K.max_sel;
    wait_for_previous();
    if (write_plain(P.K, R, row, out)) return;
    uint32_t* const key = s_bits + P.A.key();
    int* const id = reinterpret_cast<int*>(s_bits + P.A.id());
    if (tid == 0) S.total = S.bad = 0;
    if (tid < 32) S.most[tid] = 0;
    __syncthreads();
    if (R.need > 0) {
        const int rt = row / PAIR_ROWS;
        const int lists = PARTS * P.T.runs[rt];
        const long long at = P.D.list_at(P.T.first[rt] + rt, row);
        const long long run_step = (long long)P.D.tile_rows * PARTS;
        // List l is run l / PARTS of the row tile, part l % PARTS.
        for (int l = tid; l < lists; l += BEST_THREADS) {
            const int n = P.D.counts[at + l / PARTS * run_step + l % PARTS];
            const bool bad = n < 0 || n > P.D.cap;
            const int to = bad ? 0 : atomicAdd(&S.total, n);
            if (bad || to + n > P.A.room) S.bad = 1;
            s_n[l] = n;
            s_at[l] = to;
        }
        __syncthreads();
        // A warp per part; the loads of four lists in flight together.
        uint32_t most = 0;
        if (!S.bad) {
            auto keep = [&](int i, const uint2& e) {
                const uint32_t k = ordered(__uint_as_float(e.x));
                key[i] = k;
                id[i] = (int)e.y;
                most = max(most, k);
            };
            constexpr int TOGETHER = 4;
            static_assert(BEST_THREADS / 32 == PARTS, "a warp per part");
            const long long step = run_step * P.D.cap;
            const uint2* list = P.D.list + (at + warp) * P.D.cap + lane;
            for (int l0 = warp; l0 < lists; l0 += PARTS * TOGETHER, list += step * TOGETHER) {
                uint2 e[TOGETHER];
                int n[TOGETHER];
#pragma unroll
                for (int u = 0; u < TOGETHER; ++u) {
                    const int l = l0 + u * PARTS;
                    n[u] = l < lists ? s_n[l] - lane : 0;    // this lane's and those behind
                    if (n[u] > 0) e[u] = list[u * step];
                }
#pragma unroll
                for (int u = 0; u < TOGETHER; ++u) {
                    if (n[u] <= 0) continue;
                    const int to = s_at[l0 + u * PARTS] + lane;
                    keep(to, e[u]);
                    for (int i = 32; i < n[u]; i += 32) keep(to + i, list[u * step + i]);
                }
            }
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) S.most[warp] = most;
    }
    __syncthreads();
    const int total = S.total;
    if (!S.bad && total >= R.need) {
        // Every candidate reaches the bound.
        const uint32_t least = R.need ? ordered(P.bound[row]) : 0;
        const uint32_t most = __reduce_max_sync(0xffffffffu, S.most[lane % (BEST_THREADS / 32)]);
        best_of<BEST_THREADS, false>(R, key, id, total, least, most, out, s_bits, S);
        return;
    }
    // Searched block by block; a row of zero codes, and blocks with a scale of zero
    // (an index not filled yet), need no products.
    const uint4* q = reinterpret_cast<const uint4*>(P.codes + (long long)row * P.V.width);
    bool any = false;
    for (int i = tid; i < P.V.width / 16; i += BEST_THREADS) {
        const uint4 u = q[i];
        any = any || (u.x | u.y | u.z | u.w);
    }
    const bool zero = !__syncthreads_or(any);
    scan_best<BEST_THREADS>(
        R,
        [&](int b) {
            const long long block = physical_block(P.V, b);
            const float scale = P.V.scale[block];
            int dot = 0;
            if (!zero && scale != 0.f) {
                const uint4* k = reinterpret_cast<const uint4*>(P.V.index + block * P.V.width);
#pragma unroll 8
                for (int i = 0; i < P.V.width / 16; ++i) {
                    const uint4 x = q[i], y = k[i];
                    dot = __dp4a((int)x.x, (int)y.x, dot);
                    dot = __dp4a((int)x.y, (int)y.y, dot);
                    dot = __dp4a((int)x.z, (int)y.z, dot);
                    dot = __dp4a((int)x.w, (int)y.w, dot);
                }
            }
            return __fmul_rn((float)dot, scale);
        },
        out, S);
}

// ------------------------------------------------------------ host side
size_t round256(size_t n) { return (n + 255) / 256 * 256; }
int round_up(int n, int m) { return (n + m - 1) / m * m; }

// Calls of few rows take the dp4a path.  In us by it and by the tensor cores (rows x
// blocks, 64 or 128 taken): width 256, 8 x 8192 12 and 16, 32 x 8192 17 and 17, 40 x
// 16384 24 and 22; width 512, 32 x 16384 36 and 25; width 1024, 8 x 16384 23 and 31,
// 16 x 16384 35 and 31.  Over the longest contexts: width 256, 8 x 65472 22 and 56,
// 32 x 65472 45 and 58; width 512, 8 x 65472 31 and 85; width 1024, 8 x 50000 44 and
// 108.  (A width above the call's own, as the workspace is sized for, never makes it
// few where the call is not.)
bool few_rows(int rows, int width) { return rows <= (width > 256 ? 8 : 32); }

constexpr size_t SCORE_BYTES = 128ull << 20;   // scores or maxima held at once
constexpr size_t LIST_BYTES = 1024ull << 20;   // candidates held at once

// A launch as a programmatic dependent of the kernel before it on the stream.
template <typename... Params, typename... Args>
bool launch_next(void (*kernel)(Params...), int grid, int threads, size_t smem,
                 cudaStream_t stream, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

// More rows: a sample where the scores are many and few of the blocks are taken, or
// a row has more blocks than its CTA holds.  All scores and a sample, in us (rows x
// blocks : taken): 4096 x 2048 : 8 and : 64 48 and 40, 52 and 46; 4096 x 1024 : 16
// 37 and 39; 512 x 8192 : 128 39 and 35; 284 x 16384 : 64 58 and 37; 1024 x 8192 :
// 128 56 and 41; 4096 x 32000 : 128 2890 and 120.  Less than 30 blocks per block
// taken: 4096 x 2048 : 128 54 and 52, 8000 x 2000 : 128 81 and 105, 512 x 8192 : 512
// 41 and 43; an 8th of the blocks taken: 4096 x 4096 86 and 94, 8192 204 and 184,
// 16384 857 and 382.
constexpr int SAMPLE_MIN_RATIO = 8;            // blocks per block taken
bool sampled(int rows, int n, int max_sel) {
    if (n / SAMPLE_MIN_RATIO < max_sel) return false;
    if (n > PICK_SMEM / 8) return true;
    const long long scores = (long long)rows * n;
    return n / 30 >= max_sel ? n >= 1536 && scores >= 4000000 : n >= 4000 && scores >= 16000000;
}

// The sample's products cost n / 2^skip columns and leave about 2^skip candidates
// per block taken, so it thins out with n / max_sel: at 32 skips of 0 and 1 take
// 103 and 136 us (4096 x 8192), at 64 76 and 72 (4096 x 8192), at 128 skips of 1
// and 2 89 and 91 (4096 x 16384), at 250 141 and 121 (4096 x 32000), at 511 skips
// of 2 and 3 204 and 197, at 1023 198 and 175 (4096 x 65472).
constexpr int MAX_SKIP = 3;
constexpr int SKIP_RATIO[MAX_SKIP + 1] = {SAMPLE_MIN_RATIO, 48, 160, 700};
static_assert(SAMPLE_MIN_RATIO >= 8 && 48 >= 8 << 1 && 160 >= 8 << 2 && 700 >= 8 << 3,
              "eight columns of a sample per block taken");

Sample sample_of(int n, int max_sel) {
    int skip = 0;
    while (skip < MAX_SKIP && n / SKIP_RATIO[skip + 1] >= max_sel) ++skip;
    Sample S = {skip, ((n - 1) >> skip) + 1, 0, 1, 1};
    S.cols = round_up(S.count, 8);
    int bits = 1;
    for (; S.mask < (uint32_t)S.cols - 1; S.mask = 2 * S.mask + 1) ++bits;
    S.half = bits / 2;
    return S;
}
// Groups as large as leave four times as many maxima as blocks taken (of two at
// least: a sample has eight columns per block taken).
int sample_group(const Sample& S, int max_sel) {
    int g = 1;
    while (g < 3 && (S.cols >> (g + 1)) >= 4 * max_sel) ++g;
    return g;
}
// max_sel << skip of a call on n blocks is at most this.
int most_expected(int n) {
    int most = 0;
    for (int s = 0; s <= MAX_SKIP; ++s)
        most = std::max(most, std::min((int)kMaxSelect, n / SKIP_RATIO[s]) << s);
    return most;
}

// Where a call keeps what in the workspace.  Every area grows with the rows
// and the blocks and is sized for any max_sel, so the size for a context's
// last block holds for every call on it.
struct Layout {
    long long stride;         // scores (or sampled columns) of a row
    int chunk;                // most rows of a launch, by the scores
    size_t codes, scores, maxima, codes16, cols, scale, sample_cols, sample_scale, sample_block,
        bound, list;
    size_t list_bytes, bytes;
};

// Entries of a list when max_sel << skip candidates of a row are expected: twice as
// many may be in one run, even over its parts.
int list_cap(int expected, long long tiles_per_pair) {
    const long long most = tiles_per_pair * PART, want = 2ll * expected / PARTS + 64;
    return (int)(most < want ? most : want);
}
// Lists of `rows` rows' products over `tiles` column tiles, and their numbers.
size_t list_bytes(int runs, int tile_rows, int cap) {
    return (size_t)runs * tile_rows * PARTS * (cap * sizeof(uint2) + sizeof(int));
}

// n: blocks scored; kept: columns of which a row's scores or, of 2^log2_group
// together, maxima are kept.
Layout layout(int rows, int n, int kept, int log2_group, int width, int pairs) {
    Layout L = {};
    const bool few = few_rows(rows, width);
    L.stride = round_up(kept > 0 ? kept : 1, TILE) >> log2_group;
    const size_t row_bytes = (size_t)L.stride * 4;
    size_t at = kWorkspaceCounterBytes;
    auto take = [&](size_t bytes) {
        const size_t was = at;
        at += round256(bytes);
        return was;
    };
    const size_t rows_up = few ? rows : round_up(rows, PAIR_ROWS);
    size_t scores = SCORE_BYTES > PAIR_ROWS * row_bytes ? SCORE_BYTES : PAIR_ROWS * row_bytes;
    if (rows_up * row_bytes < scores) scores = rows_up * row_bytes;
    L.chunk = rows < PAIR_ROWS * MAX_ROW_TILES ? rows : PAIR_ROWS * MAX_ROW_TILES;
    if (!few && scores / row_bytes < rows_up)
        L.chunk = min(L.chunk, (int)(scores / row_bytes / PAIR_ROWS) * PAIR_ROWS);
    L.codes = take((size_t)rows * width);
    L.scores = take(scores);
    if (few) {
        L.maxima = take(scores / 8);
    } else {
        L.codes16 = take((size_t)rows * width * 2);
        L.cols = take((size_t)n * width * 2);
        L.scale = take((size_t)round_up(n, TILE) * 4);
        L.sample_cols = take((size_t)(n + 8) * width * 2);
        L.sample_scale = take((size_t)round_up(n + 8, TILE) * 4);
        L.sample_block = take((size_t)round_up(n + 8, TILE) * 4);
        L.bound = take(rows_up * 4);
        // For any max_sel: all rows together, or as many row tiles as LIST_BYTES hold.
        auto lists = [&](int row_tiles) {
            const long long total = (long long)row_tiles * (round_up(n, TILE) / TILE);
            const int G = (int)std::min<long long>(std::max(total, 1ll), pairs);
            return list_bytes(G + row_tiles, std::min(rows, PAIR_ROWS),
                              list_cap(most_expected(n), (total + G - 1) / G));
        };
        L.list_bytes = std::min(lists(std::min((int)(rows_up / PAIR_ROWS), MAX_ROW_TILES)),
                                std::max(LIST_BYTES, lists(1)));
        L.list = take(L.list_bytes);
    }
    L.bytes = at;
    return L;
}

// Pairs that can be resident at once (both SMs of a pair in one GPC).
int max_pairs(const DeviceInfo* di) {
    static std::atomic<int> cached[64];
    if (di->device < 64) {
        const int c = cached[di->device].load(std::memory_order_relaxed);
        if (c) return c;
    }
    if (ensure_smem_limit(reinterpret_cast<const void*>(dot_kernel<SCORES, true>),
                          DotCfg<true>::SMEM) != GQA_OK)
        return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(DOT_THREADS, 1, 1);
    cfg.dynamicSmemBytes = DotCfg<true>::SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, dot_kernel<SCORES, true>, &cfg) != cudaSuccess ||
        n < 1) {
        cudaGetLastError();
        return 0;
    }
    if (n > di->num_sms / 2) n = di->num_sms / 2;
    if (n > MAX_PAIRS) n = MAX_PAIRS;
    if (di->device < 64) cached[di->device].store(n, std::memory_order_relaxed);
    return n;
}

// The schedule of a launch's products, and each row tile's runs.
template <int MODE>
void schedule(DotParams& D, int pairs, RunTable* table = nullptr) {
    D.row_tiles = (D.rows + PAIR_ROWS - 1) / PAIR_ROWS;
    D.total = 0;
    for (int t = 0; t < D.row_tiles; ++t) D.total += col_tiles<MODE>(D, t);
    D.G = (int)(D.total < pairs ? D.total : pairs);
    if (!table) return;
    long long cum = 0;
    for (int t = 0; t < D.row_tiles; ++t) {
        const int n = col_tiles<MODE>(D, t);
        table->first[t] = table->runs[t] = 0;
        if (n > 0) {
            table->first[t] = (uint8_t)pair_of(D, cum);
            table->runs[t] = (uint8_t)(pair_of(D, cum + n - 1) - table->first[t] + 1);
        }
        cum += n;
    }
}

// cols: [n, width].
template <int MODE>
int launch_dots(const __half* rows16, const __half* cols, int n, const DotParams& D,
                cudaStream_t stream) {
    if (D.total == 0) return GQA_OK;
    const int width = D.chunks * 64;
    CUtensorMap tr, tc;
    if (!make_map_2d_f16(&tr, rows16, D.rows, width, width, CTA_ROWS, 64) ||
        !make_map_2d_f16(&tc, cols, n, width, width, CTA_ROWS, 64))
        return GQA_ERR_CUDA;
    const bool resident = D.chunks <= RES_CHUNKS;
    const int smem = resident ? DotCfg<true>::SMEM : DotCfg<false>::SMEM;
    auto* kernel = resident ? dot_kernel<MODE, true> : dot_kernel<MODE, false>;
    if (ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem) != GQA_OK)
        return GQA_ERR_CUDA;
    return launch_next(kernel, 2 * D.G, DOT_THREADS, smem, stream, tr, tc, D) ? GQA_OK
                                                                             : GQA_ERR_CUDA;
}

template <int THREADS>
int launch_pick(const PickParams& K, int rows, const float* scores, long long stride,
                const float* maxima, int n, cudaStream_t stream) {
    static_assert(PICK_MOST_TAKEN == kMaxSelect, "room for the groups that are reached");
    const ScorePick P = {K, scores, stride, maxima,
                         pick_areas(((K.pos0 + rows - 1) >> 2) + 1, n, K.max_sel, maxima)};
    if (ensure_smem_limit(reinterpret_cast<const void*>(pick_kernel<THREADS>), PICK_MOST_BYTES) !=
        GQA_OK)
        return GQA_ERR_CUDA;
    return launch_next(pick_kernel<THREADS>, rows, THREADS, P.A.bytes(), stream, P)
               ? GQA_OK
               : GQA_ERR_CUDA;
}

}  // namespace select

size_t select_blocks_workspace_bytes(int rows, int ctx_len, int width) {
    using namespace select;
    const DeviceInfo* di = device_info();
    const int pairs = di ? max_pairs(di) : 0;
    if (pairs < 1) return 0;
    const int n = (ctx_len - 1) / 4 + 1;
    return layout(rows, n, n, 0, width, pairs).bytes;
}

int select_blocks_launch(const void* q, const int8_t* index, const float* index_scale,
                         const int32_t* block_table, int num_pages, int page, int ctx_len,
                         int rows, int Hq, int Hkv, int D, int max_sel, int n_first, int n_last,
                         int32_t* sel_idx, int32_t* sel_cnt, cudaStream_t stream) {
    using namespace select;
    const DeviceInfo* di = device_info();
    if (!di) return GQA_ERR_CUDA;
    const int width = Hkv * D;
    const bool few = few_rows(rows, width);
    // Blocks below the last row's always-taken ones.
    int n = ((ctx_len - 1) >> 2) + 1 - n_last;
    // Nothing to score: no block is left, every row takes all it sees, or only the
    // first and last ones.
    if (n <= n_first || n + n_last <= max_sel || n_first + n_last == max_sel) n = 0;
    const bool sample = !few && sampled(rows, n, max_sel);
    const Sample S = sample ? sample_of(n, max_sel) : Sample{};
    const int log2_group = sample ? sample_group(S, max_sel) : 0;
    const int kept = sample ? S.cols : n;
    const int pairs = max_pairs(di);
    if (pairs < 1) return GQA_ERR_CUDA;
    const Layout L = layout(rows, n, kept, log2_group, width, pairs);
    void* ws;
    size_t ws_bytes;
    current_workspace(&ws, &ws_bytes);
    if (!ws || ws_bytes < L.bytes) return GQA_ERR_WORKSPACE;
    uint8_t* w = static_cast<uint8_t*>(ws);
    int8_t* codes = reinterpret_cast<int8_t*>(w + L.codes);
    float* scores = reinterpret_cast<float*>(w + L.scores);
    const IndexView V = {index, index_scale, block_table, num_pages,
                         __builtin_ctz((unsigned)page) - 2, width, di->err_word};
    CodeParams C = {static_cast<const __half*>(q), rows, Hq, D, Hq / Hkv, width, codes, nullptr};
    const int pos0 = ctx_len - rows;
    PickParams K = {pos0, max_sel, n_first, n_last, sel_idx, sel_cnt};
    int rc = GQA_OK;
    if (few) {
        float* maxima = reinterpret_cast<float*>(w + L.maxima);
        if (n > 0) {
            const FewParams F = {C, V, n, pos0, n_first, n_last, scores, L.stride, maxima};
            if (width <= 256) launch_score_few<1>(F, di, stream);
            else launch_score_few<4>(F, di, stream);
        }
        rc = launch_pick<1024>(K, rows, scores, L.stride, maxima, n, stream);
        if (rc != GQA_OK) return rc;
        return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
    }
    __half* codes16 = reinterpret_cast<__half*>(w + L.codes16);
    __half* cols = reinterpret_cast<__half*>(w + L.cols);
    float* scale = reinterpret_cast<float*>(w + L.scale);
    __half* sample_cols = reinterpret_cast<__half*>(w + L.sample_cols);
    float* sample_scale = reinterpret_cast<float*>(w + L.sample_scale);
    int* sample_block = reinterpret_cast<int*>(w + L.sample_block);
    C.codes16 = codes16;
    if (n > 0) {
        const ExpandParams E = {V, n, cols, scale, sample ? sample_cols : nullptr, sample_scale,
                                sample_block, S, n_first};
        const int code_ctas = (rows + 7) / 8;
        const int a_cta = 256 / (width / 16) * EXPAND_PASSES;
        const int ctas = code_ctas + (n + a_cta - 1) / a_cta;
        if (width <= 256) prepare_kernel<1><<<ctas, 256, 0, stream>>>(C, E, code_ctas);
        else prepare_kernel<4><<<ctas, 256, 0, stream>>>(C, E, code_ctas);
    }
    if (sample && ensure_smem_limit(reinterpret_cast<const void*>(best_kernel),
                                    BEST_MOST_BYTES) != GQA_OK)
        return GQA_ERR_CUDA;
    int step = L.chunk;
    for (int r0 = 0; r0 < rows; r0 += step) {
        DotParams P = {};
        P.rows = rows - r0 < step ? rows - r0 : step;
        P.chunks = width / 64;
        P.pos0 = pos0 + r0;
        P.n_first = n_first;
        P.n_last = n_last;
        P.scores = scores;
        P.stride = L.stride;
        P.err = di->err_word;
        K.pos0 = pos0 + r0;
        K.sel_idx = sel_idx + (size_t)r0 * max_sel;
        K.sel_cnt = sel_cnt + r0;
        const __half* rows16 = codes16 + (size_t)r0 * width;
        if (!sample) {
            P.scale = scale;
            schedule<SCORES>(P, pairs);
            if (n > 0) rc = launch_dots<SCORES>(rows16, cols, n, P, stream);
            // More threads a row where rows are few, or so long that one or two fill an
            // SM (rows x blocks, 256 and 1024 threads: 128 x 16384 36 and 25 us, 300 x
            // 5000 28 and 26, 474 x 10311 63 and 61; 900 x 8192 50 and 63, 200 x 2048
            // 22 and 25).
            const bool wide = n >= 4096 && (P.rows <= 2 * di->num_sms || n >= 10000);
            if (rc == GQA_OK)
                rc = wide ? launch_pick<1024>(K, P.rows, scores, L.stride, nullptr, n, stream)
                          : launch_pick<256>(K, P.rows, scores, L.stride, nullptr, n, stream);
            if (rc != GQA_OK) return rc;
            continue;
        }
        DotParams R = P;     // the candidates' products
        RunTable table;
        // Fewer rows a launch if their candidate lists would not fit.
        for (;;) {
            schedule<CANDIDATES>(R, pairs, &table);
            R.tile_rows = R.rows < PAIR_ROWS ? R.rows : PAIR_ROWS;
            R.cap = R.G > 0 ? list_cap(max_sel << S.skip, (R.total + R.G - 1) / R.G) : 32;
            if (list_bytes(R.runs(), R.tile_rows, R.cap) <= L.list_bytes) break;
            if (R.rows <= PAIR_ROWS) return GQA_ERR_WORKSPACE;   // layout() leaves room for these
            step = round_up(R.rows, PAIR_ROWS) - PAIR_ROWS;
            P.rows = R.rows = step;
        }
        P.scale = sample_scale;
        P.cols = S.cols;
        P.block = sample_block;
        P.log2_group = log2_group;
        schedule<MAXIMA>(P, pairs);
        rc = launch_dots<MAXIMA>(rows16, sample_cols, S.cols, P, stream);
        if (rc != GQA_OK) return rc;
        float* bound = reinterpret_cast<float*>(w + L.bound);
        const BoundParams B = {scores, P.stride, kept >> log2_group, P.rows, K.pos0, max_sel, n_first,
                               n_last, bound};
        if (!(B.groups <= BOUND_ONE_WARP
                  ? launch_next(bound_kernel<1>, (P.rows + 7) / 8, 256, 0, stream, B)
                  : launch_next(bound_kernel<8>, P.rows, 256, 0, stream, B)))
            return GQA_ERR_CUDA;
        R.scale = scale;
        R.bound = bound;
        R.list = reinterpret_cast<uint2*>(w + L.list);
        R.counts = reinterpret_cast<int*>(
            R.list + (size_t)R.runs() * R.tile_rows * PARTS * R.cap);
        rc = launch_dots<CANDIDATES>(rows16, cols, n, R, stream);
        if (rc != GQA_OK) return rc;
        const BestParams T = {
            K, R, table, bound,
            best_areas(((K.pos0 + R.rows - 1) >> 2) + 1, max_sel << S.skip, max_sel), V,
            codes + (size_t)r0 * width};
        if (!launch_next(best_kernel, R.rows, BEST_THREADS, T.A.bytes(), stream, T))
            return GQA_ERR_CUDA;
    }
    return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace gqa

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
// Few rows: every block's scores by dp4a straight from the int8 index, then
// one CTA a row finds the best.  More rows: the tensor cores (dot_kernel).
// With many blocks, writing rows x blocks scores and reading them back would
// cost several times the products themselves, so only every 8th block's are
// written; the k-th best of those bounds the k-th best of all from below
// (bound_kernel), and the other blocks' products are compared with that bound
// as they leave the tensor memory, keeping about 7 k candidates a row.  One
// CTA a row then takes the best of the candidates (best_kernel).  A row whose
// candidates do not fit (thousands of equal scores) is searched block by block.
#include <atomic>
#include <cuda_fp16.h>

#include "internal.h"
#include "pair_mma.cuh"
#include "sm100.cuh"

namespace gqa {
namespace select {

constexpr int STRIDE = 8;   // every STRIDE-th block is in the sample

// Columns of the score products: all blocks in order, the sampled blocks
// (0, 8, 16, ...), or the rest in order.
enum Order { ALL = 0, SAMPLE = 1, REST = 2 };

template <int ORDER>
__host__ __device__ __forceinline__ int col_block(int c) {
    return ORDER == ALL ? c : ORDER == SAMPLE ? c * STRIDE
                                              : c / (STRIDE - 1) * STRIDE + c % (STRIDE - 1) + 1;
}
// Columns whose block is below hi (a prefix in each order).
template <int ORDER>
__host__ __device__ __forceinline__ int cols_below(int hi) {
    if (hi <= 0) return 0;
    const int s = (hi + STRIDE - 1) / STRIDE;
    return ORDER == ALL ? hi : ORDER == SAMPLE ? s : hi - s;
}

// What a row takes: blocks below n_first and from hi on always, `need` of the
// scored blocks [n_first, hi).
struct RowRange {
    int n_vis, take, lo, hi, need;
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

// A float's order as whole numbers; NaN below everything.  Adding zero makes
// the two zeros one.
__device__ __forceinline__ uint32_t ordered(float f) {
    if (f != f) return 0;
    const uint32_t u = __float_as_uint(f + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
constexpr uint32_t kOrderedMinusInf = 0x007fffffu;

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
// heads of KV head g.  fp16 values are whole multiples of 2^-24 below 2^41 of
// them, so the sums are exact as 64-bit whole numbers; S is rounded to 32 bits
// once.  A row with an infinity or NaN gets codes of zero.  One warp a row.
struct CodeParams {
    const __half* q;
    int rows, Hq, D, group, width;
    int8_t* codes;
    __half* codes16;   // the same codes as fp16 (null: not wanted)
};

__device__ __forceinline__ void query_codes(const CodeParams& P, int row, int lane) {
    float s[8][4];
    float most = 0.f;
    bool fine = true;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        if (c * 128 >= P.width) break;
        const int g = c * 128 / P.D;
        const __half* src = P.q + ((long long)row * P.Hq + g * P.group) * P.D +
                            (c * 128 - g * P.D) + lane * 4;
        long long sum[4] = {0, 0, 0, 0};
        for (int h = 0; h < P.group; ++h) {
            const uint2 u = *reinterpret_cast<const uint2*>(src + (long long)h * P.D);
            const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
            const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
            const float f[4] = {f0.x, f0.y, f1.x, f1.y};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                fine = fine && fabsf(f[j]) <= 65504.f;
                sum[j] += __float2ll_rn(f[j] * 16777216.f);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[c][j] = __ll2float_rn(sum[j]);
            most = fmaxf(most, fabsf(s[c][j]));
        }
    }
    fine = __all_sync(0xffffffffu, fine);
    most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
    fine = fine && most > 0.f;
    // The sums carry a factor 2^24, as `most` does: the codes see their ratio.
    const float inv = fine ? 127.f / (most * (1.f / 16777216.f)) : 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        if (c * 128 >= P.width) break;
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int code =
                fine ? (int)rintf(__fmul_rn(s[c][j] * (1.f / 16777216.f), inv)) : 0;
            w |= (uint32_t)(code & 0xff) << (8 * j);
        }
        const long long at = (long long)row * P.width + c * 128 + lane * 4;
        *reinterpret_cast<uint32_t*>(P.codes + at) = w;
        if (P.codes16) *reinterpret_cast<uint2*>(P.codes16 + at) = codes_half4(w);
    }
}

// The index's columns as the tensor cores read them: fp16 codes in column
// order and the columns' scales.
struct ExpandParams {
    IndexView V;
    int n_first_cols;    // columns of the first map (ALL or SAMPLE)
    int n_rest_cols;     // columns of the REST map (0 when all are in the first)
    bool sampled;
    __half* first;
    __half* rest;
    float* first_scale;
    float* rest_scale;
};

// The first `code_ctas` CTAs make query codes (8 rows each), the others
// expand columns (16 codes a thread).
__global__ void __launch_bounds__(256) prepare_kernel(const CodeParams C, const ExpandParams E,
                                                      int code_ctas) {
    if ((int)blockIdx.x < code_ctas) {
        const int row = blockIdx.x * 8 + threadIdx.x / 32;
        if (row < C.rows) query_codes(C, row, threadIdx.x % 32);
        return;
    }
    const int per_col = E.V.width / 16;
    const long long i = (long long)(blockIdx.x - code_ctas) * 256 + threadIdx.x;
    const int c = (int)(i / per_col), part = (int)(i - (long long)c * per_col);
    if (c >= E.n_first_cols + E.n_rest_cols) return;
    const bool rest = c >= E.n_first_cols;
    const int col = rest ? c - E.n_first_cols : c;
    const int b = rest ? col_block<REST>(col) : E.sampled ? col_block<SAMPLE>(col) : col;
    const long long block = physical_block(E.V, b);
    const uint4 w = *reinterpret_cast<const uint4*>(E.V.index + block * E.V.width + part * 16);
    __half* dst = (rest ? E.rest : E.first) + (long long)col * E.V.width + part * 16;
    const uint2 x = codes_half4(w.x), y = codes_half4(w.y), z = codes_half4(w.z),
                u = codes_half4(w.w);
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(x.x, x.y, y.x, y.y);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(z.x, z.y, u.x, u.y);
    if (part == 0) (rest ? E.rest_scale : E.first_scale)[col] = E.V.scale[block];
}

// ------------------------------------------------------------ products
// rows x columns products on CTA pairs: a pair takes 256 rows (128 a CTA) and
// walks 256-column tiles, each CTA holding half of every column tile, one
// M = 256, N = 256 UMMA stream issued by the even CTA into two tensor-memory
// buffers.  Up to width 256 a pair keeps its rows' codes in shared memory for
// all its tiles; beyond, they stream with the columns.  Warp 0 loads, warp 1
// issues, warps 2..9 take the products: each thread one row and half of a
// tile's columns.
constexpr int CTA_ROWS = 128;
constexpr int PAIR_ROWS = 256;
constexpr int TILE = 256;                    // columns of a tile
constexpr int CHUNK_BYTES = 128 * 128;       // 128 rows x 64 fp16
constexpr int RES_CHUNKS = 4;                // row chunks kept (width 256)
constexpr int EPI_WARPS = 8;
constexpr int DOT_THREADS = 32 * (2 + EPI_WARPS);
constexpr uint32_t DOT_TMEM = 512;
constexpr uint32_t IDESC = idesc_f16_f32(256, TILE, false, false);

template <bool RESIDENT>
struct DotCfg {
    static constexpr int SLOTS = RESIDENT ? 8 : 6;
    static constexpr int SLOT_BYTES = RESIDENT ? CHUNK_BYTES : 2 * CHUNK_BYTES;
    static constexpr int ROW_BYTES = RESIDENT ? RES_CHUNKS * CHUNK_BYTES : 0;
    static constexpr int NUM_BARS = 2 * SLOTS + 7;
    static constexpr int SMEM = 1024 + ROW_BYTES + SLOTS * SLOT_BYTES + NUM_BARS * 8 + 16;
    static_assert(SMEM <= 232448, "shared memory");
};

struct DotParams {
    int rows;                  // rows of the launch
    int chunks;                // width / 64
    int row_tiles;
    int G;                     // pairs
    long long total;           // (row tile, column tile) products
    int pos0;                  // position of the first row
    int max_sel, n_first, n_last;
    const float* scale;        // per column, allocated to a multiple of TILE
    float* scores;             // ALL, SAMPLE: [rows, stride]
    long long stride;
    const float* bound;        // REST: per row
    uint2* list;               // REST: (score, column) [rows][segs][2][cap]
    int* counts;               // REST: entries found [rows][segs][2]
    int segs, cap;
    unsigned* err;
};

template <int ORDER>
__host__ __device__ __forceinline__ int col_tiles(const DotParams& P, int rt) {
    const int last = min(rt * PAIR_ROWS + PAIR_ROWS, P.rows) - 1;
    const int hi = ((P.pos0 + last) >> 2) + 1 - P.n_last;
    return (cols_below<ORDER>(hi) + TILE - 1) / TILE;
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
template <int ORDER>
struct Runs {
    long long pos, end, cum;
    int rt;
    __device__ void init(const DotParams& P, int pair) {
        pos = pair_begin(P, pair);
        end = pair_begin(P, pair + 1);
        cum = 0;
        rt = 0;
        while (rt < P.row_tiles) {
            const int n = col_tiles<ORDER>(P, rt);
            if (cum + n > pos) break;
            cum += n;
            ++rt;
        }
    }
    // seg: this run's number among its row tile's runs.
    __device__ bool next(const DotParams& P, int pair, int& t, int& jb, int& je, int& seg) {
        if (pos >= end) return false;
        int n = col_tiles<ORDER>(P, rt);
        while (n == 0) n = col_tiles<ORDER>(P, ++rt);
        t = rt;
        jb = (int)(pos - cum);
        je = (int)min((long long)n, end - cum);
        seg = pair - pair_of(P, cum);
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

template <int ORDER, bool RESIDENT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(DOT_THREADS, 1)
dot_kernel(const __grid_constant__ CUtensorMap tm_rows, const __grid_constant__ CUtensorMap tm_cols,
           const DotParams P) {
    using C = DotCfg<RESIDENT>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* base_ptr = smem_raw + (base - smem_u32(smem_raw));
    const uint32_t s_rows = base;
    const uint32_t s_ring = base + C::ROW_BYTES;
    const uint32_t bars = s_ring + C::SLOTS * C::SLOT_BYTES;
    auto full = [&](int s) { return bars + 8 * s; };
    auto empty = [&](int s) { return bars + 8 * (C::SLOTS + s); };
    const uint32_t rows_full = bars + 8 * (2 * C::SLOTS), rows_empty = rows_full + 8;
    auto tfull = [&](int i) { return rows_full + 16 + 8 * i; };    // products in buffer i
    auto tempty = [&](int i) { return rows_full + 32 + 8 * i; };   // buffer i read out
    const uint32_t drain = rows_full + 48;
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(base_ptr + C::ROW_BYTES +
                                                     C::SLOTS * C::SLOT_BYTES + C::NUM_BARS * 8);
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

    Runs<ORDER> runs;
    runs.init(P, pair);
    int rt, jb, je, seg;
    if (warp == 0) {
        // ------------------------------------------------------------ loads
        // Completions of both CTAs' halves land on the even CTA's barriers.
        if (lane == 0) {
            uint32_t n = 0;     // slots filled
            int run = 0;
            bool ok = true;
            while (ok && runs.next(P, pair, rt, jb, je, seg)) {
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
            while (ok && runs.next(P, pair, rt, jb, je, seg)) {
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
        const int half = (warp - 2) >> 2;      // which 128 columns of a tile
        const int quarter = warp & 3;          // TMEM lanes this warp may read
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16) + half * 128;
        uint32_t t = 0;
        bool ok = true;
        while (ok && runs.next(P, pair, rt, jb, je, seg)) {
            const int row0 = rt * PAIR_ROWS + CTA_ROWS * (int)rank + quarter * 32;
            const int row = row0 + lane;
            const bool valid = row < P.rows;
            const int hi = ((P.pos0 + row) >> 2) + 1 - P.n_last;     // this row's scored blocks end
            const int hi0 = ((P.pos0 + row0) >> 2) + 1 - P.n_last;   // the warp's smallest
            const float bound = ORDER == REST ? (valid ? P.bound[row] : INFINITY) : 0.f;
            const long long at = (((long long)row * P.segs + seg) * 2 + half);
            uint2* list = ORDER == REST ? P.list + at * P.cap : nullptr;
            int found = 0;
            const int last = P.cap - 1;
            for (int j = jb; j < je; ++j, ++t) {
                ok = mbar_wait(tfull(t & 1), (t >> 1) & 1, abort_flag, P.err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const int col0 = j * TILE + half * 128;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    uint32_t r[32];
                    tmem_ld32(t_lane + (t & 1) * TILE + g * 32, r);
                    float sc[32];
                    const float4* src = reinterpret_cast<const float4*>(P.scale + col0 + g * 32);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 f = __ldg(src + i);
                        sc[4 * i] = f.x;
                        sc[4 * i + 1] = f.y;
                        sc[4 * i + 2] = f.z;
                        sc[4 * i + 3] = f.w;
                    }
                    tmem_ld_wait<32>(r);
                    if (g == 3) {
                        // The buffer is read out.
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) pairs::remote_arrive(pairs::leader_addr(tempty(t & 1)));
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        sc[i] = __fmul_rn(__uint_as_float(r[i]), sc[i]);
                    const int c0 = col0 + g * 32;
                    if (ORDER != REST) {
                        if (valid) {
                            float* dst = P.scores + row * P.stride + c0;
#pragma unroll
                            for (int i = 0; i < 4; ++i) store8(dst + 8 * i, sc + 8 * i);
                        }
                    } else {
                        const bool whole = col_block<ORDER>(c0) >= P.n_first &&
                                           col_block<ORDER>(c0 + 31) < hi0;
                        if (!whole) {
                            // A tile on the rows' own blocks, or on the first ones.
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const int b = col_block<ORDER>(c0 + i);
                                if (b < P.n_first || b >= hi) sc[i] = __int_as_float(0x7fc00000);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (sc[i] >= bound) {
                                list[min(found, last)] =
                                    make_uint2(__float_as_uint(sc[i]), (uint32_t)(c0 + i));
                                ++found;
                            }
                    }
                }
            }
            if (ORDER == REST && valid) P.counts[at] = found;
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

// Few rows: eight lanes read one block's codes (16 bytes at a time) and take
// its dots with up to SMALL_ROWS rows.
constexpr int SMALL_ROWS = 8;

struct SmallParams {
    IndexView V;
    const int8_t* codes;
    int rows;
    int n;                       // blocks
    float* scores;               // [rows, stride]
    long long stride;
};

__global__ void __launch_bounds__(256) score_small_kernel(const SmallParams P) {
    __shared__ __align__(16) int8_t s_q[SMALL_ROWS][kMaxIndexWidth];
    const int width = P.V.width;
    const int r0 = blockIdx.y * SMALL_ROWS;
    const int nr = min(SMALL_ROWS, P.rows - r0);
    for (int i = threadIdx.x; i < SMALL_ROWS * width / 16; i += 256) {
        const int r = i / (width / 16), c = i - r * (width / 16);
        reinterpret_cast<uint4*>(s_q[r])[c] =
            r < nr ? *reinterpret_cast<const uint4*>(P.codes + (long long)(r0 + r) * width + c * 16)
                   : make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    const int lane = threadIdx.x % 8;
    for (int b0 = blockIdx.x * 32; b0 < P.n; b0 += gridDim.x * 32) {
        const int b = b0 + threadIdx.x / 8;
        const bool live = b < P.n;
        const long long block = physical_block(P.V, live ? b : b0);
        const uint4* src = reinterpret_cast<const uint4*>(P.V.index + block * width);
        int dot[SMALL_ROWS];
#pragma unroll
        for (int r = 0; r < SMALL_ROWS; ++r) dot[r] = 0;
        for (int c = lane; c < width / 16; c += 8) {
            const uint4 k = src[c];
#pragma unroll
            for (int r = 0; r < SMALL_ROWS; ++r) {
                if (r >= nr) break;
                const uint4 x = reinterpret_cast<const uint4*>(s_q[r])[c];
                dot[r] = __dp4a((int)k.x, (int)x.x, dot[r]);
                dot[r] = __dp4a((int)k.y, (int)x.y, dot[r]);
                dot[r] = __dp4a((int)k.z, (int)x.z, dot[r]);
                dot[r] = __dp4a((int)k.w, (int)x.w, dot[r]);
            }
        }
        const float scale = P.V.scale[block];
#pragma unroll
        for (int r = 0; r < SMALL_ROWS; ++r) {
            if (r >= nr) break;
            int d = dot[r];
            d += __shfl_xor_sync(0xffffffffu, d, 4);
            d += __shfl_xor_sync(0xffffffffu, d, 2);
            d += __shfl_xor_sync(0xffffffffu, d, 1);
            if (lane == 0 && live) P.scores[(r0 + r) * P.stride + b] = __fmul_rn((float)d, scale);
        }
    }
}

// ------------------------------------------------------------ the best blocks
struct PickParams {
    int pos0;                    // position of the launch's first row
    int max_sel, n_first, n_last;
    int32_t* sel_idx;            // of the launch's first row
    int32_t* sel_cnt;
};

// Largest digit d of a 256-bin histogram with at least *left entries in bins
// >= d; *left becomes what is left to take from bin d.  One warp; the result
// in every lane.
__device__ __forceinline__ int pick_digit(const int* hist, int lane, int* left) {
    // Lane l holds bins 255 - 8 l .. 248 - 8 l, highest first.
    int c[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = hist[255 - 8 * lane - i];
        sum += c[i];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    const uint32_t m = __ballot_sync(0xffffffffu, incl >= *left);
    const int who = m ? __ffs(m) - 1 : 31;
    int rest = *left - (incl - sum), d = 255 - 8 * lane;
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (rest > c[i] && 255 - 8 * lane - i == d) {
            rest -= c[i];
            --d;
        }
    *left = __shfl_sync(0xffffffffu, rest, who);
    return __shfl_sync(0xffffffffu, d, who);
}

struct ScanShared {
    int hist[256];
    uint32_t prefix;
    int need;
    int above[32], equal[32];
};

// The best blocks of one row by its scores, one after the other (score(b) for
// lo <= b < hi): the key of the last one taken is found eight bits at a time,
// then one pass over the blocks in order writes those above it and the first
// of those equal to it.  Called by all threads of a CTA.
template <int THREADS, typename Score>
__device__ void scan_best(const RowRange& R, const Score& score, int32_t* out, ScanShared& S) {
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    uint32_t prefix = 0;
    int need = R.need;
    if (need > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += THREADS) S.hist[i] = 0;
            __syncthreads();
            for (int b = R.lo + tid; b < R.hi; b += THREADS) {
                const uint32_t k = ordered(score(b));
                if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
                    atomicAdd(&S.hist[(k >> shift) & 255], 1);
            }
            __syncthreads();
            if (warp == 0) {
                int left = need;
                const int d = pick_digit(S.hist, lane, &left);
                if (lane == 0) {
                    S.need = left;
                    S.prefix = prefix | ((uint32_t)d << shift);
                }
            }
            __syncthreads();
            prefix = S.prefix;
            need = S.need;
        }
    } else {
        prefix = 0xffffffffu;
    }
    // need = how many of the blocks with key == prefix are taken (lowest ids).
    int n_above = 0, n_equal = 0;   // so far, in blocks below b0
    for (int b0 = 0; b0 < R.n_vis; b0 += THREADS) {
        const int b = b0 + tid;
        bool above = false, equal = false;
        if (b < R.n_vis) {
            if (b < R.lo || b >= R.hi) above = true;
            else {
                const uint32_t k = ordered(score(b));
                above = k > prefix;
                equal = k == prefix && need > 0;
            }
        }
        const uint32_t ma = __ballot_sync(0xffffffffu, above);
        const uint32_t me = __ballot_sync(0xffffffffu, equal);
        if (lane == 0) {
            S.above[warp] = __popc(ma);
            S.equal[warp] = __popc(me);
        }
        __syncthreads();
        int a = n_above, e = n_equal;
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) {
                a += S.above[w];
                e += S.equal[w];
            }
            n_above += S.above[w];
            n_equal += S.equal[w];
        }
        const uint32_t below = (1u << lane) - 1;
        a += __popc(ma & below);
        e += __popc(me & below);
        if (above || (equal && e < need)) out[a + min(e, need)] = b;
        __syncthreads();
    }
}

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

// One CTA a row, from all its scores.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) pick_kernel(const PickParams P, const float* scores,
                                                       long long stride) {
    __shared__ ScanShared S;
    const int row = blockIdx.x;
    const RowRange R = row_range(P.pos0 + row, P.max_sel, P.n_first, P.n_last);
    int32_t* out = P.sel_idx + (long long)row * P.max_sel;
    if (write_plain(P, R, row, out)) return;
    const float* s = scores + row * stride;
    scan_best<THREADS>(R, [&](int b) { return s[b]; }, out, S);
}

// ------------------------------------------------------------ the bound
struct BoundParams {
    const float* scores;     // the sampled blocks' [rows, stride]
    long long stride;
    int pos0, max_sel, n_first, n_last;
    float* bound;            // per row
    uint2* list;             // (score, column) of the sample's own candidates [rows][cap]
    int* counts;             // their number; -1: too many, the row is searched block by block
    int cap;
};

// A lower bound on the need-th best score, from the sample: the leading 22 bits
// of the sample's need-th best (11 bits at a time), -inf if the sample is
// smaller than need, +inf for a row that needs none.
__global__ void __launch_bounds__(256) bound_kernel(const BoundParams P) {
    __shared__ int s_hist[2048];
    __shared__ int s_sum[8];
    __shared__ int s_digit, s_left, s_count;
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const RowRange R = row_range(P.pos0 + row, P.max_sel, P.n_first, P.n_last);
    if (R.need == 0) {
        if (tid == 0) {
            P.bound[row] = INFINITY;
            P.counts[row] = 0;
        }
        return;
    }
    const float* s = P.scores + row * P.stride;
    const int c0 = (R.lo + STRIDE - 1) / STRIDE, c1 = cols_below<SAMPLE>(R.hi);
    uint32_t prefix = 0;
    if (c1 - c0 >= R.need) {
        int need = R.need;
        for (int shift = 21; shift >= 10; shift -= 11) {
            for (int i = tid; i < 2048; i += 256) s_hist[i] = 0;
            __syncthreads();
            for (int c = c0 + tid; c < c1; c += 256) {
                const uint32_t k = ordered(s[c]);
                if (shift == 21 || (k >> 21) == (prefix >> 21))
                    atomicAdd(&s_hist[(k >> shift) & 2047], 1);
            }
            __syncthreads();
            // Thread t holds bins 2047 - 8 t .. 2040 - 8 t, highest first.
            int cnt[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                cnt[i] = s_hist[2047 - 8 * tid - i];
                sum += cnt[i];
            }
            int incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (lane == 31) s_sum[warp] = incl;
            __syncthreads();
            for (int w = 0; w < warp; ++w) incl += s_sum[w];
            int before = incl - sum;
            if (before < need && need <= incl) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (before < need && need <= before + cnt[i]) {
                        s_digit = 2047 - 8 * tid - i;
                        s_left = need - before;
                    }
                    before += cnt[i];
                }
            }
            __syncthreads();
            prefix |= (uint32_t)s_digit << shift;
            need = s_left;
        }
    }
    float bound = -INFINITY;
    if (prefix > kOrderedMinusInf)
        bound = __uint_as_float(prefix & 0x80000000u ? prefix & 0x7fffffffu : ~prefix);
    if (tid == 0) s_count = 0;
    __syncthreads();
    uint2* list = P.list + (long long)row * P.cap;
    for (int c = c0 + tid; c < c1; c += 256) {
        const float v = s[c];
        if (v >= bound) {
            const int i = atomicAdd(&s_count, 1);
            if (i < P.cap) list[i] = make_uint2(__float_as_uint(v), (uint32_t)c);
        }
    }
    __syncthreads();
    if (tid == 0) {
        const bool fits = s_count <= P.cap;
        P.bound[row] = fits ? bound : INFINITY;
        P.counts[row] = fits ? s_count : -1;
    }
}

// ------------------------------------------------------------ best of the candidates
struct BestParams {
    PickParams K;
    DotParams D;             // the REST products' (lists, counts, schedule)
    const uint2* list;       // the sample's
    const int* counts;
    int cap;
    int room;                // candidates a CTA holds
    IndexView V;             // for rows searched block by block
    const int8_t* codes;
};

constexpr int BEST_THREADS = 256;

__global__ void __launch_bounds__(BEST_THREADS) best_kernel(const BestParams P) {
    extern __shared__ unsigned long long s_key[];   // [room]
    __shared__ ScanShared S;
    __shared__ int s_total, s_bad, s_count;
    __shared__ unsigned long long s_prefix;
    __shared__ int s_ids[kMaxSelect];
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const RowRange R = row_range(P.K.pos0 + row, P.K.max_sel, P.K.n_first, P.K.n_last);
    int32_t* out = P.K.sel_idx + (long long)row * P.K.max_sel;
    if (write_plain(P.K, R, row, out)) return;
    if (tid == 0) {
        s_total = s_bad = 0;
        s_count = 0;
    }
    __syncthreads();
    if (R.need > 0) {
        // Runs of this row's row tile.
        const int rt = row / PAIR_ROWS;
        long long cum = 0;
        for (int t = 0; t < rt; ++t) cum += col_tiles<REST>(P.D, t);
        const int nt = col_tiles<REST>(P.D, rt);
        const int runs =
            nt ? pair_of(P.D, cum + nt - 1) - pair_of(P.D, cum) + 1 : 0;
        // A warp per list: the sample's, then two per run.
        for (int l = warp; l < 1 + 2 * runs; l += BEST_THREADS / 32) {
            const long long at = (long long)row * P.D.segs * 2 + (l - 1);
            const int n = l == 0 ? P.counts[row] : P.D.counts[at];
            const int cap = l == 0 ? P.cap : P.D.cap;
            if (n < 0 || n > cap) {
                s_bad = 1;
                continue;
            }
            const uint2* src = l == 0 ? P.list + (long long)row * P.cap : P.D.list + at * cap;
            int to = 0;
            if (lane == 0) to = atomicAdd(&s_total, n);
            to = __shfl_sync(0xffffffffu, to, 0);
            if (to + n > P.room) {
                s_bad = 1;
                continue;
            }
            for (int i = lane; i < n; i += 32) {
                const uint2 e = src[i];
                const uint32_t b = l == 0 ? (uint32_t)col_block<SAMPLE>((int)e.y)
                                          : (uint32_t)col_block<REST>((int)e.y);
                // Higher is better: the score's order, then the lower id.
                s_key[to + i] =
                    ((unsigned long long)ordered(__uint_as_float(e.x)) << 32) | (0xffffffffu - b);
            }
        }
    }
    __syncthreads();
    const int total = s_total;
    if (s_bad || total < R.need) {
        // Searched block by block; a row of zero codes needs no products.
        __syncthreads();
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
                int dot = 0;
                if (!zero) {
                    const uint4* k =
                        reinterpret_cast<const uint4*>(P.V.index + block * P.V.width);
                    for (int i = 0; i < P.V.width / 16; ++i) {
                        const uint4 x = q[i], y = k[i];
                        dot = __dp4a((int)x.x, (int)y.x, dot);
                        dot = __dp4a((int)x.y, (int)y.y, dot);
                        dot = __dp4a((int)x.z, (int)y.z, dot);
                        dot = __dp4a((int)x.w, (int)y.w, dot);
                    }
                }
                return __fmul_rn((float)dot, P.V.scale[block]);
            },
            out, S);
        return;
    }
    // The need-th best key, eight bits at a time, until the keys that share
    // the bits found are all taken.
    unsigned long long prefix = 0;
    int need = R.need;
    for (int shift = 56; need > 0; shift -= 8) {
        for (int i = tid; i < 256; i += BEST_THREADS) S.hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < total; i += BEST_THREADS) {
            const unsigned long long k = s_key[i];
            if (shift == 56 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
                atomicAdd(&S.hist[(int)(k >> shift) & 255], 1);
        }
        __syncthreads();
        if (warp == 0) {
            int left = need;
            const int d = pick_digit(S.hist, lane, &left);
            if (lane == 0) {
                // All of bin d taken: what is above or in it is the answer.
                S.need = S.hist[d] == left ? 0 : left;
                s_prefix = prefix | ((unsigned long long)d << shift);
            }
        }
        __syncthreads();
        prefix = s_prefix;
        need = S.need;
        __syncthreads();
    }
    for (int i = tid; i < total; i += BEST_THREADS) {
        const unsigned long long k = s_key[i];
        if (R.need > 0 && k >= prefix)
            s_ids[atomicAdd(&s_count, 1)] = (int)(0xffffffffu - (uint32_t)k);
    }
    __syncthreads();
    // The blocks that are always taken, and room for a power of two.
    for (int i = tid; i < R.lo; i += BEST_THREADS) s_ids[R.need + i] = i;
    for (int i = tid; i < R.n_vis - R.hi; i += BEST_THREADS) s_ids[R.need + R.lo + i] = R.hi + i;
    int pow2 = 1;
    while (pow2 < R.take) pow2 <<= 1;
    for (int i = R.take + tid; i < pow2; i += BEST_THREADS) s_ids[i] = 0x7fffffff;
    // Ids ascending: bitonic sort.
    for (int k = 2; k <= pow2; k <<= 1)
        for (int j = k >> 1; j > 0; j >>= 1) {
            __syncthreads();
            for (int i = tid; i < pow2 / 2; i += BEST_THREADS) {
                const int a = (i / j) * 2 * j + i % j, b = a + j;
                const int x = s_ids[a], y = s_ids[b];
                if ((x > y) == ((a & k) == 0)) {
                    s_ids[a] = y;
                    s_ids[b] = x;
                }
            }
        }
    __syncthreads();
    for (int i = tid; i < R.take; i += BEST_THREADS) out[i] = s_ids[i];
}

// ------------------------------------------------------------ host side
size_t round256(size_t n) { return (n + 255) / 256 * 256; }
int round_up(int n, int m) { return (n + m - 1) / m * m; }

// Calls of up to this many rows take the dp4a path.
constexpr int FEW_ROWS = 32;
// Below this many blocks, or this many per block taken, all scores are kept.
constexpr int SAMPLE_MIN_BLOCKS = 2048;
constexpr int SAMPLE_MIN_RATIO = 16;
constexpr size_t SCORE_BYTES = 128ull << 20;   // scores held at once
constexpr size_t LIST_BYTES = 256ull << 20;    // candidates held at once

// Where a call keeps what in the workspace.  Every area grows with the rows
// and the blocks, so the size for a context's last block holds for any n_last
// and max_sel.
struct Layout {
    long long stride;         // scores of a row
    int chunk;                // most rows of a launch, by the scores
    size_t codes, scores, codes16, cols, first_scale, rest_scale, bound, scounts, counts, list;
    size_t counts_bytes, list_bytes, bytes;
};

size_t list_row_bytes(int segs, int cap, int cap_sample) {
    return ((size_t)segs * 2 * cap + cap_sample) * 8;
}
int list_cap(int max_sel, long long tiles_per_pair) {
    const long long most = tiles_per_pair * (TILE / 2);
    return (int)(most < 4 * max_sel + 64 ? most : 4 * max_sel + 64);
}
int sample_cap(int max_sel, int n_sample) {
    return n_sample < 2 * max_sel + 64 ? n_sample : 2 * max_sel + 64;
}

// n: blocks scored; n_first: columns whose scores are kept (n, or the sample).
Layout layout(int rows, int n, int n_first, int width, int pairs) {
    Layout L = {};
    const bool few = rows <= FEW_ROWS;
    L.stride = round_up(n_first > 0 ? n_first : 1, TILE);
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
    L.chunk = rows;
    if (!few && scores / row_bytes < rows_up)
        L.chunk = (int)(scores / row_bytes / PAIR_ROWS) * PAIR_ROWS;
    L.codes = take((size_t)rows * width);
    L.scores = take(scores);
    if (!few) {
        L.codes16 = take((size_t)rows * width * 2);
        L.cols = take((size_t)n * width * 2);
        L.first_scale = take(row_bytes);
        L.rest_scale = take((size_t)round_up(n, TILE) * 4);
        L.bound = take(rows_up * 4);
        L.scounts = take(rows_up * 4);
        L.counts_bytes = ((size_t)PAIR_ROWS * pairs + 2 * rows_up) * 2 * 4;
        L.counts = take(L.counts_bytes);
        // One row tile fits with any max_sel.
        const long long tiles = (round_up(n, TILE) / TILE + pairs - 1) / pairs + 1;
        const size_t one = PAIR_ROWS * list_row_bytes(pairs, list_cap(kMaxSelect, tiles),
                                                      sample_cap(kMaxSelect, n_first));
        L.list_bytes = one > LIST_BYTES ? one : LIST_BYTES;
        L.list = take(L.list_bytes);
    }
    L.bytes = at;
    return L;
}

bool sampled(int n, int max_sel) {
    return n >= SAMPLE_MIN_BLOCKS && n / SAMPLE_MIN_RATIO >= max_sel;
}

// Pairs that can be resident at once (both SMs of a pair in one GPC).
int max_pairs(const DeviceInfo* di) {
    static std::atomic<int> cached[64];
    if (di->device < 64) {
        const int c = cached[di->device].load(std::memory_order_relaxed);
        if (c) return c;
    }
    if (ensure_smem_limit(reinterpret_cast<const void*>(dot_kernel<ALL, true>),
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
    if (cudaOccupancyMaxActiveClusters(&n, dot_kernel<ALL, true>, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        return 0;
    }
    if (n > di->num_sms / 2) n = di->num_sms / 2;
    if (di->device < 64) cached[di->device].store(n, std::memory_order_relaxed);
    return n;
}

// The schedule of a launch's products: pairs and, per row tile, the most runs.
template <int ORDER>
void schedule(DotParams& D, int pairs) {
    D.row_tiles = (D.rows + PAIR_ROWS - 1) / PAIR_ROWS;
    D.total = 0;
    for (int t = 0; t < D.row_tiles; ++t) D.total += col_tiles<ORDER>(D, t);
    D.G = (int)(D.total < pairs ? D.total : pairs);
    D.segs = 1;
    long long cum = 0;
    for (int t = 0; t < D.row_tiles && D.total > 0; ++t) {
        const int n = col_tiles<ORDER>(D, t);
        if (n > 0) {
            const int s = pair_of(D, cum + n - 1) - pair_of(D, cum) + 1;
            if (s > D.segs) D.segs = s;
        }
        cum += n;
    }
}

template <int ORDER>
int launch_dots(const __half* rows16, const __half* cols, int n_cols, const DotParams& D,
                cudaStream_t stream) {
    if (D.total == 0) return GQA_OK;
    const int width = D.chunks * 64;
    CUtensorMap tr, tc;
    if (!make_map_2d_f16(&tr, rows16, D.rows, width, width, CTA_ROWS, 64) ||
        !make_map_2d_f16(&tc, cols, n_cols, width, width, CTA_ROWS, 64))
        return GQA_ERR_CUDA;
    const bool resident = D.chunks <= RES_CHUNKS;
    const int smem = resident ? DotCfg<true>::SMEM : DotCfg<false>::SMEM;
    auto* kernel = resident ? dot_kernel<ORDER, true> : dot_kernel<ORDER, false>;
    if (ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem) != GQA_OK)
        return GQA_ERR_CUDA;
    kernel<<<2 * D.G, DOT_THREADS, smem, stream>>>(tr, tc, D);
    return GQA_OK;
}

constexpr int BEST_SMEM = 200 << 10;

}  // namespace select

size_t select_blocks_workspace_bytes(int rows, int ctx_len, int width) {
    using namespace select;
    const DeviceInfo* di = device_info();
    const int pairs = di ? max_pairs(di) : 0;
    if (pairs < 1) return 0;
    const int n = (ctx_len - 1) / 4 + 1;
    const size_t all = layout(rows, n, n, width, pairs).bytes;
    const size_t some = layout(rows, n, cols_below<SAMPLE>(n), width, pairs).bytes;
    return all > some ? all : some;
}

int select_blocks_launch(const void* q, const int8_t* index, const float* index_scale,
                         const int32_t* block_table, int num_pages, int page, int ctx_len,
                         int rows, int Hq, int Hkv, int D, int max_sel, int n_first, int n_last,
                         int32_t* sel_idx, int32_t* sel_cnt, cudaStream_t stream) {
    using namespace select;
    const DeviceInfo* di = device_info();
    if (!di) return GQA_ERR_CUDA;
    const int width = Hkv * D;
    const bool few = rows <= FEW_ROWS;
    // Blocks below the last row's always-taken ones.
    int n = ((ctx_len - 1) >> 2) + 1 - n_last;
    if (n <= n_first) n = 0;   // nothing to score
    const bool sample = !few && sampled(n, max_sel);
    const int n_kept = sample ? cols_below<SAMPLE>(n) : n;
    const int pairs = max_pairs(di);
    if (pairs < 1) return GQA_ERR_CUDA;
    const Layout L = layout(rows, n, n_kept, width, pairs);
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
    const int code_ctas = (rows + 7) / 8;
    const int pos0 = ctx_len - rows;
    PickParams K = {pos0, max_sel, n_first, n_last, sel_idx, sel_cnt};
    if (few) {
        if (n > 0) {
            prepare_kernel<<<code_ctas, 256, 0, stream>>>(C, ExpandParams{}, code_ctas);
            const SmallParams S = {V, codes, rows, n, scores, L.stride};
            const int tiles = (n + 31) / 32, cap = di->num_sms * 8;
            const dim3 grid(tiles < cap ? tiles : cap, (rows + SMALL_ROWS - 1) / SMALL_ROWS);
            score_small_kernel<<<grid, 256, 0, stream>>>(S);
        }
        pick_kernel<1024><<<rows, 1024, 0, stream>>>(K, scores, L.stride);
        return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
    }
    __half* codes16 = reinterpret_cast<__half*>(w + L.codes16);
    __half* first = reinterpret_cast<__half*>(w + L.cols);
    float* first_scale = reinterpret_cast<float*>(w + L.first_scale);
    float* rest_scale = reinterpret_cast<float*>(w + L.rest_scale);
    C.codes16 = codes16;
    const ExpandParams E = {V, n_kept, n - n_kept, sample, first, first + (size_t)n_kept * width,
                            first_scale, rest_scale};
    if (n > 0) {
        const long long threads = (long long)n * (width / 16);
        const long long ctas = code_ctas + (threads + 255) / 256;
        prepare_kernel<<<(unsigned)ctas, 256, 0, stream>>>(C, E, code_ctas);
    }
    if (sample && ensure_smem_limit(reinterpret_cast<const void*>(best_kernel), BEST_SMEM) != GQA_OK)
        return GQA_ERR_CUDA;
    int step = L.chunk;
    for (int r0 = 0; r0 < rows; r0 += step) {
        DotParams P = {};
        P.chunks = width / 64;
        P.pos0 = pos0 + r0;
        P.max_sel = max_sel;
        P.n_first = n_first;
        P.n_last = n_last;
        P.scale = first_scale;
        P.scores = scores;
        P.stride = L.stride;
        P.err = di->err_word;
        DotParams R = P;     // the REST products
        const int cap_sample = sample_cap(max_sel, n_kept);
        // Fewer rows a launch if their candidate lists would not fit.
        for (;;) {
            P.rows = R.rows = rows - r0 < step ? rows - r0 : step;
            if (!sample) break;
            schedule<REST>(R, pairs);
            R.cap = R.G > 0 ? list_cap(max_sel, (R.total + R.G - 1) / R.G) : 1;
            if (R.rows * list_row_bytes(R.segs, R.cap, cap_sample) <= L.list_bytes &&
                (size_t)R.rows * R.segs * 2 * 4 <= L.counts_bytes)
                break;
            if (step <= PAIR_ROWS) return GQA_ERR_WORKSPACE;   // does not happen: see layout()
            step = round_up(R.rows, PAIR_ROWS) - PAIR_ROWS;
        }
        K.pos0 = pos0 + r0;
        K.sel_idx = sel_idx + (size_t)r0 * max_sel;
        K.sel_cnt = sel_cnt + r0;
        const __half* rows16 = codes16 + (size_t)r0 * width;
        int rc;
        if (!sample) {
            schedule<ALL>(P, pairs);
            if (n == 0) P.total = 0;
            rc = launch_dots<ALL>(rows16, first, n_kept, P, stream);
            if (rc != GQA_OK) return rc;
            pick_kernel<256><<<P.rows, 256, 0, stream>>>(K, scores, L.stride);
            continue;
        }
        schedule<SAMPLE>(P, pairs);
        rc = launch_dots<SAMPLE>(rows16, first, n_kept, P, stream);
        if (rc != GQA_OK) return rc;
        float* bound = reinterpret_cast<float*>(w + L.bound);
        int* scounts = reinterpret_cast<int*>(w + L.scounts);
        uint2* slist = reinterpret_cast<uint2*>(w + L.list);
        const BoundParams B = {scores, L.stride, K.pos0, max_sel, n_first, n_last,
                               bound, slist, scounts, cap_sample};
        bound_kernel<<<P.rows, 256, 0, stream>>>(B);
        R.scale = rest_scale;
        R.scores = nullptr;
        R.bound = bound;
        R.list = slist + (size_t)R.rows * cap_sample;
        R.counts = reinterpret_cast<int*>(w + L.counts);
        rc = launch_dots<REST>(rows16, E.rest, E.n_rest_cols, R, stream);
        if (rc != GQA_OK) return rc;
        BestParams T = {};
        T.K = K;
        T.D = R;
        T.list = slist;
        T.counts = scounts;
        T.cap = cap_sample;
        T.room = 12 * max_sel + 1024;
        if (T.room > BEST_SMEM / 8) T.room = BEST_SMEM / 8;
        T.V = V;
        T.codes = codes + (size_t)r0 * width;
        best_kernel<<<R.rows, BEST_THREADS, (size_t)T.room * 8, stream>>>(T);
    }
    return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace gqa

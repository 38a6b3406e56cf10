// paged_fp4.cu -- causal GQA tails over a 4-bit paged cache (rows as in
// fp4_rows.cuh), for a batch of sequences, with a sliding window and first tokens
// that stay visible ("sinks").
//
//   out = softmax_j(scale * q . k_j) v_j over the keys j of the sequence with
//   j <= p and (no window, or j > p - window, or j < sinks), p the row's position.
//
// One pass over the visible tiles of 128 keys, with a running maximum and sum.
//
// * Work split.  The visible tiles of all (sequence, KV head, group of up to
//   8 NT packed rows) units, one behind the other, are cut into one equal
//   contiguous range per CTA, from the context lengths on the device.  A unit that
//   lies in one range is finished there; a unit that is cut leaves (O, m, l)
//   partials, at most two for a CTA, which a second kernel joins in range order.
// * Copies.  One warp brings the pages of a tile (a page of one head is one
//   contiguous run) into a ring of stages by bulk copies, table entries two tiles
//   ahead.
// * Products.  Eight warps take 16 keys of a tile each and never meet before the
//   end of a piece.  A warp decodes its codes from shared memory straight into the
//   fragments of m16n8k16 products, keys (for K) or values' places (for V) along M,
//   packed query rows along N, so eight rows waste nothing: the order of the places
//   within a product is free, so a lane loads whole words of one key, K's pairs are
//   a byte's two nibbles and V's pairs come from two keys' nibbles put together.
//   With the operands in registers nothing decoded goes through shared memory,
//   which an operand of tcgen05.mma would have to (4 times the codes' bytes, written
//   and read).
// * Softmax.  A row's reference moves only when a score passes it by more than 8
//   (log2 units), so P <= 256 in fp16; each warp keeps its own references.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <type_traits>

#include "fp4_rows.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace gqa {
namespace paged4 {

constexpr int TILE = 128;                  // keys of a tile
constexpr int NW = 8;                      // warps with products, 16 keys of a tile each
// And a warpgroup of which one warp copies: at three warps for each quarter of an SM a
// kernel starts with 168 registers a thread, of which the products take 240 and the
// copies leave all but 24 (256 * 240 + 128 * 24 = 384 * 168).
constexpr int THREADS = 32 * NW + 128;
constexpr int REGS_PRODUCTS = 240, REGS_COPIES = 24;
constexpr int STAGES = 5;
constexpr int JOIN_BYTES = 16384;          // the warps' O on their way to one sum
constexpr int MAX_BATCH = 1024;
constexpr float RESCALE_THRESHOLD = 8.0f;

struct Params {
    const __half* q;
    const uint8_t* cache[2];     // K, V
    const float* scale_dev[2];   // their fp32 scales
    const int32_t* tables;
    const int* ctx_lens;
    int table_stride, num_pages, page, log2_page, max_ctx, batch;
    int R, hq, hkv;
    FastDiv grp;                 // query heads of one KV head
    int nq;                      // packed rows of one KV head (R * grp)
    int groups;                  // groups of 8 NT packed rows
    int window, sinks;           // window 0: none
    float scale;
    int G;                       // ranges (CTAs)
    float* ws_o;                 // [G][2][8 NT][DH]
    float* ws_ml;                // [G][2][8 NT][2]
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
    s.first_tile = s.lo / TILE;
    s.sink_tiles = (min(P.sinks, s.first_tile * TILE) + TILE - 1) / TILE;
    s.tiles = s.ctx > 0 ? s.sink_tiles + (s.ctx + TILE - 1) / TILE - s.first_tile : 0;
    return s;
}

// starts[b] = tiles of the sequences before b, for b = 0 .. batch.  All `N` threads
// of the CTA (at least 256), with two barriers.
template <int N>
__device__ void tile_starts(const Params& P, long long* starts, long long* totals) {
    constexpr int EACH = MAX_BATCH / 256;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int n[EACH];
    long long sum = 0, incl = 0;
    if (tid < 256) {
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int b = tid * EACH + i;
            n[i] = b < P.batch ? span_of(P, P.ctx_lens[b]).tiles : 0;
            sum += n[i];
        }
        incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        if (lane == 31) totals[warp] = incl;
    }
    __syncthreads();
    if (tid < 256) {
        long long at = incl - sum;
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

// Range c of G equal ones over `total` tiles, and the range a tile lies in.
__device__ __forceinline__ long long range_begin(long long total, int G, int c) {
    return (long long)c * total / G;
}
__device__ __forceinline__ int range_of(long long total, int G, long long pos) {
    return (int)(((pos + 1) * G - 1) / total);
}

// The sequence whose tiles hold position pos (units of a sequence are one behind
// the other, `per` of them).
__device__ __forceinline__ int sequence_of(const Params& P, const long long* starts, int per,
                                           long long pos) {
    int lo = 0, hi = P.batch;   // starts[lo] * per <= pos < starts[hi] * per
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] * per <= pos) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Walks the pieces (unit, tiles [jb, je)) of one range.
struct Pieces {
    long long pos, end;
    bool first;
    int b, h, g;      // sequence, KV head, group of packed rows
    int jb, je;
    bool whole;
    Span s;
    __device__ void init(long long begin, long long end_) {
        pos = begin;
        end = end_;
    }
    __device__ bool next(const Params& P, const long long* starts, long long begin) {
        if (pos >= end) return false;
        const int per = P.hkv * P.groups;
        first = pos == begin;
        b = sequence_of(P, starts, per, pos);
        s = span_of(P, P.ctx_lens[b]);
        // (at most 2^24 tiles of 192 units)
        const uint32_t off = (uint32_t)(pos - starts[b] * per);
        const uint32_t n = (uint32_t)(starts[b + 1] - starts[b]);
        const int u = (int)(off / n);
        jb = (int)(off - (uint32_t)u * n);
        const long long left = end - pos;
        je = (long long)jb + left < (long long)n ? jb + (int)left : (int)n;
        whole = jb == 0 && je == (int)n;
        h = u / P.groups;
        g = u - h * P.groups;
        pos += je - jb;
        return true;
    }
};

__device__ __forceinline__ int tile_key(const Span& s, int j) {
    return (j < s.sink_tiles ? j : s.first_tile + j - s.sink_tiles) * TILE;
}

// Element offset of packed row r of a KV head in q / out.
__device__ __forceinline__ long long row_offset(const Params& P, int b, int h, int r, int dh) {
    const int pos = P.grp.div(r);
    return (((long long)b * P.R + pos) * P.hq + h * P.grp.d + (r - pos * P.grp.d)) * dh;
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

template <int DH, int NT>
struct Layout {
    static constexpr int ROWB = fp4::row_bytes(DH);
    static constexpr int STAGE = 2 * TILE * ROWB;
    static constexpr int ROWS = 8 * NT;
    // Query rows in shared memory (NT > 1): a lane's quarter of a row padded by 16
    // bytes, so that the eight lanes of a load's phase use different banks.
    static constexpr int QUARTER = DH / 4 * 2 + 16;
    static constexpr int OFF_RING = 0;
    static constexpr int OFF_JOIN = OFF_RING + STAGES * STAGE;
    static constexpr int OFF_Q = OFF_JOIN + JOIN_BYTES;
    static constexpr int OFF_ML = OFF_Q + (NT > 1 ? ROWS * 4 * QUARTER : 0);
    static constexpr int OFF_STARTS = OFF_ML + NW * ROWS * 8;
    static constexpr int OFF_TOTALS = OFF_STARTS + (MAX_BATCH + 1) * 8;
    static constexpr int OFF_BARS = OFF_TOTALS + 8 * 8;
    static constexpr int OFF_ABORT = OFF_BARS + (2 * STAGES + 1) * 8;
    static constexpr int BYTES = OFF_ABORT + 16;
    static_assert(BYTES <= 232448, "shared memory");
};

template <int DH, int NT>
__global__ void __launch_bounds__(THREADS, 1) split_kernel(const Params P) {
    using L = Layout<DH, NT>;
    constexpr int ROWB = L::ROWB;
    constexpr int ROWS = L::ROWS;
    constexpr int MT = DH / 16;         // products along D
    extern __shared__ __align__(128) uint8_t smem[];
    float* join = reinterpret_cast<float*>(smem + L::OFF_JOIN);
    uint8_t* sq = smem + L::OFF_Q;
    float* sml = reinterpret_cast<float*>(smem + L::OFF_ML);   // [NW][ROWS][2]
    long long* starts = reinterpret_cast<long long*>(smem + L::OFF_STARTS);
    long long* totals = reinterpret_cast<long long*>(smem + L::OFF_TOTALS);
    const uint32_t bars = smem_u32(smem + L::OFF_BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_ABORT);
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (STAGES + s); };
    const uint32_t meet_bar = bars + 8u * (2 * STAGES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), NW);
        }
        mbar_init(meet_bar, NW);
        *abort_flag = 0;
        fence_mbar_init();
    }
    // Nothing of global memory is read or written before the kernel in front has
    // completed; this kernel's launch overlaps it.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    tile_starts<THREADS>(P, starts, totals);
    asm volatile("griddepcontrol.launch_dependents;");
    const long long total = starts[P.batch] * (P.hkv * P.groups);
    const int G = (int)min((long long)P.G, total);
    const int cta = blockIdx.x;
    // Sequences without a key: their rows are zeros.
    for (int b = cta; b < P.batch; b += gridDim.x) {
        const int raw = P.ctx_lens[b];
        if ((raw < 0 || raw > P.max_ctx) && threadIdx.x == 0) atomicOr(P.err, kErrBadCtxLen);
        if (raw <= 0) {
            uint4* o = reinterpret_cast<uint4*>(P.out + (long long)b * P.R * P.hq * DH);
            for (int i = threadIdx.x; i < P.R * P.hq * DH / 8; i += THREADS)
                o[i] = make_uint4(0, 0, 0, 0);
        }
    }
    const bool works = cta < G;
    const long long begin = works ? range_begin(total, G, cta) : 0;
    const long long end = works ? range_begin(total, G, cta + 1) : 0;
    Pieces it;
    it.init(begin, end);

    if (warp >= NW) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_COPIES));
      if (warp == NW) {
        // ------------------------------------------------------------ copies
        // Lanes 0 .. 15 copy K's pages of a tile, 16 .. 31 V's.
        const int kv = lane >> 4, p = lane & 15;
        const int rows = min(P.page, TILE), ppt = TILE / rows;   // rows of a copy, copies of a tile
        uint32_t n = 0;   // tiles so far
        bool ok = true;
        while (ok && it.next(P, starts, begin)) {
            const int pages = (it.s.ctx + P.page - 1) >> P.log2_page;
            const int32_t* table = P.tables + (long long)it.b * P.table_stride;
            auto entry = [&](int j) {
                if (j >= it.je) return 0;
                const int lp = (tile_key(it.s, j) >> P.log2_page) + p;
                return p < ppt && lp < pages ? __ldg(table + lp) : 0;
            };
            int id = entry(it.jb), id1 = entry(it.jb + 1);
            for (int j = it.jb; j < it.je; ++j) {
                const int id2 = entry(j + 2);
                const int key0 = tile_key(it.s, j);
                const int copies = min(ppt, pages - (key0 >> P.log2_page));
                if (p < copies && (id < 0 || id >= P.num_pages)) {
                    atomicOr(P.err, kErrBadPageId);
                    id = 0;
                }
                const int st = n % STAGES;
                int okw = 1;
                if (lane == 0) {
                    okw = mbar_wait(empty(st), ((n / STAGES) & 1) ^ 1, abort_flag, P.err);
                    if (okw) mbar_arrive_expect_tx(full(st), 2 * copies * rows * ROWB);
                }
                ok = __shfl_sync(0xffffffffu, okw, 0);
                if (!ok) break;
                if (p < copies) {
                    const long long row = ((long long)id * P.hkv + it.h) * P.page +
                                          (key0 & (P.page - 1));
                    bulk_load(smem_u32(smem) + L::OFF_RING + st * L::STAGE + kv * (TILE * ROWB) +
                                  p * rows * ROWB,
                              P.cache[kv] + row * ROWB, rows * ROWB, full(st));
                }
                ++n;
                id = id1;
                id1 = id2;
            }
        }
        if (!ok && lane == 0) {
            // Unwind: every copy in flight lands before the CTA exits.
            for (int s = 0; s < STAGES; ++s) {
                const uint32_t fills = n > (uint32_t)s ? (n - s + STAGES - 1) / STAGES : 0;
                if (!fills) continue;
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(full(s), (fills - 1) & 1))
                    if (global_timer_ns() - t0 > 100000000ull) break;
            }
        }
      }
    } else {
        // ------------------------------------------------------------ products
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_PRODUCTS));
        const int gid = lane >> 2, t = lane & 3;
        uint32_t meet_phase = 0;
        // All warps with products: a barrier that shares the bounded wait.
        auto meet = [&]() -> bool {
            __syncwarp();
            if (lane == 0) mbar_arrive(meet_bar);
            const bool ok = mbar_wait(meet_bar, meet_phase, abort_flag, P.err);
            meet_phase ^= 1;
            return __all_sync(0xffffffffu, ok);
        };
        const float sl2 = P.scale * *P.scale_dev[0] * 1.4426950408889634f;
        const float vscale = *P.scale_dev[1];
        uint32_t n = 0;
        bool ok = true;
        while (ok && it.next(P, starts, begin)) {
            const Span s = it.s;
            const int row0 = it.g * ROWS;
            // Q: the lane's quarter of row gid of each eight (products' B operand).
            uint32_t qf[NT == 1 ? MT : 1][2];
            if constexpr (NT == 1) {
                const bool there = row0 + gid < P.nq;
                const uint4* src = reinterpret_cast<const uint4*>(
                    P.q + (there ? row_offset(P, it.b, it.h, row0 + gid, DH) : 0) + t * (DH / 4));
#pragma unroll
                for (int i = 0; i < MT / 2; ++i) {
                    const uint4 v = there ? src[i] : make_uint4(0, 0, 0, 0);
                    qf[2 * i][0] = v.x;
                    qf[2 * i][1] = v.y;
                    qf[2 * i + 1][0] = v.z;
                    qf[2 * i + 1][1] = v.w;
                }
            } else {
                for (int i = threadIdx.x; i < ROWS * DH / 8; i += 32 * NW) {
                    const int r = i / (DH / 8), c = i % (DH / 8);
                    const uint4 v = row0 + r < P.nq
                                        ? *reinterpret_cast<const uint4*>(
                                              P.q + row_offset(P, it.b, it.h, row0 + r, DH) + c * 8)
                                        : make_uint4(0, 0, 0, 0);
                    const int quarter = c / (DH / 32);
                    *reinterpret_cast<uint4*>(sq + (r * 4 + quarter) * L::QUARTER +
                                              (c % (DH / 32)) * 16) = v;
                }
                ok = meet();
                if (!ok) break;
            }
            // Positions of the lane's packed rows 2 t, 2 t + 1 of each eight.
            int pos[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    pos[nt][e] = s.ctx - P.R +
                                 min(P.grp.div(row0 + nt * 8 + 2 * t + e), P.R - 1);
            float o[MT][NT][4];
            float mref[NT][2], l[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mref[nt][0] = mref[nt][1] = -INFINITY;
                l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[m][nt][e] = 0.f;
            }

            for (int j = it.jb; j < it.je; ++j) {
                const int st = n % STAGES;
                ok = mbar_wait(full(st), (n / STAGES) & 1, abort_flag, P.err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ++n;
                const int k0 = tile_key(s, j) + warp * 16;
                const int last = s.ctx - 1;
                const bool skip = k0 > last || (k0 + 15 < s.lo && k0 >= P.sinks);
                if (!skip) {
                    const uint8_t* kst = smem + L::OFF_RING + st * L::STAGE + warp * 16 * ROWB;
                    const uint8_t* vst = kst + TILE * ROWB;
                    // Some key of the 16 is hidden from some row.
                    const bool edge = k0 + 15 > s.ctx - P.R ||
                                      (P.window > 0 && k0 <= last - P.window && k0 + 15 >= P.sinks);
                    // ---- scores of keys gid and gid + 8
                    float sc[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[nt][e] = 0.f;
                    {
                        constexpr int KW = DH / 32;   // words of a lane and key
                        uint32_t w[2][KW], u[2][DH / 64];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint8_t* row = kst + (gid + 8 * e) * ROWB;
                            if constexpr (DH == 256) {
                                const uint4* src = reinterpret_cast<const uint4*>(row + t * 32);
                                const uint4 x = src[0], y = src[1];
                                w[e][0] = x.x, w[e][1] = x.y, w[e][2] = x.z, w[e][3] = x.w;
                                w[e][4] = y.x, w[e][5] = y.y, w[e][6] = y.z, w[e][7] = y.w;
                                const uint32_t c =
                                    *reinterpret_cast<const uint32_t*>(row + DH / 2 + t * 4);
                                const uint32_t c01 = fp4::scales2(c), c23 = fp4::scales2(c >> 16);
                                u[e][0] = __byte_perm(c01, 0, 0x1010);
                                u[e][1] = __byte_perm(c01, 0, 0x3232);
                                u[e][2] = __byte_perm(c23, 0, 0x1010);
                                u[e][3] = __byte_perm(c23, 0, 0x3232);
                            } else {
                                const uint2* src = reinterpret_cast<const uint2*>(row + t * 16);
                                const uint2 x = src[0], y = src[1];
                                w[e][0] = x.x, w[e][1] = x.y, w[e][2] = y.x, w[e][3] = y.y;
                                const uint32_t c = fp4::scales2(
                                    *reinterpret_cast<const uint16_t*>(row + DH / 2 + t * 2));
                                u[e][0] = __byte_perm(c, 0, 0x1010);
                                u[e][1] = __byte_perm(c, 0, 0x3232);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < KW; ++i) {
                            uint32_t a[4], b[4];
                            fp4::decode8(w[0][i], a);
                            fp4::decode8(w[1][i], b);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                a[e] = fp4::mul2(a[e], u[0][i / 2]);
                                b[e] = fp4::mul2(b[e], u[1][i / 2]);
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                uint4 qv;
                                if constexpr (NT == 1)
                                    qv = make_uint4(qf[2 * i][0], qf[2 * i][1], qf[2 * i + 1][0],
                                                    qf[2 * i + 1][1]);
                                else
                                    qv = *reinterpret_cast<const uint4*>(
                                        sq + ((nt * 8 + gid) * 4 + t) * L::QUARTER + i * 16);
                                mma16816(sc[nt], a[0], b[0], a[1], b[1], qv.x, qv.y);
                                mma16816(sc[nt], a[2], b[2], a[3], b[3], qv.z, qv.w);
                            }
                        }
                    }
                    bool exceed = false;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            sc[nt][e] *= sl2;
                            if (edge) {
                                const int key = k0 + gid + (e & 2) * 4, at = pos[nt][e & 1];
                                const bool seen =
                                    key <= at && (P.window == 0 || key > at - P.window ||
                                                  key < P.sinks);
                                if (!seen) sc[nt][e] = -INFINITY;
                            }
                            exceed |= sc[nt][e] > mref[nt][e & 1] + RESCALE_THRESHOLD;
                        }
                    if (__any_sync(0xffffffffu, exceed)) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float f[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float m = fmaxf(sc[nt][e], sc[nt][e + 2]);
#pragma unroll
                                for (int x = 4; x < 32; x <<= 1)
                                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
                                f[e] = 1.f;
                                if (m > mref[nt][e] + RESCALE_THRESHOLD) {
                                    f[e] = ex2(mref[nt][e] - m);
                                    mref[nt][e] = m;
                                }
                                l[nt][e] *= f[e];
                            }
#pragma unroll
                            for (int m = 0; m < MT; ++m) {
                                o[m][nt][0] *= f[0];
                                o[m][nt][1] *= f[1];
                                o[m][nt][2] *= f[0];
                                o[m][nt][3] *= f[1];
                            }
                        }
                    }
                    // ---- P, transposed into the second product's B operand: keys
                    // 2 t, 2 t + 1 (and 8 more) of packed row gid.
                    uint32_t pf[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float m0 = mref[nt][0] == -INFINITY ? 0.f : mref[nt][0];
                        const float m1 = mref[nt][1] == -INFINITY ? 0.f : mref[nt][1];
                        const float p0 = ex2(sc[nt][0] - m0), p1 = ex2(sc[nt][1] - m1);
                        const float p2 = ex2(sc[nt][2] - m0), p3 = ex2(sc[nt][3] - m1);
                        l[nt][0] += p0 + p2;
                        l[nt][1] += p1 + p3;
                        pf[nt][0] = transpose8(pack_half2(p0, p1));
                        pf[nt][1] = transpose8(pack_half2(p2, p3));
                    }
                    // ---- O += V^T P^T over keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
                    constexpr int VW = DH / 64;   // words of a lane and key
                    uint32_t w[4][VW];
                    uint32_t c[4];                // their scales, one byte each 16 values
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint8_t* row = vst + (2 * t + (e & 1) + (e >> 1) * 8) * ROWB;
                        if constexpr (DH == 256) {
                            const uint4 x = *reinterpret_cast<const uint4*>(row + gid * 16);
                            w[e][0] = x.x, w[e][1] = x.y, w[e][2] = x.z, w[e][3] = x.w;
                            c[e] = *reinterpret_cast<const uint16_t*>(row + DH / 2 + gid * 2);
                        } else {
                            const uint2 x = *reinterpret_cast<const uint2*>(row + gid * 8);
                            w[e][0] = x.x, w[e][1] = x.y;
                            c[e] = row[DH / 2 + gid];
                        }
                    }
                    // One pass over the values for all rows (pass < 0), or for the rows of
                    // one position alone: the others' sums stay as they are.
                    auto values = [&](auto one, int pass) {
                        constexpr bool ONE = decltype(one)::value;
                        uint32_t cc[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            cc[e] = c[e];
                            if constexpr (ONE) {
                                const int key = k0 + 2 * t + (e & 1) + (e >> 1) * 8;
                                const int at = s.ctx - P.R + pass;
                                if (key > at || (P.window > 0 && key <= at - P.window &&
                                                 key >= P.sinks))
                                    cc[e] = 0;
                            }
                        }
#pragma unroll
                        for (int i = 0; i < VW; ++i) {
                            // (words 2 k and 2 k + 1 share a scale)
                            const int sh = DH == 256 ? (i / 2) * 8 : 0;
                            const uint32_t u01 = fp4::scales2(((cc[0] >> sh) & 0xff) |
                                                              ((cc[1] >> sh) & 0xff) << 8);
                            const uint32_t u23 = fp4::scales2(((cc[2] >> sh) & 0xff) |
                                                              ((cc[3] >> sh) & 0xff) << 8);
                            uint32_t lo0[4], hi0[4], lo1[4], hi1[4];
                            fp4::decode8(low_nibbles(w[0][i], w[1][i]), lo0);
                            fp4::decode8(high_nibbles(w[0][i], w[1][i]), hi0);
                            fp4::decode8(low_nibbles(w[2][i], w[3][i]), lo1);
                            fp4::decode8(high_nibbles(w[2][i], w[3][i]), hi1);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t a0 = fp4::mul2(lo0[e], u01);
                                const uint32_t a1 = fp4::mul2(hi0[e], u01);
                                const uint32_t a2 = fp4::mul2(lo1[e], u23);
                                const uint32_t a3 = fp4::mul2(hi1[e], u23);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    float(&to)[4] = o[4 * i + e][nt];
                                    const float kept[4] = {to[0], to[1], to[2], to[3]};
                                    mma16816(to, a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
                                    if constexpr (ONE) {
#pragma unroll
                                        for (int x = 0; x < 4; ++x)
                                            if (pos[nt][x & 1] != s.ctx - P.R + pass)
                                                to[x] = kept[x];
                                    }
                                }
                            }
                        }
                    };
                    // Keys no row sees may hold anything: scales of zero.  A key that
                    // some rows see and others do not must not reach those others even
                    // if it is NaN (0 * NaN): the rows of one position at a time then.
                    bool apart = false;
                    if (edge) {
                        bool bad = false;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = k0 + 2 * t + (e & 1) + (e >> 1) * 8;
                            if (key > last || (key < s.lo && key >= P.sinks)) c[e] = 0;
                            bad |= (c[e] & 0x7f) == 0x7f || (c[e] & 0x7f00) == 0x7f00;
                        }
                        apart = P.R > 1 && __any_sync(0xffffffffu, bad);
                    }
                    if (!apart) {
                        values(std::false_type{}, -1);
                    } else {
                        for (int pass = 0; pass < P.R; ++pass) values(std::true_type{}, pass);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty(st));
            }
            if (!ok) break;

            // ---------------------------------------------------------- end of the piece
            // The warps' references and sums, then their O in a fixed order: warp x
            // gathers the products [x MT / NW, (x + 1) MT / NW) of all.
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1)
                        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], x);
                    if (gid == 0) {
                        float* to = sml + (warp * ROWS + nt * 8 + 2 * t + e) * 2;
                        to[0] = mref[nt][e];
                        to[1] = l[nt][e];
                    }
                }
            ok = meet();
            if (!ok) break;
            float M[NT][2], sum[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float* from = sml + (nt * 8 + 2 * t + e) * 2;
                    float m = -INFINITY;
#pragma unroll
                    for (int x = 0; x < NW; ++x) m = fmaxf(m, from[x * ROWS * 2]);
                    float a = 0.f;
#pragma unroll
                    for (int x = 0; x < NW; ++x) {
                        const float mx = from[x * ROWS * 2];
                        a += (mx == -INFINITY ? 0.f : ex2(mx - m)) * from[x * ROWS * 2 + 1];
                    }
                    M[nt][e] = m;
                    sum[nt][e] = a;
                    const float f = mref[nt][e] == -INFINITY ? 0.f : ex2(mref[nt][e] - m);
#pragma unroll
                    for (int k = 0; k < MT; ++k) {
                        o[k][nt][e] *= f;
                        o[k][nt][e + 2] *= f;
                    }
                }
            constexpr int MINE = MT / NW;                          // products of a target
            constexpr int PIECE = MINE * NT * 128;                 // floats of one source
            constexpr int TARGETS = JOIN_BYTES / (NW * PIECE * 4); // of one round
            static_assert(TARGETS >= 1 && NW % TARGETS == 0, "rounds");
            float acc[MINE][NT][4];
#pragma unroll
            for (int r = 0; r < NW / TARGETS; ++r) {
                if (r) {
                    ok = meet();
                    if (!ok) break;
                }
#pragma unroll
                for (int x = 0; x < TARGETS; ++x)
#pragma unroll
                    for (int k = 0; k < MINE; ++k)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const float(&v)[4] = o[(r * TARGETS + x) * MINE + k][nt];
                            *reinterpret_cast<float4*>(join + (x * NW + warp) * PIECE +
                                                       ((k * NT + nt) * 32 + lane) * 4) =
                                make_float4(v[0], v[1], v[2], v[3]);
                        }
                ok = meet();
                if (!ok) break;
                if (warp / TARGETS == r) {
#pragma unroll
                    for (int k = 0; k < MINE; ++k)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                            for (int x = 0; x < NW; ++x) {
                                const float4 v = *reinterpret_cast<const float4*>(
                                    join + ((warp % TARGETS) * NW + x) * PIECE +
                                    ((k * NT + nt) * 32 + lane) * 4);
                                a.x += v.x;
                                a.y += v.y;
                                a.z += v.z;
                                a.w += v.w;
                            }
                            acc[k][nt][0] = a.x;
                            acc[k][nt][1] = a.y;
                            acc[k][nt][2] = a.z;
                            acc[k][nt][3] = a.w;
                        }
                }
            }
            if (!ok) break;
            const int slot = cta * 2 + (it.first ? 0 : 1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = nt * 8 + 2 * t + e;
                    if (row0 + r >= P.nq) continue;
                    const float inv = sum[nt][e] > 0.f ? vscale / sum[nt][e]
                                      : isnan(sum[nt][e]) ? NAN : 0.f;
#pragma unroll
                    for (int k = 0; k < MINE; ++k) {
                        // Product i * 4 + x is the places 8 i + 2 x, 8 i + 2 x + 1 of
                        // every gid's DH / 8.
                        const int m = warp * MINE + k;
                        const int d = gid * (DH / 8) + (m / 4) * 8 + (m % 4) * 2;
                        if (it.whole)
                            *reinterpret_cast<uint32_t*>(
                                P.out + row_offset(P, it.b, it.h, row0 + r, DH) + d) =
                                pack_half2(acc[k][nt][e] * inv, acc[k][nt][e + 2] * inv);
                        else
                            *reinterpret_cast<float2*>(P.ws_o + ((long long)slot * ROWS + r) * DH +
                                                       d) =
                                make_float2(acc[k][nt][e], acc[k][nt][e + 2]);
                    }
                    if (!it.whole && warp == 0 && gid == 0)
                        *reinterpret_cast<float2*>(P.ws_ml + ((long long)slot * ROWS + r) * 2) =
                            make_float2(M[nt][e], sum[nt][e]);
                }
            // (sml and join are written again only behind the next piece's barriers:
            // sml by warps that may be ahead of this piece's last readers)
            ok = meet();
        }
    }
    __syncthreads();
}

// Joins the partials of the units that lie in several ranges: a block for a
// packed row of a unit, found by its number (by_unit) or by the first range that
// begins inside it.  Pieces are added in range order within each of the block's
// lanes of pieces, which are then added in order.
constexpr int MERGE_THREADS = 512;

template <int DH, int NT>
__global__ void __launch_bounds__(MERGE_THREADS) merge_kernel(const Params P, int by_unit) {
    constexpr int ROWS = 8 * NT;
    constexpr int LANES = MERGE_THREADS / (DH / 4);   // pieces side by side
    __shared__ long long starts[MAX_BATCH + 1];
    __shared__ long long totals[8];
    __shared__ float w_s[MERGE_THREADS];
    __shared__ float red[2][MERGE_THREADS / 32];
    __shared__ float4 part[LANES][DH / 4];
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    tile_starts<MERGE_THREADS>(P, starts, totals);
    const int per = P.hkv * P.groups;
    const long long total = starts[P.batch] * per;
    const int G = (int)min((long long)P.G, total);
    long long unit_start, unit_end;
    int b, u;
    if (by_unit) {
        b = (int)(blockIdx.x / (unsigned)per);
        u = (int)(blockIdx.x - (unsigned)b * per);
        const long long n = starts[b + 1] - starts[b];
        if (n == 0) return;
        unit_start = starts[b] * per + u * n;
        unit_end = unit_start + n;
    } else {
        const int c = blockIdx.x + 1;
        if (c >= G) return;
        const long long pos = range_begin(total, G, c);
        b = sequence_of(P, starts, per, pos);
        const uint32_t off = (uint32_t)(pos - starts[b] * per);
        const uint32_t n = (uint32_t)(starts[b + 1] - starts[b]);
        u = (int)(off / n);
        unit_start = starts[b] * per + (long long)u * n;
        unit_end = unit_start + n;
        if (unit_start == pos || range_of(total, G, unit_start) != c - 1) return;
    }
    const int c0 = range_of(total, G, unit_start), c1 = range_of(total, G, unit_end - 1);
    if (c0 == c1) return;
    const int h = u / P.groups, g = u - h * P.groups;
    const int r = blockIdx.y;
    if (g * ROWS + r >= P.nq) return;
    const int slot0 = range_begin(total, G, c0) == unit_start ? 0 : 1;
    const int pieces = c1 - c0 + 1;   // at most MERGE_THREADS
    auto row_of = [&](int i) {
        return ((long long)(c0 + i) * 2 + (i == 0 ? slot0 : 0)) * ROWS + r;
    };
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (tid < pieces) ml = __ldcg(reinterpret_cast<const float2*>(P.ws_ml + row_of(tid) * 2));
    float m = ml.x;
#pragma unroll
    for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    if (lane == 0) red[0][warp] = m;
    __syncthreads();
    m = red[0][0];
#pragma unroll
    for (int x = 1; x < MERGE_THREADS / 32; ++x) m = fmaxf(m, red[0][x]);
    const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - m);
    w_s[tid] = w;
    float sum = w * ml.y;
#pragma unroll
    for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    if (lane == 0) red[1][warp] = sum;
    __syncthreads();
    const int at = tid % (DH / 4), first = tid / (DH / 4);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = first; i < pieces; i += LANES) {
        const float4 v =
            __ldcg(reinterpret_cast<const float4*>(P.ws_o + row_of(i) * DH) + at);
        const float f = w_s[i];
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
    }
    part[first][at] = acc;
    __syncthreads();
    if (first == 0) {
        float L = 0.f;
#pragma unroll
        for (int x = 0; x < MERGE_THREADS / 32; ++x) L += red[1][x];
#pragma unroll
        for (int x = 1; x < LANES; ++x) {
            const float4 v = part[x][at];
            acc.x += v.x;
            acc.y += v.y;
            acc.z += v.z;
            acc.w += v.w;
        }
        const float inv = L > 0.f ? *P.scale_dev[1] / L : isnan(L) ? NAN : 0.f;
        uint2 v;
        v.x = pack_half2(acc.x * inv, acc.y * inv);
        v.y = pack_half2(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2*>(P.out + row_offset(P, b, h, g * ROWS + r, DH) + at * 4) = v;
    }
}

template <int DH, int NT>
int launch(const Params& P, cudaStream_t stream) {
    using L = Layout<DH, NT>;
    if (ensure_smem_limit(reinterpret_cast<const void*>(split_kernel<DH, NT>), L::BYTES) != GQA_OK)
        return GQA_ERR_CUDA;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(P.G);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = L::BYTES;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, split_kernel<DH, NT>, P) != cudaSuccess) return GQA_ERR_CUDA;
    if (P.G == 1) return GQA_OK;   // nothing is cut
    // A block for each unit or for each cut, whichever are fewer.
    const long long units = (long long)P.batch * P.hkv * P.groups;
    const int by_unit = units < P.G - 1;
    cfg.gridDim = dim3(by_unit ? (unsigned)units : P.G - 1, P.nq < 8 * NT ? P.nq : 8 * NT);
    cfg.blockDim = dim3(MERGE_THREADS);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, merge_kernel<DH, NT>, P, by_unit) != cudaSuccess)
        return GQA_ERR_CUDA;
    return GQA_OK;
}

// Packed rows of a unit: 8, or 16 where there are more.
int unit_rows(int nq) { return nq <= 8 ? 8 : 16; }

}  // namespace paged4

size_t paged_fp4_workspace_bytes(int nq, int num_sms, int Dh) {
    return kWorkspaceCounterBytes +
           (size_t)2 * num_sms * paged4::unit_rows(nq) * (Dh + 2) * sizeof(float);
}

int paged_fp4_launch(const void* q, const uint8_t* kcache, const uint8_t* vcache,
                     const float* kscale, const float* vscale, const int32_t* block_tables,
                     int table_stride, int num_pages, int page, const int* ctx_lens_dev,
                     int max_ctx_len, int batch, int R, int Hq, int Hkv, int Dh, float scale,
                     int window, int sinks, void* out, cudaStream_t stream) {
    using namespace paged4;
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
    P.groups = (P.nq + rows - 1) / rows;
    // A window that holds every context hides nothing.
    P.window = window >= max_ctx_len ? 0 : window;
    P.sinks = P.window > 0 ? sinks : 0;
    P.scale = scale;
    // No more ranges than tiles.
    const long long tiles = (long long)batch * Hkv * P.groups * ((max_ctx_len + TILE - 1LL) / TILE);
    P.G = (int)(tiles < di->num_sms ? tiles : di->num_sms);
    if (P.G > MERGE_THREADS) P.G = MERGE_THREADS;
    P.out = static_cast<__half*>(out);
    P.err = di->err_word;
    void* ws;
    size_t ws_bytes;
    current_workspace(&ws, &ws_bytes);
    if (!ws || ws_bytes < paged_fp4_workspace_bytes(P.nq, di->num_sms, Dh))
        return GQA_ERR_WORKSPACE;
    P.ws_o = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kWorkspaceCounterBytes);
    P.ws_ml = P.ws_o + (size_t)2 * P.G * rows * Dh;
    if (Dh == 256) return rows == 8 ? launch<256, 1>(P, stream) : launch<256, 2>(P, stream);
    return rows == 8 ? launch<128, 1>(P, stream) : launch<128, 2>(P, stream);
}

}  // namespace gqa

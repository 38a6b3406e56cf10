// cache_ops.cu -- the operators that fill and read back the paged cache: the
// cache write (per-head RMS norm, position rotation and the store of K and V,
// quantised or not), the cache read (dense K / V rows of cached tokens) and
// the block index (an int8 summary of every finished 4-token block).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <type_traits>

#include "cache_rows.cuh"

namespace gqa {
namespace cacheops {

constexpr int THREADS = 256;
constexpr int MAX_TILE = 16;            // most tokens of one write CTA
constexpr int WRITE_CTAS = 4;           // write CTAs resident on an SM (64 registers a thread)
constexpr int MAX_ROT_PAIRS = 128;      // rotated pairs of a head (rot_dim <= 256)

// 1 / (2 pi) as the sum of two floats.
constexpr double kInvTwoPi = 0.15915494309189533577;
constexpr float kInvTwoPiHi = (float)kInvTwoPi;
constexpr float kInvTwoPiLo = (float)(kInvTwoPi - (double)kInvTwoPiHi);

struct WriteParams {
    RowMap rows;
    const uint16_t* x[3];        // q, k, v: 16-bit floats
    long long token_stride[3];   // elements
    long long head_stride[3];
    const uint16_t* weight[2];   // q, k norm weights (null: no norm)
    float eps;
    const float* inv_freq;
    int pairs;                   // rot_dim / 2 (0: no rotation)
    int interleaved;
    const float* kscale;
    const float* vscale;
    __half* q_out;
    void* kcache;
    void* vcache;
    int nq;                      // query heads handled (0 without q)
    int hkv;
    FastDiv heads;               // nq + 2 * hkv
    FastDiv by_pairs;
    int tile;                    // tokens per CTA
};

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if (BF16) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

template <bool BF16>
__device__ __forceinline__ void unpack4(const uint2& u, float* x) {
    const float2 a = unpack2<BF16>(u.x), b = unpack2<BF16>(u.y);
    x[0] = a.x;
    x[1] = a.y;
    x[2] = b.x;
    x[3] = b.y;
}

__device__ __forceinline__ uint2 pack4_half(const float* x) {
    return make_uint2(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]));
}

// Two values to E4M3 codes: round to nearest even, +-448 beyond the range.
__device__ __forceinline__ uint32_t pack2_e4m3(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// cos and sin of position * frequency, as a fraction of a turn: the product
// position * frequency / (2 pi) is formed to about 48 bits (two floats and
// the product's own rounding error), so that far positions keep their angle.
__device__ __forceinline__ float2 turn(int pos, float hi, float lo) {
    float frac = 0.f;
    // Parts of at most 24 bits, each exact as a float.
    const int low = pos & 0xffffff, high = pos - low;
    {
        const float p = (float)low;
        const float u = __fmul_rn(p, hi);
        const float e = __fmaf_rn(p, hi, -u);
        frac = (u - rintf(u)) + __fmaf_rn(p, lo, e);
    }
    if (high) {
        const float p = (float)high;
        const float u = __fmul_rn(p, hi);
        const float e = __fmaf_rn(p, hi, -u);
        const float l = __fmul_rn(p, lo);
        frac += (u - rintf(u)) + ((e - rintf(e)) + (l - rintf(l)) + __fmaf_rn(p, lo, -l));
    }
    frac -= rintf(frac);
    float2 cs;
    sincospif(2.f * frac, &cs.y, &cs.x);
    return cs;
}

// One CTA takes `tile` tokens: it finds their cache rows, computes each
// rotated pair's cos / sin once for all heads of the token into shared
// memory, then groups of DH / 8 lanes take one head each, WRITE_AHEAD heads'
// loads in flight together (the first ones issued before the addresses are
// known).  y = x / sqrt(mean(x^2) + eps) * w and the rotation in 32 bits; one
// rounding at the end (fp16 for q, the cache's type for K and V).
//
// A lane holds two runs of four values: in the rotated part both members of
// four pairs, so no value crosses lanes.  Pairs (i, i + rot / 2): runs 4 l and
// rot / 2 + 4 l; pairs (2 i, 2 i + 1), and the values that do not turn: runs 8 l
// and 8 l + 4.
constexpr int WRITE_AHEAD = 4;

template <int DH, bool E4M3, bool BF16>
__global__ void __launch_bounds__(THREADS, WRITE_CTAS) write_kernel(const WriteParams P) {
    constexpr int LANES = DH / 8;
    constexpr int GROUPS = THREADS / LANES;
    __shared__ int s_starts[kRowsMaxBatch + 1];
    __shared__ int s_pos[MAX_TILE];
    __shared__ long long s_slot[MAX_TILE];
    __shared__ __align__(16) float s_cos[MAX_TILE][MAX_ROT_PAIRS];
    __shared__ __align__(16) float s_sin[MAX_TILE][MAX_ROT_PAIRS];
    const int t0 = blockIdx.x * P.tile;
    const int nt = min(P.tile, P.rows.tokens - t0);
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
    const bool turns = lane < P.pairs / 4;
    const bool split = turns && !P.interleaved;
    const int run0 = split ? lane * 4 : lane * 8;
    const int run1 = split ? P.pairs + lane * 4 : lane * 8 + 4;
    const int n_items = nt * P.heads.d;

    struct Item {
        int t, kind, head;
    };
    auto item_of = [&](int item) {
        Item m;
        m.t = P.heads.div(item);
        const int h = item - m.t * P.heads.d;
        m.kind = h < P.nq ? 0 : h < P.nq + P.hkv ? 1 : 2;
        m.head = m.kind == 0 ? h : m.kind == 1 ? h - P.nq : h - P.nq - P.hkv;
        return m;
    };
    uint2 raw[WRITE_AHEAD][2];
    auto load = [&](int it) {
#pragma unroll
        for (int u = 0; u < WRITE_AHEAD; ++u) {
            // (a group without an item reads the last one and stores nothing)
            const Item m = item_of(min(it + u * GROUPS + group, n_items - 1));
            const uint16_t* x = P.x[m.kind] + (long long)(t0 + m.t) * P.token_stride[m.kind] +
                                m.head * P.head_stride[m.kind];
            raw[u][0] = *reinterpret_cast<const uint2*>(x + run0);
            raw[u][1] = *reinterpret_cast<const uint2*>(x + run1);
        }
    };
    load(0);
    uint2 weight[2][2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (P.weight[k]) {
            weight[k][0] = *reinterpret_cast<const uint2*>(P.weight[k] + run0);
            weight[k][1] = *reinterpret_cast<const uint2*>(P.weight[k] + run1);
        }
    const float inv[2] = {E4M3 ? 1.f / *P.kscale : 1.f, E4M3 ? 1.f / *P.vscale : 1.f};

    if (P.rows.row_starts) {
        load_row_starts(P.rows, s_starts);
        __syncthreads();
    }
    if (threadIdx.x < nt)
        locate_row(P.rows, s_starts, t0 + threadIdx.x, &s_pos[threadIdx.x], &s_slot[threadIdx.x]);
    __syncthreads();
    if (P.pairs) {
        for (int i = threadIdx.x; i < nt * P.pairs; i += THREADS) {
            const int t = P.by_pairs.div(i), j = i - t * P.pairs;
            const float f = P.inv_freq[j];
            const float hi = __fmul_rn(f, kInvTwoPiHi);
            const float lo = __fmaf_rn(f, kInvTwoPiLo, __fmaf_rn(f, kInvTwoPiHi, -hi));
            const float2 cs = turn(max(s_pos[t], 0), hi, lo);
            s_cos[t][j] = cs.x;
            s_sin[t][j] = cs.y;
        }
        __syncthreads();
    }

    // Every lane of a warp takes the same number of turns (the shuffles need it).
    for (int it = 0; it < n_items; it += WRITE_AHEAD * GROUPS) {
        if (it > 0) load(it);
#pragma unroll
        for (int u = 0; u < WRITE_AHEAD; ++u) {
            if (it + u * GROUPS >= n_items) break;
            const bool live = it + u * GROUPS + group < n_items;
            const Item m = item_of(min(it + u * GROUPS + group, n_items - 1));
            float x[8];
            unpack4<BF16>(raw[u][0], x);
            unpack4<BF16>(raw[u][1], x + 4);
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
            for (int o = LANES / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (m.kind < 2) {
                if (P.weight[m.kind]) {
                    float w[8];
                    unpack4<BF16>(m.kind ? weight[1][0] : weight[0][0], w);
                    unpack4<BF16>(m.kind ? weight[1][1] : weight[0][1], w + 4);
                    const float r = rsqrtf(ss * (1.f / DH) + P.eps);
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
                }
                if (turns) {
                    const float4 c4 = *reinterpret_cast<const float4*>(&s_cos[m.t][lane * 4]);
                    const float4 s4 = *reinterpret_cast<const float4*>(&s_sin[m.t][lane * 4]);
                    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
                    if (split) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float a = x[i], b = x[4 + i];
                            x[i] = a * c[i] - b * s[i];
                            x[4 + i] = b * c[i] + a * s[i];
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float a = x[2 * i], b = x[2 * i + 1];
                            x[2 * i] = a * c[i] - b * s[i];
                            x[2 * i + 1] = b * c[i] + a * s[i];
                        }
                    }
                }
            }
            if (!live || s_pos[m.t] < 0) continue;
            if (m.kind == 0) {
                __half* q = P.q_out + ((long long)(t0 + m.t) * P.nq + m.head) * DH;
                *reinterpret_cast<uint2*>(q + run0) = pack4_half(x);
                *reinterpret_cast<uint2*>(q + run1) = pack4_half(x + 4);
                continue;
            }
            if (s_slot[m.t] < 0) continue;
            const long long at = (s_slot[m.t] * P.hkv + m.head) * DH;
            void* cache = m.kind == 1 ? P.kcache : P.vcache;
            if (E4M3) {
                uint8_t* c = static_cast<uint8_t*>(cache) + at;
                const float f = inv[m.kind - 1];
                *reinterpret_cast<uint32_t*>(c + run0) =
                    pack2_e4m3(x[0] * f, x[1] * f) | pack2_e4m3(x[2] * f, x[3] * f) << 16;
                *reinterpret_cast<uint32_t*>(c + run1) =
                    pack2_e4m3(x[4] * f, x[5] * f) | pack2_e4m3(x[6] * f, x[7] * f) << 16;
            } else {
                __half* c = static_cast<__half*>(cache) + at;
                *reinterpret_cast<uint2*>(c + run0) = pack4_half(x);
                *reinterpret_cast<uint2*>(c + run1) = pack4_half(x + 4);
            }
        }
    }
}

struct ReadParams {
    RowMap rows;
    const uint8_t* cache[2];   // K, V
    const float* scale[2];     // E4M3 dequantisation scales (null: rows as they are)
    uint8_t* out[2];
    int row_bytes;             // cached bytes of one token of K (or V)
    FastDiv chunks;            // pieces of one token's K (or V)
    int tile;                  // tokens per CTA
};

constexpr int MAX_READ_TILE = 64;
constexpr int READ_AHEAD = 4;

// Dense rows of cached tokens: DEQUANT reads 8 codes and writes 8 fp16 values
// a thread, the other form copies 16 bytes.  READ_AHEAD pieces of K and of V
// each are in flight together.
template <bool DEQUANT>
__global__ void __launch_bounds__(THREADS) read_kernel(const ReadParams P) {
    constexpr int IN = DEQUANT ? 8 : 16;
    using Piece = typename std::conditional<DEQUANT, uint2, uint4>::type;
    __shared__ int s_starts[kRowsMaxBatch + 1];
    __shared__ int s_pos[MAX_READ_TILE];
    __shared__ long long s_slot[MAX_READ_TILE];
    const int t0 = blockIdx.x * P.tile;
    const int nt = min(P.tile, P.rows.tokens - t0);
    if (P.rows.row_starts) {
        load_row_starts(P.rows, s_starts);
        __syncthreads();
    }
    if (threadIdx.x < nt)
        locate_row(P.rows, s_starts, t0 + threadIdx.x, &s_pos[threadIdx.x], &s_slot[threadIdx.x]);
    const float scale[2] = {DEQUANT ? *P.scale[0] : 1.f, DEQUANT ? *P.scale[1] : 1.f};
    __syncthreads();
    const int n = nt * P.chunks.d;
    for (int i0 = threadIdx.x; i0 < n; i0 += READ_AHEAD * THREADS) {
        Piece in[READ_AHEAD][2];
#pragma unroll
        for (int u = 0; u < READ_AHEAD; ++u) {
            const int i = i0 + u * THREADS;
            in[u][0] = in[u][1] = Piece{};
            if (i >= n) continue;
            const int t = P.chunks.div(i), c = i - t * P.chunks.d;
            if (s_slot[t] < 0) continue;
            const long long at = s_slot[t] * P.row_bytes + c * IN;
            in[u][0] = *reinterpret_cast<const Piece*>(P.cache[0] + at);
            in[u][1] = *reinterpret_cast<const Piece*>(P.cache[1] + at);
        }
#pragma unroll
        for (int u = 0; u < READ_AHEAD; ++u) {
            const int i = i0 + u * THREADS;
            if (i >= n) break;
            const int t = P.chunks.div(i);
            if (s_pos[t] < 0) continue;
            const long long to = ((long long)t0 * P.chunks.d + i) * 16;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                uint4 v;
                if constexpr (DEQUANT) {
                    uint32_t h[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t w = k < 2 ? in[u][kv].x : in[u][kv].y;
                        const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
                            (__nv_fp8x2_storage_t)(w >> (16 * (k & 1))), __NV_E4M3);
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
                        h[k] = pack_half2(f.x * scale[kv], f.y * scale[kv]);
                    }
                    v = make_uint4(h[0], h[1], h[2], h[3]);
                } else {
                    v = in[u][kv];
                }
                *reinterpret_cast<uint4*>(P.out[kv] + to) = v;
            }
        }
    }
}

struct IndexParams {
    RowMap rows;
    const uint8_t* kcache;
    const float* kscale;   // null for an fp16 cache
    int8_t* index;
    float* index_scale;
    int width;             // Hkv * D, a multiple of 128, at most 1024
    int tile;              // rows per CTA
};

constexpr int MAX_INDEX_TILE = 128;

// Eight keys' values of 16 (fp16) or 8 (E4M3) bytes.
template <bool E4M3>
struct Keys8 {
    typename std::conditional<E4M3, uint2, uint4>::type u;
    __device__ __forceinline__ void load(const uint8_t* cache, long long element) {
        u = *reinterpret_cast<const decltype(u)*>(cache + element * (E4M3 ? 1 : 2));
    }
    __device__ __forceinline__ float2 pair(int j) const {
        if constexpr (E4M3) {
            const uint32_t w = j < 2 ? u.x : u.y;
            const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
                (__nv_fp8x2_storage_t)(w >> (16 * (j & 1))), __NV_E4M3);
            return __half22float2(*reinterpret_cast<const __half2*>(&hr));
        } else {
            const uint32_t w = j == 0 ? u.x : j == 1 ? u.y : j == 2 ? u.z : u.w;
            return __half22float2(*reinterpret_cast<const __half2*>(&w));
        }
    }
};

// Summaries of the 4-token blocks whose last token is a row of this step: one
// warp a block, 8 values a lane of each 256 (CHUNKS of them), the keys of
// TOGETHER blocks in flight together.  The sums, the largest magnitude and the
// codes follow fixed 32-bit operations, so the codes are the same wherever and
// in whatever batch a block is summarised.
template <bool E4M3, int CHUNKS>
__global__ void __launch_bounds__(THREADS) index_kernel(const IndexParams P) {
    constexpr int TOGETHER = CHUNKS == 1 ? 2 : 1;
    constexpr int WARPS = THREADS / 32;
    __shared__ int s_starts[kRowsMaxBatch + 1];
    __shared__ long long s_block[MAX_INDEX_TILE];
    __shared__ int s_count;
    const int t0 = blockIdx.x * P.tile;
    const int nt = min(P.tile, P.rows.tokens - t0);
    if (P.rows.row_starts) load_row_starts(P.rows, s_starts);
    if (threadIdx.x == 0) s_count = 0;
    __syncthreads();
    if (threadIdx.x < nt) {
        int pos;
        long long slot;
        locate_row(P.rows, s_starts, t0 + threadIdx.x, &pos, &slot);
        if ((pos & 3) == 3 && slot >= 0) s_block[atomicAdd(&s_count, 1)] = slot >> 2;
    }
    const float unit = E4M3 ? *P.kscale / 508.f : 1.f / 508.f;
    __syncthreads();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int count = s_count;
    for (int i0 = warp; i0 < count; i0 += WARPS * TOGETHER) {
        Keys8<E4M3> k[TOGETHER][CHUNKS][4];
#pragma unroll
        for (int b = 0; b < TOGETHER; ++b) {
            const long long first = s_block[min(i0 + b * WARPS, count - 1)] * 4 * P.width;
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) {
                // (lanes past the width read its last values and store nothing)
                const int e = min(c * 256 + lane * 8, P.width - 8);
#pragma unroll
                for (int t = 0; t < 4; ++t) k[b][c][t].load(P.kcache, first + t * P.width + e);
            }
        }
#pragma unroll
        for (int b = 0; b < TOGETHER; ++b) {
            if (i0 + b * WARPS >= count) break;
            const long long block = s_block[i0 + b * WARPS];
            float s[CHUNKS][8];
            uint32_t most = 0;
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 x0 = k[b][c][0].pair(j), x1 = k[b][c][1].pair(j),
                                 x2 = k[b][c][2].pair(j), x3 = k[b][c][3].pair(j);
                    s[c][2 * j] = (x0.x + x1.x) + (x2.x + x3.x);
                    s[c][2 * j + 1] = (x0.y + x1.y) + (x2.y + x3.y);
                    // As whole numbers magnitudes keep their order, NaN above all.
                    most = max(most, __float_as_uint(s[c][2 * j]) & 0x7fffffffu);
                    most = max(most, __float_as_uint(s[c][2 * j + 1]) & 0x7fffffffu);
                }
            most = __reduce_max_sync(0xffffffffu, most);
            const bool fine = most != 0 && most < 0x7f800000u;
            const float inv = fine ? 127.f / __uint_as_float(most) : 0.f;
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) {
                const int e = c * 256 + lane * 8;
                if (e >= P.width) break;
                uint32_t w[2] = {0, 0};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int code = fine ? (int)rintf(__fmul_rn(s[c][j], inv)) : 0;
                    w[j / 4] |= (uint32_t)(code & 0xff) << (8 * (j % 4));
                }
                *reinterpret_cast<uint2*>(P.index + block * P.width + e) = make_uint2(w[0], w[1]);
            }
            if (lane == 0)
                P.index_scale[block] = fine ? __fmul_rn(__uint_as_float(most), unit) : 0.f;
        }
    }
}

template <bool E4M3>
void launch_index(const IndexParams& P, int grid, cudaStream_t stream) {
    if (P.width <= 256) index_kernel<E4M3, 1><<<grid, THREADS, 0, stream>>>(P);
    else if (P.width <= 512) index_kernel<E4M3, 2><<<grid, THREADS, 0, stream>>>(P);
    else index_kernel<E4M3, 4><<<grid, THREADS, 0, stream>>>(P);
}

RowMap make_rows(const CacheRows& r, const DeviceInfo* di) {
    RowMap m;
    m.tables = r.block_tables;
    m.row_starts = r.row_starts;
    m.ctx_lens = r.ctx_lens_dev;
    m.table_stride = r.table_stride;
    m.num_pages = r.num_pages;
    m.log2_page = __builtin_ctz((unsigned)r.page);
    m.max_ctx = r.max_ctx_len;
    m.batch = r.batch;
    m.tokens = r.tokens;
    m.rows_per_seq = make_fastdiv(r.row_starts ? 1 : r.tokens / r.batch);
    m.err = di->err_word;
    return m;
}

template <int DH, bool E4M3>
void launch_write(const WriteParams& P, bool bf16, int grid, cudaStream_t stream) {
    if (bf16) write_kernel<DH, E4M3, true><<<grid, THREADS, 0, stream>>>(P);
    else write_kernel<DH, E4M3, false><<<grid, THREADS, 0, stream>>>(P);
}

}  // namespace cacheops

int cache_write_launch(const CacheRows& r, const CacheWriteArgs& a, cudaStream_t stream) {
    using namespace cacheops;
    const DeviceInfo* di = device_info();
    if (!di) return GQA_ERR_CUDA;
    WriteParams P;
    P.rows = make_rows(r, di);
    for (int i = 0; i < 3; ++i) {
        P.x[i] = static_cast<const uint16_t*>(a.x[i]);
        P.token_stride[i] = a.token_stride[i];
        P.head_stride[i] = a.head_stride[i];
    }
    P.weight[0] = static_cast<const uint16_t*>(a.q_weight);
    P.weight[1] = static_cast<const uint16_t*>(a.k_weight);
    P.eps = a.eps;
    P.inv_freq = a.inv_freq;
    P.pairs = a.rot_dim / 2;
    P.interleaved = a.interleaved;
    P.kscale = a.kscale;
    P.vscale = a.vscale;
    P.q_out = static_cast<__half*>(a.q_out);
    P.kcache = a.kcache;
    P.vcache = a.vcache;
    P.nq = a.x[0] ? a.Hq : 0;
    P.hkv = a.Hkv;
    P.heads = make_fastdiv(P.nq + 2 * a.Hkv);
    P.by_pairs = make_fastdiv(P.pairs > 0 ? P.pairs : 1);
    // As many tokens a CTA as let all CTAs be resident at once.
    const int resident = di->num_sms * WRITE_CTAS;
    const int tile = (r.tokens + resident - 1) / resident;
    P.tile = tile < MAX_TILE ? tile : MAX_TILE;
    const int grid = (r.tokens + P.tile - 1) / P.tile;
    const bool bf16 = a.dtype == GQA_DTYPE_BF16;
    if (a.e4m3) {
        if (a.D == 256) launch_write<256, true>(P, bf16, grid, stream);
        else launch_write<128, true>(P, bf16, grid, stream);
    } else {
        if (a.D == 256) launch_write<256, false>(P, bf16, grid, stream);
        else launch_write<128, false>(P, bf16, grid, stream);
    }
    return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

int cache_read_launch(const CacheRows& r, const void* kcache, const void* vcache,
                      const float* kscale, const float* vscale, int row_bytes, void* k_out,
                      void* v_out, cudaStream_t stream) {
    using namespace cacheops;
    const DeviceInfo* di = device_info();
    if (!di) return GQA_ERR_CUDA;
    ReadParams P;
    P.rows = make_rows(r, di);
    P.cache[0] = static_cast<const uint8_t*>(kcache);
    P.cache[1] = static_cast<const uint8_t*>(vcache);
    P.scale[0] = kscale;
    P.scale[1] = vscale;
    P.out[0] = static_cast<uint8_t*>(k_out);
    P.out[1] = static_cast<uint8_t*>(v_out);
    P.row_bytes = row_bytes;
    P.chunks = make_fastdiv(row_bytes / (kscale ? 8 : 16));
    P.tile = r.tokens <= 2048 ? 8 : 32;
    const int grid = (r.tokens + P.tile - 1) / P.tile;
    if (kscale) read_kernel<true><<<grid, THREADS, 0, stream>>>(P);
    else read_kernel<false><<<grid, THREADS, 0, stream>>>(P);
    return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

int block_index_launch(const CacheRows& r, const void* kcache, const float* kscale, int width,
                       int8_t* index, float* index_scale, cudaStream_t stream) {
    using namespace cacheops;
    const DeviceInfo* di = device_info();
    if (!di) return GQA_ERR_CUDA;
    IndexParams P;
    P.rows = make_rows(r, di);
    P.kcache = static_cast<const uint8_t*>(kcache);
    P.kscale = kscale;
    P.index = index;
    P.index_scale = index_scale;
    P.width = width;
    P.tile = r.tokens <= 4096 ? 32 : MAX_INDEX_TILE;
    const int grid = (r.tokens + P.tile - 1) / P.tile;
    if (kscale) launch_index<true>(P, grid, stream);
    else launch_index<false>(P, grid, stream);
    return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace gqa

// cache_ops.cu -- the operators that fill and read back the paged cache: the
// cache write (per-head RMS norm, position rotation and the store of K and V,
// quantised or not), the cache read (dense K / V rows of cached tokens) and
// the block index (an int8 summary of every finished 4-token block).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "cache_rows.cuh"

namespace gqa {
namespace cacheops {

constexpr int THREADS = 256;
constexpr int MAX_TILE = 8;             // most tokens of one write CTA
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
    int tile;                    // tokens per CTA
};

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 f;
        if (BF16) f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
        else f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ uint4 pack8_half(const float (&x)[8]) {
    return make_uint4(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]), pack_half2(x[4], x[5]),
                      pack_half2(x[6], x[7]));
}

// Eight values to E4M3 codes: round to nearest even, +-448 beyond the range.
__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8], float inv) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * inv, x[2 * i + 1] * inv),
                                        __NV_SATFINITE, __NV_E4M3);
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
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
// memory, then groups of DH / 8 lanes take one head each (8 values a lane).
// y = x / sqrt(mean(x^2) + eps) * w and the rotation in 32 bits; one rounding
// at the end (fp16 for q, the cache's type for K and V).
template <int DH, bool E4M3, bool BF16>
__global__ void __launch_bounds__(THREADS) write_kernel(const WriteParams P) {
    constexpr int LANES = DH / 8;
    constexpr int GROUPS = THREADS / LANES;
    __shared__ int s_starts[kRowsMaxBatch + 1];
    __shared__ int s_pos[MAX_TILE];
    __shared__ long long s_slot[MAX_TILE];
    __shared__ float s_cos[MAX_TILE][MAX_ROT_PAIRS];
    __shared__ float s_sin[MAX_TILE][MAX_ROT_PAIRS];
    const int t0 = blockIdx.x * P.tile;
    const int nt = min(P.tile, P.rows.tokens - t0);
    load_row_starts(P.rows, s_starts);
    __syncthreads();
    if (threadIdx.x < nt)
        locate_row(P.rows, s_starts, t0 + threadIdx.x, &s_pos[threadIdx.x], &s_slot[threadIdx.x]);
    __syncthreads();
    for (int i = threadIdx.x; i < nt * P.pairs; i += THREADS) {
        const int t = i / P.pairs, j = i - t * P.pairs;
        const float f = P.inv_freq[j];
        const float hi = __fmul_rn(f, kInvTwoPiHi);
        const float lo = __fmaf_rn(f, kInvTwoPiLo, __fmaf_rn(f, kInvTwoPiHi, -hi));
        const float2 cs = turn(max(s_pos[t], 0), hi, lo);
        s_cos[t][j] = cs.x;
        s_sin[t][j] = cs.y;
    }
    __syncthreads();

    const int lane = threadIdx.x % LANES;
    const int group = threadIdx.x / LANES;
    const int n_items = nt * P.heads.d;
    const float kinv = E4M3 ? 1.f / *P.kscale : 1.f;
    const float vinv = E4M3 ? 1.f / *P.vscale : 1.f;
    // Every lane of a warp runs the same number of turns (the shuffles need it).
    for (int it = 0; it < n_items; it += GROUPS) {
        const int item = min(it + group, n_items - 1);
        const bool live = it + group < n_items;
        const int t = P.heads.div(item), h = item - t * P.heads.d;
        const int kind = h < P.nq ? 0 : h < P.nq + P.hkv ? 1 : 2;
        const int head = kind == 0 ? h : kind == 1 ? h - P.nq : h - P.nq - P.hkv;
        const uint4 raw = *reinterpret_cast<const uint4*>(
            P.x[kind] + (long long)(t0 + t) * P.token_stride[kind] + head * P.head_stride[kind] +
            lane * 8);
        float x[8];
        unpack8<BF16>(raw, x);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (kind < 2 && P.weight[kind]) {
            float w[8];
            unpack8<BF16>(*reinterpret_cast<const uint4*>(P.weight[kind] + lane * 8), w);
            const float r = rsqrtf(ss * (1.f / DH) + P.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
        }
        if (P.pairs) {
            if (P.interleaved) {
                if (kind < 2 && lane * 4 < P.pairs) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float c = s_cos[t][lane * 4 + i], s = s_sin[t][lane * 4 + i];
                        const float a = x[2 * i], b = x[2 * i + 1];
                        x[2 * i] = a * c - b * s;
                        x[2 * i + 1] = b * c + a * s;
                    }
                }
            } else {
                // Value i of the first half turns with value i of the second:
                // the partner sits pairs / 8 lanes away.
                const int half = P.pairs / 8;
                const bool first = lane < half;
                const int partner = first ? lane + half : lane < 2 * half ? lane - half : lane;
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], partner, LANES);
                if (kind < 2 && lane < 2 * half) {
                    const int j = (first ? lane : partner) * 8;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float c = s_cos[t][j + i], s = s_sin[t][j + i];
                        x[i] = x[i] * c + (first ? -y[i] : y[i]) * s;
                    }
                }
            }
        }
        if (!live || s_pos[t] < 0) continue;
        if (kind == 0) {
            *reinterpret_cast<uint4*>(P.q_out + ((long long)(t0 + t) * P.nq + head) * DH +
                                      lane * 8) = pack8_half(x);
            continue;
        }
        if (s_slot[t] < 0) continue;
        const long long at = (s_slot[t] * P.hkv + head) * DH + lane * 8;
        void* cache = kind == 1 ? P.kcache : P.vcache;
        if (E4M3)
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + at) =
                pack8_e4m3(x, kind == 1 ? kinv : vinv);
        else
            *reinterpret_cast<uint4*>(static_cast<__half*>(cache) + at) = pack8_half(x);
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

// Dense rows of cached tokens: DEQUANT reads 8 codes and writes 8 fp16 values
// a thread, the other form copies 16 bytes.
template <bool DEQUANT>
__global__ void __launch_bounds__(THREADS) read_kernel(const ReadParams P) {
    constexpr int IN = DEQUANT ? 8 : 16;
    __shared__ int s_starts[kRowsMaxBatch + 1];
    __shared__ int s_pos[MAX_READ_TILE];
    __shared__ long long s_slot[MAX_READ_TILE];
    const int t0 = blockIdx.x * P.tile;
    const int nt = min(P.tile, P.rows.tokens - t0);
    load_row_starts(P.rows, s_starts);
    __syncthreads();
    if (threadIdx.x < nt)
        locate_row(P.rows, s_starts, t0 + threadIdx.x, &s_pos[threadIdx.x], &s_slot[threadIdx.x]);
    __syncthreads();
    const int n = nt * P.chunks.d;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const float scale = DEQUANT ? *P.scale[kv] : 1.f;
#pragma unroll 4
        for (int i = threadIdx.x; i < n; i += THREADS) {
            const int t = P.chunks.div(i), c = i - t * P.chunks.d;
            if (s_pos[t] < 0) continue;
            const long long slot = s_slot[t];
            uint8_t* dst = P.out[kv] + ((long long)(t0 + t) * P.chunks.d + c) * 16;
            const uint8_t* src = P.cache[kv] + slot * P.row_bytes + c * IN;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (slot >= 0) {
                if (DEQUANT) {
                    const uint2 u = *reinterpret_cast<const uint2*>(src);
                    float x[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t w = k < 2 ? u.x : u.y;
                        const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
                            (__nv_fp8x2_storage_t)(w >> (16 * (k & 1))), __NV_E4M3);
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
                        x[2 * k] = f.x * scale;
                        x[2 * k + 1] = f.y * scale;
                    }
                    v = pack8_half(x);
                } else {
                    v = *reinterpret_cast<const uint4*>(src);
                }
            }
            *reinterpret_cast<uint4*>(dst) = v;
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

// Summaries of the 4-token blocks whose last token is a row of this step: one
// warp a block, 4 values a lane of each 128.  The sums, the largest magnitude
// and the codes follow fixed 32-bit operations, so the codes are the same
// wherever and in whatever batch a block is summarised.
template <bool E4M3>
__global__ void __launch_bounds__(THREADS) index_kernel(const IndexParams P) {
    __shared__ int s_starts[kRowsMaxBatch + 1];
    __shared__ long long s_block[MAX_INDEX_TILE];
    __shared__ int s_count;
    const int t0 = blockIdx.x * P.tile;
    const int nt = min(P.tile, P.rows.tokens - t0);
    load_row_starts(P.rows, s_starts);
    if (threadIdx.x == 0) s_count = 0;
    __syncthreads();
    if (threadIdx.x < nt) {
        int pos;
        long long slot;
        locate_row(P.rows, s_starts, t0 + threadIdx.x, &pos, &slot);
        if ((pos & 3) == 3 && slot >= 0) s_block[atomicAdd(&s_count, 1)] = slot >> 2;
    }
    __syncthreads();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const float unit = E4M3 ? *P.kscale / 508.f : 1.f / 508.f;
    for (int i = warp; i < s_count; i += THREADS / 32) {
        const long long block = s_block[i];
        float s[8][4];
        uint32_t most = 0;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            if (c * 128 >= P.width) break;
            float k[4][4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const long long at = (block * 4 + t) * P.width + c * 128 + lane * 4;
                if (E4M3) {
                    const uint32_t u = *reinterpret_cast<const uint32_t*>(P.kcache + at);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
                            (__nv_fp8x2_storage_t)(u >> (16 * j)), __NV_E4M3);
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
                        k[t][2 * j] = f.x;
                        k[t][2 * j + 1] = f.y;
                    }
                } else {
                    const uint2 u = *reinterpret_cast<const uint2*>(P.kcache + at * 2);
                    const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
                    const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
                    k[t][0] = f0.x;
                    k[t][1] = f0.y;
                    k[t][2] = f1.x;
                    k[t][3] = f1.y;
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[c][j] = (k[0][j] + k[1][j]) + (k[2][j] + k[3][j]);
                // As whole numbers magnitudes keep their order, NaN above all.
                most = max(most, __float_as_uint(s[c][j]) & 0x7fffffffu);
            }
        }
        most = __reduce_max_sync(0xffffffffu, most);
        const bool fine = most != 0 && most < 0x7f800000u;
        const float inv = fine ? 127.f / __uint_as_float(most) : 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            if (c * 128 >= P.width) break;
            uint32_t w = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int code = fine ? (int)rintf(__fmul_rn(s[c][j], inv)) : 0;
                w |= (uint32_t)(code & 0xff) << (8 * j);
            }
            *reinterpret_cast<uint32_t*>(P.index + block * P.width + c * 128 + lane * 4) = w;
        }
        if (lane == 0)
            P.index_scale[block] = fine ? __fmul_rn(__uint_as_float(most), unit) : 0.f;
    }
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
    P.tile = r.tokens <= 1024 ? 1 : MAX_TILE;
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
    if (kscale) index_kernel<true><<<grid, THREADS, 0, stream>>>(P);
    else index_kernel<false><<<grid, THREADS, 0, stream>>>(P);
    return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace gqa

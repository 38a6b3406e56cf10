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
constexpr int WRITE_WARPS = 16;         // write warps an SM is given before heads are shared out

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
    FastDiv shares;              // warps a token's heads are shared out to
    int heads_per_share;
    int tokens_per_warp;         // 1 if the heads are shared out
};

// Two floats as one operand of the packed 32-bit operations.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pack(float lo, float hi) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
    return p;
}
__device__ __forceinline__ float2 unpack(Pair p) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
    return f;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

template <bool BF16>
__device__ __forceinline__ Pair unpack16(uint32_t w) {
    const float2 f = BF16 ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w))
                          : __half22float2(*reinterpret_cast<const __half2*>(&w));
    return pack(f.x, f.y);
}
__device__ __forceinline__ uint32_t to_half2(Pair p) {
    const float2 f = unpack(p);
    return pack_half2(f.x, f.y);
}
// Two values to E4M3 codes: round to nearest even, +-448 beyond the range.
__device__ __forceinline__ uint32_t to_e4m3x2(Pair p) {
    return __nv_cvt_float2_to_fp8x2(unpack(p), __NV_SATFINITE, __NV_E4M3);
}

// cos and sin of position * frequency, as a fraction of a turn: the product
// position * frequency / (2 pi) is formed to about 48 bits (two floats and
// the product's own rounding error), so that far positions keep their angle;
// then the hardware's approximations (error below 2^-20 within half a turn).
__device__ __forceinline__ float2 turn(int pos, float hi, float lo) {
    // Parts of at most 24 bits, each exact as a float.
    const int low = pos & 0xffffff, high = pos - low;
    float frac;
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
    const float angle = frac * 6.283185307179586f;
    return make_float2(__cosf(angle), __sinf(angle));
}

// A warp takes some tokens, one after the other, or when there are few a share
// of one token's heads.  It finds all its tokens' cache rows at once (a lane
// each), and always has the next WRITE_AHEAD heads' loads in flight while it
// works on the present ones.  It computes the cos and sin of its lanes' own
// pairs once for all heads of a token.  No thread waits for another warp.
// (Tokens of a CTA sharing addresses and cos / sin through shared memory kept
// 8000 rows at 21 us whatever the tile, and so did a warp for each token with
// all loads in front: in both the loads of a warp and its work took turns.)
//
// y = x / sqrt(mean(x^2) + eps) * w and the rotation in 32 bits; one rounding
// at the end (fp16 for q, the cache's type for K and V).
//
// DH / 8 lanes take a head (two heads a warp at DH = 128), each lane two runs of
// four values: in the rotated part both members of four pairs, so no value
// crosses lanes.  Pairs (i, i + rot / 2): runs 4 l and rot / 2 + 4 l; pairs
// (2 i, 2 i + 1), and the values that do not turn: runs 8 l and 8 l + 4.
constexpr int WRITE_AHEAD = 4;
constexpr int WRITE_THREADS = 128;

template <int DH, bool E4M3, bool BF16>
__global__ void __launch_bounds__(WRITE_THREADS) write_kernel(const WriteParams P) {
    constexpr int LANES = DH / 8;
    constexpr int GROUPS = 32 / LANES;     // heads a warp takes at once
    constexpr int AHEAD = WRITE_AHEAD;
    __shared__ int s_starts[kRowsMaxBatch + 1];
    const int warp = blockIdx.x * (WRITE_THREADS / 32) + threadIdx.x / 32;
    const int part = P.shares.div(warp), share = warp - part * P.shares.d;
    const int token0 = part * P.tokens_per_warp;
    const int n_tokens = min(P.tokens_per_warp, P.rows.tokens - token0);
    const int wlane = threadIdx.x % 32, lane = wlane % LANES, group = wlane / LANES;
    const bool turns = lane < P.pairs / 4;
    const bool split = turns && !P.interleaved;
    const int run0 = split ? lane * 4 : lane * 8;
    const int run1 = split ? P.pairs + lane * 4 : lane * 8 + 4;
    const int k0 = P.nq, v0 = k0 + P.hkv, heads = v0 + P.hkv;   // heads: q, then K, then V
    const int h0 = share * P.heads_per_share, h1 = min(h0 + P.heads_per_share, heads);

    // The loads walk the tokens, and in each the heads of this group of lanes (h0
    // + group, + GROUPS, ...), AHEAD at a time: where the next one's values are,
    // up to the last head of its kind.
    int load_token = token0, load_i = 0, load_h = h0 + group, load_end = 0;
    const uint16_t* src = nullptr;
    long long src_step = 0;
    auto load = [&](uint2 (&raw)[AHEAD][2]) {
        if (load_token >= token0 + n_tokens) return;
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            if (load_h >= h1) break;
            if (load_h >= load_end) {
                const int kind = load_h < k0 ? 0 : load_h < v0 ? 1 : 2;
                const int begin = kind == 0 ? 0 : kind == 1 ? k0 : v0;
                load_end = kind == 0 ? k0 : kind == 1 ? v0 : heads;
                src = P.x[kind] + load_token * P.token_stride[kind] +
                      (load_h - begin) * P.head_stride[kind];
                src_step = GROUPS * P.head_stride[kind];
            }
            raw[u][0] = *reinterpret_cast<const uint2*>(src + run0);
            raw[u][1] = *reinterpret_cast<const uint2*>(src + run1);
            src += src_step;
            load_h += GROUPS;
        }
        load_i += AHEAD * GROUPS;
        if (load_i >= h1 - h0) {
            ++load_token;
            load_i = 0;
            load_h = h0 + group;
            load_end = 0;
        }
    };
    uint2 next[AHEAD][2];
    load(next);

    if (P.rows.row_starts) {
        load_row_starts(P.rows, s_starts);
        __syncthreads();
    }
    if (n_tokens <= 0) return;
    int my_pos = -1;             // lane i: token token0 + i
    long long my_slot = -1;
    if (wlane < n_tokens) locate_row(P.rows, s_starts, token0 + wlane, &my_pos, &my_slot);
    const float inv[2] = {E4M3 ? 1.f / *P.kscale : 1.f, E4M3 ? 1.f / *P.vscale : 1.f};
    float4 freq = make_float4(0.f, 0.f, 0.f, 0.f);
    if (turns) {
        freq.x = P.inv_freq[lane * 4];
        freq.y = P.inv_freq[lane * 4 + 1];
        freq.z = P.inv_freq[lane * 4 + 2];
        freq.w = P.inv_freq[lane * 4 + 3];
    }

    for (int i_token = 0; i_token < n_tokens; ++i_token) {
    const int token = token0 + i_token;
    const int pos = __shfl_sync(0xffffffffu, my_pos, i_token);
    const long long slot = __shfl_sync(0xffffffffu, my_slot, i_token);
    Pair c[2], s[2];     // cos and sin of pairs 4 l .. 4 l + 3
    if (turns) {
        float cs[4], sn[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float f = i == 0 ? freq.x : i == 1 ? freq.y : i == 2 ? freq.z : freq.w;
            const float hi = __fmul_rn(f, kInvTwoPiHi);
            const float lo = __fmaf_rn(f, kInvTwoPiLo, __fmaf_rn(f, kInvTwoPiHi, -hi));
            const float2 t = turn(max(pos, 0), hi, lo);
            cs[i] = t.x;
            sn[i] = t.y;
        }
        c[0] = pack(cs[0], cs[1]);
        c[1] = pack(cs[2], cs[3]);
        s[0] = pack(sn[0], sn[1]);
        s[1] = pack(sn[2], sn[3]);
    }

    // The head at hand: its kind until `end`, that kind's weights (or 1 / scale
    // for V), and where it goes.
    int h = h0 + group, end = 0, kind = 0;
    bool norm = false, store = true;
    float scale = 1.f;
    Pair w[4];
    uint8_t* out = nullptr;
    long long out_step = 0;
    const int warp_end = h1 - h0;
    // Every lane of a warp takes the same number of heads (the shuffles need it);
    // one past the last is not stored.
    for (int i0 = 0; i0 < warp_end; i0 += AHEAD * GROUPS) {
        uint2 raw[AHEAD][2];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            raw[u][0] = next[u][0];
            raw[u][1] = next[u][1];
        }
        load(next);
        if (pos < 0) continue;
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            if (i0 + u * GROUPS >= warp_end) break;
            if (h >= end) {
                kind = h < k0 ? 0 : h < v0 ? 1 : 2;
                end = kind == 0 ? k0 : kind == 1 ? v0 : heads;
                const int head = h - (kind == 0 ? 0 : kind == 1 ? k0 : v0);
                if (kind == 0) {
                    out = reinterpret_cast<uint8_t*>(P.q_out +
                                                     ((long long)token * P.nq + head) * DH);
                    out_step = GROUPS * DH * 2;
                } else {
                    constexpr int SIZE = E4M3 ? 1 : 2;
                    out = static_cast<uint8_t*>(kind == 1 ? P.kcache : P.vcache) +
                          (slot * P.hkv + head) * (DH * SIZE);
                    out_step = GROUPS * DH * SIZE;
                    scale = inv[kind - 1];
                }
                store = h < h1 && (kind == 0 || slot >= 0);
                const uint16_t* weight = kind < 2 ? P.weight[kind] : nullptr;
                norm = weight != nullptr;
                if (norm) {
                    const uint2 a = *reinterpret_cast<const uint2*>(weight + run0);
                    const uint2 b = *reinterpret_cast<const uint2*>(weight + run1);
                    w[0] = unpack16<BF16>(a.x);
                    w[1] = unpack16<BF16>(a.y);
                    w[2] = unpack16<BF16>(b.x);
                    w[3] = unpack16<BF16>(b.y);
                }
            }
            Pair x[4] = {unpack16<BF16>(raw[u][0].x), unpack16<BF16>(raw[u][0].y),
                         unpack16<BF16>(raw[u][1].x), unpack16<BF16>(raw[u][1].y)};
            if (i0 + u * GROUPS + h0 < v0) {      // (not all V)
                Pair sq = mul2(x[0], x[0]);
#pragma unroll
                for (int i = 1; i < 4; ++i) sq = fma2(x[i], x[i], sq);
                const float2 halves = unpack(sq);
                float ss = halves.x + halves.y;
#pragma unroll
                for (int o = LANES / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                if (norm) {
                    const float r = rsqrtf(ss * (1.f / DH) + P.eps);
                    const Pair rr = pack(r, r);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = mul2(mul2(x[i], rr), w[i]);
                }
                if (turns && kind < 2) {
                    if (split) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const Pair a = x[i], b = x[2 + i];
                            // (the sign of a packed operand is one bit each)
                            const Pair minus_s = s[i] ^ 0x8000000080000000ull;
                            x[i] = fma2(b, minus_s, mul2(a, c[i]));
                            x[2 + i] = fma2(a, s[i], mul2(b, c[i]));
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 ab = unpack(x[i]);
                            const float2 c2 = unpack(c[i / 2]), s2 = unpack(s[i / 2]);
                            const float ci = i & 1 ? c2.y : c2.x, si = i & 1 ? s2.y : s2.x;
                            x[i] = pack(ab.x * ci - ab.y * si, ab.y * ci + ab.x * si);
                        }
                    }
                }
            }
            h += GROUPS;
            uint8_t* const to = out;
            out += out_step;
            if (!store || h - GROUPS >= h1) continue;
            if (E4M3 && kind > 0) {
                const Pair f = pack(scale, scale);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = mul2(x[i], f);
                *reinterpret_cast<uint32_t*>(to + run0) = to_e4m3x2(x[0]) | to_e4m3x2(x[1]) << 16;
                *reinterpret_cast<uint32_t*>(to + run1) = to_e4m3x2(x[2]) | to_e4m3x2(x[3]) << 16;
            } else {
                *reinterpret_cast<uint2*>(to + 2 * run0) = make_uint2(to_half2(x[0]), to_half2(x[1]));
                *reinterpret_cast<uint2*>(to + 2 * run1) = make_uint2(to_half2(x[2]), to_half2(x[3]));
            }
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
};

// Eight keys' values of 16 (fp16) or 8 (E4M3) bytes.
template <bool E4M3>
struct Keys8 {
    typename std::conditional<E4M3, uint2, uint4>::type u;
    __device__ __forceinline__ void load(const uint8_t* cache, long long element) {
        u = *reinterpret_cast<const decltype(u)*>(cache + element * (E4M3 ? 1 : 2));
    }
    // Values 2 j and 2 j + 1 as fp16.
    __device__ __forceinline__ uint32_t pair(int j) const {
        if constexpr (E4M3) {
            const uint32_t w = j < 2 ? u.x : u.y;
            const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
                (__nv_fp8x2_storage_t)(w >> (16 * (j & 1))), __NV_E4M3);
            return *reinterpret_cast<const uint32_t*>(&hr);
        } else {
            return j == 0 ? u.x : j == 1 ? u.y : j == 2 ? u.z : u.w;
        }
    }
};

// fp16 + fp32 with one 32-bit rounding.
__device__ __forceinline__ float add_half(uint16_t h, float c) {
    float d;
    asm("add.f32.f16 %0, %1, %2;" : "=f"(d) : "h"(h), "f"(c));
    return d;
}
// (a + b) + (c + d) of four fp16 values in 32 bits.
__device__ __forceinline__ float sum4(uint16_t a, uint16_t b, uint16_t c, uint16_t d) {
    return __fadd_rn(add_half(b, __half2float(__ushort_as_half(a))),
                     add_half(d, __half2float(__ushort_as_half(c))));
}
// The largest magnitude; NaN if there is one.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Summaries of the 4-token blocks whose last token is a row of this step.  A
// warp takes 32 rows, a lane each to find the blocks they finish, then block
// after block: 8 values a lane of each 256 (CHUNKS of them), the keys of
// TOGETHER blocks in flight together.  The sums, the largest magnitude and the
// codes follow fixed 32-bit operations, so the codes are the same wherever and
// in whatever batch a block is summarised.
constexpr int INDEX_THREADS = 128;

template <bool E4M3, int CHUNKS>
__global__ void __launch_bounds__(INDEX_THREADS) index_kernel(const IndexParams P) {
    constexpr int TOGETHER = CHUNKS == 1 ? 4 : CHUNKS == 2 ? 2 : 1;
    __shared__ int s_starts[kRowsMaxBatch + 1];
    if (P.rows.row_starts) {
        load_row_starts(P.rows, s_starts);
        __syncthreads();
    }
    const int lane = threadIdx.x % 32;
    const int row = blockIdx.x * INDEX_THREADS + threadIdx.x;
    int pos = -1;
    long long slot = -1;
    if (row < P.rows.tokens) locate_row(P.rows, s_starts, row, &pos, &slot);
    const float unit = E4M3 ? *P.kscale / 508.f : 1.f / 508.f;
    uint32_t ends = __ballot_sync(0xffffffffu, (pos & 3) == 3 && slot >= 0);
    while (ends) {
        long long block[TOGETHER];
        Keys8<E4M3> k[TOGETHER][CHUNKS][4];
        const uint32_t all = ends;
#pragma unroll
        for (int b = 0; b < TOGETHER; ++b) {
            // (none left: the last one again, stored once)
            block[b] = __shfl_sync(0xffffffffu, slot, __ffs(ends ? ends : all) - 1) >> 2;
            ends &= ends - 1;
            const long long first = block[b] * 4 * P.width;
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
            if (b >= __popc(all)) break;
            float s[CHUNKS][8];
            float largest = 0.f;
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t x0 = k[b][c][0].pair(j), x1 = k[b][c][1].pair(j),
                                   x2 = k[b][c][2].pair(j), x3 = k[b][c][3].pair(j);
                    s[c][2 * j] = sum4(x0 & 0xffff, x1 & 0xffff, x2 & 0xffff, x3 & 0xffff);
                    s[c][2 * j + 1] = sum4(x0 >> 16, x1 >> 16, x2 >> 16, x3 >> 16);
                    largest = max3_abs(s[c][2 * j], s[c][2 * j + 1], largest);
                }
            // As whole numbers magnitudes keep their order, NaN above all.
            const uint32_t most =
                __reduce_max_sync(0xffffffffu, __float_as_uint(largest) & 0x7fffffffu);
            const bool fine = most != 0 && most < 0x7f800000u;
            const float inv = fine ? 127.f / __uint_as_float(most) : 0.f;
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) {
                const int e = c * 256 + lane * 8;
                if (e >= P.width) break;
                // Adding 1.5 * 2^23 rounds to the nearest whole number, whose low
                // byte is then the sum's.
                uint32_t y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y[j] = __float_as_uint(__fadd_rn(__fmul_rn(s[c][j], inv), 12582912.f));
                uint2 w;
                w.x = __byte_perm(__byte_perm(y[0], y[1], 0x0040), __byte_perm(y[2], y[3], 0x0040),
                                  0x5410);
                w.y = __byte_perm(__byte_perm(y[4], y[5], 0x0040), __byte_perm(y[6], y[7], 0x0040),
                                  0x5410);
                if (!fine) w = make_uint2(0, 0);
                *reinterpret_cast<uint2*>(P.index + block[b] * P.width + e) = w;
            }
            if (lane == 0)
                P.index_scale[block[b]] = fine ? __fmul_rn(__uint_as_float(most), unit) : 0.f;
        }
    }
}

template <bool E4M3>
void launch_index(const IndexParams& P, int grid, cudaStream_t stream) {
    if (P.width <= 256) index_kernel<E4M3, 1><<<grid, INDEX_THREADS, 0, stream>>>(P);
    else if (P.width <= 512) index_kernel<E4M3, 2><<<grid, INDEX_THREADS, 0, stream>>>(P);
    else index_kernel<E4M3, 4><<<grid, INDEX_THREADS, 0, stream>>>(P);
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
    if (bf16) write_kernel<DH, E4M3, true><<<grid, WRITE_THREADS, 0, stream>>>(P);
    else write_kernel<DH, E4M3, false><<<grid, WRITE_THREADS, 0, stream>>>(P);
}

}  // namespace cacheops

int cache_write_launch(const CacheRows& r, const gqa_cache_write_args& a, bool e4m3,
                       cudaStream_t stream) {
    using namespace cacheops;
    const DeviceInfo* di = device_info();
    if (!di) return GQA_ERR_CUDA;
    WriteParams P;
    P.rows = make_rows(r, di);
    const void* const x[3] = {a.q, a.k, a.v};
    const int64_t token_stride[3] = {a.q_token_stride, a.k_token_stride, a.v_token_stride};
    const int64_t head_stride[3] = {a.q_head_stride, a.k_head_stride, a.v_head_stride};
    for (int i = 0; i < 3; ++i) {
        P.x[i] = static_cast<const uint16_t*>(x[i]);
        P.token_stride[i] = token_stride[i];
        P.head_stride[i] = head_stride[i];
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
    P.nq = a.q ? a.Hq : 0;
    P.hkv = a.Hkv;
    // About as many warps as the device holds: few tokens share out their heads
    // (at most one for each head, or pair of heads at D = 128, that a warp takes
    // at once), many go several to a warp.
    const int heads = P.nq + 2 * P.hkv, at_once = 256 / a.D;
    const int warps = di->num_sms * WRITE_WARPS;
    int shares = (heads + at_once - 1) / at_once;
    const int full = (warps + r.tokens - 1) / r.tokens;
    if (shares > full) shares = full;
    P.heads_per_share = (heads + shares - 1) / shares;
    P.heads_per_share = (P.heads_per_share + at_once - 1) / at_once * at_once;
    shares = (heads + P.heads_per_share - 1) / P.heads_per_share;
    P.shares = make_fastdiv(shares);
    const int per = shares > 1 ? 1 : (r.tokens + warps - 1) / warps;
    P.tokens_per_warp = per < 32 ? per : 32;
    const long long parts = (r.tokens + P.tokens_per_warp - 1) / P.tokens_per_warp;
    const int grid = (int)((parts * shares + WRITE_THREADS / 32 - 1) / (WRITE_THREADS / 32));
    const bool bf16 = a.dtype == GQA_DTYPE_BF16;
    if (e4m3) {
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
    const int grid = (r.tokens + INDEX_THREADS - 1) / INDEX_THREADS;
    if (kscale) launch_index<true>(P, grid, stream);
    else launch_index<false>(P, grid, stream);
    return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace gqa

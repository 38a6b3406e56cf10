// cache_ops.cu -- the operators that fill and read back the paged cache: the
// cache write (per-head RMS norm, position rotation and the store of K and V,
// quantised or not), the cache read (dense K / V rows of cached tokens) and
// the block index (an int8 summary of every finished 4-token block).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <type_traits>

#include "cache_rows.cuh"
#include "fp4_rows.cuh"

namespace gqa {
namespace cacheops {

constexpr int THREADS = 256;
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
    FastDiv by_pairs;
    int tile;                    // tokens per CTA
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
// The largest magnitude; NaN if there is one.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float max4_abs(float a, float b, float c, float d) {
    return max3_abs(max3_abs(a, b, c), d, 0.f);
}
__device__ __forceinline__ float max4_abs(Pair a, Pair b) {
    const float2 x = unpack(a), y = unpack(b);
    return max4_abs(x.x, x.y, y.x, y.y);
}
// A block's scale and its reciprocal: {s, r}.
//
// A value's code is that of its true quotient with the scale: values and scales have
// few bits, so that many quotients lie half way between two codes, where the product
// with a reciprocal goes either way.  A division a value is most of the arithmetic,
// though (8000 rows: 26.4 us, against 22.2).  So the product with the rounded
// reciprocal is corrected by its remainder (Markstein's method): q0 = x r,
// q = q0 + (x - q0 s) r with two fused operations.  The remainder is exact, so the
// error is that of r times that of q0, 2^-47 of the quotient before q's own rounding:
// a half-way quotient comes out exact.  It needs every product finite: blocks with an
// infinity, a NaN or a magnitude from 2^100 on have r = 0, and divide.  (Products that
// underflow belong to quotients that round to zero.)
__device__ __forceinline__ float corrected_quotient(float x, float s, float r) {
    const float q = x * r;
    return fmaf(fmaf(-q, s, x), r, q);
}
__device__ __forceinline__ float2 block_scale(float most, uint32_t* code) {
    constexpr float kHuge = 0x1p100f;
    const float sixth =
        most < kHuge ? corrected_quotient(most, 6.f, 1.f / 6.f) : most / 6.f;
    *code = __nv_cvt_float_to_fp8(sixth, __NV_SATFINITE, __NV_E4M3);
    const __half_raw hr = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)*code, __NV_E4M3);
    const float s = __half2float(*reinterpret_cast<const __half*>(&hr));
    return make_float2(s, s > 0.f && most < kHuge ? __frcp_rn(s) : 0.f);
}
// Four values over their block's scale as E2M1 codes, the first in the lowest nibble:
// round to nearest even, +-6 beyond the range; zeros for a scale of zero or NaN.
__device__ __forceinline__ uint32_t to_e2m1x4(Pair a, Pair b, float2 sr) {
    const float s = sr.x;
    float2 x, y;
    if (sr.y > 0.f) {
        const Pair r = pack(sr.y, sr.y), m = pack(-s, -s);
        const Pair qa = mul2(a, r), qb = mul2(b, r);
        x = unpack(fma2(fma2(qa, m, a), r, qa));
        y = unpack(fma2(fma2(qb, m, b), r, qb));
    } else {
        if (!(s > 0.f)) return 0;
        x = unpack(a), y = unpack(b);
        x.x /= s, x.y /= s, y.x /= s, y.y /= s;
    }
    return __nv_cvt_float2_to_fp4x2(x, __NV_E2M1, cudaRoundNearest) |
           (uint32_t)__nv_cvt_float2_to_fp4x2(y, __NV_E2M1, cudaRoundNearest) << 8;
}

// cos and sin of position * frequency, as a fraction of a turn: frequency / (2 pi)
// as hi + lo, to 1.5 2^-47 of it, and the products' own rounding errors, whose
// fractions are taken before they are added, so that far positions keep their
// angle.  Then the hardware's approximations: within half a turn 2^-21.4 for the
// sine and 2^-21.2 for the cosine, and 2^-21.8 of the angle's product with 2 pi.
// With the sums' roundings (2^-25 of a turn; 5 2^-24 with a high part) the results
// hold to 2^-20 + |position * frequency| 2^-45, from position 2^24 on to 2^-18 and
// the same.
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

// A CTA takes up to four tokens and a share of their heads.  Groups of DH / 8
// lanes take one head of all its tokens at a time: the tokens' loads, sums,
// products and stores run side by side (one token's head after the other, each
// waiting for its own sum of squares, took 22 us for 8000 rows however they were
// shared out), the next head's loads are in flight meanwhile, and a head's
// weights serve all tokens.  The cos and sin of the tokens' pairs are computed
// once for all heads, in shared memory, while the first loads are on their way.
//
// y = x / sqrt(mean(x^2) + eps) * w and the rotation in 32 bits, two products
// an instruction; one rounding at the end (fp16 for q, the cache's type for K
// and V).  The root is rsqrtf, to 2 units in the last place of 32 bits; codes are
// those of the product with the scale's rounded reciprocal.
//
// 8000 rows of 6 + 1 + 1 heads of 256 into an E4M3 cache move 61 MB, 9.0 us at the
// copy rate, and take 16.9 us (a plain copy of the same buffers, 11.7): between
// the loads a head's chain of sum, shuffles and products is exposed, with 20
// warps an SM to cover it; 8 rows take 2.8 us, most of it the launch.  Into a 4-bit
// cache, 60 MB, 20.5 us: its blocks' largest magnitudes cross lanes as well.
//
// A lane holds two runs of four values: in the rotated part both members of
// four pairs, so no value crosses lanes.  Pairs (i, i + rot / 2): runs 4 l and
// rot / 2 + 4 l; pairs (2 i, 2 i + 1), and the values that do not turn: runs 8 l
// and 8 l + 4.
constexpr int UNIT = 4;                 // tokens of a unit
constexpr int WRITE_THREADS = 128;
constexpr int WRITE_CTAS = 5;           // resident on an SM
constexpr int MAX_ROT_PAIRS = 128;      // rotated pairs of a head (rot_dim <= 256)

// What the cache holds.
enum Cache { F16, E4M3, FP4 };

template <int DH, Cache KIND, bool BF16>
__global__ void __launch_bounds__(WRITE_THREADS, WRITE_CTAS) write_kernel(const WriteParams P) {
    constexpr int LANES = DH / 8;
    constexpr int GROUPS = WRITE_THREADS / LANES;
    __shared__ int s_starts[kRowsMaxBatch + 1];
    __shared__ int s_pos[UNIT];
    __shared__ long long s_cache[UNIT];    // element offset of the token, -1: none
    __shared__ __align__(16) float s_cos[UNIT][MAX_ROT_PAIRS];
    __shared__ __align__(16) float s_sin[UNIT][MAX_ROT_PAIRS];
    // FP4: the largest magnitude of every run of four values of a group's head.
    __shared__ __align__(16) float s_most[KIND == FP4 ? GROUPS : 1][UNIT][DH / 4];
    __shared__ float2 s_block[KIND == FP4 ? GROUPS : 1][UNIT][DH / 16];   // its blocks' scales
    const int t0 = blockIdx.x * P.tile;
    const int nt = min(P.tile, P.rows.tokens - t0);
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
    // The lanes of this group within the warp.
    const uint32_t mates = LANES == 32 ? 0xffffffffu : 0xffffu << (16 * (group & 1));
    const bool turns = lane < P.pairs / 4;
    const bool split = turns && !P.interleaved;
    const int run0 = split ? lane * 4 : lane * 8;
    const int run1 = split ? P.pairs + lane * 4 : lane * 8 + 4;
    const int k0 = P.nq, v0 = k0 + P.hkv, heads = v0 + P.hkv;   // heads: q, then K, then V
    // This group's heads: neighbours, which share their weights.  For a 4-bit cache every
    // groups-th one: K's and V's heads cost more than q's there, and neighbours of them
    // would fall to the same groups (8000 rows: 20.5 us, 22.2 with neighbours).
    const int groups = gridDim.y * GROUPS, per = (heads + groups - 1) / groups;
    const int my_group = blockIdx.y * GROUPS + group;
    const int head_step = KIND == FP4 ? groups : 1;
    int head = KIND == FP4 ? my_group : my_group * per;
    const int head_end = KIND == FP4 ? heads : min(head + per, heads);

    struct Place {
        int kind, in_kind;
    };
    auto place = [&](int h) {
        Place p;
        p.kind = h < k0 ? 0 : h < v0 ? 1 : 2;
        p.in_kind = h - (p.kind == 0 ? 0 : p.kind == 1 ? k0 : v0);
        return p;
    };
    auto load = [&](const Place& p, uint2 (&raw)[UNIT][2]) {
        const long long step = P.token_stride[p.kind];
        const uint16_t* y = P.x[p.kind] + t0 * step + p.in_kind * P.head_stride[p.kind];
#pragma unroll
        for (int i = 0; i < UNIT; ++i) {
            if (i >= nt) break;
            raw[i][0] = *reinterpret_cast<const uint2*>(y + run0);
            raw[i][1] = *reinterpret_cast<const uint2*>(y + run1);
            y += step;
        }
    };
    uint2 next[UNIT][2];
    Place at_next = place(head);
    if (head < head_end) load(at_next, next);

    if (P.rows.row_starts) {
        load_row_starts(P.rows, s_starts);
        __syncthreads();
    }
    if (threadIdx.x < nt) {
        long long slot;
        locate_row(P.rows, s_starts, t0 + threadIdx.x, &s_pos[threadIdx.x], &slot);
        if (KIND == FP4) {
            // (the row of the first head, the others a page of rows apart)
            const int lp = P.rows.log2_page;
            s_cache[threadIdx.x] =
                slot < 0 ? -1 : ((slot >> lp) * P.hkv << lp) + (slot & ((1 << lp) - 1));
        } else {
            s_cache[threadIdx.x] = slot < 0 ? -1 : slot * (P.hkv * DH);
        }
    }
    const float kinv = KIND != F16 ? 1.f / *P.kscale : 1.f;
    const float vinv = KIND != F16 ? 1.f / *P.vscale : 1.f;
    __syncthreads();
    if (P.pairs) {
        for (int i = threadIdx.x; i < nt * P.pairs; i += WRITE_THREADS) {
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

    int weights_of = -1;     // the kind w belongs to
    Pair w[4];
    for (; head < head_end; head += head_step) {
        const Place p = at_next;
        Pair x[UNIT][4];
#pragma unroll
        for (int i = 0; i < UNIT; ++i) {
            x[i][0] = unpack16<BF16>(next[i][0].x);
            x[i][1] = unpack16<BF16>(next[i][0].y);
            x[i][2] = unpack16<BF16>(next[i][1].x);
            x[i][3] = unpack16<BF16>(next[i][1].y);
        }
        if (head + head_step < head_end) {
            at_next = place(head + head_step);
            load(at_next, next);
        }
        const uint16_t* weight = p.kind < 2 ? P.weight[p.kind] : nullptr;
        if (weight) {
            if (weights_of != p.kind) {
                const uint2 a = *reinterpret_cast<const uint2*>(weight + run0);
                const uint2 b = *reinterpret_cast<const uint2*>(weight + run1);
                w[0] = unpack16<BF16>(a.x);
                w[1] = unpack16<BF16>(a.y);
                w[2] = unpack16<BF16>(b.x);
                w[3] = unpack16<BF16>(b.y);
                weights_of = p.kind;
            }
            float ss[UNIT];
#pragma unroll
            for (int i = 0; i < UNIT; ++i) {
                Pair sq = mul2(x[i][0], x[i][0]);
#pragma unroll
                for (int k = 1; k < 4; ++k) sq = fma2(x[i][k], x[i][k], sq);
                const float2 halves = unpack(sq);
                ss[i] = halves.x + halves.y;
            }
#pragma unroll
            for (int o = LANES / 2; o; o >>= 1)
#pragma unroll
                for (int i = 0; i < UNIT; ++i) ss[i] += __shfl_xor_sync(mates, ss[i], o);
#pragma unroll
            for (int i = 0; i < UNIT; ++i) {
                const float r = rsqrtf(ss[i] * (1.f / DH) + P.eps);
                const Pair rr = pack(r, r);
#pragma unroll
                for (int k = 0; k < 4; ++k) x[i][k] = mul2(mul2(x[i][k], rr), w[k]);
            }
        }
        if (turns && p.kind < 2) {
#pragma unroll
            for (int i = 0; i < UNIT; ++i) {
                // (past the last token: whatever is there, for values that go nowhere)
                const float4 c4 = *reinterpret_cast<const float4*>(&s_cos[i][lane * 4]);
                const float4 s4 = *reinterpret_cast<const float4*>(&s_sin[i][lane * 4]);
                if (split) {
                    const Pair c[2] = {pack(c4.x, c4.y), pack(c4.z, c4.w)};
                    const Pair s[2] = {pack(s4.x, s4.y), pack(s4.z, s4.w)};
                    const Pair m[2] = {pack(-s4.x, -s4.y), pack(-s4.z, -s4.w)};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const Pair a = x[i][k], b = x[i][2 + k];
                        x[i][k] = fma2(b, m[k], mul2(a, c[k]));
                        x[i][2 + k] = fma2(a, s[k], mul2(b, c[k]));
                    }
                } else {
                    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 ab = unpack(x[i][k]);
                        x[i][k] = pack(ab.x * c[k] - ab.y * s[k], ab.y * c[k] + ab.x * s[k]);
                    }
                }
            }
        }
        if (p.kind == 0) {
            __half* to = P.q_out + ((long long)t0 * P.nq + p.in_kind) * DH;
#pragma unroll
            for (int i = 0; i < UNIT; ++i) {
                if (i < nt && s_pos[i] >= 0) {
                    *reinterpret_cast<uint2*>(to + run0) =
                        make_uint2(to_half2(x[i][0]), to_half2(x[i][1]));
                    *reinterpret_cast<uint2*>(to + run1) =
                        make_uint2(to_half2(x[i][2]), to_half2(x[i][3]));
                }
                to += P.nq * DH;
            }
            continue;
        }
        void* const cache = p.kind == 1 ? P.kcache : P.vcache;
        const float f = p.kind == 1 ? kinv : vinv;
        const Pair ff = pack(f, f);
        if constexpr (KIND == FP4) {
            // A block of 16 is four runs of up to four lanes, which meet in shared memory;
            // each lane takes the scales of two neighbouring blocks of one token.
            auto row_of = [&](int i) {
                return static_cast<uint8_t*>(cache) +
                       (s_cache[i] + ((long long)p.in_kind << P.rows.log2_page)) *
                           fp4::row_bytes(DH);
            };
#pragma unroll
            for (int i = 0; i < UNIT; ++i) {
#pragma unroll
                for (int k = 0; k < 4; ++k) x[i][k] = mul2(x[i][k], ff);
                s_most[group][i][run0 / 4] = max4_abs(x[i][0], x[i][1]);
                s_most[group][i][run1 / 4] = max4_abs(x[i][2], x[i][3]);
            }
            __syncwarp(mates);
            {
                static_assert(UNIT * DH / 16 == 2 * LANES, "two blocks a lane");
                const int i = lane / (LANES / UNIT), block = lane % (LANES / UNIT) * 2;
                const float4* m = reinterpret_cast<const float4*>(&s_most[group][i][block * 4]);
                uint32_t codes[2];
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    s_block[group][i][block + k] =
                        block_scale(max4_abs(m[k].x, m[k].y, m[k].z, m[k].w), &codes[k]);
                if (i < nt && s_cache[i] >= 0)
                    *reinterpret_cast<uint16_t*>(row_of(i) + DH / 2 + block) =
                        (uint16_t)(codes[0] | codes[1] << 8);
            }
            __syncwarp(mates);
#pragma unroll
            for (int i = 0; i < UNIT; ++i) {
                if (i >= nt || s_cache[i] < 0) continue;
                uint8_t* row = row_of(i);
                *reinterpret_cast<uint16_t*>(row + run0 / 2) =
                    (uint16_t)to_e2m1x4(x[i][0], x[i][1], s_block[group][i][run0 / 16]);
                *reinterpret_cast<uint16_t*>(row + run1 / 2) =
                    (uint16_t)to_e2m1x4(x[i][2], x[i][3], s_block[group][i][run1 / 16]);
            }
            continue;
        }
#pragma unroll
        for (int i = 0; i < UNIT; ++i) {
            if (i >= nt || s_cache[i] < 0) continue;
            const long long at = s_cache[i] + p.in_kind * DH;
            if (KIND == E4M3) {
                uint8_t* to = static_cast<uint8_t*>(cache) + at;
                *reinterpret_cast<uint32_t*>(to + run0) =
                    to_e4m3x2(mul2(x[i][0], ff)) | to_e4m3x2(mul2(x[i][1], ff)) << 16;
                *reinterpret_cast<uint32_t*>(to + run1) =
                    to_e4m3x2(mul2(x[i][2], ff)) | to_e4m3x2(mul2(x[i][3], ff)) << 16;
            } else {
                __half* to = static_cast<__half*>(cache) + at;
                *reinterpret_cast<uint2*>(to + run0) =
                    make_uint2(to_half2(x[i][0]), to_half2(x[i][1]));
                *reinterpret_cast<uint2*>(to + run1) =
                    make_uint2(to_half2(x[i][2]), to_half2(x[i][3]));
            }
        }
    }
}

struct ReadParams {
    RowMap rows;
    const uint8_t* cache[2];   // K, V
    const float* scale[2];     // E4M3 dequantisation scales (null: rows as they are)
    uint8_t* out[2];
    int row_bytes;             // cached bytes of one token of K (or V); unused by read_fp4_kernel
    FastDiv chunks;            // pieces of one token's K (or V)
    int tile;                  // tokens per CTA
};

constexpr int MAX_READ_TILE = 64;
constexpr int READ_AHEAD = 4;

// Dense rows of cached tokens: DEQUANT reads 8 codes and writes 8 fp16 values
// a thread, the other form copies 16 bytes.  READ_AHEAD pieces of K and of V
// each are in flight together.  Bound by the bytes: 261888 rows of 256 E4M3 codes
// to fp16 move 402 MB in 62.0 us, 6.5 TB/s, 0.95 of a copy (71.5 us with one piece
// at a time).
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

// 32 bytes, in one store where the address allows it.  (Two of 16 leave every other 16
// bytes of a warp's lines to the second: 261888 rows 71.9 us, against 54.2.)
__device__ __forceinline__ void store32(uint8_t* to, const uint32_t (&h)[8], bool aligned) {
    if (aligned) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to),
                     "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]), "r"(h[4]), "r"(h[5]),
                     "r"(h[6]), "r"(h[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(to)[0] = make_uint4(h[0], h[1], h[2], h[3]);
        reinterpret_cast<uint4*>(to)[1] = make_uint4(h[4], h[5], h[6], h[7]);
    }
}

// Dense fp16 rows of a 4-bit cache: a block of 16 codes a thread, with its scale.  code
// * scale is exact, its product with the tensor's scale rounded to 32 bits, then to
// fp16.  FP4_AHEAD blocks of K and of V each are in flight together.  Bound by the
// bytes, mostly those written: 261888 rows of 256 move 344 MB in 54.2 us, 6.3 TB/s,
// 0.95 of a copy (58.2 us with half a block a thread and the same bytes in flight, 57.7
// with four blocks ahead, 54.5 with one).
constexpr int FP4_AHEAD = 2;
template <int DH>
__global__ void __launch_bounds__(THREADS) read_fp4_kernel(const ReadParams P) {
    constexpr int A_HEAD = DH / 16;     // pieces of one head's row
    __shared__ int s_starts[kRowsMaxBatch + 1];
    __shared__ int s_pos[MAX_READ_TILE];
    __shared__ long long s_row[MAX_READ_TILE];   // the row of the first head, -1: none
    const int t0 = blockIdx.x * P.tile;
    const int nt = min(P.tile, P.rows.tokens - t0);
    if (P.rows.row_starts) {
        load_row_starts(P.rows, s_starts);
        __syncthreads();
    }
    if (threadIdx.x < nt) {
        long long slot;
        locate_row(P.rows, s_starts, t0 + threadIdx.x, &s_pos[threadIdx.x], &slot);
        const int lp = P.rows.log2_page, heads = P.chunks.d / A_HEAD;
        s_row[threadIdx.x] = slot < 0 ? -1 : ((slot >> lp) * heads << lp) + (slot & ((1 << lp) - 1));
    }
    const float scale[2] = {*P.scale[0], *P.scale[1]};
    const bool aligned = ((uintptr_t)P.out[0] | (uintptr_t)P.out[1]) % 32 == 0;
    __syncthreads();
    const int n = nt * P.chunks.d;
    for (int i0 = threadIdx.x; i0 < n; i0 += FP4_AHEAD * THREADS) {
        uint2 in[FP4_AHEAD][2];
        uint8_t unit[FP4_AHEAD][2];
#pragma unroll
        for (int u = 0; u < FP4_AHEAD; ++u) {
            const int i = i0 + u * THREADS;
            in[u][0] = in[u][1] = make_uint2(0, 0), unit[u][0] = unit[u][1] = 0;
            if (i >= n) continue;
            const int t = P.chunks.div(i), piece = i - t * P.chunks.d;
            if (s_row[t] < 0) continue;
            const int head = piece / A_HEAD, c = piece % A_HEAD;
            const long long at =
                (s_row[t] + ((long long)head << P.rows.log2_page)) * fp4::row_bytes(DH);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                in[u][kv] = *reinterpret_cast<const uint2*>(P.cache[kv] + at + c * 8);
                unit[u][kv] = P.cache[kv][at + DH / 2 + c];
            }
        }
#pragma unroll
        for (int u = 0; u < FP4_AHEAD; ++u) {
            const int i = i0 + u * THREADS;
            if (i >= n) break;
            if (s_pos[P.chunks.div(i)] < 0) continue;
            const long long to = ((long long)t0 * P.chunks.d + i) * 32;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                uint32_t h[8];
                fp4::decode8(in[u][kv].x, h);
                fp4::decode8(in[u][kv].y, h + 4);
                const uint32_t s = fp4::scales2(unit[u][kv] * 0x101u);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t e = fp4::mul2(h[k], s);
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&e));
                    h[k] = pack_half2(f.x * scale[kv], f.y * scale[kv]);
                }
                store32(P.out[kv] + to, h, aligned);
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
    int rows_per_warp;
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
// (a + b) + (c + d) of four fp16 values in 32 bits; of E4M3 values, whose sums are
// exact in any order (20 bits from 2^-9 up), one after the other.
template <bool E4M3>
__device__ __forceinline__ float sum4(uint16_t a, uint16_t b, uint16_t c, uint16_t d) {
    if (E4M3) return add_half(d, add_half(c, add_half(b, __half2float(__ushort_as_half(a)))));
    return __fadd_rn(add_half(b, __half2float(__ushort_as_half(a))),
                     add_half(d, __half2float(__ushort_as_half(c))));
}

// Summaries of the 4-token blocks whose last token is a row of this step.  A
// warp takes rows_per_warp rows, a lane each to find the blocks they finish,
// then block after block: 8 values a lane of each 256 (CHUNKS of them), the keys
// of TOGETHER blocks in flight together.  The sums, the largest magnitude and the
// codes follow fixed 32-bit operations, so the codes are the same wherever and
// in whatever batch a block is summarised.
//
// Bound by the keys' bytes: 261888 E4M3 rows of 256 are 84 MB with what is
// written, 12.4 us at the copy rate, and take 16.2 us (5.2 TB/s; 2 or 8 blocks
// together, 16 rows a warp or other CTAs are no faster).
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
    // (unsigned: the last CTA's rows may pass 2^31)
    const uint32_t row =
        (blockIdx.x * (INDEX_THREADS / 32) + threadIdx.x / 32) * P.rows_per_warp + lane;
    int pos = -1;
    long long slot = -1;
    if (lane < P.rows_per_warp && row < (uint32_t)P.rows.tokens)
        locate_row(P.rows, s_starts, (int)row, &pos, &slot);
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
                    s[c][2 * j] = sum4<E4M3>(x0 & 0xffff, x1 & 0xffff, x2 & 0xffff, x3 & 0xffff);
                    s[c][2 * j + 1] = sum4<E4M3>(x0 >> 16, x1 >> 16, x2 >> 16, x3 >> 16);
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

template <Cache KIND>
void launch_write(const WriteParams& P, int D, bool bf16, dim3 grid, cudaStream_t stream) {
    if (D == 256) {
        if (bf16) write_kernel<256, KIND, true><<<grid, WRITE_THREADS, 0, stream>>>(P);
        else write_kernel<256, KIND, false><<<grid, WRITE_THREADS, 0, stream>>>(P);
    } else {
        if (bf16) write_kernel<128, KIND, true><<<grid, WRITE_THREADS, 0, stream>>>(P);
        else write_kernel<128, KIND, false><<<grid, WRITE_THREADS, 0, stream>>>(P);
    }
}

}  // namespace cacheops

int cache_write_launch(const CacheRows& r, const gqa_cache_write_args& a, int cache_bits,
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
    P.by_pairs = make_fastdiv(P.pairs > 0 ? P.pairs : 1);
    // Few tokens go one to a CTA, and while all CTAs are resident at once the heads
    // are shared out among more of them (6 + 1 + 1 heads of 256: 400 rows 3.5 us,
    // 4.0 with a unit's heads in one CTA, 1500 rows 4.7 and 5.1; 16 + 4 + 4 heads:
    // 400 rows 4.4 and 7.5).  Of many tokens a CTA takes all heads of its unit (8000
    // rows: 2000 CTAs, 760 of them at once).
    const int heads = P.nq + 2 * P.hkv, groups = WRITE_THREADS * 8 / a.D;
    const long long resident = (long long)di->num_sms * WRITE_CTAS;
    P.tile = (long long)r.tokens * heads <= resident * groups ? 1 : UNIT;
    const int tiles = (r.tokens + P.tile - 1) / P.tile;
    long long shares = (heads + groups - 1) / groups;
    if (shares > resident / tiles) shares = resident / tiles > 0 ? resident / tiles : 1;
    const dim3 grid(tiles, (unsigned)shares);
    const bool bf16 = a.dtype == GQA_DTYPE_BF16;
    if (cache_bits == 4) launch_write<FP4>(P, a.D, bf16, grid, stream);
    else if (cache_bits == 8) launch_write<E4M3>(P, a.D, bf16, grid, stream);
    else launch_write<F16>(P, a.D, bf16, grid, stream);
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
    // Few rows are shared out among more CTAs (333 rows: 2.0 us with 8 a CTA, 2.3 with
    // 32); many share the work of finding their pages (261888 rows: 62 us with 32,
    // 70 with 8).
    P.tile = r.tokens <= 2048 ? 8 : 32;
    const int grid = (r.tokens + P.tile - 1) / P.tile;
    if (kscale) read_kernel<true><<<grid, THREADS, 0, stream>>>(P);
    else read_kernel<false><<<grid, THREADS, 0, stream>>>(P);
    return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

int cache_read_fp4_launch(const CacheRows& r, const void* kcache, const void* vcache,
                          const float* kscale, const float* vscale, int Hkv, int D, void* k_out,
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
    P.chunks = make_fastdiv(Hkv * D / 16);
    P.tile = r.tokens <= 2048 ? 8 : 32;
    const int grid = (r.tokens - 1) / P.tile + 1;
    if (D == 256) read_fp4_kernel<256><<<grid, THREADS, 0, stream>>>(P);
    else read_fp4_kernel<128><<<grid, THREADS, 0, stream>>>(P);
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
    // Few rows are shared out among more warps: 64 rows 2.1 us instead of 3.2, 8000
    // rows 2.6 instead of 3.6; many make as many warps anyway.
    P.rows_per_warp = r.tokens <= di->num_sms * 128 ? 8 : 32;
    const int a_cta = INDEX_THREADS / 32 * P.rows_per_warp;
    const int grid = (r.tokens - 1) / a_cta + 1;
    if (kscale) launch_index<true>(P, grid, stream);
    else launch_index<false>(P, grid, stream);
    return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace gqa

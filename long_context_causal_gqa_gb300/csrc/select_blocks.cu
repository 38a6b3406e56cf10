// select_blocks.cu -- the 4-token blocks each query row attends, by a cheap
// score: the dot of the row's summed queries and the block's summed keys, both
// as int8 codes.
//
// The dot is a whole number below 2^24 in magnitude (127^2 * 1024 at most), so
// it is exact in any order of the sum; the score is that number times the
// block's scale, one 32-bit rounding.  Equal scores go to the lower block id.
// The selection is therefore a function of the inputs alone.
#include <cuda_fp16.h>

#include "internal.h"
#include "sm100.cuh"

namespace gqa {
namespace select {

// ------------------------------------------------------------ query codes
// codes[row, g * D + d] = rint(S * 127 / max |S|), S = sum of q over the query
// heads of KV head g.  fp16 values are whole multiples of 2^-24 below 2^41 of
// them, so the sums are exact as 64-bit whole numbers; S is rounded to 32 bits
// once.  A row with an infinity or NaN gets codes of zero.
__global__ void __launch_bounds__(256) query_codes_kernel(const __half* __restrict__ q, int rows,
                                                          int Hq, int D, int group, int width,
                                                          int8_t* __restrict__ codes) {
    const int row = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x % 32;
    if (row >= rows) return;
    float s[8][4];
    float most = 0.f;
    bool fine = true;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        if (c * 128 >= width) break;
        const int g = c * 128 / D;
        const __half* src = q + ((long long)row * Hq + g * group) * D + (c * 128 - g * D) + lane * 4;
        long long sum[4] = {0, 0, 0, 0};
        for (int h = 0; h < group; ++h) {
            const uint2 u = *reinterpret_cast<const uint2*>(src + (long long)h * D);
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
        if (c * 128 >= width) break;
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int code =
                fine ? (int)rintf(__fmul_rn(s[c][j] * (1.f / 16777216.f), inv)) : 0;
            w |= (uint32_t)(code & 0xff) << (8 * j);
        }
        *reinterpret_cast<uint32_t*>(codes + (long long)row * width + c * 128 + lane * 4) = w;
    }
}

// ------------------------------------------------------------ scores
struct ScoreParams {
    const int8_t* codes;         // query codes of the launch's first row
    const int8_t* index;
    const float* index_scale;
    const int32_t* table;
    int num_pages;
    int log2_ppb;                // log2 of the blocks of a page
    int n_blocks;
    int rows;
    int width;
    float* scores;               // [rows, stride]
    long long stride;
    unsigned* err;
};

// Physical block of logical block b; a table entry outside the cache reads
// page 0 (flagged), as the attention kernels do.
__device__ __forceinline__ long long physical_block(const ScoreParams& P, int b) {
    int id = P.table[b >> P.log2_ppb];
    if (id < 0 || id >= P.num_pages) {
        atomicOr(P.err, kErrBadPageId);
        id = 0;
    }
    return ((long long)id << P.log2_ppb) + (b & ((1 << P.log2_ppb) - 1));
}

constexpr int SMALL_ROWS = 8;

// Few rows: eight lanes read one block's codes (16 bytes at a time) and take
// its dots with up to SMALL_ROWS rows.
__global__ void __launch_bounds__(256) score_small_kernel(const ScoreParams P) {
    __shared__ __align__(16) int8_t s_q[SMALL_ROWS][kMaxIndexWidth];
    const int r0 = blockIdx.y * SMALL_ROWS;
    const int nr = min(SMALL_ROWS, P.rows - r0);
    for (int i = threadIdx.x; i < SMALL_ROWS * P.width / 16; i += 256) {
        const int r = i / (P.width / 16), c = i - r * (P.width / 16);
        reinterpret_cast<uint4*>(s_q[r])[c] =
            r < nr ? *reinterpret_cast<const uint4*>(P.codes + (long long)(r0 + r) * P.width +
                                                     c * 16)
                   : make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    const int lane = threadIdx.x % 8;
    for (int b0 = blockIdx.x * 32; b0 < P.n_blocks; b0 += gridDim.x * 32) {
        const int b = b0 + threadIdx.x / 8;
        const bool live = b < P.n_blocks;
        const long long block = physical_block(P, live ? b : b0);
        const uint4* src = reinterpret_cast<const uint4*>(P.index + block * P.width);
        int dot[SMALL_ROWS];
#pragma unroll
        for (int r = 0; r < SMALL_ROWS; ++r) dot[r] = 0;
        for (int c = lane; c < P.width / 16; c += 8) {
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
        const float scale = P.index_scale[block];
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
    const float* scores;
    long long stride;
    int row0;                    // first row of this launch in the call
    int pos0;                    // position of that row
    int max_sel, n_first, n_last;
    int32_t* sel_idx;            // the call's
    int32_t* sel_cnt;
};

// A float's order as whole numbers; NaN below everything.  Adding zero makes
// the two zeros one.
__device__ __forceinline__ uint32_t ordered(float f) {
    if (f != f) return 0;
    const uint32_t u = __float_as_uint(f + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int PICK_THREADS = 256;

// One CTA a row.  The key of the k-th best block is found eight bits at a time
// (counts of the keys that share the bits found so far); then one pass over
// the blocks in order writes those above it and the first of those equal to it.
__global__ void __launch_bounds__(PICK_THREADS) pick_kernel(const PickParams P) {
    __shared__ int s_hist[256];
    __shared__ uint32_t s_prefix;
    __shared__ int s_need;
    __shared__ int s_above[PICK_THREADS / 32], s_equal[PICK_THREADS / 32];
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const float* scores = P.scores + row * P.stride;
    const int own = (P.pos0 + row) >> 2;       // the row's own block
    const int n_vis = own + 1;
    const int take = min(P.max_sel, n_vis);
    int32_t* out = P.sel_idx + (long long)(P.row0 + row) * P.max_sel;
    if (tid == 0) P.sel_cnt[P.row0 + row] = take;
    for (int i = take + tid; i < P.max_sel; i += PICK_THREADS) out[i] = -1;
    if (take == n_vis) {
        for (int i = tid; i < take; i += PICK_THREADS) out[i] = i;
        return;
    }
    // take = max_sel < n_vis: at least one block is left out, so first and last
    // blocks do not meet.
    const int lo = P.n_first, hi = n_vis - P.n_last;   // scored blocks
    int need = take - P.n_first - P.n_last;
    uint32_t prefix = 0;
    if (need > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            s_hist[tid] = 0;
            __syncthreads();
            for (int b = lo + tid; b < hi; b += PICK_THREADS) {
                const uint32_t k = ordered(scores[b]);
                if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
                    atomicAdd(&s_hist[(k >> shift) & 255], 1);
            }
            __syncthreads();
            if (tid == 0) {
                int left = need, d = 255;
                while (d > 0 && s_hist[d] < left) left -= s_hist[d--];
                s_need = left;
                s_prefix = prefix | ((uint32_t)d << shift);
            }
            __syncthreads();
            prefix = s_prefix;
            need = s_need;
        }
    } else {
        prefix = 0xffffffffu;
    }
    // need = how many of the blocks with key == prefix are taken (lowest ids).
    int n_above = 0, n_equal = 0;   // so far, in blocks below b0
    for (int b0 = 0; b0 < n_vis; b0 += PICK_THREADS) {
        const int b = b0 + tid;
        bool above = false, equal = false;
        if (b < n_vis) {
            if (b < lo || b >= hi) above = true;
            else {
                const uint32_t k = ordered(scores[b]);
                above = k > prefix;
                equal = k == prefix && need > 0;
            }
        }
        const uint32_t ma = __ballot_sync(0xffffffffu, above);
        const uint32_t me = __ballot_sync(0xffffffffu, equal);
        if (lane == 0) {
            s_above[warp] = __popc(ma);
            s_equal[warp] = __popc(me);
        }
        __syncthreads();
        int a = n_above, e = n_equal, ta = 0, te = 0;
        for (int w = 0; w < PICK_THREADS / 32; ++w) {
            if (w < warp) {
                a += s_above[w];
                e += s_equal[w];
            }
            ta += s_above[w];
            te += s_equal[w];
        }
        const uint32_t below = (1u << lane) - 1;
        a += __popc(ma & below);
        e += __popc(me & below);
        if (above || (equal && e < need)) out[a + min(e, need)] = b;
        n_above += ta;
        n_equal += te;
        __syncthreads();
    }
}

// Rows whose scores are held at once: their scores take at most 64 MB (which
// stays in L2), at least one row.
int chunk_rows(int rows, int n_blocks) {
    const long long per_row = (long long)((n_blocks + 3) / 4 * 4) * 4;
    long long n = (64ll << 20) / per_row;
    n = n < 1 ? 1 : n;
    return n < rows ? (int)n : rows;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace select

size_t select_blocks_workspace_bytes(int rows, int ctx_len, int width) {
    using namespace select;
    const int n_blocks = (ctx_len - 1) / 4 + 1;
    const size_t stride = (size_t)(n_blocks + 3) / 4 * 4;
    return kWorkspaceCounterBytes + round256((size_t)rows * width) +
           round256((size_t)chunk_rows(rows, n_blocks) * stride * 4);
}

int select_blocks_launch(const void* q, const int8_t* index, const float* index_scale,
                         const int32_t* block_table, int num_pages, int page, int ctx_len,
                         int rows, int Hq, int Hkv, int D, int max_sel, int n_first, int n_last,
                         int32_t* sel_idx, int32_t* sel_cnt, cudaStream_t stream) {
    using namespace select;
    const DeviceInfo* di = device_info();
    if (!di) return GQA_ERR_CUDA;
    const int width = Hkv * D;
    void* ws;
    size_t ws_bytes;
    current_workspace(&ws, &ws_bytes);
    if (!ws || ws_bytes < select_blocks_workspace_bytes(rows, ctx_len, width))
        return GQA_ERR_WORKSPACE;
    uint8_t* w = static_cast<uint8_t*>(ws) + kWorkspaceCounterBytes;
    int8_t* codes = reinterpret_cast<int8_t*>(w);
    float* scores = reinterpret_cast<float*>(w + round256((size_t)rows * width));
    const int n_blocks = (ctx_len - 1) / 4 + 1;
    const int chunk = chunk_rows(rows, n_blocks);
    query_codes_kernel<<<(rows + 7) / 8, 256, 0, stream>>>(static_cast<const __half*>(q), rows,
                                                           Hq, D, Hq / Hkv, width, codes);
    for (int r0 = 0; r0 < rows; r0 += chunk) {
        const int n = rows - r0 < chunk ? rows - r0 : chunk;
        ScoreParams S;
        S.codes = codes + (size_t)r0 * width;
        S.index = index;
        S.index_scale = index_scale;
        S.table = block_table;
        S.num_pages = num_pages;
        S.log2_ppb = __builtin_ctz((unsigned)page) - 2;
        S.n_blocks = n_blocks;
        S.rows = n;
        S.width = width;
        S.scores = scores;
        S.stride = (n_blocks + 3) / 4 * 4;
        S.err = di->err_word;
        const int tiles = (n_blocks + 31) / 32;
        const int cap = di->num_sms * 8;
        const dim3 grid(tiles < cap ? tiles : cap, (n + SMALL_ROWS - 1) / SMALL_ROWS);
        score_small_kernel<<<grid, 256, 0, stream>>>(S);
        PickParams K;
        K.scores = scores;
        K.stride = S.stride;
        K.row0 = r0;
        K.pos0 = ctx_len - rows + r0;
        K.max_sel = max_sel;
        K.n_first = n_first;
        K.n_last = n_last;
        K.sel_idx = sel_idx;
        K.sel_cnt = sel_cnt;
        pick_kernel<<<n, PICK_THREADS, 0, stream>>>(K);
    }
    return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace gqa

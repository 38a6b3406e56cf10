// fp4_rows.cuh -- the rows of the 4-bit paged cache: E2M1 codes, one E4M3 scale
// for every 16 of them, one fp32 scale for the tensor.
//
// A token's row for one KV head is D / 2 bytes of codes (value 2 i in the low
// nibble of byte i) and D / 16 scales behind them: 9 D / 16 bytes.  The cache is
// [num_pages, Hkv, page, 9 D / 16], heads in front of tokens: a row is 144 or 72
// bytes, which at Hkv rows apart could not be copied in 16-byte pieces, while a
// page of one head is one contiguous run of them for every D and page.  Rows 36
// (18) words apart also spread a fragment's loads over the banks.
//
// A value is e2m1(code) * e4m3(scale) * tensor scale.  The first product has at
// most 2 + 4 significant bits between 2^-10 and 2688, so it is exact in fp16: the
// attention's operands are the cached values themselves, in units of the tensor's
// scale.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace gqa {
namespace fp4 {

// Bytes of one token's row of one head.
__host__ __device__ constexpr int row_bytes(int d) { return d / 2 + d / 16; }

// Eight codes (a word) as fp16 pairs: r[i] holds the two nibbles of byte i, the
// low one in the low half.
__device__ __forceinline__ void decode8(uint32_t w, uint32_t* r) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}

// Two E4M3 scales (low 16 bits) as fp16.
__device__ __forceinline__ uint32_t scales2(uint32_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
    return r;
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&a),
                              *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace fp4
}  // namespace gqa

// block_scale.cuh -- the number format of an int8 cache: a value is code * 2^e, code in [-127, 127], e one exponent
// for each block of tokens and kv head, kept as the byte e + 127.
//
// e stays where code * 2^e is a number of the 16-bit type that the cache goes with (127 2^121 is below bf16's largest
// number and 127 2^9 below fp16's; 2^-126 is bf16's smallest normal number and 2^-24 fp16's smallest at all), so
// widening rounds nothing.  A byte outside is read as the nearest one inside: whatever lies in an exponent that nobody has
// written, the value of a code is finite.  (-128 is no code; beside the largest exponent it would be infinite.)
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace dspark {

template <bool BF16>
struct ExpRange {
    static constexpr int kLo = BF16 ? -126 : -24, kHi = BF16 ? 121 : 9;
};

// 2^e as fp32, e in [-126, 127].
__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

template <bool BF16>
__device__ __forceinline__ int exponent_of(uint32_t byte) {
    return min(max((int)byte - 127, ExpRange<BF16>::kLo), ExpRange<BF16>::kHi);
}

// Where the exponents of an int8 cache lie: strides in bytes, shift = log2 of a block's tokens.
struct BlockExp {
    const unsigned char* k;
    const unsigned char* v;
    long long page, block, head;
    int shift;
};

// The pools and exponents of an int8 cache in 32-bit steps: codes in units that all three strides are multiples of,
// exponents in bytes (a stride that meets 0 alone, of a pool's only page or head, may be cut off).
struct Steps32 {
    uint32_t unit, page, token, head;
    uint32_t e_page, e_block, e_head;
};

// The four codes of a word as fp32: byte + 128 beside the exponent of 2^23 is 2^23 + 128 + code.
__device__ __forceinline__ void widen4(uint32_t w, float (&f)[4]) {
    const uint32_t u = w ^ 0x80808080u;
    f[0] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440)) - 8388736.f;
    f[1] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441)) - 8388736.f;
    f[2] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7442)) - 8388736.f;
    f[3] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7443)) - 8388736.f;
}

}  // namespace dspark

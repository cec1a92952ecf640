// tb_fp4.h -- elements held in 4 bits on the device, as tb_serve.h lays them out.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tb_serve.h"

namespace tbk {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// The i-th byte of x as what a block's elements are multiplied by.
__device__ __forceinline__ float power_of(uint32_t x, uint32_t i) {
    return __uint_as_float((x >> (8 * i) & 0xff) << 23);
}

// Byte I of x, two elements times `power`, as elements of T.  The conversion is the hardware's, exact here.
template <typename T, int I>
__device__ __forceinline__ uint32_t two_of(uint32_t x, float power) {
    if constexpr (sizeof(T) == 2 && __is_same(T, __bf16))
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, power, I));
    else
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(x, power, I));
}
template <typename T>
__device__ __forceinline__ u32x4 eight_of(uint32_t x, float power) {
    return (u32x4){two_of<T, 0>(x, power), two_of<T, 1>(x, power), two_of<T, 2>(x, power), two_of<T, 3>(x, power)};
}
template <typename T>
__device__ __forceinline__ uint32_t two_at(uint32_t x, int i, float power) {   // i is known when this is compiled
    return i == 0 ? two_of<T, 0>(x, power) : (i == 1 ? two_of<T, 1>(x, power)
            : (i == 2 ? two_of<T, 2>(x, power) : two_of<T, 3>(x, power)));
}

// N dwords at 4-byte alignment.
template <int N>
__device__ __forceinline__ void load_words(uint32_t *r, uint64_t at) {
    typedef uint32_t u32x4a __attribute__((ext_vector_type(4), aligned(4)));
    typedef uint32_t u32x3a __attribute__((ext_vector_type(3), aligned(4)));
    typedef uint32_t u32x2a __attribute__((ext_vector_type(2), aligned(4)));
    if constexpr (N >= 4) {
        const u32x4a x = *(const __attribute__((address_space(1))) u32x4a *)at;
        r[0] = x.x, r[1] = x.y, r[2] = x.z, r[3] = x.w;
        if constexpr (N > 4)
            load_words<N - 4>(r + 4, at + 16);
    } else if constexpr (N == 3) {
        const u32x3a x = *(const __attribute__((address_space(1))) u32x3a *)at;
        r[0] = x.x, r[1] = x.y, r[2] = x.z;
    } else if constexpr (N == 2) {
        const u32x2a x = *(const __attribute__((address_space(1))) u32x2a *)at;
        r[0] = x.x, r[1] = x.y;
    } else {
        static_assert(N == 1, "words");
        r[0] = *(const __attribute__((address_space(1))) uint32_t *)at;
    }
}

// Element e of the head at `at`, as a number.
template <int D>
__device__ __forceinline__ float fp4_number(uint64_t at, uint32_t e) {
    const uint8_t *const p = reinterpret_cast<const uint8_t *>(at);
    const uint32_t code = p[e / 2] >> (4 * (e & 1));
    typedef __bf16 two __attribute__((ext_vector_type(2)));
    const two x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, power_of(p[D / 2 + e / 32], 0), 0);
    return (float)x[0];
}

}  // namespace tbk

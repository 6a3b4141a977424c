// Exchanges between the lanes of a wavefront (not part of the C ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp4idx {

// Partner exchange inside each 16-lane row through the data-parallel-primitive network (a few
// cycles, no LDS round trip): the value of lane li ^ M. M = 1, 2: quad permutations; M = 8: a
// rotation of the row by 8; M = 4: a shift by 4 up or down, chosen by the lane's bit 2.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp32(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
template <int M>
__device__ __forceinline__ uint32_t xor_lane32(uint32_t v, int li) {
    if constexpr (M == 1) return dpp32<0xB1>(v);   // quad_perm [1,0,3,2]
    if constexpr (M == 2) return dpp32<0x4E>(v);   // quad_perm [2,3,0,1]
    if constexpr (M == 8) return dpp32<0x128>(v);  // row_ror:8
    if constexpr (M == 4) {
        const uint32_t up = dpp32<0x104>(v);  // row_shl:4, the value of lane li + 4
        const uint32_t dn = dpp32<0x114>(v);  // row_shr:4, the value of lane li - 4
        return (li & 4) ? dn : up;
    }
    if constexpr (M == 32) {
        // swap of the two 32-lane halves: the first result holds (low, low), the second (high, high)
        const auto sw = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return (li & 32) ? sw[0] : sw[1];
    }
    if constexpr (M == 16) {
        // swap of neighbouring 16-lane rows: the first result holds rows (0, 0, 2, 2), the
        // second rows (1, 1, 3, 3)
        const auto sw = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return (li & 16) ? sw[0] : sw[1];
    }
    return v;
}
template <int M>
__device__ __forceinline__ double xor_lane(double v, int li) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = xor_lane32<M>((uint32_t)b, li), hi = xor_lane32<M>((uint32_t)(b >> 32), li);
    return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
// the value of lane li ^ 7 (row_half_mirror)
__device__ __forceinline__ double mirror8(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = dpp32<0x141>((uint32_t)b), hi = dpp32<0x141>((uint32_t)(b >> 32));
    return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ float mirror8f(float v) { return __uint_as_float(dpp32<0x141>(__float_as_uint(v))); }
template <int M>
__device__ __forceinline__ float xor_lanef(float v, int li) {
    return __uint_as_float(xor_lane32<M>(__float_as_uint(v), li));
}

}  // namespace fp4idx

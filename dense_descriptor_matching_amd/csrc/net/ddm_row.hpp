// ddm_row.hpp -- sums over a wave and 16-byte chunks of rows, shared by the kernels that hold a row in registers.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>
#include <type_traits>

namespace ddm {

// Sum over the 64 lanes, in every lane: DPP exchanges within 16 lanes, then the swaps of rows and halves.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
    return x + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float wave_sum(float x) {
    x = dpp_add<0xb1>(x);            // quad_perm 1,0,3,2
    x = dpp_add<0x4e>(x);            // quad_perm 2,3,0,1
    x = dpp_add<0x141>(x);           // row_half_mirror
    x = dpp_add<0x140>(x);           // row_mirror
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// VE elements from any aligned address of elements, from column C on zeros or (AGAIN) the last columns again.
template <class T, int VE, bool AGAIN = false>
__device__ __forceinline__ void load_chunk(const T *row, int c, int C, float (&out)[VE]) {
    if (AGAIN && c >= C) c = max(C - VE, 0);
    if (c + VE <= C) {
        struct __attribute__((packed, aligned(sizeof(T)))) Raw { T v[VE]; };
        const Raw r = *reinterpret_cast<const Raw *>(row + c);
#pragma unroll
        for (int e = 0; e < VE; ++e) out[e] = (float)r.v[e];
    } else {
#pragma unroll
        for (int e = 0; e < VE; ++e) out[e] = c + e < C ? (float)row[c + e] : AGAIN && e ? out[e ? e - 1 : 0] : 0.f;
    }
}
// 16 bytes at an address of so many, of whatever type.
typedef uint32_t Bytes16Of2 __attribute__((ext_vector_type(4), aligned(2), may_alias));
typedef uint32_t Bytes16Of4 __attribute__((ext_vector_type(4), aligned(4), may_alias));
typedef uint32_t Bytes16Of16 __attribute__((ext_vector_type(4), aligned(16), may_alias));
template <int ALIGN> using Bytes16 = std::conditional_t<ALIGN == 2, Bytes16Of2, std::conditional_t<ALIGN == 4, Bytes16Of4, Bytes16Of16>>;
// VE elements to any aligned address of elements, those before column C.
template <class T, int VE>
__device__ __forceinline__ void store_chunk(T *row, int c, int C, const float (&in)[VE]) {
    static_assert(VE * sizeof(T) % 16 == 0, "whole 16-byte pieces");
    if (c + VE <= C) {
        struct __attribute__((aligned(16))) Raw { T v[VE]; } r;
#pragma unroll
        for (int e = 0; e < VE; ++e) r.v[e] = (T)in[e];
#pragma unroll
        for (int i = 0; i < VE * (int)sizeof(T) / 16; ++i)
            *reinterpret_cast<Bytes16<sizeof(T)> *>((char *)(row + c) + 16 * i) = reinterpret_cast<const Bytes16Of16 *>(&r)[i];
    } else {
#pragma unroll
        for (int e = 0; e < VE; ++e)
            if (c + e < C) row[c + e] = (T)in[e];
    }
}

// f(T, W) for the types of the rows and of their parameters (float or the rows').
template <class F>
inline void with_types(int dtype, int wtype, F f) {
    if (dtype == DDM_F32) f(float{}, float{});
    else if (dtype == DDM_F16) wtype == DDM_F32 ? f(_Float16{}, float{}) : f(_Float16{}, _Float16{});
    else wtype == DDM_F32 ? f(__bf16{}, float{}) : f(__bf16{}, __bf16{});
}

}  // namespace ddm

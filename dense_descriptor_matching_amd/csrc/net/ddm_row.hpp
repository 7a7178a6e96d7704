// ddm_row.hpp -- sums over a wave and 16-byte chunks of rows, shared by the kernels that hold a row in registers.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>

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

// VE elements from any aligned address of elements, zeros from column C on.
template <class T, int VE>
__device__ __forceinline__ void load_chunk(const T *row, int c, int C, float (&out)[VE]) {
    if (c + VE <= C) {
        struct __attribute__((packed, aligned(sizeof(T)))) Raw { T v[VE]; };
        const Raw r = *reinterpret_cast<const Raw *>(row + c);
#pragma unroll
        for (int e = 0; e < VE; ++e) out[e] = (float)r.v[e];
    } else {
#pragma unroll
        for (int e = 0; e < VE; ++e) out[e] = c + e < C ? (float)row[c + e] : 0.f;
    }
}
template <class T, int VE>
__device__ __forceinline__ void store_chunk(T *row, int c, int C, const float (&in)[VE]) {
    if (c + VE <= C) {
        struct __attribute__((packed, aligned(sizeof(T)))) Raw { T v[VE]; } r;
#pragma unroll
        for (int e = 0; e < VE; ++e) r.v[e] = (T)in[e];
        *reinterpret_cast<Raw *>(row + c) = r;
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

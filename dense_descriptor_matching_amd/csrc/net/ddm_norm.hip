// ddm_norm.hip -- layer norm, forward and backward (ddm_layer_norm_*).
//
//   xh = (x - mean) rstd,  rstd = (var + eps)^-1/2,  y = xh w + b
//   u = dy w,  dx = rstd (u - mean(u) - xh mean(u xh)),  dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Bound by memory: each of x (and dy) is read once and y (dx) written once. A row lies in the registers of a team of
// threads (a wave, or four for wide rows) in chunks of 16 bytes, so the variance is taken about the mean without
// reading again. A team keeps its columns' w, b and, backward, its share of dw and db in registers over all its rows;
// the shares of a workgroup meet in LDS and those of all workgroups in a second, small kernel, always in the same
// order. Measured at 24576 x 1024 bf16: forward 17.7 us (100 MB, 5.7 TB/s; a copy of 2 x 200 MB reaches 5.4 here),
// backward 31.6 us (150 MB, 4.8 TB/s) and 4.2 us for the last sums; grids of 1024 to all workgroups, and half or twice
// the backward ones, made no difference.
#include "../../../include/ddm.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

namespace {

struct NormArgs {
    const void *x, *dy, *w, *b;
    void *y, *dx;
    float *mean, *rstd, *part;       // part: [workgroup][2][C]
    int64_t ldx, N;
    int C;
    float eps;
};

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
// Over a team. Two scratch rows are used in turn, so one barrier per sum is enough.
template <int TEAM>
__device__ __forceinline__ float team_sum(float x, float (*scratch)[4], int &turn) {
    x = wave_sum(x);
    if constexpr (TEAM == 64) return x;
    scratch[turn][threadIdx.x >> 6] = x;
    __syncthreads();
    x = (scratch[turn][0] + scratch[turn][1]) + (scratch[turn][2] + scratch[turn][3]);
    turn ^= 1;
    return x;
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

template <class T, class W, int TEAM, int V>
__global__ __launch_bounds__(256) void norm_fwd_kernel(NormArgs p) {
    constexpr int VE = 16 / sizeof(T);
    __shared__ float scratch[2][4];
    const int t = threadIdx.x % TEAM;
    const int64_t first = (int64_t)blockIdx.x * (256 / TEAM) + threadIdx.x / TEAM, pitch = (int64_t)gridDim.x * (256 / TEAM);
    float w[V][VE], b[V][VE];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = (j * TEAM + t) * VE;
#pragma unroll
        for (int e = 0; e < VE; ++e) { w[j][e] = 1.f; b[j][e] = 0.f; }
        if (p.w) load_chunk<W, VE>((const W *)p.w, c, p.C, w[j]);
        if (p.b) load_chunk<W, VE>((const W *)p.b, c, p.C, b[j]);
    }
    int turn = 0;
    for (int64_t n = first; n < p.N; n += pitch) {
        const T *row = (const T *)p.x + n * p.ldx;
        float x[V][VE], sum = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            load_chunk<T, VE>(row, (j * TEAM + t) * VE, p.C, x[j]);
#pragma unroll
            for (int e = 0; e < VE; ++e) sum += x[j][e];
        }
        const float mean = team_sum<TEAM>(sum, scratch, turn) / (float)p.C;
        sum = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                x[j][e] = (j * TEAM + t) * VE + e < p.C ? x[j][e] - mean : 0.f;
                sum = __builtin_fmaf(x[j][e], x[j][e], sum);
            }
        const float rstd = 1.f / sqrtf(team_sum<TEAM>(sum, scratch, turn) / (float)p.C + p.eps);
        T *out = (T *)p.y + n * p.C;
#pragma unroll
        for (int j = 0; j < V; ++j) {
#pragma unroll
            for (int e = 0; e < VE; ++e) x[j][e] = __builtin_fmaf(x[j][e] * rstd, w[j][e], b[j][e]);
            store_chunk<T, VE>(out, (j * TEAM + t) * VE, p.C, x[j]);
        }
        if (t == 0) { p.mean[n] = mean; p.rstd[n] = rstd; }
    }
}

template <class T, class W, int TEAM, int V, bool PARAMS>
__global__ __launch_bounds__(256) void norm_bwd_kernel(NormArgs p) {
    constexpr int VE = 16 / sizeof(T);
    __shared__ float scratch[2][4];
    extern __shared__ float share[];                       // TEAM == 64: [4][C]
    const int t = threadIdx.x % TEAM;
    const int64_t first = (int64_t)blockIdx.x * (256 / TEAM) + threadIdx.x / TEAM, pitch = (int64_t)gridDim.x * (256 / TEAM);
    float w[V][VE], dw[V][VE], db[V][VE];
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
        for (int e = 0; e < VE; ++e) { w[j][e] = 1.f; dw[j][e] = 0.f; db[j][e] = 0.f; }
        if (p.w) load_chunk<W, VE>((const W *)p.w, (j * TEAM + t) * VE, p.C, w[j]);
    }
    int turn = 0;
    for (int64_t n = first; n < p.N; n += pitch) {
        const T *row = (const T *)p.x + n * p.ldx, *grow = (const T *)p.dy + n * p.C;
        const float mean = p.mean[n], rstd = p.rstd[n];
        float x[V][VE], g[V][VE], s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            load_chunk<T, VE>(row, (j * TEAM + t) * VE, p.C, x[j]);
            load_chunk<T, VE>(grow, (j * TEAM + t) * VE, p.C, g[j]);
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int e = 0; e < VE; ++e) {                 // past column C: dy = 0, so nothing is added
                x[j][e] = (x[j][e] - mean) * rstd;
                if constexpr (PARAMS) {
                    dw[j][e] = __builtin_fmaf(g[j][e], x[j][e], dw[j][e]);
                    db[j][e] += g[j][e];
                }
                g[j][e] *= w[j][e];
                s1 += g[j][e];
                s2 = __builtin_fmaf(g[j][e], x[j][e], s2);
            }
        if (!p.dx) continue;
        s1 = team_sum<TEAM>(s1, scratch, turn) / (float)p.C;
        s2 = team_sum<TEAM>(s2, scratch, turn) / (float)p.C;
        T *out = (T *)p.dx + n * p.C;
#pragma unroll
        for (int j = 0; j < V; ++j) {
#pragma unroll
            for (int e = 0; e < VE; ++e) x[j][e] = rstd * (g[j][e] - __builtin_fmaf(x[j][e], s2, s1));
            store_chunk<T, VE>(out, (j * TEAM + t) * VE, p.C, x[j]);
        }
    }
    if constexpr (PARAMS) {
        float *part = p.part + (int64_t)blockIdx.x * 2 * p.C;
        if constexpr (TEAM == 256) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                store_chunk<float, VE>(part, (j * TEAM + t) * VE, p.C, dw[j]);
                store_chunk<float, VE>(part + p.C, (j * TEAM + t) * VE, p.C, db[j]);
            }
        } else {
            float *mine = share + (threadIdx.x / TEAM) * p.C;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                __syncthreads();
#pragma unroll
                for (int j = 0; j < V; ++j) store_chunk<float, VE>(mine, (j * TEAM + t) * VE, p.C, k ? db[j] : dw[j]);
                __syncthreads();
                for (int c = threadIdx.x; c < p.C; c += 256)
                    part[k * p.C + c] = (share[c] + share[p.C + c]) + (share[2 * p.C + c] + share[3 * p.C + c]);
            }
        }
    }
}

// dw (blockIdx.y = 0) and db (1) from the workgroups' shares: 32 columns a workgroup, 32 of its threads share a column.
template <class W>
__global__ __launch_bounds__(1024) void norm_reduce_kernel(const float *part, int parts, int C, W *dw, W *db) {
    __shared__ float s[32][33];
    W *out = blockIdx.y ? db : dw;
    if (!out) return;
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
    float sum = 0.f;
    if (c < C)
#pragma unroll 4
        for (int n = g; n < parts; n += 32) sum += part[((int64_t)n * 2 + blockIdx.y) * C + c];
    s[g][threadIdx.x & 31] = sum;
    __syncthreads();
    if (g == 0 && c < C) {
        float total = 0.f;
        for (int k = 0; k < 32; ++k) total += s[k][threadIdx.x];
        out[c] = (W)total;
    }
}

int esize(int dtype) { return dtype == DDM_F32 ? 4 : 2; }

// A wave holds a row of up to four chunks a lane; wider rows take four waves.
struct Shape { int team, v; };
Shape shape_of(int C, int dtype) {
    const int ve = 16 / esize(dtype);
    const int team = C <= 64 * ve * 4 ? 64 : 256;
    int v = 1;
    while (team * ve * v < C) v *= 2;
    return {team, v};
}
// The shapes that shape_of gives for some C.
template <class T>
constexpr bool reached(int team, int v) {
    return team == 64 ? v <= 4 : v >= 2 && team * v * 16 / (int)sizeof(T) <= DDM_MAX_NORM_C;
}
// Workgroups of the backward pass: at least 8 rows a team, so that its partial sums stay small beside its rows.
int bwd_groups(int64_t N, int C, int dtype) {
    const int teams = 256 / shape_of(C, dtype).team;
    return (int)std::min<int64_t>((N + teams * 8 - 1) / (teams * 8), 1024);
}

bool types_ok(int dtype, int wtype) {
    return (dtype == DDM_F32 || dtype == DDM_F16 || dtype == DDM_BF16) && (wtype == DDM_F32 || wtype == dtype);
}

template <class F>
void with_shape(Shape s, F f) {
    auto go = [&](auto team) {
        switch (s.v) {
            case 1: f(team, std::integral_constant<int, 1>{}); break;
            case 2: f(team, std::integral_constant<int, 2>{}); break;
            case 4: f(team, std::integral_constant<int, 4>{}); break;
            default: f(team, std::integral_constant<int, 8>{}); break;
        }
    };
    if (s.team == 64) go(std::integral_constant<int, 64>{});
    else go(std::integral_constant<int, 256>{});
}
template <class F>
void with_types(int dtype, int wtype, F f) {
    if (dtype == DDM_F32) f(float{}, float{});
    else if (dtype == DDM_F16) wtype == DDM_F32 ? f(_Float16{}, float{}) : f(_Float16{}, _Float16{});
    else wtype == DDM_F32 ? f(__bf16{}, float{}) : f(__bf16{}, __bf16{});
}

bool off(const void *p, int e) { return !p || (uintptr_t)p % e; }

}  // namespace

extern "C" {

int ddm_layer_norm_forward(const void *x, int64_t ldx, const void *weight, const void *bias, int64_t N, int C, int dtype,
                           int wtype, double eps, void *y, float *mean, float *rstd, hipStream_t stream) {
    if (!types_ok(dtype, wtype) || C < 1 || C > DDM_MAX_NORM_C) return DDM_ERR_UNSUPPORTED;
    const int e = esize(dtype), we = esize(wtype);
    if (N < 0 || N > INT_MAX || ldx < C || !(eps >= 0) || !std::isfinite(eps)) return DDM_ERR_INVALID;
    if (N == 0) return DDM_OK;
    if (off(x, e) || off(y, e) || off(mean, 4) || off(rstd, 4) || (uintptr_t)weight % we || (uintptr_t)bias % we)
        return DDM_ERR_INVALID;
    NormArgs a{};
    a.x = x; a.w = weight; a.b = bias; a.y = y; a.mean = mean; a.rstd = rstd;
    a.ldx = ldx; a.N = N; a.C = C; a.eps = (float)eps;
    const Shape s = shape_of(C, dtype);
    const int teams = 256 / s.team;
    const unsigned grid = (unsigned)std::min<int64_t>((N + teams - 1) / teams, 2048);
    with_types(dtype, wtype, [&](auto t, auto w) {
        with_shape(s, [&](auto team, auto v) {
            if constexpr (reached<decltype(t)>(decltype(team)::value, decltype(v)::value))
                hipLaunchKernelGGL((norm_fwd_kernel<decltype(t), decltype(w), decltype(team)::value, decltype(v)::value>),
                                   dim3(grid), dim3(256), 0, stream, a);
        });
    });
    return hipGetLastError() == hipSuccess ? DDM_OK : DDM_ERR_HIP;
}

size_t ddm_layer_norm_backward_workspace_bytes(int64_t N, int C, int dtype) {
    if (!types_ok(dtype, DDM_F32) || C < 1 || C > DDM_MAX_NORM_C || N < 0 || N > INT_MAX) return 0;
    return std::max<size_t>((size_t)bwd_groups(N, C, dtype) * 2 * C * sizeof(float), 16);
}

int ddm_layer_norm_backward(const void *dy, const void *x, int64_t ldx, const void *weight, const float *mean,
                            const float *rstd, int64_t N, int C, int dtype, int wtype, void *dx, void *dweight,
                            void *dbias, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!types_ok(dtype, wtype) || C < 1 || C > DDM_MAX_NORM_C) return DDM_ERR_UNSUPPORTED;
    const int e = esize(dtype), we = esize(wtype);
    if (N < 0 || N > INT_MAX || ldx < C) return DDM_ERR_INVALID;
    if (N && (off(dy, e) || off(x, e) || off(mean, 4) || off(rstd, 4))) return DDM_ERR_INVALID;
    if ((uintptr_t)weight % we || (uintptr_t)dx % e || (uintptr_t)dweight % we || (uintptr_t)dbias % we)
        return DDM_ERR_INVALID;
    const bool params = dweight || dbias;
    if (params && (off(workspace, 16) || workspace_bytes < ddm_layer_norm_backward_workspace_bytes(N, C, dtype)))
        return DDM_ERR_WORKSPACE;
    NormArgs a{};
    a.x = x; a.dy = dy; a.w = weight; a.dx = dx; a.mean = const_cast<float *>(mean); a.rstd = const_cast<float *>(rstd);
    a.part = (float *)workspace; a.ldx = ldx; a.N = N; a.C = C;
    const Shape s = shape_of(C, dtype);
    const int groups = bwd_groups(N, C, dtype);
    if (N && (dx || params)) {
        with_types(dtype, wtype, [&](auto t, auto w) {
            with_shape(s, [&](auto team, auto v) {
                constexpr int TEAM = decltype(team)::value, V = decltype(v)::value;
                if constexpr (reached<decltype(t)>(TEAM, V)) {
                    using T = decltype(t);
                    using W = decltype(w);
                    if (params)
                        hipLaunchKernelGGL((norm_bwd_kernel<T, W, TEAM, V, true>), dim3(groups), dim3(256),
                                           TEAM == 64 ? 4 * C * sizeof(float) : 0, stream, a);
                    else
                        hipLaunchKernelGGL((norm_bwd_kernel<T, W, TEAM, V, false>), dim3(groups), dim3(256), 0, stream, a);
                }
            });
        });
        if (hipGetLastError() != hipSuccess) return DDM_ERR_HIP;
    }
    if (params) {
        with_types(dtype, wtype, [&](auto, auto w) {
            using W = decltype(w);
            hipLaunchKernelGGL((norm_reduce_kernel<W>), dim3((C + 31) / 32, 2), dim3(1024), 0, stream, a.part, groups, C,
                               (W *)dweight, (W *)dbias);
        });
    }
    return hipGetLastError() == hipSuccess ? DDM_OK : DDM_ERR_HIP;
}

}  // extern "C"

// ddm_residual.hip -- the sum of a residual stream and a branch with the norms around it (ddm_residual_norm_*).
//
//   t = branch, or norm(branch) wb + bb;   s = x + scale sigmoid(gate) t;   y = norm(s) w + b
//   norm(z) = (z - mean) rstd,  rstd = (var + eps)^-1/2;  rms: mean = 0
//   backward, with zh = norm(s), th = norm(branch), o = sigmoid(gate):
//   u = dy w,  dx = ds + rstd (u - mean(u) - zh mean(u zh));  dw = sum over rows of dy zh,  db = sum of dy
//   dscale = sum of dx o t,  v = dx scale,  dgate = v t o',  v' = v o
//   dwb = sum of v' th,  dbb = sum of v',  r = v' wb,  dbranch = rstd_b (r - mean(r) - th mean(r th))   (or v')
//   rms: without the means of u and r.
//
// Bound by memory: each input is read once, each output written once. A row lies in the registers of a team of threads
// (a wave, or four or eight for wide rows), 16 columns a thread at most, so that backward keeps its share of up to five
// sums over rows beside a row of five inputs. Measured, 24576 x 1024 bf16 with gate, scale and both norms: forward 47 us
// (252 MB, 5.3 TB/s; a copy of 2 x 200 MB reaches 5.4 here), backward 96 us (403 MB, 4.2 TB/s, one wave to a SIMD: 328
// registers) and 4 us for the last sums; 10007 x 1285 fp32, rms: 44 and 84 us (206 and 309 MB). From 4097 columns on, teams of eight
// waves spill backward's registers (4096 x 8192 bf16, everything: 110 and 671 us). Backward takes s again from x and the branch
// in 32 bits: the s that forward gives back is rounded, and what that costs dw would not average out.
#include "../../../include/ddm.h"
#include "ddm_row.hpp"

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

// Fused multiply-adds stand where they are written: chosen by the compiler, they would differ with the gradients that a
// call wants, and so would their last bits.
#pragma clang fp contract(off)

using namespace ddm;

namespace {

struct ResArgs {
    const void *x, *branch, *gate, *dy, *ds;
    const void *w, *b, *scale, *bw, *bb;
    void *s, *y, *dx, *dbranch, *dgate;
    float *stats, *part;                        // stats: [2 or 4][N]; part: [workgroup][3 or 5][C]
    int64_t ldx, ldb, ldg, N;
    int C;
    float eps;
    bool rms;
};

constexpr int threads_of(int team) { return team > 256 ? team : 256; }

// Sums over a team, K at a time. Two scratch rows are used in turn, so one barrier is enough.
typedef float Scratch[2][8][2];
template <int TEAM, int K>
__device__ __forceinline__ void team_sums(float (&x)[K], Scratch &scratch, int &turn) {
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = wave_sum(x[k]);
    if constexpr (TEAM == 64) return;
#pragma unroll
    for (int k = 0; k < K; ++k) scratch[turn][threadIdx.x >> 6][k] = x[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        x[k] = scratch[turn][0][k];
#pragma unroll
        for (int i = 1; i < TEAM / 64; ++i) x[k] += scratch[turn][i][k];
    }
    turn ^= 1;
}

// Columns of a row, x in: x - mean and rstd out. Columns past C are and stay zeros.
template <int TEAM, int V, int VE>
__device__ __forceinline__ float2 normed(float (&x)[V][VE], const ResArgs &p, int t, Scratch &scratch, int &turn) {
    float mean = 0.f, sum[1] = {0.f};
    if (!p.rms) {
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int e = 0; e < VE; ++e) sum[0] += x[j][e];
        team_sums<TEAM>(sum, scratch, turn);
        mean = sum[0] / (float)p.C;
        sum[0] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            x[j][e] = (j * TEAM + t) * VE + e < p.C ? x[j][e] - mean : 0.f;
            sum[0] = __builtin_fmaf(x[j][e], x[j][e], sum[0]);
        }
    team_sums<TEAM>(sum, scratch, turn);
    return {mean, 1.f / sqrtf(sum[0] / (float)p.C + p.eps)};
}

// sigmoid(g) and its derivative, with e = exp(-|g|): 1 / (1 + e) or e / (1 + e), and e / (1 + e)^2. As o (1 - o) the derivative of a
// gate that is far open would lose the digits that 1 - o has (half of them at g = 10, all at 17).
struct Gate { float open, slope; };
__device__ __forceinline__ Gate gate_of(float g) {
    const float e = __expf(-fabsf(g)), r = __builtin_amdgcn_rcpf(1.f + e), shut = e * r;
    return {g >= 0.f ? r : shut, shut * r};
}

// A chunk of a row as it lies in memory: what the next row needs waits in half the registers.
template <class T>
struct Chunk {
    static constexpr int VE = 16 / sizeof(T);
    T v[VE];
    // Past column C zeros, or (AGAIN) the last columns again: backward's sums take those times a gradient of zero, where the norm of
    // a zero, (0 - mean) rstd, may be infinite: in rows of large values that hardly vary. Lanes that have none of the columns load a
    // whole chunk then instead of missing elements one by one (24576 x 1000 bf16 backward 166 -> 106 us, x 768 fp16 58 -> 47).
    template <bool AGAIN = false>
    __device__ __forceinline__ void load(const T *row, int c, int C) {
        if (AGAIN && c >= C) c = max(C - VE, 0);
        if (c + VE <= C) {
            const Bytes16<sizeof(T)> x = *reinterpret_cast<const Bytes16<sizeof(T)> *>(row + c);
            __builtin_memcpy(v, &x, 16);
        } else {
#pragma unroll
            for (int e = 0; e < VE; ++e) v[e] = c + e < C ? row[c + e] : AGAIN && e ? v[e ? e - 1 : 0] : (T)0.f;
        }
    }
    __device__ __forceinline__ void take(float (&to)[VE]) const {
#pragma unroll
        for (int e = 0; e < VE; ++e) to[e] = (float)v[e];
    }
};

// Parameters' columns, in LDS for the workgroup: registers are for sums and rows. Zeros behind the last: what rows have
// there counts for nothing. So for a wave a row, and the next row is fetched ahead (24576 x 1024 bf16 forward 63 -> 47 us,
// backward 189 -> 96). Four and eight waves' rows have 8 to 16 columns a thread and more parameters than LDS has room for in
// as many workgroups: in registers, without fetching ahead (10007 x 1285 fp32 forward 44 us, with LDS 60 to 66).
template <class T, class W, int TEAM, int V>
struct Params {
    static constexpr int VE = 16 / sizeof(T), WIDTH = TEAM * V * VE, THREADS = threads_of(TEAM);
    static constexpr bool IN_LDS = TEAM == 64;
    static constexpr size_t BYTES = IN_LDS ? WIDTH * sizeof(float) : 0;
    float *lds;
    int C, t;
    float own[IN_LDS ? 1 : 5][V][VE];
    __device__ __forceinline__ void put(int k, const void *from, float none) {
        if constexpr (IN_LDS) {
#pragma unroll
            for (int i = 0; i < WIDTH / THREADS; ++i) {
                const int c = i * THREADS + threadIdx.x;
                lds[k * WIDTH + c] = c >= C ? 0.f : from ? (float)((const W *)from)[c] : none;
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
#pragma unroll
                for (int e = 0; e < VE; ++e) own[k][j][e] = (j * TEAM + t) * VE + e < C ? none : 0.f;
                if (from) load_chunk<W, VE>((const W *)from, (j * TEAM + t) * VE, C, own[k][j]);
            }
        }
    }
    __device__ __forceinline__ void get(int k, int j, float (&to)[VE]) const {
#pragma unroll
        for (int e = 0; e < VE; e += 4) {
            if constexpr (IN_LDS) {
                const float4 x = *reinterpret_cast<const float4 *>(lds + k * WIDTH + (j * TEAM + t) * VE + e);
                to[e] = x.x; to[e + 1] = x.y; to[e + 2] = x.z; to[e + 3] = x.w;
            } else {
#pragma unroll
                for (int i = e; i < e + 4; ++i) to[i] = own[k][j][i];
            }
        }
    }
};

template <class T, class W, int TEAM, int V, bool BN>
__global__ __launch_bounds__(threads_of(TEAM)) void residual_fwd_kernel(ResArgs p) {
    constexpr int VE = 16 / sizeof(T), THREADS = threads_of(TEAM), TEAMS = THREADS / TEAM;
    __shared__ Scratch scratch;
    extern __shared__ __attribute__((aligned(16))) float param[];      // w, b, scale, bw, bb
    using Pr = Params<T, W, TEAM, V>;
    const int t = threadIdx.x % TEAM;
    Pr pr{param, p.C, t};
    const int64_t first = (int64_t)blockIdx.x * TEAMS + threadIdx.x / TEAM, pitch = (int64_t)gridDim.x * TEAMS;
    Chunk<T> x0[V], r0[V], g0[V] = {};                     // zeros of a gate that is not there
    auto fetch = [&](int64_t n) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (j * TEAM + t) * VE;
            r0[j].load((const T *)p.branch + n * p.ldb, c, p.C);
            x0[j].load((const T *)p.x + n * p.ldx, c, p.C);
            if (p.gate) g0[j].load((const T *)p.gate + n * p.ldg, c, p.C);
        }
    };
    if (Pr::IN_LDS && first < p.N) fetch(first);
    pr.put(0, p.w, 1.f);
    pr.put(1, p.b, 0.f);
    pr.put(2, p.scale, 1.f);
    if constexpr (BN) {
        pr.put(3, p.bw, 1.f);
        pr.put(4, p.bb, 0.f);
    }
    __syncthreads();
    int turn = 0;
    for (int64_t n = first; n < p.N; n += pitch) {
        if constexpr (Pr::IN_LDS) asm volatile("" ::: "memory");       // parameters are read again, not kept in registers
        else fetch(n);
        float x[V][VE], g[V][VE], r[V][VE];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            r0[j].take(r[j]);
            x0[j].take(x[j]);
            g0[j].take(g[j]);
        }
        if (Pr::IN_LDS && n + pitch < p.N) fetch(n + pitch);
        if constexpr (BN) {
            const float2 m = normed<TEAM>(r, p, t, scratch, turn);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float bw[VE], bb[VE];
                pr.get(3, j, bw);
                pr.get(4, j, bb);
#pragma unroll
                for (int e = 0; e < VE; ++e) r[j][e] = __builtin_fmaf(r[j][e] * m.y, bw[e], bb[e]);
            }
            if (t == 0) { p.stats[2 * p.N + n] = m.x; p.stats[3 * p.N + n] = m.y; }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float scale[VE];
            pr.get(2, j, scale);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                if (p.gate) r[j][e] *= gate_of(g[j][e]).open;
                r[j][e] = __builtin_fmaf(r[j][e], scale[e], x[j][e]);
            }
            store_chunk<T, VE>((T *)p.s + n * p.C, (j * TEAM + t) * VE, p.C, r[j]);
        }
        const float2 m = normed<TEAM>(r, p, t, scratch, turn);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float w[VE], b[VE];
            pr.get(0, j, w);
            pr.get(1, j, b);
#pragma unroll
            for (int e = 0; e < VE; ++e) r[j][e] = __builtin_fmaf(r[j][e] * m.y, w[e], b[e]);
            store_chunk<T, VE>((T *)p.y + n * p.C, (j * TEAM + t) * VE, p.C, r[j]);
        }
        if (t == 0) { p.stats[n] = m.x; p.stats[p.N + n] = m.y; }
    }
}

// Two waves to a SIMD where that takes a few registers less than the compiler would like (24576 x 768 fp16, no norm of the branch: 46 us,
// 60 with one); others would spill, or have two anyway.
template <class T, class W, int TEAM, int V, bool BN, bool PARAMS>
__global__ __launch_bounds__(threads_of(TEAM), TEAM == 64 && sizeof(T) == 2 && !BN ? 2 : 1) void residual_bwd_kernel(ResArgs p) {
    constexpr int VE = 16 / sizeof(T), THREADS = threads_of(TEAM), TEAMS = THREADS / TEAM, NP = BN ? 5 : 3;
    __shared__ Scratch scratch;
    extern __shared__ __attribute__((aligned(16))) float param[];      // w, scale, bw, bb; at the end a sum's columns of four teams
    using Pr = Params<T, W, TEAM, V>;
    const int t = threadIdx.x % TEAM;
    Pr pr{param, p.C, t};
    const int64_t first = (int64_t)blockIdx.x * TEAMS + threadIdx.x / TEAM, pitch = (int64_t)gridDim.x * TEAMS;
    const float inv_c = 1.f / (float)p.C;
    Chunk<T> x0[V], r0[V], o0[V] = {}, u0[V] = {}, d0[V] = {};         // zeros of what is not there
    float mean0 = 0.f, rstd0 = 0.f, bmean0 = 0.f, brstd0 = 0.f;
    auto fetch = [&](int64_t n) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (j * TEAM + t) * VE;
            r0[j].template load<true>((const T *)p.branch + n * p.ldb, c, p.C);
            x0[j].template load<true>((const T *)p.x + n * p.ldx, c, p.C);
            if (p.gate) o0[j].template load<true>((const T *)p.gate + n * p.ldg, c, p.C);
            if (p.dy) u0[j].template load<true>((const T *)p.dy + n * p.C, c, p.C);
            if (p.ds) d0[j].template load<true>((const T *)p.ds + n * p.C, c, p.C);
        }
        mean0 = p.stats[n];
        rstd0 = p.stats[p.N + n];
        if constexpr (BN) { bmean0 = p.stats[2 * p.N + n]; brstd0 = p.stats[3 * p.N + n]; }
    };
    if (Pr::IN_LDS && first < p.N) fetch(first);
    pr.put(0, p.w, 1.f);
    pr.put(1, p.scale, 1.f);
    if constexpr (BN) {
        pr.put(2, p.bw, 1.f);
        pr.put(3, p.bb, 0.f);
    }
    float sum[NP][V][VE];
    if constexpr (PARAMS)
#pragma unroll
        for (int k = 0; k < NP; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int e = 0; e < VE; ++e) sum[k][j][e] = 0.f;
    __syncthreads();
    int turn = 0;
    for (int64_t n = first; n < p.N; n += pitch) {
        if constexpr (Pr::IN_LDS) asm volatile("" ::: "memory");       // parameters are read again, not kept in registers
        else fetch(n);
        const float mean = mean0, rstd = rstd0, bmean = bmean0, brstd = brstd0;
        float x[V][VE], r[V][VE], o[V][VE], slope[V][VE], u[V][VE], d[V][VE], m[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < V; ++j) {
            r0[j].take(r[j]);
            x0[j].take(x[j]);
            o0[j].take(o[j]);
            u0[j].take(u[j]);
            d0[j].take(d[j]);
        }
        if (Pr::IN_LDS && n + pitch < p.N) fetch(n + pitch);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (j * TEAM + t) * VE;
            float w[VE], scale[VE], bw[VE], bb[VE];
            pr.get(0, j, w);
            pr.get(1, j, scale);
            if constexpr (BN) { pr.get(2, j, bw); pr.get(3, j, bb); }
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                if constexpr (BN) r[j][e] = (r[j][e] - bmean) * brstd;
                float part = r[j][e];
                if constexpr (BN) part = __builtin_fmaf(part, bw[e], bb[e]);
                if (p.gate) {
                    const Gate g = gate_of(o[j][e]);
                    part *= o[j][e] = g.open;
                    slope[j][e] = g.slope;
                }
                x[j][e] = (__builtin_fmaf(part, scale[e], x[j][e]) - mean) * rstd;
                if constexpr (PARAMS) {
                    sum[0][j][e] = __builtin_fmaf(u[j][e], x[j][e], sum[0][j][e]);
                    sum[1][j][e] += u[j][e];
                }
                u[j][e] *= w[e];
                m[0] += u[j][e];
                m[1] = __builtin_fmaf(u[j][e], x[j][e], m[1]);
            }
        }
        team_sums<TEAM>(m, scratch, turn);
        const float s1 = p.rms ? 0.f : m[0] * inv_c, s2 = m[1] * inv_c;
        m[0] = m[1] = 0.f;
        if constexpr (Pr::IN_LDS) asm volatile("" ::: "memory");
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (j * TEAM + t) * VE;
            float scale[VE], bw[VE], bb[VE];
            pr.get(1, j, scale);
            if constexpr (BN) { pr.get(2, j, bw); pr.get(3, j, bb); }
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                d[j][e] = __builtin_fmaf(rstd, u[j][e] - __builtin_fmaf(x[j][e], s2, s1), d[j][e]);
            }
            if (p.dx) store_chunk<T, VE>((T *)p.dx + n * p.C, c, p.C, d[j]);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                float full = r[j][e];                      // t
                if constexpr (BN) full = __builtin_fmaf(full, bw[e], bb[e]);
                if constexpr (PARAMS) sum[2][j][e] = __builtin_fmaf(d[j][e], p.gate ? full * o[j][e] : full, sum[2][j][e]);
                d[j][e] *= scale[e];
                x[j][e] = d[j][e] * full * slope[j][e];
                if (p.gate) d[j][e] *= o[j][e];
                if constexpr (BN) {
                    if constexpr (PARAMS) {
                        sum[3][j][e] = __builtin_fmaf(d[j][e], r[j][e], sum[3][j][e]);
                        sum[4][j][e] += d[j][e];
                    }
                    d[j][e] *= bw[e];
                    m[0] += d[j][e];
                    m[1] = __builtin_fmaf(d[j][e], r[j][e], m[1]);
                }
            }
            if (p.dgate) store_chunk<T, VE>((T *)p.dgate + n * p.C, c, p.C, x[j]);
        }
        if (!p.dbranch) continue;
        if constexpr (BN) {
            team_sums<TEAM>(m, scratch, turn);
            m[0] = p.rms ? 0.f : m[0] * inv_c;
            m[1] *= inv_c;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if constexpr (BN)
#pragma unroll
                for (int e = 0; e < VE; ++e) d[j][e] = brstd * (d[j][e] - __builtin_fmaf(r[j][e], m[1], m[0]));
            store_chunk<T, VE>((T *)p.dbranch + n * p.C, (j * TEAM + t) * VE, p.C, d[j]);
        }
    }
    if constexpr (PARAMS) {
        float *part = p.part + (int64_t)blockIdx.x * NP * p.C;
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            if constexpr (TEAM > 64) {
#pragma unroll
                for (int j = 0; j < V; ++j) store_chunk<float, VE>(part + k * p.C, (j * TEAM + t) * VE, p.C, sum[k][j]);
            } else {
                float *mine = param + (threadIdx.x / TEAM) * p.C;
                __syncthreads();
#pragma unroll
                for (int j = 0; j < V; ++j) store_chunk<float, VE>(mine, (j * TEAM + t) * VE, p.C, sum[k][j]);
                __syncthreads();
                for (int c = threadIdx.x; c < p.C; c += 256)
                    part[k * p.C + c] = (param[c] + param[p.C + c]) + (param[2 * p.C + c] + param[3 * p.C + c]);
            }
        }
    }
}

struct Sums { void *out[5]; };

// The parameters' gradients (blockIdx.y) from the workgroups' shares: 32 columns a workgroup, 32 of its threads share a column.
template <class W>
__global__ __launch_bounds__(1024) void residual_reduce_kernel(const float *part, int parts, int np, int C, Sums to) {
    __shared__ float s[32][33];
    W *out = (W *)to.out[blockIdx.y];
    if (!out) return;
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
    float sum = 0.f;
    if (c < C)
#pragma unroll 4
        for (int n = g; n < parts; n += 32) sum += part[((int64_t)n * np + blockIdx.y) * C + c];
    s[g][threadIdx.x & 31] = sum;
    __syncthreads();
    if (g == 0 && c < C) {
        float total = 0.f;
        for (int k = 0; k < 32; ++k) total += s[k][threadIdx.x];
        out[c] = (W)total;
    }
}

int esize(int dtype) { return dtype == DDM_F32 ? 4 : 2; }

// A thread has at most 16 columns: a wave, four or eight of them to a row.
struct Shape { int team, v; };
Shape shape_of(int C, int dtype) {
    const int ve = 16 / esize(dtype);
    const int team = C <= 1024 ? 64 : C <= 4096 ? 256 : 512;
    int v = 1;
    while (team * ve * v < C) v *= 2;
    return {team, v};
}
// Workgroups of the backward pass: two to a CU, which the card holds at once, and at least 4 rows a team beside the
// partial sums.
int bwd_groups(int64_t N, int C, int dtype) {
    const int team = shape_of(C, dtype).team, teams = threads_of(team) / team;
    return (int)std::max<int64_t>(std::min<int64_t>((N + teams * 4 - 1) / (teams * 4), 512), 1);
}

bool types_ok(int dtype, int wtype) {
    return (dtype == DDM_F32 || dtype == DDM_F16 || dtype == DDM_BF16) && (wtype == DDM_F32 || wtype == dtype);
}

// The shapes that shape_of gives: of the wider teams only those that a smaller one does not hold.
template <class T>
constexpr bool reached(int team, int v) {
    const int most = team * v * 16 / (int)sizeof(T);
    return team == 64 ? most <= 1024 : team == 256 ? most > 1024 && most <= 4096 : most > 4096 && most <= 8192;
}
template <class T, class F>
void with_shape(Shape s, F f) {
    auto go = [&](auto team) {
        constexpr int TEAM = decltype(team)::value;
        if constexpr (reached<T>(TEAM, 1)) { if (s.v == 1) f(team, std::integral_constant<int, 1>{}); }
        if constexpr (reached<T>(TEAM, 2)) { if (s.v == 2) f(team, std::integral_constant<int, 2>{}); }
        if constexpr (reached<T>(TEAM, 4)) { if (s.v == 4) f(team, std::integral_constant<int, 4>{}); }
    };
    if (s.team == 64) go(std::integral_constant<int, 64>{});
    else if (s.team == 256) go(std::integral_constant<int, 256>{});
    else go(std::integral_constant<int, 512>{});
}

template <void (*KERNEL)(ResArgs), int TEAM>
void launch_rows(unsigned grid, size_t lds, hipStream_t stream, const ResArgs &a) {
    hipLaunchKernelGGL(KERNEL, dim3(grid), dim3(threads_of(TEAM)), lds, stream, a);
}

bool off(const void *p, int e) { return !p || (uintptr_t)p % e; }
bool odd(const void *p, int e) { return (uintptr_t)p % e; }

}  // namespace

extern "C" {

int ddm_residual_norm_forward(const void *x, int64_t ldx, const void *branch, int64_t ldb, const void *gate, int64_t ldg,
                              const void *scale, const void *branch_weight, const void *branch_bias, const void *weight,
                              const void *bias, int64_t N, int C, int dtype, int wtype, int branch_norm, int rms,
                              double eps, void *s, void *y, float *stats, hipStream_t stream) {
    if (!types_ok(dtype, wtype) || C < 1 || C > DDM_MAX_NORM_C) return DDM_ERR_UNSUPPORTED;
    const int e = esize(dtype), we = esize(wtype);
    if (N < 0 || N > INT_MAX || ldx < C || ldb < C || (gate && ldg < C) || !(eps >= 0) || !std::isfinite((float)eps)) return DDM_ERR_INVALID;
    if ((branch_norm != 0 && branch_norm != 1) || (rms != 0 && rms != 1)) return DDM_ERR_INVALID;
    if (!branch_norm && (branch_weight || branch_bias)) return DDM_ERR_INVALID;
    if (N == 0) return DDM_OK;
    if (off(x, e) || off(branch, e) || off(s, e) || off(y, e) || off(stats, 4) || odd(gate, e)) return DDM_ERR_INVALID;
    for (const void *w : {scale, branch_weight, branch_bias, weight, bias})
        if (odd(w, we)) return DDM_ERR_INVALID;
    ResArgs a{};
    a.x = x; a.branch = branch; a.gate = gate; a.scale = scale; a.bw = branch_weight; a.bb = branch_bias; a.w = weight; a.b = bias;
    a.s = s; a.y = y; a.stats = stats; a.ldx = ldx; a.ldb = ldb; a.ldg = ldg; a.N = N; a.C = C; a.eps = (float)eps; a.rms = rms;
    const Shape shape = shape_of(C, dtype);
    const int teams = threads_of(shape.team) / shape.team;
    const unsigned grid = (unsigned)std::min<int64_t>((N + teams - 1) / teams, shape.team == 64 ? 1024 : 2048);
    with_types(dtype, wtype, [&](auto t, auto w) {
        using T = decltype(t);
        using W = decltype(w);
        with_shape<T>(shape, [&](auto team, auto v) {
            constexpr int TEAM = decltype(team)::value, V = decltype(v)::value;
            constexpr size_t lds = Params<T, W, TEAM, V>::BYTES;
            if (branch_norm) launch_rows<residual_fwd_kernel<T, W, TEAM, V, true>, TEAM>(grid, 5 * lds, stream, a);
            else launch_rows<residual_fwd_kernel<T, W, TEAM, V, false>, TEAM>(grid, 3 * lds, stream, a);
        });
    });
    return hipGetLastError() == hipSuccess ? DDM_OK : DDM_ERR_HIP;
}

size_t ddm_residual_norm_backward_workspace_bytes(int64_t N, int C, int dtype, int branch_norm) {
    if (!types_ok(dtype, DDM_F32) || C < 1 || C > DDM_MAX_NORM_C || N < 0 || N > INT_MAX) return 0;
    return (size_t)bwd_groups(N, C, dtype) * (branch_norm ? 5 : 3) * C * sizeof(float);
}

int ddm_residual_norm_backward(const void *dy, const void *ds, const void *x, int64_t ldx, const void *branch, int64_t ldb,
                               const void *gate, int64_t ldg, const void *scale, const void *branch_weight,
                               const void *branch_bias, const void *weight, const float *stats, int64_t N, int C, int dtype,
                               int wtype, int branch_norm, int rms, void *dx, void *dbranch, void *dgate, void *dscale,
                               void *dbranch_weight, void *dbranch_bias, void *dweight, void *dbias, void *workspace,
                               size_t workspace_bytes, hipStream_t stream) {
    if (!types_ok(dtype, wtype) || C < 1 || C > DDM_MAX_NORM_C) return DDM_ERR_UNSUPPORTED;
    const int e = esize(dtype), we = esize(wtype);
    if (N < 0 || N > INT_MAX || ldx < C || ldb < C || (gate && ldg < C)) return DDM_ERR_INVALID;
    if ((branch_norm != 0 && branch_norm != 1) || (rms != 0 && rms != 1)) return DDM_ERR_INVALID;
    if (!branch_norm && (branch_weight || branch_bias || dbranch_weight || dbranch_bias)) return DDM_ERR_INVALID;
    if (dgate && !gate) return DDM_ERR_INVALID;
    if (N && (off(x, e) || off(branch, e) || off(stats, 4))) return DDM_ERR_INVALID;
    for (const void *t : {dy, ds, gate, (const void *)dx, (const void *)dbranch, (const void *)dgate})
        if (odd(t, e)) return DDM_ERR_INVALID;
    Sums sums{{dweight, dbias, dscale, dbranch_weight, dbranch_bias}};
    for (const void *t : {scale, branch_weight, branch_bias, weight})
        if (odd(t, we)) return DDM_ERR_INVALID;
    bool params = false;
    for (const void *t : sums.out) {
        if (odd(t, we)) return DDM_ERR_INVALID;
        params |= t != nullptr;
    }
    if (params && (off(workspace, 16) || workspace_bytes < ddm_residual_norm_backward_workspace_bytes(N, C, dtype, branch_norm)))
        return DDM_ERR_WORKSPACE;
    if (!params && (N == 0 || (!dx && !dbranch && !dgate))) return DDM_OK;
    ResArgs a{};
    a.x = x; a.branch = branch; a.gate = gate; a.dy = dy; a.ds = ds; a.scale = scale; a.bw = branch_weight; a.bb = branch_bias;
    a.w = weight; a.dx = dx; a.dbranch = dbranch; a.dgate = dgate; a.stats = const_cast<float *>(stats);
    a.part = (float *)workspace; a.ldx = ldx; a.ldb = ldb; a.ldg = ldg; a.N = N; a.C = C; a.rms = rms;
    const Shape shape = shape_of(C, dtype);
    const int groups = bwd_groups(N, C, dtype);            // without rows, one that leaves zeros
    with_types(dtype, wtype, [&](auto t, auto w) {
        using T = decltype(t);
        using W = decltype(w);
        with_shape<T>(shape, [&](auto team, auto v) {
            constexpr int TEAM = decltype(team)::value, V = decltype(v)::value;
            auto go = [&](auto bn, auto with_params) {
                constexpr bool BN = decltype(bn)::value, PARAMS = decltype(with_params)::value;
                constexpr size_t lds = Params<T, W, TEAM, V>::BYTES;
                launch_rows<residual_bwd_kernel<T, W, TEAM, V, BN, PARAMS>, TEAM>(groups, (BN || (PARAMS && TEAM == 64) ? 4 : 2) * lds, stream, a);
            };
            if (branch_norm) params ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
            else params ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
        });
        if (params)
            hipLaunchKernelGGL((residual_reduce_kernel<W>), dim3((C + 31) / 32, branch_norm ? 5 : 3), dim3(1024), 0, stream,
                               a.part, groups, branch_norm ? 5 : 3, C, sums);
    });
    return hipGetLastError() == hipSuccess ? DDM_OK : DDM_ERR_HIP;
}

}  // extern "C"

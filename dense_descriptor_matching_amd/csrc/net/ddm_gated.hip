// ddm_gated.hip -- gated linear layer (ddm_gated_linear_*).
//
//   g = x Wg^T + bg,  u = x Wu^T + bu,  h = act(g) u          (rows of W: the F of Wg, then the F of Wu)
//   dg = dh u act'(g),  du = dh act(g)
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x,  dbg = sum over rows of dg,  dbu = sum of du
#include "../../../include/ddm.h"
#include "ddm_gemm.hpp"
#include "ddm_row.hpp"

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

using namespace ddm;

namespace {

enum { FORWARD, BY_X, BY_W };                  // the three products

struct GatedArgs {
    const void *p, *q;                         // the product's operands
    int64_t ldp, ldq, ldo;                     // their row strides and the output's, elements
    int64_t seg_p, seg_q;                      // BY_X: from gate to up; BY_W: q alone
    int np, nq, k;                             // FORWARD: np = F pairs of rows
    int tiles_q, tiles_p, splits;
    const void *bias;
    void *out, *kept;
    float *part;                               // splits > 1: [split][output rows][outputs of a row]
    int act;
};

// act(g) and act'(g). sigmoid(g) = t: silu g t, gelu g Phi(g) with Phi the normal distribution's.
__device__ __forceinline__ float2 activation(float g, int kind) {
    if (kind == DDM_GELU) {
        const float phi = 0.5f * erfcf(g * -0.70710678118654752f);
        return {g * phi, __builtin_fmaf(g * 0.39894228040143268f, __expf(-0.5f * g * g), phi)};
    }
    const float t = __builtin_amdgcn_rcpf(1.f + __expf(-g));
    if (kind == DDM_SIGMOID) return {t, t * (1.f - t)};
    return {g * t, __builtin_fmaf(g * t, 1.f - t, t)};
}

// A wave's block of 32 rows q of W columns p, four neighbouring p at a time in a lane, to rows in memory: through LDS of
// its own, so that a row's columns are written together.
template <class T, int W>
struct Stage {
    static constexpr int PITCH = W * (int)sizeof(T) + 16, BYTES = 32 * PITCH, PE = 16 / (int)sizeof(T), NP = W / PE;
    __device__ static __forceinline__ void put(unsigned char *t, int lane, int sub, const f32x16 &c) {
        typedef T T4 __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
            const T4 v = {(T)c[r], (T)c[r + 1], (T)c[r + 2], (T)c[r + 3]};
            *reinterpret_cast<T4 *>(t + (lane & 31) * PITCH + (sub * 32 + 2 * r + 4 * (lane >> 5)) * (int)sizeof(T)) = v;
        }
    }
    // rows, cols: how many of the block's there are
    __device__ static __forceinline__ void store(const unsigned char *t, int lane, T *out, int64_t ld, int rows, int cols) {
        __builtin_amdgcn_wave_barrier();               // the wave's own writes and reads of LDS keep their order
#pragma unroll
        for (int i = 0; i < 32 * NP / 64; ++i) {
            const int r = (i * 64 + lane) / NP, c = (i * 64 + lane) % NP * PE;
            if (r >= rows || c >= cols) continue;
            const T *from = reinterpret_cast<const T *>(t + r * PITCH) + c;
            struct __attribute__((packed, aligned(sizeof(T)))) Out { T v[PE]; };
            struct __attribute__((aligned(16))) In { T v[PE]; };
            const In v = *reinterpret_cast<const In *>(from);
            T *to = out + r * ld + c;
            if (c + PE <= cols) {
                Out o;
#pragma unroll
                for (int e = 0; e < PE; ++e) o.v[e] = v.v[e];
                *reinterpret_cast<Out *>(to) = o;
            } else {
#pragma unroll
                for (int e = 0; e < PE; ++e)
                    if (c + e < cols) to[e] = v.v[e];
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
};

// WQ x WP waves of MQ x MP blocks of 32 x 32 outputs. FORWARD: half of a wave's blocks along p are of Wg, half of the
// same rows of Wu.
template <class T, int KIND, int WQ, int WP, int MQ, int MP>
__global__ __launch_bounds__(WQ *WP * 64) void gated_product_kernel(GatedArgs a) {
    constexpr int NW = WQ * WP, BQ = WQ * MQ * 32, BP = WP * MP * 32, BK = 128 / (int)sizeof(T);
    using P = Side<T, BP, KIND != FORWARD, NW>;
    using Q = Side<T, BQ, KIND == BY_W, NW>;
    constexpr int STEP = P::BYTES + Q::BYTES;
    constexpr int W = (KIND == FORWARD ? MP / 2 : MP) * 32;            // columns of a wave's outputs
    constexpr int LDS = 2 * STEP > NW * Stage<T, W>::BYTES ? 2 * STEP : NW * Stage<T, W>::BYTES;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[LDS];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wq = w / WP, wp = w % WP;
    const int tiles = a.tiles_q * a.tiles_p, split = blockIdx.x / tiles;
    TileAt t = tile_at(blockIdx.x - split * tiles, a.tiles_q, a.tiles_p);
    // BY_W: the upper half of the tiles along q is that of dWu
    const int part = KIND == BY_W && t.q >= a.tiles_q / 2;
    if (part) t.q -= a.tiles_q / 2;
    constexpr int PAIRS = KIND == FORWARD ? BP / 2 : BP;
    const int q0 = t.q * BQ, p0 = t.p * PAIRS;
    const int per = (a.k + BK - 1) / BK, all = KIND == BY_X ? 2 * per : per;
    const int each = (all + a.splits - 1) / a.splits, begin = split * each, end = min(begin + each, all);

    P feed_p;
    Q feed_q;
    auto start = [&](int step) {                                       // at step `step` of all
        const int seg = KIND == BY_X && step >= per, s = step - seg * per, k = s * BK;
        const T *p = (const T *)a.p, *q = (const T *)a.q + part * a.seg_q;
        if (KIND == BY_X) { p += seg * a.seg_p; q += seg * a.seg_q; }
        if constexpr (KIND == FORWARD) {
            feed_p.start(p + p0 * a.ldp + k, a.ldp, a.k - k, 0, w, lane, [&](int i) {
                const int sub = i / 32 % MP, f = i / 32 / MP * (MP / 2 * 32) + sub % (MP / 2) * 32 + i % 32;
                return p0 + f < a.np ? (int64_t)f + (sub >= MP / 2 ? a.np : 0) : -1;
            });
        } else {
            feed_p.start(p + k * a.ldp + p0, a.ldp, a.k - k, a.np - p0, w, lane, [](int) { return -1; });
        }
        if constexpr (KIND == BY_W) {
            feed_q.start(q + k * a.ldq + q0, a.ldq, a.k - k, a.nq - q0, w, lane, [](int) { return -1; });
        } else {
            feed_q.start(q + q0 * a.ldq + k, a.ldq, a.k - k, 0, w, lane, [&](int i) { return q0 + i < a.nq ? i : -1; });
        }
    };
    auto next = [&](int step, unsigned char *to) {
        if (KIND == BY_X && step == per) start(step);
        feed_q.next(to, w, lane);
        feed_p.next(to + Q::BYTES, w, lane);
    };

    f32x16 c[MQ][MP];
#pragma unroll
    for (int i = 0; i < MQ; ++i)
#pragma unroll
        for (int j = 0; j < MP; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) c[i][j][r] = 0.f;
    const int at_q = Q::frag_base(lane), at_p = P::frag_base(lane);
    if (begin < end) {
        start(begin);
        next(begin, lds);
    }
    for (int step = begin; step < end; ++step) {
        const unsigned char *now = lds + ((step - begin) & 1) * STEP;
        tiles_ready();
        if (step + 1 < end) next(step + 1, lds + ((step + 1 - begin) & 1) * STEP);
#pragma unroll
        for (int s = 0; s < BK / 16; ++s) {
            Frag<T> fq[MQ], fp[MP];
#pragma unroll
            for (int i = 0; i < MQ; ++i) fq[i] = Q::frag(now, at_q, wq * MQ + i, s);
#pragma unroll
            for (int j = 0; j < MP; ++j) fp[j] = P::frag(now + Q::BYTES, at_p, wp * MP + j, s);
#pragma unroll
            for (int i = 0; i < MQ; ++i)
#pragma unroll
                for (int j = 0; j < MP; ++j) mma(c[i][j], fp[j], fq[i]);
        }
    }

    // lane: row q of block i, columns 8 (r / 4) + 4 h + r % 4 of block j
    const int h = lane >> 5;
    const int first_q = q0 + wq * MQ * 32, first_p = p0 + wp * W, out_q = part * a.nq;
    if (a.splits > 1) {
        // FORWARD: all of g, then all of u
        const int64_t rows = KIND == BY_W ? 2 * (int64_t)a.nq : a.nq, width = KIND == FORWARD ? 2 * (int64_t)a.np : a.np;
        float *to = a.part + split * rows * width;
#pragma unroll
        for (int i = 0; i < MQ; ++i) {
            const int q = first_q + i * 32 + (lane & 31);
            if (q >= a.nq) continue;
#pragma unroll
            for (int j = 0; j < MP; ++j) {
                const bool up = KIND == FORWARD && j >= MP / 2;
                float *row = to + (out_q + q) * width + (up ? a.np : 0);
#pragma unroll
                for (int r = 0; r < 16; r += 4) {
                    const int p = first_p + (up ? j - MP / 2 : j) * 32 + 2 * r + 4 * h;
                    const float v[4] = {c[i][j][r], c[i][j][r + 1], c[i][j][r + 2], c[i][j][r + 3]};
                    store_chunk<float, 4>(row, p, a.np, v);
                }
            }
        }
        return;
    }
    __syncthreads();                                                   // the last step's tiles have been read
    unsigned char *mine = lds + w * Stage<T, W>::BYTES;
    const T *bias = (const T *)a.bias;
#pragma unroll
    for (int i = 0; i < MQ; ++i) {
        const int q = first_q + i * 32, rows = a.nq - q, cols = a.np - first_p;
        T *out = (T *)a.out + (int64_t)(out_q + q) * a.ldo + first_p;
        if constexpr (KIND == FORWARD) {
            if (bias) {
#pragma unroll
                for (int j = 0; j < MP; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int f = first_p + j % (MP / 2) * 32 + r / 4 * 8 + 4 * h + r % 4;
                        c[i][j][r] += (float)bias[min(f, a.np - 1) + (j >= MP / 2 ? a.np : 0)];
                    }
            }
            if (a.kept) {
                T *to = (T *)a.kept + (int64_t)q * (2 * (int64_t)a.np) + first_p;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int j = 0; j < MP / 2; ++j) Stage<T, W>::put(mine, lane, j, c[i][half * (MP / 2) + j]);
                    Stage<T, W>::store(mine, lane, to + (half ? a.np : 0), 2 * (int64_t)a.np, rows, cols);
                }
            }
#pragma unroll
            for (int j = 0; j < MP / 2; ++j) {
                f32x16 y;
#pragma unroll
                for (int r = 0; r < 16; ++r) y[r] = activation(c[i][j][r], a.act).x * c[i][j + MP / 2][r];
                Stage<T, W>::put(mine, lane, j, y);
            }
        } else {
#pragma unroll
            for (int j = 0; j < MP; ++j) Stage<T, W>::put(mine, lane, j, c[i][j]);
        }
        Stage<T, W>::store(mine, lane, out, a.ldo, rows, cols);
    }
}

// The sums of all splits, n = rows * width of them, in their order.
template <class T>
__global__ __launch_bounds__(256) void gated_join_kernel(const float *part, int splits, int64_t n, T *out) {
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n; i += (int64_t)gridDim.x * 1024) {
        float sum[4] = {};
        if (i + 4 <= n) {
            for (int s = 0; s < splits; ++s) {
                struct __attribute__((packed, aligned(4))) Raw { float v[4]; };
                const Raw r = *reinterpret_cast<const Raw *>(part + s * n + i);
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] += r.v[e];
            }
            struct __attribute__((packed, aligned(sizeof(T)))) Out { T v[4]; } o;
#pragma unroll
            for (int e = 0; e < 4; ++e) o.v[e] = (T)sum[e];
            *reinterpret_cast<Out *>(out + i) = o;
        } else {
            for (int64_t j = i; j < n; ++j) {
                float total = 0.f;
                for (int s = 0; s < splits; ++s) total += part[s * n + j];
                out[j] = (T)total;
            }
        }
    }
}
// The same for the forward pass, with what its product does at its end.
template <class T>
__global__ __launch_bounds__(256) void gated_join_forward_kernel(GatedArgs a) {
    const int64_t n = (int64_t)a.nq * a.np;
    const T *bias = (const T *)a.bias;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t q = i / a.np;
        const int p = (int)(i - q * a.np);
        float g = 0.f, u = 0.f;
        const float *from = a.part + q * 2 * a.np + p;
        for (int s = 0; s < a.splits; ++s) {
            g += from[s * 2 * n];
            u += from[s * 2 * n + a.np];
        }
        if (bias) { g += (float)bias[p]; u += (float)bias[p + a.np]; }
        if (a.kept) {
            T *kept = (T *)a.kept + q * 2 * a.np + p;
            kept[0] = (T)g;
            kept[a.np] = (T)u;
        }
        ((T *)a.out)[i] = (T)(activation(g, a.act).x * u);
    }
}

// Rows of at most 32 MQ tokens: the weights' bytes count. A workgroup takes 16 columns of h, as a block of 16 rows of Wg
// and the same 16 of Wu; its waves share k, each reading its rows' pieces straight into the operands' registers. In the
// block, rows 8..15 and 24..31 are those of Wu: a lane then holds g and u of the same columns.
template <class T, int MQ, int NW>
__global__ __launch_bounds__(NW * 64) void gated_tokens_kernel(GatedArgs a) {
    constexpr int PE = 16 / (int)sizeof(T), BK = 128 / (int)sizeof(T), PIECES = 8 / PE;
    __shared__ f32x16 sums[NW][MQ][64];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5, i = lane & 31;
    const int f0 = blockIdx.x * 16, f = f0 + (i & 7) + (i >> 4) * 8;
    const bool up = i & 8;
    const auto bp = buffer_of((const T *)a.p + f0 * a.ldp, OUTSIDE), bq = buffer_of(a.q, OUTSIDE);
    const int row_p = f < a.np ? (int)((f - f0 + (up ? (int64_t)a.np : 0)) * a.ldp * (int64_t)sizeof(T)) : OUTSIDE;
    int row_q[MQ];
#pragma unroll
    for (int j = 0; j < MQ; ++j) row_q[j] = j * 32 + i < a.nq ? (int)((j * 32 + i) * a.ldq * (int64_t)sizeof(T)) : OUTSIDE;
    f32x16 c[MQ];
#pragma unroll
    for (int j = 0; j < MQ; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) c[j][r] = 0.f;
    // the operand of k positions k + 8 h .. k + 8 h + 7
    auto load = [&](__amdgpu_buffer_rsrc_t b, int row, int k) {
        union { u32x4 v[PIECES]; Frag<T> f; } u;
#pragma unroll
        for (int s = 0; s < PIECES; ++s) {
            const int at = k + 8 * h + s * PE;
            u.v[s] = __builtin_amdgcn_raw_buffer_load_b128(b, row != OUTSIDE && at < a.k ? row + at * (int)sizeof(T) : OUTSIDE, 0, 0);
        }
        return u.f;
    };
    for (int k = w * BK; k < a.k; k += NW * BK) {
        Frag<T> fp[BK / 16], fq[MQ][BK / 16];
#pragma unroll
        for (int s = 0; s < BK / 16; ++s) {
            fp[s] = load(bp, row_p, k + 16 * s);
#pragma unroll
            for (int j = 0; j < MQ; ++j) fq[j][s] = load(bq, row_q[j], k + 16 * s);
        }
#pragma unroll
        for (int s = 0; s < BK / 16; ++s)
#pragma unroll
            for (int j = 0; j < MQ; ++j) mma(c[j], fp[s], fq[j][s]);
    }
#pragma unroll
    for (int j = 0; j < MQ; ++j) sums[w][j][lane] = c[j];
    __syncthreads();
    // 16 columns of 32 MQ rows: a thread takes pairs (g, u) of one row and column
    const T *bias = (const T *)a.bias;
    for (int n = threadIdx.x; n < MQ * 32 * 16; n += NW * 64) {
        const int col = n % 16, q = n / 16, p = f0 + col;
        if (q >= a.nq || p >= a.np) continue;
        // column col of g is row m = col % 8 + 16 (col / 8) of the block: half (m / 4) % 2, element 4 (m / 8) + m % 4
        const int m = col % 8 + col / 8 * 16, at = (m / 4 & 1) * 32 + q % 32, r = m / 8 * 4 + m % 4;
        float g = 0.f, u = 0.f;
#pragma unroll
        for (int s = 0; s < NW; ++s) {
            const float *from = reinterpret_cast<const float *>(&sums[s][q / 32][at]);
            g += from[r];
            u += from[r + 4];
        }
        if (bias) { g += (float)bias[p]; u += (float)bias[p + a.np]; }
        if (a.kept) {
            T *kept = (T *)a.kept + (int64_t)q * 2 * a.np + p;
            kept[0] = (T)g;
            kept[a.np] = (T)u;
        }
        ((T *)a.out)[(int64_t)q * a.ldo + p] = (T)(activation(g, a.act).x * u);
    }
}

struct SlopeArgs {
    const void *dh, *kept;
    void *dp;                                  // [N][2][pitch]
    float *part;                               // [rows' workgroup][2][F], or NULL
    int64_t N;
    int F, pitch, act, rows;                   // rows of a workgroup
};

// dg and du from dh and the projections; the columns' sums over a workgroup's rows. A thread has eight columns, a wave
// 512, and the workgroup's four waves every fourth row.
template <class T>
__global__ __launch_bounds__(256) void gated_slope_kernel(SlopeArgs a) {
    constexpr int VE = 8;
    __shared__ float sums[4][2][64 * VE];
    const int across = (a.pitch + 64 * VE - 1) / (64 * VE), group = blockIdx.x / across, block = blockIdx.x % across;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, c = (block * 64 + lane) * VE;
    const int64_t first = (int64_t)group * a.rows, last = min(first + a.rows, a.N);
    float sg[VE] = {}, su[VE] = {};
    if (c < a.pitch)
        for (int64_t n = first + w; n < last; n += 4) {
            float d[VE], g[VE], u[VE];
            load_chunk<T, VE>((const T *)a.dh + n * a.F, c, a.F, d);
            load_chunk<T, VE>((const T *)a.kept + n * 2 * a.F, c, a.F, g);
            load_chunk<T, VE>((const T *)a.kept + n * 2 * a.F + a.F, c, a.F, u);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float2 s = activation(g[e], a.act);
                g[e] = d[e] * u[e] * s.y;      // past column F all three are zeros
                u[e] = d[e] * s.x;
                sg[e] += g[e];
                su[e] += u[e];
            }
            store_chunk<T, VE>((T *)a.dp + n * 2 * a.pitch, c, a.pitch, g);
            store_chunk<T, VE>((T *)a.dp + n * 2 * a.pitch + a.pitch, c, a.pitch, u);
        }
    if (!a.part) return;
#pragma unroll
    for (int e = 0; e < VE; ++e) {
        sums[w][0][lane * VE + e] = sg[e];
        sums[w][1][lane * VE + e] = su[e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * 64 * VE; i += 256) {
        const int half = i / (64 * VE), j = i % (64 * VE), col = block * 64 * VE + j;
        if (col < a.F)
            a.part[((int64_t)group * 2 + half) * a.F + col] = (sums[0][half][j] + sums[1][half][j]) + (sums[2][half][j] + sums[3][half][j]);
    }
}

// The bias' gradient from the workgroups' sums: 32 columns a workgroup, 32 of its threads share a column.
template <class T>
__global__ __launch_bounds__(1024) void gated_bias_kernel(const float *part, int parts, int cols, T *out) {
    __shared__ float s[32][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
    float sum = 0.f;
    if (c < cols)
        for (int n = g; n < parts; n += 32) sum += part[(int64_t)n * cols + c];
    s[g][threadIdx.x & 31] = sum;
    __syncthreads();
    if (g == 0 && c < cols) {
        float total = 0.f;
        for (int k = 0; k < 32; ++k) total += s[k][threadIdx.x];
        out[c] = (T)total;
    }
}

// Rows of any address as rows of `pitch` elements, with zeros behind the C.
template <class T>
__global__ __launch_bounds__(256) void gated_repack_kernel(const T *in, int64_t ld, int64_t rows, int C, int pitch, T *out) {
    constexpr int VE = 16 / sizeof(T);
    const int per = pitch / VE;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * per; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per;
        const int c = (int)(i - r * per) * VE;
        float v[VE];
        load_chunk<T, VE>(in + r * ld, c, C, v);
        store_chunk<T, VE>(out + r * pitch, c, pitch, v);
    }
}

template <class T>
__global__ __launch_bounds__(256) void gated_zero_kernel(T *out, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) out[i] = (T)0.f;
}

// ------------------------------------------------------------------------------------------------------- host side
int esize(int dtype) { return dtype == DDM_F32 ? 4 : 2; }
int padded(int n, int dtype) { const int pe = 16 / esize(dtype); return (n + pe - 1) / pe * pe; }
size_t whole(size_t bytes) { return (bytes + 255) / 256 * 256; }

int check(int64_t N, int C, int F, int dtype) {
    if (dtype != DDM_F32 && dtype != DDM_F16 && dtype != DDM_BF16) return DDM_ERR_UNSUPPORTED;
    if (C < 1 || C > DDM_MAX_GATED || F < 1 || F > DDM_MAX_GATED) return DDM_ERR_UNSUPPORTED;
    if (N < 0 || N > DDM_MAX_GATED_ROWS) return DDM_ERR_INVALID;
    // a launch has fewer than 2^32 threads
    if ((N + 127) / 128 * ((std::max(2 * (int64_t)F, (int64_t)C) + 127) / 128) >= 1 << 24) return DDM_ERR_INVALID;
    // a row of Wu lies within 31-bit offsets of one of Wg
    if ((int64_t)F * padded(C, dtype) * esize(dtype) >= 1 << 30) return DDM_ERR_INVALID;
    return DDM_OK;
}

// How a product is cut up: tiles of bq x bp outputs, splits of k.
struct Cut { int bq, bp, splits; };
Cut cut_of(int kind, int64_t nq, int64_t np, int64_t k, int dtype) {
    // np, nq: the whole output's (FORWARD: 2 F)
    auto tiles = [&](int bq, int bp) { return ((nq + bq - 1) / bq) * ((np + bp - 1) / bp); };
    Cut c = tiles(256, 256) >= 192 && dtype != DDM_F32 ? Cut{256, 256, 1} : Cut{128, 128, 1};
    const int64_t n = std::max<int64_t>(tiles(c.bq, c.bp), 1), steps = k * esize(dtype) / 128 + 1;     // no rows: nothing is launched
    const int64_t places = c.bq == 256 ? 256 : 512;
    c.splits = (int)std::max<int64_t>(1, std::min<int64_t>(places / n, steps / 8));
    return c;
}
Cut cut_forward(int64_t N, int C, int F, int dtype) { return cut_of(FORWARD, N, 2 * (int64_t)F, C, dtype); }
Cut cut_by_x(int64_t N, int C, int F, int dtype) { return cut_of(BY_X, N, C, 2 * (int64_t)F, dtype); }
Cut cut_by_w(int64_t N, int C, int F, int dtype) { return cut_of(BY_W, 2 * (int64_t)F, C, N, dtype); }

constexpr int TOKENS = 64;                     // rows of gated_tokens_kernel

size_t repacked(int64_t rows, int C, int dtype) { return whole((size_t)rows * padded(C, dtype) * esize(dtype)); }
size_t parts_bytes(const Cut &c, int64_t rows, int64_t width) { return c.splits > 1 ? whole((size_t)c.splits * rows * width * 4) : 0; }

constexpr int SLOPE_ROWS = 128;
int64_t slope_groups(int64_t N) { return (N + SLOPE_ROWS - 1) / SLOPE_ROWS; }

// Workspaces, in order. Both operands' repacked rows have room whether or not they are needed: that depends on addresses.
struct ForwardPlan { Cut cut; size_t x, w, part, bytes; };
ForwardPlan forward_plan(int64_t N, int C, int F, int dtype) {
    ForwardPlan p{};
    if (N > TOKENS) p.cut = cut_forward(N, C, F, dtype);
    p.w = repacked(N, C, dtype);
    p.part = p.w + (C % (16 / esize(dtype)) ? repacked(2 * (int64_t)F, C, dtype) : 0);
    p.bytes = p.part + (N > TOKENS ? parts_bytes(p.cut, N, 2 * (int64_t)F) : 0);
    return p;
}

template <class F>
void with_type(int dtype, F f) {
    if (dtype == DDM_F32) f(float{});
    else if (dtype == DDM_F16) f(_Float16{});
    else f(__bf16{});
}

template <class T, int KIND>
void launch_product(GatedArgs a, const Cut &c, hipStream_t s) {
    const int pairs = KIND == FORWARD ? c.bp / 2 : c.bp;
    a.tiles_q = (a.nq + c.bq - 1) / c.bq * (KIND == BY_W ? 2 : 1);
    a.tiles_p = (a.np + pairs - 1) / pairs;
    a.splits = c.splits;
    const dim3 grid((unsigned)((int64_t)a.tiles_q * a.tiles_p * a.splits));
    if constexpr (sizeof(T) == 2) {
        if (c.bq == 256) {
            hipLaunchKernelGGL((gated_product_kernel<T, KIND, 2, 4, 4, 2>), grid, dim3(512), 0, s, a);
            return;
        }
    }
    hipLaunchKernelGGL((gated_product_kernel<T, KIND, 2, 2, 2, 2>), grid, dim3(256), 0, s, a);
}

unsigned blocks(int64_t items, int64_t each) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>((items + each - 1) / each, 8192)); }

// x or the weight as rows of whole 16-byte pieces: themselves, or a copy in the workspace.
template <class T>
const T *whole_rows(const void *from, int64_t &ld, int64_t rows, int C, void *copy, hipStream_t s) {
    constexpr int PE = 16 / sizeof(T);
    if ((uintptr_t)from % 16 == 0 && C % PE == 0 && (ld % PE == 0 || rows == 1)) return (const T *)from;
    const int pitch = (C + PE - 1) / PE * PE;
    hipLaunchKernelGGL((gated_repack_kernel<T>), dim3(blocks(rows * (pitch / PE), 256)), dim3(256), 0, s, (const T *)from, ld, rows, C, pitch, (T *)copy);
    ld = pitch;
    return (const T *)copy;
}

bool bad_act(int act) { return act != DDM_SILU && act != DDM_GELU && act != DDM_SIGMOID; }
bool bad_stride(int64_t ld, int C, int e) { return ld < C || ld * e > 1 << 22; }
bool off(const void *p, int e) { return !p || (uintptr_t)p % e; }

}  // namespace

extern "C" {

size_t ddm_gated_linear_forward_workspace_bytes(int64_t N, int C, int F, int dtype) {
    if (check(N, C, F, dtype) != DDM_OK) return 0;
    return std::max<size_t>(forward_plan(N, C, F, dtype).bytes, 16);
}

int ddm_gated_linear_forward(const void *x, int64_t ldx, const void *weight, const void *bias, int64_t N, int C, int F, int dtype,
                             int activation, void *h, void *kept, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if (int rc = check(N, C, F, dtype)) return rc;
    const int e = esize(dtype);
    if (bad_act(activation) || bad_stride(ldx, C, e)) return DDM_ERR_INVALID;
    if (N == 0) return DDM_OK;
    if (off(x, e) || off(weight, 16) || off(h, e) || (uintptr_t)bias % e || (uintptr_t)kept % e) return DDM_ERR_INVALID;
    const ForwardPlan pl = forward_plan(N, C, F, dtype);
    if (off(workspace, 16) || workspace_bytes < pl.bytes) return DDM_ERR_WORKSPACE;
    char *ws = (char *)workspace;
    with_type(dtype, [&](auto t) {
        using T = decltype(t);
        GatedArgs a{};
        a.ldq = ldx; a.ldp = C; a.ldo = F;
        a.q = whole_rows<T>(x, a.ldq, N, C, ws, stream);
        a.p = whole_rows<T>(weight, a.ldp, 2 * (int64_t)F, C, ws + pl.w, stream);
        a.np = F; a.nq = (int)N; a.k = C; a.bias = bias; a.out = h; a.kept = kept; a.act = activation;
        a.part = (float *)(ws + pl.part); a.splits = 1;
        if (N <= 32) hipLaunchKernelGGL((gated_tokens_kernel<T, 1, 8>), dim3((F + 15) / 16), dim3(512), 0, stream, a);
        else if (N <= TOKENS) hipLaunchKernelGGL((gated_tokens_kernel<T, 2, 8>), dim3((F + 15) / 16), dim3(512), 0, stream, a);
        else {
            launch_product<T, FORWARD>(a, pl.cut, stream);
            a.splits = pl.cut.splits;
            if (a.splits > 1)
                hipLaunchKernelGGL((gated_join_forward_kernel<T>), dim3(blocks(N * F, 256)), dim3(256), 0, stream, a);
        }
    });
    return hipGetLastError() == hipSuccess ? DDM_OK : DDM_ERR_HIP;
}

}  // extern "C"

namespace {

struct BackPlan { Cut by_x, by_w; size_t x, w, dp, bias, part, bytes; };
BackPlan back_plan(int64_t N, int C, int F, int dtype) {
    BackPlan p{};
    p.by_x = cut_by_x(N, C, F, dtype);
    p.by_w = cut_by_w(N, C, F, dtype);
    p.w = repacked(N, C, dtype);
    p.dp = p.w + (C % (16 / esize(dtype)) ? repacked(2 * (int64_t)F, C, dtype) : 0);
    p.bias = p.dp + whole((size_t)N * 2 * padded(F, dtype) * esize(dtype));
    p.part = p.bias + whole((size_t)slope_groups(N) * 2 * F * 4);
    p.bytes = p.part + std::max(parts_bytes(p.by_x, N, C), parts_bytes(p.by_w, 2 * (int64_t)F, C));
    return p;
}

}  // namespace

extern "C" {

size_t ddm_gated_linear_backward_workspace_bytes(int64_t N, int C, int F, int dtype) {
    if (check(N, C, F, dtype) != DDM_OK) return 0;
    return std::max<size_t>(back_plan(N, C, F, dtype).bytes, 16);
}

int ddm_gated_linear_backward(const void *dh, const void *x, int64_t ldx, const void *weight, const void *kept, int64_t N, int C,
                              int F, int dtype, int activation, void *dx, void *dweight, void *dbias, void *workspace,
                              size_t workspace_bytes, hipStream_t stream) {
    if (int rc = check(N, C, F, dtype)) return rc;
    const int e = esize(dtype);
    if (bad_act(activation) || bad_stride(ldx, C, e)) return DDM_ERR_INVALID;
    if (N && (off(dh, e) || off(kept, e) || (dweight && off(x, e)) || (dx && off(weight, 16)))) return DDM_ERR_INVALID;
    if ((uintptr_t)dx % e || (uintptr_t)dweight % e || (uintptr_t)dbias % e) return DDM_ERR_INVALID;
    const BackPlan pl = back_plan(N, C, F, dtype);
    if (off(workspace, 16) || workspace_bytes < pl.bytes) return DDM_ERR_WORKSPACE;
    if (!dx && !dweight && !dbias) return DDM_OK;
    char *ws = (char *)workspace;
    with_type(dtype, [&](auto t) {
        using T = decltype(t);
        if (N == 0) {
            if (dweight) hipLaunchKernelGGL((gated_zero_kernel<T>), dim3(blocks(2 * (int64_t)F * C, 256)), dim3(256), 0, stream, (T *)dweight, 2 * (int64_t)F * C);
            if (dbias) hipLaunchKernelGGL((gated_zero_kernel<T>), dim3(blocks(2 * (int64_t)F, 256)), dim3(256), 0, stream, (T *)dbias, 2 * (int64_t)F);
            return;
        }
        SlopeArgs sl{};
        sl.dh = dh; sl.kept = kept; sl.dp = ws + pl.dp; sl.part = dbias ? (float *)(ws + pl.bias) : nullptr;
        sl.N = N; sl.F = F; sl.pitch = padded(F, dtype); sl.act = activation; sl.rows = SLOPE_ROWS;
        hipLaunchKernelGGL((gated_slope_kernel<T>), dim3((unsigned)((sl.pitch + 511) / 512 * slope_groups(N))), dim3(256), 0, stream, sl);
        if (dbias)
            hipLaunchKernelGGL((gated_bias_kernel<T>), dim3((2 * F + 31) / 32), dim3(1024), 0, stream, sl.part, (int)slope_groups(N), 2 * F, (T *)dbias);
        GatedArgs a{};
        a.part = (float *)(ws + pl.part);
        a.ldo = C; a.np = C; a.ldq = 2 * (int64_t)sl.pitch; a.q = sl.dp; a.seg_q = sl.pitch;
        auto join = [&](int64_t n, void *out) {
            if (a.splits > 1)
                hipLaunchKernelGGL((gated_join_kernel<T>), dim3(blocks(n, 1024)), dim3(256), 0, stream, a.part, a.splits, n, (T *)out);
        };
        if (dx) {
            a.ldp = C;
            a.p = whole_rows<T>(weight, a.ldp, 2 * (int64_t)F, C, ws + pl.w, stream);
            a.seg_p = F * a.ldp; a.nq = (int)N; a.k = F; a.out = dx; a.splits = pl.by_x.splits;
            launch_product<T, BY_X>(a, pl.by_x, stream);
            join(N * C, dx);
        }
        if (dweight) {
            a.ldp = ldx;
            a.p = whole_rows<T>(x, a.ldp, N, C, ws, stream);
            a.nq = F; a.k = (int)N; a.out = dweight; a.splits = pl.by_w.splits;
            launch_product<T, BY_W>(a, pl.by_w, stream);
            join(2 * (int64_t)F * C, dweight);
        }
    });
    return hipGetLastError() == hipSuccess ? DDM_OK : DDM_ERR_HIP;
}

}  // extern "C"

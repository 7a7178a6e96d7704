// ddm_gated.hip -- gated linear layer (ddm_gated_linear_*).
//
//   g = x Wg^T + bg,  u = x Wu^T + bu,  h = act(g) u          (rows of W: the F of Wg, then the F of Wu)
//   dg = dh u act'(g),  du = dh act(g)
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x,  dbg = sum over rows of dg,  dbu = sum of du
//
// Bound by the matrix cores with rows, by the weight's bytes with single tokens. The forward product takes rows of Wg and the same
// rows of Wu into one tile, so that a lane has g and u of an element and finishes it in registers. The gradient makes dg and du in a
// pass over memory (each is an operand of two products, and rounding them to the inputs' type is what the matrix cores take) and then
// runs two more products from the same loop. Measured, 24576 x 1024 to 2736 bf16 (275 GFLOP a product; a product of 8192^3 reaches
// 1454 TFLOP/s here, the library takes 329, 229 and 389 us for the three): forward with g and u kept 350 us (a tile's three outputs
// are written while no matrix core works: 250 without them), dg and du 158 us behind it (672 MB, 4.3 TB/s; 144 where g and u are in
// the caches, which that forward's outputs pass by), by x 270 + 14 us to join tiles cut along k, by W 265 + 24. 256 tiles in step take
// 1.45 to 1.6 us for 64 of k, 32 tiles 1.1: where all CUs work, memory and power count. Tiles of 128 everywhere: 435, 354 and 320 us;
// 64 of k a step with two steps ahead: 385, 332, 313.
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
    int tiles_q, tiles_p;
    Shares cut;
    const void *bias;
    void *out, *kept;
    f32x4 *part;                               // slots of a tile's sums
    const float *unit;                         // float16, BY_X and BY_W: what one of dg and du as held stands for
    int act;
    bool past_l2;                              // FORWARD: outputs are more than the L2s hold (32 MB)
};

// act(g) and act'(g). sigmoid(g) = t: silu g t, gelu g Phi(g) with Phi the normal distribution's: with z = |g| / sqrt 2 and
// t = 1 / (1 + z / 2), Phi(-|g|) = erfc(z) / 2 = exp(-z^2) t p(t) / 2, where the polynomial p (fitted to erfcx(z) / t with the
// least relative error over 0 <= z <= 14) is off by 9.4e-8 of its value, so that tails keep their digits. The products' ends
// are as long as these formulas: the library's erfc took 43 us for 1536 x 1024 to 2736, this one 35.
// The exponential's argument, rounded twice, is off by up to 2^-24 g^2: 2^-17 of the value at |g| = 13. In 16 bits that is below
// a hundredth of a rounding; for T = float its rest is carried along (five instructions more; what is left is 2^-21).
template <class T>
__device__ __forceinline__ float2 activation(float g, int kind) {
    if (kind == DDM_GELU) {
        const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(fabsf(g), 0.35355339059327376f, 1.f));
        float e;
        if constexpr (sizeof(T) == 4) {
            const float z = fminf(fabsf(g), 16.f), s = z * z, c = -0.72134752044448170f;       // at 16 it is 0; no infinity less infinity
            const float a = s * c, rest = __builtin_fmaf(__builtin_fmaf(z, z, -s), c, __builtin_fmaf(s, c, -a));
            e = exp2_fast(a);
            e = __builtin_fmaf(e * 0.69314718f, __builtin_fmaf(s, -9.6298144e-9f, rest), e);     // the last of c in 32 bits
        } else {
            e = exp2_fast(g * g * -0.72134752044448170f);
        }
        float q = -0.0593863577f;
        q = __builtin_fmaf(q, t, 0.286123514f);
        q = __builtin_fmaf(q, t, -0.490405619f);
        q = __builtin_fmaf(q, t, 0.281732619f);
        q = __builtin_fmaf(q, t, -0.0291482322f);
        q = __builtin_fmaf(q, t, 0.203752473f);
        q = __builtin_fmaf(q, t, 0.242835104f);
        q = __builtin_fmaf(q, t, 0.282412112f);
        q = __builtin_fmaf(q, t, 0.282084346f);
        const float below = 0.5f * q * t * e, phi = g < 0.f ? below : 1.f - below;
        return {g * phi, __builtin_fmaf(g * 0.39894228040143268f, e, phi)};
    }
    const float t = __builtin_amdgcn_rcpf(1.f + exp2_fast(g * -1.4426950408889634f));
    // sigmoid(-g) by itself: 1 - t has lost its digits where t is near one. (The products' ends take the value alone.)
    if (kind == DDM_SIGMOID) return {t, t * __builtin_amdgcn_rcpf(1.f + exp2_fast(g * 1.4426950408889634f))};
    return {g * t, __builtin_fmaf(g * t, 1.f - t, t)};
}

// past_l2: through the L2 without staying there, for outputs larger than it that would push out what is read again.
template <int ALIGN>
__device__ __forceinline__ void store16(void *to, Bytes16Of16 v, bool past_l2) {
    if (past_l2) __builtin_nontemporal_store((Bytes16<ALIGN>)v, reinterpret_cast<Bytes16<ALIGN> *>(to));
    else *reinterpret_cast<Bytes16<ALIGN> *>(to) = v;
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
    __device__ static __forceinline__ void store(const unsigned char *t, int lane, T *out, int64_t ld, int rows, int cols, bool past_l2 = false) {
        __builtin_amdgcn_wave_barrier();               // the wave's own writes and reads of LDS keep their order
#pragma unroll
        for (int i = 0; i < 32 * NP / 64; ++i) {
            const int r = (i * 64 + lane) / NP, c = (i * 64 + lane) % NP * PE;
            if (r >= rows || c >= cols) continue;
            const T *from = reinterpret_cast<const T *>(t + r * PITCH) + c;
            const u32x4 v = *reinterpret_cast<const Bytes16<16> *>(from);
            T *to = out + r * ld + c;
            if (c + PE <= cols) {
                store16<sizeof(T)>(to, v, past_l2);
            } else {
#pragma unroll
                for (int e = 0; e < PE; ++e)
                    if (c + e < cols) to[e] = from[e];
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
};

// N matrix instructions with so many reads of LDS and loads between them, evenly, so that none waits for all of the
// others.
template <int N, int READS, int LOADS, int I = 0>
__device__ __forceinline__ void interleave() {
    constexpr int reads = (I + 1) * READS / N - I * READS / N, loads = (I + 1) * LOADS / N - I * LOADS / N;
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (reads > 0) __builtin_amdgcn_sched_group_barrier(0x100, reads, 0);
    if constexpr (loads > 0) __builtin_amdgcn_sched_group_barrier(0x020, loads, 0);
    if constexpr (I + 1 < N) interleave<N, READS, LOADS, I + 1>();
}

// WQ x WP waves of MQ x MP blocks of 32 x 32 outputs. FORWARD: half of a wave's blocks along p are of Wg, half of the
// same rows of Wu.
template <class T, int KIND, int WQ, int WP, int MQ, int MP>
struct Product {
    static constexpr int NW = WQ * WP, BQ = WQ * MQ * 32, BP = WP * MP * 32, PAIRS = KIND == FORWARD ? BP / 2 : BP;
    static constexpr int W = (KIND == FORWARD ? MP / 2 : MP) * 32;     // columns of a wave's outputs
    static constexpr int SLOT = NW * MQ * MP * 4 * 64;                 // f32x4 of a tile's sums
    using St = Stage<T, W>;
    using P = Side<T, BP, KIND != FORWARD, NW>;
    using Q = Side<T, BQ, KIND == BY_W, NW>;

    // First q and p of tile i of all. BY_W: the upper half of the tiles along q is that of dWu.
    struct At { int q0, p0, part; };
    __device__ static __forceinline__ At at(const GatedArgs &a, int i) {
        TileAt t = tile_at(i, a.tiles_q, a.tiles_p);
        const int part = KIND == BY_W && t.q >= a.tiles_q / 2;
        if (part) t.q -= a.tiles_q / 2;
        return {t.q * BQ, t.p * PAIRS, part};
    }

    // What is done with row block i of a wave's sums, c. A lane has row l % 32, columns 8 (r / 4) + 4 h + r % 4 of block j.
    __device__ static __forceinline__ void finish(const GatedArgs &a, At t, int i, int w, int lane, f32x16 (&c)[MP], unsigned char *mine) {
        const int q = t.q0 + (w / WP * MQ + i) * 32, p = t.p0 + w % WP * W, rows = a.nq - q, cols = a.np - p, h = lane >> 5;
        T *out = (T *)a.out + (int64_t)(t.part * a.nq + q) * a.ldo + p;
        if constexpr (KIND == FORWARD) {
            if (const T *bias = (const T *)a.bias) {
#pragma unroll
                for (int j = 0; j < MP; ++j) {
#pragma unroll
                    for (int r = 0; r < 16; r += 4) {
                        float b[4];
                        load_chunk<T, 4>(bias + (j >= MP / 2 ? a.np : 0), p + j % (MP / 2) * 32 + 2 * r + 4 * h, a.np, b);
#pragma unroll
                        for (int e = 0; e < 4; ++e) c[j][r + e] += b[e];
                    }
                    __builtin_amdgcn_sched_barrier(0);                 // few registers at a time
                }
            }
            if (a.kept) {
                T *to = (T *)a.kept + (int64_t)q * (2 * (int64_t)a.np) + p;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int j = 0; j < MP / 2; ++j) St::put(mine, lane, j, c[half * (MP / 2) + j]);
                    St::store(mine, lane, to + (half ? a.np : 0), 2 * (int64_t)a.np, rows, cols, a.past_l2);
                }
            }
#pragma unroll
            for (int j = 0; j < MP / 2; ++j) {
                f32x16 y;
#pragma unroll
                for (int r = 0; r < 16; ++r) y[r] = activation<T>(c[j][r], a.act).x * c[j + MP / 2][r];
                St::put(mine, lane, j, y);
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            if constexpr (std::is_same_v<T, _Float16>) {
                const float unit = *a.unit;
#pragma unroll
                for (int j = 0; j < MP; ++j) c[j] *= unit;
            }
#pragma unroll
            for (int j = 0; j < MP; ++j) St::put(mine, lane, j, c[j]);
        }
        St::store(mine, lane, out, a.ldo, rows, cols, KIND == FORWARD && a.past_l2);
    }
};

template <class T, int KIND, int WQ, int WP, int MQ, int MP, int PLACES, int WGS>
__global__ __launch_bounds__(WQ *WP * 64, WGS * WQ * WP / 4) void gated_product_kernel(GatedArgs a) {
    using Pr = Product<T, KIND, WQ, WP, MQ, MP>;
    using P = typename Pr::P;
    using Q = typename Pr::Q;
    constexpr int NW = Pr::NW, BK = STEP_BYTES / (int)sizeof(T);
    constexpr int TILE = P::BYTES + Q::BYTES, LOADS = P::LOADS + Q::LOADS, READS = MQ * Q::READS + MP * P::READS;
    constexpr int LDS = PLACES * TILE > NW * Pr::St::BYTES ? PLACES * TILE : NW * Pr::St::BYTES;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[LDS];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wq = w / WP, wp = w % WP;
    const int per = (a.k + BK - 1) / BK, all = KIND == BY_X ? 2 * per : per;       // steps of a segment, of a tile
    const int at_q = Q::frag_base(lane), at_p = P::frag_base(lane);
    // this workgroup's steps of a row of tiles' steps
    int share = 0, from = 0, to = all, tile;
    if ((int)blockIdx.x < a.cut.whole) {
        tile = by_xcd(blockIdx.x, a.cut.whole);
    } else {
        share = by_xcd(blockIdx.x - a.cut.whole, a.cut.tail * a.cut.of);
        tile = a.cut.whole + share / a.cut.of;
        from = share % a.cut.of * a.cut.each;
        to = min(from + a.cut.each, all);
    }

    {
        const typename Pr::At t = Pr::at(a, tile);
        P feed_p;
        Q feed_q;
        auto start = [&](int step) {                                   // at step `step` of the tile's
            const int seg = KIND == BY_X && step >= per, s = step - seg * per, k = s * BK;
            const T *p = (const T *)a.p, *q = (const T *)a.q + t.part * a.seg_q;
            if (KIND == BY_X) { p += seg * a.seg_p; q += seg * a.seg_q; }
            if constexpr (KIND == FORWARD) {
                feed_p.start(p + t.p0 * a.ldp + k, a.ldp, a.k - k, 0, w, lane, [&](int i) {
                    const int sub = i / 32 % MP, f = i / 32 / MP * (MP / 2 * 32) + sub % (MP / 2) * 32 + i % 32;
                    return t.p0 + f < a.np ? (int64_t)f + (sub >= MP / 2 ? a.np : 0) : -1;
                });
            } else {
                feed_p.start(p + k * a.ldp + t.p0, a.ldp, a.k - k, a.np - t.p0, w, lane, [](int) { return -1; });
            }
            if constexpr (KIND == BY_W) {
                feed_q.start(q + k * a.ldq + t.q0, a.ldq, a.k - k, a.nq - t.q0, w, lane, [](int) { return -1; });
            } else {
                feed_q.start(q + t.q0 * a.ldq + k, a.ldq, a.k - k, 0, w, lane, [&](int i) { return t.q0 + i < a.nq ? i : -1; });
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
        struct Frags { Frag<T> q[MQ], p[MP]; };
        auto read = [&](Frags &f, const unsigned char *from, int s) {
#pragma unroll
            for (int i = 0; i < MQ; ++i) f.q[i] = Q::frag(from, at_q, wq * MQ + i, s);
#pragma unroll
            for (int j = 0; j < MP; ++j) f.p[j] = P::frag(from + Q::BYTES, at_p, wp * MP + j, s);
        };
        auto multiply = [&](const Frags &f) {
#pragma unroll
            for (int i = 0; i < MQ; ++i)
#pragma unroll
                for (int j = 0; j < MP; ++j) mma(c[i][j], f.p[j], f.q[i]);
        };
        // A step's first operands are in registers when it begins, and its tile and the next one's are in LDS; the tile
        // that is asked for goes to the place of the last step's, which every wave has read by then. The pointers do
        // not alias, or each step would wait for the tiles of the next ones.
        Frags f0, f1;
        auto body = [&](int step, const unsigned char *__restrict now, const unsigned char *__restrict after, unsigned char *__restrict to) {
            loaded<(PLACES - 3) * LOADS>();                            // the next step's tile; those behind it may take their time
            __builtin_amdgcn_sched_barrier(0);
            next(step + PLACES - 1, to);
            if constexpr (sizeof(T) == 2) {
                read(f1, now, 1);
                multiply(f0);
                interleave<MQ * MP, READS, LOADS>();
                __builtin_amdgcn_sched_barrier(0);
                read(f0, after, 0);
                multiply(f1);
                interleave<MQ * MP, READS, 0>();
            } else {
                read(f1, after, 0);
                __builtin_amdgcn_sched_barrier(0);
                multiply(f0);
                f0 = f1;
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        start(from);
#pragma unroll
        for (int i = 0; i < PLACES - 1; ++i) next(from + i, lds + i * TILE);
        loaded<(PLACES - 2) * LOADS>();
        read(f0, lds, 0);
        int at = 0;
        for (int step = from; step < to; ++step) {
            const int after = at == (PLACES - 1) * TILE ? 0 : at + TILE, before = at == 0 ? (PLACES - 1) * TILE : at - TILE;
            body(step, lds + at, lds + after, lds + before);
            at = after;
        }
        tiles_ready();                                                 // nothing reads or fills LDS any more
        if (tile < a.cut.whole) {
#pragma unroll
            for (int i = 0; i < MQ; ++i) Pr::finish(a, t, i, w, lane, c[i], lds + w * Pr::St::BYTES);
            return;
        }
        f32x4 *part = a.part + (int64_t)share * Pr::SLOT + w * (MQ * MP * 4 * 64) + lane;
#pragma unroll
        for (int i = 0; i < MQ; ++i)
#pragma unroll
            for (int j = 0; j < MP; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    part[((i * MP + j) * 4 + r) * 64] = f32x4{c[i][j][4 * r], c[i][j][4 * r + 1], c[i][j][4 * r + 2], c[i][j][4 * r + 3]};
    }
}

// Adds the slots of a shared tile (blockIdx.x) and finishes row blocks blockIdx.y of its waves.
template <class T, int KIND, int WQ, int WP, int MQ, int MP>
__global__ __launch_bounds__(WQ *WP * 64) void gated_join_kernel(GatedArgs a) {
    using Pr = Product<T, KIND, WQ, WP, MQ, MP>;
    __shared__ __attribute__((aligned(16))) unsigned char lds[Pr::NW * Pr::St::BYTES];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i = blockIdx.y, t = blockIdx.x;
    const f32x4 *part = a.part + (int64_t)t * a.cut.of * Pr::SLOT + (w * MQ + i) * (MP * 4 * 64) + lane;
    f32x16 c[MP];
#pragma unroll
    for (int j = 0; j < MP; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) c[j][r] = 0.f;
    for (int s = 0; s < a.cut.of; ++s, part += Pr::SLOT)
#pragma unroll
        for (int j = 0; j < MP; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const f32x4 v = part[(j * 4 + r) * 64];
#pragma unroll
                for (int e = 0; e < 4; ++e) c[j][4 * r + e] += v[e];
            }
    Pr::finish(a, Pr::at(a, t + a.cut.whole), i, w, lane, c, lds + w * Pr::St::BYTES);
}

// Rows of at most 32 MQ tokens: the weight's bytes count (2 x 1024 to 2736 bf16 5.5 us for 11 MB; a wave's loads of 32
// bytes from each of 32 rows take the address units as long as whole lines would for twice as many; fetching a piece of k
// ahead made no difference). A workgroup takes 16 columns of h, as a block of 16 rows of Wg and the same 16 of Wu; its waves
// share k, each reading its rows' pieces straight into the operands' registers. In the block, rows 8..15 and 24..31 are
// those of Wu: a lane then holds g and u of the same columns.
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
        ((T *)a.out)[(int64_t)q * a.ldo + p] = (T)(activation<T>(g, a.act).x * u);
    }
}

struct SlopeArgs {
    const void *dh, *kept;
    void *dp;                                  // [N][2][pitch]
    float *part;                               // [rows' workgroup][2][F], or NULL
    int64_t N;
    int F, pitch, act, rows;                   // rows of a workgroup
    float *most, *unit;                        // float16: the largest |dg|, |du| of each workgroup, and the unit; or NULL
};

// dg and du of VE columns from c on.
template <class T, int VE>
__device__ __forceinline__ void slopes(const SlopeArgs &a, int64_t n, int c, float (&dg)[VE], float (&du)[VE]) {
    float d[VE];
    load_chunk<T, VE>((const T *)a.dh + n * a.F, c, a.F, d);
    load_chunk<T, VE>((const T *)a.kept + n * 2 * a.F, c, a.F, dg);
    load_chunk<T, VE>((const T *)a.kept + n * 2 * a.F + a.F, c, a.F, du);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
        const float2 s = activation<T>(dg[e], a.act);
        dg[e] = d[e] * du[e] * s.y;            // past column F all three are zeros
        du[e] = d[e] * s.x;
    }
}

// The largest of a workgroup's 256 values.
__device__ __forceinline__ float workgroup_max(float x, float (&scratch)[4]) {
#pragma unroll
    for (int i = 1; i < 64; i *= 2) x = fmaxf(x, __shfl_xor(x, i));
    scratch[threadIdx.x >> 6] = x;
    __syncthreads();
    return fmaxf(fmaxf(scratch[0], scratch[1]), fmaxf(scratch[2], scratch[3]));
}

// float16 has five bits for exponents: gradients of a mean over many rows lie below its numbers, scaled ones beyond them. Where the
// largest finite dg or du is not between 1 and 65504, all are held in units of a power of two in which it is between 2^14 and 2^15, so
// that those down to 2^-28 of it keep their digits; the products' sums are multiplied by the unit. (Between them those down to
// 2^-14 keep theirs.) Finding it first would read everything twice (24576 x 2736: 119 to 148 us); so the first pass has no unit
// and notes its largest, and a second one does nothing (6 us) or takes them again in a unit.
__device__ __forceinline__ int unit_exponent(const SlopeArgs &a, float (&scratch)[4]) {
    float most = 0.f;
    for (int i = threadIdx.x; i < (int)gridDim.x; i += 256) most = fmaxf(most, a.most[i]);
    most = workgroup_max(most, scratch);
    return most == 0.f || (most >= 1.f && most <= 65504.f) ? 0 : max(ilogbf(most) - 14, -100);
}

// dg and du from dh and the projections; the columns' sums over a workgroup's rows. A thread has eight columns, a wave
// 512, and the workgroup's four waves every fourth row. AGAIN: float16's second pass.
template <class T, bool AGAIN = false>
__global__ __launch_bounds__(256) void gated_slope_kernel(SlopeArgs a) {
    constexpr int VE = 8;
    constexpr bool HALF = std::is_same_v<T, _Float16>;
    __shared__ float sums[4][2][64 * VE], scratch[4];
    const int across = (a.pitch + 64 * VE - 1) / (64 * VE), group = blockIdx.x / across, block = blockIdx.x % across;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, c = (block * 64 + lane) * VE;
    const int64_t first = (int64_t)group * a.rows, last = min(first + a.rows, a.N);
    float sg[VE] = {}, su[VE] = {}, most = 0.f, to_unit = 1.f;
    if constexpr (AGAIN) {
        const int exponent = unit_exponent(a, scratch);
        if (blockIdx.x == 0 && threadIdx.x == 0) *a.unit = ldexpf(1.f, exponent);
        if (exponent == 0) return;
        to_unit = ldexpf(1.f, -exponent);
    }
    if (c < a.pitch)
        for (int64_t n = first + w; n < last; n += 4) {
            float g[VE], u[VE];
            slopes<T, VE>(a, n, c, g, u);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                if constexpr (AGAIN) {
                    g[e] *= to_unit;
                    u[e] *= to_unit;
                } else {
                    sg[e] += g[e];
                    su[e] += u[e];
                    if constexpr (HALF) {      // infinities and NaN are what they are in any unit
                        most = fmaxf(most, fabsf(g[e]) < INFINITY ? fabsf(g[e]) : 0.f);
                        most = fmaxf(most, fabsf(u[e]) < INFINITY ? fabsf(u[e]) : 0.f);
                    }
                }
            }
            store_chunk<T, VE>((T *)a.dp + n * 2 * a.pitch, c, a.pitch, g);
            store_chunk<T, VE>((T *)a.dp + n * 2 * a.pitch + a.pitch, c, a.pitch, u);
        }
    if constexpr (AGAIN) return;
    if (HALF && a.most) {
        most = workgroup_max(most, scratch);
        if (threadIdx.x == 0) a.most[blockIdx.x] = most;
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

// How a product is cut up: tiles of `size` x `size` outputs, and how they are shared out.
struct Cut { int size, tiles_q, tiles_p; Shares s; };

// The cut that takes the least time by a measured model, in microseconds. The card has room for 256 tiles of 256 at a time or
// 512 of 128 (two to a CU); a step of k takes `step` of such a round, its start and end `round` (FORWARD's activations and
// three outputs more). Tiles that are left when all places have had as many can be cut along k, every one alike, so that
// workgroups that run together share what they read, if writing and reading their sums at 4 TB/s and the join cost less
// than leaving places idle.
Cut cut_of(int kind, int64_t nq, int64_t np, int64_t k, int dtype) {
    const int bk = STEP_BYTES / esize(dtype);
    const int64_t all = (k + bk - 1) / bk * (kind == BY_X ? 2 : 1);
    Cut best{};
    double least = 0;
    for (int size : {128, 256}) {
        if (size == 256 && dtype == DDM_F32) continue;     // a round of as many tiles of 128 has work for all matrix cores
        const int64_t places = size == 256 || dtype == DDM_F32 ? 256 : 512;
        const double step = dtype == DDM_F32 ? 0.85 : size == 256 ? 0.8 : 0.56, round = kind == FORWARD ? 12 : 6;
        const int64_t tq = (nq + size - 1) / size * (kind == BY_W ? 2 : 1);
        const int64_t tp = kind == FORWARD ? (np + size / 2 - 1) / (size / 2) : (np + size - 1) / size, n = tq * tp;
        for (int of = 1; of <= 128 && of * 4 <= std::max<int64_t>(all, 4); ++of) {
            const int64_t whole = of == 1 ? n : n / places * places, tail = n - whole, each = (all + of - 1) / of;
            if (of > 1 && (tail == 0 || tail * of > 2 * places)) break;        // at most 128 MB of sums
            double t = (double)((whole + places - 1) / places) * (all * step + round);
            if (of > 1) t += (double)((tail * of + places - 1) / places) * (each * step + round) + 10 + (double)tail * of * size * size * 8 / 4e6;
            if (best.size == 0 || t < least) {
                least = t;
                best = Cut{size, (int)tq, (int)tp, Shares{(int)whole, (int)tail, of, (int)each}};
            }
        }
    }
    return best;
}
Cut cut_forward(int64_t N, int C, int F, int dtype) { return cut_of(FORWARD, N, F, C, dtype); }
Cut cut_by_x(int64_t N, int C, int F, int dtype) { return cut_of(BY_X, N, C, F, dtype); }
Cut cut_by_w(int64_t N, int C, int F, int dtype) { return cut_of(BY_W, F, C, N, dtype); }

// Whether gated_tokens_kernel is sooner done than the tiles' product, by models of both in microseconds that follow what was measured
// over C of 64 to 16384, F of 64 to 16384 and 1 to 64 rows. A workgroup of it walks along k at a pace that its rows and, from 33 on, a
// second operand set; workgroups beyond one to a CU (4096 of F) wait. Tiles cost a start, a join and the weight's bytes, in 32 bits
// a matrix product of rows that are mostly not there. By tokens and by tiles, bf16: 48 x 1024 to 1024 9 and 22 us, 64 x 1024 to 2736
// 9.8 and 14.5, 33 x 2048 to 5461 22.2 and 23.9, 64 rows of it 29.6 and 25.5, 32 x 16384 to 2048 66 and 54, 64 x 4096 to 8192 55 and 39; fp32:
// 64 x 1024 to 2736 16.5 and 28, 8 x 8192 to 512 46 and 40, 32 x 8192 to 1024 65 and 52, 64 x 4096 to 8192 108 and 155. Among those sizes the
// worse one is taken by 20% at most (64 x 4096 to 1024 bf16).
bool by_tokens(int64_t N, int C, int F, int dtype) {
    if (N == 0 || N > 64) return N == 0;
    const double k = C / 1024., product = 1e-6 * F * C, second = N > 32;
    if (dtype == DDM_F32) return 3 + k * (5.2 + 0.075 * N + 2 * second) * std::max(1., F / 4096.) < 18 + 4.2 * product;
    const int rounds = (F + 4095) / 4096;
    return 3.5 + k * (2.2 + 0.043 * N + 0.5 * second) * (rounds == 1 ? 1 : 1.2 * rounds) < 13.5 + 1.6 * k + 0.6 * product;
}

size_t repacked(int64_t rows, int C, int dtype) { return whole((size_t)rows * padded(C, dtype) * esize(dtype)); }
size_t parts_bytes(const Cut &c) { return (size_t)c.s.tail * c.s.of * c.size * c.size * 4; }

// Rows of a workgroup of gated_slope_kernel: some 1024 workgroups, of 16 rows at least and 64 at most (24576 x 2736 bf16:
// 144 us with 64, 149 with 128, 189 with 256), and 4096 workgroups at most.
int slope_rows(int64_t N, int F) {
    const int64_t across = (F + 511) / 512, least = (N * across / 4096 + 15) / 16 * 16;
    return (int)std::max(std::min<int64_t>(std::max<int64_t>((N * across / 1024 + 15) / 16 * 16, 16), 64), least);
}
int64_t slope_groups(int64_t N, int F) { return (N + slope_rows(N, F) - 1) / slope_rows(N, F); }
int64_t slope_blocks(int64_t N, int F) { return slope_groups(N, F) * ((F + 511) / 512); }

// Workspaces, in order. x's repacked rows come last: whether they are needed depends on its address and stride.
struct ForwardPlan { bool tokens; Cut cut; size_t w, part, x, bytes; };
ForwardPlan forward_plan(int64_t N, int C, int F, int dtype) {
    ForwardPlan p{};
    p.tokens = by_tokens(N, C, F, dtype);
    if (!p.tokens) p.cut = cut_forward(N, C, F, dtype);
    p.part = p.w + (C % (16 / esize(dtype)) ? repacked(2 * (int64_t)F, C, dtype) : 0);
    p.x = p.part + (p.tokens ? 0 : parts_bytes(p.cut));
    p.bytes = p.x + repacked(N, C, dtype);
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
    a.tiles_q = c.tiles_q; a.tiles_p = c.tiles_p; a.cut = c.s;
    const unsigned grid = (unsigned)(c.s.whole + c.s.tail * c.s.of);
    auto go = [&](auto wq, auto wp, auto mq, auto mp, auto places, auto wgs) {
        constexpr int WQ = decltype(wq)::value, WP = decltype(wp)::value, MQ = decltype(mq)::value, MP = decltype(mp)::value;
        hipLaunchKernelGGL((gated_product_kernel<T, KIND, WQ, WP, MQ, MP, decltype(places)::value, decltype(wgs)::value>), dim3(grid),
                           dim3(WQ * WP * 64), 0, s, a);
        if (c.s.tail)
            hipLaunchKernelGGL((gated_join_kernel<T, KIND, WQ, WP, MQ, MP>), dim3(c.s.tail, MQ), dim3(WQ * WP * 64), 0, s, a);
    };
    using std::integral_constant;
    if constexpr (sizeof(T) == 2) {
        if (c.size == 256) {
            if constexpr (KIND == FORWARD)
                go(integral_constant<int, 4>{}, integral_constant<int, 2>{}, integral_constant<int, 2>{}, integral_constant<int, 4>{},
                   integral_constant<int, 5>{}, integral_constant<int, 1>{});
            else
                go(integral_constant<int, 2>{}, integral_constant<int, 4>{}, integral_constant<int, 4>{}, integral_constant<int, 2>{},
                   integral_constant<int, 4>{}, integral_constant<int, 1>{});
            return;
        }
    }
    go(integral_constant<int, 2>{}, integral_constant<int, 2>{}, integral_constant<int, 2>{}, integral_constant<int, 2>{},
       integral_constant<int, 5>{}, integral_constant<int, 2>{});
}

unsigned blocks(int64_t items, int64_t each) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>((items + each - 1) / each, 8192)); }

// Whether rows are whole 16-byte pieces where they are.
bool are_whole(const void *from, int64_t ld, int64_t rows, int C, int e) {
    return (uintptr_t)from % 16 == 0 && C * (int64_t)e % 16 == 0 && (ld * e % 16 == 0 || rows == 1);
}
// x or the weight as rows of whole 16-byte pieces: themselves, or a copy in the workspace.
template <class T>
const T *whole_rows(const void *from, int64_t &ld, int64_t rows, int C, void *copy, hipStream_t s) {
    constexpr int PE = 16 / sizeof(T);
    if (are_whole(from, ld, rows, C, sizeof(T))) return (const T *)from;
    const int pitch = (C + PE - 1) / PE * PE;
    hipLaunchKernelGGL((gated_repack_kernel<T>), dim3(blocks(rows * (pitch / PE), 256)), dim3(256), 0, s, (const T *)from, ld, rows, C, pitch, (T *)copy);
    ld = pitch;
    return (const T *)copy;
}

bool bad_act(int act) { return act != DDM_SILU && act != DDM_GELU && act != DDM_SIGMOID; }
bool bad_stride(int64_t ld, int C, int e) { return ld < C || ld > (1 << 22) / e; }
bool off(const void *p, int e) { return !p || (uintptr_t)p % e; }
// What a plan's workspace comes to for this x.
template <class Plan>
size_t needed(const Plan &p, const void *x, int64_t ldx, int64_t N, int C, int e) {
    return std::max<size_t>(are_whole(x, ldx, N, C, e) ? p.x : p.bytes, 16);
}
// The weight's rows are read in place, in pieces of 16 bytes, or repacked, where they are not made of whole ones.
bool off_weight(const void *w, int C, int e) { return off(w, C * (int64_t)e % 16 ? e : 16); }

}  // namespace

extern "C" {

size_t ddm_gated_linear_repack_bytes(int64_t N, int C, int dtype) {
    return check(N, C, 1, dtype) != DDM_OK ? 0 : repacked(N, C, dtype);
}

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
    if (off(x, e) || off_weight(weight, C, e) || off(h, e) || (uintptr_t)bias % e || (uintptr_t)kept % e) return DDM_ERR_INVALID;
    const ForwardPlan pl = forward_plan(N, C, F, dtype);
    if (off(workspace, 16) || workspace_bytes < needed(pl, x, ldx, N, C, e)) return DDM_ERR_WORKSPACE;
    char *ws = (char *)workspace;
    with_type(dtype, [&](auto t) {
        using T = decltype(t);
        GatedArgs a{};
        a.ldq = ldx; a.ldp = C; a.ldo = F;
        a.q = whole_rows<T>(x, a.ldq, N, C, ws + pl.x, stream);
        a.p = whole_rows<T>(weight, a.ldp, 2 * (int64_t)F, C, ws + pl.w, stream);
        a.np = F; a.nq = (int)N; a.k = C; a.bias = bias; a.out = h; a.kept = kept; a.act = activation;
        a.part = (f32x4 *)(ws + pl.part);
        // 24576 x 1024 to 2736 bf16 with kept: 336 us past the L2s, which then keep x and the weight, 373 through them
        a.past_l2 = (kept ? 3 : 1) * N * F * e > 32 << 20;
        const dim3 tokens((F + 15) / 16);
        if (pl.tokens && N <= 32) hipLaunchKernelGGL((gated_tokens_kernel<T, 1, 8>), tokens, dim3(512), 0, stream, a);
        else if (pl.tokens) hipLaunchKernelGGL((gated_tokens_kernel<T, 2, 8>), tokens, dim3(512), 0, stream, a);
        else launch_product<T, FORWARD>(a, pl.cut, stream);
    });
    return hipGetLastError() == hipSuccess ? DDM_OK : DDM_ERR_HIP;
}

}  // extern "C"

namespace {

struct BackPlan { Cut by_x, by_w; size_t w, dp, bias, most, part, x, bytes; };
BackPlan back_plan(int64_t N, int C, int F, int dtype) {
    BackPlan p{};
    p.by_x = cut_by_x(N, C, F, dtype);
    p.by_w = cut_by_w(N, C, F, dtype);
    p.dp = p.w + (C % (16 / esize(dtype)) ? repacked(2 * (int64_t)F, C, dtype) : 0);
    p.bias = p.dp + whole((size_t)N * 2 * padded(F, dtype) * esize(dtype));
    p.most = p.bias + whole((size_t)slope_groups(N, F) * 2 * F * 4);
    p.part = p.most + (dtype == DDM_F16 ? whole((size_t)(slope_blocks(N, F) + 1) * 4) : 0);
    p.x = p.part + std::max(parts_bytes(p.by_x), parts_bytes(p.by_w));
    p.bytes = p.x + repacked(N, C, dtype);
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
    if (N && (off(dh, e) || off(kept, e) || (dweight && off(x, e)) || (dx && off_weight(weight, C, e)))) return DDM_ERR_INVALID;
    if ((uintptr_t)dx % e || (uintptr_t)dweight % e || (uintptr_t)dbias % e) return DDM_ERR_INVALID;
    const BackPlan pl = back_plan(N, C, F, dtype);
    if (off(workspace, 16) || workspace_bytes < needed(pl, x, ldx, N, C, e)) return DDM_ERR_WORKSPACE;
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
        sl.N = N; sl.F = F; sl.pitch = padded(F, dtype); sl.act = activation; sl.rows = slope_rows(N, F);
        const dim3 slope_grid((unsigned)slope_blocks(N, F));
        if (std::is_same_v<T, _Float16> && (dx || dweight)) { sl.unit = (float *)(ws + pl.most); sl.most = sl.unit + 1; }
        hipLaunchKernelGGL((gated_slope_kernel<T>), slope_grid, dim3(256), 0, stream, sl);
        if constexpr (std::is_same_v<T, _Float16>)
            if (sl.unit) hipLaunchKernelGGL((gated_slope_kernel<T, true>), slope_grid, dim3(256), 0, stream, sl);
        if (dbias)
            hipLaunchKernelGGL((gated_bias_kernel<T>), dim3((2 * F + 31) / 32), dim3(1024), 0, stream, sl.part, (int)slope_groups(N, F), 2 * F, (T *)dbias);
        GatedArgs a{};
        a.part = (f32x4 *)(ws + pl.part);
        a.unit = sl.unit;
        a.ldo = C; a.np = C; a.ldq = 2 * (int64_t)sl.pitch; a.q = sl.dp; a.seg_q = sl.pitch;
        if (dx) {
            a.ldp = C;
            a.p = whole_rows<T>(weight, a.ldp, 2 * (int64_t)F, C, ws + pl.w, stream);
            a.seg_p = F * a.ldp; a.nq = (int)N; a.k = F; a.out = dx;
            launch_product<T, BY_X>(a, pl.by_x, stream);
        }
        if (dweight) {
            a.ldp = ldx;
            a.p = whole_rows<T>(x, a.ldp, N, C, ws + pl.x, stream);
            a.nq = F; a.k = (int)N; a.out = dweight;
            launch_product<T, BY_W>(a, pl.by_w, stream);
        }
    });
    return hipGetLastError() == hipSuccess ? DDM_OK : DDM_ERR_HIP;
}

}  // extern "C"

// ddm_loss.hip -- the matching loss and its gradient (ddm_matching_loss_*).
//
//   z_ij = a_i . b_j / t,  loss_i = (lse_a_i + lse_b_i) / 2 - z_ii
//   dz_ij = (g_i e^{z_ij - lse_a_i} + g_j e^{z_ij - lse_b_j}) / 2 - g_i [i = j]
//   da_i = sum_j dz_ij b_j / t,  db_j = sum_i dz_ij a_i / t
// within each packed set. Scores exist only as matrix-core tiles. With some 24 to 64 components a score costs far less
// on the matrix cores than its exponentials on the vector units. In general each direction has its own pass: rows of
// one side stay in registers and the other side's go by, and no sum crosses workgroups except over the S pieces that a
// set's columns are cut into when there are too few rows to fill the card; those are joined in order. Forward, sets
// whose scores cannot leave +-32 need no maximum, and one exponential a score serves both directions (one_pass()).
#include "../../../include/ddm.h"
#include "ddm_attn.hpp"

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

using namespace ddm;

namespace {

constexpr float LOG2E = 1.44269504088896341f, LN2 = 0.69314718055994531f;

struct LossArgs {
    const void *a, *b;               // [P][ld] rows, of which w elements are read (w = d, or the padded d of copied rows)
    const int32_t *cu;
    int B, P, d, w, ld, S;
    float c, inv_t;                  // c = log2(e) / t
    float2 *ml;                      // forward: [2][S][P] largest a_i.b_j and the sum of exponentials about it
    float *hit;                      // forward: a_i.b_i
    float *top;                      // [2][slots] largest |a_i|^2, |b_i|^2 of 128 rows, or null: no set takes one pass
    float *row_sum, *col_sum;        // one pass: [pieces][P], [chunks][P] sums of e^z without the match
    int slots, one_rows, one_pieces;
    const float *g, *lse_a, *lse_b;  // backward
    void *da, *db;
    float *part;                     // backward: [2][S][P][DP], or null: written straight to da, db
};

// Columns [from, to) of piece `s` of S of a set of n.
__device__ __forceinline__ void piece_of(int n, int S, int s, int tile, int *from, int *to) {
    const int each = ((n + S - 1) / S + tile - 1) / tile * tile;
    *from = min(n, s * each);
    *to = min(n, *from + each);
}

// Largest |a_i|^2 (blockIdx.y = 0) or |b_i|^2 (1) of each slot of 128 rows: two lanes a row, 16 bytes a load.
template <class T>
__global__ __launch_bounds__(256) void loss_top_kernel(LossArgs p) {
    constexpr int PE = 16 / sizeof(T);
    __shared__ float wave_top[4];
    int index;
    const int s = find_slot(p.cu, p.B, p.P, 1, 128, blockIdx.x, &index);
    const Span span = span_of(p.cu, p.B, p.P, s);
    const int row = index * 128 + (threadIdx.x >> 1);
    if (index * 128 >= span.hi - span.lo) return;
    float sq = 0.f;
    if (row < span.hi - span.lo) {
        const T *x = (const T *)(blockIdx.y ? p.b : p.a) + (int64_t)(span.lo + row) * p.ld;
        for (int c = (threadIdx.x & 1) * PE; c < p.w; c += 2 * PE) {
            union { u32x4 u; T e[PE]; } v;
            v.u = *reinterpret_cast<const u32x4 *>(x + c);
#pragma unroll
            for (int e = 0; e < PE; ++e) sq = __builtin_fmaf((float)v.e[e], (float)v.e[e], sq);
        }
    }
    sq += __shfl_xor(sq, 1);
#pragma unroll
    for (int x = 32; x > 1; x >>= 1) sq = fmaxf(sq, __shfl_xor(sq, x));
    if ((threadIdx.x & 63) == 0) wave_top[threadIdx.x >> 6] = sq;
    __syncthreads();
    if (threadIdx.x == 0)
        p.top[(int64_t)blockIdx.y * p.slots + blockIdx.x] = fmaxf(fmaxf(wave_top[0], wave_top[1]), fmaxf(wave_top[2], wave_top[3]));
}

// Whether set s takes one pass: |z_ij| <= |a_i| |b_j| / t is at most 32, so that e^z and sums of up to ONE_N of them, and
// those by e^-z_ii, stay inside fp32's range; and it is not too long for its sums' places. For the whole workgroup.
constexpr int ONE_N = 32768, ONE_COLS = 1024;
__device__ __forceinline__ bool takes_one_pass(const LossArgs &p, int s, Span span, float (*red)[4]) {
    const int n = span.hi - span.lo;
    if (!p.top || s == 0 || s == p.B + 1 || n > ONE_N) return false;
    const float *at = p.top + span.lo / 128 + s;
    float ta = 0.f, tb = 0.f;
    for (int i = threadIdx.x; i < (n + 127) / 128; i += 256) {
        ta = fmaxf(ta, at[i]);
        tb = fmaxf(tb, at[p.slots + i]);
    }
#pragma unroll
    for (int x = 32; x; x >>= 1) {
        ta = fmaxf(ta, __shfl_xor(ta, x));
        tb = fmaxf(tb, __shfl_xor(tb, x));
    }
    __syncthreads();                                           // red may still be read from before
    if ((threadIdx.x & 63) == 0) { red[0][threadIdx.x >> 6] = ta; red[1][threadIdx.x >> 6] = tb; }
    __syncthreads();
    ta = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    tb = fmaxf(fmaxf(red[1][0], red[1][1]), fmaxf(red[1][2], red[1][3]));
    return __builtin_amdgcn_readfirstlane(ta * tb * (p.inv_t * p.inv_t) <= 1024.f);
}
// Its columns in pieces: p.one_pieces of them, or of at most ONE_COLS each; at least 128. one_pieces makes some 1024
// workgroups: twice or four times as many gain 3% for sets of unlike lengths and lose 2% for one of 16384.
__device__ __forceinline__ int one_piece(const LossArgs &p, int n) {
    return min(ONE_COLS, ((n + p.one_pieces - 1) / p.one_pieces + 127) / 128 * 128);
}

// 16 elements over 32 lanes: at each exchange a lane hands over the half of the elements that it stops summing, and ends
// with element (lane / 2) % 16 over the lanes of its parity.
template <int K>
__device__ __forceinline__ void hand_over(float (&v)[16], int lane) {
    const bool up = lane & (2 * K);
#pragma unroll
    for (int r = 0; r < K; ++r) {
        const float give = up ? v[r] : v[r + K], keep = up ? v[r + K] : v[r];
        v[r] = keep + __shfl_xor(give, 2 * K);
    }
    if constexpr (K > 1) hand_over<K / 2>(v, lane);
}

// Forward, both directions at once: rows a of one chunk, columns b of one piece. e^z is summed as it is, without a
// maximum: a wave keeps 32 rows, whose sums gather in the 16 elements of its score tiles over all columns, and adds each
// tile's column sums (16 of a column's 32 in each lane half) to its own row of LDS. The match itself is left out:
// lse - z_ii = log1p(e^-z_ii sum of the others) is exact where that is small. Per score 3.1 instructions and one
// exponential, for which two passes take twice 3.75 and one. With the gradient: 16384 x 64 bf16 270 us against 293 in two
// passes, 8000 x 24 fp32 234 against 272, 16 sets of up to 4096 x 24 fp16 169 against 167. Alone 79 us and 60 us for the first
// and the last, 310 and 400 ns a tile of 32 x 32 on a SIMD: 95 and 103 vector and some 24 and 42 scalar instructions, and
// waits for a quarter of the wave cycles. Chunks of 256 rows (with 512 the first of the two has 1024
// workgroups, whose last third the card runs alone: 287 us), longer ones in calls of very many matches (see the plan).
template <class T, int D, int BN>
__global__ __launch_bounds__(256, 2) void loss_one_kernel(LossArgs p) {
    using TL = Tile<T, D>;
    constexpr int DC = D / 16, KB = BN / 32, BM = 128;
    // One array: of several, the compiler takes the loads to LDS to alias what is read, and waits for the next tile in
    // every step (295 against 287 us for the first of the two above).
    constexpr int TILE = BN * TL::ROW;
    __shared__ __attribute__((aligned(16))) unsigned char lds[2 * TILE + 4 * ONE_COLS * 4 + 32];
    float *const col = (float *)(lds + 2 * TILE);
    float (*const red)[4] = (float (*)[4])(col + 4 * ONE_COLS);
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), h = lane >> 5;
    int chunk;
    const int s = find_slot(p.cu, p.B, p.P, 1, p.one_rows, blockIdx.x, &chunk), piece = blockIdx.y;
    const Span span = span_of(p.cu, p.B, p.P, s);
    const int n = span.hi - span.lo;
    if ((int64_t)chunk * p.one_rows >= n) return;
    const int each = one_piece(p, n), from = min((int64_t)n, (int64_t)piece * each), to = min(n, from + each);
    if (from >= n || !takes_one_pass(p, s, span, red)) return;
    const T *xs = (const T *)p.a + (int64_t)span.lo * p.ld, *ys = (const T *)p.b + (int64_t)span.lo * p.ld;
    const int row_at = TL::row_base(lane);
    for (int j = lane; j < to - from; j += 64) col[w * ONE_COLS + j] = 0.f;
    for (int row0 = chunk * p.one_rows; row0 < min(n, (chunk + 1) * p.one_rows); row0 += BM) {
        const int wave0 = row0 + 32 * w, row = wave0 + (lane & 31);
        Frag<T> xf[DC];
#pragma unroll
        for (int c = 0; c < DC; ++c) xf[c] = global_rows<T>(xs + (int64_t)min(row, n - 1) * p.ld, 16 * c + 8 * h, p.w, row < n);
        Walk<T, D, 4, BN> tiles(ys + (int64_t)from * p.ld, to - from, p.ld, p.w, w, lane);
        const int t_end = (to - from + BN - 1) / BN;
        f32x16 sum = 0.f;
        auto step = [&](int t, const unsigned char *__restrict cur, unsigned char *__restrict next,
                        float *__restrict my_col, auto special) {
            if (t + 1 < t_end) tiles.next(next, w);
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                float *at = my_col + t * BN + 32 * b + (lane & 31);
                const float before = *at;
                f32x16 z = 0.f;
#pragma unroll
                for (int c = 0; c < DC; ++c) mma(z, xf[c], TL::rows(cur, row_at, 32 * b, c));
                const int j = from + t * BN + 32 * b + (lane & 31);
                float hit = 0.f;
                bool has = false;
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    float e = exp2_fast(z[r] * p.c);
                    if constexpr (decltype(special)::value) {
                        const int i = wave0 + 8 * (r / 4) + 4 * h + r % 4;
                        if (i == j) { hit = z[r]; has = true; }
                        if (i == j || i >= n || j >= to) e = 0.f;
                    }
                    z[r] = e;
                }
                sum += z;
                float c4[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) c4[r] = (z[r] + z[r + 4]) + (z[r + 8] + z[r + 12]);
                const float total = half_sum((c4[0] + c4[1]) + (c4[2] + c4[3]));
                if constexpr (decltype(special)::value) {
                    if (has && j < to) p.hit[span.lo + j] = hit;
                }
                *at = before + total;                          // the same from both lane halves
            }
        };
        tiles.next(lds, w);
        tiles_ready();
        for (int t = 0; t < t_end; ++t) {
            const int j0 = from + t * BN;
            const bool special = j0 + BN > to || row0 + BM > n || (j0 < row0 + BM && row0 < j0 + BN);
            if (special) step(t, lds + (t & 1) * TILE, lds + (~t & 1) * TILE, col + w * ONE_COLS, std::integral_constant<bool, true>{});
            else step(t, lds + (t & 1) * TILE, lds + (~t & 1) * TILE, col + w * ONE_COLS, std::integral_constant<bool, false>{});
            tiles_ready();
        }
        float v[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = sum[r];
        hand_over<8>(v, lane);
        v[0] += __shfl_xor(v[0], 1);
        const int r = (lane >> 1) & 15, i = wave0 + 8 * (r / 4) + 4 * h + r % 4;
        if (!(lane & 1) && i < n) p.row_sum[(int64_t)piece * p.P + span.lo + i] = v[0];
    }
    for (int j = tid; j < to - from; j += 256)
        p.col_sum[(int64_t)chunk * p.P + span.lo + from + j] = (col[j] + col[ONE_COLS + j]) + (col[2 * ONE_COLS + j] + col[3 * ONE_COLS + j]);
}

// Forward, one direction (blockIdx.z), of the sets that do not take one pass: rows x of one side, columns y of the other.
// As attention's forward without values; the maximum is exact here, since the loss of a clear match is the logarithm of
// a sum next to 1. Bound by the vector units, 3.75 instructions and an exponential (four more's time) a score, and the
// matrix cores behind them: 110 us for 2 x 16384 x 16384 scores of 64 components (bf16), 74 us for 16 sets of up to 4096
// matches of 24 (fp16; 3.2e8 scores). Where every set takes one pass its workgroups end at once (5 us).
template <class T, int D, int BN>
__global__ __launch_bounds__(256, 2) void loss_fwd_kernel(LossArgs p) {
    using TL = Tile<T, D>;
    constexpr int DC = D / 16, KB = BN / 32, BM = 128;
    constexpr int TILE = BN * TL::ROW;
    __shared__ __attribute__((aligned(16))) unsigned char lds[2 * TILE + 32];      // one array, as above
    float (*const red)[4] = (float (*)[4])(lds + 2 * TILE);
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), h = lane >> 5;
    const int dir = blockIdx.z;
    int index;
    const int s = find_slot(p.cu, p.B, p.P, 1, BM, blockIdx.x, &index);
    const Span span = span_of(p.cu, p.B, p.P, s);
    const int n = span.hi - span.lo, row0 = index * BM;
    if (row0 >= n || takes_one_pass(p, s, span, red)) return;
    int from = 0, to = 0;
    if (s != 0 && s != p.B + 1) piece_of(n, p.S, blockIdx.y, BN, &from, &to);
    const T *xs = (const T *)(dir ? p.b : p.a) + (int64_t)span.lo * p.ld, *ys = (const T *)(dir ? p.a : p.b) + (int64_t)span.lo * p.ld;
    const int row = row0 + w * 32 + (lane & 31);
    const bool in = row < n;
    Frag<T> xf[DC];
#pragma unroll
    for (int c = 0; c < DC; ++c) xf[c] = global_rows<T>(xs + (int64_t)(in ? row : n - 1) * p.ld, 16 * c + 8 * h, p.w, in);
    Walk<T, D, 4, BN> tiles(ys + (int64_t)from * p.ld, to - from, p.ld, p.w, w, lane);
    const int row_at = TL::row_base(lane);
    float m = -INFINITY, l = 0.f, hit = -INFINITY;
    const int t_end = (to - from + BN - 1) / BN;
    auto step = [&](int t, const unsigned char *__restrict cur, unsigned char *__restrict next, auto special) {
        if (t + 1 < t_end) tiles.next(next, w);
        f32x16 z[KB];
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            z[b] = 0.f;
#pragma unroll
            for (int c = 0; c < DC; ++c) mma(z[b], TL::rows(cur, row_at, 32 * b, c), xf[c]);
        }
        if constexpr (decltype(special)::value) {
            const int j0 = from + t * BN + 4 * h;
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int j = j0 + 32 * b + 8 * (r / 4) + r % 4;
                    if (j == row) hit = z[b][r];
                    if (j >= to) z[b][r] = -INFINITY;
                }
        }
        // four running maxima and sums: one chain of dependent instructions would wait for each
        float m4[4] = {z[0][0], z[0][1], z[0][2], z[0][3]};
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) m4[r % 4] = fmaxf(m4[r % 4], z[b][r]);
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        const float next_m = fmaxf(m, half_max(mx)), ref = next_m * p.c;
        float sum = 0.f, s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                // with the match among them the largest score counts as exactly 1; elsewhere ref's rounding is a factor of
                // up to 1 + |ref| 2^-24 on what this tile adds, no more than lse's own rounding, and saves an instruction a
                // score
                if constexpr (decltype(special)::value) sum += exp2_fast((z[b][r] - next_m) * p.c);
                else s4[r % 4] += exp2_fast(__builtin_fmaf(z[b][r], p.c, -ref));
            }
        sum += (s4[0] + s4[1]) + (s4[2] + s4[3]);
        l = __builtin_fmaf(l, exp2_fast((m - next_m) * p.c), sum);
        m = next_m;
    };
    if (t_end > 0) {
        tiles.next(lds, w);
        tiles_ready();
        for (int t = 0; t < t_end; ++t) {
            const int j0 = from + t * BN;
            const bool special = j0 + BN > to || (j0 < row0 + BM && row0 < j0 + BN);
            if (special) step(t, lds + (t & 1) * TILE, lds + (~t & 1) * TILE, std::integral_constant<bool, true>{});
            else step(t, lds + (t & 1) * TILE, lds + (~t & 1) * TILE, std::integral_constant<bool, false>{});
            tiles_ready();
        }
    }
    l = half_sum(l);
    hit = half_max(hit);
    if (!in || h) return;
    p.ml[((int64_t)dir * p.S + blockIdx.y) * p.P + span.lo + row] = make_float2(m, l);
    if (dir == 0) {
        if (row >= from && row < to) p.hit[span.lo + row] = hit;
    }
}

__global__ __launch_bounds__(256) void loss_join_kernel(LossArgs p, float *loss, float *lse_a, float *lse_b) {
    __shared__ float red[2][4];
    int index;
    const int s = find_slot(p.cu, p.B, p.P, 1, 256, blockIdx.x, &index);
    const Span span = span_of(p.cu, p.B, p.P, s);
    const int n = span.hi - span.lo;
    if ((int64_t)index * 256 >= n) return;
    const bool one = takes_one_pass(p, s, span, red);
    const int i = span.lo + index * 256 + threadIdx.x;
    if (i >= span.hi) return;
    if (one) {
        const int each = one_piece(p, n), pieces = (n + each - 1) / each, chunks = (n + p.one_rows - 1) / p.one_rows;
        float a = 0.f, b = 0.f;
#pragma unroll 8
        for (int k = 0; k < pieces; ++k) a += p.row_sum[(int64_t)k * p.P + i];
#pragma unroll 8
        for (int k = 0; k < chunks; ++k) b += p.col_sum[(int64_t)k * p.P + i];
        const float hit = p.hit[i], by = exp2_fast(-hit * p.c);
        a = log1pf(a * by);
        b = log1pf(b * by);
        lse_a[i] = __builtin_fmaf(hit, p.inv_t, a);
        lse_b[i] = __builtin_fmaf(hit, p.inv_t, b);
        loss[i] = 0.5f * (a + b);
        return;
    }
    float top[2], log_sum[2];
    bool any = false;
    for (int dir = 0; dir < 2; ++dir) {
        const float2 *ml = p.ml + (int64_t)dir * p.S * p.P + i;
        float m = -INFINITY, l = 0.f;
        for (int k = 0; k < p.S; ++k) m = fmaxf(m, ml[(int64_t)k * p.P].x);
        for (int k = 0; k < p.S; ++k) {
            const float2 v = ml[(int64_t)k * p.P];
            if (v.y != 0.f) l += v.y * exp2_fast((v.x - m) * p.c);    // an empty piece has 0; NaN goes on into the loss
        }
        any = l != 0.f;                                        // rows outside every set have no piece
        top[dir] = m;
        log_sum[dir] = __builtin_amdgcn_logf(l);
    }
    const float hit = p.hit[i];
    lse_a[i] = any ? __builtin_fmaf(top[0], p.inv_t, log_sum[0] * LN2) : 0.f;
    lse_b[i] = any ? __builtin_fmaf(top[1], p.inv_t, log_sum[1] * LN2) : 0.f;
    loss[i] = any ? 0.5f * __builtin_fmaf((top[0] - hit) + (top[1] - hit), p.inv_t, (log_sum[0] + log_sum[1]) * LN2) : 0.f;
}

// Backward, one direction: dx of the rows, the gradient by the scores made tile by tile. fp16 holds it to few bits
// below 2^-14, where a mean over many matches lies: there g is divided by a power of two next to its largest value in
// reach first. The exponentials bound it, two a score, and waits, a third
// of its wave cycles. Where all lse in reach lie within 2^+-30 of a common e^mid, as
// they do for unit-norm rows unless t is tiny, one is enough: e^{z - lse_y} = e^{z - lse_x} e^{lse_x - mid} e^{mid -
// lse_y}, the last two known by row and column (what the first loses to underflow is below 2^-66 of g there). fp32
// inputs, bound by their products, keep both. Measured on the same: 196 us (298 with two exponentials) and 111 us
// (161). More registers for more tiles at once cost the third wave of a SIMD and were slower (372 us for forward and
// gradient against 298).
template <class T, int D, int BN>
__global__ __launch_bounds__(256, 2) void loss_bwd_kernel(LossArgs p) {
    using TL = Tile<T, D>;
    constexpr int DC = D / 16, DB = D / 32, BM = 128;
    constexpr bool exact_exp = sizeof(T) == 4;
    constexpr int TILE = BN * TL::ROW;
    __shared__ __attribute__((aligned(16))) unsigned char lds[2 * TILE + 4 * BN * 4 + 32];      // one array, as above
    float (*const st)[2 * BN] = (float (*)[2 * BN])(lds + 2 * TILE);                 // lse, then g, of a tile's columns
    float (*const reach)[4] = (float (*)[4])(lds + 2 * TILE + 4 * BN * 4);
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), h = lane >> 5;
    const int dir = blockIdx.z;
    int index;
    const int s = find_slot(p.cu, p.B, p.P, 1, BM, blockIdx.x, &index);
    const Span span = span_of(p.cu, p.B, p.P, s);
    const int n = span.hi - span.lo, row0 = index * BM;
    if (row0 >= n) return;
    int from = 0, to = 0;
    if (s != 0 && s != p.B + 1) piece_of(n, p.S, blockIdx.y, BN, &from, &to);
    const T *xs = (const T *)(dir ? p.b : p.a) + (int64_t)span.lo * p.ld, *ys = (const T *)(dir ? p.a : p.b) + (int64_t)span.lo * p.ld;
    const float *lse_x = (dir ? p.lse_b : p.lse_a) + span.lo, *lse_y = (dir ? p.lse_a : p.lse_b) + span.lo, *g = p.g + span.lo;
    const int row = row0 + w * 32 + (lane & 31);
    const bool in = row < n;
    const float unit = exact_exp ? 1.f : LOG2E;                // exponents in natural or base-2 units
    const float slope = exact_exp ? p.inv_t : p.c;
    float scale = 1.f, mid = 0.f;
    bool near = false;
    if constexpr (!exact_exp) {
        mid = lse_x[row0] * LOG2E;
        float big = 0.f, off = 0.f;
        for (int j = from + tid; j < to; j += 256) {
            off = fmaxf(off, fabsf(lse_y[j] * LOG2E - mid));
            if constexpr (scaled_ds<T>) big = fmaxf(big, fabsf(g[j]));
        }
        if (tid < BM && row0 + tid < n) {
            off = fmaxf(off, fabsf(lse_x[row0 + tid] * LOG2E - mid));
            if constexpr (scaled_ds<T>) big = fmaxf(big, fabsf(g[row0 + tid]));
        }
#pragma unroll
        for (int x = 32; x; x >>= 1) {
            off = fmaxf(off, __shfl_xor(off, x));
            if constexpr (scaled_ds<T>) big = fmaxf(big, __shfl_xor(big, x));
        }
        if (lane == 0) { reach[0][w] = off; reach[1][w] = big; }
        __syncthreads();
        off = fmaxf(fmaxf(reach[0][0], reach[0][1]), fmaxf(reach[0][2], reach[0][3]));
        big = fmaxf(fmaxf(reach[1][0], reach[1][1]), fmaxf(reach[1][2], reach[1][3]));
        near = __builtin_amdgcn_readfirstlane(off < 30.f);
        if (scaled_ds<T> && big > 0.f) scale = exp2_fast(fminf(100.f, -(float)__builtin_amdgcn_frexp_expf(big)));
    }
    const float my_g = in ? g[row] * scale : 0.f, half_g = 0.5f * my_g, my_lse = in ? lse_x[row] * unit : INFINITY;
    const float lift = near && in ? exp2_fast(my_lse - mid) : 0.f;
    Frag<T> xf[DC];
#pragma unroll
    for (int c = 0; c < DC; ++c) xf[c] = global_rows<T>(xs + (int64_t)(in ? row : n - 1) * p.ld, 16 * c + 8 * h, p.w, in);
    Walk<T, D, 4, BN> tiles(ys + (int64_t)from * p.ld, to - from, p.ld, p.w, w, lane);
    const int row_at = TL::row_base(lane), col_at = TL::col_base(lane);
    float diag = 0.f;                                          // dz_ii, kept out of the rounded products: it is the largest
    f32x16 dx[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d) dx[d] = 0.f;
    const int t_end = (to - from + BN - 1) / BN;
    float s_lse = INFINITY, s_g = 0.f;
    auto fetch = [&](int t, unsigned char *dst) {
        const int j0 = from + t * BN;
        tiles.next(dst, w);
        if (tid < BN) {
            const bool ok = j0 + tid < to;
            s_lse = ok ? lse_y[j0 + tid] : INFINITY;
            s_g = ok ? g[j0 + tid] : 0.f;
        }
    };
    auto put_stats = [&](int b) {                              // after the step: nothing waits for these loads before it
        if (tid < BN) {
            const float l = s_lse * unit, half = 0.5f * scale * s_g;
            st[b][tid] = l;
            st[b][BN + tid] = near && s_lse != INFINITY ? half * exp2_fast(mid - l) : half;    // NaN too
        }
    };
    auto step = [&](int t, const unsigned char *__restrict cur, unsigned char *__restrict next,
                    const float *__restrict st_lse, bool special) {
        if (t + 1 < t_end) fetch(t + 1, next);
#pragma unroll
        for (int b = 0; b < BN / 32; ++b) {
            f32x16 z = 0.f;
#pragma unroll
            for (int c = 0; c < DC; ++c) mma(z, TL::rows(cur, row_at, 32 * b, c), xf[c]);
            if (near) {
#pragma unroll
                for (int r4 = 0; r4 < 4; ++r4) {
                    const f32x4 gy = *reinterpret_cast<const f32x4 *>(st_lse + BN + 32 * b + 8 * r4 + 4 * h);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        z[4 * r4 + e] = exp2_fast(__builtin_fmaf(z[4 * r4 + e], slope, -my_lse)) *
                                        __builtin_fmaf(gy[e], lift, half_g);
                }
            } else {
#pragma unroll
                for (int r4 = 0; r4 < 4; ++r4) {
                    const int k0 = 32 * b + 8 * r4 + 4 * h;
                    const f32x4 ly = *reinterpret_cast<const f32x4 *>(st_lse + k0);
                    const f32x4 gy = *reinterpret_cast<const f32x4 *>(st_lse + BN + k0);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float v = z[4 * r4 + e];
                        float ux = __builtin_fmaf(v, slope, -my_lse), uy = __builtin_fmaf(v, slope, -ly[e]);
                        if constexpr (exact_exp) { ux *= LOG2E; uy *= LOG2E; }
                        z[4 * r4 + e] = __builtin_fmaf(gy[e], exp2_fast(uy), half_g * exp2_fast(ux));
                    }
                }
            }
            if (special) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int j = from + t * BN + 32 * b + 8 * (r / 4) + 4 * h + r % 4;
                    if (j == row) diag = z[r] - my_g;
                    if (j == row || j >= to) z[r] = 0.f;
                }
            }
#pragma unroll
            for (int kc = 0; kc < 2; ++kc) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = z[kc * 8 + e];
                const Frag<T> zf = to_frag<T>(v);
#pragma unroll
                for (int d = 0; d < DB; ++d) mma(dx[d], TL::cols(cur, col_at, 32 * b + 16 * kc, 32 * d), zf);
            }
        }
    };
    if (t_end > 0) {
        fetch(0, lds);
        put_stats(0);
        tiles_ready();
        for (int t = 0; t < t_end; ++t) {
            const int j0 = from + t * BN;
            const bool special = j0 + BN > to || (j0 < row0 + BM && row0 < j0 + BN);
            step(t, lds + (t & 1) * TILE, lds + (~t & 1) * TILE, st[t & 1], special);
            if (t + 1 < t_end) put_stats((t + 1) & 1);
            tiles_ready();
        }
    }
    diag = half_sum(diag);
    if (!in) return;
    const float f = p.inv_t / scale;
    if (diag != 0.f) {
        const T *match = ys + (int64_t)row * p.ld;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int col = 32 * d + 8 * (r / 4) + 4 * h + r % 4;
                if (col < p.d) dx[d][r] = __builtin_fmaf(diag, (float)match[col], dx[d][r]);
            }
    }
    if (p.part) {
        float *out = p.part + (((int64_t)dir * p.S + blockIdx.y) * p.P + span.lo + row) * D;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int r = 0; r < 16; r += 4)
                store4<float>(out + 32 * d + 8 * (r / 4) + 4 * h, dx[d][r] * f, dx[d][r + 1] * f, dx[d][r + 2] * f, dx[d][r + 3] * f);
    } else {
        T *out = (T *)(dir ? p.db : p.da) + (int64_t)(span.lo + row) * p.d;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const int col = 32 * d + 8 * (r / 4) + 4 * h;
                if (col < p.d) store4<T>(out + col, dx[d][r] * f, dx[d][r + 1] * f, dx[d][r + 2] * f, dx[d][r + 3] * f);
            }
    }
}

// da (blockIdx.y = 0) and db (1) from the pieces.
template <class T>
__global__ __launch_bounds__(256) void loss_sum_kernel(LossArgs p, int dp) {
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= (int64_t)p.P * p.d) return;
    const int64_t i = e / p.d, c = e % p.d;
    const float *part = p.part + ((int64_t)blockIdx.y * p.S * p.P + i) * dp + c;
    float sum = 0.f;
    for (int s = 0; s < p.S; ++s) sum += part[(int64_t)s * p.P * dp];
    ((T *)(blockIdx.y ? p.db : p.da))[e] = (T)sum;
}

// Rows that are not whole 16-byte pieces at 16-byte boundaries: copied with zeros up to dp elements.
template <class T>
__global__ __launch_bounds__(256) void loss_repack_kernel(const T *a, const T *b, int P, int d, int dp, T *out) {
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= (int64_t)P * dp) return;
    const int64_t i = e / dp, c = e % dp;
    out[(int64_t)blockIdx.y * P * dp + e] = c < d ? (blockIdx.y ? b : a)[i * d + c] : (T)0.f;
}

int esize(int dtype) { return dtype == DDM_F32 ? 4 : 2; }

struct Plan {
    int dp, S;                       // padded components, pieces of a set's columns
    bool direct;                     // backward writes da and db straight away
    bool one;                        // sets may take one pass
    int slots, one_rows, one_slots, pieces, one_pieces;
    // what the workspace holds: repacked rows first, then what the forward pass keeps between its kernels, or the backward's parts
    size_t rows, ml, hit, top, row_sum, col_sum, part, forward_bytes, backward_bytes;
};

constexpr size_t ONE_BYTES = (size_t)1 << 30;

// Some 512 row tiles of 128 and pieces: two directions make 1024 workgroups, four on each CU.
Plan make_plan(int B, int P, int d, int dtype) {
    Plan p{};
    p.dp = d <= 32 ? 32 : d <= 64 ? 64 : 128;
    const long long tiles = P / 128 + B;
    p.S = (int)std::min<long long>(std::max<long long>(512 / tiles, 1), 16);
    while (p.S > 1 && (long long)P / B / p.S < 64) p.S /= 2;     // a piece has a tile of columns on average
    p.direct = p.S == 1 && d % 4 == 0;
    size_t at = 0;
    auto take = [&](size_t n) { const size_t o = at; at += (n + 255) / 256 * 256; return o; };
    p.rows = take(2 * (size_t)P * p.dp * esize(dtype));
    p.part = at;
    p.backward_bytes = std::max<size_t>(at + (p.direct ? 0 : 2 * (size_t)p.S * P * p.dp * 4), 256);
    p.ml = take(2 * (size_t)p.S * P * sizeof(float2));
    p.hit = take((size_t)P * 4);
    // From 4096 matches on the two launches more are paid back, with the gradient: 4096 x 24 bf16 51 us against 55 in two
    // passes, fp32 100 against 109, 8000 x 24 fp32 234 against 272, 16384 x 64 bf16 270 against 293 (not quite for 24
    // components in 16 bits between: 8000 x 24 bf16 82 against 79); below they are not: 3000 x 24 bf16 49 against 48.
    p.one = P >= 4096;
    p.slots = (int)slot_count(B, P, 1, 128);
    // A chunk of rows leaves a sum for each column of its set, which may be any length up to ONE_N: 512 bytes a match with
    // chunks of 256. Longer ones bound that where there are workgroups enough without (200 sets of 4000 x 24 fp16, with the
    // gradient: 2057 us against 2129 with 256; 1000 of 1000: 1039 against 1273); past ONE_BYTES for
    // all sums, 4 M matches, every set takes two passes, which need none of them.
    p.one_rows = P <= 1 << 18 ? 256 : P <= 1 << 19 ? 512 : 1024;
    p.one_pieces = (int)std::min<long long>(std::max<long long>(1024 / (P / p.one_rows + B), 1), 32);
    p.pieces = std::max(p.one_pieces, (std::min(P, ONE_N) + ONE_COLS - 1) / ONE_COLS);
    p.one_slots = (int)slot_count(B, P, 1, p.one_rows);
    const size_t row_bytes = (size_t)p.pieces * P * 4, col_bytes = (size_t)((std::min(P, ONE_N) + p.one_rows - 1) / p.one_rows) * P * 4;
    p.one = p.one && row_bytes + col_bytes <= ONE_BYTES;
    p.top = take(p.one ? 2 * (size_t)p.slots * 4 : 0);
    p.row_sum = take(p.one ? row_bytes : 0);
    p.col_sum = take(p.one ? col_bytes : 0);
    p.forward_bytes = std::max<size_t>(at, 256);
    return p;
}

int check(int B, int P, int d, int dtype) {
    if (dtype != DDM_F32 && dtype != DDM_F16 && dtype != DDM_BF16) return DDM_ERR_UNSUPPORTED;
    if (d < 1 || d > DDM_MAX_D) return DDM_ERR_UNSUPPORTED;
    if (B < 1 || B > (1 << 20) || P < 0 || P > (1 << 24)) return DDM_ERR_INVALID;
    return DDM_OK;
}
// The kernels' 32-bit 1 / t and log2(e) / t: as 0 or infinity they would make NaN of a -inf or of a zero.
bool bad_temperature(double t) {
    return !(t > 0) || !std::isnormal((float)(1.0 / t)) || !std::isnormal((float)(1.4426950408889634 / t));
}
bool off(const void *p, int e) { return !p || (uintptr_t)p % e; }

template <class F>
hipError_t with_type(int dtype, int dp, F f) {
    auto go = [&](auto t) {
        if (dp == 32) return f(t, std::integral_constant<int, 32>{});
        if (dp == 64) return f(t, std::integral_constant<int, 64>{});
        return f(t, std::integral_constant<int, 128>{});
    };
    if (dtype == DDM_F32) return go(float{});
    if (dtype == DDM_F16) return go(_Float16{});
    return go(__bf16{});
}

// Rows as the kernels read them: in place, or repacked.
template <class T>
hipError_t rows_for(LossArgs &p, const Plan &pl, unsigned char *ws, hipStream_t s) {
    p.ld = p.w = p.d;
    if (p.d * sizeof(T) % 16 == 0 && (uintptr_t)p.a % 16 == 0 && (uintptr_t)p.b % 16 == 0) return hipSuccess;
    T *out = (T *)(ws + pl.rows);
    const int64_t n = (int64_t)p.P * pl.dp;
    hipLaunchKernelGGL((loss_repack_kernel<T>), dim3((unsigned)((n + 255) / 256), 2), dim3(256), 0, s, (const T *)p.a,
                       (const T *)p.b, p.P, p.d, pl.dp, out);
    p.a = out;
    p.b = out + n;
    p.ld = p.w = pl.dp;
    return hipGetLastError();
}

}  // namespace

extern "C" {

size_t ddm_matching_loss_forward_workspace_bytes(int B, int P, int d, int dtype) {
    return check(B, P, d, dtype) == DDM_OK ? make_plan(B, P, d, dtype).forward_bytes : 0;
}
size_t ddm_matching_loss_backward_workspace_bytes(int B, int P, int d, int dtype) {
    return check(B, P, d, dtype) == DDM_OK ? make_plan(B, P, d, dtype).backward_bytes : 0;
}
size_t ddm_matching_loss_workspace_bytes(int B, int P, int d, int dtype) {
    return std::max(ddm_matching_loss_forward_workspace_bytes(B, P, d, dtype),
                    ddm_matching_loss_backward_workspace_bytes(B, P, d, dtype));
}

int ddm_matching_loss_forward(const void *a, const void *b, const int32_t *cu, int B, int P, int d, int dtype,
                              double temperature, float *loss, float *lse_a, float *lse_b, void *workspace,
                              size_t workspace_bytes, hipStream_t stream) {
    if (int rc = check(B, P, d, dtype)) return rc;
    if (bad_temperature(temperature) || (!cu && B != 1)) return DDM_ERR_INVALID;
    if (P == 0) return DDM_OK;
    if (off(a, esize(dtype)) || off(b, esize(dtype)) || off(loss, 4) || off(lse_a, 4) || off(lse_b, 4)) return DDM_ERR_INVALID;
    const Plan pl = make_plan(B, P, d, dtype);
    if (off(workspace, 16) || workspace_bytes < pl.forward_bytes) return DDM_ERR_WORKSPACE;
    unsigned char *ws = (unsigned char *)workspace;
    LossArgs p{};
    p.a = a; p.b = b; p.cu = cu; p.B = B; p.P = P; p.d = d; p.S = pl.S;
    p.c = (float)(1.4426950408889634 / temperature); p.inv_t = (float)(1.0 / temperature);
    p.ml = (float2 *)(ws + pl.ml); p.hit = (float *)(ws + pl.hit);
    p.slots = pl.slots; p.one_rows = pl.one_rows; p.one_pieces = pl.one_pieces;
    if (pl.one) {
        p.top = (float *)(ws + pl.top); p.row_sum = (float *)(ws + pl.row_sum); p.col_sum = (float *)(ws + pl.col_sum);
    }
    const hipError_t e = with_type(dtype, pl.dp, [&](auto t, auto dp) {
        using T = decltype(t);
        if (hipError_t r = rows_for<T>(p, pl, ws, stream)) return r;
        // 16-bit rows: tiles of 128 columns (16384 x 64 bf16, with the gradient: 300 us against 325 with 64, 342 with
        // 32); fp32 ones would fill LDS with one workgroup
        constexpr int BN = sizeof(T) == 4 ? 64 : 128;
        if (pl.one) {
            hipLaunchKernelGGL((loss_top_kernel<T>), dim3(pl.slots, 2), dim3(256), 0, stream, p);
            if (hipError_t r = hipGetLastError()) return r;
            hipLaunchKernelGGL((loss_one_kernel<T, decltype(dp)::value, 64>), dim3(pl.one_slots, pl.pieces), dim3(256), 0,
                               stream, p);
            if (hipError_t r = hipGetLastError()) return r;
        }
        hipLaunchKernelGGL((loss_fwd_kernel<T, decltype(dp)::value, BN>), dim3(pl.slots, pl.S, 2), dim3(256), 0, stream, p);
        if (hipError_t r = hipGetLastError()) return r;
        hipLaunchKernelGGL(loss_join_kernel, dim3((unsigned)slot_count(B, P, 1, 256)), dim3(256), 0, stream, p, loss, lse_a,
                           lse_b);
        return hipGetLastError();
    });
    return e == hipSuccess ? DDM_OK : DDM_ERR_HIP;
}

int ddm_matching_loss_backward(const float *dloss, const void *a, const void *b, const float *lse_a, const float *lse_b,
                               const int32_t *cu, int B, int P, int d, int dtype, double temperature, void *da, void *db,
                               void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if (int rc = check(B, P, d, dtype)) return rc;
    if (bad_temperature(temperature) || (!cu && B != 1)) return DDM_ERR_INVALID;
    if (P == 0) return DDM_OK;
    const int es = esize(dtype);
    if (off(a, es) || off(b, es) || off(dloss, 4) || off(lse_a, 4) || off(lse_b, 4) || off(da, es) || off(db, es))
        return DDM_ERR_INVALID;
    const Plan pl = make_plan(B, P, d, dtype);
    if (off(workspace, 16) || workspace_bytes < pl.backward_bytes) return DDM_ERR_WORKSPACE;
    unsigned char *ws = (unsigned char *)workspace;
    LossArgs p{};
    p.a = a; p.b = b; p.cu = cu; p.B = B; p.P = P; p.d = d; p.S = pl.S;
    p.c = (float)(1.4426950408889634 / temperature); p.inv_t = (float)(1.0 / temperature);
    p.g = dloss; p.lse_a = lse_a; p.lse_b = lse_b; p.da = da; p.db = db;
    const bool aligned = (uintptr_t)da % 16 == 0 && (uintptr_t)db % 16 == 0;
    if (!pl.direct) p.part = (float *)(ws + pl.part);
    else if (!aligned) return DDM_ERR_INVALID;
    const hipError_t e = with_type(dtype, pl.dp, [&](auto t, auto dp) {
        using T = decltype(t);
        if (hipError_t r = rows_for<T>(p, pl, ws, stream)) return r;
        hipLaunchKernelGGL((loss_bwd_kernel<T, decltype(dp)::value, 64>), dim3((unsigned)slot_count(B, P, 1, 128), pl.S, 2),
                           dim3(256), 0, stream, p);
        hipError_t r = hipGetLastError();
        if (r == hipSuccess && p.part) {
            const int64_t n = (int64_t)P * d;
            hipLaunchKernelGGL((loss_sum_kernel<T>), dim3((unsigned)((n + 255) / 256), 2), dim3(256), 0, stream, p,
                               decltype(dp)::value);
            r = hipGetLastError();
        }
        return r;
    });
    return e == hipSuccess ? DDM_OK : DDM_ERR_HIP;
}

}  // extern "C"

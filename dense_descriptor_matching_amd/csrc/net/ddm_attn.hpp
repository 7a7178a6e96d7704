// ddm_attn.hpp -- attention over packed sequences, forward and backward.
//
//   z_ij = scale q_i . k_j,  lse_i = log sum_j e^{z_ij},  P_ij = e^{z_ij - lse_i},  o_i = sum_j P_ij v_j
//   D_i = do_i . o_i,  dS_ij = P_ij (do_i . v_j - D_i)
//   dv_j = sum_i P_ij do_i,  dk_j = scale sum_i dS_ij q_i,  dq_i = scale sum_j dS_ij k_j
// over the keys j that query i of its sequence sees: all, or with causal j <= i + Lk - Lq.
//
// The G = Hq / Hkv query heads that share a key head are rows of one problem: row r of a sequence is query r / G, head
// r % G of the group, so a key tile in LDS serves all of them and the sum of dk and dv over the group is a product's.
#pragma once
#include "ddm_tile.hpp"

namespace ddm {

struct AttnArgs {
    const void *q, *k, *v, *o, *dout;     // o: forward writes it through `out`, backward reads it here
    void *out, *dq, *dk, *dv;
    float *lse;                           // [Tq][Hq]
    float *stats;                         // backward: [Tq][Hq] of lse_i log2(e) (infinity for an empty row), of D_i and, for fp16,
                                          // of the exponent of the row's largest |do| less NO_EXPONENT
    const int32_t *cu_q, *cu_k;
    int B, Tq, Tk, Hq, Hkv, D;
    Div group;
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, g_ts, g_hs;   // token and head strides in elements (g: dout)
    float scale, c;                       // c = scale log2(e)
    int causal;
    int rt, parts;                        // attn_dkv_kernel: rows of a tile, most parts of a key tile's rows
    int chunk, cap;                       // split form: keys of a chunk, rows of a sequence that are split
    float *part;                          // split form: [slot][Hkv][cap][D + 4]; attn_dkv_kernel: [slot][Hkv][parts][2][keys][padded D]
};

// Workgroups go round-robin to the 8 XCDs, each with its own L2: with 8 | Hkv a key head's workgroups stay on one XCD.
__device__ __forceinline__ int key_head(int x, int heads) { return (heads & 7) ? x : (x & 7) * (heads >> 3) + (x >> 3); }

// Bytes from row 0 of `rows` strided rows of d elements to the end of the last.
template <class T>
__device__ __forceinline__ int64_t rows_bytes(int rows, int64_t ts, int d) {
    return rows <= 0 ? 0 : ((int64_t)(rows - 1) * ts + d) * (int64_t)sizeof(T);
}

// Operand rows straight from global memory: 8 elements at k positions 16 c + 8 h of a row, zeros past d or without a
// row.
template <class T>
__device__ __forceinline__ Frag<T> global_rows(const T *row, int k, int d, bool in) {
    Frag<T> f = {};
    if (!in) return f;
    if constexpr (sizeof(T) == 2) {
        if (k < d) f = *reinterpret_cast<const Frag<T> *>(row + k);
    } else {
        if (k < d) {
            const f32x4 a = *reinterpret_cast<const f32x4 *>(row + k);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = a[i];
        }
        if (k + 4 < d) {
            const f32x4 a = *reinterpret_cast<const f32x4 *>(row + k + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i + 4] = a[i];
        }
    }
    return f;
}

// Four consecutive elements of an output row, rounded once.
template <class T>
__device__ __forceinline__ void store4(T *p, float a, float b, float c, float d) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<f32x4 *>(p) = f32x4{a, b, c, d};
    } else {
        typedef T t4 __attribute__((ext_vector_type(4)));
        *reinterpret_cast<t4 *>(p) = t4{(T)a, (T)b, (T)c, (T)d};
    }
}

// --------------------------------------------------------------------------------------------------------- forward
// A workgroup takes BM = 32 NW rows (each wave 32) and walks over the keys in tiles of BN, which have two places in
// LDS: while one is used, the next is on its way. Running maximum m (in units of log2) and sum l per row; the
// accumulator is rescaled only when a row's maximum has grown by more than 8 since the last time (any reference gives
// the same quotient; p stays below 2^8, far inside fp16 and bf16). p is rounded to the inputs' type for the second
// product, which the matrix cores take; l sums it before that. Bound by the matrix cores and the vector units together,
// which overlap by a quarter here: 64 components are 16 matrix and some 16 vector cycles a score (the exponential alone
// 8), 128 are 32 and 16. Four waves of 32 rows: two row blocks a wave, eight waves, 32 or 128 keys a tile, and scores
// of the next tile begun before a tile's exponentials were all slower. Measured: 114 us for 32 x 768 tokens of 16 heads
// of 64 fp16 (680 TFLOP/s), 345 us for 11949 causal tokens of 32 over 8 heads of 128 bf16 (955 TFLOP/s; a large library
// product reaches 1185 here).
// SPLIT: the workgroup takes a chunk of the keys, for few rows and many keys; attn_join joins the chunks. Bound by
// memory: one wave with 32 KB of tiles, so that five are on a CU; 56 us for 67469 keys of 8 heads of 128 bf16 (276 MB,
// 4.9 TB/s; a large copy 4.8).
template <class T, int D, int NW, int BN, bool SPLIT>
__global__ __launch_bounds__(NW * 64, 2) void attn_fwd_kernel(AttnArgs p) {
    using TL = Tile<T, D>;
    constexpr int BM = NW * 32, KB = BN / 32, DC = D / 16, DB = D / 32;
    constexpr int TILE_BYTES = BN * TL::ROW;
    __shared__ __attribute__((aligned(16))) unsigned char lds[2][2 * TILE_BYTES];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = lane >> 5, n = lane & 31;
    const int G = p.group.g;

    int hk, s, index, row_tile;
    if constexpr (SPLIT) {
        hk = blockIdx.x % p.Hkv;
        row_tile = blockIdx.y;
        s = find_slot(p.cu_k, p.B, p.Tk, 1, p.chunk, blockIdx.x / p.Hkv, &index);
        if (s == 0 || s == p.B + 1) return;
    } else {
        const int heads = p.Hkv;
        hk = key_head(blockIdx.x % heads, heads);
        const int slots = gridDim.x / heads;
        // the last rows of a causal sequence see the most keys: they start first
        s = find_slot(p.cu_q, p.B, p.Tq, G, BM, slots - 1 - blockIdx.x / heads, &index);
        row_tile = index;
    }
    const Span sq = span_of(p.cu_q, p.B, p.Tq, s);
    Span sk = span_of(p.cu_k, p.B, p.Tk, s);
    if (s == 0 || s == p.B + 1) sk.hi = sk.lo;
    const int rows = (sq.hi - sq.lo) * G, Lk = sk.hi - sk.lo, shift = Lk - (sq.hi - sq.lo);
    int k_from = 0, k_to = Lk;
    bool whole = !SPLIT;
    int chunks = 1;
    if constexpr (SPLIT) {
        chunks = (Lk + p.chunk - 1) / p.chunk;
        if (index >= chunks) return;
        k_from = index * p.chunk;
        k_to = min(Lk, k_from + p.chunk);
    }
    const T *kb = (const T *)p.k + (int64_t)sk.lo * p.k_ts + (int64_t)hk * p.k_hs;
    const T *vb = (const T *)p.v + (int64_t)sk.lo * p.v_ts + (int64_t)hk * p.v_hs;
    const int row_at = TL::row_base(lane), col_at = TL::col_base(lane);

    for (;;) {
        const int row0 = row_tile * BM;
        if (row0 >= rows) return;
        const int row = row0 + w * 32 + n;                   // this lane's
        const bool in = row < rows;
        const int rr = in ? row : rows - 1, qi = (int)div_by(rr, p.group), head = hk * G + (rr - qi * G);
        const int lim = p.causal ? min(k_to, qi + shift + 1) : k_to;
        const T *qr = (const T *)p.q + (int64_t)(sq.lo + qi) * p.q_ts + (int64_t)head * p.q_hs;
        Frag<T> qf[DC];
#pragma unroll
        for (int c = 0; c < DC; ++c) qf[c] = global_rows<T>(qr, 16 * c + 8 * h, p.D, in);
        int top = k_to, low = k_to;                          // keys that the last and the first row see
        if (p.causal) {
            top = min(k_to, (int)div_by(min(row0 + BM, rows) - 1, p.group) + shift + 1);
            low = min(k_to, (int)div_by(row0, p.group) + shift + 1);
        }
        const int t_end = top > k_from ? (top - k_from + BN - 1) / BN : 0;
        int wave_top = 0;                                    // keys from here on no row of this wave sees
        if (const int last = min(row0 + (w + 1) * 32, rows) - 1; last >= row0 + w * 32)
            wave_top = p.causal ? min(k_to, (int)div_by(last, p.group) + shift + 1) : k_to;

        f32x16 o[DB];
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int d = 0; d < DB; ++d) o[d] = 0.f;

        Walk<T, D, NW, BN> ks(kb + (int64_t)k_from * p.k_ts, k_to - k_from, p.k_ts, p.D, w, lane);
        Walk<T, D, NW, BN> vs(vb + (int64_t)k_from * p.v_ts, k_to - k_from, p.v_ts, p.D, w, lane);
        auto fetch = [&](unsigned char *to) {
            ks.next(to, w);
            vs.next(to + TILE_BYTES, w);
        };
        auto step = [&](int t, const unsigned char *__restrict cur, unsigned char *__restrict next, bool masked) {
            if (t + 1 < t_end) fetch(next);
            if (k_from + t * BN >= wave_top) return;
            const unsigned char *kt = cur, *vt = cur + TILE_BYTES;
            f32x16 z[KB];
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                z[b] = 0.f;
#pragma unroll
                for (int c = 0; c < DC; ++c) mma(z[b], TL::rows(kt, row_at, 32 * b, c), qf[c]);
            }
            if (masked) {
                const int j0 = k_from + t * BN + 4 * h;
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (j0 + 32 * b + 8 * (r / 4) + r % 4 >= lim) z[b][r] = -INFINITY;
            }
            float mx = z[0][0];
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) mx = fmaxf(mx, z[b][r]);
            mx = half_max(mx) * p.c;
            if (__any(mx > m + 8.f)) {
                const float next = fmaxf(m, mx);
                const float a = next == -INFINITY ? 1.f : exp2_fast(m - next);
                l *= a;
#pragma unroll
                for (int d = 0; d < DB; ++d) o[d] *= a;
                m = next;
            }
            const float ref = m == -INFINITY ? 0.f : m;
            float sum = 0.f;
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    z[b][r] = exp2_fast(__builtin_fmaf(z[b][r], p.c, -ref));
                    sum += z[b][r];
                }
            l += sum;
#pragma unroll
            for (int kc = 0; kc < BN / 16; ++kc) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = z[kc / 2][(kc & 1) * 8 + e];
                const Frag<T> pf = to_frag<T>(x);
#pragma unroll
                for (int d = 0; d < DB; ++d) mma(o[d], TL::cols(vt, col_at, 16 * kc, 32 * d), pf);
            }
        };

        if (t_end > 0) {
            fetch(lds[0]);
            tiles_ready();
            const int t_full = max(0, min(t_end, (low - k_from) / BN));      // tiles that every row sees whole
            for (int t = 0; t < t_end; ++t) {
                step(t, lds[t & 1], lds[(t + 1) & 1], t >= t_full);
                tiles_ready();
            }
        }

        // the row's sum over both lane halves; the row is this lane's column
        const float sum = half_sum(l);
        if (in && whole) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;   // 0: no key seen; a NaN among the scores goes on into out and lse
            const int64_t at = (int64_t)(sq.lo + qi) * p.Hq + head;
            T *orow = (T *)p.out + at * p.D;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int r = 0; r < 16; r += 4) {
                    const int col = 32 * d + 8 * (r / 4) + 4 * h;
                    if (col < p.D)
                        store4<T>(orow + col, o[d][r] * inv, o[d][r + 1] * inv, o[d][r + 2] * inv, o[d][r + 3] * inv);
                }
            if (h == 0) p.lse[at] = sum == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(sum)) * 0.69314718055994531f;
        } else if (in) {
            float *part = p.part + ((int64_t)blockIdx.x * p.cap + row) * (p.D + 4);
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int r = 0; r < 16; r += 4) {
                    const int col = 32 * d + 8 * (r / 4) + 4 * h;
                    if (col < p.D) store4<float>(part + 4 + col, o[d][r], o[d][r + 1], o[d][r + 2], o[d][r + 3]);
                }
            if (h == 0) { part[0] = m; part[1] = sum; }
        }
        if constexpr (!SPLIT) return;
        // rows past the split ones (longer sequences than the call's average): whole tiles, shared out over the chunks
        if (!whole && row_tile != 0) return;
        row_tile = whole ? row_tile + chunks : p.cap / BM + index;
        whole = true;
        k_from = 0;
        k_to = Lk;
        __syncthreads();
    }
}

// Joins the chunks of the split form: a workgroup for each (query, head). Every chunk's weight first, one thread each;
// then DP / 4 threads a chunk add up its row, 1024 / DP chunks at a time, eight 16-byte loads in flight a thread. Bound
// by latency: 5.7 us for 192 rows of up to 79 chunks.
constexpr int MAX_CHUNKS = 1040;          // of one sequence; the plan's chunks are at least 1024th parts of all keys
template <class T, int DP>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs p) {
    constexpr int TP = DP / 4, GROUPS = 256 / TP;             // threads of a chunk, chunks at a time
    __shared__ float weight[MAX_CHUNKS], red[2][4];
    __shared__ __attribute__((aligned(16))) f32x4 rows[GROUPS][TP];
    const int tid = threadIdx.x, lane = tid & 63;
    const int tok = blockIdx.x / p.Hq, head = blockIdx.x % p.Hq;
    int sq = -1;                                                // the last sequence that begins at or before the token
    for (int base = 0; base < p.B + 2; base += 64) {
        const int x = base + lane;
        const int c = __popcll(__ballot(x < p.B + 2 && bound_at(p.cu_q, p.B, p.Tq, x) <= tok));
        sq += c;
        if (c < 64) break;
    }
    sq = __builtin_amdgcn_readfirstlane(sq);
    const Span q = span_of(p.cu_q, p.B, p.Tq, sq);
    Span k = span_of(p.cu_k, p.B, p.Tk, sq);
    if (sq == 0 || sq == p.B + 1) k.hi = k.lo;
    const int G = p.group.g, hk = head / G, r = (tok - q.lo) * G + head % G;
    const int chunks = (k.hi - k.lo + p.chunk - 1) / p.chunk;
    if (r < 0 || (chunks > 0 && r >= p.cap)) return;            // cu out of order; rows that were written whole
    const int slot0 = k.lo / p.chunk + sq;
    const float *part = p.part + (((int64_t)slot0 * p.Hkv + hk) * p.cap + r) * (p.D + 4);
    const int64_t pitch = (int64_t)p.Hkv * p.cap * (p.D + 4);
    float top = -INFINITY;
    for (int c = tid; c < chunks; c += 256) {
        weight[c] = part[c * pitch];
        top = fmaxf(top, weight[c]);
    }
#pragma unroll
    for (int x = 32; x; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
    if (lane == 0) red[0][tid >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    for (int c = tid; c < chunks; c += 256) {
        const float f = exp2_fast(weight[c] - ref);
        weight[c] = f;
        sum = __builtin_fmaf(f, part[c * pitch + 1], sum);
    }
#pragma unroll
    for (int x = 32; x; x >>= 1) sum += __shfl_xor(sum, x);
    if (lane == 0) red[1][tid >> 6] = sum;
    __syncthreads();
    sum = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
    const int col = tid % TP * 4, g = tid / TP;
    f32x4 a = 0.f;
    if (col < p.D) {
#pragma unroll 8
        for (int c = g; c < chunks; c += GROUPS) a += weight[c] * *reinterpret_cast<const f32x4 *>(part + c * pitch + 4 + col);
    }
    rows[g][tid % TP] = a;
    __syncthreads();
    if (g == 0 && col < p.D) {
#pragma unroll
        for (int x = 1; x < GROUPS; ++x) a += rows[x][tid];
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        store4<T>((T *)p.out + (int64_t)blockIdx.x * p.D + col, a[0] * inv, a[1] * inv, a[2] * inv, a[3] * inv);
        if (col == 0) p.lse[blockIdx.x] = sum == 0.f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * 0.69314718055994531f;
    }
}

// -------------------------------------------------------------------------------------------------------- backward
// fp16 holds dS to few bits once it is below 2^-14, which small gradients make it; there each row's dS is divided by
// the power of two next to its largest |do| before it is rounded, and the products are multiplied back in fp32. So
// |P (do.v - D)| may be up to some 2^16 times the row's largest |do|: v of several thousand in every component.
template <class T> constexpr bool scaled_ds = sizeof(T) == 2 && !std::is_same_v<T, __bf16>;
constexpr float NO_EXPONENT = -100.f;

// dq and D_i, one row block at a time as in the forward pass: S and dO V^T of 32 keys from two key tiles' rows, then dS
// times K from the key tile's columns. No sum crosses workgroups, so the result does not depend on their order; the
// price is that S and dO V^T are computed here and again in attn_dkv_kernel (7 products instead of 5). A row's dS sum
// to zero before they are rounded and about to zero after (D_i is taken from the rounded out), so that a mean which all
// keys share reaches dq by the sum of the roundings: with keys of mean 1 and spread 1 the error is 0.0039 of dq's norm in
// bfloat16, with keys of mean 0 0.0024. No centre is subtracted from the keys: one that lies far from those that a row
// attends carries that sum into dq without bound. Measured: 200 us for 8634 causal tokens of 16 over 4 heads of 128 bf16
// (830 TFLOP/s), 47 us for 6446 tokens over 6453 of 12 heads of 64 (490 TFLOP/s); bound as the forward pass is.
template <class T, int D, int NW, int BN>
__global__ __launch_bounds__(NW * 64, sizeof(T) == 2 && D == 64 ? 3 : 2) void attn_dq_kernel(AttnArgs p) {
    using TL = Tile<T, D>;
    constexpr int BM = NW * 32, DC = D / 16, DB = D / 32;
    constexpr int TILE_BYTES = BN * TL::ROW;
    // One array: of several, the compiler takes the loads to LDS to alias what is read, and waits for the next tile in
    // every step (training, with the dk/dv kernel's: 32 x 768 tokens of 64 bf16 446 us against 451, of 32 105 against 112).
    // 64 components in 16 bits: held to the registers of three waves a SIMD (cross pairs 122 us, with two 128).
    __shared__ __attribute__((aligned(16))) unsigned char lds[4 * TILE_BYTES];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = lane >> 5, n = lane & 31;
    const int G = p.group.g;

    const int heads = p.Hkv, hk = key_head(blockIdx.x % heads, heads);
    int row_tile;
    const int s = find_slot(p.cu_q, p.B, p.Tq, G, BM, gridDim.x / heads - 1 - blockIdx.x / heads, &row_tile);
    const Span sq = span_of(p.cu_q, p.B, p.Tq, s);
    Span sk = span_of(p.cu_k, p.B, p.Tk, s);
    if (s == 0 || s == p.B + 1) sk.hi = sk.lo;
    const int rows = (sq.hi - sq.lo) * G, Lk = sk.hi - sk.lo, shift = Lk - (sq.hi - sq.lo), row0 = row_tile * BM;
    if (row0 >= rows) return;
    const T *kb = (const T *)p.k + (int64_t)sk.lo * p.k_ts + (int64_t)hk * p.k_hs;
    const T *vb = (const T *)p.v + (int64_t)sk.lo * p.v_ts + (int64_t)hk * p.v_hs;
    const int row_at = TL::row_base(lane), col_at = TL::col_base(lane);

    const int r = row0 + w * 32 + n;
    const bool in = r < rows;
    const int rr = in ? r : rows - 1, qi = (int)div_by(rr, p.group), head = hk * G + (rr - qi * G);
    const int lim = p.causal ? min(Lk, qi + shift + 1) : Lk;
    const int64_t tok = sq.lo + qi, at = tok * p.Hq + head;
    const T *qr = (const T *)p.q + tok * p.q_ts + (int64_t)head * p.q_hs;
    const T *gr = (const T *)p.dout + tok * p.g_ts + (int64_t)head * p.g_hs;
    const T *orow = (const T *)p.o + at * p.D;
    Frag<T> qf[DC], gf[DC];
    float delta = 0.f, big = 0.f;
#pragma unroll
    for (int c = 0; c < DC; ++c) {
        qf[c] = global_rows<T>(qr, 16 * c + 8 * h, p.D, in);
        gf[c] = global_rows<T>(gr, 16 * c + 8 * h, p.D, in);
        const Frag<T> of = global_rows<T>(orow, 16 * c + 8 * h, p.D, in);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            delta = __builtin_fmaf((float)gf[c][e], (float)of[e], delta);
            if constexpr (scaled_ds<T>) big = fmaxf(big, fabsf((float)gf[c][e]));
        }
    }
    delta = half_sum(delta);
    const float z = in ? p.lse[at] : -INFINITY;
    const float lse = z == -INFINITY ? INFINITY : z * 1.44269504088896341f;      // a row that sees no key: every P is 0
    float inv = 1.f, ex = NO_EXPONENT;
    if constexpr (scaled_ds<T>) {
        big = half_max(big);
        if (big > 0.f) ex = fmaxf(NO_EXPONENT, (float)__builtin_amdgcn_frexp_expf(big));
        inv = exp2_fast(-ex);
    }
    if (in && h == 0) {
        const int64_t all = (int64_t)p.Tq * p.Hq;
        p.stats[at] = lse;
        p.stats[at + all] = delta;
        if constexpr (scaled_ds<T>) p.stats[at + 2 * all] = ex - NO_EXPONENT;
    }
    int top = Lk, low = Lk;
    if (p.causal) {
        top = min(Lk, (int)div_by(min(row0 + BM, rows) - 1, p.group) + shift + 1);
        low = min(Lk, (int)div_by(row0, p.group) + shift + 1);
    }
    const int t_end = top > 0 ? (top + BN - 1) / BN : 0;
    int wave_top = 0;
    if (const int last = min(row0 + (w + 1) * 32, rows) - 1; last >= row0 + w * 32)
        wave_top = p.causal ? min(Lk, (int)div_by(last, p.group) + shift + 1) : Lk;

    f32x16 dq[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d) dq[d] = 0.f;

    Walk<T, D, NW, BN> ks(kb, Lk, p.k_ts, p.D, w, lane), vs(vb, Lk, p.v_ts, p.D, w, lane);
    auto fetch = [&](unsigned char *to) {
        ks.next(to, w);
        vs.next(to + TILE_BYTES, w);
    };
    auto step = [&](int t, const unsigned char *__restrict cur, unsigned char *__restrict next, bool masked) {
        if (t + 1 < t_end) fetch(next);
        if (t * BN >= wave_top) return;
        const unsigned char *kt = cur, *vt = cur + TILE_BYTES;
#pragma unroll
        for (int b = 0; b < BN / 32; ++b) {
            f32x16 z = 0.f, y = 0.f;
#pragma unroll
            for (int c = 0; c < DC; ++c) {
                mma(z, TL::rows(kt, row_at, 32 * b, c), qf[c]);
                mma(y, TL::rows(vt, row_at, 32 * b, c), gf[c]);
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float pr = exp2_fast(__builtin_fmaf(z[r], p.c, -lse));
                float ds = pr * (y[r] - delta);
                if constexpr (scaled_ds<T>) ds *= inv;
                z[r] = ds;
            }
            if (masked) {
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (t * BN + 32 * b + 4 * h + 8 * (r / 4) + r % 4 >= lim) z[r] = 0.f;
            }
#pragma unroll
            for (int kc = 0; kc < 2; ++kc) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = z[kc * 8 + e];
                const Frag<T> sf = to_frag<T>(v);
#pragma unroll
                for (int d = 0; d < DB; ++d) mma(dq[d], TL::cols(kt, col_at, 32 * b + 16 * kc, 32 * d), sf);
            }
        }
    };
    if (t_end > 0) {
        fetch(lds);
        tiles_ready();
        const int t_full = max(0, min(t_end, low / BN));
        for (int t = 0; t < t_end; ++t) {
            step(t, lds + (t & 1) * 2 * TILE_BYTES, lds + (~t & 1) * 2 * TILE_BYTES, t >= t_full);
            tiles_ready();
        }
    }
    if (!in) return;
    const float f = scaled_ds<T> ? p.scale / inv : p.scale;
    T *row = (T *)p.dq + at * p.D;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
            const int col = 32 * d + 8 * (r / 4) + 4 * h;
            if (col >= p.D) continue;
            store4<T>(row + col, dq[d][r] * f, dq[d][r + 1] * f, dq[d][r + 2] * f, dq[d][r + 3] * f);
        }
}

// dk and dv: a workgroup of KW waves keeps 32 KW keys (their K, and V where there is room, as operands in registers)
// and walks over the rows of the key head's whole group in tiles of BQ = 32 BL, Q and dO in LDS. S = Q K^T and dO V^T
// come out with the keys as columns, so P and dS feed the products with dO and Q (read as columns) without leaving
// their lanes. Where there are few key tiles, or causal ones with very different numbers of rows, a sequence's rows are
// cut into up to `most` parts of at least PART_ROWS, at the same rows for every tile, so that workgroups that run
// together read the same rows through their L2. The parts' sums go to the workspace in fp32 and attn_dkv_join_kernel
// adds them in order. Four waves in step, two workgroups to a CU; eight waves that also share out the rows of a tile
// were slower (376 us against 330 for the whole call at 2 x 2048 x 16 heads of 128) but where one sequence of 768
// tokens is all there is (50, 61). Measured: 293 us for the causal tokens named above (755 TFLOP/s), 576 us for 2 x
// 4096 of 16 heads of 128 (955 TFLOP/s), 53 us for the 12 heads of 64 (585); it waits for 45% of its wave cycles in the
// first and 38% in the last.
constexpr int PART_ROWS = 512;
struct RowPart { int from, to, begin, parts; };    // rows of one part for a tile; the tile's first part and the end of its parts
__device__ __forceinline__ RowPart part_of(int first, int rows, int most, int rt, int part) {
    const int want = max(1, min(most, rows / PART_ROWS));
    const int each = max(1, ((rows + want - 1) / want + rt - 1) / rt) * rt;      // whole tiles
    RowPart r;
    r.parts = max(1, (rows + each - 1) / each);
    r.begin = min(first / each, r.parts - 1);
    r.from = min(rows, max(first, part * each));
    r.to = min(rows, max(r.from, (part + 1) * each));
    return r;
}

template <class T, int D, int KW, int BL>
__global__ __launch_bounds__(KW * 64, sizeof(T) == 4 && D == 128 ? 1 : 2) void attn_dkv_kernel(AttnArgs p) {
    using TL = Tile<T, D>;
    constexpr int NW = KW, BK = KW * 32, BQ = BL * 32, DC = D / 16, DB = D / 32;
    constexpr int TILE_BYTES = BQ * TL::ROW;
    // 128 16-bit components: with V in registers too, the accumulators would be spilled
    constexpr bool V_LDS = D == 128 && sizeof(T) == 2;
    constexpr int STATS = scaled_ds<T> ? 3 : 2;
    static_assert(BQ % 64 == 0 || BQ == 32, "a wave loads 64 rows' statistics");
    // A buffer: Q, dO and their rows' statistics. One array, as in the dq kernel.
    constexpr int SR = BQ < 64 ? 64 : BQ, BUFFER = 2 * TILE_BYTES + STATS * SR * 4;
    __shared__ __attribute__((aligned(16))) unsigned char lds[2 * BUFFER + (V_LDS ? BK * TL::ROW : 0)];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = lane >> 5, n = lane & 31;
    const int G = p.group.g;

    const int heads = p.Hkv, hk = key_head(blockIdx.x % heads, heads);
    int key_tile;
    const int s = find_slot(p.cu_k, p.B, p.Tk, 1, BK, blockIdx.x / heads, &key_tile);
    Span sq = span_of(p.cu_q, p.B, p.Tq, s);
    const Span sk = span_of(p.cu_k, p.B, p.Tk, s);
    if (s == 0 || s == p.B + 1) sq.hi = sq.lo;
    const int all_rows = (sq.hi - sq.lo) * G, Lk = sk.hi - sk.lo, shift = Lk - (sq.hi - sq.lo), j0 = key_tile * BK;
    if (j0 >= Lk) return;
    const int j_end = min(j0 + BK, Lk);

    Frag<T> kf[DC], vf[V_LDS ? 1 : DC];
    const int key = j0 + w * 32 + n;
    {
        const bool in = key < Lk;
        const int64_t tok = sk.lo + (in ? key : Lk - 1);
        const T *kr = (const T *)p.k + tok * p.k_ts + (int64_t)hk * p.k_hs;
        const T *vr = (const T *)p.v + tok * p.v_ts + (int64_t)hk * p.v_hs;
#pragma unroll
        for (int c = 0; c < DC; ++c) {
            kf[c] = global_rows<T>(kr, 16 * c + 8 * h, p.D, in);
            if constexpr (!V_LDS) vf[c] = global_rows<T>(vr, 16 * c + 8 * h, p.D, in);
        }
    }
    const int first = p.causal ? min(all_rows, max(0, j0 - shift) * G) : 0;     // earlier rows see none of these keys
    const RowPart part = part_of(first, all_rows, p.parts, p.rt, blockIdx.y);
    if ((int)blockIdx.y < part.begin || (int)blockIdx.y >= part.parts) return;
    const int rows = part.to, t_end = (rows - part.from + p.rt - 1) / p.rt, wave_key = j0 + w * 32;

    f32x16 dk[DB], dv[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d) { dk[d] = 0.f; dv[d] = 0.f; }
    float ref = NO_EXPONENT;                                  // dk is held in units of 2^ref (fp16)

    using In = Dma<T, D, NW, BQ>;
    const int row_at = TL::row_base(lane), col_at = TL::col_base(lane);
    // A tile has rt <= BQ rows: whole queries, or a whole part of one with more heads than BQ (see the plan). So a
    // lane's offsets are the same for every tile, but for the rows that a last tile lacks.
    auto in_tile = [&](int row, int64_t ts, int64_t hs) {
        const int qi = G <= BQ ? (int)div_by(row, p.group) : 0;
        return qi * (int)ts + (row - qi * G * (G <= BQ)) * (int)hs;
    };
    int qo[In::N], go[In::N];
    const int lane_row = In::row(0, w, lane);
#pragma unroll
    for (int i = 0; i < In::N; ++i) {
        const int row = In::row(i, w, lane), pc = In::piece(i, w, lane);
        const bool in = pc * TL::PE < p.D && row < p.rt;
        qo[i] = in ? in_tile(row, p.q_ts, p.q_hs) * (int)sizeof(T) + pc * 16 : OUTSIDE;
        go[i] = in ? in_tile(row, p.g_ts, p.g_hs) * (int)sizeof(T) + pc * 16 : OUTSIDE;
    }
    constexpr int PER = (BQ + 63) / 64, JOBS = (PER * STATS + NW - 1) / NW;   // wave loads of a statistic of a tile; of a wave
    int so[JOBS];
#pragma unroll
    for (int i = 0; i < JOBS; ++i) {
        const int row = (w + i * NW) % PER * 64 + lane;
        so[i] = row < p.rt ? in_tile(row, p.Hq, 1) * 4 : OUTSIDE;
    }
    auto fetch = [&](int t, unsigned char *to) {
        const int r0 = part.from + t * p.rt, q0 = (int)div_by(r0, p.group), head = hk * G + (r0 - q0 * G);
        const int64_t tok = sq.lo + q0;
        const int left = rows - r0;                            // rows from here on are not there
        const auto qb = buffer_of((const T *)p.q + tok * p.q_ts + head * p.q_hs, OUTSIDE);
        const auto gb = buffer_of((const T *)p.dout + tok * p.g_ts + head * p.g_hs, OUTSIDE);
        if (left >= p.rt) {
            In::load(qb, qo, to, w);
            In::load(gb, go, to + TILE_BYTES, w);
        } else {
            int q2[In::N], g2[In::N];
#pragma unroll
            for (int i = 0; i < In::N; ++i) {
                const bool in = lane_row + i * (64 / TL::NP) < left;
                q2[i] = in ? qo[i] : OUTSIDE;
                g2[i] = in ? go[i] : OUTSIDE;
            }
            In::load(qb, q2, to, w);
            In::load(gb, g2, to + TILE_BYTES, w);
        }
#pragma unroll
        for (int i = 0; i < JOBS; ++i) {
            const int which = (w + i * NW) / PER, part = (w + i * NW) % PER;
            if (which >= STATS) continue;
            const auto sb = buffer_of(p.stats + (int64_t)which * p.Tq * p.Hq + tok * p.Hq + head, OUTSIDE);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                sb, (void __attribute__((address_space(3))) *)(to + 2 * TILE_BYTES + (which * SR + part * 64) * 4), 4,
                part * 64 + lane < left ? so[i] : OUTSIDE, 0, 0, 0);
        }
    };
    auto step = [&](int t, const unsigned char *__restrict cur, unsigned char *__restrict next,
                    const unsigned char *__restrict v_lds, unsigned busy, unsigned masked) {
        if (t + 1 < t_end) fetch(t + 1, next);
        if (!busy) return;
        const unsigned char *qt = cur, *gt = cur + TILE_BYTES;
        const float *stats = (const float *)(cur + 2 * TILE_BYTES);
#pragma unroll
        for (int b = 0; b < BL; ++b) {
            if (!(busy >> b & 1)) continue;
            float inv = 1.f;
            if constexpr (scaled_ds<T>) {
                float e = stats[(STATS - 1) * SR + 32 * b + n];  // from NO_EXPONENT on: rows that are not there read 0
#pragma unroll
                for (int x = 16; x; x >>= 1) e = fmaxf(e, __shfl_xor(e, x));
                e += NO_EXPONENT;
                if (e > ref) {
                    const float f = exp2_fast(ref - e);
#pragma unroll
                    for (int d = 0; d < DB; ++d) dk[d] *= f;
                    ref = e;
                }
                inv = exp2_fast(-ref);
            }
            f32x16 z = 0.f, y = 0.f;
#pragma unroll
            for (int c = 0; c < DC; ++c) {
                mma(z, TL::rows(qt, row_at, 32 * b, c), kf[c]);
                if constexpr (V_LDS) mma(y, TL::rows(gt, row_at, 32 * b, c), TL::rows(v_lds, row_at, 32 * w, c));
                else mma(y, TL::rows(gt, row_at, 32 * b, c), vf[c]);
            }
            if (masked >> b & 1) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int row = part.from + t * p.rt + 32 * b + 8 * (r / 4) + 4 * h + r % 4;
                    if (key > (int)div_by(row, p.group) + shift) z[r] = -INFINITY;
                }
            }
#pragma unroll
            for (int r4 = 0; r4 < 4; ++r4) {
                const int r0 = 32 * b + 8 * r4 + 4 * h;
                const f32x4 ls = *reinterpret_cast<const f32x4 *>(stats + r0);
                const f32x4 de = *reinterpret_cast<const f32x4 *>(stats + SR + r0);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = 4 * r4 + e;
                    const float pr = exp2_fast(__builtin_fmaf(z[r], p.c, -ls[e]));
                    z[r] = pr;
                    y[r] = pr * (y[r] - de[e]);
                    if constexpr (scaled_ds<T>) y[r] *= inv;
                }
            }
            if constexpr (D == 128) __builtin_amdgcn_sched_barrier(0);   // loads hoisted further up would not fit the registers
#pragma unroll
            for (int kc = 0; kc < 2; ++kc) {
                float a[8], c[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) { a[e] = z[kc * 8 + e]; c[e] = y[kc * 8 + e]; }
                const Frag<T> pf = to_frag<T>(a), sf = to_frag<T>(c);
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    mma(dv[d], TL::cols(gt, col_at, 32 * b + 16 * kc, 32 * d), pf);
                    mma(dk[d], TL::cols(qt, col_at, 32 * b + 16 * kc, 32 * d), sf);
                }
            }
        }
    };
    if (t_end > 0) {
        if constexpr (V_LDS) {
            using Iv = Dma<T, D, NW, BK>;
            int off[Iv::N];
#pragma unroll
            for (int i = 0; i < Iv::N; ++i) off[i] = Iv::offset(i, w, lane, p.v_ts, p.D);
            Iv::load(buffer_of((const T *)p.v + (int64_t)(sk.lo + j0) * p.v_ts + (int64_t)hk * p.v_hs,
                               rows_bytes<T>(j_end - j0, p.v_ts, p.D)), off, lds + 2 * BUFFER, w);
        }
        fetch(0, lds);
        tiles_ready();
        for (int t = 0; t < t_end; ++t) {
            unsigned busy = 0, masked = 0;                      // by blocks of 32 rows: this wave's keys see it, not all see it whole
#pragma unroll
            for (int b = 0; b < BL; ++b) {
                const int w0 = part.from + t * p.rt + 32 * b;
                const int w1 = min(min(w0 + 32, part.from + (t + 1) * p.rt), rows);
                if (wave_key >= Lk || w0 >= w1) continue;
                if (p.causal) {
                    if (wave_key >= (int)div_by(w1 - 1, p.group) + shift + 1) continue;
                    if (min(wave_key + 32, Lk) > (int)div_by(w0, p.group) + shift + 1) masked |= 1u << b;
                }
                busy |= 1u << b;
            }
            step(t, lds + (t & 1) * BUFFER, lds + (~t & 1) * BUFFER, lds + 2 * BUFFER, busy, masked);
            tiles_ready();
        }
    }
    const float f = scaled_ds<T> ? p.scale * exp2_fast(ref) : p.scale;
    if (part.parts - part.begin > 1) {
        // as the lanes hold it: four elements a lane, 1 KB a store
        f32x4 *out = reinterpret_cast<f32x4 *>(p.part) + (((int64_t)blockIdx.x * p.parts + blockIdx.y) * 2 * BK + w * 32) * (D / 4) + lane;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int r = 4 * q;
                out[(d * 4 + q) * 64] = f32x4{dk[d][r], dk[d][r + 1], dk[d][r + 2], dk[d][r + 3]} * f;
                out[BK * (D / 4) + (d * 4 + q) * 64] = f32x4{dv[d][r], dv[d][r + 1], dv[d][r + 2], dv[d][r + 3]};
            }
        return;
    }
    if (key >= Lk) return;
    const int64_t at = ((int64_t)(sk.lo + key) * p.Hkv + hk) * p.D;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
            const int col = 32 * d + 8 * (r / 4) + 4 * h;
            if (col >= p.D) continue;
            store4<T>((T *)p.dk + at + col, dk[d][r] * f, dk[d][r + 1] * f, dk[d][r + 2] * f, dk[d][r + 3] * f);
            store4<T>((T *)p.dv + at + col, dv[d][r], dv[d][r + 1], dv[d][r + 2], dv[d][r + 3]);
        }
}

// dk and dv of the key tiles whose rows were cut into parts: a workgroup for 32 keys of one of them. Bound by memory:
// 34 us for up to 7 parts of 8634 x 4 heads of 128.
template <class T, int D, int KW>
__global__ __launch_bounds__(256) void attn_dkv_join_kernel(AttnArgs p) {
    constexpr int BK = KW * 32;
    const int hk = key_head(blockIdx.x % p.Hkv, p.Hkv);
    int key_tile;
    const int s = find_slot(p.cu_k, p.B, p.Tk, 1, BK, blockIdx.x / p.Hkv, &key_tile);
    if (s == 0 || s == p.B + 1) return;
    const Span sq = span_of(p.cu_q, p.B, p.Tq, s), sk = span_of(p.cu_k, p.B, p.Tk, s);
    const int G = p.group.g, rows = (sq.hi - sq.lo) * G, Lk = sk.hi - sk.lo, w = blockIdx.y % KW, which = blockIdx.y / KW;
    const int tile0 = key_tile * BK, j0 = tile0 + w * 32;
    if (j0 >= Lk) return;
    const int first = p.causal ? min(rows, max(0, tile0 - (Lk - (sq.hi - sq.lo))) * G) : 0;
    const RowPart part = part_of(first, rows, p.parts, p.rt, 0);
    if (part.parts - part.begin == 1) return;
    constexpr int ALL = BK * (D / 4);                          // f32x4 of one gradient of one part
    const f32x4 *in = reinterpret_cast<const f32x4 *>(p.part) + ((int64_t)blockIdx.x * p.parts * 2 + which) * ALL + w * (8 * D);
    T *out = (T *)(which ? p.dv : p.dk);
#pragma unroll
    for (int i = threadIdx.x; i < 8 * D; i += 256) {
        const int lane = i % 64, q = i / 64 % 4, d = i / 256;
        const int row = lane % 32, col = 32 * d + 8 * q + 4 * (lane / 32);
        f32x4 sum = 0.f;
#pragma unroll 4
        for (int k = part.begin; k < part.parts; ++k) sum += in[(int64_t)k * 2 * ALL + i];
        if (j0 + row < Lk && col < p.D)
            store4<T>(out + ((int64_t)(sk.lo + j0 + row) * p.Hkv + hk) * p.D + col, sum[0], sum[1], sum[2], sum[3]);
    }
}

}  // namespace ddm

// ddm_gemm.hpp -- products of matrices on the matrix cores, out[q][p] = sum_k Q(q, k) P(p, k), with what is to be done
// with a tile of them left to the caller.
//
// A workgroup takes a tile of BQ x BP outputs and walks along k in steps of 64 bytes (32 or 16 elements): the rows of
// steps to come go from memory straight to LDS while the matrix cores work on this one's. An operand's rows may run
// along k (TRANS = false: tiles of BQ rows of 64 bytes) or along its own index (TRANS = true: panels of 128 columns of
// as many rows as the step has k), read with transposing reads: no product needs a transposed copy of its inputs in
// memory. P is the matrix instructions' first operand, so that a lane holds runs of four
// neighbouring p of one q.
#pragma once
#include "ddm_tile.hpp"

namespace ddm {

constexpr int STEP_BYTES = 64;                  // of k in a step

// One operand of a tile: R of its indices.
template <class T, int R, bool TRANS, int NW>
struct Side {
    static constexpr int BK = STEP_BYTES / (int)sizeof(T), PE = 16 / (int)sizeof(T);
    static constexpr int COLS = !TRANS ? BK : R < 128 ? R : 128;      // elements of a row in LDS
    static constexpr int ROWS = !TRANS ? R : BK;                      // rows of a panel
    static constexpr int PANELS = !TRANS ? 1 : R / COLS, BYTES = R * STEP_BYTES;
    using TL = Tile<T, COLS>;
    using In = Dma<T, COLS, NW, ROWS>;
    static constexpr int READS = TRANS && sizeof(T) == 2 ? 2 : 1;     // of LDS for an operand of a matrix instruction
    static constexpr int LOADS = PANELS * In::N;                      // of a wave in a step
    static_assert(In::ALL % NW == 0, "every wave has as many");

    const T *at;
    int64_t pitch;                              // elements from one step to the next
    int off[PANELS][In::N], left;               // left: of k

    // source(i): the row of `base` that is index i of the tile, or a negative number (TRANS: i is the index itself, of
    // `most`).
    template <class F>
    __device__ __forceinline__ void start(const T *base, int64_t ld, int k, int most, int w, int lane, F source) {
        at = base;
        left = k;
        pitch = TRANS ? BK * ld : BK;
#pragma unroll
        for (int a = 0; a < PANELS; ++a)
#pragma unroll
            for (int n = 0; n < In::N; ++n) {
                const int row = In::row(n, w, lane), piece = In::piece(n, w, lane);
                if constexpr (TRANS) {
                    const int c = a * COLS + piece * PE;
                    off[a][n] = c < most ? (int)(row * ld + c) * (int)sizeof(T) : OUTSIDE;
                } else {
                    const int64_t r = source(row);
                    off[a][n] = r < 0 ? OUTSIDE : (int)((r * ld + piece * PE) * (int64_t)sizeof(T));
                }
            }
    }
    // The next step's tile; what lies past k is zeros.
    __device__ __forceinline__ void next(unsigned char *to, int w, int lane) {
        const auto b = buffer_of(at, OUTSIDE);
#pragma unroll
        for (int a = 0; a < PANELS; ++a) {
            unsigned char *panel = to + a * (ROWS * COLS * (int)sizeof(T));
            if (left >= BK) {
                In::load(b, off[a], panel, w);
            } else {
                int o[In::N];
#pragma unroll
                for (int n = 0; n < In::N; ++n)
                    o[n] = (TRANS ? In::row(n, w, lane) : In::piece(n, w, lane) * PE) < left ? off[a][n] : OUTSIDE;
                In::load(b, o, panel, w);
            }
        }
        at += pitch;
        left -= BK;
    }

    // Operand of indices 32 sub .. 32 sub + 31, k positions 16 c + 8 h + 0..7 of lane half h.
    __device__ static __forceinline__ int frag_base(int lane) {
        if constexpr (!TRANS) return TL::row_base(lane);
        const int h = lane >> 5, i = lane & 15;
        if constexpr (sizeof(T) == 2) return TL::place(8 * h + (i >> 2), ((lane & 16) >> 3) + ((i >> 1) & 1)) + 8 * (i & 1);
        return TL::place(8 * h, (lane & 31) >> 2) + 4 * (lane & 3);
    }
    __device__ static __forceinline__ Frag<T> frag(const unsigned char *t, int base, int sub, int c) {
        if constexpr (!TRANS) {
            return TL::rows(t, base, 32 * sub, c);
        } else {
            constexpr int PER = COLS / 32;
            const unsigned char *panel = t + sub / PER * (ROWS * COLS * (int)sizeof(T));
            const int d0 = sub % PER * 32, r0 = 16 * c;
            if constexpr (sizeof(T) == 2) {            // four rows on, the swizzle's lowest bit flips
                typedef __attribute__((address_space(3))) i16x4 lds4;
                const int a = base ^ (d0 >> 3 << 4);
                union { i16x4 s[2]; Frag<T> f; } u;
                u.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(panel + r0 * TL::ROW + a));
                u.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(panel + (r0 + 4) * TL::ROW + (a ^ (1 << 4))));
                return u.f;
            } else {
                const int a = base ^ (d0 >> 2 << 4);
                f32x8 f;
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = *reinterpret_cast<const float *>(panel + (r0 + j) * TL::ROW + (a ^ (j << 4)));
                return f;
            }
        }
    }
};

// All but this wave's N latest loads to LDS have landed, then everyone's.
template <int N>
__device__ __forceinline__ void loaded() {
    static_assert(N < 64, "vmcnt has six bits");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | (N >> 4 << 14));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Workgroups of one XCD (every eighth) get numbers that follow one another.
__device__ __forceinline__ int by_xcd(int b, int n) {
    const int x = b % 8;
    return b / 8 + x * (n / 8) + min(x, n % 8);
}
// Tile i of nq x np: tiles follow one another down bands of eight q, so that what an XCD works on at a time shares rows
// of both operands in its L2.
struct TileAt { int q, p; };
__device__ __forceinline__ TileAt tile_at(int i, int nq, int np) {
    const int band = i / (8 * np), high = min(8, nq - band * 8), j = i - band * 8 * np;
    return {band * 8 + j % high, j / high};
}

// How a product's tiles are shared out: each of the first `whole` to a workgroup, and each of the other `tail` to `of` workgroups
// that take `each` steps of k one after another; a join adds up what they found, in their order.
struct Shares { int whole, tail, of, each; };

}  // namespace ddm

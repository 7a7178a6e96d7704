// ddm_tile.hpp -- 32 x 32 matrix-core tiles, LDS tiles and packed sets, shared by the attention and matching-loss
// kernels.
//
// A product C[m][n] = sum_k A[m][k] B[n][k] runs in steps of 16 along k. Lane l of a wave holds row l % 32 of A and of
// B and, with h = l / 32, eight of the step's k positions; any assignment of k positions to (h, element) is right as
// long as A and B agree. C element r of lane l is column n = l % 32, row m = 8 (r / 4) + 4 h + r % 4. So the transposed
// score tile (m = key, n = query) holds one query's scores in two lanes: a row's softmax statistics need one exchange
// between lane halves, and its elements 8t..8t+7 are, as they lie, the B operand of a product over keys 16t + 4h +
// {0..3} and 16t + 8 + 4h + {0..3}: probabilities go from one product to the next in registers.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>
#include <type_traits>

namespace ddm {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <class T> struct FragOf;
template <> struct FragOf<_Float16> { typedef f16x8 type; };
template <> struct FragOf<__bf16> { typedef bf16x8 type; };
template <> struct FragOf<float> { typedef f32x8 type; };
template <class T> using Frag = typename FragOf<T>::type;

__device__ __forceinline__ void mma(f32x16 &c, f16x8 a, f16x8 b) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x16 &c, bf16x8 a, bf16x8 b) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
// fp32: element i of both operands in step i, whose two k positions are the lane halves.
__device__ __forceinline__ void mma(f32x16 &c, f32x8 a, f32x8 b) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
}

template <class T>
__device__ __forceinline__ Frag<T> to_frag(const float (&x)[8]) {
    Frag<T> f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (T)x[i];       // round to nearest even
    return f;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Over the two lanes n and n + 32: v_permlane32_swap of a value with itself leaves the low half's in one register and
// the high half's in the other, in both lanes.
__device__ __forceinline__ float half_max(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// ------------------------------------------------------------------------------------------------------ LDS tiles
// A tile holds rows of D elements as 16-byte pieces; piece p of row r lies at place p ^ swizzle(r) of its row, so that
// both the reads of one piece column over 32 rows and the transposing reads of four rows spread over the banks.
template <class T, int D>
struct Tile {
    static constexpr int PE = 16 / (int)sizeof(T);   // elements of a piece
    static constexpr int NP = D / PE;                // pieces of a row
    static constexpr int ROW = D * (int)sizeof(T);   // bytes of a row

    __device__ static __forceinline__ int swizzle(int r) {
        if constexpr (NP == 4) return (r >> 2) & 3;
        if constexpr (sizeof(T) == 4) return r & 7;    // NP = 8, 16, 32
        if constexpr (NP == 16) return ((r & 3) << 2) | ((r >> 2) & 3);
        return ((r & 2) << 1) | ((r >> 2) & 3);        // NP = 8
    }
    __device__ static __forceinline__ int place(int r, int p) { return r * ROW + ((p ^ swizzle(r)) << 4); }

    // Operand rows: lane's row r0 + l % 32, k positions 16 c + 8 h + 0..7. at = row_base(lane); r0 is a multiple of 32,
    // which leaves the swizzle alone, and the k step only flips piece bits of the address.
    __device__ static __forceinline__ int row_base(int lane) { return place(lane & 31, (PE == 8 ? 1 : 2) * (lane >> 5)); }
    __device__ static __forceinline__ Frag<T> rows(const unsigned char *t, int at, int r0, int c) {
        if constexpr (sizeof(T) == 2) {
            return *reinterpret_cast<const Frag<T> *>(t + r0 * ROW + (at ^ (2 * c << 4)));
        } else {
            const f32x4 a = *reinterpret_cast<const f32x4 *>(t + r0 * ROW + (at ^ (4 * c << 4)));
            const f32x4 b = *reinterpret_cast<const f32x4 *>(t + r0 * ROW + (at ^ ((4 * c + 1) << 4)));
            return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
        }
    }
    // Operand of the tile's transpose: lane's column d0 + l % 32, k positions = rows r0 + 4 h + {0..3}, r0 + 8 + 4 h +
    // {0..3}. 16-bit: ds_read_b64_tr_b16 hands lane i of 16 the i-th column of the 4 x 16 block whose 8-byte quarters
    // of rows the 16 lanes point at. at = col_base(lane); r0 is a multiple of 16, d0 of 32; eight rows on, one swizzle
    // bit flips.
    __device__ static __forceinline__ int col_base(int lane) {
        const int h = lane >> 5, i = lane & 15;
        if constexpr (sizeof(T) == 2) return place(4 * h + (i >> 2), ((lane & 16) >> 3) + ((i >> 1) & 1)) + 8 * (i & 1);
        return place(4 * h, (lane & 31) >> 2) + 4 * (lane & 3);
    }
    __device__ static __forceinline__ Frag<T> cols(const unsigned char *t, int at, int r0, int d0) {
        if constexpr (sizeof(T) == 2) {
            typedef __attribute__((address_space(3))) i16x4 lds4;
            const int a = at ^ (d0 >> 3 << 4);
            union { i16x4 s[2]; Frag<T> f; } u;
            u.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(t + r0 * ROW + a));
            u.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(t + (r0 + 8) * ROW + (a ^ (2 << 4))));
            return u.f;
        } else {                                       // rows j and j + 8 share the swizzle of row j of eight
            const int a = at ^ (d0 >> 2 << 4);
            f32x8 f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f[j] = *reinterpret_cast<const float *>(t + (r0 + (j & 3) + 8 * (j >> 2)) * ROW + (a ^ ((j & 3) << 4)));
            return f;
        }
    }
};

// Buffer loads with bounds: every dword at or past `bytes` reads as zero. A buffer ends at OUTSIDE at the latest, so
// that a piece placed there is outside with all of its dwords.
constexpr int OUTSIDE = 0x7ffffff0;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *p, int64_t bytes) {
    const int n = (int)(bytes < 0 ? 0 : bytes > OUTSIDE ? OUTSIDE : bytes);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, n, 0x00027000);
}

// A tile of ROWS rows from global memory straight to LDS (buffer_load_dwordx4 ... lds): a wave's 64 lanes fill 64
// consecutive places, and each lane names the piece that belongs there. Pieces past the row's elements or the buffer's
// bytes are zeros.
template <class T, int D, int NW, int ROWS>
struct Dma {
    using TL = Tile<T, D>;
    static constexpr int ALL = ROWS * TL::NP / 64, N = (ALL + NW - 1) / NW;      // loads of the tile, and of a wave
    static_assert(ALL * 64 == ROWS * TL::NP, "whole waves");
    __device__ static __forceinline__ int row(int n, int w, int lane) { return ((w * N + n) * 64 + lane) / TL::NP; }
    __device__ static __forceinline__ int piece(int n, int w, int lane) {
        return ((w * N + n) * 64 + lane) % TL::NP ^ TL::swizzle(row(n, w, lane));
    }
    // Byte offset of the lane's piece in rows of stride ts elements.
    __device__ static __forceinline__ int offset(int n, int w, int lane, int64_t ts, int d) {
        const int pc = piece(n, w, lane);
        return pc * TL::PE < d ? (int)(row(n, w, lane) * ts * (int)sizeof(T)) + pc * 16 : OUTSIDE;
    }
    __device__ static __forceinline__ void load(__amdgpu_buffer_rsrc_t b, const int (&off)[N], unsigned char *t, int w) {
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (ALL % NW == 0 || w * N + n < ALL)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (void __attribute__((address_space(3))) *)(t + (w * N + n) * 1024), 
                                                         16, off[n], 0, 0, 0);
    }
};

// The tiles of ROWS rows of a strided matrix, one after another from `at` on; `rows` counts those that are left.
template <class T, int D, int NW, int ROWS>
struct Walk {
    using In = Dma<T, D, NW, ROWS>;
    const T *at;
    int64_t pitch;                                     // elements from one tile to the next
    int off[In::N], rows, lane_row;
    __device__ __forceinline__ Walk(const T *first, int rows, int64_t ts, int d, int w, int lane)
        : at(first), pitch(ROWS * ts), rows(rows), lane_row(In::row(0, w, lane)) {
#pragma unroll
        for (int i = 0; i < In::N; ++i) off[i] = In::offset(i, w, lane, ts, d);
    }
    // The next tile; rows that are not there are zeros. Whole tiles cost a few scalar instructions.
    __device__ __forceinline__ void next(unsigned char *to, int w) {
        const auto b = buffer_of(at, OUTSIDE);
        if (rows >= ROWS) {
            In::load(b, off, to, w);
        } else {
            int o[In::N];
#pragma unroll
            for (int i = 0; i < In::N; ++i) o[i] = lane_row + i * (64 / In::TL::NP) < rows ? off[i] : OUTSIDE;
            In::load(b, o, to, w);
        }
        at += pitch;
        rows -= ROWS;
    }
};

// This wave's loads to LDS have landed, then everyone's.
__device__ __forceinline__ void tiles_ready() {
    __builtin_amdgcn_s_waitcnt(0x0f70);                // vmcnt(0)
    __syncthreads();
}

// ----------------------------------------------------------------------------------------------------- packed sets
// Sequence s of the boundaries 0, cu[0], ..., cu[B], T is [lo, hi); s = 0 and s = B + 1 are the tokens before and after
// every sequence. cu == nullptr stands for one sequence of all T tokens. Contents are clamped and no length is
// negative, so that no bad value of cu leads outside the tensor.
struct Span { int lo, hi; };

__device__ __forceinline__ int bound_at(const int32_t *cu, int B, int T, int s) {
    if (s <= 0) return 0;
    if (s > B + 1) return T;
    const int x = cu ? cu[s - 1] : (s == 1 ? 0 : T);
    return min(max(x, 0), T);
}
__device__ __forceinline__ Span span_of(const int32_t *cu, int B, int T, int s) {
    Span r;
    r.lo = bound_at(cu, B, T, s);
    r.hi = max(bound_at(cu, B, T, s + 1), r.lo);
    return r;
}

// Work slots over packed sequences without their lengths on the host: sequence s takes the slots from
// floor(lo mul / tile) + s on, which leaves it at least ceil(length mul / tile) before the next one's first.
// slot_count() of them cover every sequence. A wave counts the first slots that are at most `slot`.
__device__ __forceinline__ int find_slot(const int32_t *cu, int B, int T, int mul, int tile, int slot, int *index) {
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int base = 0; base < B + 2; base += 64) {
        const int s = base + lane;
        const bool in = s < B + 2 && (int)((uint32_t)(bound_at(cu, B, T, s) * mul) / (uint32_t)tile) + s <= slot;
        const int c = __popcll(__ballot(in));
        n += c;
        if (c < 64) break;
    }
    const int s = __builtin_amdgcn_readfirstlane(n - 1);
    // at least 0 also where cu decreases somewhere, so that no slot begins before its sequence
    *index = max(0, slot - ((int)((uint32_t)(bound_at(cu, B, T, s) * mul) / (uint32_t)tile) + s));
    return s;
}
inline __host__ __device__ long long slot_count(int B, int T, int mul, int tile) {
    return (long long)T * mul / tile + B + 2;
}

// r / g by multiplication, exact for r < 2^31: with 2^(k-1) < g <= 2^k and m = ceil(2^(31 + k) / g), which has 32 bits, r m /
// 2^(31 + k) exceeds r / g by less than 1 / g. g == 1 has no such m.
struct Div { uint32_t g, m, shift; };
inline Div make_div(uint32_t g) {
    if (g <= 1) return Div{g, 0, 0};
    const int k = 32 - __builtin_clz(g - 1);
    return Div{g, (uint32_t)(((1ull << (31 + k)) + g - 1) / g), (uint32_t)(k - 1)};
}
__host__ __device__ __forceinline__ uint32_t div_by(uint32_t r, Div d) {
    return ((uint32_t)((uint64_t)r * d.m >> 32) >> d.shift) + (d.m ? 0 : r);
}

}  // namespace ddm

// ddm_rotary.hip -- rotary positions (ddm_rotary).
//
//   angle = position of the token on the pair's axis * the pair's frequency,  c = m cos(angle),  s = m sin(angle)
//   (a, b) -> (a c - b s, a s + b c)
//
// Bound by memory: every element of q and k is read once and written once. A workgroup takes a few tokens, puts the
// sines and cosines of their pairs into LDS and then walks over the tokens' heads, q's and k's, in the order of their
// addresses: one angle serves all heads. 24576 tokens x 32 heads of 64 bf16, two axes: 41 us (201 MB, 4.9 TB/s; a copy
// of 2 x 200 MB reaches 5.4 here); 40001 x 40 heads of 128 fp16, half of each turned: 158 us (819 MB, 5.2 TB/s). Six
// tokens x 40 heads take 3 us, beside some 10 of the host's call.
#include "../../../include/ddm.h"
#include "ddm_tile.hpp"

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

using namespace ddm;

namespace {

struct Heads {
    const char *in;
    char *out;
    int64_t in_ts, in_hs, out_ts, out_hs;      // bytes
};

struct RotArgs {
    Heads q, k;
    const int32_t *pos;
    const double *freq;
    int T, Hq, axes, pairs;                    // pairs of an axis
    int group;                                 // tokens of a workgroup's step
    int slices, slice;                         // a token's items go to that many workgroups, so many to each
    int tail;                                  // elements of a head behind the rotated ones
    Div token, unit, axis;                     // items of a token, units of a head, units of an axis
    float magnitude, sign;
};

// cos and sin of position times frequency. The product and its rest about the nearest quarter turn are taken in 64
// bits: a far position's angle has lost its digits behind the point in 32. The rest, at most pi / 4, goes into the
// Taylor series, whose first terms left out are below 2^-29.
__device__ __forceinline__ float2 cos_sin(double x) {
    const double n = __builtin_rint(x * 0.63661977236758134308);
    double r = __builtin_fma(n, -1.57079632679489655800, x);
    r = __builtin_fma(n, -6.12323399573676603587e-17, r);
    const int quarter = (int)(n - 4.0 * __builtin_floor(n * 0.25));
    const float t = (float)r, u = t * t;
    const float sn = __builtin_fmaf(t * u, __builtin_fmaf(u, __builtin_fmaf(u, __builtin_fmaf(u, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), t);
    const float cs = __builtin_fmaf(u, __builtin_fmaf(u, __builtin_fmaf(u, __builtin_fmaf(u, __builtin_fmaf(u, -1.f / 3628800, 1.f / 40320), -1.f / 720),
                                                                      1.f / 24), -0.5f), 1.f);
    const float a = quarter & 1 ? sn : cs, b = quarter & 1 ? cs : sn;
    return {quarter == 1 || quarter == 2 ? -a : a, quarter >= 2 ? -b : b};
}

// The 32-bit value is there before it is rounded: fused into one instruction with the sum before it, as the compiler does
// in some variants for float16, rounding would differ between them.
template <class T>
__device__ __forceinline__ T rounded(float x) {
    asm("" : "+v"(x));
    return (T)x;
}

template <class T, int VE>
struct __attribute__((aligned(VE * sizeof(T)))) Piece { T v[VE]; };

// VE pairs at a time, as two pieces of VE elements: the first and the second elements of the pairs, or, interleaved,
// the pairs one after another. Pieces lie on addresses of whole pieces.
template <class T, int VE, bool INTERLEAVED>
__global__ __launch_bounds__(256) void rotary_kernel(RotArgs p) {
    extern __shared__ float2 table[];
    const int all = p.axes * p.pairs, rotated = all / VE;
    const int64_t steps = ((int64_t)p.T + p.group - 1) / p.group * p.slices;
    for (int64_t step = blockIdx.x; step < steps; step += gridDim.x) {
        const int t0 = (int)(step / p.slices) * p.group, tokens = min(p.group, p.T - t0);
        const int begin = (int)(step % p.slices) * p.slice;
        const int end = min(begin + p.slice, tokens * (int)p.token.g);
        __syncthreads();                       // the table of the step before has been read
        for (int i = threadIdx.x; i < tokens * all; i += 256) {
            const int t = i / all, j = i - t * all, axis = j / p.pairs;
            const float2 c = cos_sin((double)p.pos[(int64_t)(t0 + t) * p.axes + axis] * p.freq[j]);
            table[i] = {p.magnitude * c.x, p.magnitude * p.sign * c.y};
        }
        __syncthreads();
        for (int i = begin + threadIdx.x; i < end; i += 256) {
            const int t = div_by(i, p.token), j = i - t * p.token.g;
            int h = div_by(j, p.unit);
            const int u = j - h * p.unit.g;
            const bool is_q = h < p.Hq;
            const Heads &x = is_q ? p.q : p.k;
            h -= is_q ? 0 : p.Hq;
            const T *in = (const T *)(x.in + (t0 + t) * x.in_ts + h * x.in_hs);
            T *out = (T *)(x.out + (t0 + t) * x.out_ts + h * x.out_hs);
            if (u < rotated) {
                const int axis = div_by(u, p.axis), first = (u - axis * p.axis.g) * VE;
                const int a = 2 * p.pairs * axis + (INTERLEAVED ? 2 * first : first), b = a + (INTERLEAVED ? VE : p.pairs);
                Piece<T, VE> lo = *(const Piece<T, VE> *)(in + a), hi = *(const Piece<T, VE> *)(in + b);
                const float2 *cs = table + t * all + axis * p.pairs + first;
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float2 w = cs[e];
                    T &first_of = !INTERLEAVED ? lo.v[e] : 2 * e < VE ? lo.v[2 * e] : hi.v[2 * e - VE];
                    T &second_of = !INTERLEAVED ? hi.v[e] : 2 * e + 1 < VE ? lo.v[2 * e + 1] : hi.v[2 * e + 1 - VE];
                    const float v0 = (float)first_of, v1 = (float)second_of;
                    first_of = rounded<T>(__builtin_fmaf(v0, w.x, -(v1 * w.y)));
                    second_of = rounded<T>(__builtin_fmaf(v0, w.y, v1 * w.x));
                }
                *(Piece<T, VE> *)(out + a) = lo;
                *(Piece<T, VE> *)(out + b) = hi;
            } else {
                const int from = 2 * all + (u - rotated) * VE;
                *(Piece<T, VE> *)(out + from) = *(const Piece<T, VE> *)(in + from);
            }
        }
    }
}

int esize(int dtype) { return dtype == DDM_F32 ? 4 : 2; }

bool bad_heads(const void *p, int64_t ts, int64_t hs, int e) {
    return !p || (uintptr_t)p % e || ts < 0 || hs < 0 || ts >= (1ll << 40) || hs >= (1ll << 40);
}

// Whether rows of n elements at t ts + h hs, t < T, h < H, share some.
bool rows_meet(int64_t ts, int64_t hs, int T, int H, int n) {
    if ((T > 1 && ts < n) || (H > 1 && hs < n)) return true;
    if (T <= 1 || H <= 1) return false;
    if (ts >= hs * (H - 1) + n || hs >= ts * (T - 1) + n) return false;        // one within the other, as in dense tensors
    for (int64_t h = 1; h < H; ++h) {
        const int64_t t = h * hs / ts;                                         // the tokens whose rows are nearest to head h of the first
        if ((t < T && h * hs - t * ts < n) || (t + 1 < T && (t + 1) * ts - h * hs < n)) return true;
    }
    return false;
}
bool near(const void *a, const void *b, int bytes) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return (x < y ? y - x : x - y) < (uintptr_t)bytes;
}

template <class T, int VE>
void launch(const RotArgs &a, unsigned grid, size_t lds, bool interleaved, hipStream_t s) {
    if (interleaved) hipLaunchKernelGGL((rotary_kernel<T, VE, true>), dim3(grid), dim3(256), lds, s, a);
    else hipLaunchKernelGGL((rotary_kernel<T, VE, false>), dim3(grid), dim3(256), lds, s, a);
}

template <class T>
void launch_pieces(const RotArgs &a, int ve, unsigned grid, size_t lds, bool interleaved, hipStream_t s) {
    if (ve == 1) launch<T, 1>(a, grid, lds, interleaved, s);
    else if (ve == 2) launch<T, 2>(a, grid, lds, interleaved, s);
    else if (ve == 4) launch<T, 4>(a, grid, lds, interleaved, s);
    else if constexpr (sizeof(T) == 2) launch<T, 8>(a, grid, lds, interleaved, s);
}

}  // namespace

extern "C" {

int ddm_rotary(const void *q, int64_t q_ts, int64_t q_hs, int Hq, const void *k, int64_t k_ts, int64_t k_hs, int Hk,
               const int32_t *positions, const double *frequencies, int T, int D, int axes, int pairs, int dtype,
               int interleaved, int inverse, double magnitude, void *q_out, int64_t qo_ts, int64_t qo_hs, void *k_out,
               int64_t ko_ts, int64_t ko_hs, hipStream_t stream) {
    if (dtype != DDM_F32 && dtype != DDM_F16 && dtype != DDM_BF16) return DDM_ERR_UNSUPPORTED;
    if (D < 1 || D > DDM_MAX_ROTARY_D) return DDM_ERR_UNSUPPORTED;
    if (T < 0 || Hq < 0 || Hk < 0 || Hq > DDM_MAX_ROTARY_HEADS || Hk > DDM_MAX_ROTARY_HEADS) return DDM_ERR_INVALID;
    if (axes < 1 || pairs < 1 || axes > D || pairs > D || 2 * axes * pairs > D) return DDM_ERR_INVALID;
    if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1) || !std::isfinite((float)magnitude)) return DDM_ERR_INVALID;
    if (T == 0 || Hq + Hk == 0) return DDM_OK;
    // an only token's or head's stride says nothing
    for (int64_t *ts : {&q_ts, &k_ts, &qo_ts, &ko_ts}) *ts = T > 1 ? *ts : 0;
    for (int64_t *hs : {&q_hs, &qo_hs}) *hs = Hq > 1 ? *hs : 0;
    for (int64_t *hs : {&k_hs, &ko_hs}) *hs = Hk > 1 ? *hs : 0;
    const int e = esize(dtype);
    if (!positions || (uintptr_t)positions % 4 || !frequencies || (uintptr_t)frequencies % 8) return DDM_ERR_INVALID;
    if (Hq && (bad_heads(q, q_ts, q_hs, e) || bad_heads(q_out, qo_ts, qo_hs, e))) return DDM_ERR_INVALID;
    if (Hk && (bad_heads(k, k_ts, k_hs, e) || bad_heads(k_out, ko_ts, ko_hs, e))) return DDM_ERR_INVALID;
    // outputs that lie over one another, or over inputs that other threads still read
    const int row = D * e;
    if (Hq && (rows_meet(qo_ts, qo_hs, T, Hq, D) || (near(q_out, q, row) && !(q_out == q && qo_ts == q_ts && qo_hs == q_hs)))) return DDM_ERR_INVALID;
    if (Hk && (rows_meet(ko_ts, ko_hs, T, Hk, D) || (near(k_out, k, row) && !(k_out == k && ko_ts == k_ts && ko_hs == k_hs)))) return DDM_ERR_INVALID;
    if (Hq && Hk && (near(q_out, k_out, row) || near(q_out, k, row) || near(k_out, q, row))) return DDM_ERR_INVALID;
    RotArgs a{};
    a.q = {(const char *)q, (char *)q_out, q_ts * e, q_hs * e, qo_ts * e, qo_hs * e};
    a.k = {(const char *)k, (char *)k_out, k_ts * e, k_hs * e, ko_ts * e, ko_hs * e};
    a.pos = positions; a.freq = frequencies;
    a.T = T; a.Hq = Hq; a.axes = axes; a.pairs = pairs;
    a.magnitude = (float)magnitude; a.sign = inverse ? -1.f : 1.f;
    const int rest = D - 2 * axes * pairs;
    // the widest pieces that every row, axis and address is made of
    int64_t grain = (pairs | rest) * e;
    for (const Heads *x : {&a.q, &a.k}) {
        const int heads = x == &a.q ? Hq : Hk;
        if (heads) grain |= (int64_t)((uintptr_t)x->in | (uintptr_t)x->out);
        if (heads && T > 1) grain |= x->in_ts | x->out_ts;
        if (heads > 1) grain |= x->in_hs | x->out_hs;
    }
    int ve = 16 / e;
    while (grain % (ve * e)) ve /= 2;
    const int units = (axes * pairs + rest) / ve, items = units * (Hq + Hk);
    a.token = make_div(items); a.unit = make_div(units); a.axis = make_div(pairs / ve);
    // four items a thread where the tokens are many; fewer tokens a workgroup where they would not fill the card, and a token's
    // items over several where tokens are few
    const int table = axes * pairs * (int)sizeof(float2);
    a.group = (int)std::min<long long>({std::max(1024 / items, 1), std::max((int)(((int64_t)T + 511) / 512), 1), std::max(32768 / table, 1)});
    a.slices = a.group > 1 ? 1 : std::max(1, std::min((items + 255) / 256, std::max((items + 1023) / 1024, 512 / T)));
    a.slice = a.group > 1 ? a.group * items : ((items + a.slices - 1) / a.slices + 255) / 256 * 256;
    const long long steps = ((long long)T + a.group - 1) / a.group * a.slices;
    const unsigned grid = (unsigned)std::min<long long>(steps, 1 << 20);
    const size_t lds = (size_t)a.group * table;
    if (dtype == DDM_F32) launch_pieces<float>(a, ve, grid, lds, interleaved, stream);
    else if (dtype == DDM_F16) launch_pieces<_Float16>(a, ve, grid, lds, interleaved, stream);
    else launch_pieces<__bf16>(a, ve, grid, lds, interleaved, stream);
    return hipGetLastError() == hipSuccess ? DDM_OK : DDM_ERR_HIP;
}

}  // extern "C"

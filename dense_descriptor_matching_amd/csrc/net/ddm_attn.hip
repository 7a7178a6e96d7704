// ddm_attn.hip -- host side of ddm_attention_*: checks, variants and launches.
#include "../../../include/ddm.h"
#include "ddm_attn.hpp"

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

using namespace ddm;

namespace {

constexpr int SPLIT_ROWS = 32;            // rows of a workgroup of the split form

constexpr int KEYS = 128;                 // keys of a workgroup of the dk/dv kernel

struct Plan {
    int d;                                // padded head dimension: 32, 64 or 128
    bool split;
    int chunk, cap;
    size_t bytes;                         // forward workspace
};

int esize(int dtype) { return dtype == DDM_F32 ? 4 : 2; }

// Which form the forward pass takes, from the sizes alone (the lengths are on the device).
Plan make_plan(int dtype, int B, int Tq, int Tk, int Hq, int Hkv, int D) {
    Plan p{};
    p.d = D <= 32 ? 32 : D <= 64 ? 64 : 128;
    const long long rows = (long long)Tq * (Hq / Hkv);
    // Split the keys where that is sooner done, in microseconds: a whole row tile walks over its keys at 0.85 a step of
    // 64 where 512 workgroups of 128 rows run at once; split, a step of 32 rows takes its 3 ns of the whole card, and
    // the second launch and the join take 10. (1 row of 12 heads of 64 over 8 x 1500 keys: 24 whole, 19 split; 64 rows
    // over 8 x 1000: 19, 28; 100 rows of 16 heads over 40000: 531, 100; 1 row over 256 x 2000 keys of 8 heads of 128:
    // 359, 432.) The step is a long call's: the first twelve take 14 us. Lengths count by their mean: of 256 single tokens
    // with 500 keys on average, one with 40000 walks over them in one workgroup a key head.
    const double mean_rows = (double)rows / B, steps = Tk / 64.0, wgs = ((double)rows / 128 + B) * Hkv;
    const double whole = steps / B * 0.85 * std::max(1.0, wgs / 512);
    const double apart = 10 + std::ceil(mean_rows / 32) * Hkv * steps * 0.003;
    p.split = mean_rows <= 128 && whole > apart && (long long)Tq * Hq < 1 << 24;
    if (p.split) {
        // some 1024 workgroups of one wave over all keys, which the card holds at once with their tiles; whole tiles of
        // 64 keys. 67469 keys of 8 heads of 128 bf16: 61 us, against 65 with 2048, 71 with 1152 and 64 with 512 (5.3
        // TB/s at 32 x 4096 keys)
        const long long avg = ((long long)Tk * Hkv + 1023) / 1024;
        p.chunk = (int)std::max<long long>((avg + 63) / 64 * 64, 64);
        const long long mean = (rows + B - 1) / B;
        p.cap = (int)std::min<long long>((2 * mean + SPLIT_ROWS - 1) / SPLIT_ROWS * SPLIT_ROWS, 4 * SPLIT_ROWS);
        if (mean <= SPLIT_ROWS / 2) p.cap = SPLIT_ROWS;
        p.bytes = (size_t)(slot_count(B, Tk, 1, p.chunk) * Hkv) * p.cap * (D + 4) * sizeof(float);
    }
    return p;
}

// Backward: the statistics of the rows, then the parts of the dk/dv kernel. Parts are taken where key tiles alone are
// few and their sequences have rows enough: so many that equal ones fill the card's 512 places (two workgroups of four
// waves to a CU) once (16 heads over 4 key heads of 128 bf16, 2 x 2048 tokens: 339 us for the whole call with 4 parts,
// 393 with 5, 362 with 7), or four times with causal ones, whose rows differ (4096, 3001, 1024 and 513 tokens: 648 us
// with 3 parts, 627 with 6). The workspace holds the larger number for either.
struct BackPlan { int parts; size_t stats, bytes; };
BackPlan make_back_plan(int dtype, int B, int Tq, int Tk, int Hq, int Hkv, int D, int causal = 1) {
    BackPlan p{};
    const long long tiles = slot_count(B, Tk, 1, KEYS) * Hkv, rows = (long long)Tq * (Hq / Hkv);
    const long long full = std::max<long long>((long long)Tk * Hkv / KEYS, 1);
    const long long most = std::min<long long>(std::max<long long>(rows / B / PART_ROWS, 1), 8);
    p.parts = (int)std::min<long long>(std::max<long long>((causal ? 2048 : 512) / full, 1), most);
    p.stats = ((size_t)Tq * Hq * sizeof(float) * (dtype == DDM_F16 ? 3 : 2) + 255) / 256 * 256;
    const int d = D <= 32 ? 32 : D <= 64 ? 64 : 128;
    p.bytes = p.stats + (p.parts > 1 ? (size_t)tiles * p.parts * 2 * KEYS * d * sizeof(float) : 0);
    return p;
}

// Sizes that every entry point checks alike.
int check(int dtype, int B, int Tq, int Tk, int Hq, int Hkv, int D) {
    if (dtype != DDM_F32 && dtype != DDM_F16 && dtype != DDM_BF16) return DDM_ERR_UNSUPPORTED;
    if (B < 1 || Tq < 0 || Tk < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv) return DDM_ERR_INVALID;
    if (D < 1 || D > DDM_MAX_D || D * esize(dtype) % 16) return DDM_ERR_UNSUPPORTED;
    const long long G = Hq / Hkv;
    // rows and keys are counted in 31 bits, with room for the tile or parts of tiles past the last
    if (B > (1 << 20) || Tq * G > INT_MAX - 4096 || Tk >= INT_MAX - (1 << 22)) return DDM_ERR_INVALID;
    // a launch has fewer than 2^32 threads
    if (slot_count(B, Tq, (int)G, 128) * Hkv >= 1 << 24 || slot_count(B, Tk, 1, KEYS) * Hkv >= 1 << 24) return DDM_ERR_INVALID;
    return DDM_OK;
}

// Rows are whole 16-byte pieces at 16-byte boundaries, and 64 tokens of a tile, with `heads` heads of each, lie within
// 31-bit offsets.
bool bad_view(const void *p, int64_t ts, int64_t hs, int dtype, int heads = 1) {
    const int e = esize(dtype);
    if (!p || (uintptr_t)p % 16 || ts < 0 || hs < 0 || ts >= (1ll << 40) || hs >= (1ll << 40)) return true;
    if (ts * e % 16 || hs * e % 16 || ts * e >= (1ll << 24)) return true;
    return heads > 1 && hs * e >= (1ll << 29) / heads;
}
// The kernels' 32-bit scale and scale log2(e): as 0 or infinity they would make NaN of a hidden key's -inf or of a zero.
bool bad_scale(double scale) {
    return !(scale > 0) || !std::isnormal((float)scale) || !std::isnormal((float)(scale * 1.4426950408889634));
}
bool bad_ptr(const void *p) { return !p || (uintptr_t)p % 16; }

template <class T, int D>
hipError_t forward(const AttnArgs &a, const Plan &pl, hipStream_t s) {
    const int G = a.group.g;
    constexpr bool wide = sizeof(T) == 2;
    if (pl.split) {
        constexpr int BN = 32;
        const long long slots = slot_count(a.B, a.Tk, 1, pl.chunk);
        hipLaunchKernelGGL((attn_fwd_kernel<T, D, 1, BN, true>), dim3((unsigned)(slots * a.Hkv), pl.cap / SPLIT_ROWS),
                           dim3(64), 0, s, a);
        if (hipError_t e = hipGetLastError()) return e;
        hipLaunchKernelGGL((attn_join_kernel<T, D>), dim3((unsigned)((long long)a.Tq * a.Hq)), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    constexpr int BN = wide ? 64 : 32;
    const long long n = slot_count(a.B, a.Tq, G, 128) * a.Hkv;
    hipLaunchKernelGGL((attn_fwd_kernel<T, D, 4, BN, false>), dim3((unsigned)n), dim3(256), 0, s, a);
    return hipGetLastError();
}

// Rows of a tile of at most `most` in the dk/dv kernel: whole queries of G heads, or where G is larger a whole part of
// one.
int tile_rows(int most, int G) {
    if (G <= most) return most / G * G;
    int r = most;
    while (G % r) --r;
    return r;
}

template <class T, int D>
hipError_t backward(AttnArgs a, hipStream_t s) {
    const int G = a.group.g;
    constexpr bool wide = sizeof(T) == 2;
    constexpr int BN = wide ? 64 : 32;
    if (a.Tq) {
        const long long n = slot_count(a.B, a.Tq, G, 128) * a.Hkv;
        hipLaunchKernelGGL((attn_dq_kernel<T, D, 4, BN>), dim3((unsigned)n), dim3(256), 0, s, a);
        if (hipError_t e = hipGetLastError()) return e;
    }
    if (a.Tk) {
        constexpr int BL = wide && D < 128 ? 2 : 1;
        const long long n = slot_count(a.B, a.Tk, 1, KEYS) * a.Hkv;
        a.rt = tile_rows(32 * BL, G);
        hipLaunchKernelGGL((attn_dkv_kernel<T, D, KEYS / 32, BL>), dim3((unsigned)n, a.parts), dim3(KEYS * 2), 0, s, a);
        if (hipError_t e = hipGetLastError()) return e;
        if (a.parts > 1)
            hipLaunchKernelGGL((attn_dkv_join_kernel<T, D, KEYS / 32>), dim3((unsigned)n, 2 * KEYS / 32), dim3(256), 0, s, a);
    }
    return hipGetLastError();
}

template <class F>
hipError_t with_type(int dtype, int d, F f) {
    if (dtype == DDM_F16) return d == 32 ? f(_Float16{}, std::integral_constant<int, 32>{})
                                 : d == 64 ? f(_Float16{}, std::integral_constant<int, 64>{})
                                           : f(_Float16{}, std::integral_constant<int, 128>{});
    if (dtype == DDM_BF16) return d == 32 ? f(__bf16{}, std::integral_constant<int, 32>{})
                                  : d == 64 ? f(__bf16{}, std::integral_constant<int, 64>{})
                                            : f(__bf16{}, std::integral_constant<int, 128>{});
    return d == 32 ? f(float{}, std::integral_constant<int, 32>{})
           : d == 64 ? f(float{}, std::integral_constant<int, 64>{})
                     : f(float{}, std::integral_constant<int, 128>{});
}

}  // namespace

extern "C" {

size_t ddm_attention_forward_workspace_bytes(int B, int Tq, int Tk, int Hq, int Hkv, int D, int dtype) {
    if (check(dtype, B, Tq, Tk, Hq, Hkv, D) != DDM_OK) return 0;
    return std::max<size_t>(make_plan(dtype, B, Tq, Tk, Hq, Hkv, D).bytes, 16);
}

int ddm_attention_forward(const void *q, int64_t q_ts, int64_t q_hs, const void *k, int64_t k_ts, int64_t k_hs,
                          const void *v, int64_t v_ts, int64_t v_hs, const int32_t *cu_q, const int32_t *cu_k, int B,
                          int Tq, int Tk, int Hq, int Hkv, int D, int dtype, int causal, double scale, void *out,
                          float *lse, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if (int rc = check(dtype, B, Tq, Tk, Hq, Hkv, D)) return rc;
    if (bad_scale(scale) || (causal != 0 && causal != 1)) return DDM_ERR_INVALID;
    if ((!cu_q || !cu_k) && B != 1) return DDM_ERR_INVALID;
    if (Tq == 0) return DDM_OK;
    if (bad_view(q, q_ts, q_hs, dtype) || bad_ptr(out) || bad_ptr(lse)) return DDM_ERR_INVALID;
    if (Tk && (bad_view(k, k_ts, k_hs, dtype) || bad_view(v, v_ts, v_hs, dtype))) return DDM_ERR_INVALID;
    const Plan pl = make_plan(dtype, B, Tq, Tk, Hq, Hkv, D);
    if (pl.bytes && (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < pl.bytes)) return DDM_ERR_WORKSPACE;
    AttnArgs a{};
    a.q = q; a.k = k; a.v = v; a.out = out; a.lse = lse;
    a.cu_q = cu_q; a.cu_k = cu_k;
    a.B = B; a.Tq = Tq; a.Tk = Tk; a.Hq = Hq; a.Hkv = Hkv; a.D = D;
    a.group = make_div(Hq / Hkv);
    a.q_ts = q_ts; a.q_hs = q_hs; a.k_ts = k_ts; a.k_hs = k_hs; a.v_ts = v_ts; a.v_hs = v_hs;
    a.scale = (float)scale; a.c = (float)(scale * 1.4426950408889634); a.causal = causal;
    a.chunk = pl.chunk; a.cap = pl.cap; a.part = (float *)workspace;
    const hipError_t e = with_type(dtype, pl.d, [&](auto t, auto d) {
        return forward<decltype(t), decltype(d)::value>(a, pl, stream);
    });
    return e == hipSuccess ? DDM_OK : DDM_ERR_HIP;
}

size_t ddm_attention_backward_workspace_bytes(int B, int Tq, int Tk, int Hq, int Hkv, int D, int dtype) {
    if (check(dtype, B, Tq, Tk, Hq, Hkv, D) != DDM_OK) return 0;
    return std::max<size_t>(make_back_plan(dtype, B, Tq, Tk, Hq, Hkv, D).bytes, 16);
}

int ddm_attention_backward(const void *dout, int64_t g_ts, int64_t g_hs, const void *q, int64_t q_ts, int64_t q_hs,
                           const void *k, int64_t k_ts, int64_t k_hs, const void *v, int64_t v_ts, int64_t v_hs,
                           const void *out, const float *lse, const int32_t *cu_q, const int32_t *cu_k, int B, int Tq,
                           int Tk, int Hq, int Hkv, int D, int dtype, int causal, double scale, void *dq, void *dk,
                           void *dv, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if (int rc = check(dtype, B, Tq, Tk, Hq, Hkv, D)) return rc;
    if (bad_scale(scale) || (causal != 0 && causal != 1)) return DDM_ERR_INVALID;
    if ((!cu_q || !cu_k) && B != 1) return DDM_ERR_INVALID;
    if (Tq && (bad_view(q, q_ts, q_hs, dtype, Hq / Hkv) || bad_view(dout, g_ts, g_hs, dtype, Hq / Hkv) || bad_ptr(out) || bad_ptr(lse) ||
               bad_ptr(dq)))
        return DDM_ERR_INVALID;
    if (Tk && (bad_view(k, k_ts, k_hs, dtype) || bad_view(v, v_ts, v_hs, dtype) || bad_ptr(dk) || bad_ptr(dv)))
        return DDM_ERR_INVALID;
    const BackPlan bp = make_back_plan(dtype, B, Tq, Tk, Hq, Hkv, D);
    if (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < bp.bytes) return DDM_ERR_WORKSPACE;
    const Plan pl = make_plan(dtype, B, Tq, Tk, Hq, Hkv, D);
    AttnArgs a{};
    a.q = q; a.k = k; a.v = v; a.o = out; a.dout = dout; a.lse = const_cast<float *>(lse); a.stats = (float *)workspace;
    a.parts = make_back_plan(dtype, B, Tq, Tk, Hq, Hkv, D, causal).parts; a.part = (float *)((char *)workspace + bp.stats);
    a.dq = dq; a.dk = dk; a.dv = dv;
    a.cu_q = cu_q; a.cu_k = cu_k;
    a.B = B; a.Tq = Tq; a.Tk = Tk; a.Hq = Hq; a.Hkv = Hkv; a.D = D;
    a.group = make_div(Hq / Hkv);
    a.q_ts = q_ts; a.q_hs = q_hs; a.k_ts = k_ts; a.k_hs = k_hs; a.v_ts = v_ts; a.v_hs = v_hs; a.g_ts = g_ts; a.g_hs = g_hs;
    a.scale = (float)scale; a.c = (float)(scale * 1.4426950408889634); a.causal = causal;
    const hipError_t e = with_type(dtype, pl.d, [&](auto t, auto d) {
        return backward<decltype(t), decltype(d)::value>(a, stream);
    });
    return e == hipSuccess ? DDM_OK : DDM_ERR_HIP;
}

}  // extern "C"

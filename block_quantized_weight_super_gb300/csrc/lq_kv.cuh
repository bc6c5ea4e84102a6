// lq_kv.cuh -- what the KV cache kernels share: the cache view, the step's
// token -> sequence map and the exact 8-bit rounding.
#pragma once
#include <cstdint>

#include "lq_device.cuh"

namespace lq {

// One layer's cache (include/lq.h, lq_kv8); page = 1 << pshift.
struct KvView {
    int8_t* k;          // [n_pages][n_kv][page][d]
    int8_t* v;          // [n_pages][n_kv][d][page]
    float* ks;          // [n_pages][n_kv]
    float* vs;
    int64_t n_pages;
    int32_t n_kv, pshift, d;
};

// The step: sequences, their new token rows and the page table.
struct KvStep {
    const int32_t* table;   // [nseq][max_pages]
    const int32_t* start;   // [nseq]
    const int32_t* cu;      // [nseq + 1], or null: one token per sequence
    int32_t max_pages, nseq, ntok;
};

__device__ __forceinline__ int kv_cu(const KvStep& S, int s) { return S.cu ? __ldg(S.cu + s) : s; }

// The last sequence s with key(s) <= x, for an ascending key with
// key(0) <= x: the sequence that holds item x.
template <class Key>
__device__ __forceinline__ int kv_find(int nseq, int64_t x, Key key) {
    int lo = 0, hi = nseq - 1;
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if ((int64_t)key(m) <= x) lo = m;
        else hi = m - 1;
    }
    return lo;
}

// x / s rounded to the nearest integer, ties to even, exactly, in
// [-127, 127]; s > 0 finite, both already multiplied by kv_up(s), inv the
// fp32 reciprocal of s.  x * inv is within 3 ulps of the quotient, so its
// rounding is off by one at most, and only next to a half-integer h; there the
// sign of x - h s decides, which the fused multiply-add gives exactly (h s has
// at most 32 significant bits, and kv_up keeps it out of the subnormals).
__device__ __forceinline__ int kv_round(float x, float s, float inv) {
    const float r = fminf(fmaxf(x * inv, -127.f), 127.f);
    float n = rintf(r);
    const float up = fmaf(-(n + 0.5f), s, x), dn = fmaf(-(n - 0.5f), s, x);
    const bool odd = ((int)n & 1) != 0;
    if (up > 0.f || (up == 0.f && odd)) n += 1.f;
    else if (dn < 0.f || (dn == 0.f && odd)) n -= 1.f;
    return (int)fminf(fmaxf(n, -127.f), 127.f);
}

// Power of two that keeps the arithmetic of kv_round normal for tiny scales.
__device__ __forceinline__ float kv_up(float s) { return s < 1e-30f ? 18446744073709551616.f : 1.f; }

// Bits of |x|: they order like the values, with infinities and NaN above all
// finite values, so a maximum over them keeps a NaN.
__device__ __forceinline__ uint32_t kv_absbits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

}  // namespace lq

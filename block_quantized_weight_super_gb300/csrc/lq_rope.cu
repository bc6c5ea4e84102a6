// lq_rope.cu -- rotary positions with one or several axes.
//
// Pair i of a token at position p of the pair's axis is rotated by p * freq[i].
// The angle is taken in turns, p * (freq[i] / 2 pi) in fp64, and only its
// fractional part in [-1/2, 1/2] goes to fp32: at p = 2^20 the reduction error
// is below 2^-35 turns, where an fp32 product would have lost 2^-7.  sincospi
// of twice that fraction is accurate to fp32 rounding.  Two fp64 products and
// one rounding per (token, pair), shared by all heads, are small beside the
// memory traffic (8 bytes per element), which bounds the kernel.
#include "lq_internal.h"
#include "lq_kv.cuh"

namespace lq {
namespace {

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_MAX_PAIRS = 512;

// One token (blockIdx.x) and a range of its heads (blockIdx.y).  The table of
// (cos, sin) per pair lies in shared memory; V = 4: a thread rotates four
// adjacent pairs with 16-byte accesses (ROPE_HALF, widths and addresses
// multiples of four floats), V = 1: one pair.
template <int V>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(const RopeParams P) {
    __shared__ float2 cs[ROPE_MAX_PAIRS];
    const int t = blockIdx.x, half = P.rot / 2;
    for (int i = threadIdx.x; i < half; i += ROPE_THREADS) {
        const int a = P.axis ? P.axis[i] : 0;
        float s = 0.f, c = 1.f;
        if (a < P.n_axes) {
            const double turns = (double)P.pos[(int64_t)a * P.ntok + t] * (P.freq[i] * 0.15915494309189533577);
            sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
        } else {
            record_status(P.status, STATUS_BADARG);
        }
        cs[i] = make_float2(c, s);
    }
    __syncthreads();
    const int heads = P.n_q + P.n_k, h0 = (int)((int64_t)heads * blockIdx.y / gridDim.y),
              h1 = (int)((int64_t)heads * (blockIdx.y + 1) / gridDim.y);
    const int units = half / V, tail = (P.d - P.rot) / V, per = units + tail;   // work items of a head
    for (int u = threadIdx.x; u < (h1 - h0) * per; u += ROPE_THREADS) {
        const int h = h0 + u / per, i = u % per;
        const float* x = h < P.n_q ? P.q + t * P.ld_q + (int64_t)h * P.d : P.k + t * P.ld_k + (int64_t)(h - P.n_q) * P.d;
        float* y = h < P.n_q ? P.qo + t * P.ld_qo + (int64_t)h * P.d : P.ko + t * P.ld_ko + (int64_t)(h - P.n_q) * P.d;
        if (V == 4) {
            if (i < units) {
                const float4 a = *reinterpret_cast<const float4*>(x + 4 * i);
                const float4 b = *reinterpret_cast<const float4*>(x + half + 4 * i);
                const float2 c0 = cs[4 * i], c1 = cs[4 * i + 1], c2 = cs[4 * i + 2], c3 = cs[4 * i + 3];
                *reinterpret_cast<float4*>(y + 4 * i) = make_float4(a.x * c0.x - b.x * c0.y, a.y * c1.x - b.y * c1.y,
                                                                    a.z * c2.x - b.z * c2.y, a.w * c3.x - b.w * c3.y);
                *reinterpret_cast<float4*>(y + half + 4 * i) =
                    make_float4(b.x * c0.x + a.x * c0.y, b.y * c1.x + a.y * c1.y, b.z * c2.x + a.z * c2.y,
                                b.w * c3.x + a.w * c3.y);
            } else {
                const int e = P.rot + 4 * (i - units);
                *reinterpret_cast<float4*>(y + e) = *reinterpret_cast<const float4*>(x + e);
            }
        } else {
            if (i < units) {
                const int ia = P.adjacent ? 2 * i : i, ib = P.adjacent ? 2 * i + 1 : half + i;
                const float a = x[ia], b = x[ib];
                const float2 c = cs[i];
                y[ia] = a * c.x - b * c.y;
                y[ib] = b * c.x + a * c.y;
            } else {
                const int e = P.rot + (i - units);
                y[e] = x[e];
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& P, int sms, cudaStream_t st) {
    const int heads = P.n_q + P.n_k;
    // few tokens: the heads of one are spread over blocks (one token of 40
    // heads: 10 blocks)
    int split = 1;
    while (split * 4 < heads && (int64_t)P.ntok * split < sms) split *= 2;
    const dim3 grid((unsigned)P.ntok, (unsigned)split);
    auto al16 = [](const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 4 == 0; };
    const bool vec = !P.adjacent && (P.rot / 2) % 4 == 0 && P.d % 4 == 0 && al16(P.q, P.ld_q) && al16(P.qo, P.ld_qo) &&
                     (P.n_k == 0 || (al16(P.k, P.ld_k) && al16(P.ko, P.ld_ko)));
    if (vec) rope_kernel<4><<<grid, ROPE_THREADS, 0, st>>>(P);
    else rope_kernel<1><<<grid, ROPE_THREADS, 0, st>>>(P);
    return cudaGetLastError();
}

}  // namespace lq

// lq_kv8_attn.cu -- attention over the 8-bit paged cache.
//
// One warp per (token, query head): a running maximum and sum of the softmax
// over the visible keys, one key at a time.
#include "lq_internal.h"
#include "lq_kv.cuh"

namespace lq {
namespace {

__global__ void __launch_bounds__(32) kv8_attn_simple_kernel(const AttnParams P) {
    const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x, D = P.c.d, g = P.n_q / P.c.n_kv, hk = h / g;
    const int s = kv_find(P.s.nseq, t, [&](int i) { return kv_cu(P.s, i); });
    const int row0 = kv_cu(P.s, s), n = kv_cu(P.s, s + 1) - row0;
    if (t >= row0 + n) return;
    const int64_t p = (int64_t)P.s.start[s] + (t - row0);
    const int64_t end = (int64_t)P.s.start[s] + n;
    const int64_t pre = P.prefix ? P.prefix[s] : 0;
    float q[8], o[8];
    const int per = D / 32;
    for (int i = 0; i < 8; ++i) {
        q[i] = i < per ? P.q[t * P.ld_q + (int64_t)h * D + lane + 32 * i] : 0.f;
        o[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int64_t j = 0; p >= 0 && j < end; ++j) {
        if (!(j < pre || (j <= p && (P.window == 0 || p - j < P.window)))) continue;
        const int64_t pj = j >> P.c.pshift;
        const int page = pj < P.s.max_pages ? P.s.table[(int64_t)s * P.s.max_pages + pj] : -1;
        if (page < 0 || page >= P.c.n_pages) {
            if (lane == 0) record_status(P.status, STATUS_BADARG);
            continue;
        }
        const int slot = (int)(j & ((1 << P.c.pshift) - 1));
        const int64_t ph = (int64_t)page * P.c.n_kv + hk, base = ph * ((int64_t)D << P.c.pshift);
        float a = 0.f;
        for (int i = 0; i < per; ++i) a = fmaf(q[i], (float)P.c.k[base + (int64_t)slot * D + lane + 32 * i], a);
        for (int o2 = 16; o2; o2 >>= 1) a += __shfl_xor_sync(~0u, a, o2);
        a = a * P.c.ks[ph] * P.scale;
        if (P.softcap > 0.f) a = P.softcap * tanhf(a / P.softcap);
        if (P.slopes) a -= P.slopes[h] * fabsf((float)(p - j));
        const float m2 = fmaxf(m, a), r = expf(m - m2), w = expf(a - m2);
        l = l * r + w;
        m = m2;
        for (int i = 0; i < per; ++i)
            o[i] = o[i] * r + w * P.c.vs[ph] * (float)P.c.v[base + ((int64_t)(lane + 32 * i) << P.c.pshift) + slot];
    }
    for (int i = 0; i < per; ++i) P.out[t * P.ld_out + (int64_t)h * D + lane + 32 * i] = l > 0.f || l != l ? o[i] / l : 0.f;
}

}  // namespace

size_t kv8_attn_workspace(int n_q, int n_kv, int d, int nseq, int ntok) { return 256; }

cudaError_t launch_kv8_attn(const AttnParams& P, int sms, cudaStream_t st) {
    kv8_attn_simple_kernel<<<dim3((unsigned)P.s.ntok, (unsigned)P.n_q), 32, 0, st>>>(P);
    return cudaGetLastError();
}

}  // namespace lq

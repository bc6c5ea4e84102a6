// lq_kv8.cu -- writing the 8-bit KV cache: append (quantise new rows) and
// page copies.
#include "lq_internal.h"
#include "lq_kv.cuh"

namespace lq {
namespace {

constexpr int APP_THREADS = 256;

// Sequence s owns the work items [base(s), base(s + 1)), base(s) =
// floor(cu[s] / page) + 2 s: at least as many as the pages its new tokens
// can touch (n new tokens at any offset touch at most floor(n / page) + 2), so
// the grid's size follows from ntok and nseq alone.  One new token per
// sequence (cu null): one item each.
__device__ __forceinline__ int64_t app_base(const KvStep& S, int pshift, int s) {
    return S.cu ? (int64_t)(__ldg(S.cu + s) >> pshift) + 2 * s : s;
}

// One page, kv head and K (blockIdx.z = 0) or V (1).  Two passes over the
// page's new rows: the largest |x|, then the codes (the second read comes from
// L2).  A thread makes 4 codes of adjacent dims (K) or of adjacent slots (V),
// one 32-bit word of the cache; a word that also holds earlier codes keeps
// or rescales them.
__global__ void __launch_bounds__(APP_THREADS) kv8_append_kernel(const KvView C, const KvStep S, const float* k,
                                                                 int64_t ld_k, const float* v, int64_t ld_v,
                                                                 unsigned* status) {
    __shared__ uint32_t red[APP_THREADS / 32];
    const int head = blockIdx.y, tid = threadIdx.x;
    const bool isv = blockIdx.z != 0;
    const int s = kv_find(S.nseq, blockIdx.x, [&](int i) { return app_base(S, C.pshift, i); });
    const int row0 = kv_cu(S, s), n = kv_cu(S, s + 1) - row0, start = S.start[s];
    const int64_t end = (int64_t)start + n;                              // one past the last position
    const int64_t p0 = max(start, 0);                                    // first stored position
    const int64_t pj = (p0 >> C.pshift) + ((int64_t)blockIdx.x - app_base(S, C.pshift, s));
    const int64_t a = max(p0, pj << C.pshift), b = min(end, (pj + 1) << C.pshift);   // the page's new positions
    if (n <= 0 || a >= b) return;
    const int page = pj < S.max_pages ? S.table[(int64_t)s * S.max_pages + pj] : -1;
    if (page < 0 || page >= C.n_pages || row0 < 0 || row0 + n > S.ntok) {
        if (tid == 0) record_status(status, STATUS_BADARG);
        return;
    }
    const int s0 = (int)(a - (pj << C.pshift)), s1 = (int)(b - (pj << C.pshift));     // its new slots
    const int64_t ld = isv ? ld_v : ld_k;
    const float* x = (isv ? v : k) + (row0 + (a - start)) * ld + (int64_t)head * C.d;  // row of slot s0
    const int64_t ph = (int64_t)page * C.n_kv + head;
    float* scale = (isv ? C.vs : C.ks) + ph;
    int8_t* codes = (isv ? C.v : C.k) + ph * ((int64_t)C.d << C.pshift);

    uint32_t m = 0;
    for (int e = tid; e < (s1 - s0) * C.d; e += APP_THREADS) m = max(m, kv_absbits(x[(e / C.d) * ld + e % C.d]));
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((tid & 31) == 0) red[tid >> 5] = m;
    __syncthreads();
    for (int i = 0; i < APP_THREADS / 32; ++i) m = max(m, red[i]);
    const float was = s0 > 0 ? *scale : 0.f;
    const float mine = m < 0x7F800000u ? __uint_as_float(m) * (1.f / 127.f) : __uint_as_float(0x7FC00000u);
    const float now = kv_absbits(was) >= kv_absbits(mine) ? was : mine;  // NaN stays
    const bool good = kv_absbits(now) < 0x7F800000u && now > 0.f;
    const bool again = s0 > 0 && good && now > was;                      // earlier codes get the new scale
    __syncthreads();                                                     // every thread has read *scale
    if (tid == 0) *scale = now;
    const float up = kv_up(now), su = now * up, inv = 1.f / su;

    // code of (slot, dim), given the code there now
    auto code = [&](int slot, int d, int had) -> int {
        if (slot >= s0 && slot < s1) return good ? kv_round(x[(slot - s0) * ld + d] * up, su, inv) : 0;
        if (slot < s0 && again) return kv_round((float)had * was * up, su, inv);
        return had;
    };
    const int first = again ? 0 : s0;                                    // slots to rewrite: [first, s1)
    if (!isv) {
        const int dw = C.d / 4;                                          // words per slot
        for (int w = first * dw + tid; w < s1 * dw; w += APP_THREADS) {
            const int slot = w / dw, d = 4 * (w % dw);
            char4* p = reinterpret_cast<char4*>(codes) + w;
            char4 c = slot < s0 ? *p : make_char4(0, 0, 0, 0);
            *p = make_char4(code(slot, d, c.x), code(slot, d + 1, c.y), code(slot, d + 2, c.z), code(slot, d + 3, c.w));
        }
    } else {
        const int w0 = first / 4, nw = (s1 + 3) / 4 - w0;                // slot words to rewrite
        for (int u = tid; u < nw * C.d; u += APP_THREADS) {
            const int d = u % C.d, slot = 4 * (w0 + u / C.d);
            char4* p = reinterpret_cast<char4*>(codes + ((int64_t)d << C.pshift) + slot);
            char4 c = *p;
            *p = make_char4(code(slot, d, c.x), code(slot + 1, d, c.y), code(slot + 2, d, c.z), code(slot + 3, d, c.w));
        }
    }
}

// Block (piece, pair, layer): a piece of the K and V codes of the pair's page
// in 16-byte units, and the scales with piece 0.
__global__ void __launch_bounds__(256) kv8_copy_kernel(const __grid_constant__ KvLayers L, const int32_t* src,
                                                       const int32_t* dst, int i0, const int32_t* count,
                                                       int64_t n_pages, int n_kv, int64_t units, unsigned* status) {
    const int i = i0 + (int)blockIdx.y;
    if (count && i >= *count) return;
    const int a = src[i], b = dst[i];
    if (a < 0 || b < 0) return;
    if (a >= n_pages || b >= n_pages) {
        if (threadIdx.x == 0) record_status(status, STATUS_BADARG);
        return;
    }
    const int l = blockIdx.z;
    if (blockIdx.x == 0)
        for (int h = threadIdx.x; h < n_kv; h += 256) {
            L.ks[l][(int64_t)b * n_kv + h] = L.ks[l][(int64_t)a * n_kv + h];
            L.vs[l][(int64_t)b * n_kv + h] = L.vs[l][(int64_t)a * n_kv + h];
        }
    const uint4* ka = reinterpret_cast<const uint4*>(L.k[l]) + a * units;
    const uint4* va = reinterpret_cast<const uint4*>(L.v[l]) + a * units;
    uint4* kb = reinterpret_cast<uint4*>(L.k[l]) + b * units;
    uint4* vb = reinterpret_cast<uint4*>(L.v[l]) + b * units;
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < units; u += (int64_t)gridDim.x * 256) {
        kb[u] = ka[u];
        vb[u] = va[u];
    }
}

}  // namespace

cudaError_t launch_kv8_append(const KvView& C, const KvStep& S, const float* k, int64_t ld_k, const float* v,
                              int64_t ld_v, unsigned* status, cudaStream_t st) {
    const int64_t items = S.cu ? (int64_t)(S.ntok >> C.pshift) + 2 * (int64_t)S.nseq : S.nseq;
    kv8_append_kernel<<<dim3((unsigned)items, (unsigned)C.n_kv, 2), APP_THREADS, 0, st>>>(C, S, k, ld_k, v, ld_v, status);
    return cudaGetLastError();
}

cudaError_t launch_kv8_copy(const KvLayers& L, int n_layers, const int32_t* src, const int32_t* dst, int n,
                            const int32_t* count, int64_t n_pages, int n_kv, int64_t units, unsigned* status,
                            cudaStream_t st) {
    const unsigned pieces = (unsigned)((units + 1023) / 1024);           // 16 KB of K and of V per block
    for (int i = 0; i < n; i += 65535) {                                 // (the grid's y limit)
        const int m = n - i < 65535 ? n - i : 65535;
        kv8_copy_kernel<<<dim3(pieces, (unsigned)m, (unsigned)n_layers), 256, 0, st>>>(
            L, src, dst, i, count, n_pages, n_kv, units, status);
    }
    return cudaGetLastError();
}

}  // namespace lq

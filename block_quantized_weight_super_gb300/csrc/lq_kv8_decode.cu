// lq_kv8_decode.cu -- attention over the 8-bit paged cache for few query rows
// per sequence (decoding): bound by the HBM reads of the codes.
//
// Rows.  The query rows of one kv head (tokens x the heads of its group) are
// taken 8 at a time.  mma.sync.m16n8k16 with A = those 8 rows as fp16 hi
// pieces (A rows 0-7) and lo pieces (8-15): the two halves of a D fragment lie
// in one thread and their sum is the fp32-accurate product, for the price of
// the M = 16 tile that 8 rows would cost anyway.  B = the codes, exact in
// fp16: S = Q K^T takes 8 keys x 16 dims per MMA, O += W V 16 keys x 8 dims.
// The D fragment of S (row g, keys 2t, 2t + 1) is the A fragment of the second
// product, so the weights never leave the thread.
//
// Keys.  Thread t of a quad owns T / 4 adjacent keys of a T-key chunk (the
// key a column stands for is free to choose): they lie in one page, so both
// scales are one register per thread, the K bytes of a key are 16-byte pieces
// and the V bytes of a dim (pages hold V with the tokens adjacent) one 8- or
// 16-byte piece.  Four codes become two fp16 pairs in five instructions.
//
// Split.  (sequence, kv head, row tile, chunk) are numbered in one line and
// dealt to the warps of one CTA per SM in equal shares, whatever the
// lengths; warps never meet.  A warp keeps a running maximum, sum and O for
// its stretch of a tile; a tile that spans several warps leaves one partial
// result per warp and kv8_combine_kernel joins them in order.  The share
// boundaries depend on the lengths and the SM count only, so results are
// reproducible.
//
// Loads.  Each warp streams its chunks through its own ring of half-chunks
// (K, then V) with 16-byte cp.async, two or more halves in flight: 8 warps x
// 16 KB cover 6.8 TB/s x 1 us = 45 KB per SM with room.  Shared memory is
// swizzled so that both the copies and the fragment reads are free of bank
// conflicts.
#include "lq_kv8_attn.cuh"

namespace lq {
namespace {

template <int D>
struct Dc {
    static constexpr int T = D == 256 ? 32 : 64;             // keys of a chunk
    static constexpr int TQ = T / 4;                         // keys of a thread of a quad
    static constexpr int NW = D == 256 ? 6 : 8;              // warps of a CTA
    static constexpr int NSLOT = D == 64 ? 6 : 3;            // half-chunks of a warp's ring
    static constexpr int HB = T * D;                         // bytes of a half-chunk
    static constexpr bool QS = D == 256;                     // q fragments in shared memory (registers are full)
    static constexpr int QB = QS ? D * 32 : 0;
    static constexpr int NMETA = 4;                          // chunks whose scales are held
    static constexpr int WB = NSLOT * HB + QB + NMETA * 64;  // shared memory of a warp
    static constexpr int SMEM = NW * WB;
    static constexpr int SUB = D / 16;                       // 16-byte pieces of a key
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 ld_s128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 ld_s64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ float ld_sf(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ void st_sf(uint32_t a, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory"); }
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A sequence as the split sees it: `tiles` row tiles per kv head, each over
// the same nc chunks: the first na, then those from cb on.
struct DecSeq {
    AttSeq q;
    int32_t tiles, na, cb, nc;
};
template <int T>
__device__ __forceinline__ DecSeq dec_seq(const AttnParams& P, int s) {
    DecSeq d;
    d.q = att_seq(P, s);
    d.tiles = (int)(((int64_t)d.q.n * (P.n_q / P.c.n_kv) + 7) >> 3);
    const int ce = (d.q.len + T - 1) / T;
    d.cb = min(d.q.lo / T, ce);
    d.na = min((d.q.pre + T - 1) / T, d.cb);
    d.nc = d.na + ce - d.cb;
    return d;
}
__device__ __forceinline__ int64_t dec_units(const AttnParams& P, const DecSeq& d) {
    return (int64_t)P.c.n_kv * d.tiles * d.nc;
}

// A place in the line.
struct Cur {
    DecSeq d;
    int32_t hk, tile, c;
};
template <int T>
__device__ __forceinline__ void cur_next(const AttnParams& P, Cur& k) {
    if (++k.c < k.d.nc) return;
    k.c = 0;
    if (++k.tile < k.d.tiles) return;
    k.tile = 0;
    if (++k.hk < P.c.n_kv) return;
    k.hk = 0;
    int s = k.d.q.s + 1;
    for (; s < P.s.nseq; ++s) {
        k.d = dec_seq<T>(P, s);
        if (dec_units(P, k.d) > 0) return;
    }
}
__device__ __forceinline__ int cur_chunk(const Cur& k) { return k.c < k.d.na ? k.c : k.d.cb + (k.c - k.d.na); }

// Workspace: base [nseq + 1] int64 (padded), then the partial results:
// 2 per worker, [8 rows][D] of O, then [8][2] of (max, sum).
__host__ __device__ constexpr int64_t part_floats(int d) { return 8 * (int64_t)d + 16; }
__host__ __device__ inline size_t base_bytes(int nseq) { return ((size_t)(nseq + 1) * 8 + 255) & ~size_t(255); }

// First worker of W whose share [U w / W, U (w + 1) / W) holds unit u.
__device__ __forceinline__ int owner(int64_t u, int64_t U, int W) { return (int)(((u + 1) * W - 1) / U); }

template <int D, bool EXTRA>
__global__ void __launch_bounds__(Dc<D>::NW * 32, 1) kv8_decode_kernel(const AttnParams P) {
    using F = Dc<D>;
    constexpr int T = F::T, TQ = F::TQ, NS = TQ / 4, NT = F::NW * 32;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t tb[NT + 1];
    __shared__ int64_t wsum[F::NW];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    pdl_launch_dependents();
    pdl_wait();

    // ---- the line: thread i sums the units of its sequences
    const int per = (P.s.nseq + NT - 1) / NT;
    int64_t mine = 0;
    for (int s = tid * per; s < min((tid + 1) * per, P.s.nseq); ++s) mine += dec_units(P, dec_seq<T>(P, s));
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int64_t before = 0, U = 0;
    for (int i = 0; i < F::NW; ++i) {
        if (i < warp) before += wsum[i];
        U += wsum[i];
    }
    tb[tid] = before + inc - mine;
    if (blockIdx.x == 0) {
        int64_t* base = reinterpret_cast<int64_t*>(P.ws);
        int64_t b = before + inc - mine;
        for (int s = tid * per; s < min((tid + 1) * per, P.s.nseq); ++s) {
            base[s] = b;
            b += dec_units(P, dec_seq<T>(P, s));
        }
        if (tid == 0) base[P.s.nseq] = U;
    }
    __syncthreads();

    // warps in use (none without a unit) and this one: few units go to different SMs
    const int W = (int)min((int64_t)gridDim.x * F::NW, U), w = warp * gridDim.x + blockIdx.x;
    if (w >= W) return;                                   // warps never meet again
    const int64_t u0 = U * w / W, u1 = U * (w + 1) / W;
    const int nu = (int)(u1 - u0);
    Cur cc;                                               // what is computed
    {
        int i = kv_find(NT, u0, [&](int x) { return tb[x]; });
        int64_t b = tb[i];
        int s = i * per;
        for (;; ++s) {
            cc.d = dec_seq<T>(P, s);
            const int64_t n = dec_units(P, cc.d);
            if (b + n > u0) break;
            b += n;
        }
        const int64_t r = u0 - b, item = r / cc.d.nc;
        cc.c = (int)(r % cc.d.nc);
        cc.tile = (int)(item % cc.d.tiles);
        cc.hk = (int)(item / cc.d.tiles);
    }
    Cur ci = cc;                                          // what is loaded

    const uint32_t wbase = smem_u32(smem) + warp * F::WB, qbase = wbase + F::NSLOT * F::HB, mbase = qbase + F::QB;
    const int pshift = P.c.pshift, Pg = 1 << pshift;
    const int64_t blk = (int64_t)D << pshift;             // bytes of a page's head
    int pg = -1;                                          // page of this thread's keys in the chunk to load
    auto load_page = [&]() {
        const int pos = cur_chunk(ci) * T + TQ * t;
        pg = pos < ci.d.q.len ? att_page(P, ci.d.q.s, pos) : -1;
    };
    load_page();
    int64_t gb = -1;                                      // byte offset of that page and head, -1: none
    int iu = 0;                                           // units whose K was loaded

    // half-chunk h: K (even) or V (odd) of unit h / 2
    auto issue = [&](int h) {
        if (h < 2 * nu) {
            const uint32_t slot = wbase + (h % F::NSLOT) * F::HB;
            const int tok = cur_chunk(ci) * T + TQ * t;
            if ((h & 1) == 0) {
                gb = pg < 0 ? -1 : ((int64_t)pg * P.c.n_kv + ci.hk) * blk;
                const int64_t kb = gb < 0 ? -1 : gb + (int64_t)(tok & (Pg - 1)) * D;
#pragma unroll
                for (int i = 0; i < F::HB / 512; ++i) {
                    const int idx = i * 32 + lane, r = idx / F::SUB, u = idx % F::SUB;
                    const int64_t b = __shfl_sync(0xFFFFFFFFu, kb, r / TQ);
                    const int sw = D >= 128 ? (r & 1) << 2 : 0;
                    if (b >= 0) cp16(slot + r * D + ((u ^ sw) << 4), P.c.k + b + (r % TQ) * D + u * 16);
                }
                // scales: threads 0-3 K's, 4-7 V's of key groups 0-3
                if (lane < 8) {
                    const uint32_t m = mbase + (iu % F::NMETA) * 64 + (lane >> 2) * 16 + t * 4;
                    const int64_t ph = gb < 0 ? 0 : (int64_t)pg * P.c.n_kv + ci.hk;
                    if (gb >= 0) cp4(m, (lane < 4 ? P.c.ks : P.c.vs) + ph);
                    else st_sf(m, 0.f);
                    if (lane < 4) st_sf(m + 32, gb < 0 ? 0.f : 1.f);
                }
            } else {
                // V: `upd` 16-byte pieces per dim in each of the chunk's pages
                const int lu = min(pshift - 4, T == 64 ? 2 : 1);
                const int64_t vb = gb < 0 ? -1 : gb + ((tok & (Pg - 1)) & ~15);
#pragma unroll
                for (int i = 0; i < F::HB / 512; ++i) {
                    const int idx = i * 32 + lane;
                    const int pi = idx / D >> lu, rem = idx - ((pi << lu) * D), d = rem >> lu, u = rem & ((1 << lu) - 1);
                    const int unit = (pi << lu) + u;                         // 16-byte piece of the chunk's row of dim d
                    const int64_t b = __shfl_sync(0xFFFFFFFFu, vb, T == 64 ? (pi << lu) : (pi << lu) * 2);
                    const int sw = T == 64 ? (d >> 1) & 3 : (d >> 2) & 1;
                    if (b >= 0) cp16(slot + d * T + ((unit ^ sw) << 4), P.c.v + b + ((int64_t)d << pshift) + u * 16);
                }
                if (++iu < nu) {
                    cur_next<T>(P, ci);
                    load_page();
                }
            }
        }
        cp_commit();
    };
    for (int h = 0; h < F::NSLOT - 1; ++h) issue(h);

    const int grp = P.n_q / P.c.n_kv;
    float* part = reinterpret_cast<float*>(P.ws + base_bytes(P.s.nseq));
    float o[D / 8][4];
    uint32_t qf[F::QS ? 1 : D / 16][4];
    float m = -INFINITY, l = 0.f, qs = 0.f, slope = 0.f;
    int p = 0, e0 = 0;
    bool rowok = false, fresh = true, from_start = false;
    int64_t qrow = 0;
    int head = 0;
    float is = 1.f;                                       // 2^-e0

    for (int u = 0; u < nu; ++u) {
        const AttSeq& q = cc.d.q;
        if (fresh) {
            // ---- a tile begins (or this warp's stretch of it): its rows
            fresh = false;
            from_start = cc.c == 0;
            const int r = cc.tile * 8 + g;
            rowok = r < q.n * grp;
            const int i = rowok ? r / grp : 0;
            head = cc.hk * grp + (rowok ? r % grp : 0);
            qrow = q.row0 + i;
            p = (int)min(max(q.start + i, (int64_t)-1), (int64_t)INT32_MAX - 1);
            slope = P.slopes ? __ldg(P.slopes + head) : 0.f;
            const int pe = att_page(P, q.s, cc.d.na > 0 ? 0 : min(cc.d.cb * T, q.len - 1));
            e0 = pe >= 0 ? att_e0(__ldg(P.c.vs + (int64_t)pe * P.c.n_kv + cc.hk)) : 0;
            is = att_pow2(-e0);
            const float* x = P.q + qrow * P.ld_q + (int64_t)head * D;
            // the row's largest |q| and its power of two
            float mx = 0.f;
            float v[D / 64][16];
#pragma unroll
            for (int a = 0; a < D / 64; ++a)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    v[a][e] = rowok ? __ldg(x + 64 * a + 16 * t + e) : 0.f;
                    mx = fmaxf(mx, fabsf(v[a][e]));
                }
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
            const int es = max(1, (int)((__float_as_uint(mx) >> 23) & 0xFFu) - 14);
            const float inv = __uint_as_float((uint32_t)(254 - es) << 23);
            qs = __uint_as_float((uint32_t)es << 23) * P.scale;
            if (F::QS) __syncwarp();                      // every lane has read the last tile's fragments
#pragma unroll
            for (int a = 0; a < D / 64; ++a)
#pragma unroll
                for (int k = 0; k < 4; ++k) {             // MMA step 4 a + k: dims 64 a + 16 t + 4 k .. + 3
                    uint32_t f[4];
                    att_split(v[a][4 * k] * inv, v[a][4 * k + 1] * inv, f[0], f[1]);
                    att_split(v[a][4 * k + 2] * inv, v[a][4 * k + 3] * inv, f[2], f[3]);
                    if (F::QS) {
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(qbase + ((4 * a + k) * 32 + lane) * 16),
                                     "r"(f[0]), "r"(f[1]), "r"(f[2]), "r"(f[3])
                                     : "memory");
                    } else {
#pragma unroll
                        for (int z = 0; z < 4; ++z) qf[F::QS ? 0 : 4 * a + k][z] = f[z];
                    }
                }
            m = -INFINITY;
            l = 0.f;
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int z = 0; z < 4; ++z) o[n][z] = 0.f;
        }

        // ---- S = Q K^T
        const int hK = 2 * u;
        cp_wait<F::NSLOT - 2>();
        __syncwarp();
        issue(hK + F::NSLOT - 1);
        const uint32_t mt = mbase + (u % F::NMETA) * 64 + t * 4;
        const float ks = ld_sf(mt), vs = ld_sf(mt + 16);
        const bool held = ld_sf(mt + 32) != 0.f;
        float s[NS][2][4];
#pragma unroll
        for (int x = 0; x < NS; ++x)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int z = 0; z < 4; ++z) s[x][j][z] = 0.f;
        {
            const uint32_t slot = wbase + (hK % F::NSLOT) * F::HB;
#pragma unroll
            for (int a = 0; a < D / 64; ++a) {
                uint32_t qa[4][4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (F::QS) {
                        const uint4 f = ld_s128(qbase + ((4 * a + k) * 32 + lane) * 16);
                        qa[k][0] = f.x;
                        qa[k][1] = f.y;
                        qa[k][2] = f.z;
                        qa[k][3] = f.w;
                    } else {
#pragma unroll
                        for (int z = 0; z < 4; ++z) qa[k][z] = qf[F::QS ? 0 : 4 * a + k][z];
                    }
                }
#pragma unroll
                for (int x = 0; x < NS; ++x)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int r = TQ * (g >> 1) + 4 * x + 2 * j + (g & 1);
                        const int sw = D >= 128 ? (g & 1) << 2 : 0;
                        const uint4 kw = ld_s128(slot + r * D + (((4 * a + t) ^ sw) << 4));
                        const uint32_t wv[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t b0, b1;
                            att_codes(wv[k], b0, b1);
                            mma16816(s[x][j], qa[k], b0, b1);
                        }
                    }
            }
        }

        // ---- weights
        const int chunk = cur_chunk(cc), j0 = chunk * T, jt = j0 + TQ * t;
        const bool full = held && j0 + T <= q.len &&
                          (!rowok || (p >= 0 && (j0 + T <= q.pre ||
                                                 (j0 + T - 1 <= p && (P.window == 0 || p - j0 < P.window)))));
        const bool all_full = __all_sync(0xFFFFFFFFu, full);
        bool vzero;
        const float rel = att_rel(vs * is, vzero), lv = log2f(rel);
        const float f = qs * ks * (EXTRA ? 1.f : ATT_LOG2E);
        float mx = -INFINITY;
#pragma unroll
        for (int x = 0; x < NS; ++x)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = s[x][j][e] + s[x][j][2 + e];
                    const int jj = jt + 4 * x + 2 * j + e;
                    if (EXTRA) {
                        v *= f;
                        if (P.softcap > 0.f) v = P.softcap * att_tanh(__fdividef(v, P.softcap));
                        v -= slope * fabsf((float)(p - jj));
                        v = fmaf(v, ATT_LOG2E, lv);
                    } else {
                        v = fmaf(v, f, lv);
                    }
                    if (!all_full && rowok) {
                        const bool see = att_sees(P, q, p, jj);
                        if (see && !held) record_status(P.status, STATUS_BADARG);
                        if (!see || !held) v = -INFINITY;
                    }
                    s[x][j][e] = v;
                    mx = fmaxf(mx, v);
                }
        // no key of this thread seen: its page's scale, which may be NaN, does
        // not count (a seen key of a NaN page still makes its weight NaN)
        const float il = mx == -INFINITY ? 0.f : 1.f / rel;
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
        if (__any_sync(0xFFFFFFFFu, mx > m)) {
            const float mn = fmaxf(m, mx), r = m == mn ? 1.f : att_ex2(m - mn);
            m = mn;
            l *= r;
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int z = 0; z < 4; ++z) o[n][z] *= r;
        }
        const float ref = m == -INFINITY ? 0.f : m - ATT_SHIFT;
        const uint32_t vmask = vzero ? 0u : 0xFFFFFFFFu;
        uint32_t wa[NS][4];
#pragma unroll
        for (int x = 0; x < NS; ++x)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float w0 = att_ex2(s[x][j][0] - ref), w1 = att_ex2(s[x][j][1] - ref);
                l = fmaf(w0 + w1, il, l);
                att_split(w0, w1, wa[x][2 * j], wa[x][2 * j + 1]);
                wa[x][2 * j] &= vmask;
                wa[x][2 * j + 1] &= vmask;
            }

        // ---- O += W V
        const int hV = hK + 1;
        cp_wait<F::NSLOT - 2>();
        __syncwarp();
        issue(hV + F::NSLOT - 1);
        {
            const uint32_t slot = wbase + (hV % F::NSLOT) * F::HB;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
                const int d = 8 * n + g;
                uint32_t wv[4];
                if (T == 64) {
                    const uint4 vw = ld_s128(slot + d * T + ((t ^ ((d >> 1) & 3)) << 4));
                    wv[0] = vw.x;
                    wv[1] = vw.y;
                    wv[2] = vw.z;
                    wv[3] = vw.w;
                } else {
                    const uint2 vw = ld_s64(slot + d * T + (((t >> 1) ^ ((d >> 2) & 1)) << 4) + (t & 1) * 8);
                    wv[0] = vw.x;
                    wv[1] = vw.y;
                }
#pragma unroll
                for (int x = 0; x < NS; ++x) {
                    uint32_t b0, b1;
                    att_codes(wv[x], b0, b1);
                    mma16816(o[n], wa[x], b0, b1);
                }
            }
        }

        // ---- the tile, or this warp's stretch of it, ends
        const bool tile_end = cc.c == cc.d.nc - 1;
        if (tile_end || u == nu - 1) {
            l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
            l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
            const float up = att_pow2(e0);
            if (tile_end && from_start) {
                const float r = l == 0.f ? 0.f : up / l;
                if (rowok) {
                    float* y = P.out + qrow * P.ld_out + (int64_t)head * D + 2 * t;
                    const bool vec = (reinterpret_cast<uintptr_t>(y) & 7) == 0;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        const float a = (o[n][0] + o[n][2]) * r, b = (o[n][1] + o[n][3]) * r;
                        if (vec) {
                            *reinterpret_cast<float2*>(y + 8 * n) = make_float2(a, b);
                        } else {
                            y[8 * n] = a;
                            y[8 * n + 1] = b;
                        }
                    }
                }
            } else {
                float* y = part + (2 * (int64_t)w + (from_start ? 1 : 0)) * part_floats(D);
                if (rowok) {
#pragma unroll
                    for (int n = 0; n < D / 8; ++n)
                        *reinterpret_cast<float2*>(y + g * D + 8 * n + 2 * t) =
                            make_float2((o[n][0] + o[n][2]) * up, (o[n][1] + o[n][3]) * up);
                    if (t == 0) *reinterpret_cast<float2*>(y + 8 * D + 2 * g) = make_float2(m, l);
                }
            }
            fresh = true;
        }
        if (u < nu - 1) cur_next<T>(P, cc);
    }
}

// Block (head, token): joins the partial results of one query row where
// several warps hold some, in the order of the line; zeros for rows that no
// chunk reaches.
constexpr int CMB_WARPS = 8;
template <int D>
__global__ void __launch_bounds__(CMB_WARPS * 32) kv8_combine_kernel(const AttnParams P, int warps) {
    constexpr int T = Dc<D>::T, V = D / 32;
    __shared__ float acc[CMB_WARPS][D];
    __shared__ float red[CMB_WARPS][2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, head = blockIdx.x, tok = blockIdx.y + blockIdx.z * 65535;
    pdl_wait();
    if (tok >= P.s.ntok) return;
    const int s = kv_find(P.s.nseq, tok, [&](int i) { return kv_cu(P.s, i); });
    const DecSeq d = dec_seq<T>(P, s);
    if (tok >= d.q.row0 + d.q.n) return;
    const int64_t* base = reinterpret_cast<const int64_t*>(P.ws);
    const int64_t U = base[P.s.nseq];
    const int grp = P.n_q / P.c.n_kv, hk = head / grp;
    const int r = (tok - d.q.row0) * grp + head % grp, tile = r >> 3, g = r & 7;
    float* y = P.out + (int64_t)tok * P.ld_out + (int64_t)head * D;
    if (d.nc == 0) {
        for (int i = threadIdx.x; i < D; i += CMB_WARPS * 32) y[i] = 0.f;
        return;
    }
    const int64_t b = base[s] + ((int64_t)hk * d.tiles + tile) * d.nc;
    const int W = (int)min((int64_t)warps, U);
    const int a = owner(b, U, W), z = owner(b + d.nc - 1, U, W);
    if (a == z) return;                                   // that warp wrote the row
    const float* part = reinterpret_cast<const float*>(P.ws + base_bytes(P.s.nseq));
    auto slot = [&](int k) { return part + (2 * (int64_t)k + (k == a ? 1 : 0)) * part_floats(D); };
    // the first warp's stretch begins with the tile; the later ones' at their first unit
    float m = -INFINITY;
    for (int k = a + (int)threadIdx.x; k <= z; k += CMB_WARPS * 32) m = fmaxf(m, slot(k)[8 * D + 2 * g]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (lane == 0) red[warp][0] = m;
    __syncthreads();
    for (int i = 0; i < CMB_WARPS; ++i) m = fmaxf(m, red[i][0]);
    float l = 0.f, o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int k = a + warp; k <= z; k += CMB_WARPS) {
        const float* x = slot(k);
        const float2 ml = *reinterpret_cast<const float2*>(x + 8 * D + 2 * g);
        const float c = ml.x == m ? 1.f : att_ex2(ml.x - m);
        l = fmaf(ml.y, c, l);
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = fmaf(x[g * D + lane + 32 * e], c, o[e]);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) acc[warp][lane + 32 * e] = o[e];
    if (lane == 0) red[warp][1] = l;
    __syncthreads();
    l = 0.f;
    for (int i = 0; i < CMB_WARPS; ++i) l += red[i][1];
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int i = threadIdx.x; i < D; i += CMB_WARPS * 32) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < CMB_WARPS; ++k) v += acc[k][i];
        y[i] = v * inv;
    }
}

constexpr int DEC_MAX_SMS = 160;

template <int D>
cudaError_t decode_launch(const AttnParams& P, int sms, cudaStream_t st) {
    using F = Dc<D>;
    const bool extra = P.softcap > 0.f || P.slopes;
    auto kern = extra ? kv8_decode_kernel<D, true> : kv8_decode_kernel<D, false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, F::SMEM);
    if (e != cudaSuccess) return e;
    const int grid = sms < DEC_MAX_SMS ? sms : DEC_MAX_SMS;
    kern<<<grid, F::NW * 32, F::SMEM, st>>>(P);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t c{};
    const int ty = P.s.ntok < 65535 ? P.s.ntok : 65535;
    c.gridDim = dim3((unsigned)P.n_q, (unsigned)ty, (unsigned)((P.s.ntok + 65534) / 65535));
    c.blockDim = dim3(CMB_WARPS * 32);
    c.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kv8_combine_kernel<D>, P, grid * F::NW);
}

}  // namespace

size_t kv8_attn_workspace(int n_q, int n_kv, int d, int nseq, int ntok) {
    const int nw = d == 64 ? Dc<64>::NW : d == 128 ? Dc<128>::NW : Dc<256>::NW;
    return base_bytes(nseq) + (size_t)DEC_MAX_SMS * nw * 2 * part_floats(d) * sizeof(float);
}

cudaError_t launch_kv8_attn(const AttnParams& P, int sms, cudaStream_t st) {
    return P.c.d == 64    ? decode_launch<64>(P, sms, st)
           : P.c.d == 128 ? decode_launch<128>(P, sms, st)
                          : decode_launch<256>(P, sms, st);
}

}  // namespace lq

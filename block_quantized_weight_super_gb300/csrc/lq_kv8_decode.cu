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
// dealt to the warps of one CTA per SM in equal shares, whatever the lengths;
// they never meet.  A warp keeps a running maximum, sum and O for its stretch
// of a tile; a tile that spans several warps leaves one partial result per
// warp and kv8_combine_kernel joins them in order.  The shares depend on the
// lengths and the SM count only, so results are reproducible.
//
// Loads.  Each warp streams its chunks through its own ring of half-chunks
// (K, then V), always all but one of them in flight: bulk copies by its first
// lanes, one per page (a tensor copy where a chunk is a slice of a page's V
// rows).  The lanes hold the next 32 page indices of the table in a register.
#include "lq_kv8_attn.cuh"

namespace lq {
namespace {

template <int D>
struct Dc {
    static constexpr int T = D == 64 ? 64 : 32;              // keys of a chunk
    static constexpr int TQ = T / 4;                         // keys of a thread of a quad
    static constexpr int NC = D == 64 ? 15 : D == 128 ? 12 : 8;    // warps: 4, 3 or 2 per scheduler, as registers allow
    static constexpr int NT = NC * 32;
    static constexpr int NSLOT = D == 256 ? 2 : 3;   // half-chunks of a warp's ring
    static constexpr int HB = T * D;                         // bytes of a half-chunk
    static constexpr int HBP = HB + 128;                     // with the padding between pages of V
    static constexpr int QB = D * 32;                        // q fragments
    static constexpr int NMETA = 4;                          // chunks whose scales are held
    static constexpr int WB = NSLOT * HBP + QB + NMETA * 64; // shared memory of a warp (a multiple of 128)
    static constexpr int SMEM = NC * WB;
};

__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives on the barrier (one of its expected arrivals) once this thread's
// cp.async so far have landed.
__device__ __forceinline__ void cp_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
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
__global__ void __launch_bounds__(Dc<D>::NT, 1) kv8_decode_kernel(const AttnParams P, const __grid_constant__ CUtensorMap vmap) {
    using F = Dc<D>;
    constexpr int T = F::T, TQ = F::TQ, NS = TQ / 4, NT = F::NT, NC = F::NC, NSLOT = F::NSLOT;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t tb[NT];
    __shared__ int64_t wsum[NC];
    __shared__ uint64_t full[NC][NSLOT];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    pdl_launch_dependents();
    if (tid < NC * NSLOT) {
        mbar_init(&full[0][0] + tid, 1 + T / 16);         // the copies' bytes, the scales' lanes
        fence_mbar_init();
    }

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
    for (int i = 0; i < NC; ++i) {
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
    const int W = (int)min((int64_t)gridDim.x * NC, U), w = warp * gridDim.x + blockIdx.x;
    if (w >= W) return;                                   // warps never meet again
    const int64_t u0 = U * w / W;
    const int nu = (int)(U * (w + 1) / W - u0);
    Cur cc;                                               // the unit at hand
    {
        const int i = kv_find(NT, u0, [&](int x) { return tb[x]; });
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
    uint64_t* const bars = full[warp];
    const uint32_t wbase = smem_u32(smem) + warp * F::WB, qbase = wbase + NSLOT * F::HBP, mbase = qbase + F::QB;
    const int pshift = P.c.pshift, Pg = 1 << pshift;

    // ---- loading, ahead of the computation
    Cur ci = cc;                                          // the unit to load
    const int lpw = min(pshift, T == 64 ? 6 : 5), lnp = (T == 64 ? 6 : 5) - lpw;   // log2 of the keys a page gives a chunk, of its pages
    int wc = ci.c, win = -1;                              // lane x: the page x & (pages - 1) of chunk wc + x / pages of this item
    auto window = [&]() {
        wc = ci.c;
        Cur k = ci;
        k.c += lane >> lnp;
        const int pos = cur_chunk(k) * T + ((lane & ((1 << lnp) - 1)) << lpw);
        win = k.c < k.d.nc && pos < k.d.q.len ? att_page(P, k.d.q.s, pos) : -1;
    };
    window();
    auto issue = [&](int h) {                             // half-chunk h: K (even) or V (odd) of unit h / 2
        if (h >= 2 * nu) return;
        const int slot = h % NSLOT, np = 1 << lnp;
        uint64_t* bar = bars + slot;
        const uint32_t dst = wbase + slot * F::HBP, pb = (uint32_t)D << lpw;
        const int pg = __shfl_sync(0xFFFFFFFFu, win, ((ci.c - wc) << lnp) + (lane & (np - 1)));   // lane i: the chunk's page i
        const int pm = __shfl_sync(0xFFFFFFFFu, pg, (lane & 3) << 4 >> lpw);   // lane i: the page of the chunk's i-th 16 keys
        const bool have = lane < np && pg >= 0;
        const int n = __popc(__ballot_sync(0xFFFFFFFFu, have));
        const int off = cur_chunk(ci) * T & (Pg - 1);     // the chunk's place in its page (0 unless it is a part of it)
        const int64_t ph = (int64_t)pg * P.c.n_kv + ci.hk;
        if ((h & 1) == 0) {
            if (lane < T / 16) {
                const uint32_t m = mbase + (h / 2 % F::NMETA) * 64 + 4 * lane;
                st_sf(m + 32, pm < 0 ? 0.f : 1.f);
                if (pm < 0) {
                    st_sf(m, 0.f);
                    st_sf(m + 16, 0.f);
                } else {
                    cp4(m, P.c.ks + (int64_t)pm * P.c.n_kv + ci.hk);
                    cp4(m + 16, P.c.vs + (int64_t)pm * P.c.n_kv + ci.hk);
                }
                cp_arrive(bar);
            }
            if (have) bulk_copy(dst + lane * pb, P.c.k + ((ph * D) << pshift) + (int64_t)off * D, pb, bar);
        } else {
            if (lane < T / 16) mbar_arrive(bar);
            if (have) {
                if (lpw == pshift) bulk_copy(dst + lane * (pb + (lnp ? 128 >> lnp : 0)), P.c.v + ((ph * D) << pshift), pb, bar);
                else tma_load_3d(dst, &vmap, off, 0, (int)ph, bar);
            }
        }
        if (lane == 0) {
            if (n > 0) mbar_arrive_expect_tx(bar, n * pb);
            else mbar_arrive(bar);
        }
        if ((h & 1) && h / 2 + 1 < nu) {
            cur_next<T>(P, ci);
            if (ci.c == 0 || ci.c - wc >= 32 >> lnp) window();
        }
    };
    for (int h = 0; h < NSLOT - 1; ++h) issue(h);

    const int grp = P.n_q / P.c.n_kv;
    float* part = reinterpret_cast<float*>(P.ws + base_bytes(P.s.nseq));
    const int vw = min(Pg, T);                            // keys per row of V in shared memory
    const uint32_t voff = (uint32_t)(TQ * t / vw) * ((uint32_t)vw * D + (vw < T ? 128u / (T / vw) : 0u)) + (TQ * t) % vw + g * vw;
    float o[D / 8][4];
    float m = -INFINITY, l = 0.f, qs = 0.f, slope = 0.f;
    int p = 0, e0 = 0;
    bool rowok = false, fresh = true, from_start = false;
    int64_t qrow = 0;
    int head = 0;
    float is = 1.f;                                       // 2^-e0

    // Waits for half-chunk h; every lane is past the half before it then,
    // whose slot is the next to fill.  On a timeout the halves in flight
    // still land (bounded) before the warp leaves.
    auto arrived = [&](int h) -> bool {
        if (__all_sync(0xFFFFFFFFu, mbar_wait_bounded(bars + h % NSLOT, (uint32_t)((h / NSLOT) & 1), P.timeout_ns))) return true;
        record_status(P.status, STATUS_TIMEOUT);
        for (int k = h; k < min(h + NSLOT - 1, 2 * nu); ++k)
            mbar_wait_bounded(bars + k % NSLOT, (uint32_t)((k / NSLOT) & 1), drain_bound(P.timeout_ns));
        return false;
    };
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
            const float* x = P.q + qrow * P.ld_q + (int64_t)head * D + 16 * t;
            const int pe = att_page(P, q.s, cc.d.na > 0 ? 0 : min(cc.d.cb * T, q.len - 1));
            // the row's largest |q| and its power of two
            float mx = 0.f;
            float v[D / 64][16];
            const bool vec = ((reinterpret_cast<uintptr_t>(P.q) | (P.ld_q * 4)) & 15) == 0;
#pragma unroll
            for (int a = 0; a < D / 64; ++a)
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
                    const float* y = x + 64 * a + e;
                    if (rowok) z = vec ? __ldg(reinterpret_cast<const float4*>(y)) : make_float4(__ldg(y), __ldg(y + 1), __ldg(y + 2), __ldg(y + 3));
                    v[a][e] = z.x;
                    v[a][e + 1] = z.y;
                    v[a][e + 2] = z.z;
                    v[a][e + 3] = z.w;
                }
            slope = P.slopes ? __ldg(P.slopes + head) : 0.f;
            e0 = pe >= 0 ? att_e0(__ldg(P.c.vs + (int64_t)pe * P.c.n_kv + cc.hk)) : 0;
            is = att_pow2(-e0);
#pragma unroll
            for (int a = 0; a < D / 64; ++a)
#pragma unroll
                for (int e = 0; e < 16; ++e) mx = fmaxf(mx, fabsf(v[a][e]));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
            const int es = max(1, (int)((__float_as_uint(mx) >> 23) & 0xFFu) - 14);
            const float inv = __uint_as_float((uint32_t)(254 - es) << 23);
            qs = __uint_as_float((uint32_t)es << 23) * P.scale;
            __syncwarp();                                 // every lane has read the last tile's fragments
#pragma unroll
            for (int a = 0; a < D / 64; ++a)
#pragma unroll
                for (int k = 0; k < 4; ++k) {             // MMA step 4 a + k: dims 64 a + 16 t + 4 k .. + 3
                    uint32_t f[4];
                    att_split(v[a][4 * k] * inv, v[a][4 * k + 1] * inv, f[0], f[1]);
                    att_split(v[a][4 * k + 2] * inv, v[a][4 * k + 3] * inv, f[2], f[3]);
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(qbase + ((4 * a + k) * 32 + lane) * 16),
                                 "r"(f[0]), "r"(f[1]), "r"(f[2]), "r"(f[3])
                                 : "memory");             // (read back by this lane alone)
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
        if (!arrived(hK)) return;
        issue(hK + NSLOT - 1);
        const uint32_t mt = mbase + (u % F::NMETA) * 64 + (TQ * t / 16) * 4;
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
            const uint32_t kb = wbase + (hK % NSLOT) * F::HBP + (TQ * (g >> 1) + (g & 1)) * D + 16 * t;
#pragma unroll
            for (int a = 0; a < D / 64; ++a) {
                uint32_t qa[4][4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint4 f = ld_s128(qbase + ((4 * a + k) * 32 + lane) * 16);
                    qa[k][0] = f.x;
                    qa[k][1] = f.y;
                    qa[k][2] = f.z;
                    qa[k][3] = f.w;
                }
#pragma unroll
                for (int x = 0; x < NS; ++x)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint4 kw = ld_s128(kb + (4 * x + 2 * j) * D + 64 * a);
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
        const int j0 = cur_chunk(cc) * T, jt = j0 + TQ * t;
        const bool whole = held && j0 + T <= q.len &&
                           (!rowok || (p >= 0 && (j0 + T <= q.pre ||
                                                  (j0 + T - 1 <= p && (P.window == 0 || p - j0 < P.window)))));
        const bool all_whole = __all_sync(0xFFFFFFFFu, whole);
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
                    if (!all_whole && rowok) {
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
        if (!arrived(hV)) return;
        issue(hV + NSLOT - 1);
        {
            const uint32_t vb = wbase + (hV % NSLOT) * F::HBP + voff;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
                uint32_t wv[4];
                if (T == 64) {
                    const uint4 z = ld_s128(vb + 8 * n * vw);
                    wv[0] = z.x;
                    wv[1] = z.y;
                    wv[2] = z.z;
                    wv[3] = z.w;
                } else {
                    const uint2 z = ld_s64(vb + 8 * n * vw);
                    wv[0] = z.x;
                    wv[1] = z.y;
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
    // slices of T keys of a page's V rows, where a page holds more
    CUtensorMap vmap{};
    const int64_t pg = (int64_t)1 << P.c.pshift;
    if (pg > F::T && api_byte_map(&vmap, P.c.v, pg, D, P.c.n_pages * P.c.n_kv, F::T, D) != 0) return cudaErrorInvalidValue;
    const bool extra = P.softcap > 0.f || P.slopes;
    auto kern = extra ? kv8_decode_kernel<D, true> : kv8_decode_kernel<D, false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, F::SMEM);
    if (e != cudaSuccess) return e;
    const int grid = sms < DEC_MAX_SMS ? sms : DEC_MAX_SMS;
    kern<<<grid, F::NT, F::SMEM, st>>>(P, vmap);
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
    return cudaLaunchKernelEx(&c, kv8_combine_kernel<D>, P, grid * F::NC);
}

}  // namespace

size_t kv8_attn_workspace(int n_q, int n_kv, int d, int nseq, int ntok) {
    const int nw = d == 64 ? Dc<64>::NC : d == 128 ? Dc<128>::NC : Dc<256>::NC;
    return base_bytes(nseq) + (size_t)DEC_MAX_SMS * nw * 2 * part_floats(d) * sizeof(float);
}

cudaError_t launch_kv8_attn(const AttnParams& P, int sms, cudaStream_t st) {
    return P.c.d == 64    ? decode_launch<64>(P, sms, st)
           : P.c.d == 128 ? decode_launch<128>(P, sms, st)
                          : decode_launch<256>(P, sms, st);
}

}  // namespace lq

// kv_attn_wide.cuh -- attention over the quantised cache for many query rows:
// a question's tokens against what the session holds.
//
// With more than 16 query rows a line, k_kv_attn would read and widen every
// code once per 16 rows; here 128 rows share one pass, on the fifth-generation
// tensor cores.  A CTA (one per SM) walks tiles of 128 tokens:
//   - all warps widen the tile's codes to fp16 in shared memory (exact; rows
//     of 8 channels are the operands' 16-byte core-matrix rows for keys, K-major,
//     and values, MN-major, alike), two buffers deep;
//   - S = Q K^T, M = N = 128, fp32 in tensor memory, Q in one (bf16) or two
//     (fp32) fp16 parts from shared memory;
//   - each thread takes a quarter of one query row's scores: scales, mask,
//     running reference, sum and value exponent of the row as in k_kv_attn, the
//     weights packed to fp16 parts back into tensor memory;
//   - O += P V with P from tensor memory, while the next tile's S is formed.
// Measured on 17 fp32 queries of 7 heads over 20 to 8190 e4m3 tokens of 4 sessions, 4
// heads, 2 layers: 52 us (k_kv_attn in tiles of 16 rows: 102 us; the bytes alone would take 6).
// A tile takes about 6400 cycles: 3000 in which the thread that issues the 32
// products (two parts) waits at the tensor cores' queue, 1500 for the
// exponentials, 1800 for widening; a line's begin and end take 20000 more.  A
// warp of its own for the issue leaves 96 registers a thread, and what spills waits
// for its loads at once: 56 to 73 us.  At 128 registers INT8 still spills 96 to 112 bytes
// a thread, e4m3 60, INT4 none to 24.
#pragma once
#include "kv_attn.cuh"
#include "tc_common.cuh"

namespace milo {

constexpr int KW_ROWS = 128, KW_TOK = 128, KW_THREADS = 512;
static_assert(KW_TOK == D, "a thread's columns of the scores are also its columns of the output");
constexpr int KW_SPLIT = KW_THREADS / KW_ROWS, KW_COLS = KW_TOK / KW_SPLIT;   // threads of a query row, tokens of each
static_assert(KW_SPLIT == 4, "a row's threads exchange four values");
constexpr int KW_WARPS = KW_THREADS / 32, KW_TAKE = KW_TOK * 8 / KW_THREADS;  // 16-channel pieces of a tile that a thread widens
constexpr uint32_t KW_TMEM = 512, KW_S = 0, KW_O = 128, KW_P = 256;   // columns: scores, output, weights (2 parts of 64)
constexpr int KW_TILE = KW_TOK * D * 2;                               // bytes of a widened tile

template <typename T> struct KwSmem {
    static constexpr int PARTS = sizeof(T) == 4 ? 2 : 1;
    unsigned char q[PARTS][KW_TILE], k[2][KW_TILE], v[2][KW_TILE];
    float ks[2][KW_TOK], vs[2][KW_TOK];       // scales of a tile's rows
    float top[2][4];                          // greatest value scale of 32 rows each
    float x[KW_SPLIT][KW_ROWS];               // exchange between a row's threads: scores, sums
    float y[KW_SPLIT][KW_ROWS];               // value scales of the tokens that the row sees
    float sc[KW_ROWS];
    int seen[KW_ROWS];
    int least;                                // tokens that every row sees
    KaScan scan;
    uint64_t bar_s, bar_o;                    // S formed; P V added
    uint32_t tmem;
};

// A thread's share of a tile: KW_TAKE times 16 channels of a row (row kw_row(j), channels 16 kw_c16(j) ..)
__device__ __forceinline__ int kw_row(int j) { return 8 * ((threadIdx.x / 32 + KW_WARPS * j) / 2) + threadIdx.x % 8; }
__device__ __forceinline__ int kw_c16(int j) { return 4 * ((threadIdx.x / 32 + KW_WARPS * j) % 2) + (threadIdx.x % 32) / 8; }

// Loads that stay where they are written: their results are used a tile later, and a load that may be moved is moved
// behind the wait that it is meant to pass
__device__ __forceinline__ uint4 kw_ldg16(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 kw_ldg8(const void *p) {
    uint2 v;
    asm volatile("ld.global.nc.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t kw_ldg4(const void *p) {
    uint32_t v;
    asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

template <int DT> struct KwRaw {
    uint4 w[KW_TAKE];                         // 4 bits: x and y
    uint32_t p[DT == MILO_INT4 ? KW_TAKE : 1];      // 4 bits: (scale, zero) of the channels' group
    __device__ __forceinline__ void load(const unsigned char *codes, const unsigned char *par, int t0, int end) {
#pragma unroll
        for (int j = 0; j < KW_TAKE; ++j) {
            const int64_t t = t0 + kw_row(j);
            w[j] = make_uint4(0u, 0u, 0u, 0u);
            if (DT == MILO_INT4) p[j] = 0u;
            if (t < end) {
                if constexpr (DT == MILO_INT4) {
                    const uint2 u = kw_ldg8(codes + t * 64 + 8 * kw_c16(j));
                    w[j].x = u.x;
                    w[j].y = u.y;
                    p[j] = kw_ldg4(par + t * 16 + 4 * (kw_c16(j) / 2));
                } else {
                    w[j] = kw_ldg16(codes + t * 128 + 16 * kw_c16(j));
                }
            }
        }
    }
    // widened into a tile [token / 8][channel / 8][token % 8][channel % 8].  4-bit codes come out in the order
    // 0 4 1 5 2 6 3 7 of each 8 channels (kw_order).
    __device__ __forceinline__ void store(unsigned char *tile) const {
#pragma unroll
        for (int j = 0; j < KW_TAKE; ++j) {
            uint32_t o[8];
            if constexpr (DT == MILO_INT4) {
                const __half2 s = ka_h(__byte_perm(p[j], 0u, 0x1010)), z = ka_h(__byte_perm(p[j], 0u, 0x3232));
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t x = e ? w[j].y : w[j].x, y = x >> 8;
                    o[4 * e] = ka_int4<false>(x, s, z);
                    o[4 * e + 1] = ka_int4<true>(x, s, z);
                    o[4 * e + 2] = ka_int4<false>(y, s, z);
                    o[4 * e + 3] = ka_int4<true>(y, s, z);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t x = ka_word(w[j], e);
                    if constexpr (DT == MILO_INT8) {
                        x ^= 0x80808080u;
                        o[2 * e] = ka_int8(x, 0x4140);
                        o[2 * e + 1] = ka_int8(x, 0x4342);
                    } else {
                        o[2 * e] = ka_fp8(x, 0x1404);
                        o[2 * e + 1] = ka_fp8(x, 0x3424);
                    }
                }
            }
            unsigned char *to = tile + (kw_row(j) / 8) * 2048 + 2 * kw_c16(j) * 128 + (threadIdx.x % 8) * 16;
            *reinterpret_cast<uint4 *>(to) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4 *>(to + 128) = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
};
// channel (of 8) at place p of a widened row
template <int DT> __device__ __forceinline__ constexpr int kw_order(int p) { return DT == MILO_INT4 ? p / 2 + 4 * (p % 2) : p; }

__device__ __forceinline__ void kw_rows_sync(int warp) {   // the warps that share 32 query rows
    asm volatile("bar.sync %0, %1;" ::"r"(1 + warp % 4), "n"(32 * KW_SPLIT) : "memory");
}

template <typename T, int DT> __global__ void __launch_bounds__(KW_THREADS, 1) k_kv_attn_wide(const __grid_constant__ KvAttnArgs a) {
    using Sm = KwSmem<T>;
    constexpr int PARTS = Sm::PARTS, BEGIN = KaShape<16>::BEGIN;
    constexpr bool PAR = DT != MILO_INT4;
    constexpr float UP = DT == MILO_FP8 ? KA_FP8_UP : 1.f;
    extern __shared__ __align__(128) unsigned char kw_raw[];
    Sm &sm = *reinterpret_cast<Sm *>(kw_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    KaRun<false, 16> run;
    const bool any_work = run.begin(a, sm.scan);
    if (tid == 0) a.split[blockIdx.x] = make_int4(-1, 0, 0, 0);
    kv_launch_next();
    if (!any_work) return;
    const KaClass<false, 16> &cl = run.cl;
    if (tid == 0) {
        tc::mbar_init(&sm.bar_s, 1);
        tc::mbar_init(&sm.bar_o, 1);
        tc::fence_barrier_init();
    }
    if (warp == 0) {
        tc::tmem_alloc(&sm.tmem, KW_TMEM);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = sm.tmem;
    const int row = 32 * (warp % 4) + lane, col = KW_COLS * (warp / 4);   // this thread's query row and first token of a tile
    const uint32_t lanes = (uint32_t)(32 * (warp % 4)) << 16;      // its warp's tensor-memory lanes
    const uint32_t sq = tc::smem_u32(sm.q), sk = tc::smem_u32(sm.k), sv = tc::smem_u32(sm.v);
    uint32_t n_s = 0, n_o = 0;                                     // phases of the two barriers
    bool ok = true;

    // one thread issues; the descriptors of a product's steps differ by constants in their address field (16-byte units),
    // so that a step costs an addition
    const uint64_t d_q = tc::smem_desc(sq, 128, 2048, tc::LAYOUT_NONE), d_k = tc::smem_desc(sk, 128, 2048, tc::LAYOUT_NONE);
    const uint64_t d_v = tc::smem_desc(sv, 2048, 128, tc::LAYOUT_NONE);
    auto issue_s = [&](int buf) {
        constexpr uint32_t id = tc::idesc_f16(KW_ROWS, KW_TOK, 0, 0, 0);
        const uint64_t k = d_k + (uint64_t)(buf * (KW_TILE / 16));
#pragma unroll
        for (int p = 0; p < PARTS; ++p)
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
                tc::mma_ss(tmem + KW_S, d_q + p * (KW_TILE / 16) + j * 16, k + j * 16, id, (p | j) != 0);
        tc::mma_commit(&sm.bar_s);
    };
    auto issue_o = [&](int buf, bool first) {
        constexpr uint32_t id = tc::idesc_f16(KW_ROWS, D, 0, 0, 1);
        const uint64_t v = d_v + (uint64_t)(buf * (KW_TILE / 16));
#pragma unroll
        for (int p = 0; p < PARTS; ++p)
#pragma unroll
            for (int j = 0; j < KW_TOK / 16; ++j)
                tc::mma_ts(tmem + KW_O, tmem + KW_P + 64 * p + 8 * j, v + j * 256, id, (p | j) != 0 || !first);
        tc::mma_commit(&sm.bar_o);
    };

    while (run.u0 < run.u1 && ok) {
        const int s0 = run.s0(), s1 = run.s1(), l = run.l, h = run.h;
        const int64_t sh = (int64_t)cl.s * a.c.H + h;
        const unsigned char *kc = a.c.codes(l, sh, 0), *vc = a.c.codes(l, sh, 1);
        const unsigned char *kp = a.c.params(l, sh, 0), *vp = a.c.params(l, sh, 1);
        const int first = max(s0 - BEGIN, 0), end = cl.end;        // tiles [first, first + n)
        const int n = max(min((end + KW_TOK - 1) / KW_TOK, s1 - BEGIN) - first, 0);
        const bool whole = s0 == 0 && s1 == run.per;
        const int64_t part = 2 * (int64_t)blockIdx.x + (s0 == 0 ? 1 : 0);
        if (n == 0 && !whole) {                                    // the units that stand for a line's begin alone
            if (tid < KW_ROWS) a.part_ml[part * KW_ROWS + tid] = make_float2(-INFINITY, 0.f);
            if (s0 == 0 && tid == 0) a.split[blockIdx.x] = run.split();
            run.next(a, s1);
            continue;
        }
        KwRaw<DT> rk, rv;
        float rks = 0.f, rvs = 0.f;
        auto load_k = [&](int i) { rk.load(kc, kp, (first + i) * KW_TOK, end); };
        auto load_v = [&](int i) {
            rv.load(vc, vp, (first + i) * KW_TOK, end);
            if (PAR && tid < KW_TOK) {
                const int t = (first + i) * KW_TOK + tid;
                rks = rvs = 0.f;
                if (t < end) {
                    rks = __uint_as_float(kw_ldg4(kp + 4 * (int64_t)t));
                    rvs = __uint_as_float(kw_ldg4(vp + 4 * (int64_t)t));
                }
            }
        };
        auto store_scales = [&](int buf) {
            if (PAR && tid < KW_TOK) {
                sm.ks[buf][tid] = rks;
                sm.vs[buf][tid] = rvs;
                const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(rvs));
                if (lane == 0) sm.top[buf][warp] = __uint_as_float(top);
            }
        };
        if (n > 0) {
            load_k(0);
            load_v(0);
        }
        // the queries, eight rows a warp: a lane holds 8-channel chunks x, x + 4, x + 8, x + 12 of its row
        const int x = lane / 8;
#pragma unroll
        for (int g = 0; g < 16 / KW_WARPS; ++g) {
            const int r = 8 * (warp + KW_WARPS * g) + lane % 8;
            const bool live = r < cl.rows;
            float q[4][8], mx = 0.f;
            const T *src = (const T *)a.q + (live ? cl.row(a, l, h, r) : 0) * D;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint4 w[sizeof(T) / 2];                            // 8 channels
#pragma unroll
                for (int e = 0; e < (int)sizeof(T) / 2; ++e) {
                    w[e] = make_uint4(0u, 0u, 0u, 0u);
                    if (live) w[e] = __ldg(reinterpret_cast<const uint4 *>(src + 8 * (x + 4 * i)) + e);
                }
                const T *t = reinterpret_cast<const T *>(w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    q[i][e] = to_f32(t[kw_order<DT>(e)]);
                    mx = fmaxf(mx, fabsf(q[i][e]));
                }
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const int e2 = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 127);
            const float up = __uint_as_float((uint32_t)(135 - e2) << 23), down = __uint_as_float((uint32_t)(119 + e2) << 23);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float y0 = isfinite(q[i][2 * e]) ? q[i][2 * e] * up : NAN;
                    const float y1 = isfinite(q[i][2 * e + 1]) ? q[i][2 * e + 1] * up : NAN;
                    const __half2 hh = __floats2half2_rn(y0, y1);
                    hi[e] = ka_u(hh);
                    lo[e] = ka_u(__floats2half2_rn(y0 - __low2float(hh), y1 - __high2float(hh)));
                }
                const int at = (r / 8) * 2048 + (x + 4 * i) * 128 + (r % 8) * 16;
                *reinterpret_cast<uint4 *>(&sm.q[0][at]) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                if (PARTS == 2) *reinterpret_cast<uint4 *>(&sm.q[PARTS - 1][at]) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            if (x == 0) {
                sm.sc[r] = a.scale * UP * down;
                sm.seen[r] = live ? cl.seen(a, r) : end;
                if (r == 0) sm.least = sm.seen[0];
            }
        }
        if (n > 0) {
            rk.store(sm.k[0]);
            rv.store(sm.v[0]);
            store_scales(0);
        }
        tc::fence_async_smem();
        tc::tc_fence_before();
        __syncthreads();
        if (n > 0 && tid == 0) {
            tc::tc_fence_after();
            issue_s(0);
        }
        if (n > 1) {
            load_k(1);
            load_v(1);
        }
        const float sc = sm.sc[row];
        const int seen = sm.seen[row];
        const bool idle = 32 * (warp % 4) >= cl.rows;              // a warp of rows behind the last: their weights are never read
        float ref = -INFINITY, sum = 0.f, e_max = 0.f, e_inv = 0.f;

        for (int i = 0; i < n; ++i) {
            const int buf = i & 1, t0 = (first + i) * KW_TOK + col;
            if (i + 1 < n) {
                rk.store(sm.k[buf ^ 1]);                           // S of the tile before it is formed
                if (i + 2 < n) load_k(i + 2);
            }
            ok = tc::mbar_wait(&sm.bar_s, n_s & 1u) && ok;
            ++n_s;
            tc::tc_fence_after();
            float z[KW_COLS];
            float fac = 1.f;
            bool rescale = false;
            if (!idle) {
                float top = -INFINITY;
                {
                    uint32_t r[KW_COLS];
                    tc::tmem_ld32(tmem + KW_S + lanes + col, r);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < KW_COLS; c += 4) {
                        float4 f = make_float4(sc, sc, sc, sc);
                        if (PAR) {
                            const float4 k4 = *reinterpret_cast<const float4 *>(&sm.ks[buf][col + c]);
                            f = make_float4(k4.x * sc, k4.y * sc, k4.z * sc, k4.w * sc);
                        }
                        z[c] = __uint_as_float(r[c]) * f.x;
                        z[c + 1] = __uint_as_float(r[c + 1]) * f.y;
                        z[c + 2] = __uint_as_float(r[c + 2]) * f.z;
                        z[c + 3] = __uint_as_float(r[c + 3]) * f.w;
                    }
                }
                if (t0 + KW_COLS > seen) {
#pragma unroll
                    for (int c = 0; c < KW_COLS; ++c)
                        if (t0 + c >= seen) z[c] = -INFINITY;
                }
#pragma unroll
                for (int c = 0; c < KW_COLS; ++c) top = fmaxf(top, z[c]);
                sm.x[warp / 4][row] = top;
                const bool edge = PAR && (first + i + 1) * KW_TOK > sm.least;   // some row does not see all of the tile
                if (edge) {
                    float w = 0.f;
                    for (int c = 0; c < min(KW_COLS, seen - t0); ++c) w = fmaxf(w, sm.vs[buf][col + c]);
                    sm.y[warp / 4][row] = w;
                }
                kw_rows_sync(warp);
#pragma unroll
                for (int y = 0; y < KW_SPLIT; ++y) top = fmaxf(top, sm.x[y][row]);
                if (top > ref + KA_RAISE) {
                    fac = ref == -INFINITY ? 0.f : ka_exp2(ref - top);
                    ref = top;
                    rescale = true;
                }
                if (PAR) {
                    float4 t4 = *reinterpret_cast<const float4 *>(sm.top[buf]);
                    if (edge) t4 = make_float4(sm.y[0][row], sm.y[1][row], sm.y[2][row], sm.y[3][row]);
                    const uint32_t bits = __float_as_uint(fmaxf(fmaxf(t4.x, t4.y), fmaxf(t4.z, t4.w))) & 0x7f800000u;
                    const float pw = __uint_as_float(min(max(bits, KA_E_MIN), 0x7e800000u));   // 2^E
                    sum *= fac;
                    if (pw > e_max) {
                        fac *= e_max * (1.f / pw);
                        e_max = pw;
                        e_inv = KA_UP / pw;
                        rescale = true;
                    }
                } else {
                    sum *= fac;
                }
            }
            if (i > 0) {                                           // P and O are free, and the value tile before this one
                ok = tc::mbar_wait(&sm.bar_o, n_o & 1u) && ok;
                ++n_o;
                tc::tc_fence_after();
            }
            if (!idle) {
                if (i > 0 && __any_sync(0xffffffffu, rescale)) {
                    const uint32_t at = tmem + KW_O + lanes + col;   // as many columns of the output
                    uint32_t r[KW_COLS];
                    tc::tmem_ld32(at, r);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < KW_COLS; c += 8) {
                        uint32_t w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(__uint_as_float(r[c + e]) * fac);
                        tc::tmem_st8(at + c, w);
                    }
                }
                const float off = ref == -INFINITY ? 0.f : -ref;
#pragma unroll
                for (int b = 0; b < KW_COLS / 16; ++b) {           // 16 tokens: 8 columns of each part
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int c = 0; c < 16; c += 4) {
                        float p[4];
                        float4 w4 = make_float4(1.f, 1.f, 1.f, 1.f);
                        if (PAR) w4 = *reinterpret_cast<const float4 *>(&sm.vs[buf][col + 16 * b + c]);
                        const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            p[e] = ka_exp2(z[16 * b + c + e] + off);
                            sum += p[e];
                            p[e] *= PAR ? w[e] : KA_UP;
                            if (PAR) p[e] *= e_inv;        // last: 0 for a token not seen, whatever its scale is
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const __half2 hh = __floats2half2_rn(p[2 * e], p[2 * e + 1]);
                            hi[c / 2 + e] = ka_u(hh);
                            if (PARTS == 2)
                                lo[c / 2 + e] = ka_u(__floats2half2_rn(p[2 * e] - __low2float(hh), p[2 * e + 1] - __high2float(hh)));
                        }
                    }
                    tc::tmem_st8(tmem + KW_P + lanes + col / 2 + 8 * b, hi);
                    if (PARTS == 2) tc::tmem_st8(tmem + KW_P + 64 + lanes + col / 2 + 8 * b, lo);
                }
                tc::tmem_wait_st();
            }
            if (i + 1 < n) {
                rv.store(sm.v[buf ^ 1]);
                store_scales(buf ^ 1);
                if (i + 2 < n) load_v(i + 2);
            }
            tc::fence_async_smem();
            tc::tc_fence_before();
            ok = __syncthreads_and(ok);
            if (!ok) break;
            if (tid == 0) {
                tc::tc_fence_after();
                if (i + 1 < n) issue_s(buf ^ 1);
                issue_o(buf, i == 0);
            }
        }
        if (!ok) break;
        if (n > 0) {
            ok = tc::mbar_wait(&sm.bar_o, n_o & 1u);
            ++n_o;
            tc::tc_fence_after();
        }
        // the row's sums, then its output
        sm.x[warp / 4][row] = sum;
        ok = __syncthreads_and(ok);
        if (!ok) break;
        float den = 0.f;
#pragma unroll
        for (int y = 0; y < KW_SPLIT; ++y) den += sm.x[y][row];
        const float inv = den != 0.f ? 1.f / den : 0.f, scale_o = (PAR ? e_max : 1.f) * (UP / KA_UP);
        // through shared memory (the tiles' place), so that a warp writes whole rows
        float(*const out)[D + 4] = reinterpret_cast<float(*)[D + 4]>(sm.k);
        static_assert(sizeof(float) * KW_ROWS * (D + 4) <= sizeof(sm.k) + sizeof(sm.v), "the output fits in the tiles' place");
        if (!idle) {
            uint32_t r[KW_COLS];
#pragma unroll
            for (int c = 0; c < KW_COLS; ++c) r[c] = 0u;
            if (n > 0) {
                tc::tmem_ld32(tmem + KW_O + lanes + col, r);
                tc::tmem_wait_ld();
            }
            float y[KW_COLS];
#pragma unroll
            for (int c = 0; c < KW_COLS; ++c)   // den == 0: nothing seen, and the sums may be another line's leftovers
                y[c / 8 * 8 + kw_order<DT>(c % 8)] = den != 0.f ? __uint_as_float(r[c]) * inv * scale_o : 0.f;
#pragma unroll
            for (int c = 0; c < KW_COLS; c += 4)
                *reinterpret_cast<float4 *>(&out[row][col + c]) = make_float4(y[c], y[c + 1], y[c + 2], y[c + 3]);
            if (warp < 4) {
                sm.ks[0][row] = ref;   // the scales are used up
                sm.sc[row] = den;
            }
        }
        __syncthreads();
        for (int r = warp; r < cl.rows; r += KW_WARPS) {
            const float4 y = *reinterpret_cast<const float4 *>(&out[r][4 * lane]);
            if (whole) ka_finish<T>(a, cl.row(a, l, h, r), lane, y, sm.ks[0][r], sm.sc[r]);
            else {
                *reinterpret_cast<float4 *>(a.part_o + (part * KW_ROWS + r) * D + 4 * lane) = y;
                if (lane == 0) a.part_ml[part * KW_ROWS + r] = make_float2(sm.ks[0][r], sm.sc[r]);
            }
        }
        if (!whole && s0 == 0 && tid == 0) a.split[blockIdx.x] = run.split();
        tc::tc_fence_before();
        __syncthreads();                                           // queries, tiles and O used before the next line
        tc::tc_fence_after();
        run.next(a, s1);
    }
    // the tensor memory goes back with no product in flight: every one that was issued has been waited for above, or its wait ran out
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 0) tc::tmem_dealloc(tmem, KW_TMEM);
}

}  // namespace milo

// kv_select.cuh -- retrieval by query: the blocks of the recent-token cache
// whose keys are estimated to score highest.
//
// For a query q and a block whose keys lie channelwise in [lo, hi],
// sum_j max(q_j lo_j, q_j hi_j) bounds q . k from above for every key of the
// block.  Both sides are rounded to the nearest INT8 code, which makes the sum an
// estimate: it may miss the bound by half a step of the query's codes and of the
// bounds' (milo.h has the slack).  In codes it is
//   sum_j min(c_j, 0) lo_j + max(c_j, 0) hi_j,
// one dot product of 256 8-bit values, exact in integers whatever the order,
// so that equal blocks tie and every run picks the same ones.
//
// Measured on 32 sessions of 30000 to 131072 tokens, 4 KV heads of 7 query heads,
// blocks of 64: 22.5 us for 42 MB (6.6 us at the copy rate), in one kernel or in two.
// A CTA is a chain of latencies: its length, its queries' coding, then steps of one
// batch of loads (two batches in flight cost registers, 25 us in all; equal runs of steps
// by the lengths begin more rows, 24 us), and for the selection 6 to 9 us of short rounds.
// Of the 11.7 cycles between a warp's instructions in the one kernel 3.5 are loads from memory,
// 1.8 fixed latencies and 1.6 barriers; issue 35 %, DRAM 21 %.
#pragma once
#include "kv_cache.cuh"

namespace milo {

// A kernel that follows another on its stream may be set up while that one
// still runs (programmatic dependent launch): the first says that it can be, the
// second waits for the first's end before it reads anything.
__device__ __forceinline__ void kv_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void kv_wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

struct KvSelectArgs {
    KvView c;
    const void *q;                 // [L][S][n_q][Hq][D]
    const int32_t *len;
    float *scores;                 // [L][S][n_q][H][n_b]
    int32_t *selected;             // [L][S][n_q][H][n_sel]
    int n_q, G, n_sel, n_first, n_last;
};

// tokens that query i of session s sees (0 and ST_BOUNDS for a bad length)
__device__ __forceinline__ int kv_seen(const int32_t *len, int s, int n_q, int i, int cap, bool tell) {
    int n = len[s];
    if (n < 0 || n > cap) {
        if (tell) raise_status(ST_BOUNDS);
        n = 0;
    }
    return max(0, n - n_q + i + 1);
}

constexpr int KV_SCORE_WARPS = 4, KV_SCORE_G = 8, KV_SCORE_STEP = 16 * KV_SCORE_WARPS;

__device__ __forceinline__ void kv_imma(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// grid (rows = L S n_q H, ceil(n_b / per)): a CTA scores `per` blocks of one row,
// 16 blocks a warp at a time as the rows of m16n8k32 products of 8-bit integers,
// the query heads its columns.  The sum's order is free: thread c of a row's four
// reads 16-byte chunks c, c + 4, c + 8, c + 12 of a block's 256 bytes, which are the
// operands of two steps each.  Bound by reading the codes once (260 B a block).
template <typename T, int WARPS> __device__ __forceinline__ void kv_score(const KvSelectArgs &a, int per) {
    constexpr int STEP = 16 * WARPS;
    __shared__ __align__(16) uint32_t s_q[KV_SCORE_G][2 * D / 4];
    __shared__ float s_u[KV_SCORE_G];
    const int64_t row = blockIdx.x;
    const int h = (int)(row % a.c.H);
    const int64_t lsi = row / a.c.H;
    const int i = (int)(lsi % a.n_q);
    const int s = (int)((lsi / a.n_q) % a.c.S), l = (int)(lsi / a.n_q / a.c.S);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int seen = kv_seen(a.len, s, a.n_q, i, a.c.cap, tid == 0 && h == 0 && l == 0 && i == 0 && blockIdx.y == 0);
    const int cand = (seen + a.c.block_len - 1) / a.c.block_len;
    const int b0 = blockIdx.y * per, b1 = min(a.c.n_b, b0 + per);
    float *out = a.scores + row * a.c.n_b;
    kv_launch_next();
    for (int b = max(b0, cand) + tid; b < b1; b += 32 * WARPS) out[b] = -INFINITY;
    if (b0 >= cand) return;
    const int end = min(b1, cand);
    const int64_t base = ((int64_t)s * a.c.H + h) * a.c.n_b;
    const unsigned char *codes = a.c.section(l, 5) + base * 2 * D + 16 * c;
    const float *scale = reinterpret_cast<const float *>(a.c.section(l, 6)) + base;
    uint4 w[2][4];                                  // rows g and g + 8 of the warp's 16 blocks
    auto load = [&](int b) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                w[r][x] = make_uint4(0u, 0u, 0u, 0u);
                if (b + g + 8 * r < end)
                    w[r][x] = __ldg(reinterpret_cast<const uint4 *>(codes + (int64_t)(b + g + 8 * r) * 2 * D + 64 * x));
            }
    };
    load(b0 + 16 * warp);
    for (int g0 = 0; g0 < a.G; g0 += KV_SCORE_G) {
        const int gn = min(KV_SCORE_G, a.G - g0);
        if (g0) {
            __syncthreads();                        // the heads before these are used
            load(b0 + 16 * warp);
        }
        for (int gg = warp; gg < KV_SCORE_G; gg += WARPS) {   // a head's codes; lane holds channels 4 lane ..
            uint32_t neg = 0u, pos = 0u;
            float u = 0.f;
            if (gg < gn) {
                const T *q = (const T *)a.q + ((lsi * a.c.H + h) * a.G + g0 + gg) * D + 4 * lane;
                float x[4], m = 0.f;
                bool bad = false;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = to_f32(q[e]);
                    if (!isfinite(x[e])) {
                        bad = true;
                        x[e] = 0.f;
                    }
                    m = fmaxf(m, fabsf(x[e]));
                }
                if (bad) raise_status(ST_NONFINITE);
                for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                u = __fdiv_rn(m, 127.f);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int v = u > 0.f ? (int)fminf(fmaxf(rintf(__fdiv_rn(x[e], u)), -127.f), 127.f) : 0;
                    neg |= (uint32_t)(min(v, 0) & 0xff) << (8 * e);
                    pos |= (uint32_t)(max(v, 0) & 0xff) << (8 * e);
                }
            }
            s_q[gg][lane] = neg;
            s_q[gg][32 + lane] = pos;
            if (lane == 0) s_u[gg] = u;
        }
        __syncthreads();
        uint4 f[4];                                 // this thread's column of the query heads' codes
#pragma unroll
        for (int x = 0; x < 4; ++x) f[x] = *reinterpret_cast<const uint4 *>(&s_q[g][4 * c + 16 * x]);
        const float u0 = s_u[2 * c], u1 = s_u[2 * c + 1];
        for (int b = b0 + 16 * warp; b < end; b += STEP) {
            int acc[4] = {0, 0, 0, 0};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                kv_imma(acc, w[0][x].x, w[1][x].x, w[0][x].y, w[1][x].y, f[x].x, f[x].y);
                kv_imma(acc, w[0][x].z, w[1][x].z, w[0][x].w, w[1][x].w, f[x].z, f[x].w);
            }
            load(b + STEP);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float v = 2 * c < gn ? __fmul_rn((float)acc[2 * r], u0) : -INFINITY;
                if (2 * c + 1 < gn) v = fmaxf(v, __fmul_rn((float)acc[2 * r + 1], u1));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                const int at = b + g + 8 * r;
                if (c == 0 && at < end) {
                    if (g0) v = fmaxf(v, out[at]);  // the heads before; the scale comes with the last ones
                    out[at] = g0 + KV_SCORE_G >= a.G ? __fmul_rn(v, __ldg(scale + at)) : v;
                }
            }
        }
    }
}
template <typename T> __global__ void __launch_bounds__(32 * KV_SCORE_WARPS) k_kv_score(KvSelectArgs a, int per) {
    kv_score<T, KV_SCORE_WARPS>(a, per);
}

// larger float = larger key, 1 at least and below 2^32 - 1 (only NaN would be either)
__device__ __forceinline__ uint32_t kv_key(float x) {
    if (x == 0.f) x = 0.f;   // -0 ties with +0
    const uint32_t b = __float_as_uint(x);
    return min(max(b & 0x80000000u ? ~b : b | 0x80000000u, 1u), 0xfffffffeu);
}

// One CTA per row.  The n_sel-th greatest key is found two bits at a time: a
// round counts the keys at or above three thresholds.  A thread keeps KEYS
// consecutive keys in registers, so that ids come out in order after one scan;
// HELD = false reads them from the scores again in every round (more blocks than
// THREADS * KEYS).
template <int THREADS, int KEYS, bool HELD> __device__ __forceinline__ void kv_topn(const KvSelectArgs &a) {
    constexpr int WARPS = THREADS / 32;
    __shared__ int s_n[2][WARPS][4];
    const int64_t row = blockIdx.x;
    const int64_t lsi = row / a.c.H;
    const int i = (int)(lsi % a.n_q), s = (int)((lsi / a.n_q) % a.c.S);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int seen = kv_seen(a.len, s, a.n_q, i, a.c.cap, false);
    const int cand = (seen + a.c.block_len - 1) / a.c.block_len;
    const float *sc = a.scores + row * a.c.n_b;
    int32_t *out = a.selected + row * a.n_sel;
    if (cand <= a.n_sel) {
        for (int e = tid; e < a.n_sel; e += THREADS) out[e] = e < cand ? e : -1;
        return;
    }
    const int last = cand - a.n_last, n_sel = a.n_sel - a.n_first - a.n_last;   // to be found beside the forced ones
    const int mine = HELD ? KEYS : (cand + THREADS - 1) / THREADS;   // ids tid * mine ..
    const int first = tid * mine;
    auto forced = [&](int b) { return b < a.n_first || (b >= last && b < cand); };
    auto key_of = [&](int b) { return b < cand && !forced(b) ? kv_key(sc[b]) : 0u; };
    uint32_t key[KEYS];
#pragma unroll
    for (int x = 0; x < KEYS; ++x) key[x] = HELD ? key_of(first + x) : 0u;
    // greatest threshold t with at least n_sel keys >= t (a key is 0 only where there is no candidate to be found): the
    // bits that all keys share come from their least and greatest
    uint32_t lo = 0xffffffffu, hi = 0u;
    auto range = [&](uint32_t k) {
        hi = max(hi, k);
        lo = min(lo, k - 1u);                        // 0 wraps: not a key
    };
    if (HELD) {
#pragma unroll
        for (int x = 0; x < KEYS; ++x) range(key[x]);
    } else {
        for (int b = tid; b < cand; b += THREADS) range(key_of(b));
    }
    hi = __reduce_max_sync(0xffffffffu, hi);
    lo = __reduce_min_sync(0xffffffffu, lo);
    if (lane == 0) *reinterpret_cast<uint2 *>(s_n[1][warp]) = make_uint2(lo, hi);
    __syncthreads();
    {
        const uint2 v = *reinterpret_cast<const uint2 *>(s_n[1][lane % WARPS]);
        lo = __reduce_min_sync(0xffffffffu, v.x) + 1u;
        hi = __reduce_max_sync(0xffffffffu, v.y);
    }
    const uint32_t differ = lo ^ hi;
    int shift = differ ? (31 - __clz(differ)) & ~1 : -2;
    uint32_t t = n_sel == 0 ? 0xffffffffu : shift >= 30 ? 0u : hi & ~((4u << max(shift, 0)) - 1u);
    if (differ == 0u) t = n_sel == 0 ? 0xffffffffu : hi;
    if (n_sel == 0) shift = -2;
    // the first round uses the other buffer than the range did
    for (int round = 0; shift >= 0; shift -= 2, ++round) {
        const uint32_t t1 = t | (1u << shift), t2 = t | (2u << shift), t3 = t | (3u << shift);
        int n1 = 0, n2 = 0, n3 = 0;
        auto count = [&](uint32_t k) {
            n1 += k >= t1;
            n2 += k >= t2;
            n3 += k >= t3;
        };
        if (HELD) {
#pragma unroll
            for (int x = 0; x < KEYS; ++x) count(key[x]);
        } else {
            for (int b = tid; b < cand; b += THREADS) count(key_of(b));
        }
        n1 = __reduce_add_sync(0xffffffffu, n1);
        n2 = __reduce_add_sync(0xffffffffu, n2);
        n3 = __reduce_add_sync(0xffffffffu, n3);
        const int buf = round & 1;                   // two buffers: one barrier a round
        if (lane == 0) *reinterpret_cast<int4 *>(s_n[buf][warp]) = make_int4(n1, n2, n3, 0);
        __syncthreads();
        const int4 v = *reinterpret_cast<const int4 *>(s_n[buf][lane % WARPS]);   // each warp adds the warps' counts
        const bool own = lane < WARPS;
        n1 = __reduce_add_sync(0xffffffffu, own ? v.x : 0);
        n2 = __reduce_add_sync(0xffffffffu, own ? v.y : 0);
        n3 = __reduce_add_sync(0xffffffffu, own ? v.z : 0);
        const int n = n3 >= n_sel ? n3 : n2 >= n_sel ? n2 : n1;
        t = n3 >= n_sel ? t3 : n2 >= n_sel ? t2 : n1 >= n_sel ? t1 : t;
        if (n == n_sel) {                            // exactly the keys >= t: all above t - 1
            --t;
            break;
        }
    }
    // keys above t are all taken, and the first of those equal to it
    int gt = 0, eq = 0;
    auto tally = [&](uint32_t k, int b) {
        gt += k > t || forced(b);
        eq += k == t && k != 0u;
    };
    if (HELD) {
#pragma unroll
        for (int x = 0; x < KEYS; ++x) tally(key[x], first + x);
    } else {
        for (int x = 0; x < mine; ++x) tally(key_of(first + x), first + x);
    }
    int ig = gt, ie = eq;                            // inclusive over the threads
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, ig, o), y = __shfl_up_sync(0xffffffffu, ie, o);
        if (lane >= o) {
            ig += x;
            ie += y;
        }
    }
    __syncthreads();
    if (lane == 31) *reinterpret_cast<int2 *>(s_n[0][warp]) = make_int2(ig, ie);
    __syncthreads();
    int all = 0;
    ig -= gt;
    ie -= eq;
    for (int w = 0; w < WARPS; ++w) {
        const int2 v = *reinterpret_cast<const int2 *>(s_n[0][w]);
        if (w < warp) {
            ig += v.x;
            ie += v.y;
        }
        all += v.x;
    }
    const int want = a.n_sel - all;                  // how many of the equal ones
    auto put = [&](uint32_t k, int b) {
        const bool g = k > t || forced(b), e = k == t && k != 0u;
        if (g) out[ig + min(ie, want)] = b;
        else if (e && ie < want) out[ig + ie] = b;
        ig += g;
        ie += e;
    };
    if (HELD) {
#pragma unroll
        for (int x = 0; x < KEYS; ++x) put(key[x], first + x);
    } else {
        for (int x = 0; x < mine; ++x) put(key_of(first + x), first + x);
    }
}

template <int THREADS, int KEYS, bool HELD> __global__ void __launch_bounds__(THREADS) k_kv_topn(KvSelectArgs a) {
    kv_wait_previous();
    kv_topn<THREADS, KEYS, HELD>(a);
}

// Both in one CTA per row, for few blocks: the scores are the CTA's own
constexpr int KV_ROW_THREADS = 512, KV_ROW_KEYS = 4;
template <typename T> __global__ void __launch_bounds__(KV_ROW_THREADS) k_kv_select_row(KvSelectArgs a) {
    kv_score<T, KV_ROW_THREADS / 32>(a, a.c.n_b);
    __syncthreads();
    kv_topn<KV_ROW_THREADS, KV_ROW_KEYS, true>(a);
}

}  // namespace milo

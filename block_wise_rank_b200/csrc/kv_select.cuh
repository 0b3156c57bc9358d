// kv_select.cuh -- retrieval by query: the blocks of the recent-token cache
// whose keys can score highest.
//
// For a query c (INT8 codes) and a block whose keys lie channelwise in
// [lo, hi], sum_j max(c_j lo_j, c_j hi_j) bounds c . k from above for every
// key of the block.  With both sides in INT8 the sum is
//   sum_j min(c_j, 0) lo_j + max(c_j, 0) hi_j,
// one dot product of 256 8-bit values, exact in integers whatever the order,
// so that equal blocks tie and every run picks the same ones.
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

constexpr int KV_SCORE_THREADS = 128, KV_SCORE_G = 8;

// grid (rows = L S n_q H, ceil(n_b / 128)): thread = block
template <typename T> __global__ void __launch_bounds__(KV_SCORE_THREADS) k_kv_score(KvSelectArgs a) {
    __shared__ __align__(16) uint32_t s_q[KV_SCORE_G][2 * D / 4];
    __shared__ float s_u[KV_SCORE_G];
    const int64_t row = blockIdx.x;
    const int h = (int)(row % a.c.H);
    const int64_t lsi = row / a.c.H;
    const int i = (int)(lsi % a.n_q);
    const int s = (int)((lsi / a.n_q) % a.c.S), l = (int)(lsi / a.n_q / a.c.S);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int seen = kv_seen(a.len, s, a.n_q, i, a.c.cap, tid == 0 && h == 0 && l == 0 && i == 0 && blockIdx.y == 0);
    const int cand = (seen + a.c.block_len - 1) / a.c.block_len;
    const int b = blockIdx.y * KV_SCORE_THREADS + tid;
    float best = -INFINITY;
    kv_launch_next();
    for (int g0 = 0; g0 < a.G; g0 += KV_SCORE_G) {
        const int gn = min(KV_SCORE_G, a.G - g0);
        __syncthreads();
        for (int g = warp; g < gn; g += KV_SCORE_THREADS / 32) {   // lane holds channels 4 lane ..
            const T *q = (const T *)a.q + ((lsi * a.c.H + h) * a.G + g0 + g) * D + 4 * lane;
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
            const float u = __fdiv_rn(m, 127.f);
            uint32_t neg = 0u, pos = 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = u > 0.f ? (int)fminf(fmaxf(rintf(__fdiv_rn(x[e], u)), -127.f), 127.f) : 0;
                neg |= (uint32_t)(min(c, 0) & 0xff) << (8 * e);
                pos |= (uint32_t)(max(c, 0) & 0xff) << (8 * e);
            }
            s_q[g][lane] = neg;
            s_q[g][32 + lane] = pos;
            if (lane == 0) s_u[g] = u;
        }
        __syncthreads();
        if (b < cand) {
            const int64_t blk = ((int64_t)s * a.c.H + h) * a.c.n_b + b;
            const uint4 *code = reinterpret_cast<const uint4 *>(a.c.section(l, 5) + blk * 2 * D);
            int acc[KV_SCORE_G];
#pragma unroll
            for (int g = 0; g < KV_SCORE_G; ++g) acc[g] = 0;
            for (int w = 0; w < 2 * D / 16; ++w) {
                const uint4 u = __ldg(code + w);
#pragma unroll
                for (int g = 0; g < KV_SCORE_G; ++g) {
                    if (g >= gn) break;
                    const uint4 c = reinterpret_cast<const uint4 *>(s_q[g])[w];
                    acc[g] = __dp4a((int)u.x, (int)c.x, acc[g]);
                    acc[g] = __dp4a((int)u.y, (int)c.y, acc[g]);
                    acc[g] = __dp4a((int)u.z, (int)c.z, acc[g]);
                    acc[g] = __dp4a((int)u.w, (int)c.w, acc[g]);
                }
            }
#pragma unroll
            for (int g = 0; g < KV_SCORE_G; ++g)
                if (g < gn) best = fmaxf(best, __fmul_rn((float)acc[g], s_u[g]));
            if (g0 + KV_SCORE_G >= a.G) best = __fmul_rn(best, __ldg((const float *)a.c.section(l, 6) + blk));
        }
    }
    if (b < a.c.n_b) a.scores[row * a.c.n_b + b] = best;
}

// larger float = larger key; forced candidates above all
__device__ __forceinline__ uint32_t kv_key(float x, bool forced) {
    if (forced) return 0xffffffffu;
    if (x == 0.f) x = 0.f;   // -0 ties with +0
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

constexpr int KV_TOPN_THREADS = 256;

// one CTA per row: the n_sel-th greatest key by four 8-bit histogram passes,
// then the ids above it and the first of those equal to it, in order
__global__ void __launch_bounds__(KV_TOPN_THREADS) k_kv_topn(KvSelectArgs a) {
    __shared__ int s_hist[256], s_gt[KV_TOPN_THREADS / 32], s_eq[KV_TOPN_THREADS / 32], s_bin, s_above;
    kv_wait_previous();
    const int64_t row = blockIdx.x;
    const int64_t lsi = row / a.c.H;
    const int i = (int)(lsi % a.n_q), s = (int)((lsi / a.n_q) % a.c.S);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int seen = kv_seen(a.len, s, a.n_q, i, a.c.cap, false);
    const int cand = (seen + a.c.block_len - 1) / a.c.block_len;
    const float *sc = a.scores + row * a.c.n_b;
    int32_t *out = a.selected + row * a.n_sel;
    if (cand <= a.n_sel) {
        for (int e = tid; e < a.n_sel; e += KV_TOPN_THREADS) out[e] = e < cand ? e : -1;
        return;
    }
    const int last = cand - a.n_last;
    uint32_t prefix = 0u, mask = 0u;
    int want = a.n_sel;                     // how many of the keys that match the prefix are taken
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int e = tid; e < 256; e += KV_TOPN_THREADS) s_hist[e] = 0;
        __syncthreads();
        for (int b = tid; b < cand; b += KV_TOPN_THREADS) {
            const uint32_t k = kv_key(sc[b], b < a.n_first || b >= last);
            if ((k & mask) == prefix) atomicAdd(&s_hist[(k >> shift) & 255u], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int above = 0, bin = 255;
            while (above + s_hist[bin] < want) above += s_hist[bin--];
            s_bin = bin;
            s_above = above;
        }
        __syncthreads();
        prefix |= (uint32_t)s_bin << shift;
        mask |= 255u << shift;
        want -= s_above;
        __syncthreads();
    }
    int gt0 = 0, eq0 = 0;                   // ids above / equal before this round of blocks
    for (int b0 = 0; b0 < cand; b0 += KV_TOPN_THREADS) {
        const int b = b0 + tid;
        const uint32_t k = b < cand ? kv_key(sc[b], b < a.n_first || b >= last) : 0u;
        const bool gt = b < cand && k > prefix, eq = b < cand && k == prefix;
        const unsigned mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) {
            s_gt[warp] = __popc(mg);
            s_eq[warp] = __popc(me);
        }
        __syncthreads();
        int g = gt0, e = eq0;
        for (int w = 0; w < KV_TOPN_THREADS / 32; ++w) {
            if (w < warp) {
                g += s_gt[w];
                e += s_eq[w];
            }
            gt0 += s_gt[w];
            eq0 += s_eq[w];
        }
        const unsigned below = (1u << lane) - 1u;
        g += __popc(mg & below);
        e += __popc(me & below);
        if (gt || (eq && e < want)) out[g + min(e, want)] = b;
        __syncthreads();
    }
}

}  // namespace milo

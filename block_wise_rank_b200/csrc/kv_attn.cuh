// kv_attn.cuh -- attention over the quantised cache of recent tokens.
//
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q . k_t - m)
//
// over the tokens that a query sees, all of them or those of the blocks it
// selected, with the running maximum m and sum in fp32.
#pragma once
#include "kv_select.cuh"

namespace milo {

struct KvAttnArgs {
    KvView c;
    const void *q;                 // [L][S][n_q][Hq][D]
    void *out;                     // like q
    float *lse;                    // [L][S][n_q][Hq] or null
    float2 *ml;                    // [L][S][n_q][Hq] (max, sum) or null
    const int32_t *len;
    const int32_t *sel;            // [L][S][n_q][H][n_sel] or null
    int n_q, G, n_sel;
    float scale;
};

// one warp per query row; lane holds channels 16 (lane % 8) .. of the tokens
// t = lane / 8 modulo 4
template <typename T, int DT> __global__ void __launch_bounds__(128) k_kv_attn_rows(KvAttnArgs a) {
    const int64_t Hq = (int64_t)a.c.H * a.G, rows = (int64_t)a.c.L * a.c.S * a.n_q * Hq;
    const int64_t r = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
    if (r >= rows) return;
    const int lane = threadIdx.x & 31, j = lane & 7, tq = lane >> 3;
    const int hq = (int)(r % Hq), h = hq / a.G;
    const int64_t lsi = r / Hq;
    const int i = (int)(lsi % a.n_q), s = (int)((lsi / a.n_q) % a.c.S), l = (int)(lsi / a.n_q / a.c.S);
    const int seen = kv_seen(a.len, s, a.n_q, i, a.c.cap, lane == 0 && hq == 0 && l == 0 && i == 0);
    const int64_t sh = (int64_t)s * a.c.H + h;
    const unsigned char *kc = a.c.codes(l, sh, 0), *vc = a.c.codes(l, sh, 1);
    const unsigned char *kp = a.c.params(l, sh, 0), *vp = a.c.params(l, sh, 1);
    const int rb = a.c.row_bytes(), pb = a.c.par_bytes();
    float q[16], o[16], m = -INFINITY, sum = 0.f;
    kv_load16<T>((const T *)a.q + r * D + 16 * j, q);
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = 0.f;
    const int parts = a.sel ? a.n_sel : 1;
    for (int u = 0; u < parts; ++u) {
        int t0 = 0, t1 = seen;
        if (a.sel) {
            const int b = a.sel[(lsi * a.c.H + h) * a.n_sel + u];
            if (b < 0 || b >= a.c.n_b) {
                if (b != -1) raise_status(ST_BOUNDS);
                continue;
            }
            t0 = b * a.c.block_len;
            t1 = min(seen, t0 + a.c.block_len);
        }
        for (int t4 = t0; t4 < t1; t4 += 4) {
            const int64_t t = t4 + tq;
            const bool ok = t < t1;
            float x = 0.f, v[16];
            if (ok) {
                kv_dequant16<DT>(kc + t * rb, kp + t * pb, j, v);
#pragma unroll
                for (int e = 0; e < 16; ++e) x = fmaf(q[e], v[e], x);
            }
            for (int w = 1; w < 8; w <<= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
            x = ok ? x * a.scale : -INFINITY;
            float mx = fmaxf(m, x);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float f = m == -INFINITY ? 0.f : expf(m - mx), p = expf(x - mx);
            m = mx;
            sum = sum * f + p;
            if (ok) kv_dequant16<DT>(vc + t * rb, vp + t * pb, j, v);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = ok ? fmaf(p, v[e], o[e] * f) : o[e] * f;
        }
    }
#pragma unroll
    for (int w = 8; w < 32; w <<= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, w);
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] += __shfl_xor_sync(0xffffffffu, o[e], w);
    }
    if (tq == 0) {
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = sum != 0.f ? o[e] / sum : 0.f;
        kv_store16<T>((T *)a.out + r * D + 16 * j, o);
        if (j == 0 && a.lse) a.lse[r] = sum != 0.f ? m + logf(sum) : -INFINITY;
        if (j == 0 && a.ml) a.ml[r] = make_float2(m, sum);
    }
}

}  // namespace milo

// kv_api.cuh -- C entry points of the rotary positions and of the quantised
// cache of recent tokens (milo.h): argument checks and launches.  Included by
// milo.cu, whose helpers it uses.
#pragma once

namespace {

bool float_dtype(milo_dtype t) { return t == MILO_F32 || t == MILO_BF16; }

// ------------------------------------------------------------------ rotary

milo_status rope_check(const milo_rope_params *p, int *rd) {
    if (!p || p->d < 2 || p->d % 2 || p->rotary_dim < 0 || p->rotary_dim % 2 || p->rotary_dim > p->d)
        return MILO_ERR_INVALID_ARG;
    if (p->d > MILO_ROPE_MAX_D) return MILO_ERR_UNSUPPORTED;
    *rd = p->rotary_dim ? p->rotary_dim : p->d;
    if (!(p->base > 1.0) || !std::isfinite(p->base) || !std::isfinite(p->attn_factor) || p->attn_factor < 0.0)
        return MILO_ERR_INVALID_ARG;
    if (p->scaling < MILO_ROPE_NONE || p->scaling > MILO_ROPE_BANDS) return MILO_ERR_INVALID_ARG;
    if (p->scaling != MILO_ROPE_NONE && (!(p->factor > 0.0) || !std::isfinite(p->factor)))
        return MILO_ERR_INVALID_ARG;
    if (p->scaling == MILO_ROPE_NTK && *rd <= 2) return MILO_ERR_INVALID_ARG;
    if (p->scaling >= MILO_ROPE_YARN && (!(p->orig_ctx > 0.0) || !std::isfinite(p->orig_ctx)))
        return MILO_ERR_INVALID_ARG;
    if (p->scaling == MILO_ROPE_YARN && !(p->beta_slow > 0.0 && p->beta_fast >= p->beta_slow &&
                                          std::isfinite(p->beta_fast)))
        return MILO_ERR_INVALID_ARG;
    if (p->scaling == MILO_ROPE_BANDS && !(p->high_freq > p->low_freq && std::isfinite(p->low_freq) &&
                                           std::isfinite(p->high_freq)))
        return MILO_ERR_INVALID_ARG;
    return MILO_OK;
}

constexpr double kTwoPi = 6.283185307179586476925286766559;

double clamp01(double x) { return x < 0.0 ? 0.0 : (x > 1.0 ? 1.0 : x); }

// w_i and the factor on the turned channels (milo.h, milo_rope_scaling)
void rope_freqs(const milo_rope_params *p, int rd, double *w, double *m) {
    const double base = p->scaling == MILO_ROPE_NTK ? p->base * std::pow(p->factor, (double)rd / (rd - 2)) : p->base;
    double lo = 0.0, span = 1.0;
    if (p->scaling == MILO_ROPE_YARN) {
        auto channel = [&](double turns) { return rd * std::log(p->orig_ctx / (turns * kTwoPi)) / (2.0 * std::log(base)); };
        lo = std::max(std::floor(channel(p->beta_fast)), 0.0);
        const double hi = std::min(std::ceil(channel(p->beta_slow)), (double)rd - 1.0);
        span = hi > lo ? hi - lo : 0.001;
    }
    for (int i = 0; i < rd / 2; ++i) {
        const double t = std::pow(base, -2.0 * i / rd);
        switch (p->scaling) {
        case MILO_ROPE_LINEAR: w[i] = t / p->factor; break;
        case MILO_ROPE_YARN: {
            const double g = clamp01((i - lo) / span);
            w[i] = t / p->factor * g + t * (1.0 - g);
            break;
        }
        case MILO_ROPE_BANDS: {
            const double u = clamp01((p->orig_ctx * t / kTwoPi - p->low_freq) / (p->high_freq - p->low_freq));
            w[i] = (1.0 - u) * t / p->factor + u * t;
            break;
        }
        default: w[i] = t;
        }
    }
    // YaRN (Peng et al., 2023): 0.1 ln(factor) + 1 for a longer context, 1 for one that is not
    const double own = p->scaling == MILO_ROPE_YARN && p->factor > 1.0 ? 0.1 * std::log(p->factor) + 1.0 : 1.0;
    *m = p->attn_factor > 0.0 ? p->attn_factor : own;
}

// [lo, hi) bytes that n_tokens x n_heads rows of d elements cover
void rope_extent(const void *p, int64_t ts, int64_t hs, int64_t nt, int64_t nh, int d, int es, uintptr_t &lo,
                 uintptr_t &hi) {
    lo = (uintptr_t)p;
    hi = lo + (uintptr_t)(((nt - 1) * ts + (nh - 1) * hs + d) * es);
}

// ------------------------------------------------------------------- cache

bool kv_ok(const milo_kv_shape *s) {
    return s && s->L > 0 && s->S > 0 && s->H > 0 && s->cap > 0 && s->cap <= (1 << 26) && s->block_len >= 16 &&
           s->block_len <= 1024 && s->block_len % 16 == 0 &&
           (s->dtype == MILO_INT8 || s->dtype == MILO_FP8 || s->dtype == MILO_INT4) &&
           (int64_t)s->S * s->H <= INT32_MAX && (int64_t)s->L * s->S * s->H <= INT32_MAX &&
           (double)s->L * s->S * s->H * s->cap < 4e15;   // at most 600 bytes a row: sizes stay inside 64 bits
}

milo_status kv_check(const milo_kv_shape *s, const void *cache, size_t bytes) {
    if (!kv_ok(s) || !cache || !aligned(cache, kAlign)) return MILO_ERR_INVALID_ARG;
    if (s->d != D) return MILO_ERR_UNSUPPORTED;
    return bytes < milo_kv_cache_size(s) ? MILO_ERR_WORKSPACE : MILO_OK;
}

KvView kv_view(const milo_kv_shape *s, const void *cache) {
    KvView v{};
    v.base = (unsigned char *)const_cast<void *>(cache);
    v.L = s->L; v.S = s->S; v.H = s->H; v.cap = s->cap; v.block_len = s->block_len;
    v.n_b = (s->cap + s->block_len - 1) / s->block_len;
    v.dtype = s->dtype;
    const int64_t sh = (int64_t)s->S * s->H, rows = sh * s->cap, blocks = sh * v.n_b;
    const int64_t size[7] = {rows * v.row_bytes(), rows * v.row_bytes(), rows * v.par_bytes(), rows * v.par_bytes(),
                             blocks * 2 * D * 2, blocks * 2 * D, blocks * 4};
    int64_t at = 0;
    for (int i = 0; i < 7; ++i) {
        v.off[i] = at;
        at = (int64_t)align_up((size_t)(at + size[i]));
    }
    v.layer = at;
    return v;
}

// query rows within 31 bits (the product of four counts can pass 64)
bool kv_rows_fit(const milo_kv_shape *s, int32_t n_q, int32_t heads) {
    return (double)s->L * s->S * n_q * heads <= INT32_MAX;
}

// the candidates, queries and heads of a select or attention call
milo_status kv_query_check(const milo_kv_shape *s, const void *q, milo_dtype q_dtype, int32_t n_q, int32_t Hq,
                           const int32_t *len) {
    if (!q || !len || n_q <= 0 || Hq <= 0 || Hq % s->H || !aligned(q, 16) || !aligned(len, 4))
        return MILO_ERR_INVALID_ARG;
    if (!float_dtype(q_dtype)) return MILO_ERR_UNSUPPORTED;
    return kv_rows_fit(s, n_q, Hq) ? MILO_OK : MILO_ERR_UNSUPPORTED;
}

// grid size for `ctas` thread blocks in x, 0 if there are too many (2^30, so that four items a block still count in 32 bits)
unsigned grid_x(int64_t ctas) { return ctas > (1 << 30) ? 0u : (unsigned)ctas; }

template <typename T, int DT> void kv_append_run(const KvAppendArgs &a, cudaStream_t s) {
    // a warp to an item where a step takes all its tokens, or where the items fill the GPU (16 warps an SM) twice over:
    // what an item costs beside its rows is then paid once a warp, not by four
    if (a.n_new <= 4 || a.items >= 32 * sm_count())
        k_kv_append<T, DT, 1><<<(a.items + KV_APPEND_WARPS - 1) / KV_APPEND_WARPS, 32 * KV_APPEND_WARPS, 0, s>>>(a);
    else
        k_kv_append<T, DT, KV_APPEND_WARPS><<<a.items, 32 * KV_APPEND_WARPS, 0, s>>>(a);
}

template <typename T> void kv_append_launch(const KvAppendArgs &a, cudaStream_t s) {
    if (a.c.dtype == MILO_INT8) kv_append_run<T, MILO_INT8>(a, s);
    else if (a.c.dtype == MILO_FP8) kv_append_run<T, MILO_FP8>(a, s);
    else kv_append_run<T, MILO_INT4>(a, s);
}

template <typename T> void kv_read_launch(const KvReadArgs &a, dim3 grid, cudaStream_t s) {
    if (a.c.dtype == MILO_INT8) k_kv_read<T, MILO_INT8><<<grid, 256, 0, s>>>(a);
    else if (a.c.dtype == MILO_FP8) k_kv_read<T, MILO_FP8><<<grid, 256, 0, s>>>(a);
    else k_kv_read<T, MILO_INT4><<<grid, 256, 0, s>>>(a);
}

// Query rows of a line and the launch shape of an attention call.
struct KvAttnPlan {
    int nt, row_tiles, grid, classes;
    bool whole;
    size_t part_o, part_ml, split, bytes;    // workspace offsets
};

KvAttnPlan kv_attn_plan(const milo_kv_shape *s, int32_t n_q, int32_t Hq, int32_t n_sel) {
    KvAttnPlan p{};
    const int64_t G = Hq / s->H, rows = n_sel ? G : G * n_q;
    // up to 8 rows: two CTAs an SM, bound by memory; up to 16, and selected blocks, whose lines have few rows: two tiles
    // of 8 a warp; above, 128 rows share a pass.  In tiles of 16 rows and wide, in a graph, codes not in L2 (us): 17 queries
    // of 7 heads over e4m3 102 and 52; 16 lines of 30000 INT8 tokens, bf16, of 119 rows 177 and 99, 63 rows 101 and 94,
    // 49 rows 101 and 94, 35 rows 82 and 94, 21 rows 65 and 93 (fp32 235 and 115, 130 and 110, 129 and 110, 104 and 109, 79
    // and 105); e4m3 at 35 rows 102 and 99, INT4 84 and 80; of 2000 tokens 20 to 29 either way up to 63 rows.  Two tiles (17
    // to 32 rows) over long lines would take less than the wide pass that they get
    p.nt = rows <= 8 ? 1 : rows <= 16 || n_sel ? 2 : 16;
    const int rpt = 8 * p.nt;
    p.row_tiles = (int)((rows + rpt - 1) / rpt);
    p.classes = (int)((int64_t)s->S * (n_sel ? n_q : 1) * p.row_tiles);   // at most the query rows
    // units at most: a CTA with none would have nothing to do
    const int warps = p.nt == 1 ? KaShape<1>::WARPS : p.nt == 2 ? KaShape<2>::WARPS : KaShape<16>::WARPS;
    const int begin = p.nt == 1 ? KaShape<1>::BEGIN : p.nt == 2 ? KaShape<2>::BEGIN : KaShape<16>::BEGIN;
    const int ctas = p.nt == 1 ? KaShape<1>::CTAS : p.nt == 2 ? KaShape<2>::CTAS : KaShape<16>::CTAS;
    const int64_t tiles = n_sel ? (int64_t)n_sel * (s->block_len / 16) : ((int64_t)s->cap + 15) / 16;
    const int64_t lines = (int64_t)p.classes * s->L * s->H, behind = (tiles + warps - 1) / warps;
    const int most = p.nt == 1 ? KaShape<1>::WHOLE : p.nt == 2 ? KaShape<2>::WHOLE : KaShape<16>::WHOLE;
    // short lines, no more than a wave holds: a CTA for each, one launch and nothing to merge; twice as long ones where
    // they fill a quarter of the wave.  The lengths are on the device, so the limits go by capacity, and lie where lines
    // that fill up take no more time on average (1/6, 1/2 and 5/6 full), whole less split in us, in a graph, codes not in L2:
    //   up to 8 rows a line (limit 8 units, 1024 tokens), 1, 4 and 16 lines
    //     capacity 1024: INT8 bf16 7 heads -1.4 -1.6 -2.3, fp32 8 heads -0.6 -1.0 -1.8, e4m3 fp32 4 heads 0.0 -0.2 -0.7
    //     capacity 1536: -0.5 -0.8 -1.9, +0.5 +0.3 -1.2, +1.9 +2.0 +0.2
    //     full lines of 1024: 0.0 0.0 -1.0, +2.1 +1.4 0.0, +3.8 +3.4 +2.1; of 512: -1.4 -1.7 -2.1, -1.0 -1.4 -1.4, 0.0 -0.3 -0.3
    //   up to 16 rows (8 units, 512 tokens), 12 bf16 heads, 1, 4 and 16 lines: 512 -1.8 -3.0 -3.5, 1024 +1.1 +0.1 -5.5
    //   128 rows (1 unit, 128 tokens), 17 fp32 queries of 7 heads, full: 128 -2.1 to -3.7, 256 +1.7 +1.0 +0.3 (1, 4, 16 lines)
    // and for a quarter of the wave and more, full lines, whole and split: 74 lines of 2048 18.1 and 22.9, 148 20.5 and
    // 28.7, 256 30.4 and 36.9, but one of 2048 among lines of 100 tokens 17.1 and 15.7, 17.4 and 16.0, 18.4 and 16.0; 32
    // lines of 2048 17.4 and 18.8; 74 of 4096 29.4 and 28.7, 200 50.2 and 48.8
    const int wave = ctas * sm_count();
    p.whole = lines <= wave && behind <= (4 * lines >= wave ? 2 * most : most);
    p.grid = (int)(p.whole ? lines : std::min<int64_t>(lines * (begin + behind), wave));
    p.part_o = 0;
    p.part_ml = align_up(sizeof(float) * 2 * (size_t)p.grid * rpt * D);
    p.split = p.part_ml + align_up(sizeof(float2) * 2 * (size_t)p.grid * rpt);
    p.bytes = p.split + align_up(sizeof(int4) * (size_t)p.grid);
    return p;
}

// Launch of a kernel that waits for its predecessor itself (kv_wait_previous).
template <typename A> cudaError_t kv_follow(void (*kernel)(A), dim3 grid, int threads, const A &a, cudaStream_t s) {
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3((unsigned)threads);
    c.stream = s;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, a);
}

// opt-in shared memory of a kernel, once per device
template <typename K> cudaError_t kv_smem(K kernel, size_t bytes, bool (&done)[64]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && done[dev])) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && dev < 64) done[dev] = true;
    return e;
}

template <typename T, int NT, bool SEL> cudaError_t kv_attn_merge(const KvAttnArgs &a, int grid, cudaStream_t s) {
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || a.whole) return e;
    // many parts a line: a CTA per row, else one for 16 rows at most
    const int64_t lines = (int64_t)a.classes * a.c.L * a.c.H;
    const int rows = grid >= 16 * lines ? 8 * NT : (8 * NT + 15) / 16;
    return kv_follow(k_kv_attn_merge<T, NT, SEL>, dim3(grid, rows), 32 * KA_MERGE_WARPS, a, s);
}

template <typename T, int DT, int NT, bool SEL, bool OWN>
cudaError_t kv_attn_run_as(const KvAttnArgs &a, int grid, cudaStream_t s) {
    static bool done[64];
    const size_t smem = sizeof(KaSmem<T, DT, NT>);
    const cudaError_t e = kv_smem(k_kv_attn<T, DT, NT, SEL, OWN>, smem, done);
    if (e != cudaSuccess) return e;
    k_kv_attn<T, DT, NT, SEL, OWN><<<grid, 32 * KaShape<NT>::WARPS, smem, s>>>(a);
    return kv_attn_merge<T, NT, SEL>(a, grid, s);
}

template <typename T, int DT, int NT, bool SEL> cudaError_t kv_attn_run(const KvAttnArgs &a, int grid, cudaStream_t s) {
    // rows of a line that see different tokens: the queries of a session, where they are not lines of their own
    if constexpr (!SEL && DT != MILO_INT4)
        if (a.n_q > 1) return kv_attn_run_as<T, DT, NT, SEL, true>(a, grid, s);
    return kv_attn_run_as<T, DT, NT, SEL, false>(a, grid, s);
}

template <typename T, int DT> cudaError_t kv_attn_run_wide(const KvAttnArgs &a, int grid, cudaStream_t s) {
    static bool done[64];
    const size_t smem = sizeof(KwSmem<T>);
    const cudaError_t e = kv_smem(k_kv_attn_wide<T, DT>, smem, done);
    if (e != cudaSuccess) return e;
    k_kv_attn_wide<T, DT><<<grid, KW_THREADS, smem, s>>>(a);
    return kv_attn_merge<T, 16, false>(a, grid, s);
}

template <typename T, int DT> cudaError_t kv_attn_rows(const KvAttnArgs &a, int nt, int grid, cudaStream_t s) {
    if (nt == 16) return kv_attn_run_wide<T, DT>(a, grid, s);
    if (a.sel) return nt == 1 ? kv_attn_run<T, DT, 1, true>(a, grid, s) : kv_attn_run<T, DT, 2, true>(a, grid, s);
    return nt == 1 ? kv_attn_run<T, DT, 1, false>(a, grid, s) : kv_attn_run<T, DT, 2, false>(a, grid, s);
}

template <typename T> cudaError_t kv_attn_type(const KvAttnArgs &a, int nt, int grid, cudaStream_t s) {
    if (a.c.dtype == MILO_INT8) return kv_attn_rows<T, MILO_INT8>(a, nt, grid, s);
    if (a.c.dtype == MILO_FP8) return kv_attn_rows<T, MILO_FP8>(a, nt, grid, s);
    return kv_attn_rows<T, MILO_INT4>(a, nt, grid, s);
}

milo_status kv_attn_launch(const milo_kv_shape *shape, const void *cache, const void *q, milo_dtype q_dtype,
                           int32_t n_q, int32_t Hq, const int32_t *len, const int32_t *selected, int32_t n_sel,
                           double scale, void *out, float *lse, float2 *ml, void *workspace, cudaStream_t s) {
    const KvAttnPlan p = kv_attn_plan(shape, n_q, Hq, n_sel);
    KvAttnArgs a{};
    a.c = kv_view(shape, cache);
    a.q = q; a.out = out; a.lse = lse; a.ml = ml; a.len = len; a.sel = selected;
    a.n_q = n_q; a.G = Hq / shape->H; a.n_sel = n_sel;
    a.tpb = shape->block_len / 16;
    a.row_tiles = p.row_tiles; a.classes = p.classes; a.whole = p.whole;
    a.scale = (float)((scale > 0.0 ? scale : 1.0 / std::sqrt((double)D)) * 1.4426950408889634074);
    a.part_o = (float *)((char *)workspace + p.part_o);
    a.part_ml = (float2 *)((char *)workspace + p.part_ml);
    a.split = (int4 *)((char *)workspace + p.split);
    return cuda_check(q_dtype == MILO_BF16 ? kv_attn_type<__nv_bfloat16>(a, p.nt, p.grid, s)
                                           : kv_attn_type<float>(a, p.nt, p.grid, s), "kv attention launch");
}

// tokens of a selection: at most 2^30
bool kv_tokens_fit(const milo_kv_shape *s, int32_t n_sel) {
    return (int64_t)n_sel * s->block_len <= (int64_t(1) << 30);
}

// selection of a call: NULL and 0, or ids and how many
bool kv_selection_ok(const milo_kv_shape *s, const int32_t *selected, int32_t n_sel) {
    if (!selected) return n_sel == 0;
    return aligned(selected, 4) && n_sel >= 1 && kv_tokens_fit(s, n_sel);
}

}  // namespace

extern "C" {

void milo_rope_default_params(milo_rope_params *p, int32_t d, double base) {
    if (!p) return;
    *p = milo_rope_params{d, 0, 0, MILO_ROPE_NONE, base, 1.0, 0.0, 32.0, 1.0, 1.0, 4.0, 0.0};
}

milo_status milo_rope_freqs(const milo_rope_params *p, double *w, double *attn_factor) {
    int rd;
    const milo_status st = rope_check(p, &rd);
    if (st != MILO_OK) return st;
    double f[MILO_ROPE_MAX_D / 2], m;
    rope_freqs(p, rd, f, &m);
    if (w) memcpy(w, f, sizeof(double) * (rd / 2));
    if (attn_factor) *attn_factor = m;
    return MILO_OK;
}

milo_status milo_rope(const milo_rope_params *p, const void *x, milo_dtype x_dtype, int64_t xt, int64_t xh, void *y,
                      milo_dtype y_dtype, int64_t yt, int64_t yh, const int32_t *positions, int64_t n_pos,
                      int64_t n_tokens, int32_t n_heads, int32_t transpose, milo_stream_t stream) {
    int rd;
    milo_status st = rope_check(p, &rd);
    if (st != MILO_OK) return st;
    if (!float_dtype(x_dtype) || !float_dtype(y_dtype)) return MILO_ERR_UNSUPPORTED;
    if (n_tokens < 0 || n_heads < 0) return MILO_ERR_INVALID_ARG;
    if (n_tokens == 0 || n_heads == 0) return MILO_OK;
    const int ex = x_dtype == MILO_F32 ? 4 : 2, ey = y_dtype == MILO_F32 ? 4 : 2, d = p->d;
    if (!x || !y || !positions || n_pos < 1 || xt < 0 || xh < 0 || yt < 0 || yh < 0 || !aligned(x, ex) ||
        !aligned(y, ey) || !aligned(positions, 4))
        return MILO_ERR_INVALID_ARG;
    const int64_t most = int64_t(1) << 46;   // strides and counts whose products stay inside 64 bits
    if (xt > most / n_tokens || xh > most / n_heads || yt > most / n_tokens || yh > most / n_heads || n_tokens > most)
        return MILO_ERR_INVALID_ARG;
    // rows of y apart: one index strides over whole rows of the other
    const bool apart = (n_heads == 1 || yh >= d) && (n_tokens == 1 || yt >= (n_heads - 1) * yh + d);
    const bool apart2 = (n_tokens == 1 || yt >= d) && (n_heads == 1 || yh >= (n_tokens - 1) * yt + d);
    if (!apart && !apart2) return MILO_ERR_INVALID_ARG;
    const bool same = x == y && x_dtype == y_dtype && (xt == yt || n_tokens == 1) && (xh == yh || n_heads == 1);
    if (!same) {
        uintptr_t x0, x1, y0, y1;
        rope_extent(x, xt, xh, n_tokens, n_heads, d, ex, x0, x1);
        rope_extent(y, yt, yh, n_tokens, n_heads, d, ey, y0, y1);
        if (x0 < y1 && y0 < x1) return MILO_ERR_INVALID_ARG;
    }
    RopeArgs a{};
    double w[MILO_ROPE_MAX_D / 2], m;
    rope_freqs(p, rd, w, &m);
    for (int i = 0; i < rd / 2; ++i) a.turns[i] = w[i] / kTwoPi;
    a.x = x; a.y = y; a.pos = positions; a.n_pos = n_pos; a.n_tokens = n_tokens;
    a.xt = xt; a.xh = xh; a.yt = yt; a.yh = yh; a.d = d; a.rd = rd; a.heads = n_heads;
    a.m = (float)m;
    a.sgn = transpose ? -1.f : 1.f;
    // widest access that every row start and both parts of a row allow
    const bool inter = p->interleaved != 0;
    int v = 8;
    auto fits = [&](int n) {
        const int64_t unit = inter ? rd : rd / 2;
        return unit % n == 0 && d % n == 0 && xt % n == 0 && xh % n == 0 && yt % n == 0 && yh % n == 0 &&
               aligned(x, (size_t)std::min(16, n * ex)) && aligned(y, (size_t)std::min(16, n * ey));
    };
    if (!fits(8)) v = fits(4) ? 4 : (inter ? 2 : 1);
    a.rot_units = (inter ? rd : rd / 2) / v;
    a.units = a.rot_units + (same ? 0 : (d - rd) / v);   // in place, the other channels are where they belong
    // a thread takes as many heads as leave a full wave of threads
    const int64_t per_head = n_tokens * a.units, wave = (int64_t)sm_count() * 2048;
    a.hpt = (int)std::min<int64_t>(n_heads, std::max<int64_t>(1, per_head * n_heads / wave));
    a.n_hc = (n_heads + a.hpt - 1) / a.hpt;
    a.hpt = (n_heads + a.n_hc - 1) / a.n_hc;   // equal chunks
    if (grid_x((per_head * a.n_hc + 255) / 256) == 0) return MILO_ERR_UNSUPPORTED;
    a.small = per_head * a.n_hc + 255 < (int64_t(1) << 32);
    cudaStream_t s = (cudaStream_t)stream;
    cudaEvent_t t0 = tmark(s);
    auto go = [&](auto tx, auto ty) {
        using TX = decltype(tx);
        using TY = decltype(ty);
        if (v == 8) rope_launch_layout<TX, TY, 8>(a, inter, s);
        else if (v == 4) rope_launch_layout<TX, TY, 4>(a, inter, s);
        else rope_launch_layout<TX, TY, 1>(a, inter, s);
    };
    if (x_dtype == MILO_F32) y_dtype == MILO_F32 ? go(0.f, 0.f) : go(0.f, __nv_bfloat16());
    else y_dtype == MILO_F32 ? go(__nv_bfloat16(), 0.f) : go(__nv_bfloat16(), __nv_bfloat16());
    tpush(MILO_TK_ROPE, t0, tmark(s));
    return cuda_check(cudaGetLastError(), "rope launch");
}

size_t milo_kv_cache_size(const milo_kv_shape *shape) {
    if (!kv_ok(shape) || shape->d != D) return 0;
    return (size_t)kv_view(shape, nullptr).layer * shape->L;
}

milo_status milo_kv_layout(const milo_kv_shape *shape, size_t *offsets) {
    if (!kv_ok(shape) || !offsets) return MILO_ERR_INVALID_ARG;
    if (shape->d != D) return MILO_ERR_UNSUPPORTED;
    const KvView v = kv_view(shape, nullptr);
    for (int i = 0; i < 7; ++i) offsets[i] = (size_t)v.off[i];
    return MILO_OK;
}

milo_status milo_kv_append(const milo_kv_shape *shape, void *cache, size_t cache_bytes, const void *k, const void *v,
                           milo_dtype in_dtype, const int64_t *strides, int32_t n_new, const int32_t *start,
                           const int32_t *count, milo_stream_t stream) {
    milo_status st = kv_check(shape, cache, cache_bytes);
    if (st != MILO_OK) return st;
    if (!float_dtype(in_dtype)) return MILO_ERR_UNSUPPORTED;
    if (n_new < 0 || n_new > shape->cap) return MILO_ERR_INVALID_ARG;
    if (n_new == 0) return MILO_OK;
    if (!k || !v || !start || !aligned(k, 16) || !aligned(v, 16) || !aligned(start, 4) || !aligned(count, 4))
        return MILO_ERR_INVALID_ARG;
    KvAppendArgs a{};
    a.c = kv_view(shape, cache);
    a.k = k; a.v = v; a.n_new = n_new; a.start = start; a.count = count;
    a.st = D;
    a.sh = (int64_t)n_new * D;
    a.ss = a.sh * shape->H;
    a.sl = a.ss * shape->S;
    if (strides) {
        for (int i = 0; i < 4; ++i)
            if (strides[i] < 0 || strides[i] % 8) return MILO_ERR_INVALID_ARG;
        a.sl = strides[0]; a.ss = strides[1]; a.sh = strides[2]; a.st = strides[3];
    }
    a.windows = (int)(((int64_t)n_new - 2 + shape->block_len) / shape->block_len) + 1;
    a.items = (int)grid_x((int64_t)a.windows * shape->L * shape->S * shape->H * 2);
    if (!a.items) return MILO_ERR_UNSUPPORTED;
    cudaStream_t s = (cudaStream_t)stream;
    cudaEvent_t t0 = tmark(s);
    if (in_dtype == MILO_BF16) kv_append_launch<__nv_bfloat16>(a, s);
    else kv_append_launch<float>(a, s);
    tpush(MILO_TK_KV_WRITE, t0, tmark(s));
    return cuda_check(cudaGetLastError(), "kv append launch");
}

milo_status milo_kv_read(const milo_kv_shape *shape, const void *cache, size_t cache_bytes, int32_t n,
                         const int32_t *start, const int32_t *count, void *k_out, void *v_out, milo_dtype out_dtype,
                         milo_stream_t stream) {
    milo_status st = kv_check(shape, cache, cache_bytes);
    if (st != MILO_OK) return st;
    if (!float_dtype(out_dtype)) return MILO_ERR_UNSUPPORTED;
    if (n < 0 || n > shape->cap) return MILO_ERR_INVALID_ARG;
    if (n == 0) return MILO_OK;
    if ((!k_out && !v_out) || !start || !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(start, 4) ||
        !aligned(count, 4))
        return MILO_ERR_INVALID_ARG;
    KvReadArgs a{};
    a.c = kv_view(shape, cache);
    a.k = k_out; a.v = v_out; a.n = n; a.start = start; a.count = count;
    a.tiles = (n + KV_READ_ROWS - 1) / KV_READ_ROWS;
    const unsigned grid = grid_x((int64_t)shape->L * shape->S * shape->H * a.tiles);
    if (!grid) return MILO_ERR_UNSUPPORTED;
    cudaStream_t s = (cudaStream_t)stream;
    cudaEvent_t t0 = tmark(s);
    if (out_dtype == MILO_BF16) kv_read_launch<__nv_bfloat16>(a, dim3(grid, 2), s);
    else kv_read_launch<float>(a, dim3(grid, 2), s);
    tpush(MILO_TK_KV_READ, t0, tmark(s));
    return cuda_check(cudaGetLastError(), "kv read launch");
}

size_t milo_kv_select_workspace_size(const milo_kv_shape *shape, int32_t n_q) {
    if (!kv_ok(shape) || shape->d != D || n_q <= 0 || !kv_rows_fit(shape, n_q, shape->H)) return 0;
    const int64_t n_b = (shape->cap + shape->block_len - 1) / shape->block_len;
    return align_up(sizeof(float) * (size_t)((int64_t)shape->L * shape->S * shape->H * n_q * n_b));
}

milo_status milo_kv_select(const milo_kv_shape *shape, const void *cache, size_t cache_bytes, const void *q,
                           milo_dtype q_dtype, int32_t n_q, int32_t Hq, const int32_t *len, int32_t n_sel,
                           int32_t n_first, int32_t n_last, int32_t *selected, float *scores, void *workspace,
                           size_t ws_bytes, milo_stream_t stream) {
    milo_status st = kv_check(shape, cache, cache_bytes);
    if (st != MILO_OK) return st;
    st = kv_query_check(shape, q, q_dtype, n_q, Hq, len);
    if (st != MILO_OK) return st;
    KvSelectArgs a{};
    a.c = kv_view(shape, cache);
    if (!selected || !workspace || !aligned(selected, 4) || !aligned(scores, 4) || !aligned(workspace, kAlign) ||
        n_sel < 1 || n_sel > a.c.n_b || n_first < 0 || n_last < 0 || (int64_t)n_first + n_last > n_sel)
        return MILO_ERR_INVALID_ARG;
    if (ws_bytes < milo_kv_select_workspace_size(shape, n_q)) return MILO_ERR_WORKSPACE;
    a.q = q; a.len = len; a.selected = selected; a.scores = scores ? scores : (float *)workspace;
    a.n_q = n_q; a.G = Hq / shape->H; a.n_sel = n_sel; a.n_first = n_first; a.n_last = n_last;
    const unsigned rows = grid_x((int64_t)shape->L * shape->S * n_q * shape->H);
    if (!rows) return MILO_ERR_UNSUPPORTED;
    cudaStream_t s = (cudaStream_t)stream;
    cudaEvent_t t0 = tmark(s);
    cudaError_t e;
    // a CTA for each row and one launch, where the rows fill most of the SMs, or where they are short and read once.  One
    // launch and two, full rows of 7 bf16 heads, in a graph, codes not in L2 (us): 128 rows of 512 blocks 15.0 and 18.1, of 1024
    // 18.1 and 21.9, of 2048 24.6 and 27.0; 111 rows of 2048 23.6 and 25.3; 80 rows of 1024 16.7 and 16.4, of 2048 22.5
    // and 20.5.  Short rows are level in a graph and spare a host that makes the calls one by one the second launch
    // (15.8 and 18.2 for 2 rows of 512): one less two, rows 1/6, 1/2 and 5/6 full on average, 1, 8 and 32 rows of 256 blocks
    // -0.2 -0.6 -0.8, of 512 +0.6 -0.2 -0.3 (full +1.7 +1.0 +0.3), of 640 +0.9 +0.7 +0.2 (full +2.0 +2.4 +1.4); with 12
    // heads, which take two passes, full rows of 512 15.0 and 11.6
    const bool fill = 4 * (int64_t)rows >= 3 * sm_count(), brief = a.c.n_b <= 512 && a.G <= KV_SCORE_G;
    if (rows <= (unsigned)sm_count() && a.c.n_b <= KV_ROW_THREADS * KV_ROW_KEYS && (fill || brief)) {
        if (q_dtype == MILO_BF16) k_kv_select_row<__nv_bfloat16><<<rows, KV_ROW_THREADS, 0, s>>>(a);
        else k_kv_select_row<float><<<rows, KV_ROW_THREADS, 0, s>>>(a);
        e = cudaGetLastError();
    } else {
        // blocks per CTA: as many steps of its warps as leave one wave of four CTAs an SM (a CTA first codes its queries, about
        // what two steps cost)
        const int64_t steps = (a.c.n_b + KV_SCORE_STEP - 1) / KV_SCORE_STEP, wave = 4 * sm_count();
        const int per = KV_SCORE_STEP * (int)std::min<int64_t>((rows * steps + wave - 1) / wave, steps);
        const dim3 grid(rows, (unsigned)((a.c.n_b + per - 1) / per));
        if (q_dtype == MILO_BF16) k_kv_score<__nv_bfloat16><<<grid, 32 * KV_SCORE_WARPS, 0, s>>>(a, per);
        else k_kv_score<float><<<grid, 32 * KV_SCORE_WARPS, 0, s>>>(a, per);
        e = cudaGetLastError();
        if (e == cudaSuccess)
            e = a.c.n_b <= 2048   ? kv_follow(k_kv_topn<512, 4, true>, dim3(rows), 512, a, s)
                : a.c.n_b <= 8192 ? kv_follow(k_kv_topn<1024, 8, true>, dim3(rows), 1024, a, s)
                                  : kv_follow(k_kv_topn<1024, 1, false>, dim3(rows), 1024, a, s);
    }
    tpush(MILO_TK_KV_SELECT, t0, tmark(s));
    return cuda_check(e, "kv select launch");
}

size_t milo_kv_attn_workspace_size(const milo_kv_shape *shape, int32_t n_q, int32_t Hq, int32_t n_sel) {
    if (!kv_ok(shape) || shape->d != D || n_q <= 0 || Hq <= 0 || Hq % shape->H || n_sel < 0 ||
        !kv_rows_fit(shape, n_q, Hq) || !kv_tokens_fit(shape, n_sel))
        return 0;
    return kv_attn_plan(shape, n_q, Hq, n_sel).bytes;
}

milo_status milo_kv_attn(const milo_kv_shape *shape, const void *cache, size_t cache_bytes, const void *q,
                         milo_dtype q_dtype, int32_t n_q, int32_t Hq, const int32_t *len, const int32_t *selected,
                         int32_t n_sel, double scale, void *out, float *lse, void *workspace, size_t ws_bytes,
                         milo_stream_t stream) {
    milo_status st = kv_check(shape, cache, cache_bytes);
    if (st != MILO_OK) return st;
    st = kv_query_check(shape, q, q_dtype, n_q, Hq, len);
    if (st != MILO_OK) return st;
    if (!out || !workspace || !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, kAlign) ||
        !kv_selection_ok(shape, selected, n_sel) || !(scale >= 0.0) || !std::isfinite(scale))
        return MILO_ERR_INVALID_ARG;
    if (ws_bytes < milo_kv_attn_workspace_size(shape, n_q, Hq, n_sel)) return MILO_ERR_WORKSPACE;
    cudaStream_t s = (cudaStream_t)stream;
    cudaEvent_t t0 = tmark(s);
    st = kv_attn_launch(shape, cache, q, q_dtype, n_q, Hq, len, selected, n_sel, scale, out, lse, nullptr, workspace, s);
    tpush(MILO_TK_KV_ATTN, t0, tmark(s));
    return st;
}

size_t milo_decode_kv_workspace_size(const milo_factors *f, int32_t S, int32_t Hq, int32_t n_sel,
                                     const milo_kv_shape *shape, int32_t kv_n_sel) {
    const size_t base = milo_decode_tail_workspace_size(f, S, Hq, n_sel);
    const size_t kv = milo_kv_attn_workspace_size(shape, 1, Hq, kv_n_sel);
    return base && kv ? base + kv : 0;
}

milo_status milo_decode_attn_kv(const milo_factors *f, const float *q, int32_t S, int32_t Hq, const int32_t *selected,
                                const int32_t *positions, int32_t n_sel, double rope_base, const milo_kv_shape *shape,
                                const void *cache, size_t cache_bytes, const int32_t *len, const int32_t *kv_selected,
                                int32_t kv_n_sel, float *out, void *workspace, size_t ws_bytes, milo_stream_t stream) {
    milo_status st = kv_check(shape, cache, cache_bytes);
    if (st != MILO_OK) return st;
    if (!f || shape->L != f->shape.L || shape->H != f->shape.H || shape->S != S) return MILO_ERR_INVALID_ARG;
    st = kv_query_check(shape, q, MILO_F32, 1, Hq, len);
    if (st != MILO_OK) return st;
    if (!kv_selection_ok(shape, kv_selected, kv_n_sel)) return MILO_ERR_INVALID_ARG;
    TailIn t;
    t.len = len;
    t.kv = shape;
    t.kv_cache = cache;
    t.kv_selected = kv_selected;
    t.kv_n_sel = kv_n_sel;
    return decode_impl(f, q, S, Hq, selected, positions, n_sel, rope_base, t, out, workspace, ws_bytes, stream);
}

}  // extern "C"

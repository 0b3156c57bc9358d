// kv_attn.cuh -- attention over the quantised cache of recent tokens.
//
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q . k_t - m)
//
// over the tokens that a query sees, all of them or those of the blocks it
// selected.  The work is one pass over the code rows (4 d / row bytes flops per
// byte and query head), so memory bounds it as long as the codes reach the
// tensor cores cheaply:
//
// * A warp takes 16 tokens at a time straight from memory into the operand
//   registers of m16n8k16: tokens are the rows of the score product (A = K, B =
//   up to 8 NT queries from shared memory), channels those of the value
//   product (A = V^T, B = the weights, transposed between the two by movmatrix).
//   Both products sum over an index whose order is free, so a thread's 16-byte
//   loads are already fragments; codes become fp16 exactly (INT8 and e4m3 times
//   the row's scale later, INT4 as the fp16 value it stands for).
// * Row scales never touch the rows: the key's multiplies the score, the
//   value's the weight.  A weight is kept as p * v_scale / 2^E * 2^10 in fp16,
//   with E the greatest exponent of the scales so far.
// * fp32 queries go in two fp16 parts (22 bits, after a power of two that puts
//   the row's greatest value at 2^8), and so do their weights; bf16 queries fit in
//   one part, and their weights are rounded to fp16 (2^-11, an eighth of the
//   output's rounding).  Sums are fp32.
// * The reference m of the weights is raised only when a score passes it by more
//   than 4 (in powers of two), so that most tiles neither exchange maxima nor
//   rescale; the weights then reach 2^(4 + 1 + 10) at most.
//
// The (layer, session, KV head, query tile) lines are cut into units of 16 * WARPS
// tokens, and every CTA of a single wave takes an equal run of units, whatever the
// lengths are: a run that covers a line writes its result, the parts of a line that
// several CTAs share are merged by k_kv_attn_merge in a fixed order.
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
    int tpb;                       // tiles of 16 tokens per block
    uint32_t tpb_magic;            // ceil(2^32 / tpb), 0 for tpb = 1
    int row_tiles;                 // query tiles of a line's rows
    int64_t classes;               // S * row_tiles (dense), S * n_q * row_tiles (selected)
    float scale;                   // softmax scale * log2(e)
    float *part_o;                 // [2 grid][8 NT][D] normalised outputs of parts
    float2 *part_ml;               // [2 grid][8 NT] (reference, sum) of parts, in powers of two
    longlong2 *split;              // [grid] line that a CTA begins and others end, or -1; its last CTA
};

constexpr int KA_WARPS = 8, KA_THREADS = 32 * KA_WARPS, KA_UNIT = 16 * KA_WARPS;
constexpr float KA_RAISE = 4.f;        // a score this far above the reference raises it
constexpr float KA_SHIFT = 10.f;       // weights are kept times 2^10 (fp16's subnormals begin at 2^-14)

// ------------------------------------------------------------ instructions
__device__ __forceinline__ void ka_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t ka_transpose(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float ka_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t ka_u(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 ka_h(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }
__device__ __forceinline__ uint4 ka_ldg16(const unsigned char *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ka_ldg8(const unsigned char *p) {
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

// INT8: bytes (biased by 128) b0, b1 (sel 0x4140) or b2, b3 (0x4342) of x under
// the high byte of 1024 + code + 128
__device__ __forceinline__ uint32_t ka_int8(uint32_t x, uint32_t sel) {
    return ka_u(__hsub2(ka_h(__byte_perm(x, 0x64646464u, sel)), __half2half2(__ushort_as_half(0x6480))));
}
// e4m3: the fp16 with the same sign, exponent and fraction fields, which is the
// value times 2^-8 (exact, subnormals too); the 2^8 goes into the row's factors.
// The bytes come in the high halves of the result (sel 0x1404, 0x3424).
constexpr float KA_FP8_UP = 256.f;
__device__ __forceinline__ uint32_t ka_fp8(uint32_t x, uint32_t sel) {
    const uint32_t w = __byte_perm(x, 0u, sel);
    return (w & 0x80008000u) | ((w >> 1) & 0x3f803f80u);
}
// two codes of 4 bits in bits 0-3 (HI: 4-7) of a word's halves -> their fp16 values
template <bool HI> __device__ __forceinline__ uint32_t ka_int4(uint32_t x, __half2 s, __half2 z) {
    __half2 c;
    if (HI) c = __hfma2(ka_h((x & 0x00f000f0u) | 0x64006400u), __half2half2(__ushort_as_half(0x2c00)),
                        __half2half2(__ushort_as_half(0xd400)));    // (1024 + 16 code) / 16 - 64
    else c = __hsub2(ka_h((x & 0x000f000fu) | 0x64006400u), __half2half2(__ushort_as_half(0x6400)));
    return ka_u(__hfma2(c, s, z));
}

// ---------------------------------------------------------- a tile's codes
// Keys: rows t0 + g and t0 + g + 8, values: rows t0 + {2c, 2c + 1, 2c + 8, 2c + 9}
// (g = lane / 4, c = lane % 4).  Rows from `end` on are neither read nor used.
template <int DT> struct KaTile;

template <> struct KaTile<MILO_INT8> {
    uint4 k[4], v[4];
    float ks[2], vs[2];
};
template <> struct KaTile<MILO_FP8> : KaTile<MILO_INT8> {};
template <> struct KaTile<MILO_INT4> {
    uint4 k[2];
    uint2 v[4];
    uint32_t kp[2], vp[4];       // (scale, zero) of the thread's group in each row
};

template <int DT> struct KaLine {
    const unsigned char *k, *v, *kp, *vp;
};

template <int DT>
__device__ __forceinline__ void ka_load_k(KaTile<DT> &t, const KaLine<DT> &ln, int64_t t0, int64_t end, int g, int c) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int64_t row = t0 + g + 8 * r;
        const bool ok = row < end;
        if constexpr (DT == MILO_INT4) {
            t.k[r] = make_uint4(0u, 0u, 0u, 0u);
            t.kp[r] = 0u;
            if (ok) {
                t.k[r] = ka_ldg16(ln.k + row * 64 + 16 * c);
                t.kp[r] = __ldg(reinterpret_cast<const uint32_t *>(ln.kp + row * 16) + c);
            }
        } else {
            t.k[2 * r] = t.k[2 * r + 1] = make_uint4(0u, 0u, 0u, 0u);
            t.ks[r] = t.vs[r] = 0.f;
            if (ok) {
                t.k[2 * r] = ka_ldg16(ln.k + row * 128 + 16 * c);
                t.k[2 * r + 1] = ka_ldg16(ln.k + row * 128 + 64 + 16 * c);
                t.ks[r] = __ldg(reinterpret_cast<const float *>(ln.kp) + row);
                t.vs[r] = __ldg(reinterpret_cast<const float *>(ln.vp) + row);
            }
        }
    }
}

template <int DT>
__device__ __forceinline__ void ka_load_v(KaTile<DT> &t, const KaLine<DT> &ln, int64_t t0, int64_t end, int g, int c) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int64_t row = t0 + 2 * c + (r & 1) + 8 * (r >> 1);
        const bool ok = row < end;
        if constexpr (DT == MILO_INT4) {
            t.v[r] = make_uint2(0u, 0u);
            t.vp[r] = 0u;
            if (ok) {
                t.v[r] = ka_ldg8(ln.v + row * 64 + 8 * g);
                t.vp[r] = __ldg(reinterpret_cast<const uint32_t *>(ln.vp + row * 16) + g / 2);
            }
        } else {
            t.v[r] = make_uint4(0u, 0u, 0u, 0u);
            if (ok) t.v[r] = ka_ldg16(ln.v + row * 128 + 16 * g);
        }
    }
}

__device__ __forceinline__ uint32_t ka_word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// channel of element e (0..3: b0 low, b0 high, b1 low, b1 high) of the queries'
// fragment for step j of the score product, thread column c: the order in which
// the keys' codes come
template <int DT> __device__ __forceinline__ int ka_channel(int j, int c, int e) {
    if (DT == MILO_INT4) return 32 * c + 8 * (j / 2) + 2 * (j % 2) + (e / 2) + 4 * (e % 2);
    return (j < 4 ? 16 * c + 4 * j : 64 + 16 * c + 4 * (j - 4)) + e;
}

// A fragment of step j of the score product
template <int DT> __device__ __forceinline__ void ka_frag_k(const KaTile<DT> &t, int j, uint32_t (&a)[4]) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        if constexpr (DT == MILO_INT4) {
            const __half2 s = ka_h(__byte_perm(t.kp[r], 0u, 0x1010)), z = ka_h(__byte_perm(t.kp[r], 0u, 0x3232));
            const uint32_t w = ka_word(t.k[r], j / 2) >> (j % 2 ? 8 : 0);
            a[r] = ka_int4<false>(w, s, z);
            a[2 + r] = ka_int4<true>(w, s, z);
        } else {
            uint32_t w = ka_word(t.k[2 * r + j / 4], j % 4);
            if constexpr (DT == MILO_INT8) {
                w ^= 0x80808080u;
                a[r] = ka_int8(w, 0x4140);
                a[2 + r] = ka_int8(w, 0x4342);
            } else {
                a[r] = ka_fp8(w, 0x1404);
                a[2 + r] = ka_fp8(w, 0x3424);
            }
        }
    }
}

// A fragments of row tiles 2 w and 2 w + 1 of the value product: channels 16 g +
// 4 w .. + 3, tokens 2c, 2c + 1 (h = 0) and 2c + 8, 2c + 9 (h = 1)
template <int DT> __device__ __forceinline__ void ka_frag_v(const KaTile<DT> &t, int w, uint32_t (&a)[2][4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if constexpr (DT == MILO_INT4) {
            const __half2 s = ka_h(__byte_perm(t.vp[2 * h], t.vp[2 * h + 1], 0x5410));
            const __half2 z = ka_h(__byte_perm(t.vp[2 * h], t.vp[2 * h + 1], 0x7632));
            const uint32_t A = w < 2 ? t.v[2 * h].x : t.v[2 * h].y, B = w < 2 ? t.v[2 * h + 1].x : t.v[2 * h + 1].y;
            const uint32_t x = __byte_perm(A, B, w % 2 ? 0x7632 : 0x5410), y = x >> 8;
            a[0][2 * h] = ka_int4<false>(x, s, z);
            a[0][2 * h + 1] = ka_int4<true>(x, s, z);
            a[1][2 * h] = ka_int4<false>(y, s, z);
            a[1][2 * h + 1] = ka_int4<true>(y, s, z);
        } else {
            const uint32_t A = ka_word(t.v[2 * h], w), B = ka_word(t.v[2 * h + 1], w);
            uint32_t x = __byte_perm(A, B, 0x5140), y = __byte_perm(A, B, 0x7362);   // (A0 B0 A1 B1), (A2 B2 A3 B3)
            if constexpr (DT == MILO_INT8) {
                x ^= 0x80808080u;
                y ^= 0x80808080u;
                a[0][2 * h] = ka_int8(x, 0x4140);
                a[0][2 * h + 1] = ka_int8(x, 0x4342);
                a[1][2 * h] = ka_int8(y, 0x4140);
                a[1][2 * h + 1] = ka_int8(y, 0x4342);
            } else {
                a[0][2 * h] = ka_fp8(x, 0x1404);
                a[0][2 * h + 1] = ka_fp8(x, 0x3424);
                a[1][2 * h] = ka_fp8(y, 0x1404);
                a[1][2 * h + 1] = ka_fp8(y, 0x3424);
            }
        }
    }
}

// ------------------------------------------------------------------- lines
// A class is a (session, query, query tile) -- dense: all queries share their
// lines -- and holds L * H lines of equal length.
template <bool SEL> struct KaClass {
    int s, i, rt, rows, end;       // rows of the class's query tile, tokens that its last row sees

    __device__ __forceinline__ void set(const KvAttnArgs &a, int64_t k, int rpt, bool tell) {
        rt = (int)(k % a.row_tiles);
        k /= a.row_tiles;
        i = SEL ? (int)(k % a.n_q) : 0;
        s = (int)(SEL ? k / a.n_q : k);
        const int all = SEL ? a.G : a.n_q * a.G;
        rows = min(rpt, all - rt * rpt);
        end = kv_seen(a.len, s, a.n_q, SEL ? i : (rt * rpt + rows - 1) / a.G, a.c.cap, tell);
    }
    // 16-token tiles of a line (selected: of all listed blocks)
    __device__ __forceinline__ int64_t tiles(const KvAttnArgs &a) const {
        return SEL ? (int64_t)a.n_sel * a.tpb : ((int64_t)end + 15) / 16;
    }
    __device__ __forceinline__ int64_t units(const KvAttnArgs &a) const {
        const int64_t u = (tiles(a) + KA_WARPS - 1) / KA_WARPS;
        return u > 0 ? u : 1;      // an empty line still writes its zeros
    }
    // query of row r, and the row's index in [L][S][n_q][Hq]
    __device__ __forceinline__ int query(const KvAttnArgs &a, int r, int rpt) const {
        return SEL ? i : (rt * rpt + r) / a.G;
    }
    __device__ __forceinline__ int64_t row(const KvAttnArgs &a, int l, int h, int r, int rpt) const {
        const int at = rt * rpt + r, g = SEL ? at : at % a.G;
        return (((int64_t)l * a.c.S + s) * a.n_q + query(a, r, rpt)) * a.c.H * a.G + (int64_t)h * a.G + g;
    }
};

template <typename T, int NT> struct KaSmem {
    static constexpr int RPT = 8 * NT;                       // query rows of a line
    static constexpr int PARTS = sizeof(T) == 4 ? 2 : 1;     // fp16 parts of a query
    uint32_t q[NT][8][32][2 * PARTS];                        // fragments of the queries, [tile][step][lane]
    float o[KA_WARPS][RPT][D + 4];                           // the warps' outputs (channel rows padded)
    float m[KA_WARPS][RPT], l[KA_WARPS][RPT];
    float e[KA_WARPS];                                       // exponent of the warp's value scales
    float sc[RPT];                                           // factor on a row's scores
    int seen[RPT];
    int64_t scan[KA_WARPS + 1];
    int64_t cls, off;
};

// out / lse / (max, sum) of one finished row: normalised o, reference m and sum l in powers of two
template <typename T>
__device__ __forceinline__ void ka_finish(const KvAttnArgs &a, int64_t row, int ch, float o, float m, float l) {
    if constexpr (sizeof(T) == 4) ((float *)a.out)[row * D + ch] = o;
    else ((__nv_bfloat16 *)a.out)[row * D + ch] = __float2bfloat16_rn(o);
    if (ch == 0) {
        const float ln2 = 0.693147180559945309f;
        if (a.lse) a.lse[row] = l != 0.f ? (m + log2f(l)) * ln2 : -INFINITY;
        if (a.ml) a.ml[row] = l != 0.f ? make_float2(m * ln2, l) : make_float2(-INFINITY, 0.f);
    }
}

template <typename T, int DT, int NT, bool SEL>
__global__ void __launch_bounds__(KA_THREADS, 2) k_kv_attn(const __grid_constant__ KvAttnArgs a) {
    using Sm = KaSmem<T, NT>;
    constexpr int RPT = Sm::RPT, PARTS = Sm::PARTS;
    constexpr bool PAR = DT != MILO_INT4;                    // a scale per row
    extern __shared__ __align__(16) unsigned char ka_raw[];
    Sm &sm = *reinterpret_cast<Sm *>(ka_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int64_t LH = (int64_t)a.c.L * a.c.H;

    // this CTA's run of units [u0, u1) and the class that u0 falls into
    int64_t total;
    KaClass<SEL> cl;
    if (SEL) {
        cl.set(a, 0, RPT, false);
        total = a.classes * LH * cl.units(a);
    } else {
        const int64_t per = (a.classes + KA_THREADS - 1) / KA_THREADS;
        const int64_t k0 = min(a.classes, tid * per), k1 = min(a.classes, k0 + per);
        int64_t mine = 0;
        for (int64_t k = k0; k < k1; ++k) {
            cl.set(a, k, RPT, blockIdx.x == 0);   // each class once
            mine += cl.units(a) * LH;
        }
        int64_t inc = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += x;
        }
        if (lane == 31) sm.scan[warp] = inc;
        __syncthreads();
        int64_t before = 0;
        total = 0;
        for (int w = 0; w < KA_WARPS; ++w) {
            if (w < warp) before += sm.scan[w];
            total += sm.scan[w];
        }
        int64_t at = before + inc - mine;                    // first unit of class k0
        const int64_t n = (total + gridDim.x - 1) / gridDim.x, u = blockIdx.x * n;
        if (u >= at && u < at + mine) {
            int64_t k = k0;
            for (;; ++k) {
                cl.set(a, k, RPT, false);
                const int64_t w = cl.units(a) * LH;
                if (u < at + w) break;
                at += w;
            }
            sm.cls = k;
            sm.off = at;
        }
        __syncthreads();
    }
    const int64_t n_units = (total + gridDim.x - 1) / gridDim.x;
    int64_t u0 = blockIdx.x * n_units;
    const int64_t u1 = min(total, u0 + n_units);
    if (tid == 0) a.split[blockIdx.x] = make_longlong2(-1, -1);
    if (u0 >= u1) return;
    int64_t k, cls0;                                         // class, its first unit
    if (SEL) {
        const int64_t w = cl.units(a) * LH;
        k = u0 / w;
        cls0 = k * w;
    } else {
        k = sm.cls;
        cls0 = sm.off;
    }
    cl.set(a, k, RPT, SEL && tid == 0);
    int64_t per = cl.units(a);

    while (u0 < u1) {
        if (u0 >= cls0 + per * LH) {                         // next class
            cls0 += per * LH;
            cl.set(a, ++k, RPT, SEL && tid == 0);
            per = cl.units(a);
        }
        const int64_t lh = (u0 - cls0) / per, line0 = cls0 + lh * per;
        const int64_t s0 = u0 - line0, s1 = min(per, u1 - line0);   // this segment's units of the line
        const int l = (int)(lh / a.c.H), h = (int)(lh % a.c.H);
        const int64_t sh = (int64_t)cl.s * a.c.H + h;
        const KaLine<DT> ln{a.c.codes(l, sh, 0), a.c.codes(l, sh, 1), a.c.params(l, sh, 0), a.c.params(l, sh, 1)};
        const int32_t *sel = SEL ? a.sel + ((((int64_t)l * a.c.S + cl.s) * a.n_q + cl.i) * a.c.H + h) * a.n_sel : nullptr;
        const int64_t v_end = min(cl.tiles(a), s1 * KA_WARPS);       // tiles [v, v_end) in steps of KA_WARPS
        int64_t v = s0 * KA_WARPS + warp;

        // first token of tile v and the end of its rows
        auto slot = [&](int64_t x) { return a.tpb_magic ? (int)__umulhi((uint32_t)x, a.tpb_magic) : (int)x; };
        auto id_of = [&](int64_t x) { return x < v_end ? __ldg(sel + slot(x)) : -1; };
        auto place = [&](int64_t x, int id, int64_t &t0, int64_t &end) {
            if (SEL) {
                const bool ok = id >= 0 && id < a.c.n_b;
                if (!ok && id != -1 && lane == 0) raise_status(ST_BOUNDS);
                t0 = ok ? ((int64_t)id * a.tpb + (x - (int64_t)slot(x) * a.tpb)) * 16 : 0;
                end = ok ? cl.end : 0;
            } else {
                t0 = x * 16;
                end = x < v_end ? cl.end : 0;
            }
        };
        KaTile<DT> t;
        int64_t t0, end;
        int id_next = 0;
        place(v, SEL ? id_of(v) : 0, t0, end);
        if (SEL) id_next = id_of(v + KA_WARPS);
        ka_load_k<DT>(t, ln, t0, end, g, c);
        ka_load_v<DT>(t, ln, t0, end, g, c);

        // the line's queries as fragments, a warp per row
        for (int r = warp; r < RPT; r += KA_WARPS) {
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            const bool live = r < cl.rows;
            if (live) {
                const T *q = (const T *)a.q + cl.row(a, l, h, r, RPT) * D + 4 * lane;
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = to_f32(q[e]);
            }
            float mx = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
            for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const int e = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 127);
            const float up = __uint_as_float((uint32_t)(135 - e) << 23), down = __uint_as_float((uint32_t)(119 + e) << 23);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int ch = 4 * lane + w;
                int j, cc, el;                                // the inverse of ka_channel
                if (DT == MILO_INT4) {
                    cc = ch / 32;
                    j = 2 * ((ch % 32) / 8) + (ch % 4) / 2;
                    el = 2 * (ch % 2) + (ch % 8) / 4;
                } else {
                    cc = (ch % 64) / 16;
                    j = (ch / 64) * 4 + (ch % 16) / 4;
                    el = ch % 4;
                }
                const float y = isfinite(x[w]) ? x[w] * up : NAN;   // an infinity spoils its row's scores like a NaN
                const __half hi = __float2half_rn(y);
                __half *f = reinterpret_cast<__half *>(sm.q[r / 8][j][(r % 8) * 4 + cc]);
                f[el] = hi;
                if (PARTS == 2) f[4 + el] = __float2half_rn(y - __half2float(hi));
            }
            if (lane == 0) {
                sm.sc[r] = a.scale * (DT == MILO_FP8 ? KA_FP8_UP : 1.f) * down;
                // rows behind the last are zero queries that see what the others see
                sm.seen[r] = SEL || !live ? cl.end : kv_seen(a.len, cl.s, a.n_q, cl.query(a, r, RPT), a.c.cap, false);
            }
        }
        __syncthreads();
        float sc[NT][2], ref[NT][2], sum[NT][2], o[NT][8][4];
        int seen[NT][2], least = cl.end;                     // least: tokens that every row of the thread sees
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                sc[n][x] = sm.sc[8 * n + 2 * c + x];
                seen[n][x] = sm.seen[8 * n + 2 * c + x];
                least = min(least, seen[n][x]);
                ref[n][x] = -INFINITY;
                sum[n][x] = 0.f;
#pragma unroll
                for (int w = 0; w < 8; ++w) o[n][w][2 * x] = o[n][w][2 * x + 1] = 0.f;
            }
        float e_max = 0.f, e_inv = 0.f;                      // 2^E and 2^-E of the value scales so far

        for (; v < v_end; v += KA_WARPS) {
            int64_t t0n, endn;
            place(v + KA_WARPS, id_next, t0n, endn);
            if (SEL) id_next = id_of(v + 2 * KA_WARPS);
            // scores: tokens t0 + g (+ 8), queries 2c, 2c + 1 of each tile of 8
            float s[NT][4], slo[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[n][x] = slo[n][x] = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t f[4];
                ka_frag_k<DT>(t, j, f);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if constexpr (PARTS == 2) {
                        const uint4 b = *reinterpret_cast<const uint4 *>(sm.q[n][j][lane]);
                        ka_mma(s[n], f[0], f[1], f[2], f[3], b.x, b.y);
                        ka_mma(slo[n], f[0], f[1], f[2], f[3], b.z, b.w);
                    } else {
                        const uint2 b = *reinterpret_cast<const uint2 *>(sm.q[n][j][lane]);
                        ka_mma(s[n], f[0], f[1], f[2], f[3], b.x, b.y);
                    }
                }
            }
            float ks[2] = {1.f, 1.f}, vs[2] = {1.f, 1.f};
            if constexpr (PAR) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    ks[r] = t.ks[r];
                    vs[r] = t.vs[r];
                }
            }
            ka_load_k<DT>(t, ln, t0n, endn, g, c);
            bool raise = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    if (PARTS == 2) s[n][x] += slo[n][x];
                    s[n][x] *= PAR ? ks[x / 2] * sc[n][x % 2] : sc[n][x % 2];
                }
            if (t0 + 16 > least || end == 0) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (t0 + g + 8 * (x / 2) >= min((int64_t)seen[n][x % 2], end)) s[n][x] = -INFINITY;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) raise |= s[n][x] > ref[n][x % 2] + KA_RAISE;
            if (__any_sync(0xffffffffu, raise)) {            // raise the references to this tile's maxima
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float m = fmaxf(s[n][x], s[n][2 + x]);
#pragma unroll
                        for (int w = 4; w < 32; w <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
                        m = fmaxf(m, ref[n][x]);
                        const float f = ref[n][x] == -INFINITY ? 0.f : ka_exp2(ref[n][x] - m);
                        ref[n][x] = m;
                        sum[n][x] *= f;
#pragma unroll
                        for (int w = 0; w < 8; ++w) {
                            o[n][w][x] *= f;
                            o[n][w][2 + x] *= f;
                        }
                    }
            }
            if constexpr (PAR) {
                const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(vs[0], vs[1])));
                const float pw = __uint_as_float(min(max(top & 0x7f800000u, 0x00800000u), 0x7e800000u));   // 2^E
                if (pw > e_max) {
                    const float f = e_max * (1.f / pw);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int w = 0; w < 8; ++w)
#pragma unroll
                            for (int x = 0; x < 4; ++x) o[n][w][x] *= f;
                    e_max = pw;
                    e_inv = 1.f / pw;
                }
                vs[0] *= e_inv;
                vs[1] *= e_inv;
            }
            // weights, as fragments of the value product
            uint32_t b[NT][2][PARTS];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float p[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float m = ref[n][x % 2];
                    p[x] = ka_exp2(s[n][x] - (m == -INFINITY ? 0.f : m) + KA_SHIFT);
                    sum[n][x % 2] += p[x];
                    if (PAR) p[x] *= vs[x / 2];
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const __half2 hi = __floats2half2_rn(p[2 * r], p[2 * r + 1]);
                    b[n][r][0] = ka_transpose(ka_u(hi));
                    if constexpr (PARTS == 2)
                        b[n][r][1] = ka_transpose(ka_u(__floats2half2_rn(p[2 * r] - __low2float(hi),
                                                                         p[2 * r + 1] - __high2float(hi))));
                }
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t f[2][4];
                ka_frag_v<DT>(t, w, f);
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int p = 0; p < PARTS; ++p)
                            ka_mma(o[n][2 * w + y], f[y][0], f[y][1], f[y][2], f[y][3], b[n][0][p], b[n][1][p]);
            }
            ka_load_v<DT>(t, ln, t0n, endn, g, c);
            t0 = t0n;
            end = endn;
        }

        // join the warps: reference and sum per query, then the outputs
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) sum[n][x] += __shfl_xor_sync(0xffffffffu, sum[n][x], w);
                const int r = 8 * n + 2 * c + x;
                if (g == 0) {
                    sm.m[warp][r] = ref[n][x];
                    sm.l[warp][r] = sum[n][x];
                }
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    *reinterpret_cast<float4 *>(&sm.o[warp][r][16 * g + 4 * w]) =
                        make_float4(o[n][2 * w][x], o[n][2 * w][2 + x], o[n][2 * w + 1][x], o[n][2 * w + 1][2 + x]);
            }
        if (lane == 0) sm.e[warp] = PAR ? e_max : 1.f;
        __syncthreads();
        const bool whole = s0 == 0 && s1 == per;
        const int64_t part = 2 * (int64_t)blockIdx.x + (s0 == 0 ? 1 : 0);
        float e_top = 0.f;
#pragma unroll
        for (int w = 0; w < KA_WARPS; ++w) e_top = fmaxf(e_top, sm.e[w]);
        for (int x = tid; x < RPT * D; x += KA_THREADS) {
            const int r = x / D, ch = x % D;
            if (r >= cl.rows) break;
            float m = -INFINITY, num = 0.f, den = 0.f;
#pragma unroll
            for (int w = 0; w < KA_WARPS; ++w) m = fmaxf(m, sm.m[w][r]);
#pragma unroll
            for (int w = 0; w < KA_WARPS; ++w) {
                if (sm.m[w][r] == -INFINITY && sm.l[w][r] == 0.f) continue;      // saw nothing
                const float f = ka_exp2(sm.m[w][r] - m);
                den = fmaf(f, sm.l[w][r], den);
                num = fmaf(f * (e_top > 0.f ? sm.e[w] / e_top : 0.f), sm.o[w][r][ch], num);
            }
            const float y = den != 0.f ? num / den * (e_top * (DT == MILO_FP8 ? KA_FP8_UP : 1.f)) : 0.f;
            if (whole) ka_finish<T>(a, cl.row(a, l, h, r, RPT), ch, y, m - KA_SHIFT, den);
            else {
                a.part_o[(part * RPT + r) * D + ch] = y;
                if (ch == 0) a.part_ml[part * RPT + r] = make_float2(m - KA_SHIFT, den);
            }
        }
        if (!whole && s0 == 0 && tid == 0)                   // begun here, ended by a later CTA
            a.split[blockIdx.x] = make_longlong2(k * LH + lh, (line0 + per - 1) / n_units);
        __syncthreads();                                     // queries and outputs used before the next segment
        u0 = line0 + s1;
    }
}

// Joins the parts of a line that CTA blockIdx.x begins: grid (grid of k_kv_attn, 8 NT rows),
// 16 warps take the parts in turn.
constexpr int KA_MERGE_WARPS = 16;
template <typename T, int NT, bool SEL>
__global__ void __launch_bounds__(32 * KA_MERGE_WARPS) k_kv_attn_merge(const __grid_constant__ KvAttnArgs a) {
    constexpr int RPT = 8 * NT;
    __shared__ float s_o[KA_MERGE_WARPS][D], s_l[KA_MERGE_WARPS], s_m[KA_MERGE_WARPS];
    const longlong2 sp = a.split[blockIdx.x];
    if (sp.x < 0) return;
    const int64_t LH = (int64_t)a.c.L * a.c.H, lh = sp.x % LH;
    const int r = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    KaClass<SEL> cl;
    cl.set(a, sp.x / LH, RPT, false);
    if (r >= cl.rows) return;
    const int n = (int)(sp.y - blockIdx.x) + 1;              // parts: slot 1 of the first CTA, slot 0 of the others
    auto at = [&](int i) { return (2 * ((int64_t)blockIdx.x + i) + (i == 0)) * RPT + r; };
    float m = -INFINITY;
    for (int i = tid; i < n; i += 32 * KA_MERGE_WARPS) {
        const float2 x = a.part_ml[at(i)];
        if (x.y != 0.f) m = fmaxf(m, x.x);
    }
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) s_m[warp] = m;
    __syncthreads();
    for (int w = 0; w < KA_MERGE_WARPS; ++w) m = fmaxf(m, s_m[w]);
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f;
#pragma unroll 4
    for (int i = warp; i < n; i += KA_MERGE_WARPS) {
        const float2 x = a.part_ml[at(i)];
        const float4 o = *reinterpret_cast<const float4 *>(a.part_o + at(i) * D + 4 * lane);
        const float w = x.y != 0.f ? ka_exp2(x.x - m) * x.y : 0.f;
        den += w;
        num.x = fmaf(w, o.x, num.x);
        num.y = fmaf(w, o.y, num.y);
        num.z = fmaf(w, o.z, num.z);
        num.w = fmaf(w, o.w, num.w);
    }
    *reinterpret_cast<float4 *>(&s_o[warp][4 * lane]) = num;
    if (lane == 0) s_l[warp] = den;
    __syncthreads();
    if (tid < D) {
        float y = 0.f, d = 0.f;
        for (int w = 0; w < KA_MERGE_WARPS; ++w) {
            y += s_o[w][tid];
            d += s_l[w];
        }
        ka_finish<T>(a, cl.row(a, (int)(lh / a.c.H), (int)(lh % a.c.H), r, RPT), tid, d != 0.f ? y / d : 0.f, m, d);
    }
}

}  // namespace milo

// kv_attn.cuh -- attention over the quantised cache of recent tokens.
//
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q . k_t - m)
//
// over the tokens that a query sees, all of them or those of the blocks it
// selected.  The work is one pass over the code rows (4 d / row bytes flops per
// byte and query head), so memory bounds it as long as the codes reach the
// tensor cores cheaply:
//
// * A warp takes 16 tokens at a time from its own ring of asynchronous copies: tokens
//   are the rows of the score product (m16n8k16, A = K, B = up to 8 NT queries),
//   channels those of the value product (A = V^T, B = the weights, transposed
//   between the two by movmatrix).  Both products sum over an index whose order
//   is free, so a thread's 16-byte reads are already fragments; codes become
//   fp16 exactly (INT8 and e4m3 times the row's scale later, INT4 as the fp16
//   value it stands for).
// * Row scales never touch the rows: the key's multiplies the score, the
//   value's the weight.  A weight is kept as p * v_scale / 2^E * 2^10 in fp16,
//   with E the greatest exponent of the scales so far.  Where the queries of a line
//   see different tokens (OWN: several queries over all tokens) each row has an E of
//   its own, from the tokens that it sees: another query's token may be any size
//   (1 to 4 % of such a call: 2 queries of 8 heads over 30000 tokens 61.2 -> 63.2 us).
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
// several CTAs share are merged by k_kv_attn_merge in a fixed order.  Short lines
// that one wave holds are not split, and there is no merge (kv_attn_plan).
//
// Measured: 8 sessions of 1000 to 131072 tokens, 4 KV heads of 7 bf16 query heads,
// INT8: 104 us for 558 MB, 82 % of the measured copy rate (the kernel alone 93 us; codes
// loaded straight into registers, a tile ahead: 122 us; more CTAs than a wave, 2, 3 and 4
// times as many: 111, 117 and 123 us).  64 INT4 blocks of 64 tokens for 32 sessions, 2
// layers: 54 us for 169 MB; there about 470 instructions a tile of 16 tokens, 190 of them
// widening the codes, in dependent chains of 3.7 warps a scheduler take the time (2.57
// instructions a cycle of 4, DRAM 41 %).  A short line costs a CTA about 4 us beside its
// tokens.
#pragma once
#include <type_traits>

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
    int row_tiles;                 // query tiles of a line's rows
    int classes;                   // S * row_tiles (dense), S * n_q * row_tiles (selected)
    bool whole;                    // a CTA for each line, and no parts to be merged
    float scale;                   // softmax scale * log2(e)
    float *part_o;                 // [2 grid][8 NT][D] normalised outputs of parts
    float2 *part_ml;               // [2 grid][8 NT] (reference, sum) of parts, in powers of two
    int4 *split;                   // [grid] (class, layer, head, last CTA) of a line that a CTA begins and others end; -1: none
};

// CTA shape by the query tiles of a warp: 8 NT rows
// (16: the wide kernel's 128 rows)
template <int NT> struct KaShape {
    static constexpr int WARPS = NT == 2 ? 4 : 8, CTAS = NT == 1 ? 2 : NT == 2 ? 3 : 1;   // warps of a CTA, CTAs of an SM
    static constexpr int BEGIN = NT == 1 ? 1 : 2;   // units that beginning and ending a line costs, counted at its front
    static constexpr int WHOLE = NT == 16 ? 1 : 8;  // units behind them up to which few lines are not split
};
constexpr uint32_t KA_E_MIN = 0x08800000u;   // 2^-110: least 2^E, so that 2^(10 - E) is finite
constexpr float KA_RAISE = 4.f;        // a score this far above the reference raises it
constexpr float KA_UP = 1024.f;        // weights are kept times 2^10 in fp16, whose subnormals begin at 2^-14

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
// two codes of 4 bits in bits 0-3 (HI: 4-7) of a word's halves -> their fp16 values: the codes under the
// exponent whose last place is worth 1 (1024 + code), or 2^-4 (64 + code)
template <bool HI> __device__ __forceinline__ uint32_t ka_int4(uint32_t x, __half2 s, __half2 z) {
    uint32_t w;   // (x & mask) | exponent in one instruction
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(w) : "r"(x), "n"(HI ? 0x00f000f0 : 0x000f000f), "r"(HI ? 0x54005400 : 0x64006400));
    return ka_u(__hfma2(__hsub2(ka_h(w), __half2half2(__ushort_as_half(HI ? 0x5400 : 0x6400))), s, z));
}

// ---------------------------------------------------------- a tile's codes
// A warp's ring in shared memory holds a tile of 16 tokens per stage: keys,
// values, then the parameters, brought by 16-byte asynchronous copies (rows behind the
// first `rem` are filled with zeros and not read; t0 is a row of the line).  Row r of the score product is
// token ka_token(r) of the tile, and so is index r of the value product; that
// and the exchange of 16-byte chunks below let the fragments' reads touch every bank
// once.
template <int DT> struct KaTile {
    static constexpr int ROW = DT == MILO_INT4 ? D / 2 : D;
    static constexpr int PAR = DT == MILO_INT4 ? 4 * KV_NG : 4;
    static constexpr int V = 16 * ROW, KP = 32 * ROW, VP = KP + 16 * PAR, BYTES = KP + 32 * PAR;
    static constexpr int STAGES = DT == MILO_INT4 ? 5 : 3;
};

// where a lane's share of row 0's tile comes from: chunks of keys and values, and one row's parameters
template <int DT> struct KaLine {
    const unsigned char *k, *v, *p;
    __device__ __forceinline__ KaLine(const unsigned char *k0, const unsigned char *v0, const unsigned char *kp,
                                      const unsigned char *vp, int lane) {
        constexpr int PER = KaTile<DT>::ROW / 16;
        const int at = lane / PER * KaTile<DT>::ROW + 16 * (lane % PER);
        k = k0 + at;
        v = v0 + at;
        p = (lane < 16 ? kp : vp) + (lane & 15) * KaTile<DT>::PAR;
    }
};

template <int DT> __device__ __forceinline__ int ka_token(int r) { return DT == MILO_INT4 ? r ^ ((r >> 1) & 1) : r; }
// where 16-byte chunk `c` of row `t` lies in its row
template <int DT> __device__ __forceinline__ int ka_chunk(int t, int c) {
    return DT == MILO_INT4 ? c ^ ((t >> 1) & 2) : c ^ ((t & 6) ^ ((t & 1) << 2));
}

__device__ __forceinline__ void ka_copy16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ka_copy4(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}
__device__ __forceinline__ void ka_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void ka_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// rows t0 .. t0 + min(rem, 16) - 1 of a line into the stage at shared address `dst`
template <int DT>
__device__ __forceinline__ void ka_fetch(uint32_t dst, const KaLine<DT> &ln, int t0, int rem, int lane) {
    using Tl = KaTile<DT>;
    constexpr int PER = Tl::ROW / 16, STEP = 32 / PER;       // chunks of a row, rows per round of the warp
    const int c = lane % PER, r0 = lane / PER, rp = lane & 15;
    const unsigned char *k = ln.k + (int64_t)t0 * Tl::ROW, *v = ln.v + (int64_t)t0 * Tl::ROW;
    const unsigned char *p = ln.p + (int64_t)t0 * Tl::PAR;
    const uint32_t top = dst + (lane < 16 ? Tl::KP : Tl::VP) + rp * Tl::PAR;
#pragma unroll
    for (int i = 0; i < 16 / STEP; ++i) {
        const int r = r0 + STEP * i;
        const uint32_t to = dst + r * Tl::ROW + 16 * ka_chunk<DT>(r, c);
        ka_copy16(to, k + STEP * i * Tl::ROW, r < rem);
        ka_copy16(to + Tl::V, v + STEP * i * Tl::ROW, r < rem);
    }
    if (DT == MILO_INT4) ka_copy16(top, p, rp < rem);
    else ka_copy4(top, p, rp < rem);
}

// channel of element e (0..3: b0 low, b0 high, b1 low, b1 high) of the queries'
// fragment for step j of the score product, thread column c, and its inverse:
// the order in which the keys' codes come
//   8 bits: (j < 4 ? 16 c + 4 j : 64 + 16 c + 4 (j - 4)) + e
//   4 bits: 32 c + 8 (j / 2) + 2 (j % 2) + e / 2 + 4 (e % 2)
template <int DT> __device__ __forceinline__ void ka_place(int ch, int &j, int &c, int &e) {
    if (DT == MILO_INT4) {
        c = ch / 32;
        j = 2 * ((ch % 32) / 8) + (ch % 4) / 2;
        e = 2 * (ch % 2) + (ch % 8) / 4;
    } else {
        c = (ch % 64) / 16;
        j = (ch / 64) * 4 + (ch % 16) / 4;
        e = ch % 4;
    }
}

__device__ __forceinline__ uint32_t ka_word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// What a thread reads of the tile's keys: rows g and g + 8, 16-byte chunks c and c + 4 (4 bits: chunk c alone, with
// the (scale, zero) of its group)
template <int DT> struct KaKeys {
    uint4 w[2][2];
};
template <> struct KaKeys<MILO_INT4> {
    uint4 w[2];
    uint32_t p[2];
};
template <int DT> __device__ __forceinline__ void ka_read_k(const unsigned char *st, int g, int c, KaKeys<DT> &k) {
    using Tl = KaTile<DT>;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int t = ka_token<DT>(g + 8 * r);
        const unsigned char *row = st + t * Tl::ROW;
        if constexpr (DT == MILO_INT4) {
            k.w[r] = *reinterpret_cast<const uint4 *>(row + 16 * ka_chunk<DT>(t, c));
            k.p[r] = *reinterpret_cast<const uint32_t *>(st + Tl::KP + t * Tl::PAR + 4 * c);
        } else {
            k.w[r][0] = *reinterpret_cast<const uint4 *>(row + 16 * ka_chunk<DT>(t, c));
            k.w[r][1] = *reinterpret_cast<const uint4 *>(row + 16 * ka_chunk<DT>(t, c + 4));
        }
    }
}

// A fragment of step j of the score product
template <int DT> __device__ __forceinline__ void ka_frag_k(const KaKeys<DT> &k, int j, uint32_t (&a)[4]) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        if constexpr (DT == MILO_INT4) {
            const __half2 s = ka_h(__byte_perm(k.p[r], 0u, 0x1010)), z = ka_h(__byte_perm(k.p[r], 0u, 0x3232));
            const uint32_t x = ka_word(k.w[r], j / 2) >> (j % 2 ? 8 : 0);
            a[r] = ka_int4<false>(x, s, z);
            a[2 + r] = ka_int4<true>(x, s, z);
        } else {
            uint32_t x = ka_word(k.w[r][j / 4], j % 4);
            if constexpr (DT == MILO_INT8) {
                x ^= 0x80808080u;
                a[r] = ka_int8(x, 0x4140);
                a[2 + r] = ka_int8(x, 0x4342);
            } else {
                a[r] = ka_fp8(x, 0x1404);
                a[2 + r] = ka_fp8(x, 0x3424);
            }
        }
    }
}

// What a thread reads of the tile's values: channels 16 g .. + 15 of tokens
// r = 2c, 2c + 1, 2c + 8, 2c + 9, 4-bit codes with their (scale, zero)
template <int DT> struct KaValues {
    uint4 w[4];
};
template <> struct KaValues<MILO_INT4> {
    uint2 w[4];
    uint32_t p[4];
};
template <int DT> __device__ __forceinline__ void ka_read_v(const unsigned char *st, int g, int c, KaValues<DT> &v) {
    using Tl = KaTile<DT>;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = ka_token<DT>(2 * c + (i & 1) + 8 * (i >> 1));
        const unsigned char *row = st + Tl::V + t * Tl::ROW;
        if constexpr (DT == MILO_INT4) {
            v.w[i] = *reinterpret_cast<const uint2 *>(row + 16 * ka_chunk<DT>(t, g / 2) + 8 * (g % 2));
            v.p[i] = *reinterpret_cast<const uint32_t *>(st + Tl::VP + t * Tl::PAR + 4 * (g / 2));
        } else {
            v.w[i] = *reinterpret_cast<const uint4 *>(row + 16 * ka_chunk<DT>(t, g));
        }
    }
}

// A fragments of row tiles 2 w and 2 w + 1 of the value product: channels 16 g +
// 4 w .. + 3, tokens 2c, 2c + 1 (h = 0) and 2c + 8, 2c + 9 (h = 1)
template <int DT> __device__ __forceinline__ void ka_frag_v(const KaValues<DT> &t, int w, uint32_t (&a)[2][4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if constexpr (DT == MILO_INT4) {
            const __half2 s = ka_h(__byte_perm(t.p[2 * h], t.p[2 * h + 1], 0x5410));
            const __half2 z = ka_h(__byte_perm(t.p[2 * h], t.p[2 * h + 1], 0x7632));
            const uint32_t A = w < 2 ? t.w[2 * h].x : t.w[2 * h].y, B = w < 2 ? t.w[2 * h + 1].x : t.w[2 * h + 1].y;
            const uint32_t x = __byte_perm(A, B, w % 2 ? 0x7632 : 0x5410), y = x >> 8;
            a[0][2 * h] = ka_int4<false>(x, s, z);
            a[0][2 * h + 1] = ka_int4<true>(x, s, z);
            a[1][2 * h] = ka_int4<false>(y, s, z);
            a[1][2 * h + 1] = ka_int4<true>(y, s, z);
        } else {
            const uint32_t A = ka_word(t.w[2 * h], w), B = ka_word(t.w[2 * h + 1], w);
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
template <bool SEL, int NT> struct KaClass {
    static constexpr int rpt = 8 * NT, KA_WARPS = KaShape<NT>::WARPS;
    int s, i, rt, rows, end;       // rows of the class's query tile, tokens that its last row sees
    int held;                      // tokens of the session

    __device__ __forceinline__ void set(const KvAttnArgs &a, int k, bool tell) {
        rt = k % a.row_tiles;
        k /= a.row_tiles;
        i = SEL ? k % a.n_q : 0;
        s = SEL ? k / a.n_q : k;
        fill(a, tell);
    }
    __device__ __forceinline__ void fill(const KvAttnArgs &a, bool tell) {
        const int all = SEL ? a.G : a.n_q * a.G;
        rows = min(rpt, all - rt * rpt);
        held = kv_seen(a.len, s, 1, 0, a.c.cap, tell);
        end = seen(a, rows - 1);
    }
    __device__ __forceinline__ void next(const KvAttnArgs &a, bool tell) {
        if (++rt == a.row_tiles) {
            rt = 0;
            if (!SEL || ++i == a.n_q) {
                i = 0;
                ++s;
            }
        }
        fill(a, tell);
    }
    // 16-token tiles of a line (selected: of all listed blocks); at most 2^26
    __device__ __forceinline__ int tiles(const KvAttnArgs &a) const {
        return SEL ? a.n_sel * a.tpb : (end + 15) / 16;
    }
    __device__ __forceinline__ int units(const KvAttnArgs &a) const {
        return KaShape<NT>::BEGIN + (tiles(a) + KA_WARPS - 1) / KA_WARPS;
    }
    // tokens that row r sees
    __device__ __forceinline__ int seen(const KvAttnArgs &a, int r) const {
        return max(0, held - a.n_q + query(a, r) + 1);
    }
    // query of row r, and the row's index in [L][S][n_q][Hq]
    __device__ __forceinline__ int query(const KvAttnArgs &a, int r) const {
        return SEL ? i : (rt * rpt + r) / a.G;
    }
    __device__ __forceinline__ int64_t row(const KvAttnArgs &a, int l, int h, int r) const {
        const int at = rt * rpt + r, g = SEL ? at : at % a.G;
        return (((int64_t)l * a.c.S + s) * a.n_q + query(a, r)) * a.c.H * a.G + (int64_t)h * a.G + g;
    }
};

// a / b, both not negative: a 64-bit division takes several times as long as a 32-bit one, and the units nearly always fit
__device__ __forceinline__ int64_t ka_div(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// A CTA's run of units [u0, u1) of the flattened lines, and the line that it is at.
struct KaScan {
    int64_t sum[32], off;
    int cls;
};
template <bool SEL, int NT> struct KaRun {
    static constexpr int THREADS = 32 * KaShape<NT>::WARPS;
    KaClass<SEL, NT> cl;
    int64_t u0, u1, n_units, line0;    // n_units: of every CTA; line0: first unit of the line
    int k, per, l, h;                  // class, units of its lines, the line's layer and head

    __device__ __forceinline__ bool mine_of(int64_t total) {
        n_units = ka_div(total + gridDim.x - 1, gridDim.x);
        u0 = blockIdx.x * n_units;
        u1 = min(total, u0 + n_units);
        return u0 < u1;
    }
    // Finds the run (the whole CTA calls it); false if it is empty.
    __device__ __forceinline__ bool begin(const KvAttnArgs &a, KaScan &sc) {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, LH = a.c.L * a.c.H;
        int64_t total, cls0 = 0;
        if (!SEL && a.whole) {   // selected lines have equal units: their runs are whole lines by themselves
            const int lh = blockIdx.x % LH;
            k = blockIdx.x / LH;
            l = lh / a.c.H;
            h = lh - l * a.c.H;
            cl.set(a, k, tid == 0 && lh == 0);
            per = cl.units(a);
            u0 = line0 = 0;
            u1 = per;
            return true;
        }
        if (SEL) {   // every line has the same units
            per = cl.units(a);
            total = (int64_t)a.classes * LH * per;
            if (!mine_of(total)) return false;
            const int64_t w = (int64_t)per * LH;
            k = (int)ka_div(u0, w);
            cls0 = k * w;
            cl.set(a, k, tid == 0);
        } else if (a.classes <= 32) {   // a class a lane, each warp for itself: no barrier
            KaClass<SEL, NT> at;
            int64_t mine = 0;
            if (lane < a.classes) {
                at.set(a, lane, blockIdx.x == 0 && warp == 0);
                mine = (int64_t)at.units(a) * LH;
            }
            int64_t inc = mine;
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += x;
            }
            total = __shfl_sync(0xffffffffu, inc, 31);
            if (!mine_of(total)) return false;
            k = __popc(__ballot_sync(0xffffffffu, inc <= u0));   // the classes that end before u0
            cls0 = __shfl_sync(0xffffffffu, inc - mine, k);
            cl.set(a, k, false);
            per = cl.units(a);
        } else {
            const int chunk = (a.classes + THREADS - 1) / THREADS;
            const int k0 = (int)min((int64_t)a.classes, (int64_t)tid * chunk), k1 = min(a.classes - k0, chunk) + k0;
            int64_t mine = 0;
            for (int i = k0; i < k1; ++i) {
                cl.set(a, i, blockIdx.x == 0);   // each class once
                mine += (int64_t)cl.units(a) * LH;
            }
            int64_t inc = mine;
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += x;
            }
            if (lane == 31) sc.sum[warp] = inc;
            __syncthreads();
            int64_t before = 0;
            total = 0;
            for (int w = 0; w < THREADS / 32; ++w) {
                if (w < warp) before += sc.sum[w];
                total += sc.sum[w];
            }
            int64_t at = before + inc - mine;    // first unit of class k0
            const int64_t n = ka_div(total + gridDim.x - 1, gridDim.x), u = blockIdx.x * n;
            if (u >= at && u < at + mine) {
                int i = k0;
                for (;; ++i) {
                    cl.set(a, i, false);
                    const int64_t w = (int64_t)cl.units(a) * LH;
                    if (u < at + w) break;
                    at += w;
                }
                sc.cls = i;
                sc.off = at;
            }
            __syncthreads();
            if (!mine_of(total)) return false;
            k = sc.cls;
            cls0 = sc.off;
            cl.set(a, k, false);
            per = cl.units(a);
        }
        const int lh = (int)ka_div(u0 - cls0, per);
        line0 = cls0 + (int64_t)lh * per;
        l = lh / a.c.H;
        h = lh % a.c.H;
        return true;
    }
    // this segment's units [s0, s1) of the line
    __device__ __forceinline__ int s0() const { return (int)(u0 - line0); }
    __device__ __forceinline__ int s1() const { return (int)min((int64_t)per, u1 - line0); }
    // a line begun here and ended by a later CTA, for the merge
    __device__ __forceinline__ int4 split() const { return make_int4(k, l, h, (int)ka_div(line0 + per - 1, n_units)); }
    __device__ __forceinline__ void next(const KvAttnArgs &a, int s1) {
        u0 = line0 + s1;
        if (s1 < per) return;
        line0 += per;
        if (++h < a.c.H) return;
        h = 0;
        if (++l < a.c.L) return;
        l = 0;
        if (u0 < u1) {
            ++k;
            cl.next(a, SEL && threadIdx.x == 0);
            per = cl.units(a);
        }
    }
};

template <typename T, int DT, int NT> struct KaSmem {
    static constexpr int RPT = 8 * NT;                       // query rows of a line
    static constexpr int KA_WARPS = KaShape<NT>::WARPS;
    static constexpr int PARTS = sizeof(T) == 4 ? 2 : 1;     // fp16 parts of a query
    static constexpr int RING = KaTile<DT>::STAGES * KaTile<DT>::BYTES, OUT = RPT * (D + 4) * 4;
    unsigned char ring[KA_WARPS][RING > OUT ? RING : OUT];   // a warp's stages; behind its tiles its output [RPT][D + 4]
    uint32_t q[NT][8][32][2 * PARTS];                        // fragments of the queries, [tile][step][lane]
    float m[KA_WARPS][RPT], l[KA_WARPS][RPT];
    float e[KA_WARPS + 1][RPT];                              // 2^E of the warps' value scales, and the join's factor
    float sc[RPT];                                           // factor on a row's scores
    int seen[RPT];
    int t0[KA_WARPS][KaTile<DT>::STAGES];                    // first token of the tile in each stage
    KaScan scan;
};

// lse / (max, sum) of one finished row, from the reference m and the sum l in powers of two
__device__ __forceinline__ void ka_finish_sums(const KvAttnArgs &a, int64_t row, float m, float l) {
    const float ln2 = 0.693147180559945309f;
    if (a.lse) a.lse[row] = l != 0.f ? (m + log2f(l)) * ln2 : -INFINITY;
    if (a.ml) a.ml[row] = l != 0.f ? make_float2(m * ln2, l) : make_float2(-INFINITY, 0.f);
}

// Channels 4 lane .. of one finished row: normalised output; lane 0 adds the sums
template <typename T>
__device__ __forceinline__ void ka_finish(const KvAttnArgs &a, int64_t row, int lane, float4 o, float m, float l) {
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4 *>(a.out)[row * (D / 4) + lane] = o;
    } else {
        const __nv_bfloat162 x = __floats2bfloat162_rn(o.x, o.y), y = __floats2bfloat162_rn(o.z, o.w);
        reinterpret_cast<uint2 *>(a.out)[row * (D / 4) + lane] =
            make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
    }
    if (lane == 0) ka_finish_sums(a, row, m, l);
}

template <typename T, int DT, int NT, bool SEL, bool OWN>
__global__ void __launch_bounds__(32 * KaShape<NT>::WARPS, KaShape<NT>::CTAS) k_kv_attn(const __grid_constant__ KvAttnArgs a) {
    using Sm = KaSmem<T, DT, NT>;
    using Tl = KaTile<DT>;
    constexpr int RPT = Sm::RPT, PARTS = Sm::PARTS, KA_WARPS = Sm::KA_WARPS;
    constexpr int KA_BEGIN = KaShape<NT>::BEGIN;
    constexpr bool PAR = DT != MILO_INT4;                    // a scale per row
    static_assert(PAR || !OWN, "only scales per row have an E");
    constexpr int EN = OWN ? NT : 1, EX = OWN ? 2 : 1;       // its values: the lane's query rows, or one
    extern __shared__ __align__(16) unsigned char ka_raw[];
    Sm &sm = *reinterpret_cast<Sm *>(ka_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    KaRun<SEL, NT> run;
    const bool any_work = run.begin(a, sm.scan);
    if (tid == 0) a.split[blockIdx.x] = make_int4(-1, 0, 0, 0);
    kv_launch_next();
    if (!any_work) return;
    const KaClass<SEL, NT> &cl = run.cl;
    float *const my_o = reinterpret_cast<float *>(sm.ring[warp]);
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(sm.ring[warp]);

    while (run.u0 < run.u1) {
        const int s0 = run.s0(), s1 = run.s1(), l = run.l, h = run.h;
        const int64_t sh = (int64_t)cl.s * a.c.H + h;
        const KaLine<DT> ln(a.c.codes(l, sh, 0), a.c.codes(l, sh, 1), a.c.params(l, sh, 0), a.c.params(l, sh, 1), lane);
        const int32_t *sel = SEL ? a.sel + ((((int64_t)l * a.c.S + cl.s) * a.n_q + cl.i) * a.c.H + h) * a.n_sel : nullptr;
        // the line's queries, a warp per row (RPT / KA_WARPS rows each): asked for before the codes
        float qx[RPT / KA_WARPS][4];
#pragma unroll
        for (int y = 0; y < RPT / KA_WARPS; ++y) {
            const int r = warp + y * KA_WARPS;
            const T *q = (const T *)a.q + cl.row(a, l, h, min(r, cl.rows - 1)) * D + 4 * lane;
            T t[4];                                          // 16 or 8 bytes
            if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4 *>(t) = __ldg(reinterpret_cast<const uint4 *>(q));
            else *reinterpret_cast<uint2 *>(t) = __ldg(reinterpret_cast<const uint2 *>(q));
#pragma unroll
            for (int e = 0; e < 4; ++e) qx[y][e] = r < cl.rows ? to_f32(t[e]) : 0.f;
        }
        // the segment's tiles, an equal run of them to each warp: `left` of them, fetched a few ahead of their use
        const int first = max(s0 - KA_BEGIN, 0) * KA_WARPS;
        const int tiles = max(min(cl.tiles(a), (s1 - KA_BEGIN) * KA_WARPS) - first, 0);
        const int mine0 = first + (int)((int64_t)tiles * warp / KA_WARPS);
        int left = first + (int)((int64_t)tiles * (warp + 1) / KA_WARPS) - mine0;
        int to_fetch = left, t_next = 16 * mine0;            // selected: block `id`, its tile `in`, the block after it
        int in = 0, slot = 0, id = -1, id_next = -1;
        auto block_at = [&](int x) {
            const int b = x < a.n_sel ? __ldg(sel + x) : -1;
            if (b >= 0 && b < a.c.n_b) return b;
            if (b != -1 && lane == 0) raise_status(ST_BOUNDS);
            return -1;
        };
        if (SEL) {
            slot = mine0 / a.tpb;
            in = mine0 - slot * a.tpb;
            id = left > 0 ? block_at(slot) : -1;
            id_next = left > a.tpb - in ? block_at(slot + 1) : -1;
        }
        constexpr int AHEAD = Tl::STAGES - 1, NONE = 0x7fffff00;
        auto fetch = [&](int stage) {
            int t0 = NONE;                                   // no tokens: every row is masked
            if (to_fetch > 0) {
                if (!SEL) {
                    t0 = t_next;
                    t_next += 16;
                } else {
                    if (id >= 0) t0 = (id * a.tpb + in) * 16;
                    if (++in == a.tpb) {
                        in = 0;
                        id = id_next;
                        ++slot;
                        id_next = to_fetch - 1 > a.tpb ? block_at(slot + 1) : -1;
                    }
                }
                --to_fetch;
            }
            const bool any = t0 < cl.end;
            ka_fetch<DT>(ring + stage * Tl::BYTES, ln, any ? t0 : 0, any ? cl.end - t0 : 0, lane);
            if (lane == 0) sm.t0[warp][stage] = any ? t0 : NONE;
            ka_commit();
        };
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) fetch(i);

        // the line's queries as fragments, a warp per row (RPT / KA_WARPS rows each)
#pragma unroll
        for (int y = 0; y < RPT / KA_WARPS; ++y) {
            const int r = warp + y * KA_WARPS;
            const float (&x)[4] = qx[y];
            float mx = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
            for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const int e = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 127);
            const float up = __uint_as_float((uint32_t)(135 - e) << 23), down = __uint_as_float((uint32_t)(119 + e) << 23);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int ch = 4 * lane + w;
                int j, cc, el;
                ka_place<DT>(ch, j, cc, el);
                const float z = isfinite(x[w]) ? x[w] * up : NAN;   // an infinity spoils its row's scores like a NaN
                const __half hi = __float2half_rn(z);
                __half *f = reinterpret_cast<__half *>(sm.q[r / 8][j][(r % 8) * 4 + cc]);
                f[el] = hi;
                if (PARTS == 2) f[4 + el] = __float2half_rn(z - __half2float(hi));
            }
            if (lane == 0) {
                sm.sc[r] = a.scale * (DT == MILO_FP8 ? KA_FP8_UP : 1.f) * down;
                // rows behind the last are zero queries that see what the others see
                sm.seen[r] = r < cl.rows ? cl.seen(a, r) : cl.end;
            }
        }
        __syncthreads();
        float sc[NT][2], off[NT][2], sum[NT][2], o[NT][8][4];   // off: -reference
        const int least = cl.seen(a, 0);                // tokens that every row sees
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                sc[n][x] = sm.sc[8 * n + 2 * c + x];
                off[n][x] = INFINITY;
                sum[n][x] = 0.f;
#pragma unroll
                for (int w = 0; w < 8; ++w) o[n][w][2 * x] = o[n][w][2 * x + 1] = 0.f;
            }
        float e_max[EN][EX], e_inv[EN][EX];                  // 2^E and 2^(10 - E) of the value scales so far
#pragma unroll
        for (int n = 0; n < EN; ++n)
#pragma unroll
            for (int x = 0; x < EX; ++x) e_max[n][x] = e_inv[n][x] = 0.f;

        for (int stage = 0; left > 0; --left) {
            ka_wait<AHEAD - 1>();
            __syncwarp();                                    // this tile is there, and the one before it used
            fetch(stage == 0 ? AHEAD : stage - 1);
            const unsigned char *st = sm.ring[warp] + stage * Tl::BYTES;
            const int t0 = sm.t0[warp][stage];
            stage = stage == AHEAD ? 0 : stage + 1;
            // scores: tokens ka_token(g) and ka_token(g + 8), queries 2c, 2c + 1 of each tile of 8
            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[n][x] = 0.f;
            KaKeys<DT> keys;
            ka_read_k<DT>(st, g, c, keys);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t f[4];
                ka_frag_k<DT>(keys, j, f);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if constexpr (PARTS == 2) {
                        const uint4 b = *reinterpret_cast<const uint4 *>(sm.q[n][j][lane]);
                        ka_mma(s[n], f[0], f[1], f[2], f[3], b.x, b.y);
                        ka_mma(s[n], f[0], f[1], f[2], f[3], b.z, b.w);
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
                    ks[r] = *reinterpret_cast<const float *>(st + Tl::KP + 4 * (g + 8 * r));
                    vs[r] = *reinterpret_cast<const float *>(st + Tl::VP + 4 * (g + 8 * r));
                }
            }
            // exponents of the weights, relative to the references
            float y[NT][4];
            bool raise = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float f = PAR ? ks[x / 2] * sc[n][x % 2] : sc[n][x % 2];
                    y[n][x] = fmaf(s[n][x], f, off[n][x % 2]);
                    if (t0 + 16 > least && t0 + ka_token<DT>(g + 8 * (x / 2)) >= sm.seen[8 * n + 2 * c + x % 2])
                        y[n][x] = -INFINITY;
                    raise |= y[n][x] > KA_RAISE;
                }
            if (__any_sync(0xffffffffu, raise)) {            // raise the references to this tile's maxima
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float s0 = y[n][x] == -INFINITY ? -INFINITY : s[n][x] * (PAR ? ks[0] * sc[n][x] : sc[n][x]);
                        const float s1 = y[n][2 + x] == -INFINITY ? -INFINITY : s[n][2 + x] * (PAR ? ks[1] * sc[n][x] : sc[n][x]);
                        const float old = -off[n][x];
                        float m = fmaxf(s0, s1);
#pragma unroll
                        for (int w = 4; w < 32; w <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
                        m = fmaxf(m, old);
                        const float f = old == -INFINITY ? 0.f : ka_exp2(old - m);
                        off[n][x] = -m;
                        if (y[n][x] != -INFINITY) y[n][x] = s0 + off[n][x];
                        if (y[n][2 + x] != -INFINITY) y[n][2 + x] = s1 + off[n][x];
                        sum[n][x] *= f;
#pragma unroll
                        for (int w = 0; w < 8; ++w) {
                            o[n][w][x] *= f;
                            o[n][w][2 + x] *= f;
                        }
                    }
            }
            const bool edge = OWN && t0 + 16 > least;        // some row does not see all of the tile, nor of those behind it
            if constexpr (PAR) {
                // 2^E of the greatest scale; a row's (n, x), or all rows' at once
                auto raise_e = [&](uint32_t top, int n0, int n1, int x0, int step) {
                    const float pw = __uint_as_float(min(max(top & 0x7f800000u, KA_E_MIN), 0x7e800000u));
                    float &e = e_max[OWN ? n0 : 0][OWN ? x0 : 0];
                    if (pw <= e) return;
                    const float f = e * (1.f / pw);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int w = 0; w < 8; ++w)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (n >= n0 && n < n1 && i % step == x0) o[n][w][i] *= f;
#pragma unroll
                    for (int n = 0; n < EN; ++n)
#pragma unroll
                        for (int x = 0; x < EX; ++x)
                            if (n >= n0 && n < n1 && x % step == x0) {
                                e_max[n][x] = pw;
                                e_inv[n][x] = KA_UP / pw;
                            }
                };
                if (!edge) {                                 // every row has seen the same so far
                    raise_e(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(vs[0], vs[1]))), 0, NT, 0, 1);
                    vs[0] *= e_inv[0][0];
                    vs[1] *= e_inv[0][0];
                } else {
#pragma unroll
                    for (int n = 0; n < EN; ++n)
#pragma unroll
                        for (int x = 0; x < EX; ++x) {
                            const float v = fmaxf(y[n][x] == -INFINITY ? 0.f : vs[0], y[n][2 + x] == -INFINITY ? 0.f : vs[1]);
                            uint32_t u = __float_as_uint(v);
#pragma unroll
                            for (int w = 4; w < 32; w <<= 1) u = max(u, __shfl_xor_sync(0xffffffffu, u, w));
                            raise_e(u, n, n + 1, x, 2);
                        }
                }
            }
            // weights, as fragments of the value product
            uint32_t b[NT][2][PARTS];
            auto weights = [&](auto at_edge) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float p[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        p[x] = ka_exp2(y[n][x]);
                        sum[n][x % 2] += p[x];
                        p[x] *= PAR ? vs[x / 2] : KA_UP;
                        // last: 0 for a token not seen, whatever its scale is
                        if constexpr (decltype(at_edge)::value) p[x] *= e_inv[n][x % 2];
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
            };
            if (OWN && edge) weights(std::integral_constant<bool, OWN>());
            else weights(std::false_type());
            KaValues<DT> vals;
            ka_read_v<DT>(st, g, c, vals);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t f[2][4];
                ka_frag_v<DT>(vals, w, f);
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int p = 0; p < PARTS; ++p)
                            ka_mma(o[n][2 * w + y], f[y][0], f[y][1], f[y][2], f[y][3], b[n][0][p], b[n][1][p]);
            }
        }
        ka_wait<0>();
        __syncwarp();                                        // the ring is free: the warp's output goes there

        // join the warps: reference and sum per query, then the outputs
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) sum[n][x] += __shfl_xor_sync(0xffffffffu, sum[n][x], w);
                const int r = 8 * n + 2 * c + x;
                if (g == 0) {
                    sm.m[warp][r] = -off[n][x];
                    sm.l[warp][r] = sum[n][x];
                    sm.e[warp][r] = PAR ? e_max[OWN ? n : 0][OWN ? x : 0] : 1.f;
                }
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    *reinterpret_cast<float4 *>(my_o + r * (D + 4) + 16 * g + 4 * w) =
                        make_float4(o[n][2 * w][x], o[n][2 * w][2 + x], o[n][2 * w + 1][x], o[n][2 * w + 1][2 + x]);
            }
        __syncthreads();
        const bool whole = s0 == 0 && s1 == run.per;
        const int64_t part = 2 * (int64_t)blockIdx.x + (s0 == 0 ? 1 : 0);
        if (tid < RPT) {                                     // each warp's share of a row
            float e_top = 0.f, m = -INFINITY, den = 0.f;
#pragma unroll
            for (int w = 0; w < KA_WARPS; ++w) {
                e_top = fmaxf(e_top, sm.e[w][tid]);
                m = fmaxf(m, sm.m[w][tid]);
            }
            float f[KA_WARPS];
#pragma unroll
            for (int w = 0; w < KA_WARPS; ++w) {
                f[w] = sm.l[w][tid] != 0.f ? ka_exp2(sm.m[w][tid] - m) : 0.f;   // 0: saw nothing
                den = fmaf(f[w], sm.l[w][tid], den);
            }
            const float inv = den != 0.f ? 1.f / den : 0.f, down = e_top > 0.f ? 1.f / e_top : 0.f;
#pragma unroll
            for (int w = 0; w < KA_WARPS; ++w) sm.m[w][tid] = f[w] * inv * (sm.e[w][tid] * down);
            sm.l[0][tid] = den;
            sm.sc[tid] = m;
            sm.e[KA_WARPS][tid] = e_top * ((DT == MILO_FP8 ? KA_FP8_UP : 1.f) / KA_UP);
        }
        __syncthreads();
        for (int r = warp; r < cl.rows; r += KA_WARPS) {     // a row per warp, four channels a lane
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < KA_WARPS; ++w) {
                const float f = sm.m[w][r];
                const float4 x = *reinterpret_cast<const float4 *>(sm.ring[w] + (r * (D + 4) + 4 * lane) * 4);
                y.x = fmaf(f, x.x, y.x);
                y.y = fmaf(f, x.y, y.y);
                y.z = fmaf(f, x.z, y.z);
                y.w = fmaf(f, x.w, y.w);
            }
            const float up = sm.e[KA_WARPS][r];
            y = make_float4(y.x * up, y.y * up, y.z * up, y.w * up);
            if (whole) ka_finish<T>(a, cl.row(a, l, h, r), lane, y, sm.sc[r], sm.l[0][r]);
            else {
                *reinterpret_cast<float4 *>(a.part_o + (part * RPT + r) * D + 4 * lane) = y;
                if (lane == 0) a.part_ml[part * RPT + r] = make_float2(sm.sc[r], sm.l[0][r]);
            }
        }
        if (!whole && s0 == 0 && tid == 0) a.split[blockIdx.x] = run.split();
        __syncthreads();                                     // queries and outputs used before the next segment
        run.next(a, s1);
    }
}

// Joins the parts of a line that CTA blockIdx.x begins, in their order.  Each of
// the gridDim.y CTAs takes 8 NT / gridDim.y of its rows, and the 16 / that many
// warps of a row take its parts in turn.
constexpr int KA_MERGE_WARPS = 16;
template <typename T, int NT, bool SEL>
__global__ void __launch_bounds__(32 * KA_MERGE_WARPS) k_kv_attn_merge(const __grid_constant__ KvAttnArgs a) {
    constexpr int RPT = 8 * NT;
    __shared__ float s_o[KA_MERGE_WARPS][D], s_l[KA_MERGE_WARPS], s_m[KA_MERGE_WARPS];
    kv_wait_previous();
    const int4 sp = a.split[blockIdx.x];
    if (sp.x < 0) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = RPT / gridDim.y, wpr = KA_MERGE_WARPS / per;     // rows of this CTA, warps of a row
    const int r = blockIdx.y * per + warp / wpr, w0 = warp % wpr;
    KaClass<SEL, NT> cl;
    cl.set(a, sp.x, false);
    const int n = sp.w - (int)blockIdx.x + 1;                // parts: slot 1 of the first CTA, slot 0 of the others
    auto at = [&](int i) { return (2 * ((int64_t)blockIdx.x + i) + (i == 0)) * RPT + r; };
    float m = -INFINITY, den = 0.f;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int BATCH = 4;
    for (int i0 = w0; i0 < n; i0 += BATCH * wpr) {
        float2 x[BATCH];
        float4 o[BATCH];
#pragma unroll
        for (int y = 0; y < BATCH; ++y) {
            const int i = i0 + y * wpr;
            x[y] = make_float2(-INFINITY, 0.f);
            o[y] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < n) {
                x[y] = a.part_ml[at(i)];                     // a sum of 0: an empty part, whose output may not be written
                o[y] = *reinterpret_cast<const float4 *>(a.part_o + at(i) * D + 4 * lane);
                if (x[y].y == 0.f) o[y] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        float top = m;
#pragma unroll
        for (int y = 0; y < BATCH; ++y)
            if (x[y].y != 0.f) top = fmaxf(top, x[y].x);
        const float f = den != 0.f ? ka_exp2(m - top) : 0.f;
        m = top;
        den *= f;
        num = make_float4(num.x * f, num.y * f, num.z * f, num.w * f);
#pragma unroll
        for (int y = 0; y < BATCH; ++y) {
            const float w = x[y].y != 0.f ? ka_exp2(x[y].x - m) * x[y].y : 0.f;
            den += w;
            num.x = fmaf(w, o[y].x, num.x);
            num.y = fmaf(w, o[y].y, num.y);
            num.z = fmaf(w, o[y].z, num.z);
            num.w = fmaf(w, o[y].w, num.w);
        }
    }
    if (lane == 0) s_m[warp] = m;
    *reinterpret_cast<float4 *>(&s_o[warp][4 * lane]) = num;
    if (lane == 0) s_l[warp] = den;
    __syncthreads();
    if (w0 == 0 && r < cl.rows) {
        float top = m;
        for (int w = 1; w < wpr; ++w) top = fmaxf(top, s_m[warp + w]);
        num = make_float4(0.f, 0.f, 0.f, 0.f);
        den = 0.f;
        for (int w = 0; w < wpr; ++w) {
            const float4 o = *reinterpret_cast<const float4 *>(&s_o[warp + w][4 * lane]);
            const float f = s_l[warp + w] != 0.f ? ka_exp2(s_m[warp + w] - top) : 0.f;
            num = make_float4(fmaf(f, o.x, num.x), fmaf(f, o.y, num.y), fmaf(f, o.z, num.z), fmaf(f, o.w, num.w));
            den = fmaf(f, s_l[warp + w], den);
        }
        m = top;
        const float inv = den != 0.f ? 1.f / den : 0.f;
        num = make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv);
        ka_finish<T>(a, cl.row(a, sp.y, sp.z, r), lane, num, m, den);
    }
}

}  // namespace milo

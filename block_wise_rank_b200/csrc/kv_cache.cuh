// kv_cache.cuh -- the quantised cache of recent tokens: rows quantised as they
// are written, the key bounds of each block, and rows read back.
//
// The layout and the arithmetic of the codes are milo.h's (milo_kv_shape).
// Every code is decided by IEEE fp32 operations on the stored parameters, the
// bounds by minima and maxima, so nothing depends on the order of the work.
//
// Writing takes 106496 bf16 rows of 4 heads into e4m3 in 76 us, 4.4 TB/s (with the
// division's subroutine 173 us).  No unit is full: issue slots 66 %, the busiest pipe (ALU)
// 45 %, DRAM 50 %.  16 channels take about 240 instructions, 64 of them the exact
// quotients, in dependent chains, and 80 registers leave 5.3 warps a scheduler: of the 8.0
// cycles between a warp's instructions 2.4 are fixed latencies, 1.4 another warp's turn, 1.0
// loads from memory, 0.7 shared memory.  fp32 rows into INT4 alike: issue 55 %, 3.6 warps, 6.5
// cycles, of them 1.8 fixed and 1.1 loads; that instance spills 76 bytes a thread (the
// others 16 to 52 with a warp an item).  Reading is bound by memory: the same rows back to
// bf16 in 53 us, 6.2 TB/s.
#pragma once
#include <cuda_fp8.h>

#include "common.cuh"

namespace milo {

constexpr int KV_GROUP = 32;                 // channels that share an INT4 scale and zero
constexpr int KV_NG = D / KV_GROUP;
// Greatest INT4 value: a group's highest value 15 s + z passes its maximum by 60 + 16 at most, the roundings of s
// (at most 8725) and z, and has to stay below 65520, which rounds past fp16's end
constexpr float KV_INT4_MAX = 65440.f;

// One layer-strided cache buffer.
struct KvView {
    unsigned char *base;
    int64_t layer;                           // bytes of a layer
    int64_t off[7];                          // sections (milo.h)
    int L, S, H, cap, block_len, n_b, dtype;

    __host__ __device__ __forceinline__ int row_bytes() const { return dtype == MILO_INT4 ? D / 2 : D; }
    __host__ __device__ __forceinline__ int par_bytes() const { return dtype == MILO_INT4 ? 4 * KV_NG : 4; }
    __device__ __forceinline__ unsigned char *section(int l, int i) const { return base + l * layer + off[i]; }
    // codes / parameters of row 0 of (l, s, h) of kind 0 (K) or 1 (V)
    __device__ __forceinline__ unsigned char *codes(int l, int64_t sh, int kind) const {
        return section(l, kind) + sh * cap * row_bytes();
    }
    __device__ __forceinline__ unsigned char *params(int l, int64_t sh, int kind) const {
        return section(l, 2 + kind) + sh * cap * par_bytes();
    }
};

// rows [start, start + n) of session s, or n = 0 and ST_BOUNDS if they leave the cache
__device__ __forceinline__ void kv_range(const int32_t *start, const int32_t *count, int s, int n_new, int cap,
                                         bool tell, int &st, int &n) {
    st = start[s];
    n = count ? count[s] : n_new;
    if (st < 0 || n < 0 || n > n_new || (int64_t)st + n > cap) {
        if (tell) raise_status(ST_BOUNDS);
        n = 0;
    }
}

// 16 consecutive elements, raw and as fp32
template <typename T> struct KvRaw {
    uint4 w[sizeof(T)];
};
template <typename T> __device__ __forceinline__ KvRaw<T> kv_raw16(const T *p) {
    KvRaw<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) r.w[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
    return r;
}
// the bits of the greatest magnitude, as an fp32's (above 0x7f7fffff: not finite)
template <typename T> __device__ __forceinline__ uint32_t kv_top(const KvRaw<T> &r) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(r.w);
    uint32_t top = 0u;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 16; ++i) top = max(top, w[i] & 0x7fffffffu);
        return top;
    } else {   // two values an instruction
#pragma unroll
        for (int i = 0; i < 8; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
        return max(top & 0xffff0000u, top << 16);
    }
}
template <typename T> __device__ __forceinline__ void kv_f32(const KvRaw<T> &r, float (&x)[16]) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(r.w);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if constexpr (sizeof(T) == 4) x[i] = __uint_as_float(w[i]);
        else x[i] = __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
}

// x / s rounded like an IEEE division, from inv = 1 / s rounded: by Markstein
// ("Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990), one step q + (x - q s) inv of a quotient q within one place of x / s
// rounds it correctly when the remainder is exact.  The first step brings x inv,
// at most 1.5 places off, to within one.  Holds while no remainder that
// matters for a code underflows: 2^-60 < s < 2^100 (|x| <= 448 s, codes from 2^-10 on).
__device__ __forceinline__ float kv_quotient(float x, float s, float inv) {
    float q = x * inv;
    q = fmaf(fmaf(-q, s, x), inv, q);
    return fmaf(fmaf(-q, s, x), inv, q);
}
__device__ __forceinline__ bool kv_plain_scale(float s) { return s > 0x1p-60f && s < 0x1p100f; }
// x / n for a constant n
template <int N> __device__ __forceinline__ float kv_over(float x) {
    return x > 0x1p-60f ? kv_quotient(x, (float)N, 1.f / (float)N) : __fdiv_rn(x, (float)N);
}
// x[i] / s for every i; 0 where s is 0
template <int N> __device__ __forceinline__ void kv_divide(float (&x)[N], float s) {
    if (kv_plain_scale(s)) {
        const float inv = __frcp_rn(s);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = kv_quotient(x[i], s, inv);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = s > 0.f ? __fdiv_rn(x[i], s) : 0.f;
    }
}
constexpr float KV_MAGIC = 12582912.f;   // 1.5 * 2^23: the low bits of x + KV_MAGIC are the integer nearest to x, ties to even

// the low bytes of four words
__device__ __forceinline__ uint32_t kv_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
// INT8 codes of quotients within 127.5
template <int N> __device__ __forceinline__ void kv_int8(const float (&q)[N], uint32_t (&w)[N / 4]) {
    uint32_t r[N];
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = __float_as_uint(q[i] + KV_MAGIC);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) w[i] = kv_bytes(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
}

// Quantise a lane's 16 channels (lane j of 8 holds channels 16 j ..) of one row
// and store its codes and parameters where the row is `live`.  The whole warp calls it together.
template <int DT>
__device__ __forceinline__ void kv_quant_store(const float (&x)[16], float amax, int j, bool live,
                                               unsigned char *codes, unsigned char *par) {
    constexpr unsigned mask = 0xffffffffu;
    if constexpr (DT == MILO_INT4) {
        float lo = x[0], hi = x[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) {
            lo = fminf(lo, x[i]);
            hi = fmaxf(hi, x[i]);
        }
        lo = fminf(lo, __shfl_xor_sync(mask, lo, 1));
        hi = fmaxf(hi, __shfl_xor_sync(mask, hi, 1));
        const __half z = __float2half_rn(lo), s = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
        const float zf = __half2float(z), sf = __half2float(s);
        float q[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) q[i] = __fsub_rn(x[i], zf);
        kv_divide<16>(q, sf);
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int i = 0; i < 16; ++i)   // clamped before it is rounded: the same code, and within the trick's range
            w[i / 8] |= (__float_as_uint(fminf(fmaxf(q[i], 0.f), 15.f) + KV_MAGIC) & 15u) << (4 * (i % 8));
        if (live) reinterpret_cast<uint2 *>(codes)[j] = make_uint2(w[0], w[1]);
        if (live && j % 2 == 0) reinterpret_cast<__half2 *>(par)[j / 2] = __halves2half2(s, z);
    } else {
        amax = fmaxf(amax, __shfl_xor_sync(mask, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(mask, amax, 2));
        amax = fmaxf(amax, __shfl_xor_sync(mask, amax, 4));
        const float s = kv_over<DT == MILO_INT8 ? 127 : 448>(amax);
        float q[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) q[i] = x[i];
        kv_divide<16>(q, s);
        uint32_t w[4];
        if constexpr (DT == MILO_INT8) {
            if (s < 0x1p-100f) {   // a scale with few bits left: 127 can be passed
#pragma unroll
                for (int i = 0; i < 16; ++i) q[i] = fminf(fmaxf(q[i], -127.f), 127.f);
            }
            kv_int8<16>(q, w);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * i], q[4 * i + 1]), __NV_SATFINITE, __NV_E4M3) |
                       (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(q[4 * i + 2], q[4 * i + 3]), __NV_SATFINITE,
                                                          __NV_E4M3) << 16;
        }
        if (live) reinterpret_cast<uint4 *>(codes)[j] = make_uint4(w[0], w[1], w[2], w[3]);
        if (live && j == 0) *reinterpret_cast<float *>(par) = s;
    }
}

// fp32 rounded to bf16 away from zero's side it must not cross: down / up, finite
__device__ __forceinline__ __nv_bfloat16 kv_outward(float x, bool up) {
    const float m = 3.3895313892515355e38f;   // greatest finite bf16
    const __nv_bfloat16 b = up ? __float2bfloat16_ru(x) : __float2bfloat16_rd(x);
    return __float2bfloat16_rn(fminf(fmaxf(__bfloat162float(b), -m), m));
}

struct KvAppendArgs {
    KvView c;
    const void *k, *v;
    int64_t sl, ss, sh, st;                  // strides of k and v in elements
    int n_new, windows;                      // blocks of block_len that a range can touch
    int items;                               // windows * S * H * L * 2
    const int32_t *start, *count;
};

// A running channelwise minimum and maximum of 16 channels, in the elements' own type
template <typename T> struct KvBounds;
template <> struct KvBounds<float> {
    float lo[16], hi[16];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            lo[i] = INFINITY;
            hi[i] = -INFINITY;
        }
    }
    __device__ __forceinline__ void add(const KvRaw<float> &, const float (&x)[16]) { add(x); }
    __device__ __forceinline__ void add(const float (&x)[16]) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            lo[i] = fminf(lo[i], x[i]);
            hi[i] = fmaxf(hi[i], x[i]);
        }
    }
    __device__ __forceinline__ void get(float (&l)[16], float (&h)[16]) const {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            l[i] = lo[i];
            h[i] = hi[i];
        }
    }
};
template <> struct KvBounds<__nv_bfloat16> {   // two channels an instruction
    __nv_bfloat162 lo[8], hi[8];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo[i] = __float2bfloat162_rn(INFINITY);
            hi[i] = __float2bfloat162_rn(-INFINITY);
        }
    }
    __device__ __forceinline__ void add(const KvRaw<__nv_bfloat16> &r, const float (&)[16]) {
        const __nv_bfloat162 *v = reinterpret_cast<const __nv_bfloat162 *>(r.w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo[i] = __hmin2(lo[i], v[i]);
            hi[i] = __hmax2(hi[i], v[i]);
        }
    }
    __device__ __forceinline__ void add(const float (&x)[16]) {   // x are bf16 values, or +-65440: rounded outward
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const __nv_bfloat162 d = __halves2bfloat162(__float2bfloat16_rd(x[2 * i]), __float2bfloat16_rd(x[2 * i + 1]));
            const __nv_bfloat162 u = __halves2bfloat162(__float2bfloat16_ru(x[2 * i]), __float2bfloat16_ru(x[2 * i + 1]));
            lo[i] = __hmin2(lo[i], d);
            hi[i] = __hmax2(hi[i], u);
        }
    }
    __device__ __forceinline__ void get(float (&l)[16], float (&h)[16]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 a = __bfloat1622float2(lo[i]), b = __bfloat1622float2(hi[i]);
            l[2 * i] = a.x;
            l[2 * i + 1] = a.y;
            h[2 * i] = b.x;
            h[2 * i + 1] = b.y;
        }
    }
};

constexpr int KV_APPEND_WARPS = 4;

// An item is the new tokens of one block of one (layer, session, KV head) and
// kind (kind slowest, then layer, session, head, window).  WPI warps quantise it,
// four rows a warp at a time, eight lanes a row with 16 channels each; for keys the
// channelwise minima and maxima of the 4 WPI row groups are then joined in shared
// memory, CPT channels a thread.  One token a block leaves three quarters of a
// warp idle, so then a warp takes an item (WPI = 1); otherwise a CTA does.
template <typename T, int DT, int WPI>
__global__ void __launch_bounds__(32 * KV_APPEND_WARPS, sizeof(T) == 4 ? 5 : 6) k_kv_append(KvAppendArgs a) {
    constexpr int CPT = D / (32 * WPI), ITEMS = KV_APPEND_WARPS / WPI;
    __shared__ __align__(16) float s_b[ITEMS][2][4 * WPI][D];   // [item][min, max][row group][channel]
    __shared__ float s_amax[KV_APPEND_WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wi = WPI > 1 ? warp : 0, item = WPI > 1 ? 0 : warp;   // warp of the item, item of the CTA
    int id = blockIdx.x * ITEMS + item;
    if (id >= a.items) return;
    const int win = id % a.windows;
    id /= a.windows;
    const int h = id % a.c.H;
    id /= a.c.H;
    const int s = id % a.c.S;
    id /= a.c.S;
    const int l = id % a.c.L, kind = id / a.c.L;
    int start, n;
    kv_range(a.start, a.count, s, a.n_new, a.c.cap, lane == 0 && h == 0 && l == 0 && win == 0 && kind == 0, start, n);
    const int b = start / a.c.block_len + win;
    const int t0 = max(start, b * a.c.block_len), t1 = min(start + n, (b + 1) * a.c.block_len);   // tokens written here
    if (n == 0 || t0 >= t1) return;
    const int64_t sh = (int64_t)s * a.c.H + h;
    const int j = lane & 7, group = lane >> 3;
    const T *x = (const T *)(kind ? a.v : a.k) + l * a.sl + s * a.ss + h * a.sh + 16 * j - start * a.st;
    constexpr int ROW = DT == MILO_INT4 ? D / 2 : D, PAR = DT == MILO_INT4 ? 4 * KV_NG : 4;
    unsigned char *codes = a.c.codes(l, sh, kind), *par = a.c.params(l, sh, kind);
    int t = t0 + 4 * wi + group;
    KvRaw<T> next{};
    if (t < t1) next = kv_raw16<T>(x + (int64_t)t * a.st);
    // bounds that a continued block has, of this thread's channels
    const int64_t blk = sh * a.c.n_b + b;
    const int ch = (32 * wi + lane) * CPT;
    __nv_bfloat16 *held = (__nv_bfloat16 *)a.c.section(l, 4) + blk * 2 * D + ch;
    const bool goes_on = kind == 0 && start > b * a.c.block_len;
    float lo[CPT], hi[CPT];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        lo[i] = goes_on ? __bfloat162float(held[i]) : INFINITY;
        hi[i] = goes_on ? __bfloat162float(held[D + i]) : -INFINITY;
    }
    KvBounds<T> bounds;
    bounds.clear();
    bool bad = false;
    for (; t - group < t1; t += 4 * WPI) {                   // the whole warp, rows behind the last with what was there
        const bool live = t < t1;
        const KvRaw<T> raw = next;
        float r[16];
        kv_f32<T>(raw, r);
        if (t + 4 * WPI < t1) next = kv_raw16<T>(x + (int64_t)(t + 4 * WPI) * a.st);
        uint32_t top = kv_top<T>(raw);
        if (live && top > __float_as_uint(DT == MILO_INT4 ? KV_INT4_MAX : 3.402823466e38f)) {
            bad = true;
            top = 0u;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (!isfinite(r[i])) r[i] = 0.f;
                if (DT == MILO_INT4 && fabsf(r[i]) > KV_INT4_MAX) r[i] = copysignf(KV_INT4_MAX, r[i]);
                top = max(top, __float_as_uint(r[i]) & 0x7fffffffu);
            }
            if (kind == 0) bounds.add(r);
        } else if (kind == 0 && live) {
            bounds.add(raw, r);
        }
        kv_quant_store<DT>(r, __uint_as_float(top), j, live, codes + (int64_t)t * ROW, par + (int64_t)t * PAR);
    }
    if (bad) raise_status(ST_NONFINITE);
    if (kind == 1) return;
    {
        float l16[16], h16[16];
        bounds.get(l16, h16);
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            *reinterpret_cast<float4 *>(&s_b[item][0][4 * wi + group][16 * j + i]) =
                make_float4(l16[i], l16[i + 1], l16[i + 2], l16[i + 3]);
            *reinterpret_cast<float4 *>(&s_b[item][1][4 * wi + group][16 * j + i]) =
                make_float4(h16[i], h16[i + 1], h16[i + 2], h16[i + 3]);
        }
    }
    if (WPI > 1) __syncthreads();
    else __syncwarp();
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
#pragma unroll
        for (int g = 0; g < 4 * WPI; ++g) {
            lo[i] = fminf(lo[i], s_b[item][0][g][ch + i]);
            hi[i] = fmaxf(hi[i], s_b[item][1][g][ch + i]);
        }
        const __nv_bfloat16 bl = kv_outward(lo[i], false), bh = kv_outward(hi[i], true);
        held[i] = bl;
        held[D + i] = bh;
        lo[i] = __bfloat162float(bl);
        hi[i] = __bfloat162float(bh);
        m = fmaxf(m, fmaxf(fabsf(lo[i]), fabsf(hi[i])));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (WPI > 1) {
        if (lane == 0) s_amax[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WPI; ++w) m = fmaxf(m, s_amax[w]);
    }
    const float sc = __fdiv_rn(m, 127.f);
    int8_t *bcodes = (int8_t *)a.c.section(l, 5) + blk * 2 * D + ch;
    kv_divide<CPT>(lo, sc);
    kv_divide<CPT>(hi, sc);
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        bcodes[i] = (int8_t)(int)rintf(fminf(fmaxf(lo[i], -127.f), 127.f));
        bcodes[D + i] = (int8_t)(int)rintf(fminf(fmaxf(hi[i], -127.f), 127.f));
    }
    if (wi == 0 && lane == 0) ((float *)a.c.section(l, 6))[blk] = sc;
}

// What a thread reads of one row: N channels' codes and their parameters
template <int DT, int N> struct KvCodes {
    uint32_t w[DT == MILO_INT4 ? (N + 7) / 8 : N / 4];
    uint32_t p;                              // the scale's bits, or (scale, zero) of the channels' group

    __device__ __forceinline__ void load(const unsigned char *codes, const unsigned char *par, int ch) {
        if constexpr (DT == MILO_INT4) {
            if constexpr (N == 8) w[0] = __ldg(reinterpret_cast<const uint32_t *>(codes) + ch / 8);
            else w[0] = __ldg(reinterpret_cast<const uint16_t *>(codes) + ch / 4);
            p = __ldg(reinterpret_cast<const uint32_t *>(par) + ch / KV_GROUP);
        } else {
            if constexpr (N == 8) {
                const uint2 u = __ldg(reinterpret_cast<const uint2 *>(codes) + ch / 8);
                w[0] = u.x;
                w[1] = u.y;
            } else {
                w[0] = __ldg(reinterpret_cast<const uint32_t *>(codes) + ch / 4);
            }
            p = __ldg(reinterpret_cast<const uint32_t *>(par));
        }
    }
    __device__ __forceinline__ void get(float (&x)[N]) const {
        if constexpr (DT == MILO_INT4) {
            const __half2 sz = *reinterpret_cast<const __half2 *>(&p);
#pragma unroll
            for (int i = 0; i < N; ++i)
                x[i] = __half2float(__hfma(__ushort2half_rn((unsigned short)((w[i / 8] >> (4 * (i % 8))) & 15u)),
                                           __low2half(sz), __high2half(sz)));
        } else if constexpr (DT == MILO_INT8) {
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = __fmul_rn((float)(int8_t)(w[i / 4] >> (8 * (i % 4))), __uint_as_float(p));
        } else {   // an e4m3's fields as an fp16's: the value times 2^-8, exactly
            const float s8 = __uint_as_float(p) * 256.f;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const uint32_t v = __byte_perm(w[i / 2], 0u, i % 2 ? 0x3424 : 0x1404);
                const uint32_t h = (v & 0x80008000u) | ((v >> 1) & 0x3f803f80u);
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                x[2 * i] = __fmul_rn(f.x, s8);
                x[2 * i + 1] = __fmul_rn(f.y, s8);
            }
        }
    }
};

struct KvReadArgs {
    KvView c;
    void *k, *v;                             // [L][S][H][n][D] or null
    int n, tiles;                            // tiles of KV_READ_ROWS rows of a session's n
    const int32_t *start, *count;
};

constexpr int KV_READ_ROWS = 64;

// grid (L S H tiles, 2 kinds), 256 threads.  A thread writes 16 bytes of a row, so
// that the rows' threads write it in one piece, and takes several rows, whose
// reads are issued together.
template <typename T, int DT> __global__ void __launch_bounds__(256) k_kv_read(KvReadArgs a) {
    constexpr int N = 16 / (int)sizeof(T), PER = D / N;       // channels of a thread, threads of a row
    constexpr int STEP = 256 / PER, TAKE = KV_READ_ROWS / STEP;
    constexpr int ROW = DT == MILO_INT4 ? D / 2 : D, PAR = DT == MILO_INT4 ? 4 * KV_NG : 4;
    const int kind = blockIdx.y;
    T *out = (T *)(kind ? a.v : a.k);
    if (!out) return;
    const int tile = blockIdx.x % a.tiles, lsh = blockIdx.x / a.tiles;
    const int SH = a.c.S * a.c.H, l = lsh / SH, sh = lsh % SH, s = sh / a.c.H;
    const int tid = threadIdx.x, ch = N * (tid % PER);
    int start, n;
    kv_range(a.start, a.count, s, a.n, a.c.cap, tid == 0 && tile == 0 && l == 0 && sh % a.c.H == 0, start, n);
    const int i0 = tile * KV_READ_ROWS + tid / PER;
    const unsigned char *codes = a.c.codes(l, sh, kind) + (int64_t)(start + i0) * ROW;
    const unsigned char *par = a.c.params(l, sh, kind) + (int64_t)(start + i0) * PAR;
    out += ((int64_t)lsh * a.n + i0) * D + ch;
    KvCodes<DT, N> c[TAKE];
#pragma unroll
    for (int y = 0; y < TAKE; ++y)
        if (i0 + STEP * y < n) c[y].load(codes + STEP * y * ROW, par + STEP * y * PAR, ch);
#pragma unroll
    for (int y = 0; y < TAKE; ++y) {
        if (i0 + STEP * y < n) {
            float x[N];
            c[y].get(x);
            uint4 w;
            if constexpr (sizeof(T) == 4) {
                w = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
            } else {
                __nv_bfloat162 b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) b[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w = *reinterpret_cast<const uint4 *>(b);
            }
            *reinterpret_cast<uint4 *>(out + (int64_t)STEP * y * D) = w;
        }
    }
}

}  // namespace milo

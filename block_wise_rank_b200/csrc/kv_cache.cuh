// kv_cache.cuh -- the quantised cache of recent tokens: rows quantised as they
// are written, the key bounds of each block, and rows read back.
//
// The layout and the arithmetic of the codes are milo.h's (milo_kv_shape).
// Every code is decided by IEEE fp32 operations on the stored parameters, the
// bounds by minima and maxima, so nothing depends on the order of the work.
#pragma once
#include <cuda_fp8.h>

#include "common.cuh"

namespace milo {

constexpr int KV_GROUP = 32;                 // channels that share an INT4 scale and zero
constexpr int KV_NG = D / KV_GROUP;
constexpr float KV_F16_MAX = 65504.f;

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

// 16 consecutive elements as fp32
template <typename T> __device__ __forceinline__ void kv_load16(const T *p, float (&x)[16]) {
    constexpr int N = (int)sizeof(T);        // 16-byte vectors
    uint4 w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
    const T *e = reinterpret_cast<const T *>(w);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = to_f32(e[i]);
}

template <typename T> __device__ __forceinline__ void kv_store16(T *p, const float (&x)[16]) {
    constexpr int N = (int)sizeof(T);
    uint4 w[N];
    T *e = reinterpret_cast<T *>(w);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if constexpr (sizeof(T) == 4) e[i] = x[i];
        else e[i] = __float2bfloat16_rn(x[i]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) reinterpret_cast<uint4 *>(p)[i] = w[i];
}

// Quantise a lane's 16 channels (lane j of 8 holds channels 16 j ..) of one row
// and store its codes and parameters.  All 8 lanes of the row call it together.
template <int DT>
__device__ __forceinline__ void kv_quant_store(const float (&x)[16], int j, unsigned mask, unsigned char *codes,
                                               unsigned char *par) {
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
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float c = sf > 0.f ? rintf(__fdiv_rn(__fsub_rn(x[i], zf), sf)) : 0.f;
            w[i / 8] |= (uint32_t)fminf(fmaxf(c, 0.f), 15.f) << (4 * (i % 8));
        }
        reinterpret_cast<uint2 *>(codes)[j] = make_uint2(w[0], w[1]);
        if (j % 2 == 0) reinterpret_cast<__half2 *>(par)[j / 2] = __halves2half2(s, z);
    } else {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(x[i]));
        m = fmaxf(m, __shfl_xor_sync(mask, m, 1));
        m = fmaxf(m, __shfl_xor_sync(mask, m, 2));
        m = fmaxf(m, __shfl_xor_sync(mask, m, 4));
        const float s = __fdiv_rn(m, DT == MILO_INT8 ? 127.f : 448.f);
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float c = s > 0.f ? __fdiv_rn(x[i], s) : 0.f;
            uint32_t b;
            if constexpr (DT == MILO_INT8) b = (uint32_t)(int)fminf(fmaxf(rintf(c), -127.f), 127.f) & 0xffu;
            else b = __nv_cvt_float_to_fp8(c, __NV_SATFINITE, __NV_E4M3);
            w[i / 4] |= b << (8 * (i % 4));
        }
        reinterpret_cast<uint4 *>(codes)[j] = make_uint4(w[0], w[1], w[2], w[3]);
        if (j == 0) *reinterpret_cast<float *>(par) = s;
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
    const int32_t *start, *count;
};

constexpr int KV_APPEND_WARPS = 4;

// grid: windows * S * H * L * 2 CTAs (kind slowest, then layer, head, window).
// A CTA quantises the new tokens of one block of one (layer, session, KV head)
// and kind, four rows a warp at a time, eight lanes a row; for keys it then
// joins the channelwise minima and maxima and writes the block's bounds.
template <typename T, int DT>
__global__ void __launch_bounds__(32 * KV_APPEND_WARPS) k_kv_append(KvAppendArgs a) {
    __shared__ float s_mn[KV_APPEND_WARPS][D], s_mx[KV_APPEND_WARPS][D], s_amax[KV_APPEND_WARPS];
    int64_t id = blockIdx.x;
    const int win = (int)(id % a.windows);
    id /= a.windows;
    const int h = (int)(id % a.c.H);
    id /= a.c.H;
    const int s = (int)(id % a.c.S);
    id /= a.c.S;
    const int l = (int)(id % a.c.L), kind = (int)(id / a.c.L);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int start, n;
    kv_range(a.start, a.count, s, a.n_new, a.c.cap, tid == 0 && h == 0 && l == 0 && win == 0 && kind == 0, start, n);
    const int b = start / a.c.block_len + win;
    const int t0 = max(start, b * a.c.block_len), t1 = min(start + n, (b + 1) * a.c.block_len);   // tokens written here
    if (n == 0 || t0 >= t1) return;
    const int64_t sh = (int64_t)s * a.c.H + h;
    const T *x = (const T *)(kind ? a.v : a.k) + l * a.sl + s * a.ss + h * a.sh;
    unsigned char *codes = a.c.codes(l, sh, kind), *par = a.c.params(l, sh, kind);
    const int j = lane & 7;
    const unsigned mask = 0xffu << (lane & 24);
    float mn[16], mx[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        mn[i] = INFINITY;
        mx[i] = -INFINITY;
    }
    bool bad = false;
    for (int t = t0 + 4 * warp + (lane >> 3); t < t1; t += 4 * KV_APPEND_WARPS) {
        float r[16];
        kv_load16<T>(x + (int64_t)(t - start) * a.st + 16 * j, r);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (!isfinite(r[i])) {
                bad = true;
                r[i] = 0.f;
            }
            if (DT == MILO_INT4 && fabsf(r[i]) > KV_F16_MAX) {
                bad = true;
                r[i] = copysignf(KV_F16_MAX, r[i]);
            }
            mn[i] = fminf(mn[i], r[i]);
            mx[i] = fmaxf(mx[i], r[i]);
        }
        kv_quant_store<DT>(r, j, mask, codes + (int64_t)t * a.c.row_bytes(), par + (int64_t)t * a.c.par_bytes());
    }
    if (bad) raise_status(ST_NONFINITE);
    if (kind == 1) return;
    // channel 16 j + i over the four rows of a warp, then over the warps
#pragma unroll
    for (int i = 0; i < 16; ++i) {
#pragma unroll
        for (int o = 8; o < 32; o <<= 1) {
            mn[i] = fminf(mn[i], __shfl_xor_sync(0xffffffffu, mn[i], o));
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], o));
        }
        if (lane < 8) {
            s_mn[warp][16 * j + i] = mn[i];
            s_mx[warp][16 * j + i] = mx[i];
        }
    }
    __syncthreads();
    const int64_t blk = sh * a.c.n_b + b;
    __nv_bfloat16 *bounds = (__nv_bfloat16 *)a.c.section(l, 4) + blk * 2 * D;
    int8_t *bcodes = (int8_t *)a.c.section(l, 5) + blk * 2 * D;
    float lo = s_mn[0][tid], hi = s_mx[0][tid];
#pragma unroll
    for (int w = 1; w < KV_APPEND_WARPS; ++w) {
        lo = fminf(lo, s_mn[w][tid]);
        hi = fmaxf(hi, s_mx[w][tid]);
    }
    if (start > b * a.c.block_len) {   // a block that is continued keeps what it had
        lo = fminf(lo, __bfloat162float(bounds[tid]));
        hi = fmaxf(hi, __bfloat162float(bounds[D + tid]));
    }
    const __nv_bfloat16 blo = kv_outward(lo, false), bhi = kv_outward(hi, true);
    bounds[tid] = blo;
    bounds[D + tid] = bhi;
    const float flo = __bfloat162float(blo), fhi = __bfloat162float(bhi);
    float m = fmaxf(fabsf(flo), fabsf(fhi));
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) s_amax[warp] = m;
    __syncthreads();
    for (int w = 0; w < KV_APPEND_WARPS; ++w) m = fmaxf(m, s_amax[w]);
    const float sc = __fdiv_rn(m, 127.f);
    bcodes[tid] = sc > 0.f ? (int8_t)fminf(fmaxf(rintf(__fdiv_rn(flo, sc)), -127.f), 127.f) : (int8_t)0;
    bcodes[D + tid] = sc > 0.f ? (int8_t)fminf(fmaxf(rintf(__fdiv_rn(fhi, sc)), -127.f), 127.f) : (int8_t)0;
    if (tid == 0) ((float *)a.c.section(l, 6))[blk] = sc;
}

// the value of a lane's 16 channels (16 j ..) of one row
template <int DT>
__device__ __forceinline__ void kv_dequant16(const unsigned char *codes, const unsigned char *par, int j,
                                             float (&x)[16]) {
    if constexpr (DT == MILO_INT4) {
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(codes) + j);
        const __half2 p = __ldg(reinterpret_cast<const __half2 *>(par) + j / 2);   // (scale, zero)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t c = ((i < 8 ? w.x : w.y) >> (4 * (i % 8))) & 15u;
            x[i] = __half2float(__hfma(__ushort2half_rn((unsigned short)c), __low2half(p), __high2half(p)));
        }
    } else {
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(codes) + j);
        const float s = __ldg(reinterpret_cast<const float *>(par));
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t c = (u[i / 4] >> (8 * (i % 4))) & 0xffu;
            float v;
            if constexpr (DT == MILO_INT8) v = (float)(int8_t)c;
            else v = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3)));
            x[i] = __fmul_rn(v, s);
        }
    }
}

struct KvReadArgs {
    KvView c;
    void *k, *v;                             // [L][S][H][n][D] or null
    int n;
    const int32_t *start, *count;
    int64_t rows;                            // L * S * H * n
};

// grid (ceil(rows * 8 / 256), 2 kinds), 256 threads: eight threads a row
template <typename T, int DT> __global__ void __launch_bounds__(256) k_kv_read(KvReadArgs a) {
    const int kind = blockIdx.y;
    T *out = (T *)(kind ? a.v : a.k);
    if (!out) return;
    const int64_t gid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, row = gid >> 3;
    if (row >= a.rows) return;
    const int j = (int)(gid & 7);
    const int i = (int)(row % a.n);
    const int64_t lsh = row / a.n;
    const int64_t SH = (int64_t)a.c.S * a.c.H;
    const int l = (int)(lsh / SH);
    const int64_t sh = lsh % SH;
    const int s = (int)(sh / a.c.H);
    int start, n;
    kv_range(a.start, a.count, s, a.n, a.c.cap, i == 0 && j == 0 && l == 0 && sh % a.c.H == 0, start, n);
    if (i >= n) return;
    const int64_t t = (int64_t)start + i;
    float x[16];
    kv_dequant16<DT>(a.c.codes(l, sh, kind) + t * a.c.row_bytes(), a.c.params(l, sh, kind) + t * a.c.par_bytes(), j, x);
    kv_store16<T>(out + row * D + 16 * j, x);
}

}  // namespace milo

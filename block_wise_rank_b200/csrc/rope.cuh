// rope.cuh -- rotary positions for queries and keys, and their gradient.
//
// Pair i of a row turns by the angle p * w_i (Su et al., "RoFormer", 2021):
// (a, b) -> m (a cos - b sin, a sin + b cos); the transposed map negates the
// angle and is the gradient.  The turns p * w_i / (2 pi) are taken modulo 1 in
// fp64, so a position of 2^31 still leaves 22 bits of the angle, and the rest
// goes through sincospi in fp32 (its argument, at most 1, is rounded to 2^-25).
//
// Bound by memory: each row is read and written once.  A thread owns one unit
// of V pairs (or V copied channels) of one token and walks a chunk of the
// heads, so a token's angles are computed once per chunk and stay in
// registers; the loads of several heads are issued together (128 bytes a
// thread).  Measured on 32768 tokens x 32 heads x 128 bf16: 90 us, 5.9 TB/s,
// 90 % of the measured copy rate (one head at a time 120 us, two 111 us); 28 tokens
// of a decode step, 3 us in a graph.  80 registers for three CTAs an SM: bf16 rows in half
// layout spill 16 bytes a thread.
#pragma once
#include "project_simt.cuh"   // from_f32

namespace milo {

struct RopeArgs {
    double turns[MILO_ROPE_MAX_D / 2];   // w_i / (2 pi)
    const void *x;
    void *y;
    const int32_t *pos;
    int64_t n_pos, n_tokens;
    int64_t xt, xh, yt, yh;              // strides in elements
    int d, rd, heads;
    int hpt, n_hc;                       // heads per thread, chunks of heads
    int units, rot_units;                // units of a row, those that turn
    bool small;                          // the launch has fewer than 2^32 threads
    float m;                             // factor on the turned channels
    float sgn;                           // -1: transposed
};

// V elements as they lie, and as fp32
template <typename T, int V> struct RopeRaw {
    static constexpr int B = V * (int)sizeof(T);
    static constexpr bool VEC = B % 16 == 0, HALF16 = B == 8 && V >= 4;
    uint4 w[VEC ? B / 16 : 1];
    T e[VEC || HALF16 ? 1 : V];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < B / 16; ++i) w[i] = reinterpret_cast<const uint4 *>(p)[i];
        } else if constexpr (HALF16) {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            w[0].x = u.x;
            w[0].y = u.y;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) e[i] = p[i];
        }
    }
    __device__ __forceinline__ void get(float (&v)[V]) const {
        if constexpr (VEC || HALF16) {
            const T *t = reinterpret_cast<const T *>(w);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = to_f32(t[i]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = to_f32(e[i]);
        }
    }
};

template <typename T, int V> __device__ __forceinline__ void rope_store(T *p, const float (&v)[V]) {
    constexpr int B = V * (int)sizeof(T);
    if constexpr (B % 16 == 0) {
        uint4 w[B / 16];
        T *e = reinterpret_cast<T *>(w);
#pragma unroll
        for (int i = 0; i < V; ++i) e[i] = from_f32<T>(v[i]);
#pragma unroll
        for (int i = 0; i < B / 16; ++i) reinterpret_cast<uint4 *>(p)[i] = w[i];
    } else if constexpr (B == 8 && V >= 4) {
        uint2 w;
        T *e = reinterpret_cast<T *>(&w);
#pragma unroll
        for (int i = 0; i < V; ++i) e[i] = from_f32<T>(v[i]);
        *reinterpret_cast<uint2 *>(p) = w;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = from_f32<T>(v[i]);
    }
}

// V elements per access.  INTER: a unit is V neighbouring channels (V / 2
// pairs); otherwise V pairs (i, i + rd / 2), i.e. two accesses.
template <typename TX, typename TY, int V, bool INTER>
__global__ void __launch_bounds__(256, 3) k_rope(const __grid_constant__ RopeArgs a) {
    int u, hc;
    int64_t t;
    if (a.small) {   // fewer than 2^32 threads: 64-bit divisions would take as long as a small call's transfer
        const uint32_t gid = blockIdx.x * blockDim.x + threadIdx.x, r = gid / (uint32_t)a.units;
        u = (int)(gid - r * (uint32_t)a.units);
        const uint32_t q = r / (uint32_t)a.n_hc;
        hc = (int)(r - q * (uint32_t)a.n_hc);
        t = q;
    } else {
        const int64_t gid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, r = gid / a.units;
        u = (int)(gid % a.units);
        hc = (int)(r % a.n_hc);
        t = r / a.n_hc;
    }
    if (t >= a.n_tokens) return;
    const int h0 = hc * a.hpt, h1 = min(a.heads, h0 + a.hpt);
    const TX *x = (const TX *)a.x + t * a.xt;
    TY *y = (TY *)a.y + t * a.yt;
    if (u >= a.rot_units) {   // channels that do not turn
        const int c = a.rd + (u - a.rot_units) * V;
        for (int h = h0; h < h1; ++h) {
            RopeRaw<TX, V> r;
            float v[V];
            r.load(x + h * a.xh + c);
            r.get(v);
            rope_store<TY, V>(y + h * a.yh + c, v);
        }
        return;
    }
    constexpr int NP = INTER ? (V + 1) / 2 : V;   // pairs of a unit
    // heads whose loads are issued together: up to 128 bytes in flight a thread
    constexpr int FIT = 128 / (V * (int)sizeof(TX) * (INTER ? 1 : 2)), ROPE_HEADS = FIT < 4 ? FIT : 4;
    const double p = (double)a.pos[a.n_pos >= a.n_tokens ? t : t % a.n_pos];
    float cs[NP], sn[NP];
    const int i0 = u * NP;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const double n = p * a.turns[i0 + i];
        float s, c;
        sincospif((float)(2.0 * (n - rint(n))), &s, &c);
        cs[i] = c * a.m;
        sn[i] = s * a.m * a.sgn;
    }
    if constexpr (INTER) {
        static_assert(V % 2 == 0, "a unit of neighbouring channels holds whole pairs");
        for (int h = h0; h < h1; h += ROPE_HEADS) {
            RopeRaw<TX, V> r[ROPE_HEADS];
#pragma unroll
            for (int e = 0; e < ROPE_HEADS; ++e)
                if (h + e < h1) r[e].load(x + (h + e) * a.xh + u * V);
#pragma unroll
            for (int e = 0; e < ROPE_HEADS; ++e) {
                float v[V], w[V];
                r[e].get(v);
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    w[2 * i] = v[2 * i] * cs[i] - v[2 * i + 1] * sn[i];
                    w[2 * i + 1] = v[2 * i] * sn[i] + v[2 * i + 1] * cs[i];
                }
                if (h + e < h1) rope_store<TY, V>(y + (h + e) * a.yh + u * V, w);
            }
        }
    } else {
        const int c0 = u * V, c1 = a.rd / 2 + u * V;
        for (int h = h0; h < h1; h += ROPE_HEADS) {
            RopeRaw<TX, V> r0[ROPE_HEADS], r1[ROPE_HEADS];
#pragma unroll
            for (int e = 0; e < ROPE_HEADS; ++e)
                if (h + e < h1) {
                    r0[e].load(x + (h + e) * a.xh + c0);
                    r1[e].load(x + (h + e) * a.xh + c1);
                }
#pragma unroll
            for (int e = 0; e < ROPE_HEADS; ++e) {
                float v[V], w[V], p0[V], p1[V];
                r0[e].get(v);
                r1[e].get(w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    p0[i] = v[i] * cs[i] - w[i] * sn[i];
                    p1[i] = v[i] * sn[i] + w[i] * cs[i];
                }
                if (h + e < h1) {
                    rope_store<TY, V>(y + (h + e) * a.yh + c0, p0);
                    rope_store<TY, V>(y + (h + e) * a.yh + c1, p1);
                }
            }
        }
    }
}

template <typename TX, typename TY, int V, bool INTER> void rope_launch(const RopeArgs &a, cudaStream_t s) {
    const int64_t threads = a.n_tokens * a.n_hc * a.units;
    k_rope<TX, TY, V, INTER><<<(unsigned)((threads + 255) / 256), 256, 0, s>>>(a);
}

template <typename TX, typename TY, int V> void rope_launch_layout(const RopeArgs &a, bool inter, cudaStream_t s) {
    if (inter) rope_launch<TX, TY, (V < 2 ? 2 : V), true>(a, s);
    else rope_launch<TX, TY, V, false>(a, s);
}

}  // namespace milo

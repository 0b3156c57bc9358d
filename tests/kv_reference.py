"""Plain numpy forms of the rotary positions and of the quantised cache of
recent tokens: code decisions in fp32 as milo.h states them, everything else
in 64 bits (angles in extended precision)."""
import math

import numpy as np

D = 128


# ------------------------------------------------------------------ rotary
def rope_freqs(rd, base, scaling="none", factor=1.0, orig_ctx=0.0, beta_fast=32.0, beta_slow=1.0, low_freq=1.0,
               high_freq=4.0):
    i = np.arange(rd // 2, dtype=np.longdouble)
    if scaling == "ntk":
        base = base * factor ** (rd / (rd - 2))
    t = np.longdouble(base) ** (-2 * i / rd)
    if scaling == "linear":
        return t / factor
    if scaling == "yarn":
        def channel(n):
            return rd * math.log(orig_ctx / (n * 2 * math.pi)) / (2 * math.log(base))
        lo = max(math.floor(channel(beta_fast)), 0)
        hi = min(math.ceil(channel(beta_slow)), rd - 1)
        g = np.clip((i - lo) / (hi - lo if hi > lo else 0.001), 0, 1)
        return t / factor * g + t * (1 - g)
    if scaling == "bands":
        n = orig_ctx * t / (2 * math.pi)
        u = np.clip((n - low_freq) / (high_freq - low_freq), 0, 1)
        return (1 - u) * t / factor + u * t
    return t


def rope(x, pos, w, interleaved=False, m=1.0, transpose=False):
    """x [n_tokens][n_heads][d] float64 turned by pos[t % n_pos] * w."""
    n, rd = x.shape[0], 2 * len(w)
    p = np.asarray(pos, dtype=np.longdouble)[np.arange(n) % len(pos)]
    a = p[:, None] * w * (-1 if transpose else 1)
    c, s = (np.cos(a) * m).astype(np.float64)[:, None], (np.sin(a) * m).astype(np.float64)[:, None]
    y = x.copy()
    u, v = (slice(0, rd, 2), slice(1, rd, 2)) if interleaved else (slice(0, rd // 2), slice(rd // 2, rd))
    y[..., u] = x[..., u] * c - x[..., v] * s
    y[..., v] = x[..., u] * s + x[..., v] * c
    return y


def rope_pair_size(x, rd, interleaved):
    """|a| + |b| of each channel's pair (0 for channels that do not turn): what a relative error of the turn scales."""
    y = np.zeros_like(x)
    u, v = (slice(0, rd, 2), slice(1, rd, 2)) if interleaved else (slice(0, rd // 2), slice(rd // 2, rd))
    y[..., u] = y[..., v] = np.abs(x[..., u]) + np.abs(x[..., v])
    return y


# ------------------------------------------------------------------- codes
def e4m3(x):
    """fp32 rounded to the nearest e4m3 value (half to even), at most 448."""
    x = x.astype(np.float64)
    e = np.maximum(np.frexp(x)[1] - 1, -6)
    return np.clip(np.rint(x / 2.0 ** (e - 3)) * 2.0 ** (e - 3), -448, 448)


def quantise(x, dtype):
    """(codes as numbers [..., 128], params) of rows x (fp32)."""
    x = x.astype(np.float32)
    with np.errstate(all="ignore"):
        if dtype == "int4":
            g = x.reshape(x.shape[:-1] + (4, 32))
            lo, hi = g.min(-1, keepdims=True), g.max(-1, keepdims=True)
            z = lo.astype(np.float16)
            s = ((hi - lo) / np.float32(15)).astype(np.float16)
            zf, sf = z.astype(np.float32), s.astype(np.float32)
            c = np.where(sf > 0, np.clip(np.rint((g - zf) / sf), 0, 15), np.float32(0))
            return c.reshape(x.shape), np.concatenate([s, z], -1)
        s = (np.abs(x).max(-1) / np.float32(127 if dtype == "int8" else 448)).astype(np.float32)
        t = np.where(s[..., None] > 0, x / s[..., None], np.float32(0)).astype(np.float32)
        return (np.clip(np.rint(t), -127, 127) if dtype == "int8" else e4m3(t)), s


def values(codes, params, dtype):
    """The values of codes, in 64 bits."""
    c = codes.astype(np.float64)
    if dtype == "int4":
        p = np.repeat(params.astype(np.float64), 32, axis=-2)
        return (c * p[..., 0] + p[..., 1]).astype(np.float16).astype(np.float64)
    return c * params[..., None].astype(np.float64)


def outward(x, up):
    """fp32 -> nearest bf16 (as fp32) not below (up) / not above x."""
    b = x.astype(np.float32).view(np.int32)
    t = b & np.int32(-65536)
    away = (t != b) & ((b >= 0) if up else (b < 0))
    return np.where(away, t + 65536, t).astype(np.int32).view(np.float32)


def bound_codes(lo, hi):
    b = np.stack([lo, hi], -2).astype(np.float32)
    s = (np.abs(b).max((-1, -2)) / np.float32(127)).astype(np.float32)
    with np.errstate(all="ignore"):
        c = np.where(s[..., None, None] > 0, np.clip(np.rint(b / s[..., None, None]), -127, 127), 0)
    return c.astype(np.int8), s


# --------------------------------------------------------------- retrieval
def scores(q, bcodes, bscale):
    """fp32 scores [n_b] of one KV head's query heads q [G][128] (fp32)."""
    q = np.where(np.isfinite(q), q, 0).astype(np.float32)
    u = (np.abs(q).max(-1) / np.float32(127)).astype(np.float32)
    with np.errstate(all="ignore"):
        c = np.where(u[:, None] > 0, np.clip(np.rint(q / u[:, None]), -127, 127), 0).astype(np.int64)
    lo, hi = bcodes[:, 0].astype(np.int64), bcodes[:, 1].astype(np.int64)
    dot = np.minimum(c, 0) @ lo.T + np.maximum(c, 0) @ hi.T                      # [G][n_b]
    return ((dot.astype(np.float32) * u[:, None]).max(0) * bscale).astype(np.float32)


def top(score, cand, n_sel, n_first, n_last):
    """Ascending ids of the n_sel best of the first `cand` blocks, -1 behind."""
    forced = set(range(min(n_first, cand))) | set(range(max(0, cand - n_last), cand))
    order = sorted(range(cand), key=lambda b: (b not in forced, -score[b] if b not in forced else 0, b))
    ids = sorted(order[:n_sel])
    return np.array(ids + [-1] * (n_sel - len(ids)), dtype=np.int32)


# --------------------------------------------------------------- attention
def attn(q, k, v, scale, f16_weights=False, out_eps=0.0):
    """(o, lse, bound on |o' - o|, bound on |lse' - lse|) of query rows q [R][128] over
    tokens k, v [T][128] in 64 bits.

    The bound counts the roundings of a kernel with fp32 sums: a score is a sum
    of 128 products in at most 24 rounded steps (2^-23 each, where the last bit
    may be cut off), its factors are held to 2^-22; a weight adds an exponential
    and two products (2^-21) and, for 16-bit queries, its rounding to fp16
    (2^-11, or 2^-24 of the greatest weight below the normal range); the sums over T tokens
    take at most T / 8 + 32 rounded steps."""
    R, T = q.shape[0], k.shape[0]
    if T == 0:
        z = np.zeros((R, D))
        return z, np.full(R, -np.inf), z + 1e-300, np.zeros(R)
    s = (q @ k.T) * scale
    size = (np.abs(q) @ np.abs(k).T) * scale
    dz = 2.0 ** -23 * (24 + 4) * size + 2.0 ** -23 * np.abs(s)
    m = s.max(-1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(-1, keepdims=True)
    w = p / l
    o = w @ v
    steps = 2.0 ** -23 * (T / 8 + 32)
    rel = dz + 2.0 ** -21 + steps + (2.0 ** -11 if f16_weights else 0.0)
    low = 2.0 ** -24 if f16_weights else 2.0 ** -34
    big = np.abs(v).max()
    err = (w * rel) @ np.abs(v) + (w * rel).sum(-1, keepdims=True) * np.abs(o) + low * T * big / l
    err = err + out_eps * np.abs(o) + 1e-30
    lse = (m + np.log(l))[:, 0]
    return o, lse, err, (w * (dz + 2.0 ** -21 + steps)).sum(-1) + 2.0 ** -23 * (1 + np.abs(lse))


def score_floor(q, k, s):
    """The least score [G], before its own fp32 roundings, of query heads q [G][128] for a block of keys k [T][128]
    whose bound codes have the scale s.  With u = max|q| / 127 a code of q is at most u / 2 off and a code of a bound
    s / 2, so the score is at least max_t (q . k_t - u / 2 sum_j |k_tj|) - s / 2 sum_j |q'_j|, q' = u c the coded q."""
    q, k = q.astype(np.float64), k.astype(np.float64)
    u = np.abs(q).max(-1, keepdims=True) / 127
    coded = u * np.abs(np.rint(q / np.where(u > 0, u, 1)))
    off = 0.5 + 2.0 ** -15           # half a step; a code of at most 127 is decided in fp32
    return (q @ k.T - off * u * np.abs(k).sum(-1)).max(-1) - off * float(s) * coded.sum(-1)

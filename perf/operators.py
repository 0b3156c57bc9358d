"""The operators around the quantised KV cache, as cases to be measured.

Four operators, each in its plain form (elementary torch operations in 32 bits,
angles in 64) and through libmilo's entry points:

  rope    milo_rope: queries and keys turned to their positions, and the gradient
  append  milo_kv_append + milo_kv_read: keys and values quantised as they are
          written, with each block's key bounds, and read back
  select  milo_kv_select: the blocks of the cache that a query's cheap score picks
  attn    milo_kv_attn: attention over the cache, all of it or the picked blocks

The cache is one byte buffer in the layout that include/milo.h documents, so
that `prepare` can fill it with torch alone.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

D = 128
GROUP = 32           # channels that share one INT4 scale and zero
BF16_MAX = 3.3895313892515355e38


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the queries and keys of one new token, every layer of a 7B-shaped model: latency
        dict(name="rope-decode", op="rope", tokens=28, n_pos=1, heads=32, d=128, rotary=128, inter=False, scaling="none",
             dtype="bf16", back=False, pos0=131000),
        # a packed projection of a long prompt (28 query and 4 key heads), context stretched fourfold
        dict(name="rope-prompt", op="rope", tokens=32768, n_pos=32768, heads=32, d=128, rotary=128, inter=False,
             scaling="yarn", dtype="bf16", back=False, pos0=0),
        # gradient of a partly rotated head in neighbouring pairs, odd sizes
        dict(name="rope-grad-partial", op="rope", tokens=4097, n_pos=4097, heads=9, d=96, rotary=40, inter=True,
             scaling="ntk", dtype="f32", back=True, pos0=7),
        # one new token of 8 sessions in all 28 layers
        dict(name="append-decode-int8", op="append", cache="int8", dtype="bf16", L=28, S=8, H=4, n=1, cap=4096,
             block_len=64, lo=100, hi=4000, out="bf16"),
        # questions of ragged length behind earlier turns
        dict(name="append-question-int4", op="append", cache="int4", dtype="f32", L=4, S=16, H=4, n=333, cap=2048,
             block_len=32, lo=0, hi=1500, out="f32"),
        # a whole prompt of one layer
        dict(name="append-prompt-fp8", op="append", cache="fp8", dtype="bf16", L=1, S=4, H=4, n=32768, cap=32768,
             block_len=64, lo=0, hi=0, out="bf16"),
        # 512 blocks of one session and layer
        dict(name="select-32k", op="select", cache="int8", q="f32", L=1, S=1, H=2, G=8, n_q=1, cap=32768, block_len=64,
             lo=32768, hi=32768, n_sel=16),
        # 32 sessions of up to 131072 tokens
        dict(name="select-128k", op="select", cache="int8", q="bf16", L=1, S=32, H=4, G=7, n_q=1, cap=131072,
             block_len=64, lo=30000, hi=131072, n_sel=64),
        # a short tail of one session: latency
        dict(name="attn-short-int8", op="attn", cache="int8", q="f32", L=1, S=1, H=2, G=8, n_q=1, cap=1024, block_len=64,
             lo=513, hi=513, n_sel=0),
        # 8 sessions of very different length, dense
        dict(name="attn-long-int8", op="attn", cache="int8", q="bf16", L=1, S=8, H=4, G=7, n_q=1, cap=131072,
             block_len=64, lo=1000, hi=131072, n_sel=0),
        # 32 sessions, 64 of up to 1024 blocks each, 4 bits
        dict(name="attn-sparse-int4", op="attn", cache="int4", q="bf16", L=2, S=32, H=4, G=7, n_q=1, cap=65536,
             block_len=64, lo=9001, hi=65536, n_sel=64),
        # a 17-token question over what the session holds
        dict(name="attn-question-fp8", op="attn", cache="fp8", q="f32", L=2, S=4, H=4, G=7, n_q=17, cap=8192,
             block_len=64, lo=20, hi=8190, n_sel=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "select", "attn"])
    if op == "rope":
        d = rng.choice([64, 80, 96, 128, 160, 256])
        tokens, heads = _log(rng, 1, 16384), rng.randint(1, 40)
        return dict(op=op, tokens=tokens, n_pos=tokens, heads=heads, d=d,
                    rotary=rng.choice([d, d, d // 2, 2 * rng.randint(2, d // 2)]), inter=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]), dtype=rng.choice(["bf16", "f32"]),
                    back=rng.random() < 0.4, pos0=rng.choice([0, 1, _log(rng, 2, 1 << 20)]))
    c = dict(op=op, cache=rng.choice(["int8", "fp8", "int4"]), L=rng.randint(1, 3), H=rng.choice([1, 2, 4]),
             block_len=rng.choice([16, 32, 48, 64, 128]))
    if op == "append":
        n = _log(rng, 1, 4096)
        lo = rng.choice([0, rng.randint(0, 300)])
        hi = lo + rng.randint(0, 1000)
        return dict(c, dtype=rng.choice(["bf16", "f32"]), S=rng.randint(1, 6), n=n, cap=hi + n + rng.randint(0, 200),
                    lo=lo, hi=hi, out=rng.choice(["bf16", "f32"]))
    cap = _log(rng, 40, 65536)
    c.update(q=rng.choice(["bf16", "f32"]), S=rng.randint(1, 8), G=rng.choice([1, 2, 4, 5, 7, 8, 12]), n_q=1, cap=cap,
             lo=rng.randint(0, cap), hi=cap - rng.randint(0, cap // 8))
    n_b = -(-cap // c["block_len"])
    if op == "select":
        return dict(c, n_q=rng.choice([1, 1, 2, 3]), n_sel=min(n_b, _log(rng, 2, 200)))
    if rng.random() < 0.5:
        return dict(c, n_q=rng.choice([1, 1, 2]), n_sel=min(n_b, _log(rng, 2, 64)), L=1)
    return dict(c, n_q=rng.choice([1, 1, 3, 20]), n_sel=0, L=1)


# ------------------------------------------------------------- the cache
def _row(cache):
    return 64 if cache == "int4" else 128


def _par(cache):
    return 16 if cache == "int4" else 4


def _sections(c):
    """(name, byte offset in a layer, bytes) of a layer's sections, and the layer's bytes."""
    rows, n_b = c["S"] * c["H"] * c["cap"], -(-c["cap"] // c["block_len"])
    blocks = c["S"] * c["H"] * n_b
    got, at = {}, 0
    for name, n in (("k", rows * _row(c["cache"])), ("v", rows * _row(c["cache"])), ("kp", rows * _par(c["cache"])),
                    ("vp", rows * _par(c["cache"])), ("bounds", blocks * 2 * D * 2), ("codes", blocks * 2 * D),
                    ("scale", blocks * 4)):
        got[name] = (at, n)
        at = -(-(at + n) // 256) * 256
    return got, at


def _views(c, buf):
    """The sections of a cache buffer as typed tensors over every layer."""
    got, layer = _sections(c)
    L, S, H, cap, n_b = c["L"], c["S"], c["H"], c["cap"], -(-c["cap"] // c["block_len"])
    raw = buf.view(L, layer)
    cut = lambda name: raw[:, got[name][0]:got[name][0] + got[name][1]]  # noqa: E731
    kinds = {"int8": torch.int8, "fp8": torch.float8_e4m3fn, "int4": torch.uint8}
    v = {}
    for name in ("k", "v"):
        v[name] = cut(name).view(kinds[c["cache"]]).view(L, S, H, cap, _row(c["cache"]))
        p = cut(name + "p")
        v[name + "p"] = p.view(torch.float16).view(L, S, H, cap, 4, 2) if c["cache"] == "int4" else \
            p.view(torch.float32).view(L, S, H, cap)
    v["bounds"] = cut("bounds").view(torch.bfloat16).view(L, S, H, n_b, 2, D)
    v["codes"] = cut("codes").view(torch.int8).view(L, S, H, n_b, 2, D)
    v["scale"] = cut("scale").view(torch.float32).view(L, S, H, n_b)
    return v


def _over(x, n):
    """x / n, rounded once (a division by a plain number is a product with its rounded reciprocal on the GPU)."""
    return x / torch.full_like(x, n)


def _encode(x, cache):
    """Codes and parameters of rows x [..., 128] in 32 bits."""
    if cache == "int4":
        g = x.unflatten(-1, (4, GROUP))
        lo, hi = g.amin(-1), g.amax(-1)
        z, s = lo.half(), _over(hi - lo, 15.0).half()
        sf = s.float()[..., None]
        q = torch.where(sf > 0, torch.round((g - z.float()[..., None]) / sf), 0.0).clamp(0, 15).to(torch.uint8)
        q = q.flatten(-2).unflatten(-1, (64, 2))
        return q[..., 0] | (q[..., 1] << 4), torch.stack((s, z), -1)
    amax = x.abs().amax(-1)
    s = _over(amax, 127.0 if cache == "int8" else 448.0)
    q = torch.where(s[..., None] > 0, x / s[..., None], 0.0)
    if cache == "int8":
        return torch.round(q).clamp(-127, 127).to(torch.int8), s
    return q.clamp(-448, 448).to(torch.float8_e4m3fn), s


def _decode(q, p, cache):
    """The values, in 32 bits, that codes q and parameters p stand for."""
    if cache == "int4":
        u = torch.stack((q & 15, q >> 4), -1).flatten(-2).unflatten(-1, (4, GROUP)).float()
        return (u * p[..., 0, None].float() + p[..., 1, None].float()).half().float().flatten(-2)
    return q.float() * p[..., None]


def _outward(x, up):
    """x rounded to bf16 towards +inf (up) or -inf."""
    b = x.view(torch.int32)
    t = b & -65536
    away = (t != b) & ((b >= 0) if up else (b < 0))
    return torch.where(away, t + 65536, t).view(torch.float32).clamp(-BF16_MAX, BF16_MAX).to(torch.bfloat16)


def _bound_codes(mn, mx):
    """INT8 codes [..., 2, 128] and the scale of a block's key bounds."""
    b = torch.stack((mn, mx), -2).float()
    s = _over(b.abs().amax((-1, -2)), 127.0)
    q = torch.where(s[..., None, None] > 0, torch.round(b / s[..., None, None]), 0.0)
    return q.clamp(-127, 127).to(torch.int8), s


def _lens(c):
    S = c["S"]
    return [c["lo"] + (c["hi"] - c["lo"]) * s // max(1, S - 1) for s in range(S)]


def _counts(c):
    """Tokens that each session appends: ragged, the first one all of them."""
    return [max(0, c["n"] - (s * c["n"]) // (2 * c["S"])) if c["n"] > 1 else 1 for s in range(c["S"])]


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _keys(shape, g):
    """Keys with a few loud channels, as projections have them."""
    x = torch.randn(shape, generator=g, device="cuda")
    loud = 0.5 + 2.0 * torch.rand(shape[-1], generator=g, device="cuda") ** 4
    return x * loud


def _fill(c, g):
    """A cache of cap tokens in every session, filled a session at a time (bounds alone where nothing else is read)."""
    layer = _sections(c)[1]
    buf = torch.zeros(c["L"] * layer, dtype=torch.uint8, device="cuda")
    v = _views(c, buf)
    bl, cap = c["block_len"], c["cap"]
    n_b = -(-cap // bl)
    for at in range(c["L"]):
        for s in range(c["S"]):
            k = _keys((c["H"], cap, D), g)
            if c["op"] == "attn":
                x = torch.randn((c["H"], cap, D), generator=g, device="cuda")
                for name, t in (("k", k), ("v", x)):
                    q, p = _encode(t, c["cache"])
                    v[name][at, s].view(torch.uint8).copy_(q.view(torch.uint8))
                    v[name + "p"][at, s].copy_(p)
            pad = n_b * bl - cap
            mn = torch.nn.functional.pad(k, (0, 0, 0, pad), value=math.inf).unflatten(1, (n_b, bl)).amin(2)
            mx = torch.nn.functional.pad(k, (0, 0, 0, pad), value=-math.inf).unflatten(1, (n_b, bl)).amax(2)
            mn, mx = _outward(mn, False), _outward(mx, True)
            v["bounds"][at, s].copy_(torch.stack((mn, mx), -2))
            q, p = _bound_codes(mn, mx)
            v["codes"][at, s].copy_(q)
            v["scale"][at, s].copy_(p)
    return buf


_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ROPE = dict(base=1e6, factor=4.0, orig_ctx=8192, beta_fast=32.0, beta_slow=1.0, low_freq=1.0, high_freq=4.0)


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = {"case": c}
    if c["op"] == "rope":
        # the heads of a packed projection: a token's row also holds what is not rotated
        rows = torch.randn((c["tokens"], c["heads"] + 4, c["d"]), generator=g, device="cuda").to(_DT[c["dtype"]])
        st["x"] = rows[:, :c["heads"]]
        st["pos"] = torch.arange(c["pos0"], c["pos0"] + c["n_pos"], dtype=torch.int32, device="cuda")
        return st
    if c["op"] == "append":
        layer = _sections(c)[1]
        st["buf"] = torch.zeros(c["L"] * layer, dtype=torch.uint8, device="cuda")
        v = _views(c, st["buf"])
        # bounds of what the sessions hold already
        mn = -torch.rand(v["scale"].shape + (D,), generator=g, device="cuda") * 3
        mx = torch.rand(v["scale"].shape + (D,), generator=g, device="cuda") * 3
        v["bounds"].copy_(torch.stack((mn, mx), -2))
        q, p = _bound_codes(v["bounds"][..., 0, :], v["bounds"][..., 1, :])
        v["codes"].copy_(q)
        v["scale"].copy_(p)
        shape = (c["L"], c["S"], c["H"], c["n"], D)
        st["k"] = _keys(shape, g).to(_DT[c["dtype"]])
        st["v"] = torch.randn(shape, generator=g, device="cuda").to(_DT[c["dtype"]])
        st["start"] = torch.tensor(_lens(c), dtype=torch.int32, device="cuda")
        st["count"] = torch.tensor(_counts(c), dtype=torch.int32, device="cuda")
        st["k_out"] = torch.zeros(shape, dtype=_DT[c["out"]], device="cuda")
        st["v_out"] = torch.zeros(shape, dtype=_DT[c["out"]], device="cuda")
        return st
    st["buf"] = _fill(c, g)
    st["len"] = torch.tensor(_lens(c), dtype=torch.int32, device="cuda")
    shape = (c["L"], c["S"], c["n_q"], c["H"] * c["G"], D)
    st["q"] = torch.randn(shape, generator=g, device="cuda").to(_DT[c["q"]])
    if c["op"] == "attn" and c["n_sel"]:
        # distinct blocks of those that the query sees, ascending, -1 behind
        n_b = -(-c["cap"] // c["block_len"])
        r = torch.rand((c["L"], c["S"], c["n_q"], c["H"], n_b), generator=g, device="cuda")
        r = torch.where(torch.arange(n_b, device="cuda") < _seen_blocks(c, st["len"])[None, :, :, None, None], r, 2.0)
        val, idx = r.sort(-1)
        idx = torch.where(val[..., :c["n_sel"]] < 2.0, idx[..., :c["n_sel"]], n_b).sort(-1).values
        st["sel"] = torch.where(idx < n_b, idx, -1).to(torch.int32).contiguous()
    return st


def _seen(c, length):
    """Tokens that query i of session s sees, [S][n_q]."""
    i = torch.arange(c["n_q"], device=length.device)
    return (length[:, None] - c["n_q"] + i + 1).clamp(min=0)


def _seen_blocks(c, length):
    return (_seen(c, length) + c["block_len"] - 1) // c["block_len"]


# ------------------------------------------------------------- plain forms
def _inv_freq(c):
    """Angles per position of each pair (64 bits), and what the result is multiplied by."""
    rd, r = c["rotary"], _ROPE
    i = np.arange(rd // 2, dtype=np.float64)
    base, s = r["base"], c["scaling"]
    if s == "ntk" and rd > 2:
        base = base * r["factor"] ** (rd / (rd - 2))
    w = base ** (-2.0 * i / rd)
    if s == "linear":
        w = w / r["factor"]
    if s == "yarn":
        dim = lambda turns: rd * math.log(r["orig_ctx"] / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(dim(r["beta_fast"])), 0), min(math.ceil(dim(r["beta_slow"])), rd - 1)
        ramp = np.clip((i - low) / (high - low if high > low else 0.001), 0, 1)
        return w / r["factor"] * ramp + w * (1 - ramp), 0.1 * math.log(r["factor"]) + 1
    if s == "bands":
        turns = r["orig_ctx"] * w / (2 * math.pi)
        mix = np.clip((turns - r["low_freq"]) / (r["high_freq"] - r["low_freq"]), 0, 1)
        w = (1 - mix) * w / r["factor"] + mix * w
    return w, 1.0


def _rope_plain(st):
    c, x = st["case"], st["x"].float()
    w, m = _inv_freq(c)
    pos = st["pos"].double().repeat(c["tokens"] // c["n_pos"])
    a = pos[:, None] * torch.from_numpy(w).to(x.device)
    cos, sin = (torch.cos(a) * m).float()[:, None], (torch.sin(a) * m).float()[:, None]
    if c["back"]:
        sin = -sin
    rd = c["rotary"]
    r = x[..., :rd]
    u, v = (r[..., 0::2], r[..., 1::2]) if c["inter"] else (r[..., :rd // 2], r[..., rd // 2:])
    p, q = u * cos - v * sin, u * sin + v * cos
    y = torch.stack((p, q), -1).flatten(-2) if c["inter"] else torch.cat((p, q), -1)
    return torch.cat((y, x[..., rd:]), -1).to(_DT[c["dtype"]])


def _append_plain(st):
    c, v = st["case"], _views(st["case"], st["buf"])
    k, x = st["k"].float(), st["v"].float()
    n, bl, cap = c["n"], c["block_len"], c["cap"]
    live = torch.arange(n, device=k.device) < st["count"][:, None]                     # [S][n]
    out = []
    for t in (k, x):
        t = _decode(*_encode(t, c["cache"]), c["cache"])
        out.append(torch.where(live[None, :, None, :, None], t, 0.0).to(_DT[c["out"]]))
    # the blocks that the new tokens fall into, and the tokens' places in them
    nt, n_b = -(-n // bl) + 1, -(-cap // bl)
    start = st["start"].long()
    blk = start[:, None] // bl + torch.arange(nt, device=k.device)                     # [S][nt]
    i = torch.arange(nt * bl, device=k.device) - (start % bl)[:, None]                 # [S][nt bl]
    ok = ((i >= 0) & (i < st["count"][:, None]))[None, :, None, :, None]
    at = i.clamp(0, n - 1)[None, :, None, :, None].expand(c["L"], -1, c["H"], -1, D)
    new = k.gather(3, at)
    mn = torch.where(ok, new, math.inf).unflatten(3, (nt, bl)).amin(4)
    mx = torch.where(ok, new, -math.inf).unflatten(3, (nt, bl)).amax(4)
    # a block that the new tokens begin is theirs alone; one that they go on with keeps its bounds
    put = blk.clamp(max=n_b - 1)[None, :, None, :, None].expand(c["L"], -1, c["H"], -1, D)
    fresh = (blk * bl >= start[:, None])[None, :, None, :, None]
    old = v["bounds"].float()
    mn = torch.where(fresh, mn, torch.minimum(mn, old[..., 0, :].gather(3, put)))
    mx = torch.where(fresh, mx, torch.maximum(mx, old[..., 1, :].gather(3, put)))
    mn, mx = _outward(mn, False), _outward(mx, True)
    hit = ok[0, :, 0, :, 0].unflatten(1, (nt, bl)).any(2)                              # [S][nt]
    bounds, codes, scale = v["bounds"].clone(), v["codes"].clone(), v["scale"].clone()
    q, p = _bound_codes(mn, mx)
    s, t = hit.nonzero(as_tuple=True)
    b = blk[s, t]
    bounds[:, s, :, b] = torch.stack((mn, mx), -2)[:, s, :, t]
    codes[:, s, :, b] = q[:, s, :, t]
    scale[:, s, :, b] = p[:, s, :, t]
    return dict(k=out[0], v=out[1], bounds=bounds, codes=codes, scale=scale)


def _select_plain(st):
    c, v = st["case"], _views(st["case"], st["buf"])
    q = st["q"].float().unflatten(3, (c["H"], c["G"]))                                 # [L][S][n_q][H][G][D]
    sq = _over(q.abs().amax(-1), 127.0)
    qc = torch.where(sq[..., None] > 0, torch.round(q / sq[..., None]), 0.0).clamp(-127, 127)
    mn, mx = v["codes"].float().unbind(4)                                              # [L][S][H][n_b][D]
    # sums of products of whole numbers below 2^24: exact in 32 bits
    dot = qc.clamp(min=0) @ mx[:, :, None].mT + qc.clamp(max=0) @ mn[:, :, None].mT
    score = (dot * sq[..., None]).amax(-2) * v["scale"][:, :, None]
    n_b = score.shape[-1]
    ids = torch.arange(n_b, device=q.device)
    seen = _seen_blocks(c, st["len"])[None, :, :, None, None]
    score = torch.where(ids < seen, score, -math.inf)
    # the last block seen is always picked; ties go to the lower id
    key = torch.where((ids == seen - 1), math.inf, score)
    idx = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :c["n_sel"]]
    idx = torch.where(idx < seen, idx, n_b).sort(-1).values
    return dict(selected=torch.where(idx < n_b, idx, -1).to(torch.int32), scores=score)


def _attn_plain(st):
    c, v = st["case"], _views(st["case"], st["buf"])
    seen, n_q, G = _seen(c, st["len"]), c["n_q"], c["G"]                               # [S][n_q]
    q = st["q"].float().unflatten(3, (c["H"], G))                                      # [L][S][n_q][H][G][D]
    if c["n_sel"]:
        sel, bl = st["sel"].long(), c["block_len"]
        tok = sel[..., None] * bl + torch.arange(bl, device=q.device)                  # [L][S][n_q][H][n_sel][bl]
        tok = torch.where(sel[..., None] >= 0, tok, c["cap"]).flatten(-2)
        ok = (tok < seen[None, :, :, None, None])[..., None, :]
        tok = tok.clamp(max=c["cap"] - 1)
        l, s, h = (torch.arange(c[n], device=q.device).view(shape) for n, shape in
                   (("L", (-1, 1, 1, 1, 1)), ("S", (-1, 1, 1, 1)), ("H", (-1, 1))))
        k, x = (_decode(v[n][l, s, h, tok], v[n + "p"][l, s, h, tok], c["cache"]) for n in ("k", "v"))
    else:
        # every query of a session reads the same rows: they share a product
        most = max(1, max(_lens(c)))
        q = q.transpose(2, 3).flatten(3, 4)[:, :, None]                                # [L][S][1][H][n_q G][D]
        k, x = (_decode(v[n][:, :, :, :most], v[n + "p"][:, :, :, :most], c["cache"])[:, :, None] for n in ("k", "v"))
        ok = torch.arange(most, device=q.device) < seen.repeat_interleave(G, 1)[None, :, None, None, :, None]
    s = (q @ k.mT) * (1 / math.sqrt(D))
    s = torch.where(ok, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m > -math.inf, m, 0.0))
    l = p.sum(-1, keepdim=True)
    o = (p @ x) / torch.where(l > 0, l, 1.0)
    lse = m + torch.log(l)
    if not c["n_sel"]:
        o, lse = (t[:, :, 0].unflatten(3, (n_q, G)).transpose(2, 3) for t in (o, lse))
    return dict(out=o.flatten(3, 4).to(_DT[c["q"]]), lse=lse[..., 0].flatten(3, 4))


# --------------------------------------------------------------------- run
def run(st):
    c = st["case"]
    if not own:
        return {"rope": _rope_plain, "append": _append_plain, "select": _select_plain, "attn": _attn_plain}[c["op"]](st)
    from block_wise_rank_b200 import milo

    # the parameters and the cache's handle, which a program makes once and keeps
    if "plan" not in st:
        st["plan"] = milo.rope_params(c["d"], rotary_dim=c["rotary"], interleaved=c["inter"], scaling=c["scaling"],
                                      **_ROPE) if c["op"] == "rope" else \
            milo.KvCache(milo.kv_shape(c["L"], c["S"], c["H"], c["cap"], c["block_len"], c["cache"]), st["buf"])
    cache = st["plan"]
    if c["op"] == "rope":
        return milo.milo_rope(st["x"], st["pos"], st["plan"], transpose=c["back"])
    if c["op"] == "append":
        milo.milo_kv_append(cache, st["k"], st["v"], st["start"], count=st["count"])
        k, v = milo.milo_kv_read(cache, st["start"], c["n"], count=st["count"], k_out=st["k_out"], v_out=st["v_out"])
        w = _views(c, st["buf"])
        return dict(k=k, v=v, bounds=w["bounds"], codes=w["codes"], scale=w["scale"])
    if c["op"] == "select":
        sel, scores = milo.milo_kv_select(cache, st["q"], st["len"], c["n_sel"], n_last=1, return_scores=True)
        return dict(selected=sel, scores=scores)
    out, lse = milo.milo_kv_attn(cache, st["q"], st["len"], selected=st.get("sel"), return_lse=True)
    return dict(out=out, lse=lse)


# -------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "rope":
        n, e = c["tokens"] * c["heads"], 2 if c["dtype"] == "bf16" else 4
        return dict(bytes=2 * n * c["d"] * e + 4 * c["n_pos"], flops=3 * n * c["rotary"])
    per = _row(c["cache"]) + _par(c["cache"])
    if c["op"] == "append":
        rows = 2 * c["L"] * c["H"] * sum(_counts(c))
        blocks = sum(-(-(s + n) // c["block_len"]) - s // c["block_len"] for s, n in zip(_lens(c), _counts(c)))
        e = 2 if c["dtype"] == "bf16" else 4
        o = 2 if c["out"] == "bf16" else 4
        # rows in, codes out, codes in, rows out; the bounds of the blocks that are begun or gone on with
        return dict(bytes=rows * (D * e + 2 * per + D * o) + c["L"] * c["H"] * blocks * (6 * D + 4), flops=6 * rows * D)
    rows = c["L"] * c["H"]
    io = c["L"] * c["S"] * c["n_q"] * c["H"] * c["G"] * D * (2 if c["q"] == "bf16" else 4)
    seen = [[max(0, n - c["n_q"] + i + 1) for i in range(c["n_q"])] for n in _lens(c)]
    if c["op"] == "select":
        blocks = [[-(-t // c["block_len"]) for t in s] for s in seen]
        n_b = -(-c["cap"] // c["block_len"])
        return dict(bytes=rows * sum(max(b) for b in blocks) * (2 * D + 4) + io
                    + rows * c["S"] * c["n_q"] * (n_b + c["n_sel"]) * 4, flops=rows * sum(map(sum, blocks)) * 4 * D * c["G"])
    if c["n_sel"]:
        toks = sum(min(t, c["n_sel"] * c["block_len"]) for s in seen for t in s)
        read = rows * toks * 2 * per + rows * c["S"] * c["n_q"] * c["n_sel"] * 4
    else:
        toks = sum(t for s in seen for t in s)
        read = rows * sum(max(s) for s in seen) * 2 * per
    lse = c["L"] * c["S"] * c["n_q"] * c["H"] * c["G"] * 4
    return dict(bytes=read + 2 * io + lse, flops=rows * toks * c["G"] * 4 * D)


# ------------------------------------------------------------------- exact
def _values64(v, name, cache, at):
    """The 64-bit values of cache rows `at`, from codes and parameters."""
    q, p = v[name][at], v[name + "p"][at].double()
    if cache == "int4":
        u = torch.stack((q & 15, q >> 4), -1).flatten(-2).double()
        p = p.repeat_interleave(GROUP, -2)
        return (u * p[..., 0] + p[..., 1]).half().double()
    return q.to(torch.float32).double() * p[..., None]


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    if c["op"] == "rope":
        x = st["x"].double().cpu().numpy()
        w, m = _inv_freq(c)
        a = np.tile(st["pos"].cpu().numpy().astype(np.float64), c["tokens"] // c["n_pos"])[:, None] * w
        z = np.exp(-1j * a if c["back"] else 1j * a) * m
        rd, y = c["rotary"], x.copy()
        u, v = (slice(0, rd, 2), slice(1, rd, 2)) if c["inter"] else (slice(0, rd // 2), slice(rd // 2, rd))
        for h in range(c["heads"]):
            t = (x[:, h, u] + 1j * x[:, h, v]) * z
            y[:, h, u], y[:, h, v] = t.real, t.imag
        return y
    if c["op"] == "append":
        out = []
        for name in ("k", "v"):
            x = st[name].float().cpu().numpy()
            y = np.zeros(x.shape, np.float64)
            for s, n in enumerate(_counts(c)):
                r = x[:, s, :, :n]
                if c["cache"] == "int4":
                    r = r.reshape(r.shape[:-1] + (4, GROUP))
                    z = r.min(-1, keepdims=True).astype(np.float16).astype(np.float32)
                    p = ((r.max(-1, keepdims=True) - r.min(-1, keepdims=True)) / np.float32(15)).astype(np.float16).astype(np.float32)
                    with np.errstate(all="ignore"):
                        q = np.where(p > 0, np.clip(np.rint((r - z) / p), 0, 15), 0)
                    t = (q.astype(np.float64) * p + z).astype(np.float16).astype(np.float64)
                    y[:, s, :, :n] = t.reshape(t.shape[:-2] + (D,))
                    continue
                p = np.abs(r).max(-1, keepdims=True) / np.float32(127 if c["cache"] == "int8" else 448)
                with np.errstate(all="ignore"):
                    q = np.where(p > 0, r / p, np.float32(0))
                if c["cache"] == "int8":
                    q = np.clip(np.rint(q), -127, 127).astype(np.float64)
                else:  # e4m3: three bits behind the leading one, steps of 2^-9 below 2^-6
                    e = np.maximum(np.frexp(q.astype(np.float64))[1] - 1, -6)
                    q = np.rint(q.astype(np.float64) / 2.0 ** (e - 3)) * 2.0 ** (e - 3)
                y[:, s, :, :n] = q * p
            out.append(y)
        return dict(k=out[0], v=out[1], bounds=None, codes=None, scale=None)
    v = _views(c, st["buf"])
    G, H, dev = c["G"], c["H"], "cuda"
    if c["op"] == "select":
        n_b = -(-c["cap"] // c["block_len"])
        score = torch.full((c["L"], c["S"], c["n_q"], H, n_b), -math.inf, dtype=torch.float64, device=dev)
        for s, length in enumerate(_lens(c)):
            for i in range(c["n_q"]):
                nb = -(-max(0, length - c["n_q"] + i + 1) // c["block_len"])
                q = st["q"][:, s, i].float().unflatten(1, (H, G))
                sq = q.abs().amax(-1, keepdim=True)
                sq = sq / torch.full_like(sq, 127)
                qc = torch.where(sq > 0, torch.round(q / sq), 0.0).double()
                b = v["codes"][:, s, :, :nb].double()
                both = torch.maximum(qc[:, :, :, None] * b[:, :, None, :, 0], qc[:, :, :, None] * b[:, :, None, :, 1])
                score[:, s, i, :, :nb] = (both.sum(-1) * sq.double()).amax(2) * v["scale"][:, s, :, :nb].double()
        return dict(selected=None, scores=score)
    shape = st["q"].shape
    out = torch.zeros(shape, dtype=torch.float64, device=dev)
    lse = torch.full(shape[:-1], -math.inf, dtype=torch.float64, device=dev)
    for l in range(c["L"]):
        for s, length in enumerate(_lens(c)):
            for i in range(c["n_q"]):
                n = max(0, length - c["n_q"] + i + 1)
                for h in range(H):
                    if c["n_sel"]:
                        b = st["sel"][l, s, i, h].long()
                        t = (b[b >= 0, None] * c["block_len"] + torch.arange(c["block_len"], device=dev)).flatten()
                        t = t[t < n]
                    else:
                        t = torch.arange(n, device=dev)
                    if not t.numel():
                        continue
                    k, x = (_values64(v, name, c["cache"], (l, s, h, t)) for name in ("k", "v"))
                    a = st["q"][l, s, i, h * G:(h + 1) * G].double() @ k.T / math.sqrt(D)
                    out[l, s, i, h * G:(h + 1) * G] = torch.softmax(a, -1) @ x
                    lse[l, s, i, h * G:(h + 1) * G] = torch.logsumexp(a, -1)
    return dict(out=out, lse=lse)

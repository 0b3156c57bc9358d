"""Rotary positions and the quantised cache of recent tokens on the GPU,
against the plain forms of tests/kv_reference.py.

Tolerances are counted from roundings where they are used; codes, bounds and
selections have to be equal."""
import ctypes
import math

import numpy as np
import pytest
import torch

from block_wise_rank_b200 import build as milo_build
from block_wise_rank_b200 import milo, synth
from tests import kv_reference as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF: 2.0 ** -8, F32: 2.0 ** -24}     # finfo.eps / 2
KINDS = ["int8", "fp8", "int4"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    milo_build.build()
    milo.lib()
    assert torch.cuda.is_available()
    milo.milo_get_status()


def ok(status=milo.MILO_OK):
    assert milo.milo_get_status() == status


def np64(t):
    return t.detach().double().cpu().numpy()


def rnd(seed, *shape, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


# ------------------------------------------------------------------ rotary
# a turn's error relative to |a| + |b|: the reduced argument (pi 2^-25), sincospi (1 ulp: 2^-23), the factor's own
# rounding and its product (2^-23), two products and a sum (3 2^-24)
TURN = 2.0 ** -23 * (0.8 + 1 + 1 + 1.5)


def check_rope(x, pos, y, p, ref_w, inter=False, m=1.0, transpose=False, extra=0.0):
    rd = 2 * len(ref_w)
    ref = R.rope(np64(x), pos, ref_w, inter, m, transpose)
    size = R.rope_pair_size(np64(x), rd, inter)
    tol = (TURN + extra) * m * size + HALF_STEP[y.dtype] * np.abs(ref) * (1 + 2.0 ** -7) * (size > 0)
    if y.dtype != x.dtype and y.dtype == BF:     # channels that do not turn are rounded as well
        tol = tol + (size == 0) * HALF_STEP[BF] * np.abs(ref)
    assert np.all(np.abs(np64(y) - ref) <= tol), np.max(np.abs(np64(y) - ref) - tol)


SCALINGS = [("none", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=2.5)),
            ("yarn", dict(factor=4.0, orig_ctx=4096)), ("bands", dict(factor=8.0, orig_ctx=8192))]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("xd,yd", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("nt,nh,d,rd", [(1, 1, 128, 0), (5, 3, 128, 128), (33, 4, 80, 20), (7, 2, 6, 4), (3, 1, 2, 2),
                                        (2, 40, 512, 64), (300, 5, 96, 40), (1000, 28, 128, 128)])
def test_rope_types_and_sizes(inter, xd, yd, nt, nh, d, rd):
    for k, (scaling, kw) in enumerate(SCALINGS):
        if scaling == "ntk" and (rd or d) <= 2:
            continue
        x = rnd(nt * d + k, nt, nh, d, dtype=xd)
        pos = (np.arange(nt) * 37 + 11 * k).astype(np.int32)
        p = milo.rope_params(d, 1e4, rotary_dim=rd, interleaved=inter, scaling=scaling, **kw)
        m = 0.1 * math.log(kw["factor"]) + 1 if scaling == "yarn" else 1.0
        w = R.rope_freqs(rd or d, 1e4, scaling, **kw)
        for back in (False, True):
            y = milo.milo_rope(x, i32(pos.tolist()), p, out_dtype=yd, transpose=back)
            check_rope(x, pos, y, p, w, inter, m, back)
    ok()


def test_rope_far_and_negative_positions():
    pos = [2 ** 31 - 1, -2 ** 31, -1, 2 ** 24 + 1, 0]
    x = rnd(1, 5, 2, 128)
    p = milo.rope_params(128, 1e6)
    y = milo.milo_rope(x, i32(pos), p)
    # turns of at most 2^28.4, each of two factors rounded to 2^-53, and their product: 3 * 2^-24.6 turns
    check_rope(x, pos, y, p, R.rope_freqs(128, 1e6), extra=3 * 2.0 ** -24.6 * 2 * math.pi)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dt", [BF, F32])
def test_rope_strides_alignment_and_in_place(inter, dt):
    p = milo.rope_params(64, 1e4, rotary_dim=32, interleaved=inter)
    w = R.rope_freqs(32, 1e4)
    pos = list(range(3, 14))
    packed = rnd(5, 11, 7 * 64 + 3, dtype=dt)                      # odd row length: element-wise accesses
    for off in (0, 1, 8):
        x = packed[:, off:off + 5 * 64].view(11, 5, 64) if off == 8 else packed[:, off:off + 320].unflatten(1, (5, 64))
        y = milo.milo_rope(x, i32(pos), p)
        check_rope(x, pos, y, p, w, inter)
    heads_first = rnd(6, 5, 11, 64, dtype=dt).transpose(0, 1)     # [H][T][d] storage
    out = torch.full((5, 11, 64), 7.0, dtype=dt, device="cuda").transpose(0, 1)
    milo.milo_rope(heads_first, i32(pos), p, out=out)
    check_rope(heads_first, pos, out, p, w, inter)
    row = rnd(7, 1, 1, 64, dtype=dt)
    y = milo.milo_rope(row.expand(11, 5, 64), i32(pos), p)        # one row, broadcast
    check_rope(row.expand(11, 5, 64), pos, y, p, w, inter)
    big = rnd(8, 11, 9, 64, dtype=dt)
    keep = big.clone()
    milo.milo_rope(big[:, 2:7], i32(pos), p, out=big[:, 2:7])     # in place in a packed row: the others stay
    check_rope(keep[:, 2:7], pos, big[:, 2:7], p, w, inter)
    assert torch.equal(big[:, :2], keep[:, :2]) and torch.equal(big[:, 7:], keep[:, 7:])
    with pytest.raises(milo.MiloError):
        milo.milo_rope(big[:, 0:5], i32(pos), p, out=big[:, 2:7])
    e = milo.milo_rope(big[:0], i32(pos), p)
    assert e.shape == (0, 9, 64)


def test_rope_positions_repeat_over_layers():
    x = rnd(9, 12, 2, 128)
    pos = [5, 0, 900]
    p = milo.rope_params(128)
    check_rope(x, pos, milo.milo_rope(x, i32(pos), p), p, R.rope_freqs(128, 1e6))


def test_rope_more_than_2_to_32_threads():
    """One row for 2^32 + 5 tokens: indices that 32 bits do not hold."""
    n, p = 2 ** 32 + 5, milo.rope_params(2)
    x, pos = rnd(41, 1, 1, 2, dtype=BF), i32([12345])
    want = milo.milo_rope(x, pos, p).view(torch.int32).item()
    y = milo.milo_rope(x.expand(n, 1, 2), pos, p)
    assert y.shape == (n, 1, 2) and not (y.view(torch.int32) != want).any()
    ok()
    del y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradient(inter):
    """Against the formula (the transposed map) and against differences of the forward pass."""
    p = milo.rope_params(48, 100.0, rotary_dim=36, interleaved=inter, scaling="yarn", factor=4.0, orig_ctx=64)
    pos = i32([0, 1, 17, 5000])
    x, dy = rnd(10, 4, 3, 48), rnd(11, 4, 3, 48)
    dx = milo.milo_rope(dy, pos, p, transpose=True)
    check_rope(dy, pos.cpu().numpy(), dx, p, R.rope_freqs(36, 100.0, "yarn", factor=4.0, orig_ctx=64), inter,
               0.1 * math.log(4) + 1, True)
    # the map is linear: <R(x + h e) - R(x), dy> / h = dx . e for any step h; here h = 1 and e = a random direction
    e = rnd(12, 4, 3, 48)
    f = (milo.milo_rope(x + e, pos, p).double() - milo.milo_rope(x, pos, p).double())
    lhs, rhs = float((f * dy.double()).sum()), float((dx.double() * e.double()).sum())
    # 576 values with pairs of size at most 2 max: each side's roundings
    n = 576 * (2 * TURN * 1.14 + 2.0 ** -22) * 2 * float((x.abs().max() + e.abs().max()) * dy.abs().max())
    assert abs(lhs - rhs) <= n


# ------------------------------------------------------------------- cache
def make(L, S, H, cap, bl, dtype, fill=0xFF):
    """A cache whose untouched bytes are NaN scales, NaN e4m3 codes and infinite zeros."""
    c = milo.KvCache(milo.kv_shape(L, S, H, cap, bl, dtype))
    c.buf.fill_(fill)
    return c


def sections(c):
    """The cache's sections as numpy arrays over all layers (codes as numbers)."""
    s, o = c.shape, milo.milo_kv_layout(c.shape)
    layer = milo.milo_kv_cache_size(s) // s.L
    raw = c.buf[:s.L * layer].cpu().numpy().reshape(s.L, layer)
    kind = {v: k for k, v in milo.KV_DTYPES.items()}[s.dtype]
    row, par = (64, 16) if kind == "int4" else (128, 4)
    rows, n_b = s.S * s.H * s.cap, c.n_b
    got = {}
    for i, name in ((0, "k"), (1, "v")):
        b = np.ascontiguousarray(raw[:, o[i]:o[i] + rows * row]).reshape(s.L, s.S, s.H, s.cap, row)
        if kind == "int4":
            got[name] = np.stack([b & 15, b >> 4], -1).reshape(s.L, s.S, s.H, s.cap, 128).astype(np.float64)
        elif kind == "int8":
            got[name] = b.view(np.int8).astype(np.float64)
        else:
            got[name] = torch.from_numpy(b).view(torch.float8_e4m3fn).double().numpy()
        p = np.ascontiguousarray(raw[:, o[2 + i]:o[2 + i] + rows * par])
        got[name + "p"] = p.view(np.float16).reshape(s.L, s.S, s.H, s.cap, 4, 2) if kind == "int4" else \
            p.view(np.float32).reshape(s.L, s.S, s.H, s.cap)
    nb = s.S * s.H * n_b
    b = np.ascontiguousarray(raw[:, o[4]:o[4] + nb * 512]).view(np.uint16).astype(np.uint32) << 16
    got["bounds"] = b.view(np.float32).reshape(s.L, s.S, s.H, n_b, 2, 128)
    got["codes"] = np.ascontiguousarray(raw[:, o[5]:o[5] + nb * 256]).view(np.int8).reshape(s.L, s.S, s.H, n_b, 2, 128)
    got["scale"] = np.ascontiguousarray(raw[:, o[6]:o[6] + nb * 4]).view(np.float32).reshape(s.L, s.S, s.H, n_b)
    return got, kind


def append(c, k, v, start, count=None):
    milo.milo_kv_append(c, k, v, i32(start), None if count is None else i32(count))


def f32np(t):
    return t.float().cpu().numpy()


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("bl", [16, 48, 64])
def test_append_codes_bounds_and_untouched_bytes(dtype, dt, bl):
    L, S, H, cap, n = 2, 4, 3, 150, 70
    c = make(L, S, H, cap, bl, dtype)
    before, _ = sections(c)
    k, v = rnd(1, L, S, H, n, 128, dtype=dt, scale=3.0), rnd(2, L, S, H, n, 128, dtype=dt)
    k[0, 0, 0, 0] = 0.0                                         # a row of zeros
    k[0, 0, 0, 1] = 2.5                                         # a constant row
    k[0, 0, 1, 2, 5:] = 1e-30
    v[1, 1, 1, 3] *= 1e4
    start, count = [0, 80, 33, 7], [70, 70, 1, 0]
    append(c, k, v, start, count)
    ok()
    got, _ = sections(c)
    kn, vn = f32np(k), f32np(v)
    touched = np.zeros((S, cap), bool)
    for s in range(S):
        touched[s, start[s]:start[s] + count[s]] = True
        for name, x in (("k", kn), ("v", vn)):
            q, p = R.quantise(x[:, s, :, :count[s]], dtype)
            rows = slice(start[s], start[s] + count[s])
            np.testing.assert_array_equal(got[name][:, s, :, rows], q)
            np.testing.assert_array_equal(got[name + "p"][:, s, :, rows], p)
    for name in ("k", "v", "kp", "vp"):                         # the others are as they were
        a, b = np.moveaxis(got[name], 2, 1)[:, :, ~touched], np.moveaxis(before[name], 2, 1)[:, :, ~touched]
        assert a.tobytes() == b.tobytes()
    for s in range(S):
        for b in range(c.n_b):
            t = np.arange(max(b * bl, start[s]), min((b + 1) * bl, start[s] + count[s]))
            if not t.size:
                assert got["bounds"][:, s, :, b].tobytes() == before["bounds"][:, s, :, b].tobytes()
                assert got["codes"][:, s, :, b].tobytes() == before["codes"][:, s, :, b].tobytes()
            elif start[s] <= b * bl:                            # begun here: the bounds of these rows alone
                x = kn[:, s, :, t - start[s]]
                x = np.moveaxis(x, 0, 2) if x.shape[0] == t.size else x
                lo, hi = R.outward(x.min(2), False), R.outward(x.max(2), True)
                np.testing.assert_array_equal(got["bounds"][:, s, :, b], np.stack([lo, hi], -2))
                q, p = R.bound_codes(lo, hi)
                np.testing.assert_array_equal(got["codes"][:, s, :, b], q)
                np.testing.assert_array_equal(got["scale"][:, s, :, b], p)


@pytest.mark.parametrize("dtype", KINDS)
def test_append_token_by_token_equals_at_once(dtype):
    L, S, H, cap, bl, n = 1, 2, 2, 70, 32, 67
    k, v = rnd(3, L, S, H, n, 128), rnd(4, L, S, H, n, 128)
    a, b = make(L, S, H, cap, bl, dtype), make(L, S, H, cap, bl, dtype)
    append(a, k, v, [0, 3])
    append(b, k[:, :, :, :1], v[:, :, :, :1], [0, 3])
    # session 1 begins inside a block: its bounds go on from what the buffer held; give both the same
    for t in range(1, n):
        append(b, k[:, :, :, t:t + 1], v[:, :, :, t:t + 1], [t, t + 3])
    ok()
    ga, gb = sections(a)[0], sections(b)[0]
    for name in ga:
        x, y = (ga[name][:, :1], gb[name][:, :1]) if name in ("bounds", "codes", "scale") else (ga[name], gb[name])
        np.testing.assert_array_equal(x, y)


def test_append_strides_of_a_packed_projection():
    L, S, H, n = 2, 3, 2, 19
    qkv = rnd(5, L, S, n, 12, 128, dtype=BF)                     # [L][S][token][q heads | k heads | v heads][d]
    k, v = qkv[..., 8:10, :].transpose(2, 3), qkv[..., 10:12, :].transpose(2, 3)
    a, b = make(L, S, H, 32, 16, "int8"), make(L, S, H, 32, 16, "int8")
    append(a, k, v, [0, 4, 13])
    append(b, k.contiguous(), v.contiguous(), [0, 4, 13])
    ok()
    assert torch.equal(a.buf, b.buf)
    one = rnd(6, 1, 1, 1, 1, 128).expand(L, S, H, n, 128)        # one row everywhere: strides of 0
    append(a, one, one, [0, 0, 0])
    append(b, one.contiguous(), one.contiguous(), [0, 0, 0])
    assert torch.equal(a.buf, b.buf)


@pytest.mark.parametrize("dtype", KINDS)
def test_append_one_token_of_a_strided_view(dtype):
    """A dimension of one index may have any stride."""
    a, b = make(1, 2, 3, 32, 16, dtype), make(1, 2, 3, 32, 16, dtype)
    x = rnd(50, 2, 2, 3, 130 * 8)[:, :, :, :128]
    k, v = (x[i].as_strided((1, 2, 3, 1, 128), (7, 3 * 1040, 1040, 5, 1), x[i].storage_offset()) for i in (0, 1))
    append(a, k, v, [0, 31])
    append(b, k.contiguous(), v.contiguous(), [0, 31])
    ok()
    assert torch.equal(a.buf, b.buf)


@pytest.mark.parametrize("dtype", KINDS)
def test_append_bad_ranges_and_values(dtype):
    L, S, H, cap = 1, 5, 1, 40
    c = make(L, S, H, cap, 16, dtype)
    keep = c.buf.clone()
    k = rnd(7, L, S, H, 8, 128)
    append(c, k, k, [-1, 33, 2 ** 31 - 1, 0, 0], [8, 8, 8, 9, -1])
    ok(milo.MILO_ERR_BOUNDS)
    assert torch.equal(c.buf, keep)
    ok()
    k[0, 0, 0, 0, 3], k[0, 0, 0, 1, 4], k[0, 0, 0, 2, 5] = math.nan, math.inf, -math.inf
    append(c, k, k, [0] * 5)
    ok(milo.MILO_ERR_NONFINITE)
    z = f32np(torch.where(torch.isfinite(k), k, 0.0))
    got, _ = sections(c)
    q, p = R.quantise(z, dtype)
    np.testing.assert_array_equal(got["k"][:, :, :, :8], q)
    np.testing.assert_array_equal(got["vp"][:, :, :, :8], p)
    x = k.nan_to_num(0, 0, 0)
    x[0, 0, 0, 0, 0], x[0, 0, 0, 0, 1], x[0, 0, 0, 1, 0] = 1e38, -1e38, 65504.0
    append(c, x, x, [0] * 5)
    ok(milo.MILO_ERR_NONFINITE if dtype == "int4" else milo.MILO_OK)
    z = f32np(x.clamp(-65504, 65504) if dtype == "int4" else x)
    got, _ = sections(c)
    np.testing.assert_array_equal(got["k"][:, :, :, :8], R.quantise(z, dtype)[0])


def test_append_smallest_and_largest_values():
    BIG = torch.finfo(F32).max
    c = make(1, 1, 1, 16, 16, "int8")
    k = torch.zeros(1, 1, 1, 4, 128, device="cuda")
    k[..., 0, 0], k[..., 1, 0], k[..., 2, :], k[..., 3, :] = 1e-45, BIG, 1e-39, -BIG
    append(c, k, k, [0])
    ok()
    got, _ = sections(c)
    q, p = R.quantise(f32np(k), "int8")
    np.testing.assert_array_equal(got["k"][:, :, :, :4], q)
    np.testing.assert_array_equal(got["kp"][:, :, :, :4], p)
    assert np.isfinite(got["bounds"][0, 0, 0, 0]).all()


@pytest.mark.parametrize("dt", [BF, F32])
def test_int4_values_of_the_widest_groups_are_finite(dt):
    """Groups that span fp16: the highest code's value must not round past its end."""
    n = 64
    x = rnd(51, 1, 1, 1, n, 128, dtype=dt)
    x[..., 0::32] = 65504.0 if dt == F32 else 65280.0            # bf16 above 65280 is 65536
    x[..., 1::32] = -65504.0 if dt == F32 else -65280.0
    low = -40336.0 + 16 * torch.arange(n // 2, device="cuda")     # zeros that are rounded up by half a step
    x[..., :n // 2, 1::32] = low.to(dt)[:, None]
    c = make(1, 1, 1, n, 16, "int4")
    append(c, x, x, [0])
    ok(milo.MILO_ERR_NONFINITE if dt == F32 else milo.MILO_OK)
    z = f32np(x.clamp(-65440, 65440) if dt == F32 else x)
    q, p = R.quantise(z, "int4")
    got, _ = sections(c)
    np.testing.assert_array_equal(got["k"], q)
    np.testing.assert_array_equal(got["kp"], p)
    k, v = milo.milo_kv_read(c, i32([0]), n)
    assert torch.isfinite(k).all() and torch.equal(k, v)
    np.testing.assert_array_equal(f32np(k), R.values(q, p, "int4").astype(np.float32))
    for n_q in (1, 40):                                          # both attention kernels
        check_attn(c, rnd(52, 1, 1, n_q, 2, 128, scale=1e-6), [n])


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("out", [BF, F32])
def test_read_back(dtype, out):
    L, S, H, cap, n = 2, 3, 2, 90, 37
    c = make(L, S, H, cap, 32, dtype)
    k, v = rnd(8, L, S, H, cap, 128), rnd(9, L, S, H, cap, 128)
    append(c, k, v, [0] * 3)
    start, count = [0, 53, 20], [37, 37, 5]
    ko, vo = (torch.full((L, S, H, n, 128), 7.0, dtype=out, device="cuda") for _ in range(2))
    milo.milo_kv_read(c, i32(start), n, i32(count), ko, vo)
    ok()
    for x, y in ((k, ko), (v, vo)):
        q, p = R.quantise(f32np(x), dtype)
        ref = R.values(q, p, dtype).astype(np.float32)          # one rounding to fp32, as the kernel's product
        for s in range(S):
            want = torch.from_numpy(ref[:, s, :, start[s]:start[s] + count[s]]).to(out)
            assert torch.equal(y[:, s, :, :count[s]].cpu(), want)
            assert (y[:, s, :, count[s]:] == 7.0).all()
    keep = ko.clone()
    milo.milo_kv_read(c, i32([-1, 54, 2 ** 31 - 1]), n, None, ko, vo)
    ok(milo.MILO_ERR_BOUNDS)
    assert torch.equal(ko, keep)
    assert milo.lib().milo_kv_read(c.shape, c.buf.data_ptr(), c.buf.numel(), n, i32(start).data_ptr(), None, None,
                                   vo.data_ptr(), milo.MILO_BF16 if out == BF else milo.MILO_F32, None) == 0
    torch.cuda.synchronize()


# --------------------------------------------------------------- retrieval
def seen(length, n_q, i):
    return max(0, length - n_q + i + 1)


@pytest.mark.parametrize("G", [1, 3, 7, 8, 12, 20])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("bl,cap,n_q", [(16, 16, 1), (16, 1000, 2), (64, 5000, 1), (48, 333, 3)])
def test_select(G, dt, bl, cap, n_q):
    L, S, H = 2, 3, 2
    c = make(L, S, H, cap, bl, "int4")
    k = rnd(10, L, S, H, cap, 128)
    append(c, k, k, [0] * S)
    length = [cap, cap // 3, min(1, cap)]
    q = rnd(11, L, S, n_q, H * G, 128, dtype=dt)
    q[0, 0, 0, 0] = 0.0
    got, _ = sections(c)
    for n_sel, nf, nl in {(1, 0, 1), (1, 0, 0), (min(9, c.n_b), min(1, c.n_b - 1), 1), (c.n_b, 0, 0)}:
        sel, sc = milo.milo_kv_select(c, q, i32(length), n_sel, nf, nl, return_scores=True)
        assert torch.equal(sel, milo.milo_kv_select(c, q, i32(length), n_sel, nf, nl))
        sel, sc, qn = sel.cpu().numpy(), sc.cpu().numpy(), f32np(q)
        for l, s, i, h in np.ndindex(L, S, n_q, H):
            cand = -(-seen(length[s], n_q, i) // bl)
            ref = R.scores(qn[l, s, i, h * G:(h + 1) * G], got["codes"][l, s, h], got["scale"][l, s, h])
            np.testing.assert_array_equal(sc[l, s, i, h, :cand], ref[:cand])
            assert np.all(np.isneginf(sc[l, s, i, h, cand:]))
            np.testing.assert_array_equal(sel[l, s, i, h], R.top(ref, cand, n_sel, nf, nl))
    ok()


@pytest.mark.parametrize("S,H,cap,G", [(40, 4, 600, 7), (3, 2, 9000, 7), (30, 4, 9000, 8), (30, 4, 30000, 3), (4, 2, 1000, 12)])
def test_select_by_rows_and_blocks(S, H, cap, G):
    """Rows and blocks that one kernel takes, and that two do."""
    c = make(1, S, H, cap, 16, "int8")
    k = rnd(57, 1, S, H, cap, 128, dtype=BF)
    append(c, k, k, [0] * S)
    length = [cap - 7 * s for s in range(S)]
    length[:3] = [0, 1, 16 * 9]
    q = rnd(58, 1, S, H * G, 128)
    got, _ = sections(c)
    sel, sc = milo.milo_kv_select(c, q, i32(length), 9, 1, 2, return_scores=True)
    assert torch.equal(sel, milo.milo_kv_select(c, q, i32(length), 9, 1, 2))
    ok()
    sel, sc, qn = sel.cpu().numpy(), sc.cpu().numpy(), f32np(q)
    for s, h in np.ndindex(S, H):
        cand = -(-length[s] // 16)
        ref = R.scores(qn[0, s, h * G:(h + 1) * G], got["codes"][0, s, h], got["scale"][0, s, h])
        np.testing.assert_array_equal(sc[0, s, h, :cand], ref[:cand])
        assert np.all(np.isneginf(sc[0, s, h, cand:]))
        np.testing.assert_array_equal(sel[0, s, h], R.top(ref, cand, 9, 1, 2))


@pytest.mark.parametrize("n_b,n_sel,nf,nl", [(2500, 40, 2, 3), (2500, 2499, 0, 0), (9000, 100, 1, 1), (9000, 8500, 0, 0),
                                             (9000, 2, 1, 1)])
def test_select_many_blocks(n_b, n_sel, nf, nl):
    """More blocks than a small CTA's registers hold, and than a large one's; many equal scores."""
    cap = 16 * n_b
    c = make(1, 1, 1, cap, 16, "int4")
    k = rnd(14, 1, 1, 1, cap, 128)
    k[:, :, :, 16 * 100:16 * 2200] = k[:, :, :, :16].repeat(1, 1, 1, 2100, 1)
    append(c, k, k, [0])
    q = rnd(15, 1, 1, 2, 128)
    got, _ = sections(c)
    for length in (cap, cap - 16 * 50 - 3):
        sel, sc = milo.milo_kv_select(c, q, i32([length]), n_sel, nf, nl, return_scores=True)
        cand = -(-length // 16)
        ref = R.scores(f32np(q)[0, 0], got["codes"][0, 0, 0], got["scale"][0, 0, 0])
        np.testing.assert_array_equal(sc.cpu().numpy()[0, 0, 0, :cand], ref[:cand])
        np.testing.assert_array_equal(sel.cpu().numpy()[0, 0, 0], R.top(ref, cand, n_sel, nf, nl))
    ok()


def test_select_ties_lengths_and_bad_queries():
    L, S, H, cap, bl = 1, 5, 1, 640, 16
    c = make(L, S, H, cap, bl, "fp8")
    k = rnd(12, 1, 1, 1, bl, 128).repeat(L, S, H, cap // bl, 1)  # equal blocks: ties go to the lower ids
    append(c, k, k, [0] * S)
    q = rnd(13, L, S, 2, 128)
    sel = milo.milo_kv_select(c, q, i32([640, 0, 17, -3, 641]), 7, 0, 1).cpu().numpy()
    ok(milo.MILO_ERR_BOUNDS)
    assert sel[0, 0, 0].tolist() == [0, 1, 2, 3, 4, 5, 39]
    assert sel[0, 2, 0].tolist() == [0, 1, -1, -1, -1, -1, -1]
    assert (sel[0, [1, 3, 4]] == -1).all()
    q[0, 0, 0, 0], q[0, 2, 1, 5] = math.nan, math.inf
    want = milo.milo_kv_select(c, torch.where(torch.isfinite(q), q, 0.0), i32([640] * S), 3)
    ok()
    assert torch.equal(milo.milo_kv_select(c, q, i32([640] * S), 3), want)
    ok(milo.MILO_ERR_NONFINITE)
    z = milo.milo_kv_select(c, torch.zeros_like(q), i32([640] * S), 3, 0, 0)
    assert (z.cpu() == torch.tensor([0, 1, 2])).all()


def test_select_negative_and_zero_scores_order():
    """A block whose keys all point away scores below zero, and -0 ties with +0."""
    c = make(1, 1, 1, 64, 16, "int8")
    k = torch.zeros(1, 1, 1, 64, 128, device="cuda")
    k[..., :16, :], k[..., 16:32, :], k[..., 48:, :] = -1.0, 0.0, -1e-40
    append(c, k, k, [0])
    q = torch.ones(1, 1, 1, 128, device="cuda")
    assert milo.milo_kv_select(c, q, i32([64]), 2, 0, 0).flatten().tolist() == [1, 2]
    assert milo.milo_kv_select(c, -q, i32([64]), 1, 0, 0).flatten().tolist() == [0]


# --------------------------------------------------------------- attention
def check_attn(c, q, length, sel=None, scale=0.0, out=None, lse=None, status=milo.MILO_OK):
    """milo_kv_attn against 64 bits on the values that the cache holds."""
    if out is None:
        out, lse = milo.milo_kv_attn(c, q, i32(length), None if sel is None else i32(sel), scale, return_lse=True)
        ok(status)
    five = q.dim() == 5
    qn = np64(q if five else q[:, :, None])
    on = np64(out if five else out[:, :, None])
    ln = np64(lse if five else lse[:, :, None])
    got, kind = sections(c)
    L, S, n_q, Hq, _ = qn.shape
    H, bl = c.shape.H, c.shape.block_len
    G = Hq // H
    sel = None if sel is None else np.asarray(sel).reshape(L, S, n_q, H, -1)
    scale = scale or 128 ** -0.5
    for l, s, h in np.ndindex(L, S, H):
        n = length[s] if 0 <= length[s] <= c.shape.cap else 0
        k, v = (R.values(got[x][l, s, h, :n], got[x + "p"][l, s, h, :n], kind) for x in ("k", "v"))
        for i in range(n_q):
            t = np.arange(seen(n, n_q, i))
            if sel is not None:
                b = [x for x in sel[l, s, i, h] if 0 <= x < c.n_b]
                t = np.concatenate([np.arange(x * bl, min((x + 1) * bl, t.size)) for x in b] + [t[:0]]).astype(int)
            o, e, err, le = R.attn(qn[l, s, i, h * G:(h + 1) * G], k[t], v[t], scale, q.dtype == BF, HALF_STEP[q.dtype])
            g = on[l, s, i, h * G:(h + 1) * G]
            assert np.all(np.abs(g - o) <= err), (l, s, h, i, np.max(np.abs(g - o) / err))
            w = ln[l, s, i, h * G:(h + 1) * G]
            if t.size == 0:
                assert np.all(g == 0) and np.all(np.isneginf(w))
            else:
                assert np.all(np.abs(w - e) <= le), (l, s, h, i, np.max(np.abs(w - e) / le))


def filled(L, S, H, cap, bl, dtype, length, seed=20, scale=1.0):
    """A cache that holds length[s] tokens; everything behind them is 0xFF."""
    c = make(L, S, H, cap, bl, dtype)
    n = max(1, max(length))
    k, v = rnd(seed, L, S, H, n, 128, scale=scale), rnd(seed + 1, L, S, H, n, 128)
    append(c, k, v, [0] * S, [min(x, n) for x in length])
    ok()
    return c


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("G,H", [(1, 1), (7, 2), (8, 1), (12, 1), (5, 3)])
def test_attn_lengths(dtype, dt, G, H):
    length = [0, 1, 15, 16, 17, 64, 257, 300]
    c = filled(1, len(length), H, 300, 64, dtype, length)
    check_attn(c, rnd(21, 1, len(length), H * G, 128, dtype=dt), length)


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n_q,G", [(2, 1), (3, 7), (17, 4), (40, 2)])
def test_attn_several_queries(dtype, dt, n_q, G):
    length = [0, 1, n_q - 1, n_q, 100, 203]
    c = filled(2, len(length), 2, 203, 16, dtype, length)
    check_attn(c, rnd(22, 2, len(length), n_q, 2 * G, 128, dtype=dt), length)


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n_q,G,H", [(40, 7, 1), (1, 20, 2), (128, 1, 2), (129, 1, 1), (5, 4, 3)])
def test_attn_many_query_rows(dtype, dt, n_q, G, H):
    """More than 16 rows a line, below, at and above one tile of 128, over many tiles of tokens."""
    length = [3000, 0, 1500, n_q, 127, 128, 129]
    c = filled(1, len(length), H, 3000, 32, dtype, length)
    check_attn(c, rnd(43, 1, len(length), n_q, G * H, 128, dtype=dt), length)


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("cap,n_q,G", [(5000, 1, 7), (5000, 1, 12), (5000, 2, 3), (5000, 40, 4), (2048, 1, 8), (1024, 1, 12), (128, 9, 5)])
def test_attn_short_lengths_of_long_and_short_caches(cap, dtype, dt, n_q, G):
    """The same lengths where lines may be split over CTAs, and where a CTA takes a whole one."""
    length = [0, 1, 15, 16, 17, 64, 127, 128, 100, 3, 128, 0]
    for S in (2, 12):                                            # few lines and many
        c = filled(1, S, 4, cap, 64, dtype, length[-S:])
        q = rnd(56, 1, S, n_q, 4 * G, 128, dtype=dt)
        check_attn(c, q, length[-S:])
        sel = np.random.default_rng(cap).integers(-1, c.n_b, (1, S, n_q, 4, min(40, c.n_b))).astype(np.int32)
        sel[..., :2] = [1, 0]
        check_attn(c, q, length[-S:], sel.tolist())


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("dt", [BF, F32])
def test_attn_many_query_rows_large_and_small_values(dtype, dt):
    """The references and the value scales rise along the tiles: the output is rescaled."""
    L, S, H, n, n_q = 1, 2, 1, 900, 24
    c = make(L, S, H, n, 16, dtype)
    k, v = rnd(44, L, S, H, n, 128), rnd(45, L, S, H, n, 128)
    k *= torch.linspace(0.5, 6, n).cuda()[:, None]
    if dtype != "int4":
        v *= torch.exp2(torch.linspace(-30, 30, n).round()).cuda()[:, None]
    k[0, 0, 0, 5], v[0, 0, 0, 7], k[0, 1] = 0.0, 0.0, 0.0
    append(c, k, v, [0] * S)
    q = rnd(46, L, S, n_q, 2, 128, dtype=dt)
    q[0, 0, 3] *= 30.0
    q[0, 0, 4] *= 1e-20
    q[0, 0, 5] = 0.0
    check_attn(c, q, [n, 333])
    q[0, 0, 6, 1, 9], q[0, 0, 7, 0, 0] = math.nan, math.inf
    out, lse = milo.milo_kv_attn(c, q, i32([n, 333]), return_lse=True)
    ref, rl = milo.milo_kv_attn(c, torch.where(torch.isfinite(q), q, 0.0), i32([n, 333]), return_lse=True)
    bad = ~torch.isfinite(q).all(-1)
    assert torch.equal(out[~bad], ref[~bad]) and torch.equal(lse[~bad], rl[~bad])
    assert int(bad.sum()) == 2 and not torch.isfinite(out[bad]).any() and not torch.isfinite(lse[bad]).any()
    ok()


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("bl,n_q,G", [(16, 1, 7), (48, 2, 3), (64, 1, 8), (128, 1, 12), (32, 1, 20)])
def test_attn_selected_blocks(dtype, dt, bl, n_q, G):
    L, S, H, cap = 2, 4, 2, 700
    length = [700, 333, 1, 0]
    c = filled(L, S, H, cap, bl, dtype, length)
    g = np.random.default_rng(bl)
    sel = g.integers(-1, c.n_b, (L, S, n_q, H, 5)).astype(np.int32)   # any order, some twice, some none, some unseen
    sel[0, 0, 0, 0] = -1                                              # nothing selected
    sel[1, 0, 0, 1] = c.n_b - 1
    q = rnd(23, L, S, n_q, H * G, 128, dtype=dt)
    check_attn(c, q, length, sel.tolist())
    if n_q == 1:
        check_attn(c, q[:, :, 0].contiguous(), length, sel[:, :, 0].tolist())


def test_attn_bad_ids_and_lengths():
    c = filled(1, 3, 1, 64, 16, "int8", [64, 40, 64])
    q = rnd(24, 1, 3, 2, 128)
    check_attn(c, q, [64, 40, 64], [[[[0, 4, 2]], [[-2, 1, 99]], [[2 ** 31 - 1, -2 ** 31, -1]]]],
               status=milo.MILO_ERR_BOUNDS)
    check_attn(c, q, [-1, 40, 65], status=milo.MILO_ERR_BOUNDS)
    check_attn(c, q, [64, 2 ** 31 - 1, -2 ** 31], status=milo.MILO_ERR_BOUNDS)


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("dt", [BF, F32])
def test_attn_long_and_ragged(dtype, dt):
    length = [9000, 3, 4097, 640]
    c = filled(1, 4, 2, 9000, 64, dtype, length)
    q = rnd(25, 1, 4, 14, 128, dtype=dt)
    check_attn(c, q, length)
    check_attn(c, q, length, scale=0.5)
    sel = milo.milo_kv_select(c, q, i32(length), 20, 1, 2)
    check_attn(c, q, length, sel.cpu().tolist())


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("dtype", KINDS)
def test_attn_large_and_small_values(dtype, dt):
    """Scores of hundreds, tiny and huge queries, values whose scales span 2^60, rows of zeros."""
    L, S, H, n = 1, 3, 1, 130
    c = make(L, S, H, 160, 16, dtype)
    k, v = rnd(26, L, S, H, n, 128, scale=4.0), rnd(27, L, S, H, n, 128)
    if dtype != "int4":
        v *= torch.exp2(torch.randint(-30, 31, (L, S, H, n, 1), generator=torch.Generator().manual_seed(3))).cuda()
    k[0, 0, 0, 5], v[0, 0, 0, 7], k[0, 1] = 0.0, 0.0, 0.0
    append(c, k, v, [0] * S)
    q = rnd(28, L, S, 5, 128, dtype=dt)
    q[0, 0, 0] *= 100.0
    q[0, 0, 1] *= 1e-20
    q[0, 0, 2] = 0.0
    q[0, 2, 0] *= 1e-3
    q[0, 2, 1, 1:] *= 1e-6                                       # one loud channel
    check_attn(c, q, [n, n, 77])
    check_attn(c, q, [n, n, 77], [[[[0, 3, 8]], [[2, 2, 2]], [[4, 1, 0]]]])


def test_attn_query_that_is_not_finite_spoils_its_own_row_alone():
    c = filled(1, 1, 1, 40, 16, "int8", [40])
    q = rnd(29, 1, 1, 8, 128)
    q[0, 0, 3, 5], q[0, 0, 6, 0] = math.nan, math.inf
    out, lse = milo.milo_kv_attn(c, q, i32([40]), return_lse=True)
    clean = torch.where(torch.isfinite(q), q, 0.0)
    ref, rl = milo.milo_kv_attn(c, clean, i32([40]), return_lse=True)
    good = [0, 1, 2, 4, 5, 7]
    assert torch.equal(out[:, :, good], ref[:, :, good]) and torch.equal(lse[:, :, good], rl[:, :, good])
    assert not torch.isfinite(out[0, 0, [3, 6]]).any()
    ok()


def test_attn_same_call_same_bits():
    length = [9000, 3, 4097, 640]
    c = filled(1, 4, 2, 9000, 64, "int8", length)
    q = rnd(30, 1, 4, 14, 128)
    a = milo.milo_kv_attn(c, q, i32(length))
    for _ in range(3):
        assert torch.equal(a, milo.milo_kv_attn(c, q, i32(length)))


def test_attn_writes_only_its_output():
    c = filled(1, 2, 1, 50, 16, "fp8", [50, 0])
    q = rnd(31, 1, 2, 3, 128, dtype=BF)
    buf = torch.full((2 * 3 * 128 + 256,), 7.0, dtype=BF, device="cuda")
    n = milo.milo_kv_attn_workspace_size(c.shape, 1, 3)
    ws = torch.full((n + 512,), 0xAB, dtype=torch.uint8, device="cuda")
    keep = c.buf.clone()
    milo.milo_kv_attn(c, q, i32([50, 0]), out=buf[128:-128].view(1, 2, 3, 128), workspace=ws[:n])
    ok()
    assert (buf[:128] == 7).all() and (buf[-128:] == 7).all() and (ws[n:] == 0xAB).all() and torch.equal(c.buf, keep)


# ------------------------------------------------- as they are used together
def test_rows_behind_4_gigabytes():
    """A session whose last rows lie behind 2^32 bytes: written, read, picked and attended."""
    H, cap, bl, n = 2, 2 ** 25 + 4099, 1024, 50
    c = make(1, 1, H, cap, bl, "int8", fill=0)                   # zero rows: score 0, value 0
    k, v = rnd(53, 1, 1, H, n, 128), rnd(54, 1, 1, H, n, 128)
    append(c, k, v, [cap - n])
    ko, vo = milo.milo_kv_read(c, i32([cap - n]), n)
    kr, vr = (R.values(*R.quantise(f32np(x), "int8"), "int8") for x in (k, v))
    assert np.array_equal(f32np(ko), kr.astype(np.float32)) and np.array_equal(f32np(vo), vr.astype(np.float32))
    q = (2 * k[:, :, :, -1]).contiguous()                        # [1][1][Hq = H][128]
    sel = milo.milo_kv_select(c, q, i32([cap]), 2, 0, 0)
    assert sel.cpu().numpy().tolist() == [[[[c.n_b - 2, c.n_b - 1]] * H]]
    for picked in (None, sel):
        o, lse = milo.milo_kv_attn(c, q, i32([cap]), picked, return_lse=True)
        ok()
        zeros = (cap if picked is None else bl + cap % bl) - n     # the rows lie in the last two blocks
        for h in range(H):
            qn = np64(q)[0, 0, h]
            s = kr[0, 0, h] @ qn * 128 ** -0.5
            w = np.exp(s)
            total = w.sum() + zeros
            # roundings as R.attn counts them; a thread adds at most cap / 16 / 1184 * 2 < 4096 weights, the parts are fewer
            rel = 2.0 ** -23 * (28 * (np.abs(kr[0, 0, h]) @ np.abs(qn)) * 128 ** -0.5 + np.abs(s)) + 2.0 ** -21 + 2.0 ** -11
            ref = w @ vr[0, 0, h] / total
            tol = (w * rel) @ np.abs(vr[0, 0, h]) / total + rel.max() * np.abs(ref) + 2.0 ** -34 * np.abs(vr).max()
            assert np.all(np.abs(np64(o)[0, 0, h] - ref) <= tol)
            assert abs(np64(lse)[0, 0, h] - np.log(total)) <= rel.max() + 2.0 ** -23 * (1 + np.log(total))
    del c
    torch.cuda.empty_cache()


def test_attn_refuses_an_empty_selection():
    """No ids would be taken for no selection, which stands for every token."""
    c, q = filled(1, 1, 1, 32, 16, "int8", [32]), rnd(55, 1, 1, 2, 128)
    with pytest.raises(ValueError, match="at least one block"):
        milo.milo_kv_attn(c, q, i32([32]), torch.empty(1, 1, 1, 0, dtype=torch.int32, device="cuda"))


def test_one_layer_of_a_cache_is_a_cache():
    L, S, H = 3, 2, 2
    a, b = make(L, S, H, 50, 16, "int4"), make(L, S, H, 50, 16, "int4")
    k, v = rnd(32, L, S, H, 50, 128, dtype=BF), rnd(33, L, S, H, 50, 128, dtype=BF)
    q = rnd(34, L, S, 6, 128, dtype=BF)
    append(a, k, v, [0, 0])
    whole = milo.milo_kv_attn(a, q, i32([50, 31]))
    for l in range(L):
        append(b.layer(l), k[l:l + 1], v[l:l + 1], [0, 0])
        assert torch.equal(milo.milo_kv_attn(b.layer(l), q[l:l + 1], i32([50, 31])), whole[l:l + 1])
    assert torch.equal(a.buf, b.buf)


def _steps(c, qkv, start, G, n_steps, stream=None, n_sel=3):
    """A few decode steps as a model makes them: turn, append, pick blocks, attend."""
    L, S, H = c.shape.L, c.shape.S, c.shape.H
    p = milo.rope_params(128, 1e4)
    length = start.clone()
    outs = []
    for t in range(n_steps):
        x = qkv[t]                                               # [L][S][(G + 2) H][128]
        n = (G + 1) * H
        r = milo.milo_rope(x.view(L * S, (G + 2) * H, 128)[:, :n], length, p, stream=stream).view(L, S, n, 128)
        v = x[:, :, n:].unsqueeze(3)
        k = r[:, :, G * H:].unsqueeze(3)
        milo.milo_kv_append(c, k.contiguous(), v.contiguous(), length, stream=stream)
        length = length + 1
        q = r[:, :, :G * H].contiguous()
        sel = milo.milo_kv_select(c, q, length, n_sel, 1, 1, stream=stream)
        outs.append((milo.milo_kv_attn(c, q, length, sel, stream=stream), q, sel, length))
    return outs


@pytest.mark.parametrize("dtype", KINDS)
def test_decode_steps(dtype):
    L, S, H, G, bl = 2, 3, 2, 4, 16
    c = make(L, S, H, 120, bl, dtype)
    k, v = rnd(35, L, S, H, 90, 128, dtype=BF), rnd(36, L, S, H, 90, 128, dtype=BF)
    start = [90, 31, 0]
    append(c, k, v, [0] * 3, start)
    qkv = rnd(37, 6, L, S, (G + 2) * H, 128, dtype=BF)
    for out, q, sel, length in _steps(c, qkv, i32(start), G, 6):
        assert (length.cpu() <= 120).all()
    ok()
    # the last step, whose cache is the one that is held now
    _, lse = milo.milo_kv_attn(c, q, length, sel, return_lse=True)
    check_attn(c, q, length.tolist(), sel.cpu().tolist(), out=out, lse=lse)


def test_two_streams_and_a_captured_graph():
    L, S, H, G = 1, 2, 1, 3
    qkv = rnd(38, 4, L, S, (G + 2) * H, 128, dtype=BF)
    k = rnd(39, L, S, H, 40, 128, dtype=BF)

    def fresh():
        c = make(L, S, H, 64, 16, "int8")
        append(c, k, k, [0, 0], [40, 7])
        return c
    want = [o[0] for o in _steps(fresh(), qkv, i32([40, 7]), G, 4)]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    ca, cb = fresh(), fresh()
    torch.cuda.synchronize()
    got = {}
    for s, c in ((a, ca), (b, cb)):
        with torch.cuda.stream(s):
            got[s] = [o[0] for o in _steps(c, qkv, i32([40, 7]), G, 4)]
    torch.cuda.synchronize()
    for s in (a, b):
        assert all(torch.equal(x, y) for x, y in zip(got[s], want))
    # captured once, replayed on other inputs
    c, start, x = fresh(), i32([40, 7]), torch.zeros_like(qkv)
    _steps(fresh(), x, start, G, 4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = [o[0] for o in _steps(c, x, start, G, 4)]
    x.copy_(qkv)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    ok()


# -------------------------------------- with the compressed blocks, one softmax
def test_decode_over_compressed_blocks_and_cache(oracle_mod):
    w = synth.WORKLOADS["qwen3b-1layer"]
    K, V = synth.workload_cache(w)
    f = milo.milo_compress(K.cuda(), V.cuda(), w.block_len, milo.default_params(factor_dtype="bf16"))
    q, sel, pos = (t.cuda() for t in synth.decode_inputs(w))
    S = q.shape[1]
    plain = milo.milo_decode_attn(f, q, sel, pos, rope_base=w.rope_base)
    for dtype in KINDS:
        c = make(w.L, S, w.H, 200, 16, dtype)
        k, v = rnd(40, w.L, S, w.H, 150, 128), rnd(41, w.L, S, w.H, 150, 128)
        append(c, k, v, [0] * S)
        empty = milo.milo_decode_attn_kv(f, q, sel, c, i32([0] * S), positions=pos, rope_base=w.rope_base)
        assert torch.equal(empty, plain)
        kt, vt = milo.milo_kv_read(c, i32([0] * S), 150)
        for n in (1, 150):
            # the same tokens as a plain fp32 tail: the two tail kernels share the merge, so the difference is
            # theirs alone, at most that of fp32 attention over 150 tokens of size 1
            want = milo.milo_decode_attn_tail(f, q, sel, kt, vt, i32([n] * S), pos, rope_base=w.rope_base)
            got = milo.milo_decode_attn_kv(f, q, sel, c, i32([n] * S), positions=pos, rope_base=w.rope_base)
            assert float((got - want).abs().max()) <= 2e-5 * float(want.abs().max())
        ks = torch.tensor([3, 0, -1], dtype=torch.int32).repeat(w.L, S, w.H, 1).cuda()
        got = milo.milo_decode_attn_kv(f, q, sel, c, i32([150] * S), ks, pos, rope_base=w.rope_base)
        idx = torch.cat([torch.arange(48, 64), torch.arange(0, 16)]).cuda()
        want = milo.milo_decode_attn_tail(f, q, sel, kt[:, :, :, idx].contiguous(), vt[:, :, :, idx].contiguous(),
                                          i32([32] * S), pos, rope_base=w.rope_base)
        assert float((got - want).abs().max()) <= 2e-5 * float(want.abs().max())
    ok()
    L = milo.lib()
    other = milo.kv_shape(w.L, S + 1, w.H, 200, 16, "int8")
    big = torch.zeros(milo.milo_kv_cache_size(other), dtype=torch.uint8, device="cuda")
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    args = (f.handle, q.data_ptr(), S, w.Hq, sel.data_ptr(), pos.data_ptr(), sel.shape[1], 1e6, ctypes.byref(other),
            big.data_ptr(), big.numel(), i32([0] * (S + 1)).data_ptr(), None, 0, plain.data_ptr(), ws.data_ptr())
    assert L.milo_decode_attn_kv(*args, ws.numel(), None) == milo.MILO_ERR_INVALID_ARG
    n = L.milo_decode_kv_workspace_size(f.handle, S, w.Hq, sel.shape[1], ctypes.byref(c.shape), 0)
    args = args[:8] + (ctypes.byref(c.shape), c.buf.data_ptr(), c.buf.numel()) + args[11:]
    assert L.milo_decode_attn_kv(*args, n - 1, None) == milo.MILO_ERR_WORKSPACE


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("G", [3, 12, 20])
def test_decode_over_blocks_and_cache_by_group_size(dtype, G):
    """Query groups of each attention kernel, more tokens than one CTA takes."""
    w = synth.WORKLOADS["toy"]
    K, V = synth.workload_cache(w)
    f = milo.milo_compress(K.cuda(), V.cuda(), w.block_len, milo.default_params(factor_dtype="f32"))
    S = 2
    q = rnd(47, 1, S, G, 128)
    sel = i32([[0, 3], [5, 1]])
    c = make(1, S, 1, 5000, 64, dtype)
    k, v = rnd(48, 1, S, 1, 5000, 128), rnd(49, 1, S, 1, 5000, 128)
    append(c, k, v, [0] * S)
    kt, vt = milo.milo_kv_read(c, i32([0] * S), 5000)
    for length in ([5000, 17], [0, 1], [0, 0]):
        want = milo.milo_decode_attn_tail(f, q, sel, kt, vt, i32(length))
        got = milo.milo_decode_attn_kv(f, q, sel, c, i32(length))
        # both in fp32 sums over 5000 tokens of size 1: their bounds in R.attn, a few 1e-4 of the largest value
        assert float((got - want).abs().max()) <= 2e-4 * float(want.abs().max())
        if length == [0, 0]:
            assert torch.equal(got, milo.milo_decode_attn(f, q, sel))
    ok()


def test_stage_timing_counts_the_calls():
    c = filled(1, 1, 1, 40, 16, "int8", [40])
    q = rnd(42, 1, 1, 2, 128)
    milo.milo_timing_enable()
    milo.milo_rope(q.view(1, 2, 128), i32([3]), milo.rope_params(128))
    milo.milo_kv_read(c, i32([0]), 4)
    append(c, q[:, :, :1, None], q[:, :, :1, None], [3])
    milo.milo_kv_attn(c, q, i32([40]), milo.milo_kv_select(c, q, i32([40]), 2))
    t = milo.milo_timing_read()
    milo.milo_timing_enable(False)
    for name in ("rope", "kv_write", "kv_read", "kv_select", "kv_attn"):
        assert t[name][1] == 1 and t[name][0] > 0


@pytest.mark.parametrize("workload,factors", [("toy", "f32"), ("qwen3b-1layer", "bf16")])
@pytest.mark.parametrize("dtype", KINDS)
def test_decode_over_blocks_and_cache_shows_queries_that_are_not_finite(dtype, workload, factors):
    """As milo_kv_attn: such a row is not finite, and its neighbours are what they were."""
    w = synth.WORKLOADS[workload]
    K, V = synth.workload_cache(w)
    f = milo.milo_compress(K.cuda(), V.cuda(), w.block_len, milo.default_params(factor_dtype=factors))
    S, Hq = 2, 4 * w.H
    q = rnd(60, w.L, S, Hq, 128)
    sel = i32([[0, 3], [2, 1]])
    c = filled(w.L, S, w.H, 100, 16, dtype, [100, 100], seed=61)
    call = lambda x, n: milo.milo_decode_attn_kv(f, x, sel, c, i32(n))  # noqa: E731
    want = call(q, [100, 37])
    bad = q.clone()
    bad[0, 0, 1, 5], bad[0, 1, 3, 0] = math.nan, math.inf
    got = call(bad, [100, 37])
    rows = ~torch.isfinite(bad).all(-1)
    assert int(rows.sum()) == 2 and not torch.isfinite(got[rows]).any()
    # both factor types against their own call without the two rows; half precision's weights may move by a reference's change
    near = 0.0 if factors == "f32" else 1e-3
    assert float((got[~rows] - want[~rows]).abs().max()) <= near * float(want.abs().max())
    # nothing cached: milo_decode_attn's output, whatever the queries are
    alone = milo.milo_decode_attn(f, bad, sel)
    assert torch.equal(call(bad, [0, 0]).view(torch.int32), alone.view(torch.int32))
    ok()


def test_decode_over_blocks_and_cache_shows_scores_that_overflow():
    """Scores past fp32's end in the cache do not leave the blocks' output standing alone."""
    w = synth.WORKLOADS["toy"]
    K, V = synth.workload_cache(w)
    f = milo.milo_compress(K.cuda(), V.cuda(), w.block_len, milo.default_params(factor_dtype="f32"))
    c = make(1, 1, 1, 32, 16, "int8")
    k = rnd(62, 1, 1, 1, 20, 128)
    append(c, k * 1e30, k, [0])
    q = rnd(63, 1, 1, 3, 128)
    q[0, 0, 1] *= 1e12
    sel = i32([[0, 3]])
    alone = milo.milo_kv_attn(c, q, i32([20]))
    got = milo.milo_decode_attn_kv(f, q, sel, c, i32([20]))
    assert not torch.isfinite(alone[0, 0, 1]).any() and not torch.isfinite(got[0, 0, 1]).any()
    assert torch.isfinite(got[0, 0, [0, 2]]).all()
    ok()


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n_q,G,H", [(2, 3, 2), (16, 1, 1), (3, 7, 1), (100, 2, 1)])
@pytest.mark.parametrize("cap", [300, 6000])
def test_attn_tokens_that_a_query_does_not_see_cost_it_nothing(dtype, dt, n_q, G, H, cap):
    """The last tokens' values are larger and larger: a query sees its own and those before it, and is as exact as they
    alone make it (the bound counts the values that it sees)."""
    L, S, n = 1, 3, 290
    c = make(L, S, H, cap, 16, dtype)
    k, v = rnd(64, L, S, H, n, 128), rnd(65, L, S, H, n, 128)
    top = 12.0 if dtype == "int4" else 110.0                     # 2^top at the last token
    grow = torch.zeros(n)
    grow[n - n_q:] = torch.linspace(top / n_q, top, n_q)
    append(c, k, v * torch.exp2(grow.round()).cuda()[:, None], [0] * S)
    ok()
    check_attn(c, rnd(66, L, S, n_q, G * H, 128, dtype=dt), [n, n - n_q + 1, n - 17])


@pytest.mark.parametrize("loud", [1.0, 50.0, 200.0])
def test_select_scores_stay_within_their_slack(loud):
    """milo_kv_select's scores are estimates: at least q . k of every key of the block less the codes' half steps."""
    S, cap, bl = 4, 640, 64
    c = make(1, S, 1, cap, bl, "int8")
    k = rnd(67, 1, S, 1, cap, 128) + 3 * rnd(68, 1, S, 1, 1, 128)
    k[..., 7] *= loud
    k[:, 1] = k[:, 1, :, :1]                                      # blocks of equal keys: no room between the bounds
    append(c, k, k, [0] * S)
    q = rnd(69, 1, S, 3, 128)
    q[:, 2, :, 7] = 0.0                                           # the loud channel is not asked for
    _, sc = milo.milo_kv_select(c, q, i32([cap] * S), 2, return_scores=True)
    ok()
    sc, qn, kn = np64(sc), f32np(q), f32np(k)
    scale = sections(c)[0]["scale"]
    for s in range(S):
        got = sc[0, s, 0]
        for b in range(c.n_b):
            best = R.score_floor(qn[0, s], kn[0, s, 0, b * bl:(b + 1) * bl], scale[0, s, 0, b])
            assert got[b] >= best.max() - abs(got[b]) * 2.0 ** -22


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n", [3, 40])
def test_int4_bounds_of_saturated_keys_are_outward(dt, n):
    """Keys past the INT4 limit of one sign: the bounds hold the stored +-65440 between them, in both types alike."""
    c = make(1, 1, 1, 64, 16, "int4")
    x = rnd(70, 1, 1, 1, n, 128, scale=10.0).to(dt)
    x[..., 0::4], x[..., 1::4] = 70656.0, -70656.0               # both types hold them
    x[..., 1, 0], x[..., 2, 1] = 65536.0, -65536.0
    append(c, x, x, [0])
    ok(milo.MILO_ERR_NONFINITE)
    z = f32np(x).clip(-65440, 65440)
    got, _ = sections(c)
    q, p = R.quantise(z, "int4")
    for name in ("k", "v"):
        np.testing.assert_array_equal(got[name][:, :, :, :n], q)
        np.testing.assert_array_equal(got[name + "p"][:, :, :, :n], p)
    for b in range(-(-n // 16)):
        t = z[0, 0, 0, 16 * b:16 * (b + 1)]
        lo, hi = R.outward(t.min(0), False), R.outward(t.max(0), True)
        assert lo[0] == 65280.0 and hi[0] == 65536.0 and lo[1] == -65536.0 and hi[1] == -65280.0
        np.testing.assert_array_equal(got["bounds"][0, 0, 0, b], np.stack([lo, hi]))
        codes, scale = R.bound_codes(lo, hi)
        np.testing.assert_array_equal(got["codes"][0, 0, 0, b], codes)
        assert got["scale"][0, 0, 0, b] == scale


@pytest.mark.parametrize("dt", [BF, F32])
def test_int4_values_past_the_limit_are_stored_as_the_limit(dt):
    c = make(1, 1, 1, 16, 16, "int4")
    x = rnd(71, 1, 1, 1, 8, 128, dtype=dt)
    x[..., 0, 0], x[..., 0, 1], x[..., 1, 0], x[..., 2, 40] = 1e38, -1e38, 65504.0, 65441.0   # bf16: 65536
    append(c, x, x, [0])
    ok(milo.MILO_ERR_NONFINITE)
    q, p = R.quantise(f32np(x).clip(-65440, 65440), "int4")
    got, _ = sections(c)
    np.testing.assert_array_equal(got["k"][:, :, :, :8], q)
    np.testing.assert_array_equal(got["kp"][:, :, :, :8], p)


def test_results_on_another_stream_are_not_the_current_streams_memory():
    """What a call makes for `stream` does not take memory that the current stream let go and may still be using."""
    w = synth.WORKLOADS["toy"]
    K, V = (t.cuda() for t in synth.workload_cache(w))
    f = milo.milo_compress(K, V, w.block_len, milo.default_params(factor_dtype="f32"))
    c = filled(1, 2, 1, 300, 16, "int8", [300, 40])
    q, length, zero = rnd(72, 1, 2, 4, 128), i32([300, 40]), i32([0, 0])
    sel, tail = i32([[0, 3], [5, 1]]), rnd(73, 1, 2, 1, 30, 128)
    side = torch.cuda.Stream()
    calls = {
        "rope": lambda s: milo.milo_rope(q.view(1, 8, 128), i32([5]), milo.rope_params(128), stream=s),
        "read": lambda s: milo.milo_kv_read(c, zero, 40, stream=s),
        "select": lambda s: milo.milo_kv_select(c, q, length, 3, return_scores=True, stream=s),
        "attn": lambda s: milo.milo_kv_attn(c, q, length, return_lse=True, stream=s),
        "decode": lambda s: milo.milo_decode_attn(f, q, sel, stream=s),
        "tail": lambda s: milo.milo_decode_attn_tail(f, q, sel, tail, tail, i32([30, 7]), stream=s),
        "decode_kv": lambda s: milo.milo_decode_attn_kv(f, q, sel, c, length, stream=s),
    }
    for name, call in calls.items():
        want = call(None)
        torch.cuda.synchronize()
        one = isinstance(want, torch.Tensor)
        # memory of these sizes that the current stream has just let go
        torch.cuda.empty_cache()
        free = [torch.empty(x.shape, dtype=x.dtype, device="cuda") for x in ([want] if one else want) for _ in range(8)]
        held = {x.data_ptr() for x in free}
        del free
        got = call(side)
        side.synchronize()
        for x, y in zip([got] if one else got, [want] if one else want):
            assert x.data_ptr() not in held, name
            assert torch.equal(x, y), name
    ok()


def expect_blocks(got, kn, bl, s, start, n, old=None):
    """Bounds, codes and scales of session s after rows kn [L][H][n][128] went to `start`: blocks that begin inside the
    range hold these rows alone, the one that goes on holds what it held (`old`) as well."""
    for b in range(start // bl, -(-(start + n) // bl)):
        t0, t1 = max(b * bl, start) - start, min((b + 1) * bl, start + n) - start
        lo, hi = kn[:, :, t0:t1].min(2), kn[:, :, t0:t1].max(2)
        if start > b * bl:
            lo, hi = np.minimum(lo, old["bounds"][:, s, :, b, 0]), np.maximum(hi, old["bounds"][:, s, :, b, 1])
        lo, hi = R.outward(lo, False), R.outward(hi, True)
        np.testing.assert_array_equal(got["bounds"][:, s, :, b], np.stack([lo, hi], -2))
        q, p = R.bound_codes(lo, hi)
        np.testing.assert_array_equal(got["codes"][:, s, :, b], q)
        np.testing.assert_array_equal(got["scale"][:, s, :, b], p)


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n", [2, 5, 37])
def test_append_goes_on_with_a_block_and_writes_rows_again(dtype, dt, n):
    """Chunks whose seam lies inside a block, then rows written a second time: the block's bounds widen, never narrow."""
    L, S, H, cap, bl = 2, 2, 2, 160, 32
    c = make(L, S, H, cap, bl, dtype)
    first = rnd(74, L, S, H, 45, 128, dtype=dt, scale=2.0)
    append(c, first, first, [0, 0], [45, 21])
    at = [45, 21]
    for step, scale in ((0, 3.0), (1, 0.1), (2, 5.0)):            # the last two write the same rows again
        old, _ = sections(c)
        x, y = rnd(75 + step, L, S, H, n, 128, dtype=dt, scale=scale), rnd(78 + step, L, S, H, n, 128, dtype=dt)
        append(c, x, y, at)
        ok()
        got, _ = sections(c)
        for s in range(S):
            rows = slice(at[s], at[s] + n)
            for name, t in (("k", x), ("v", y)):
                q, p = R.quantise(f32np(t[:, s]), dtype)
                np.testing.assert_array_equal(got[name][:, s, :, rows], q)
                np.testing.assert_array_equal(got[name + "p"][:, s, :, rows], p)
            expect_blocks(got, f32np(x[:, s]), bl, s, at[s], n, old)


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("dt", [BF, F32])
def test_append_with_more_items_than_the_gpu_holds(dtype, dt):
    """A warp walks many rows of an item where the items fill the GPU twice over."""
    L, S, H, bl, n, cap = 2, 80, 4, 16, 45, 80
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert ((n - 2 + bl) // bl + 1) * L * S * H * 2 >= 32 * sms
    c = make(L, S, H, cap, bl, dtype)
    k, v = rnd(81, L, S, H, n, 128, dtype=dt, scale=3.0), rnd(82, L, S, H, n, 128, dtype=dt)
    old, _ = sections(c)
    old["bounds"][:] = 0.0
    c.buf.zero_()                                                 # blocks that go on hold zeros
    start, count = [(7 * s) % 36 for s in range(S)], [(11 * s) % 46 for s in range(S)]
    append(c, k, v, start, count)
    ok()
    got, _ = sections(c)
    kn, vn = f32np(k), f32np(v)
    for s in range(S):
        m, rows = count[s], slice(start[s], start[s] + count[s])
        for name, x in (("k", kn), ("v", vn)):
            q, p = R.quantise(x[:, s, :, :m], dtype)
            np.testing.assert_array_equal(got[name][:, s, :, rows], q)
            np.testing.assert_array_equal(got[name + "p"][:, s, :, rows], p)
            assert not got[name][:, s, :, :start[s]].any() and not got[name + "p"][:, s, :, start[s] + m:].any()
        if m:
            expect_blocks(got, kn[:, s, :, :m], bl, s, start[s], m, old)


def test_entry_points_on_another_stream_give_the_same():
    """Those that the test above leaves out: compression, allocation, offloaded decode, text retrieval, cache writes."""
    w = synth.WORKLOADS["toy"]
    K, V = (t.cuda() for t in synth.workload_cache(w))
    p = milo.default_params(factor_dtype="f32")
    sigma = torch.sort(rnd(83, 8, 128).abs(), descending=True).values.contiguous()
    eps = torch.full((1,), 0.5, dtype=torch.float64, device="cuda")
    q, sel, tail = rnd(84, 1, 2, 4, 128), i32([[0, 3], [5, 1]]), rnd(85, 1, 2, 1, 30, 128)
    length, start, count = i32([30, 7]), i32([0, 9]), i32([40, 3])
    host = milo.factors_to_host(milo.milo_compress(K, V, w.block_len, p))
    tables, kv = synth.bm25_tables(w), rnd(86, 1, 2, 1, 40, 128)
    caches = {}

    def append(s):
        milo.milo_kv_append(caches[s], kv, kv, start, count, stream=s)
        return caches[s].buf
    calls = {
        "compress": lambda s: milo.milo_compress(K, V, w.block_len, p, stream=s),
        "allocate": lambda s: milo.milo_allocate(sigma, eps, 1, 8, 2048, 256, 100, stream=s),
        "allocate_noalloc": lambda s: milo.milo_allocate_noalloc(sigma, eps, 1, 8, 2048, 256, 100, stream=s),
        "offload": lambda s: milo.milo_decode_attn_offload(host, q, sel, stream=s),
        "offload_tail": lambda s: milo.milo_decode_attn_offload_tail(host, q, sel, tail, tail, length, stream=s),
        "bm25": lambda s: milo.milo_bm25_select(tables, 8192, 3, stream=s),
        "append": append,
    }
    side = torch.cuda.Stream()
    for s in (None, side):
        caches[s] = make(1, 2, 1, 64, 16, "int4")
    torch.cuda.synchronize()                                      # every input is ready on both streams
    for name, call in calls.items():
        want = call(None)
        torch.cuda.synchronize()
        got = call(side)
        side.synchronize()
        if name == "compress":                                    # the arena's gaps are not written: what it decodes to
            want, got = (milo.milo_decode_attn(x, q, sel) for x in (want, got))
        for x, y in zip(*((a,) if isinstance(a, torch.Tensor) else a for a in (got, want))):
            assert torch.equal(x, y), name
    ok()

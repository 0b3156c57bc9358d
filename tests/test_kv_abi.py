"""Argument checks of the rotary positions and of the quantised cache of recent
tokens, made on the host before anything is launched, and the host-side
formulas (no GPU needed)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from block_wise_rank_b200 import build as milo_build
from block_wise_rank_b200 import milo
from tests import kv_reference as R

INV, UNS, WSP = milo.MILO_ERR_INVALID_ARG, milo.MILO_ERR_UNSUPPORTED, milo.MILO_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    milo_build.build()
    return milo.lib()


def P(x=1 << 20):
    return ctypes.c_void_p(x)


SCALINGS = [("none", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=2.5)),
            ("yarn", dict(factor=4.0, orig_ctx=8192)), ("yarn", dict(factor=32.0, orig_ctx=64, beta_fast=2)),
            ("bands", dict(factor=8.0, orig_ctx=8192)), ("bands", dict(factor=8.0, orig_ctx=10))]


@pytest.mark.parametrize("scaling,kw", SCALINGS)
@pytest.mark.parametrize("d,rd,base", [(128, 0, 1e6), (96, 40, 1e4), (512, 512, 5e5), (4, 4, 10.0)])
def test_rope_freqs(L, scaling, kw, d, rd, base):
    p = milo.rope_params(d, base, rotary_dim=rd, scaling=scaling, **kw)
    w, m = milo.milo_rope_freqs(p)
    ref = R.rope_freqs(rd or d, base, scaling, **kw).astype(np.float64)
    # a power and a few products in 64 bits; the exponent's rounding grows with ln(base) * factor
    np.testing.assert_allclose(w, ref, rtol=2.0 ** -53 * 64)
    assert m == pytest.approx(0.1 * math.log(kw["factor"]) + 1 if scaling == "yarn" else 1.0, rel=1e-15)
    assert milo.milo_rope_freqs(milo.rope_params(d, base, rotary_dim=rd, scaling=scaling, attn_factor=0.7, **kw))[1] == 0.7


@pytest.mark.parametrize("kw,status", [
    (dict(d=0), INV), (dict(d=127), INV), (dict(d=514), UNS), (dict(rotary_dim=3), INV), (dict(rotary_dim=130), INV),
    (dict(rotary_dim=-2), INV), (dict(base=1.0), INV), (dict(base=math.nan), INV), (dict(base=math.inf), INV),
    (dict(scaling=5), INV), (dict(scaling=-1), INV), (dict(scaling=1, factor=0.0), INV),
    (dict(scaling=1, factor=math.inf), INV), (dict(scaling=2, factor=2.0, rotary_dim=2), INV),
    (dict(scaling=3, factor=2.0, orig_ctx=0.0), INV), (dict(scaling=3, factor=2.0, orig_ctx=10, beta_slow=0.0), INV),
    (dict(scaling=3, factor=2.0, orig_ctx=10, beta_slow=40.0), INV),
    (dict(scaling=4, factor=2.0, orig_ctx=10, low_freq=4.0), INV), (dict(attn_factor=-1.0), INV),
    (dict(attn_factor=math.nan), INV)])
def test_rope_refuses_parameters(L, kw, status):
    p = milo.milo_rope_params()
    L.milo_rope_default_params(ctypes.byref(p), kw.pop("d", 128), kw.pop("base", 1e4))
    for k, v in kw.items():
        setattr(p, k, v)
    assert L.milo_rope_freqs(ctypes.byref(p), None, None) == status
    assert L.milo_rope(ctypes.byref(p), P(), 0, 128, 128, P(1 << 30), 0, 128, 128, P(), 1, 4, 1, 0, None) == status


def _rope(L, x=P(), xd=0, xt=512, xh=128, y=P(1 << 30), yd=0, yt=512, yh=128, pos=P(), n_pos=1, nt=4, nh=4):
    p = milo.rope_params(128)
    return L.milo_rope(ctypes.byref(p), x, xd, xt, xh, y, yd, yt, yh, pos, n_pos, nt, nh, 0, None)


def test_rope_refuses_arguments(L):
    assert L.milo_rope(None, P(), 0, 1, 1, P(), 0, 1, 1, P(), 1, 1, 1, 0, None) == INV
    assert _rope(L, x=None) == INV and _rope(L, y=None) == INV and _rope(L, pos=None) == INV
    assert _rope(L, xd=milo.MILO_INT8) == UNS and _rope(L, yd=milo.MILO_FP8) == UNS
    assert _rope(L, nt=-1) == INV and _rope(L, nh=-1) == INV and _rope(L, n_pos=0) == INV
    assert _rope(L, x=P(2)) == INV and _rope(L, pos=P(2)) == INV
    assert _rope(L, xt=-1) == INV and _rope(L, xt=1 << 62) == INV
    assert _rope(L, yh=127) == INV                       # rows of y overlap
    assert _rope(L, yt=511) == INV and _rope(L, yt=0) == INV
    assert _rope(L, y=P((1 << 20) + 4)) == INV           # y overlaps x without being it
    assert _rope(L, y=P(), yt=1024) == INV               # in place with other strides
    assert _rope(L, y=P(), yd=1) == INV                  # in place in another type
    assert _rope(L, nt=0) == milo.MILO_OK and _rope(L, nh=0, x=None) == milo.MILO_OK


SH = dict(L=2, S=3, H=4, cap=100, block_len=32, dtype="int8")


@pytest.mark.parametrize("kw", [dict(L=0), dict(S=0), dict(H=-1), dict(cap=0), dict(cap=(1 << 26) + 1), dict(d=64),
                                dict(block_len=0), dict(block_len=24), dict(block_len=1040), dict(block_len=-16),
                                dict(dtype=milo.MILO_BF16), dict(dtype=milo.MILO_INT2), dict(dtype=77),
                                dict(L=1 << 12, S=1 << 12, H=1 << 12),
                                dict(L=1 << 10, S=1 << 10, H=1 << 10, cap=1 << 26)])
def test_kv_shape_refused(L, kw):
    s = milo.kv_shape(**{**SH, **kw})
    assert milo.milo_kv_cache_size(s) == 0
    o = (ctypes.c_size_t * 7)()
    want = UNS if "d" in kw else INV
    assert L.milo_kv_layout(ctypes.byref(s), o) == want
    b = ctypes.byref(s)
    assert L.milo_kv_append(b, P(), 1 << 50, P(), P(), 0, None, 1, P(), None, None) == want
    assert L.milo_kv_read(b, P(), 1 << 50, 1, P(), None, P(), P(), 0, None) == want
    assert L.milo_kv_select(b, P(), 1 << 50, P(), 0, 1, 8, P(), 1, 0, 1, P(), None, P(), 1 << 50, None) == want
    assert L.milo_kv_attn(b, P(), 1 << 50, P(), 0, 1, 8, P(), None, 0, 0.0, P(), None, P(), 1 << 50, None) == want
    assert L.milo_kv_select_workspace_size(b, 1) == 0 and L.milo_kv_attn_workspace_size(b, 1, 8, 0) == 0
    with pytest.raises(milo.MiloError):
        milo.KvCache(s, device="cpu")


@pytest.mark.parametrize("dtype,row,par", [("int8", 128, 4), ("fp8", 128, 4), ("int4", 64, 16)])
@pytest.mark.parametrize("L_,S,H,cap,bl", [(2, 3, 4, 100, 32), (1, 1, 1, 1, 16), (28, 8, 4, 4097, 64)])
def test_kv_layout(L, dtype, row, par, L_, S, H, cap, bl):
    s = milo.kv_shape(L_, S, H, cap, bl, dtype)
    n, b = S * H * cap, S * H * -(-cap // bl)
    at, want = 0, []
    for size in (n * row, n * row, n * par, n * par, b * 512, b * 256, b * 4):
        want.append(at)
        at = (at + size + 255) // 256 * 256
    assert milo.milo_kv_layout(s) == want and milo.milo_kv_cache_size(s) == L_ * at


def test_kv_cache_object(L):
    c = milo.KvCache(milo.kv_shape(**SH), device="cpu")
    assert c.n_b == 4 and c.layer(1).buf.data_ptr() - c.buf.data_ptr() == milo.milo_kv_cache_size(c.shape) // 2
    assert milo.milo_kv_cache_size(c.layer(1).shape) == milo.milo_kv_cache_size(c.shape) // 2
    with pytest.raises(IndexError):
        c.layer(2)
    with pytest.raises(ValueError):
        milo.KvCache(c.shape, torch.zeros(10, dtype=torch.int32))


def test_kv_append_and_read_refuse(L):
    s = milo.kv_shape(**SH)
    n = milo.milo_kv_cache_size(s)

    def app(cache=P(), nb=n, k=P(), v=P(), dt=0, st=None, n_new=5, start=P(), count=None):
        st = None if st is None else (ctypes.c_int64 * 4)(*st)
        return L.milo_kv_append(ctypes.byref(s), cache, nb, k, v, dt, st, n_new, start, count, None)

    def read(cache=P(), nb=n, m=5, start=P(), count=None, k=P(), v=P(), dt=0):
        return L.milo_kv_read(ctypes.byref(s), cache, nb, m, start, count, k, v, dt, None)
    assert L.milo_kv_append(None, P(), n, P(), P(), 0, None, 1, P(), None, None) == INV
    assert app(cache=None) == INV and app(cache=P(128)) == INV and app(nb=n - 1) == WSP
    assert app(k=None) == INV and app(v=None) == INV and app(start=None) == INV
    assert app(k=P(8)) == INV and app(v=P(8)) == INV and app(start=P(2)) == INV and app(count=P(2)) == INV
    assert app(dt=milo.MILO_INT8) == UNS and app(n_new=-1) == INV and app(n_new=101) == INV
    assert app(st=(-8, 0, 0, 0)) == INV and app(st=(8, 8, 8, 4)) == INV
    assert app(n_new=0, k=None) == milo.MILO_OK
    assert read(cache=None) == INV and read(nb=n - 1) == WSP and read(start=None) == INV
    assert read(k=None, v=None) == INV and read(k=P(8)) == INV and read(v=P(8)) == INV
    assert read(dt=milo.MILO_INT4) == UNS and read(m=-1) == INV and read(m=101) == INV
    assert read(m=0, k=None, v=None) == milo.MILO_OK


def test_kv_select_and_attn_refuse(L):
    s = milo.kv_shape(**SH)
    n, W = milo.milo_kv_cache_size(s), 1 << 40

    def sel(nb=n, q=P(), dt=0, n_q=2, Hq=8, ln=P(), n_sel=2, nf=0, nl=1, out=P(), sc=None, ws=P(), wb=W):
        return L.milo_kv_select(ctypes.byref(s), P(), nb, q, dt, n_q, Hq, ln, n_sel, nf, nl, out, sc, ws, wb, None)

    def att(nb=n, q=P(), dt=0, n_q=2, Hq=8, ln=P(), se=None, n_sel=0, scale=0.0, out=P(), lse=None, ws=P(), wb=W):
        return L.milo_kv_attn(ctypes.byref(s), P(), nb, q, dt, n_q, Hq, ln, se, n_sel, scale, out, lse, ws, wb, None)
    for f in (sel, att):
        assert f(nb=n - 1) == WSP and f(q=None) == INV and f(q=P(8)) == INV and f(ln=None) == INV
        assert f(dt=milo.MILO_INT8) == UNS and f(n_q=0) == INV and f(Hq=6) == INV and f(Hq=0) == INV
        assert f(out=None) == INV and f(ws=None) == INV and f(ws=P(128)) == INV
        assert f(n_q=1 << 28) == UNS
    assert sel(n_sel=0) == INV and sel(n_sel=5) == INV and sel(nf=-1) == INV and sel(nl=-1) == INV
    assert sel(nf=2, nl=1) == INV and sel(sc=P(2)) == INV
    assert sel(wb=L.milo_kv_select_workspace_size(ctypes.byref(s), 2) - 1) == WSP
    assert att(out=P(8)) == INV and att(lse=P(2)) == INV and att(scale=-1.0) == INV and att(scale=math.nan) == INV
    assert att(scale=math.inf) == INV and att(n_sel=1) == INV and att(se=P()) == INV and att(se=P(2), n_sel=1) == INV
    assert att(wb=L.milo_kv_attn_workspace_size(ctypes.byref(s), 2, 8, 0) - 1) == WSP
    assert L.milo_kv_attn_workspace_size(ctypes.byref(s), 2, 7, 0) == 0
    assert L.milo_kv_attn_workspace_size(ctypes.byref(s), 0, 8, 0) == 0


def test_binding_refuses_tensors(L):
    c = milo.KvCache(milo.kv_shape(**SH), device="cpu")
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt)  # noqa: E731
    i = z(3, dt=torch.int32)
    p = milo.rope_params(128)
    with pytest.raises(ValueError):
        milo.milo_rope(z(4, 128), z(4, dt=torch.int32), p)
    with pytest.raises(ValueError):
        milo.milo_rope(z(4, 2, 64), z(4, dt=torch.int32), p)
    with pytest.raises(ValueError):
        milo.milo_rope(z(4, 2, 128), z(4, dt=torch.int32), p)        # not on a GPU
    with pytest.raises(ValueError):
        milo.milo_kv_append(c, z(2, 3, 4, 5, 128), z(2, 3, 4, 6, 128), i)
    with pytest.raises(ValueError):
        milo.milo_kv_append(c, z(2, 3, 4, 5, 128).transpose(3, 4), z(2, 3, 4, 5, 128), i)
    with pytest.raises(ValueError):
        milo.milo_kv_attn(c, z(2, 3, 8, 64), i)
    with pytest.raises(ValueError):
        milo.milo_kv_select(c, z(2, 3, 8, 128), z(4, dt=torch.int32), 1)


def test_binding_refuses_an_empty_selection(L):
    c = milo.KvCache(milo.kv_shape(**SH), device="cpu")
    q, i, none = torch.zeros(2, 3, 8, 128), torch.zeros(3, dtype=torch.int32), torch.zeros(2, 3, 4, 0, dtype=torch.int32)
    with pytest.raises(ValueError, match="at least one block"):
        milo.milo_kv_attn(c, q, i, none)
    with pytest.raises(ValueError, match="at least one block"):
        milo.milo_decode_attn_kv(None, q, none, c, i, none)


# ------------------------------------------------ the reference's own pins
def test_reference_codes():
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(200, 128, generator=g) * torch.exp(3 * torch.randn(200, 1, generator=g))).numpy()
    np.testing.assert_array_equal(R.e4m3(x[:, :64]), torch.from_numpy(x[:, :64]).clamp(-448, 448)
                                  .to(torch.float8_e4m3fn).double().numpy())
    for dt, step in (("int8", 1 / 254), ("int4", None), ("fp8", 2.0 ** -4)):
        c, p = R.quantise(x, dt)
        v = R.values(c, p, dt)
        if dt == "int4":       # half a step of the group's range, and the fp16 rounding of zero, scale and value
            r = x.reshape(200, 4, 32)
            lim = (r.max(-1) - r.min(-1)) / 30 * (1 + 2.0 ** -9) + np.abs(r).max(-1) * 2.0 ** -9
            assert np.all(np.abs(v - x).reshape(200, 4, 32) <= lim[..., None])
        else:
            assert np.all(np.abs(v - x) <= np.abs(x).max(-1, keepdims=True) * step * (1 + 2.0 ** -20))
    for up in (True, False):
        b = R.outward(x, up)
        assert np.all((b >= x) if up else (b <= x)) and np.all((b.view(np.int32) & 0xffff) == 0)


def test_reference_bound_is_an_upper_bound():
    g = np.random.default_rng(0)
    k = g.standard_normal((64, 128)).astype(np.float32)
    lo, hi = R.outward(k.min(0), False), R.outward(k.max(0), True)
    c, s = R.bound_codes(lo[None], hi[None])
    q = g.standard_normal((3, 128)).astype(np.float32)
    best = R.scores(q, c, s)[0]
    # the codes' rounding: half a step of q and of the bound on each of 128 products
    slack = 128 * (np.abs(q).max() / 254 * np.abs(k).max() + np.abs(q).max() * s[0] / 2) * 1.1
    assert best >= (q @ k.T).max() - slack and best >= (q @ k.T).max()


def test_reference_attention_bound_covers_fp32():
    g = np.random.default_rng(0)
    q, k, v = (g.standard_normal((n, 128)).astype(np.float32) for n in (4, 300, 300))
    o, lse, err, le = R.attn(q.astype(float), k.astype(float), v.astype(float), 128 ** -0.5)
    t = torch.from_numpy(q) @ torch.from_numpy(k).T * np.float32(128 ** -0.5)
    assert np.all(np.abs((torch.softmax(t, -1) @ torch.from_numpy(v)).numpy() - o) <= err) and err.max() < 1e-3
    assert np.all(np.abs(torch.logsumexp(t, -1).numpy() - lse) <= le)


def test_reference_score_is_an_estimate_within_its_slack():
    """The coded score may lie below the greatest q . k of a block, by the codes' half steps at most."""
    below = 0
    for seed in range(60):
        g = np.random.default_rng(seed)
        k = (g.standard_normal((64, 128)) + 3 * g.standard_normal(128)).astype(np.float32)
        if seed % 3 == 1:
            k /= 16
            k[:, 5] = 200.0                           # one loud channel, which q does not ask for
        if seed % 3 == 2:
            k[:] = k[0]                                          # equal keys: no room between the bounds
        q = g.standard_normal((3, 128)).astype(np.float32)
        if seed % 3 == 1:
            q[:, 5] = 0.0
        lo, hi = R.outward(k.min(0), False), R.outward(k.max(0), True)
        c, s = R.bound_codes(lo[None], hi[None])
        got = float(R.scores(q, c, s)[0])
        assert got >= R.score_floor(q, k, s[0]).max() - abs(got) * 2.0 ** -22
        below += got < float((q @ k.T).max())
    assert below > 0                                             # so it is no upper bound


def test_rope_yarn_factor_below_one(L):
    """The attention factor grows with the logarithm of a longer context; a shorter one leaves it at 1."""
    for factor, want in ((4.0, 0.1 * math.log(4.0) + 1), (1.0, 1.0), (0.5, 1.0), (1e-5, 1.0)):
        p = milo.rope_params(64, 1e4, scaling="yarn", factor=factor, orig_ctx=4096)
        assert milo.milo_rope_freqs(p)[1] == pytest.approx(want, rel=1e-15)
        p.attn_factor = 0.25
        assert milo.milo_rope_freqs(p)[1] == 0.25


def test_workspace_sizes_of_refused_calls_are_zero(L):
    s = milo.kv_shape(**SH)
    b = ctypes.byref(s)
    sel, att = L.milo_kv_select_workspace_size, L.milo_kv_attn_workspace_size
    assert sel(b, 2) > 0 and att(b, 2, 8, 0) > 0 and att(b, 2, 8, 4) > 0
    most = (2 ** 31 - 1) // (2 * 3 * 4)                          # L S H n_q within 31 bits
    assert sel(b, most) > 0 and sel(b, most + 1) == 0 and sel(b, 2 ** 31 - 1) == 0
    assert att(b, most, 4, 0) > 0 and att(b, most + 1, 4, 0) == 0 and att(b, 1 << 28, 8, 0) == 0
    assert att(b, 2, 2 ** 31 - 4, 0) == 0 and att(b, 2, 8, 2 ** 31 - 1) == 0 and att(b, 2, 8, -1) == 0
    assert att(b, 2, 8, 2 ** 30 // 32) > 0 and att(b, 2, 8, 2 ** 30 // 32 + 1) == 0


def test_counts_whose_product_passes_64_bits_are_refused(L):
    """2^60 query rows in each of 16 sessions: their number is 0 in 64 bits."""
    s = milo.kv_shape(1, 16, 1, 64, 16, "int8")
    b, n, W = ctypes.byref(s), milo.milo_kv_cache_size(milo.kv_shape(1, 16, 1, 64, 16, "int8")), 1 << 62
    big = 1 << 30
    assert 16 * big * big == 2 ** 64
    assert L.milo_kv_select(b, P(), n, P(), 0, big, big, P(), 1, 0, 1, P(), None, P(), W, None) == UNS
    assert L.milo_kv_attn(b, P(), n, P(), 0, big, big, P(), None, 0, 0.0, P(), None, P(), W, None) == UNS
    assert L.milo_kv_attn_workspace_size(b, big, big, 0) == 0

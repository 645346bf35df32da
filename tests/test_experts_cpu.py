"""The routed-FFN entry points on the host: refusals before any device call, the
binding's checks, and the oracle's own pins (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import experts_oracle as O

P = pytest.importorskip("free_ffn_activation_amd.prox",
                        reason="libprox.so not built (run __graft_entry__.build())")

FAKE = 1 << 40  # 256-aligned, never dereferenced by validation
BAD, UNSUP = P.PROX_ERR_INVALID_ARG, P.PROX_ERR_UNSUPPORTED


def _experts(**kw):
    e = P.prox_experts(4, 64, 128, P.PROX_BF16, 0, 0, 128, 64 * 128, FAKE, None, None, None)
    for k, v in kw.items():
        setattr(e, k, v)
    return e


def _mm(e, a=FAKE, a_rows=8, a_stride=128, a_scale=None, idx=None, off=FAKE, rows=8, out=FAKE, odt=P.PROX_BF16, ostr=64):
    return P.raw_library().prox_grouped_matmul(ctypes.byref(e) if e is not None else None, a, a_rows, a_stride, a_scale,
                                               idx, off, rows, out, odt, ostr, None)


@pytest.mark.parametrize("kw,status", [
    (dict(wdtype=3), BAD), (dict(wdtype=-1), BAD), (dict(activation=2), BAD), (dict(reserved=1), BAD),
    (dict(n_groups=0), BAD), (dict(n=0), BAD), (dict(k=0), BAD), (dict(n_groups=1025), UNSUP), (dict(k=132), UNSUP),
    (dict(row_stride=132), UNSUP), (dict(group_stride=12), UNSUP), (dict(row_stride=64), BAD),
    (dict(group_stride=-8), BAD), (dict(w=None), BAD), (dict(w=FAKE + 8), BAD), (dict(w_gate=FAKE + 2), BAD),
    (dict(wdtype=P.PROX_FP8), BAD), (dict(wdtype=P.PROX_FP8, w_scale=FAKE + 2), BAD),
    (dict(wdtype=P.PROX_FP8, w_scale=FAKE, w_gate=FAKE), BAD), (dict(n=(1 << 24) + 1), UNSUP)])
def test_product_refuses_descriptors(kw, status):
    assert _mm(_experts(**kw)) == status
    assert P.prox_last_error() != ""


def test_product_refuses_arguments():
    e = _experts()
    assert _mm(None) == BAD
    for kw in (dict(rows=-1), dict(rows=(1 << 30) + 1), dict(a_rows=-1), dict(a_rows=7), dict(a_stride=120), dict(ostr=63),
               dict(odt=P.PROX_FP8), dict(a=None), dict(a=FAKE + 8), dict(out=None), dict(out=FAKE + 1),
               dict(idx=FAKE + 1), dict(off=FAKE + 2), dict(off=None)):
        assert _mm(e, **kw) == BAD, kw
    assert _mm(e, a_stride=132) == UNSUP
    f8 = _experts(wdtype=P.PROX_FP8, w_scale=FAKE)
    assert _mm(f8) == BAD and "a_scale" in P.prox_last_error()
    assert _mm(f8, a_scale=FAKE + 1) == BAD
    # nothing to do: accepted without a device
    assert _mm(e, rows=0, a=None, out=None) == P.PROX_OK


def test_route_refusals():
    lib = P.raw_library()

    def call(logits=FAKE, dt=P.PROX_F32, t=4, e=8, k=2, rn=1, idx=FAKE, w=FAKE, off=FAKE, rt=FAKE, ro=FAKE, ws=FAKE,
             nb=1 << 20):
        return lib.prox_expert_route(logits, dt, t, e, k, rn, idx, w, off, rt, ro, ws, nb, None)
    for kw in (dict(t=-1), dict(e=0), dict(k=0), dict(k=9), dict(dt=P.PROX_FP8), dict(rn=2), dict(logits=None),
               dict(idx=None), dict(w=None), dict(off=None), dict(rt=None), dict(ro=None), dict(ws=None),
               dict(ws=FAKE + 16), dict(off=FAKE + 2), dict(logits=FAKE + 2), dict(nb=0)):
        assert call(**kw) == BAD, kw
    assert call(e=1025) == UNSUP and call(e=64, k=33) == UNSUP and call(t=1 << 30, k=2) == UNSUP
    with pytest.raises(P.ProxError):
        P.prox_expert_route_workspace_size(4, 8, 9)
    assert P.prox_expert_route_workspace_size(0, 8, 2) % 256 == 0


@pytest.mark.parametrize("es,code", [(4, P.PROX_F32), (2, P.PROX_BF16)])
def test_refuses_strides_beyond_64_bits(es, code):
    """Strides whose sizes in bytes would pass 64 bits (2^61 fp32 values wrap to
    a negative stride, which is below every upper limit)."""
    lib = P.raw_library()
    for stride in (1 << 61, 1 << 62, (1 << 63) - 16, (1 << 40) + 16):
        assert _mm(_experts(wdtype=code, row_stride=stride)) == UNSUP
        assert _mm(_experts(wdtype=code, group_stride=stride)) == UNSUP
        assert _mm(_experts(wdtype=code), a_stride=stride) == UNSUP
        assert _mm(_experts(wdtype=code), ostr=stride) == UNSUP
        assert lib.prox_fp8_quantize(FAKE, code, 4, 128, stride, 1, FAKE, 128, FAKE, None) == UNSUP
        assert lib.prox_fp8_quantize(FAKE, code, 4, 128, 128, 1, FAKE, stride, FAKE, None) == UNSUP
        assert lib.prox_expert_combine(FAKE, code, 8, stride, FAKE, FAKE, 4, 2, 64, FAKE, code, 64, None) == UNSUP
        assert lib.prox_expert_combine(FAKE, code, 8, 64, FAKE, FAKE, 4, 2, 64, FAKE, code, stride, None) == UNSUP


def test_combine_refuses_rows_whose_last_index_passes_32_bits():
    n = (1 << 31) - 1
    assert P.raw_library().prox_expert_combine(FAKE, P.PROX_BF16, 8, n, FAKE, FAKE, 1, 1, n, FAKE, P.PROX_BF16, n,
                                               None) == UNSUP


def test_moe_refuses_router_rows_of_8_mib():
    """An fp8 layer's bf16 router has rows twice as wide as its experts'."""
    lib, size = P.raw_library(), ctypes.c_size_t(0)
    f8 = dict(wdtype=P.PROX_FP8, w_scale=FAKE)
    for d, want in (((1 << 22) - 16, P.PROX_OK), (1 << 22, UNSUP)):
        up = _experts(n=16, k=d, row_stride=d, group_stride=16 * d, w_gate=FAKE, w_gate_scale=FAKE, **f8)
        down = _experts(n=d, k=16, row_stride=16, group_stride=16 * d, **f8)
        layer = P.prox_moe_layer(up, down, FAKE, 2, 1, 0)
        assert lib.prox_moe_workspace_size(ctypes.byref(layer), 4, ctypes.byref(size)) == want


def test_quantize_and_combine_refusals():
    lib = P.raw_library()

    def quant(x=FAKE, dt=P.PROX_BF16, rows=4, k=128, xs=128, br=1, q=FAKE, qs=128, sc=FAKE):
        return lib.prox_fp8_quantize(x, dt, rows, k, xs, br, q, qs, sc, None)
    for kw in (dict(dt=P.PROX_FP8), dict(rows=-1), dict(k=0), dict(br=2), dict(xs=112), dict(qs=112), dict(x=None),
               dict(q=None), dict(sc=None), dict(x=FAKE + 8), dict(q=FAKE + 8), dict(sc=FAKE + 1)):
        assert quant(**kw) == BAD, kw
    assert quant(k=120) == UNSUP and quant(xs=132) == UNSUP and quant(qs=136) == UNSUP
    assert quant(rows=0, x=None) == P.PROX_OK

    def comb(h=FAKE, hd=P.PROX_BF16, hr=8, hs=64, ro=FAKE, w=FAKE, t=4, k=2, n=64, y=FAKE, yd=P.PROX_F32, ys=64):
        return lib.prox_expert_combine(h, hd, hr, hs, ro, w, t, k, n, y, yd, ys, None)
    for kw in (dict(hd=P.PROX_FP8), dict(yd=P.PROX_FP8), dict(t=-1), dict(hr=-1), dict(k=0), dict(k=33), dict(n=0),
               dict(hs=63), dict(ys=63), dict(h=None), dict(ro=None), dict(w=None), dict(y=None), dict(h=FAKE + 1),
               dict(y=FAKE + 2), dict(ro=FAKE + 2), dict(w=FAKE + 2)):
        assert comb(**kw) == BAD, kw
    assert comb(t=0, y=None) == P.PROX_OK


def test_moe_refusals():
    lib = P.raw_library()
    up = dict(n=64, k=128, row_stride=128, group_stride=64 * 128, w_gate=FAKE)
    down = dict(n=128, k=64, row_stride=64, group_stride=64 * 128)

    def layer(u=None, d=None, router=FAKE, top_k=2, rn=1, reserved=0):
        return P.prox_moe_layer(_experts(**{**up, **(u or {})}), _experts(**{**down, **(d or {})}), router, top_k, rn,
                                reserved)

    def call(L, x=FAKE, t=4, y=FAKE, ws=FAKE, nb=1 << 40):
        return lib.prox_moe_ffn(ctypes.byref(L) if L is not None else None, x, t, y, ws, nb, None)
    size = ctypes.c_size_t(0)
    good = layer()
    assert lib.prox_moe_workspace_size(ctypes.byref(good), 4, ctypes.byref(size)) == P.PROX_OK and size.value > 0
    assert lib.prox_moe_workspace_size(ctypes.byref(good), 4, None) == BAD
    assert call(good, t=0, x=None) == P.PROX_OK
    assert call(good, nb=size.value - 1) == BAD
    for kw in (dict(x=None), dict(y=None), dict(ws=None), dict(ws=FAKE + 16), dict(x=FAKE + 8), dict(t=-1)):
        assert call(good, **kw) == BAD, kw
    for L in (None, layer(u=dict(w_gate=None)), layer(d=dict(w_gate=FAKE)), layer(u=dict(n_groups=3)),
              layer(d=dict(k=32)), layer(d=dict(wdtype=P.PROX_F32)), layer(rn=2), layer(reserved=1),
              layer(router=None), layer(router=FAKE + 4), layer(top_k=0), layer(top_k=5)):
        assert call(L) == BAD


def test_binding_refuses_tensors():
    w = torch.zeros(2, 16, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        P.ProxExperts(w[0])
    with pytest.raises(ValueError):
        P.ProxExperts(w, w[:1])
    with pytest.raises(ValueError):
        P.ProxExperts(w, scale=torch.zeros(2, 1, 1))
    with pytest.raises(TypeError):
        P.ProxExperts(w.half())
    with pytest.raises(ValueError):
        P.ProxExperts(w.to(torch.float8_e4m3fn))
    with pytest.raises(ValueError):
        P.ProxExperts(w.transpose(1, 2))
    e = P.ProxExperts(w)
    a, out, off = torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(4, 16), torch.zeros(3, dtype=torch.int32)
    for bad in (dict(a=a[:, :16]), dict(a=a.float()), dict(out=out[:, :8]), dict(offsets=off[:2]),
                dict(offsets=off.long()), dict(row_index=off), dict(a_scale=torch.zeros(4, 1)),
                dict(a=torch.zeros(32, 4, dtype=torch.bfloat16).T), dict(out=out[:1].expand(4, 16))):
        with pytest.raises(ValueError):
            P.prox_grouped_matmul(e, **{**dict(a=a, out=out, offsets=off), **bad})
    with pytest.raises(ValueError, match="GPU"):  # host tensors never reach the library
        P.prox_grouped_matmul(e, a, out, offsets=off)
    with pytest.raises(ValueError):
        P.prox_fp8_quantize(a, a, out)
    with pytest.raises(ValueError):
        P.prox_expert_combine(a, off.reshape(1, 3), torch.zeros(1, 2), torch.zeros(1, 32))


# ------------------------------------------------------------ oracle pins
def test_oracle_route_by_hand():
    inf, nan = np.inf, np.nan
    z = np.array([[1.0, 3.0, 3.0, 2.0], [-inf, -inf, 0.5, -inf], [-inf] * 4, [nan, 9.0, inf, 1.0]])
    r = O.route(z, 2)
    assert r["idx"].tolist() == [[1, 2], [2, -1], [-1, -1], [0, 2]]
    assert np.allclose(r["weight"][:3], [[0.5, 0.5], [1, 0], [0, 0]]) and np.isnan(r["weight"][3]).all()
    assert r["offsets"].tolist() == [0, 1, 2, 5, 5]
    assert r["row_token"].tolist() == [3, 0, 0, 1, 3, -1, -1, -1]
    assert r["row_of"].tolist() == [[1, 2], [3, -1], [-1, -1], [0, 4]]
    w = O.route(np.array([[0.0, np.log(3.0)]]), 1, renormalize=False)["weight"]
    assert np.allclose(w, 0.75)


def test_oracle_e4m3_is_torchs():
    """Every e4m3 value and every midpoint, against torch's own conversion."""
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    v = np.unique(v[np.isfinite(v)])
    x = np.concatenate([v, (v[1:] + v[:-1]) / 2])
    assert np.array_equal(O.round_e4m3(x.astype(np.float64)),
                          torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy().astype(np.float64))


def test_oracle_quantize_blocks():
    x = np.zeros((3, 144), np.float32)
    x[0, :128], x[0, 128:], x[2, 130] = 448.0, -7.0, np.inf
    q, s = O.quantize(x, 1)
    assert s[0].tolist() == [1.0, np.float32(7.0) / np.float32(448.0)] and np.isnan(s[2, 1]) and s[1].tolist() == [0, 0]
    assert (q[0, :128] == 448).all() and (q[0, 128:] == -448).all() and (q[1] == 0).all() and np.isnan(q[2, 128:]).all()

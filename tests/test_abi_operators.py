"""Refusals of the MXFP4, few-token and norm entry points: on the host, before
any launch (so these run without a GPU)."""
import ctypes

import pytest

from top_routing_expert_amd import binding as B
from top_routing_expert_amd import configs as C

P = 1 << 40  # 256-byte aligned, never dereferenced
bf = ctypes.byref


def _size():
    return ctypes.c_size_t(0)


def test_mxfp4_rows():
    L = B.lib()
    cfg = B.config(T=4, d=64, E=1, k=1, f=64)
    f32 = B.config(T=4, d=36, E=1, k=1, f=64, dtype=B.MOE_F32)
    assert L.moe_quantize_mxfp4(bf(f32), P, P, P, None) == B.MOE_EUNSUPPORTED  # 36 % 32
    assert L.moe_dequantize_mxfp4(bf(f32), P, None, P, P, None) == B.MOE_EUNSUPPORTED
    assert L.moe_quantize_mxfp4(None, P, P, P, None) == B.MOE_EINVAL
    for args in ((None, P, P), (P, None, P), (P, P, None), (P + 2, P, P), (P, P + 8, P),
                 (P, P, P + 2)):
        assert L.moe_quantize_mxfp4(bf(cfg), *args, None) == B.MOE_EINVAL, args
    for args in ((None, P, P, P), (P, P, None, P), (P, P, P, None), (P + 4, P, P, P),
                 (P, P, P + 2, P), (P, P, P, P + 8)):
        assert L.moe_dequantize_mxfp4(bf(cfg), *args, None) == B.MOE_EINVAL, args
    empty = B.config(T=0, d=64, E=1, k=1, f=64)
    assert L.moe_quantize_mxfp4(bf(empty), None, None, None, None) == B.MOE_OK
    assert L.moe_dequantize_mxfp4(bf(empty), None, None, None, None, None) == B.MOE_OK


def test_mxfp4_products():
    L = B.lib()
    ok = B.config(C.E8_D4096)
    gu, dn = B.mxfp4_weight_bytes(ok)
    e, d, f = C.E8_D4096.E, C.E8_D4096.d, C.E8_D4096.f
    assert gu == e * 2 * f * d * 17 // 32 and dn == e * d * f * 17 // 32
    n = _size()
    for bad in (dict(d=4096 + 64), dict(f=64), dict(dtype=B.MOE_F32)):
        cfg = B.config(C.E8_D4096, **bad)
        assert L.moe_mxfp4_weight_bytes(bf(cfg), bf(n), bf(n)) == B.MOE_EUNSUPPORTED
        assert L.moe_pack_weights_mxfp4(bf(cfg), *[P] * 8, None) == B.MOE_EUNSUPPORTED
        assert L.moe_ffn_gate_up_mxfp4_gather(bf(cfg), *[P] * 6, None) == B.MOE_EUNSUPPORTED
        assert L.moe_ffn_down_mxfp4(bf(cfg), *[P] * 5, None) == B.MOE_EUNSUPPORTED
    assert L.moe_mxfp4_weight_bytes(bf(ok), bf(n), None) == B.MOE_EINVAL
    assert L.moe_pack_weights_mxfp4(bf(ok), *[P] * 6, None, None, None) == B.MOE_EINVAL
    for i in range(8):  # any input missing or misaligned
        for bad in (None, P + 8):
            args = [P] * 8
            args[i] = bad
            if bad is None and i >= 6:
                continue  # an image may be absent
            assert L.moe_pack_weights_mxfp4(bf(ok), *args, None) == B.MOE_EINVAL, (i, bad)
    for i in range(6):
        args = [P] * 6
        args[i] = None
        assert L.moe_ffn_gate_up_mxfp4_gather(bf(ok), *args, None) == B.MOE_EINVAL, i
    for i in range(5):
        args = [P] * 5
        args[i] = None
        assert L.moe_ffn_down_mxfp4(bf(ok), *args, None) == B.MOE_EINVAL, i
    assert L.moe_ffn_down_mxfp4(bf(ok), P, P + 2, P, P, P, None) == B.MOE_EINVAL
    assert L.moe_ffn_down_mxfp4(bf(ok), P, P, P, P, P + 8, None) == B.MOE_EINVAL
    empty = B.config(C.E8_D4096, T=0)
    assert L.moe_ffn_gate_up_mxfp4_gather(bf(empty), *[None] * 6, None) == B.MOE_OK
    assert L.moe_ffn_down_mxfp4(bf(empty), *[None] * 5, None) == B.MOE_OK


def _few(cfg, args, weights=0, bufs=None, ws=P, n=1 << 40):
    x, wr, gu, dn, out = args
    return B.lib().moe_layer_fwd_few(bf(cfg), x, wr, None, gu, dn, weights, out, bufs, ws, n, None)


def test_few():
    ok = B.config(C.E8_D4096, T=7)
    need = B.workspace_bytes(ok, "layer_few")
    assert need >= 7 * 2 * C.E8_D4096.f * 2
    for T in (-1, 33, 1024):
        want = B.MOE_EINVAL if T < 0 else B.MOE_EUNSUPPORTED
        assert _few(B.config(C.E8_D4096, T=T), [P] * 5) == want
        assert B.lib().moe_workspace_bytes(bf(B.config(C.E8_D4096, T=T)), 9, bf(_size())) == want
    assert B.workspace_bytes(B.config(C.E8_D4096, T=32), "layer_few") > need
    assert _few(ok, [P] * 5, weights=2) == B.MOE_EINVAL
    assert _few(ok, [P] * 5, weights=-1) == B.MOE_EINVAL
    assert _few(B.config(C.E8_D4096, T=7, d=4160), [P] * 5, weights=1) == B.MOE_EUNSUPPORTED
    assert _few(B.config(C.TINY_F32, T=7), [P] * 5) == B.MOE_EUNSUPPORTED
    assert _few(B.config(C.E8_D4096, T=7, k=9), [P] * 5) == B.MOE_EINVAL
    for i in range(5):
        for bad in (None, P + 8):
            args = [P] * 5
            args[i] = bad
            assert _few(ok, args) == B.MOE_EINVAL, (i, bad)
    assert _few(ok, [P] * 5, ws=None) == B.MOE_EINVAL
    assert _few(ok, [P] * 5, n=need - 256) == B.MOE_EINVAL
    assert _few(ok, [P] * 5, ws=P + 16) == B.MOE_EINVAL
    for field in ("expert_offsets", "rank_offsets", "slot_of", "src_of", "x_perm", "h", "y_perm"):
        assert _few(ok, [P] * 5, bufs=bf(B.MoELayerBufs(**{field: P}))) == B.MOE_EINVAL, field
    assert _few(B.config(C.E8_D4096, T=0), [None] * 5, ws=None, n=0) == B.MOE_OK
    assert B.workspace_bytes(B.config(C.E8_D4096, T=0), "layer_few") == 0


def test_norm():
    L = B.lib()
    ok = B.config(C.E8_D4096, T=7)
    assert L.moe_norm(bf(ok), None, P, 1e-6, P, P, None) == B.MOE_EINVAL
    assert L.moe_norm(bf(ok), P, P, 1e-6, None, P, None) == B.MOE_EINVAL
    assert L.moe_norm(bf(ok), P, P + 2, 1e-6, P, P, None) == B.MOE_EINVAL
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert L.moe_norm(bf(ok), P, P, eps, P, P, None) == B.MOE_EINVAL, eps
    for d, dt in ((16384 + 64, B.MOE_BF16), (8192 + 4, B.MOE_F32)):
        wide = B.config(T=3, d=d, E=1, k=1, f=64, dtype=dt)
        assert L.moe_norm(bf(wide), P, P, 1e-6, P, P, None) == B.MOE_EUNSUPPORTED
        assert L.moe_combine_norm_backward_bytes(bf(wide), 1, bf(_size())) == B.MOE_EUNSUPPORTED
    need = B.workspace_bytes(ok, "norm_backward")
    assert need >= C.E8_D4096.d * 4
    args = [P] * 7  # d_xn, x, weight, rstd, d_residual, d_x, d_weight
    assert L.moe_norm_backward(bf(ok), *args, P, need - 256, None) == B.MOE_EINVAL
    assert L.moe_norm_backward(bf(ok), *args, None, 0, None) == B.MOE_EINVAL
    for i in (0, 1, 3, 5):
        a = list(args)
        a[i] = None
        assert L.moe_norm_backward(bf(ok), *a, P, need, None) == B.MOE_EINVAL, i
    for i in (0, 1, 2, 4, 5):
        a = list(args)
        a[i] = P + 4
        assert L.moe_norm_backward(bf(ok), *a, P, need, None) == B.MOE_EINVAL, i


def test_combine_norm():
    L = B.lib()
    ok = B.config(C.E8_D4096, T=6)
    fwd = lambda y=P, slot=P, tw=P, res=P, w=P, gate=P, n=2, eps=1e-6, sc=1.0, out=P, c=ok: (  # noqa: E731
        L.moe_combine_norm(bf(c), y, slot, tw, res, w, gate, n, eps, sc, out, P, None))
    for kw in (dict(y=None), dict(out=None), dict(slot=None), dict(tw=None), dict(gate=None),
               dict(n=0), dict(n=4), dict(n=-1), dict(n=12), dict(eps=0.0), dict(sc=float("nan")),
               dict(y=P + 8), dict(res=P + 8), dict(w=P + 8), dict(gate=P + 8), dict(out=P + 8)):
        assert fwd(**kw) == B.MOE_EINVAL, kw
    need = B.combine_norm_backward_bytes(ok, 2)
    assert B.combine_norm_backward_bytes(ok, 6) > need
    with pytest.raises(B.MoEError):
        B.combine_norm_backward_bytes(ok, 4)
    assert L.moe_combine_norm_backward_bytes(bf(ok), 2, None) == B.MOE_EINVAL
    names = ("d_out", "y", "slot", "tw", "w", "gate")
    outs = ("d_y", "d_tw", "d_res", "d_w", "d_gate")

    def bwd(n=2, sc=1.0, rstd=P, ws=P, nws=need, **kw):
        v = {m: kw.get(m, P) for m in names + outs}
        return L.moe_combine_norm_backward(bf(ok), *[v[m] for m in names], n, sc, rstd,
                                           *[v[m] for m in outs], ws, nws, None)

    for kw in (dict(d_out=None), dict(y=None), dict(slot=None), dict(tw=None), dict(rstd=None),
               dict(d_y=None), dict(gate=None), dict(gate=None, n=0), dict(n=5),
               dict(slot=None, tw=None), dict(sc=float("inf")), dict(ws=None),
               dict(nws=need - 256), dict(ws=P + 64), dict(d_out=P + 2), dict(y=P + 2),
               dict(w=P + 2), dict(gate=P + 2), dict(d_y=P + 2), dict(d_res=P + 2)):
        assert bwd(**kw) == B.MOE_EINVAL, kw

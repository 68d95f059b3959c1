"""CPU pins of the oracle of MXFP4 and of the norms around the block: hand cases
of the format, finite differences of the norms' gradients."""
import numpy as np
import pytest

from oracle import block_oracle as bo


def test_mxfp4_hand_block():
    """max 6 -> scale 1: every level, every tie, both signs, saturation."""
    x = np.zeros((1, 32), np.float32)
    vals = [6, -6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0, 7.9, 0.24, 0.26, -0.0, 0.5, 4.99]
    want = [7, 15, 0, 2, 2, 4, 4, 6, 6, 14, 7, 0, 1, 8, 1, 6]
    x[0, :16] = vals
    codes, scales = bo.mxfp4_quantize(x)
    got = np.stack([codes[0] & 15, codes[0] >> 4], -1).ravel()[:16]
    assert scales[0, 0] == 127
    assert got.tolist() == want


@pytest.mark.parametrize("top,byte", [(4.0, 127), (7.99, 127), (8.0, 128), (1.0, 125), (0.0, 0),
                                      (2.0 ** -140, 0), (2.0 ** 127, 252)])
def test_mxfp4_scale_of_the_maximum(top, byte):
    x = np.zeros((1, 32), np.float32)
    x[0, 9] = top
    assert bo.mxfp4_quantize(x)[1][0, 0] == byte


def test_mxfp4_non_finite_blocks():
    x = np.ones((1, 96), np.float32)
    x[0, 3], x[0, 40] = np.nan, -np.inf
    codes, scales = bo.mxfp4_quantize(x)
    assert scales[0].tolist() == [255, 255, 125]
    v = bo.mxfp4_decode(codes, scales)[0]
    assert np.isnan(v[:64]).all() and (v[64:] == 1.0).all()


def test_mxfp4_round_trip_is_the_nearest_level():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((7, 128)) * np.exp2(rng.integers(-20, 20, (7, 1)))).astype(np.float32)
    codes, scales = bo.mxfp4_quantize(x)
    v = bo.mxfp4_decode(codes, scales)
    step = np.repeat(np.exp2(scales.astype(float) - 127), 32, -1)
    grid = np.concatenate([-bo.MX_LEVELS, bo.MX_LEVELS])
    best = np.abs(x[..., None] / step[..., None] - grid).min(-1)
    assert np.array_equal(np.abs(x / step - v / step), best)
    # quantised values are fixed points
    c2, s2 = bo.mxfp4_quantize(v.astype(np.float32))
    assert np.array_equal(bo.mxfp4_decode(c2, s2), v)


def _numeric(f, a, da, h=1e-6):
    return (f(a + h * da) - f(a - h * da)) / (2 * h)


@pytest.mark.parametrize("n_gate,k,given", [(0, 2, True), (1, 3, True), (3, 2, False), (6, 1, True)])
def test_norm_gradients_against_differences(n_gate, k, given):
    rng = np.random.default_rng(n_gate + 10 * k)
    T, d = 6, 12
    y = rng.standard_normal((T * k, d))
    slot = rng.permutation(T * k)
    tw = rng.random((T, k)) + 0.1
    res, up = rng.standard_normal((T, d)), rng.standard_normal((T, d))
    w = rng.standard_normal(d) if given else None
    gate = rng.standard_normal((n_gate, d)) if n_gate else None
    kw = dict(eps=1e-3, scale=0.7)
    out = lambda y=y, tw=tw, res=res, w=w, gate=gate: float(  # noqa: E731
        (up * bo.combine_norm(y, slot, tw, res, w, gate, **kw)[0]).sum())
    g = bo.combine_norm_backward(up, y, slot, tw, w, gate, **kw)
    for name, a, key in (("y", y, "d_y"), ("tw", tw, "d_topk_w"), ("res", res, "d_residual"),
                         ("w", w, "d_weight"), ("gate", gate, "d_gate")):
        if a is None:
            continue
        da = rng.standard_normal(a.shape)
        num = _numeric(lambda v: out(**{name: v}), a, da)
        # central differences of O(1) curvature: h^2 + rounding / h
        assert abs(num - (g[key] * da).sum()) < 1e-7 * max(1.0, abs(num)), name
    x, dr = rng.standard_normal((T, d)), rng.standard_normal((T, d))
    f = lambda x=x, w=w: float((up * bo.rms_norm(x, w, 1e-3)[0]).sum() + (dr * x).sum())  # noqa: E731
    dx, dw = bo.rms_norm_backward(up, x, w, 1e-3, dr)
    da = rng.standard_normal(x.shape)
    assert abs(_numeric(lambda v: f(x=v), x, da) - (dx * da).sum()) < 1e-7 * 10
    if given:
        da = rng.standard_normal(d)
        assert abs(_numeric(lambda v: f(w=v), w, da) - (dw * da).sum()) < 1e-7 * 10

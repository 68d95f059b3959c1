"""MXFP4 on the GPU: quantisation and decoding bit-exact against the oracle, the
packed images, and the expert products against float64.

Tolerance of the products.  Where every scale is 1 the products of two codes are
multiples of 1/4 and their sums stay below 2^24 quarters, so float32 holds
every partial sum and the result must be the exact sum rounded once to bf16.
With free scales a product differs from the float64 sum by the one bf16 rounding
(2^-8 of the value) and by float32 sums of K terms in some order: at most
K 2^-24 sum |a b|, and 2^-11 of the largest |product| for each 64-wide step inside the
matrix instruction, which aligns its products before it adds them."""
import numpy as np
import pytest
import torch

from _gpu import host, log, rel_err
from oracle import block_oracle as bo
from oracle import moe_oracle as om
from top_routing_expert_amd import binding as B

pytestmark = pytest.mark.gpu


def _cfg(T, d, bf=True, **kw):
    base = dict(T=T, d=d, E=1, k=1, f=64, dtype=B.MOE_BF16 if bf else B.MOE_F32)
    return B.config(**{**base, **kw})


def _bits(a):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda().view(torch.bfloat16)


def _quantize(x, T, d, bf=True):
    n = T * d
    codes = torch.full((T, d // 2), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((n // 32 + 64,), 0x33, dtype=torch.uint8, device="cuda")
    B.moe_quantize_mxfp4(_cfg(T, d, bf), x, codes, scales)
    torch.cuda.synchronize()
    assert (scales[n // 32:] == 0x33).all()  # nothing behind the last block
    return host(codes), host(scales)[:n // 32].reshape(T, d // 32)


def _check(bits_or_f32, bf=True):
    T, d = bits_or_f32.shape
    x = _bits(bits_or_f32) if bf else torch.from_numpy(bits_or_f32).cuda()
    codes, scales = _quantize(x, T, d, bf)
    c_ref, s_ref = bo.mxfp4_quantize(bits_or_f32)
    assert np.array_equal(scales, s_ref)
    assert np.array_equal(codes, c_ref)


@pytest.mark.parametrize("T,d,bf", [(1, 64, True), (3, 192, True), (1, 32, False), (7, 96, False),
                                    (33, 7168, True), (300, 2048, True), (129, 4096, False)])
def test_quantize_random_rows(T, d, bf):
    log(f"[mxfp4] quantize T={T} d={d} bf16={bf}")
    rng = np.random.default_rng(T + d)
    x = (rng.standard_normal((T, d)) * np.exp2(rng.integers(-30, 30, (T, 1)))).astype(np.float32)
    x[rng.random((T, d)) < 0.05] = 0.0
    x[:, ::7] *= -1.0
    _check(om.round_bf16(x) if bf else x, bf)


def test_quantize_every_bf16_value():
    """Every finite bf16 value: as the maximum of its block (consecutive patterns
    share an exponent), and below maxima of 2^e 1.5 over the whole range."""
    log("[mxfp4] every bf16 value")
    pos = np.arange(0, 0x7F80, dtype=np.uint16)
    blocks = [pos, pos | 0x8000]
    for top in (0x0000, 0x0001, 0x0040, 0x0080, 0x0140, 0x01C0, 0x3F80, 0x3FC0, 0x4080, 0x7F00,
                0x7F40, 0x7F7F):
        below = np.concatenate([pos[pos <= top], pos[pos <= top] | 0x8000])
        below = np.resize(below, -(-below.size // 31) * 31).reshape(-1, 31)
        blocks.append(np.concatenate([below, np.full((len(below), 1), top, np.uint16)], 1).ravel())
    x = np.concatenate(blocks)
    x = np.concatenate([x, np.zeros(-x.size % 128, np.uint16)]).reshape(-1, 128)
    _check(x)


def test_quantize_float32_borders():
    """Values a float32 step beside every rounding border, for several scales."""
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 4.0], np.float32)
    near = np.concatenate([mids, np.nextafter(mids, np.float32(0)), np.nextafter(mids, np.float32(9))])
    near[near >= 8] = 7.5
    row = np.concatenate([near, -near, np.array([4.0, -6.5, 0.0, -0.0], np.float32)])
    row = row[:64]
    x = np.stack([np.resize(np.roll(row, s), 64) * np.float32(2.0 ** e)
                  for e in (-126, -120, -60, -1, 0, 1, 50, 124) for s in range(0, 64, 3)])
    _check(x.astype(np.float32), False)


def test_non_finite_blocks_decode_to_nan():
    x = np.full((2, 128), om.round_bf16(np.float32([1.5]))[0], np.uint16)
    x[0, 5], x[0, 40], x[1, 127] = 0x7FC0, 0x7F80, 0xFF80
    _check(x)
    codes, scales = _quantize(_bits(x), 2, 128)
    out = torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda")
    B.moe_dequantize_mxfp4(_cfg(2, 128), torch.from_numpy(codes).cuda(), None,
                           torch.from_numpy(scales).cuda(), out)
    nan = torch.isnan(out).cpu().numpy()
    want = np.isnan(bo.mxfp4_decode(codes, scales))
    assert np.array_equal(nan, want) and want.sum() == 96


@pytest.mark.parametrize("bf", [True, False])
def test_decode_every_code_and_scale(bf):
    codes = np.tile(np.arange(256, dtype=np.uint8), (255, 1))
    scales = np.tile(np.arange(255, dtype=np.uint8)[:, None], (1, 16))
    out = torch.full((255, 512), -3.0, dtype=torch.bfloat16 if bf else torch.float32, device="cuda")
    B.moe_dequantize_mxfp4(_cfg(255, 512, bf), torch.from_numpy(codes).cuda(), None,
                           torch.from_numpy(scales).cuda(), out)
    want = bo.mxfp4_decode(codes, scales)
    got = out.double().cpu().numpy()
    with np.errstate(over="ignore"):
        want = want.astype(np.float32).astype(np.float64)  # beyond float32: infinity
    assert np.array_equal(got, want)
    assert np.array_equal(np.signbit(got), np.signbit(want))


@pytest.mark.parametrize("T,d,E,k,bf", [(1, 64, 4, 1, True), (77, 1088, 16, 4, True),
                                        (300, 256, 8, 2, False), (1000, 7168, 64, 8, True)])
def test_payload_gather(T, d, E, k, bf):
    log(f"[mxfp4] payload T={T} d={d} k={k}")
    rng = np.random.default_rng(5)
    x = rng.standard_normal((T, d)).astype(np.float32)
    x = om.round_bf16(x) if bf else x
    dev = _bits(x) if bf else torch.from_numpy(x).cuda()
    codes, scales = _quantize(dev, T, d, bf)
    src = rng.permutation(T * k).astype(np.int32)
    if T > 2:
        src[0], src[1] = -5, 2 ** 30  # malformed: clamped into the batch
    out = torch.zeros((T * k, d), dtype=dev.dtype, device="cuda")
    B.moe_dequantize_mxfp4(_cfg(T, d, bf, E=E, k=k), torch.from_numpy(codes).cuda(),
                           torch.from_numpy(src).cuda(), torch.from_numpy(scales).cuda(), out)
    want = bo.mxfp4_decode(codes, scales)[np.clip(src // k, 0, T - 1)]
    assert np.array_equal(out.double().cpu().numpy(), want)


@pytest.mark.parametrize("bf", [True, False])
def test_large_payload_gather(bf):
    """An x_perm large enough to be stored past the cache: the rows of the smaller decoding."""
    T, d, k = (8192, 5120, 2) if bf else (4096, 5120, 2)
    x = torch.randn((T, d), device="cuda").to(torch.bfloat16 if bf else torch.float32)
    codes, scales = B.quantize_mxfp4(x)
    src = torch.randperm(T * k, device="cuda").int()
    cfg = _cfg(T, d, bf, E=8, k=k)
    rows = torch.full((T, d), 3.0, dtype=x.dtype, device="cuda")
    B.moe_dequantize_mxfp4(cfg, codes, None, scales, rows)
    out = torch.full((T * k + 1, d), 3.0, dtype=x.dtype, device="cuda")
    B.moe_dequantize_mxfp4(cfg, codes, src, scales, out)
    assert torch.equal(out[:-1], rows[(src // k).long()]) and (out[-1] == 3.0).all()


def test_quantize_helper_and_other_stream():
    x = torch.randn((5, 3, 256), dtype=torch.bfloat16, device="cuda")
    want = B.quantize_mxfp4(x)
    assert want[0].shape == (5, 3, 128) and want[1].shape == (5, 3, 8)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = B.quantize_mxfp4(x)
    st.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------ products
def _weights(rng, E, n, K, unit):
    if unit:
        codes = rng.integers(0, 256, (E, n, K // 2), dtype=np.uint8)
        return codes, np.full((E, n, K // 32), 127, np.uint8)
    w = (rng.standard_normal((E * n, K)) * 0.02 * np.exp2(rng.integers(-3, 4, (E * n, 1)))).astype(np.float32)
    c, s = bo.mxfp4_quantize(w)
    return c.reshape(E, n, -1), s.reshape(E, n, -1)


def _dev(*a):
    return tuple(torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in a)


def _acts(rng, rows, K, unit):
    if unit:
        return rng.integers(0, 256, (rows, K // 2), dtype=np.uint8), np.full((rows, K // 32), 127, np.uint8)
    x = (rng.standard_normal((rows, K)) * np.exp2(rng.integers(-4, 4, (rows, 1)))).astype(np.float32)
    x[:, ::31] *= 20.0  # outliers: neighbouring blocks of very different scale
    return bo.mxfp4_quantize(x)


def _tables():
    z = lambda *c: np.concatenate([[0], np.cumsum(c)]).astype(np.int32)  # noqa: E731
    return {
        "one-row": (z(1), 1),
        "empty-and-ragged": (z(0, 5, 0, 33, 1, 0, 64, 2), 8),
        "long": (z(700, 130, 0, 257), 4),
        "skewed": (z(1, 1400, 3), 3),
        "last-empty": (z(31, 32, 33, 0), 4),
    }


def _bound(a, w, nk):
    """float32 and instruction bound of a @ w.T (see the file's head)."""
    K = a.shape[1]
    s = np.abs(a) @ np.abs(w).T
    top = np.zeros_like(s)
    for k0 in range(0, K, 64):
        pa, pw = np.abs(a[:, k0:k0 + 64]), np.abs(w[:, k0:k0 + 64])
        top += np.max(pa, 1)[:, None] * np.max(pw, 1)[None]
    return K * 2.0 ** -24 * s + 2.0 ** -11 * top


@pytest.mark.parametrize("table", sorted(_tables()))
@pytest.mark.parametrize("unit", [True, False])
@pytest.mark.parametrize("K,N", [(128, 128), (384, 256), (1408, 640)])
def test_down(table, unit, K, N):
    offs, E = _tables()[table]
    rows = int(offs[-1])
    log(f"[mxfp4] down {table} unit={unit} K={K} N={N}")
    rng = np.random.default_rng(rows + K)
    wc, ws = _weights(rng, E, N, K, unit)
    hc, hs = _acts(rng, rows, K, unit)
    cfg = B.config(T=rows, d=N, E=E, k=1, f=K)
    _, image = B.pack_weights_mxfp4(cfg, None, None, _dev(wc, ws))
    guard = 8
    y = torch.full((rows + guard, N), 7.5, dtype=torch.bfloat16, device="cuda")
    c, s, o = _dev(hc, hs, offs)
    B.moe_ffn_down_mxfp4(cfg, c, s, o, image, y)
    torch.cuda.synchronize()
    assert (y[rows:] == 7.5).all()
    got = y[:rows].double().cpu().numpy()
    h = bo.mxfp4_decode(hc, hs)
    for e in range(E):
        r = slice(offs[e], offs[e + 1])
        if offs[e] == offs[e + 1]:
            continue
        w = bo.mxfp4_decode(wc[e], ws[e])
        want = h[r] @ w.T
        if unit:
            exact = om.widen_bf16(om.round_bf16(want.astype(np.float32)))
            assert np.array_equal(got[r], exact), (table, e)
        else:
            err = np.abs(got[r] - want)
            assert (err <= 2.0 ** -8 * np.abs(want) + 1.01 * _bound(h[r], w, K // 64)).all(), (table, e)
            assert rel_err(got[r], want) <= 1e-2  # the stage bound of bf16 outputs


@pytest.mark.parametrize("T,d,E,k,f", [(1, 128, 4, 1, 128), (9, 256, 8, 2, 384), (150, 640, 5, 3, 128),
                                       (600, 384, 4, 2, 640), (37, 1280, 33, 4, 256)])
def test_gate_up_gather(T, d, E, k, f):
    log(f"[mxfp4] gate_up T={T} d={d} E={E} k={k} f={f}")
    rng = np.random.default_rng(T)
    g, u = _weights(rng, E, f, d, False), _weights(rng, E, f, d, False)
    xc, xs = bo.mxfp4_quantize(rng.standard_normal((T, d)).astype(np.float32))
    score = rng.random((T, E)) + np.linspace(1, 0, E)
    idx = np.argsort(-score, 1)[:, :k].astype(np.int32)
    p = om.permute(idx, E)
    cfg = B.config(T=T, d=d, E=E, k=k, f=f)
    image, _ = B.pack_weights_mxfp4(cfg, _dev(*g), _dev(*u), None)
    h = torch.full((T * k, f), 3.25, dtype=torch.bfloat16, device="cuda")
    c, s, src, o = _dev(xc, xs, np.asarray(p["src_of"], np.int32), np.asarray(p["offsets"], np.int32))
    B.moe_ffn_gate_up_mxfp4_gather(cfg, c, s, src, o, image, h)
    x = bo.mxfp4_decode(xc, xs)[np.asarray(p["src_of"]) // k]
    got = h.double().cpu().numpy()
    offs = np.asarray(p["offsets"])
    want = np.zeros_like(got)
    for e in range(E):
        r = slice(offs[e], offs[e + 1])
        a = x[r] @ bo.mxfp4_decode(g[0][e], g[1][e]).T
        b = x[r] @ bo.mxfp4_decode(u[0][e], u[1][e]).T
        want[r] = om.silu(a) * b
    assert rel_err(got, want) <= 1e-2


def test_sub_table_of_experts():
    """One rank's experts: the offsets and the image advanced by its first expert
    touch that rank's rows only."""
    rng = np.random.default_rng(2)
    E, K, N = 6, 256, 128
    offs = np.array([0, 3, 40, 40, 41, 75, 80], np.int32)
    wc, ws = _weights(rng, E, N, K, False)
    hc, hs = _acts(rng, 80, K, False)
    cfg = B.config(T=80, d=N, E=E, k=1, f=K)
    _, image = B.pack_weights_mxfp4(cfg, None, None, _dev(wc, ws))
    c, s, o = _dev(hc, hs, offs)
    full = torch.zeros((80, N), dtype=torch.bfloat16, device="cuda")
    B.moe_ffn_down_mxfp4(cfg, c, s, o, image, full)
    part = torch.full((80, N), 9.0, dtype=torch.bfloat16, device="cuda")
    sub = B.config(T=80, d=N, E=3, k=1, f=K)
    B.moe_ffn_down_mxfp4(sub, c, s, o[2:], image[2 * image.numel() // E:], part)
    assert torch.equal(part[40:75], full[40:75])
    assert (part[:40] == 9.0).all() and (part[75:] == 9.0).all()


def test_products_captured_and_replayed():
    rng = np.random.default_rng(4)
    T, d, E, k, f = 40, 256, 4, 2, 384
    g, u, dn = (_dev(*_weights(rng, E, *s, False)) for s in ((f, d), (f, d), (d, f)))
    cfg = B.config(T=T, d=d, E=E, k=k, f=f)
    qh = B.config(T=T * k, d=f, E=1, k=1, f=64)
    images = B.pack_weights_mxfp4(cfg, g, u, dn)
    x = torch.randn((T, d), dtype=torch.bfloat16, device="cuda")
    idx = torch.stack([torch.randperm(E, device="cuda")[:k] for _ in range(T)]).int().contiguous()
    p = om.permute(idx.cpu().numpy(), E)
    src, offs = _dev(np.asarray(p["src_of"], np.int32), np.asarray(p["offsets"], np.int32))
    new = lambda *s, t=torch.uint8: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    xc, xs, hc, hs = new(T, d // 2), new(T, d // 32), new(T * k, f // 2), new(T * k, f // 32)
    h, y = new(T * k, f, t=torch.bfloat16), new(T * k, d, t=torch.bfloat16)

    def step():
        B.moe_quantize_mxfp4(cfg, x, xc, xs)
        B.moe_ffn_gate_up_mxfp4_gather(cfg, xc, xs, src, offs, images[0], h)
        B.moe_quantize_mxfp4(qh, h, hc, hs)
        B.moe_ffn_down_mxfp4(cfg, hc, hs, offs, images[1], y)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x.copy_(torch.randn_like(x))
        step()
        torch.cuda.synchronize()
        want = y.clone()
        y.zero_()
        h.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i


@pytest.mark.parametrize("rows_per", [3, 200])
def test_non_finite_rows_stay_to_themselves(rows_per):
    """A block with a NaN makes its own row NaN and changes no bit of another."""
    rng = np.random.default_rng(rows_per)
    E, K, N = 3, 512, 256
    rows = E * rows_per
    offs = np.arange(E + 1, dtype=np.int32) * rows_per
    wc, ws = _weights(rng, E, N, K, False)
    hc, hs = _acts(rng, rows, K, False)
    cfg = B.config(T=rows, d=N, E=E, k=1, f=K)
    _, image = B.pack_weights_mxfp4(cfg, None, None, _dev(wc, ws))
    c, s, o = _dev(hc, hs, offs)
    clean = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
    B.moe_ffn_down_mxfp4(cfg, c, s, o, image, clean)
    assert torch.isfinite(clean).all()
    bad = [1, rows_per + 2, rows - 1]
    for i, r in enumerate(bad):
        s[r, 3 + i] = 255
    got = torch.zeros_like(clean)
    B.moe_ffn_down_mxfp4(cfg, c, s, o, image, got)
    rest = [r for r in range(rows) if r not in bad]
    assert torch.isnan(got[bad]).all() and torch.equal(got[rest], clean[rest])

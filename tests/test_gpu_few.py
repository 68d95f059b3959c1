"""The layer for a few tokens: routing bit for bit as moe_route, out against the
oracle's layer (float64) on bf16 and MXFP4 images.

Tolerance: TOL_LAYER, the layer's bf16 bound (h rounded to bf16 before the second product,
out rounded once; y is not rounded here), and elementwise the worst case of those
roundings, 2^-8 sum_j g_j |h_j| |Wd_j| + 2^-8 |out|, with 2^-16 of the first for the
float32 sums (k <= 2^8 terms a wave and block of 2^-24 each)."""
import numpy as np
import pytest
import torch

import oracle
from _gpu import TOL_LAYER, host, log, rel_err, upload
from oracle import block_oracle as bo
from top_routing_expert_amd import binding as B
from top_routing_expert_amd import configs as C
from top_routing_expert_amd import inputs as I

pytestmark = pytest.mark.gpu

BASE = C.MoEShape("few", T=1, d=256, E=8, k=2, f=256)
SHAPES = {
    "e8": BASE,
    "e1": BASE.replace(E=1, k=1),
    "e3-k3": BASE.replace(E=3, k=3, d=128, f=128),
    "e16-zipf": BASE.replace(E=16, d=384, bias="zipf"),
    "e64-presel": BASE.replace(E=64, presel=8, renorm=0, bias="normal", f=384),
    "e64-all": BASE.replace(E=64, k=4, renorm=0),
    "e64-g16": BASE.replace(E=64, k=4, n_group=16, topk_group=3, d=128, f=128),
    "e64-g32": BASE.replace(E=64, k=6, n_group=32, topk_group=5, d=128, f=128, bias="normal"),
    "e64-presel32": BASE.replace(E=64, k=4, presel=32, renorm=0, d=128, f=128),
    "e256-grouped": BASE.replace(E=256, k=8, n_group=8, topk_group=4, f=128),
    "e96-g48": BASE.replace(E=96, k=4, n_group=48, topk_group=7, f=128),
    "e1024": BASE.replace(E=1024, k=16, d=128, f=128, renorm=0),
    "d64": BASE.replace(d=64, f=64),          # bf16 images only: not multiples of 128
    "odd": BASE.replace(d=448, f=192, E=12),  # the same
}


def _images(shape, inp, dev, mx):
    """The images, and the float64 expert weights they stand for."""
    cfg = B.config(shape)
    if not mx:
        return B.pack_weights(cfg, dev["w_gate"], dev["w_up"], dev["w_down"]), inp
    q = {n: B.quantize_mxfp4(dev[n]) for n in ("w_gate", "w_up", "w_down")}
    vals = {n: bo.mxfp4_decode(host(c), host(s)) for n, (c, s) in q.items()}
    return B.pack_weights_mxfp4(cfg, q["w_gate"], q["w_up"], q["w_down"]), {**inp, **vals}


def _run(shape, dev, images, mx, bufs=True, ws=None, stream=None):
    T, E, k, d = shape.T, shape.E, shape.k, shape.d
    cfg = B.config(shape)
    out = torch.full((T + 2, d), 5.5, dtype=torch.bfloat16, device="cuda")
    b = dict(logits=torch.full((T, E), 9.0, device="cuda"),
             topk_idx=torch.full((T, k), -1, dtype=torch.int32, device="cuda"),
             topk_w=torch.full((T, k), 9.0, device="cuda"))
    if ws is None:
        ws = B.workspace(cfg, "layer_few")
        ws.fill_(0xFF)  # nothing in it need be initialised
    B.moe_layer_fwd_few(cfg, dev["x"], dev["w_router"], dev["bias"], *images, int(mx), out,
                        b if bufs else None, ws, stream)
    return out, b


def _compare(shape, inp, out, b):
    T = shape.T
    assert (out[T:] == 5.5).all()  # rows behind the batch are left alone
    kw = dict(k=shape.k, n_group=shape.n_group, topk_group=shape.topk_group, presel=shape.presel,
              renorm=shape.renorm)
    ref = oracle.layer(inp["x"], inp["w_router"], inp["bias"], inp["w_gate"], inp["w_up"],
                       inp["w_down"], logits32=host(b["logits"]), **kw)
    got, want = oracle.widen_bf16(host(out[:T])), ref["out"]
    assert rel_err(got, want) <= TOL_LAYER["bf16"]
    x = oracle.moe_oracle._f64(inp["x"])
    idx, g = host(b["topk_idx"]), host(b["topk_w"]).astype(np.float64)
    wg, wu, wd = (oracle.moe_oracle._f64(inp[n]) for n in ("w_gate", "w_up", "w_down"))
    worst = np.zeros_like(want)
    for t in range(T):
        for j in range(shape.k):
            e = idx[t, j]
            h = oracle.silu(wg[e] @ x[t]) * (wu[e] @ x[t])
            worst[t] += g[t, j] * (np.abs(wd[e]) @ np.abs(h))
    assert (np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -16) * worst + 2.0 ** -8 * np.abs(want)).all()
    return rel_err(got, want)


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp4"])
@pytest.mark.parametrize("T", [1, 2, 3, 16, 17, 32])
@pytest.mark.parametrize("name", sorted(SHAPES))
def test_layer(name, T, mx):
    shape = SHAPES[name].replace(T=T)
    if mx and (shape.d % 128 or shape.f % 128):
        pytest.skip("MXFP4 products take multiples of 128")
    if T not in (1, 17) and shape.E >= 256 and mx:
        pytest.skip("covered by the other batch sizes")
    log(f"[few] {name} T={T} mx={mx}")
    inp = I.make_inputs(shape, 11 + T)
    dev = upload(inp)
    images, vals = _images(shape, inp, dev, mx)
    out, b = _run(shape, dev, images, mx)
    cfg = B.config(shape)
    r = dict(logits=torch.empty_like(b["logits"]), idx=torch.empty_like(b["topk_idx"]),
             w=torch.empty_like(b["topk_w"]))
    B.moe_route(cfg, dev["x"], dev["w_router"], dev["bias"], r["logits"], r["idx"], r["w"],
                B.workspace(cfg, "route"))
    assert torch.equal(b["logits"], r["logits"])
    assert torch.equal(b["topk_idx"], r["idx"])
    assert torch.equal(b["topk_w"], r["w"])
    err = _compare(shape, vals, out, b)
    log(f"[few] {name} T={T} mx={mx} max rel err {err:.2e}")
    again, _ = _run(shape, dev, images, mx, bufs=False)
    assert torch.equal(again, out)  # and the routing outputs are optional


@pytest.mark.parametrize("shape", [C.E16_ZIPF, C.E64_PRESEL8, C.E8_D4096], ids=lambda s: s.name)
@pytest.mark.parametrize("T,mx", [(1, False), (1, True), (19, False), (32, True)])
def test_full_size(shape, T, mx):
    """The workloads' own widths, against float64 products of the chosen experts."""
    shape = shape.replace(T=T)
    log(f"[few] full size {shape.name} T={T} mx={mx}")
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    new = lambda *s, std=0.02: torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=g)  # noqa: E731
    T, d, E, k, f = shape.T, shape.d, shape.E, shape.k, shape.f
    dev = dict(x=new(T, d, std=1.0), w_router=new(E, d), bias=None, w_gate=new(E, f, d),
               w_up=new(E, f, d), w_down=new(E, d, f))
    images, _ = _images(shape, {}, dev, mx) if not mx else (None, None)
    if mx:
        q = {n: B.quantize_mxfp4(dev[n]) for n in ("w_gate", "w_up", "w_down")}
        cfg = B.config(shape)
        images = B.pack_weights_mxfp4(cfg, q["w_gate"], q["w_up"], q["w_down"])
        for n, (c, s) in q.items():  # the values the images stand for (decoding is exact)
            rows = dev[n].numel() // dev[n].shape[-1]
            dc = B.config(T=1024, d=dev[n].shape[-1], E=1, k=1, f=64)
            flat, fc, fs = dev[n].view(rows, -1), c.view(rows, -1), s.view(rows, -1)
            for r0 in range(0, rows, 1024):
                dc.T = min(1024, rows - r0)
                B.moe_dequantize_mxfp4(dc, fc[r0:], None, fs[r0:], flat[r0:])
    out, b = _run(shape, dev, images, mx)
    x = dev["x"].double()
    want = torch.zeros((T, d), dtype=torch.float64, device="cuda")
    idx, w = b["topk_idx"].tolist(), b["topk_w"].double()
    for t in range(T):
        for j, e in enumerate(idx[t]):
            a = dev["w_gate"][e].double() @ x[t]
            h = a * torch.sigmoid(a) * (dev["w_up"][e].double() @ x[t])
            want[t] += w[t, j] * (dev["w_down"][e].double() @ h)
    err = rel_err(out[:T].double().cpu().numpy(), want.cpu().numpy())
    log(f"[few] full size {shape.name} T={T} mx={mx} max rel err {err:.2e}")
    assert err <= TOL_LAYER["bf16"]


def test_streams_side_by_side():
    """Two calls at once on streams of their own, each with its workspace."""
    shape = SHAPES["e64-all"].replace(T=5, d=512, f=512)
    inp = I.make_inputs(shape, 3)
    dev = upload(inp)
    images, _ = _images(shape, inp, dev, False)
    want, _ = _run(shape, dev, images, False)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    wss = [B.workspace(B.config(shape), "layer_few") for _ in streams]
    outs = []
    for _ in range(4):
        for st, ws in zip(streams, wss):
            with torch.cuda.stream(st):
                outs.append(_run(shape, dev, images, False, ws=ws)[0])
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp4"])
def test_captured_and_replayed(mx):
    shape = SHAPES["e8"].replace(T=4)
    inp = I.make_inputs(shape, 6)
    dev = upload(inp)
    images, _ = _images(shape, inp, dev, mx)
    cfg, ws = B.config(shape), B.workspace(B.config(shape), "layer_few")
    out = torch.empty((shape.T, shape.d), dtype=torch.bfloat16, device="cuda")
    call = lambda: B.moe_layer_fwd_few(cfg, dev["x"], dev["w_router"], dev["bias"], *images,  # noqa: E731
                                       int(mx), out, None, ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        dev["x"].copy_(torch.randn_like(dev["x"]))
        call()
        torch.cuda.synchronize()
        want = out.clone()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_empty_batch():
    cfg = B.config(BASE, T=0)
    assert B.workspace(cfg, "layer_few") is None
    B.moe_layer_fwd_few(cfg, None, None, None, None, None, 0, None)


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp4"])
def test_non_finite_tokens_stay_to_themselves(mx):
    """Tokens of NaN and infinities choose experts in range, and no other token's
    routing or output moves by more than the order of its sums."""
    shape = SHAPES["e16-zipf"].replace(T=20)
    inp = I.make_inputs(shape, 8)
    dev = upload(inp)
    images, vals = _images(shape, inp, dev, mx)
    bad = [3, 7, 19]
    good = [t for t in range(shape.T) if t not in bad]
    dev["x"][3], dev["x"][7, 5], dev["x"][19] = float("nan"), float("inf"), float("-inf")
    out, b = _run(shape, dev, images, mx)
    idx = host(b["topk_idx"])
    assert ((idx >= 0) & (idx < shape.E)).all() and (idx[:, 0] != idx[:, 1]).all()
    assert all(torch.isnan(out[t]).any() for t in bad)
    ref = oracle.layer(inp["x"], inp["w_router"], inp["bias"], vals["w_gate"], vals["w_up"],
                       vals["w_down"], k=shape.k, renorm=shape.renorm)
    assert np.array_equal(idx[good], ref["topk_idx"][good])
    assert rel_err(oracle.widen_bf16(host(out[:shape.T]))[good], ref["out"][good]) <= TOL_LAYER["bf16"]

"""moe_forward_few (the whole layer for a few tokens in two launches) on the GPU against the 64-bit form of
tests/ref64.py.  Experts have to be equal: the logits are rounded once from 64 bits on both sides.  Weights: the
softmax's exponentials, sum and quotient are each off by a few 2^-24, so 2^-20 relative.  y: the tolerances of
test_gpu_6_routed.py (the same roundings), and for fp32, with rows of up to 2^13 here, 2^-15."""
import numpy as np
import pytest
import torch

import ref64
from gpu_util import host, rel_fro, say, y_to_f64
from sparse_mixture_experts_08_amd import binding as B
from sparse_mixture_experts_08_amd import workloads as W
from test_gpu_6_routed import TYPES, TOL as TOL6, WEIGHTS, bits, make, scales

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = {**TOL6, "f32": 2.0 ** -15}


def few(inp, k, **kw):
    return B.moe_forward_few(inp["x"], inp["Wg"], inp.get("bias"), *[inp[n] for n in WEIGHTS], k, scales=scales(inp), **kw)


def ref_route(h, x, k):
    z = x @ h["Wg"].astype(np.float64).T
    if h.get("bias") is not None:
        z = z + h["bias"].astype(np.float64)
    z = z.astype(np.float32)
    idx = np.argsort(-z, axis=1, kind="stable")[:, :k]              # equal logits: the lower expert first
    v = np.take_along_axis(z, idx, 1).astype(np.float64)
    w = np.exp(v - v[:, :1])
    return idx, w / w.sum(axis=1, keepdims=True)


def check(inp, k, wt, **kw):
    y, r = few(inp, k, routing=True, **kw)
    torch.cuda.synchronize()
    h = host(inp)
    x = y_to_f64(h["x"], TYPES[wt][0])
    idx, w = ref_route(h, x, k)
    assert np.array_equal(r["idx"].cpu().numpy(), idx)
    assert np.array_equal(r["counts"].cpu().numpy(), np.bincount(idx.ravel(), minlength=h["W1"].shape[0]))
    assert np.abs(r["w"].cpu().double().numpy() / w - 1).max() <= 2.0 ** -20
    want = ref64.layer(h, x, idx, w, wt)
    got = y.float().cpu().double().numpy()
    assert np.isfinite(got).all()
    err = rel_fro(got, want)
    rows = np.linalg.norm(got - want, axis=1) / np.linalg.norm(want, axis=1)
    say(f"  rel_fro={err:.2e} worst row {rows.max():.2e} (bound {TOL[wt]:.2e})")
    assert err <= TOL[wt] and rows.max() <= 4 * TOL[wt]
    return y


SHAPES = [  # T, d, E, k, inter, inter_shared
    (1, 128, 1, 1, 128, 128),                # the smallest layer
    (1, 512, 32, 4, 256, 256),
    (2, 384, 300, 16, 128, 384),             # E > 256, k = 16, d an odd multiple of 128
    (3, 1024, 1024, 8, 128, 128),            # the largest E
    (5, 1152, 64, 6, 384, 256),              # nine units of K for eight wavefronts
    (7, 256, 20, 3, 1152, 128),              # more than one chunk of h (fp32, bf16)
    (9, 256, 8, 2, 2304, 2176),              # ... in every type
    (16, 640, 16, 16, 128, 256),             # every expert for every token
    (16, 512, 256, 16, 128, 128),            # the most slots
    (13, 896, 2, 1, 256, 640),               # many tokens on one expert
]


@pytest.mark.parametrize("wt", ["mxfp4", "fp8", "bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_parity(wt, shape):
    say(f"[few] {wt} {shape}")
    check(make(wt, *shape), shape[3], wt)


@pytest.mark.parametrize("wt", ["mxfp4", "f32"])
@pytest.mark.parametrize("T", range(1, 17))
def test_every_token_count_with_skewed_routing(wt, T):
    say(f"[few] {wt} T={T}")
    check(make(wt, T, 384, 24, 3, 128, 128, seed=T, skew=True), 3, wt)


@pytest.mark.parametrize("wt", ["mxfp4", "fp8", "bf16"])
def test_full_width_rows(wt):
    # rows as long as the decode configuration's, few experts
    say(f"[few] full width {wt}")
    check(make(wt, 4, 7168, 12, 8, 2048, 2048), 8, wt)


@pytest.mark.parametrize("wt,T,d", [("f32", 16, 2048), ("f32", 5, 7168), ("bf16", 9, 7168), ("bf16", 16, 3712),
                                    ("fp8", 16, 7296), ("mxfp4", 16, 7296)])
def test_x_longer_than_the_lds(wt, T, d):
    # the up products then take x from memory with the weights; 7296 is an odd multiple of 128
    say(f"[few] x from memory {wt} T={T} d={d}")
    check(make(wt, T, d, 10, 3, 256, 384, skew=True), 3, wt)


def test_ties_go_to_the_lower_expert():
    say("[few] ties")
    inp = make("bf16", 16, 512, 64, 6, 128, 128)
    inp["Wg"][40:60] = inp["Wg"][5:25]                   # twenty pairs of equal logits
    check(inp, 6, "bf16")
    inp["x"].zero_()                                     # all logits equal, all outputs zero
    y, r = few(inp, 6, routing=True)
    assert (r["idx"].cpu() == torch.arange(6, dtype=torch.int32)).all() and not y.any()
    assert torch.equal(r["w"].cpu(), torch.full((16, 6), 1 / 6))


@pytest.mark.parametrize("wt", ["mxfp4", "fp8", "bf16", "f32"])
@pytest.mark.parametrize("T", [1, 6])
def test_a_token_that_is_not_finite_stays_alone(wt, T):
    # a NaN in x makes all of the token's logits NaN: equal keys, so the lowest experts are its own
    say(f"[few] NaN and infinity {wt} T={T}")
    inp = make(wt, T, 384, 24, 3, 256, 128)
    y = check(inp, 3, wt)
    bad = torch.zeros(T, dtype=torch.bool)
    bad[[0, T - 1]] = True
    inp["x"][T - 1, 200] = float("inf")
    inp["x"][0, 17] = float("nan")
    z, r = few(inp, 3, routing=True)
    assert r["idx"][0].tolist() == [0, 1, 2] and int(r["counts"].sum()) == 3 * T
    assert not torch.isfinite(z[bad.to(DEV)].float()).any()
    if T > 2:                                            # other experts selected: the sums' order may differ
        a, b = z[~bad.to(DEV)].double(), y[~bad.to(DEV)].double()
        assert float((a - b).norm() / b.norm()) <= 2 * TOL[wt]


@pytest.mark.parametrize("wt", ["mxfp4", "fp8", "bf16", "f32"])
def test_near_moe_forward(wt):
    # the same layer as moe_forward up to the order of sums: each within the tolerance of the 64-bit form
    say(f"[few] against moe_forward {wt}")
    inp = make(wt, 11, 512, 32, 4, 256, 384)
    y, r = few(inp, 4, routing=True)
    y2, r2 = B.forward_inputs(inp, 4, routing=True)
    assert torch.equal(r["idx"], r2["idx"]) and torch.equal(r["counts"], r2["counts"])
    assert rel_fro(y.float().cpu().numpy(), y2.float().cpu().numpy()) <= 2 * TOL[wt]


@pytest.mark.parametrize("wt,T", [("mxfp4", 16), ("mxfp4", 1), ("bf16", 5), ("fp8", 3), ("f32", 2)])
def test_dirty_workspace_guards_and_repeats(wt, T):
    say(f"[few] guards {wt} T={T}")
    inp = make(wt, T, 512, 16, 4, 256, 384)
    y0 = few(inp, 4)
    need = B.moe_few_workspace_size(B.make_shape(T, 512, 16, 4, 256, 384, *TYPES[wt]))
    for fill in (0x00, 0xFF, 0x7F):
        ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device=DEV)
        buf = torch.full((T + 9, 512), 7.0, dtype=inp["x"].dtype, device=DEV)
        y = few(inp, 4, y=buf[:T], workspace=ws[:need])
        torch.cuda.synchronize()
        assert torch.equal(bits(y), bits(y0))
        assert bool((buf[T:] == 7).all()) and bool((ws[need:] == fill).all())
        for _ in range(20):                              # one call after another on one workspace
            few(inp, 4, y=buf[:T], workspace=ws[:need])
        assert torch.equal(bits(buf[:T]), bits(y0))


def test_captured_into_a_graph_and_replayed():
    say("[few] captured")
    inp = make("mxfp4", 6, 512, 16, 4, 256, 256)
    y = torch.empty_like(inp["x"])
    ws = torch.empty(B.moe_few_workspace_size(B.make_shape(6, 512, 16, 4, 256, 256, *TYPES["mxfp4"])), dtype=torch.uint8, device=DEV)
    few(inp, 4, y=y, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        few(inp, 4, y=y, workspace=ws)
    for i in range(4):
        inp["x"].copy_(torch.randn(6, 512, device=DEV))
        want = few(inp, 4)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(y), bits(want))


def test_streams_at_once():
    # three calls in flight together, each with more blocks than the card holds of all of them
    say("[few] three streams")
    jobs = []
    for s, wt in enumerate(("mxfp4", "bf16", "fp8")):
        inp = make(wt, 3 + 5 * s, 1024, 64, 4, 512, 512, seed=s)
        jobs.append((inp, few(inp, 4), torch.cuda.Stream()))
    torch.cuda.synchronize()
    out = [[], [], []]
    for _ in range(10):
        for s, (inp, _, stream) in enumerate(jobs):
            with torch.cuda.stream(stream):
                out[s].append(few(inp, 4))
    torch.cuda.synchronize()
    for s in range(3):
        for y in out[s]:
            assert torch.equal(bits(y), bits(jobs[s][1]))


def test_decode_steps_of_a_small_model():
    # the operators as they are used together: weights made into MXFP4 by moe_quantize_mx, a prompt through the
    # grouped routing and moe_forward_routed, then single tokens through moe_forward_few, each layer's output
    # entering the next
    say("[few] prompt and decode steps")
    d, E, k, inter = 512, 16, 4, 256
    g = torch.Generator(device=DEV).manual_seed(3)
    layers = []
    for _ in range(2):
        lay = {"Wg": torch.randn(E, d, generator=g, device=DEV) * d ** -0.5}
        for n, rows, cols in (("W1", E * inter, d), ("W3", E * inter, d), ("W2", E * d, inter), ("S1", inter, d), ("S3", inter, d), ("S2", d, inter)):
            q, s = B.moe_quantize_mx(torch.randn(rows, cols, generator=g, device=DEV) * cols ** -0.5, B.MOE_MXFP4)
            shape = (E, rows // E) if n[0] == "W" else (rows,)
            lay[n], lay[n + "s"] = q.view(*shape, cols // 2), s.view(*shape, cols // 32)
        layers.append(lay)
    x = torch.randn(21, d, generator=g, device=DEV).to(torch.bfloat16)
    outs = []
    for rows, decode in ((slice(0, 17), False), (slice(17, 18), True), (slice(18, 21), True)):
        v = x[rows].contiguous()
        for lay in layers:
            inp = dict(lay, x=v)
            if decode:
                y, r = few(inp, k, routing=True)
            else:
                r = B.moe_route(v, lay["Wg"], None, k)
                y = B.moe_forward_routed(v, r["idx"], r["w"], *[lay[n] for n in WEIGHTS], scales=scales(lay))
            h = host(lay)
            want = ref64.layer(h, v.double().cpu().numpy(), r["idx"].cpu().numpy(), r["w"].cpu().numpy(), "mxfp4")
            assert rel_fro(y.double().cpu().numpy(), want) <= TOL["mxfp4"]
            v = (v + y).contiguous()
        outs.append(v)
    # a token's result does not depend on the company it had
    again = x[19:20].contiguous()
    for lay in layers:
        again = again + few(dict(lay, x=again), k)
    assert rel_fro(again.double().cpu().numpy(), outs[2][1:2].double().cpu().numpy()) <= 2 * TOL["mxfp4"]


def test_no_tokens():
    inp = make("bf16", 2, 256, 8, 2, 128, 128)
    inp["x"] = inp["x"][:0]
    y, r = few(inp, 2, routing=True)
    assert y.shape == (0, 256) and int(r["counts"].abs().sum()) == 0

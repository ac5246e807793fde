"""moe_forward_few without a GPU: what is refused on the host, before any launch."""
import ctypes
import os

import pytest
import torch

from sparse_mixture_experts_08_amd import binding as B
from sparse_mixture_experts_08_amd import workloads as W

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libmoe.so not built")
# x, Wg, bias, W1, W3, W2, W1s, W3s, W2s, S1, S3, S2, S1s, S3s, S2s, y, idx, w, counts, workspace
REQUIRED = [0, 1] + list(range(3, 16)) + [19]


def shape(**kw):
    base = dict(T=16, d=1024, E=32, k=4, inter=256, inter_shared=256, act_dtype=B.MOE_BF16, w_dtype=B.MOE_MXFP4)
    return B.make_shape(**{**base, **kw})


def call(s, change=None, ws_bytes=1 << 30):
    p = [ctypes.c_void_p(0x1000 * (i + 1)) for i in range(20)]
    for i, v in (change or {}).items():
        p[i] = v if v is None else ctypes.c_void_p(v)
    return B.lib().moe_forward_few(None if s is None else ctypes.byref(s), *p, ctypes.c_size_t(ws_bytes), None)


def test_shapes_and_types():
    assert call(None) == 1
    assert call(shape(T=17)) == 2 and call(shape(T=1 << 40)) == 2
    assert call(shape(T=-1)) == 1 and call(shape(k=33)) == 1
    assert call(shape(d=1000)) == 2 and call(shape(k=17)) == 2 and call(shape(E=1025)) == 2
    assert call(shape(act_dtype=B.MOE_F32)) == 2 and call(shape(w_dtype=B.MOE_MXFP8)) == 2


@pytest.mark.parametrize("i", REQUIRED)
def test_required_pointers(i):
    assert call(shape(), {i: None}) == 1


def test_alignment_aliasing_and_workspace():
    for i in (0, 1, 3, 9, 15):
        assert call(shape(), {i: 0x9008}) == 1
    for i in (6, 14):
        assert call(shape(), {i: 0x9002}) == 1
    assert call(shape(), {15: 0x1000}) == 1                        # y is x
    need = B.moe_few_workspace_size(shape())
    assert call(shape(), ws_bytes=need - 1) == 3 and call(shape(), {19: 0x9010}) == 3


def test_workspace_size():
    assert B.FEW_MAX_T == 16
    for wt, act in ((B.MOE_F32, B.MOE_F32), (B.MOE_BF16, B.MOE_BF16), (B.MOE_FP8_E4M3, B.MOE_BF16), (B.MOE_MXFP4, B.MOE_BF16)):
        sizes = [B.moe_few_workspace_size(shape(T=t, act_dtype=act, w_dtype=wt)) for t in (0, 1, 16)]
        assert 0 < sizes[0] <= sizes[1] < sizes[2] < 8 << 20
    assert B.moe_few_workspace_size(shape(T=17)) == 0 and B.moe_few_workspace_size(shape(d=100)) == 0
    assert call(shape(T=0), {i: None for i in range(20)}, ws_bytes=0) == 0


def test_binding_checks_tensors():
    inp = W.generate(W.Workload("few", 3, 256, 4, 2, 128, 256, W.BF16, W.BF16), device="cpu")
    good = dict(bias=None, k=2, **{n: inp[n] for n in ("x", "Wg", "W1", "W3", "W2", "S1", "S3", "S2")})
    for change in (dict(Wg=inp["Wg"].to(torch.bfloat16)), dict(Wg=inp["Wg"][:, :128]), dict(bias=torch.zeros(5)),
                   dict(W1=inp["W1"].float()), dict(S3=inp["S3"].float()), dict(x=inp["x"].half()),
                   dict(y=torch.empty(2, 256, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            B.moe_forward_few(**{**good, **change})

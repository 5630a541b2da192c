"""Parity of the layer norm (HIP, through the binding) with its formula in 64
bits (layer_ref), forwards and backwards.  Tolerances: half a step of the
result's type, and for the fp32 arithmetic 2^-24 times the number of roundings
on a term's way times its size (block_ref.close)."""
import pytest
import torch

import block_ref
import layer_ref as ref
from gpu_util import require_gpu, say
from test_gpu_block import Maker

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def dw():
    return require_gpu()


LAYER = [  # tokens, channels, type, weight, bias, strided, mean of a row over its deviation
    (1, 1, F32, True, True, False, 0.0),
    (0, 64, BF16, True, True, False, 0.0),
    (1, 8, BF16, True, True, True, 1.0),
    (3, 7, F16, True, False, True, 1.0),
    (65, 128, BF16, True, True, False, 1.0),
    (1000, 100, F32, False, True, True, 10.0),
    (131, 136, F16, True, True, False, 1.0),
    (67, 255, F32, True, True, False, 30.0),
    (33, 512, BF16, True, False, True, 1.0),
    (70, 513, F32, True, True, True, 1.0),
    (9, 1537, F32, True, True, False, 30.0),
    (300, 2048, BF16, True, True, False, 1.0),
    (1100, 640, BF16, True, True, True, 1.0),
    (5, 8200, F16, True, True, False, 1.0),
    (4, 16384, F32, True, True, True, 1.0),
    (2, 16383, BF16, False, False, False, 1.0),
    (20000, 24, BF16, True, True, False, 1.0),
]


@pytest.mark.parametrize("case", LAYER, ids=str)
def test_layer_norm(dw, case):
    T, ch, dtype, has_w, has_b, wide, mean = case
    say("layer norm", case)
    m = Maker(T + ch, dtype, wide)
    x, dout = m.act(T, ch, mean=mean), m.act(T, ch, packed=True)
    w, b = m.par(ch, mean=1.0, scale=0.3) if has_w else None, m.par(ch) if has_b else None
    out = torch.full((T, ch), 7.0, dtype=dtype, device="cuda")
    dw.ps_layer_norm(x, w, b, out=out)
    g = dw.ps_layer_norm_bwd(x, dout, w, b)
    torch.cuda.synchronize()
    want, mag = (ref.layer_norm(x, w, b, dout=dout, bound=v) for v in (False, True))
    K = ch + 64
    block_ref.close("out", out, want["out"], mag["out"], K)
    block_ref.close("dx", g.dx, want["dx"], mag["dx"], 2 * K)
    assert (g.dweight is None) == (w is None) and (g.dbias is None) == (b is None)
    if has_w:
        block_ref.close("dweight", g.dweight, want["dweight"], mag["dweight"], K + T)
    if has_b:
        block_ref.close("dbias", g.dbias, want["dbias"], mag["dbias"], K + T)


def test_layer_norm_keeps_rows_apart(dw):
    """A row of NaN or infinities is its own, in out and dx."""
    for ch in (100, 512, 1000):
        say("layer norm, rows apart", ch)
        m = Maker(ch, F32)
        x, dout = m.act(70, ch), m.act(70, ch)
        x[3], x[20, 5], x[64, 0] = float("nan"), float("inf"), float("-inf")
        out, g = dw.ps_layer_norm(x), dw.ps_layer_norm_bwd(x, dout)
        bad = torch.zeros(70, dtype=torch.bool, device="cuda")
        bad[[3, 20, 64]] = True
        for t in (out, g.dx):
            assert torch.isfinite(t[~bad]).all() and not torch.isfinite(t[bad]).all(1).any()


def test_layer_norm_of_equal_channels(dw):
    """A row without deviation: out is the bias, with eps in the root's place."""
    x = torch.full((5, 768), 3.0, dtype=F32, device="cuda")
    b = torch.randn(768, device="cuda")
    out = dw.ps_layer_norm(x, None, b)
    assert torch.equal(out, b.expand(5, 768))

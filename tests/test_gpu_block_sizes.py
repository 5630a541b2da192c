"""Calls of the state space block's operators whose work items pass the 32 bits
in which a launch counts them: short rows, so that the reference is a closed
form over all of them at once, in 64 bits on the GPU.

Tolerances: half a step of fp32 plus, for every rounding on a term's way, 2^-24
of the terms' magnitudes; the roundings are those of block_ref and scan_bound
(an argument of size |v| <= 8: 2 |v| + 14 for a step, 2 |v| + 7 for a gate, the
products and a sum over states: below 100)."""
import pytest
import torch

from block_ref import U32
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

F32, F64 = torch.float32, torch.float64


@pytest.fixture(scope="module")
def dw():
    yield require_gpu()
    torch.cuda.empty_cache()


def _maker(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s, dtype=F32: torch.randn(*s, generator=g, device="cuda").clamp_(-4.0, 4.0).to(dtype)


def _close(name, got, want, mag, roundings=100):
    half = torch.finfo(got.dtype).eps / 2
    tol = mag * (roundings * U32 * (1 + half)) + want.abs() * half + torch.finfo(got.dtype).tiny
    bad = ~((got.to(F64) - want).abs_() <= tol)
    assert not bad.any(), "%s: %d out of tolerance, first at %s" % (name, int(bad.sum()), bad.nonzero()[0].tolist())


def test_scan_of_many_short_sequences(dw):
    """2^23 + 77 sequences of one token: workgroups of 512 threads, forwards and
    for the gradients, and 2^30 sums of dB and dC in workgroups of 256."""
    T, N = (1 << 23) + 77, 64
    say("scan of many short sequences")
    r = _maker(1)
    x, dt, z, dout, B, C = r(T, 1), r(T, 1), r(T, 1), r(T, 1), r(T, 1, N), r(T, 1, N)
    A, D, bias = -r(1, N).abs(), r(1), r(1)
    off = torch.arange(T + 1, dtype=torch.int32, device="cuda")
    kept = torch.empty(dw.ps_selective_scan_checkpoint_rows(T, N), 1, N, device="cuda")
    more = dict(D=D, z=z, dt_bias=bias, offsets=off)
    ws = torch.empty(1 << 34, dtype=torch.uint8, device="cuda")
    out = dw.ps_selective_scan(x, dt, A, B, C, checkpoints=kept, workspace=ws, **more)
    g = dw.ps_selective_scan_bwd(x, dt, A, B, C, dout, kept, workspace=ws, **more)
    torch.cuda.synchronize()
    del ws, kept
    say("the closed form")
    x6, dt6, z6, do6, B6, C6 = (v.reshape(T, -1).to(F64) for v in (x, dt, z, dout, B, C))
    D6, raw = D.to(F64), dt6 + bias.to(F64)
    step, sig, sz = torch.logaddexp(raw, torch.zeros_like(raw)), torch.sigmoid(raw), torch.sigmoid(z6)
    bc = B6 * C6
    dot, size = bc.sum(1, keepdim=True), bc.abs_().sum(1, keepdim=True)  # sum over states of B C
    del bc
    inner, inner_size = step * x6 * dot + D6 * x6, (step * x6).abs() * size + (D6 * x6).abs()
    gate = z6 * sz
    _close("out", out, inner * gate, inner_size * gate.abs())
    gy = do6 * gate
    slope = sz * (1 + z6 * (1 - sz))
    _close("dz", g.dz, do6 * inner * slope, do6.abs() * inner_size * sz * (1 + z6.abs()))
    along, along_size = gy * dot, gy.abs() * size
    _close("dx", g.dx, D6 * gy + step * along, (D6 * gy).abs() + step * along_size)
    ddt = x6 * along * sig
    _close("ddt", g.ddt, ddt, x6.abs() * along_size * sig)
    _close("dB", g.dB.view(T, N), (gy * step * x6) * C6, ((gy * step * x6) * C6).abs())
    _close("dC", g.dC.view(T, N), (gy * step * x6) * B6, ((gy * step * x6) * B6).abs())
    assert (g.dA == 0).all()  # no state before the only row
    many = 100 + T // 32  # a column of partial sums: 32 runs of additions
    _close("dD", g.dD, (gy * x6).sum(0), (gy * x6).abs().sum(0), many)
    _close("ddt_bias", g.ddt_bias, ddt.sum(0), (x6.abs() * along_size * sig).sum(0), many)


def test_scan_step_of_many_rows(dw):
    """2^27 + 9 rows, eight a workgroup of 256 threads; states in place."""
    T = (1 << 27) + 9
    say("scan step of many rows")
    r = _maker(2)
    x, dt, B, C, state = r(T, 1), r(T, 1), r(T, 1, 1), r(T, 1, 1), r(T, 1, 1)
    A = -r(1, 1).abs()
    before = state.clone()
    out = dw.ps_selective_scan_step(x, state, dt, A, B, C)
    torch.cuda.synchronize()
    step = dt.view(T).to(F64)
    step = torch.logaddexp(step, torch.zeros_like(step))
    old = torch.exp(step * A.to(F64).view(1)) * before.view(T)
    add = step * x.view(T) * B.view(T)
    _close("state", state.view(T), old + add, old.abs() + add.abs())
    _close("out", out.view(T), (old + add) * C.view(T), (old.abs() + add.abs()) * C.view(T).abs())


def test_conv_step_of_many_rows(dw):
    """2^28 + 9 rows, four a workgroup of 64 threads; rows of state in place."""
    T = (1 << 28) + 9
    say("convolution step of many rows")
    r = _maker(3)
    x, state, w = r(T, 1), r(T, 1, 1), r(1, 2)
    before = state.clone()
    out = dw.ps_causal_conv_step(x, state, w)
    torch.cuda.synchronize()
    assert torch.equal(state.view(T), x.view(T))
    w = w.to(F64).view(2)
    old, new = before.view(T).to(F64).mul_(w[0]), x.view(T).to(F64).mul_(w[1])
    pre = old + new
    _close("out", out.view(T), pre * torch.sigmoid(pre), old.abs_().add_(new.abs_()).mul_(1.1))


def test_norm_of_many_rows(dw):
    """2^26 + 5 rows, one a workgroup of 64 threads."""
    T = (1 << 26) + 5
    say("norm of many rows")
    r = _maker(4)
    y, res = r(T, 2), r(T, 2)
    total, out = dw.ps_block_norm(y, res)
    torch.cuda.synchronize()
    y6, r6 = y.to(F64), res.to(F64)
    add = y6 * torch.rsqrt(y6.square().mean(1, keepdim=True) + 1e-6)
    want = r6 + add
    mag = r6.abs() + add.abs()
    _close("residual", total, want, mag)
    n = torch.rsqrt(want.square().mean(1, keepdim=True) + 1e-6)
    lean = (mag * want.abs()).mean(1, keepdim=True)
    _close("out", out, want * n, mag * n + want.abs() * n ** 3 * lean)

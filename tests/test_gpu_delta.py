"""Parity of the gated delta rule (HIP, through the binding) with its formula in
64 bits (delta_ref): forwards, backwards and for single tokens.  Tolerances are
derived in delta_ref."""
import pytest
import torch

import delta_ref as ref
from gpu_util import require_gpu, say
from test_gpu_block import Maker, _finite_rows, _offsets

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def dw():
    return require_gpu()


DELTA = [  # tokens, cuts, kheads, heads, key_dim, value_dim, type, normalize, initial, strided
    (1, None, 1, 1, 1, 1, F32, False, False, False),
    (0, [0, 0, 0], 2, 2, 16, 16, BF16, True, True, False),
    (1, [0, 1], 1, 2, 8, 5, BF16, True, True, True),
    (63, None, 1, 1, 32, 16, F32, True, False, False),
    (64, [0, 64], 2, 2, 32, 16, BF16, True, True, False),
    (65, None, 1, 1, 32, 64, F16, True, True, False),
    (200, None, 2, 2, 64, 64, BF16, True, False, False),
    (200, None, 2, 4, 64, 64, F32, True, True, True),
    (300, [0, 1, 1, 66, 131, 300], 3, 6, 40, 36, BF16, True, True, True),
    (300, [0, 1, 1, 66, 131, 300], 1, 3, 33, 17, F16, True, True, True),
    (300, [7, 70, 70, 290], 2, 2, 72, 100, F16, True, False, False),
    (190, [0, 50, 190], 2, 2, 128, 128, BF16, True, True, False),
    (190, None, 1, 2, 128, 128, F32, False, False, False),
    (150, [0, 20, 150], 1, 1, 128, 130, BF16, False, True, True),
    (130, [0, 66, 130], 1, 2, 256, 256, BF16, True, True, False),
    (130, None, 1, 1, 256, 70, F32, True, True, False),
    (130, None, 1, 1, 256, 40, F16, True, False, True),
    (130, [0, 129, 130], 1, 1, 130, 256, F32, True, True, True),
    (90, list(range(91)), 1, 2, 16, 24, BF16, True, True, False),
    (500, None, 1, 1, 24, 8, BF16, True, True, False),
    # long sequences: segments of them side by side
    (1500, None, 1, 2, 64, 72, BF16, True, True, False),
    (1600, [0, 1300, 1310, 1310, 1600], 1, 1, 128, 128, BF16, True, True, True),
    (1500, [0, 700, 1500], 1, 1, 40, 33, F16, True, False, False),
    (1024, None, 1, 1, 256, 20, F16, True, True, False),
    (1290, [3, 1290], 1, 1, 128, 96, F32, True, True, False),
    (1100, None, 1, 1, 200, 24, BF16, False, True, False),
]


class DeltaMaker(Maker):
    def of(self, v, dtype=None):
        """v as this maker's activations are laid out."""
        v = v.to(self.dtype if dtype is None else dtype).cuda()
        if not self.wide:
            return v
        row = v[0].numel()
        big = torch.full((v.shape[0], row + 13), float("nan"), dtype=v.dtype, device="cuda")
        big[:, 3:3 + row] = v.reshape(v.shape[0], row)
        return big[:, 3:3 + row].unflatten(1, v.shape[1:]) if v.dim() > 2 else big[:, 3:3 + row]


def delta_inputs(m, T, KH, H, K, V, normalize, initial, seqs):
    def keys():
        v = torch.randn(T, KH, K, generator=m.g)
        if not normalize:
            v = 0.9 * v / v.norm(dim=-1, keepdim=True).clamp(min=1e-3)
        return m.of(v)
    a = dict(q=keys(), k=keys(), v=m.act(T, H, V), g=m.of(-torch.rand(T, H, generator=m.g) ** 3, F32),
             beta=m.of(torch.sigmoid(torch.randn(T, H, generator=m.g)), F32))
    more = dict(initial=m.par(seqs, H, K, V, scale=0.5) if initial else None, normalize=normalize)
    return a, more


def _outside(cuts, T):
    keep = torch.ones(T, dtype=torch.bool)
    keep[_finite_rows(cuts, T)] = False
    return keep


@pytest.mark.parametrize("case", DELTA, ids=str)
def test_delta(dw, case):
    T, cuts, KH, H, K, V, dtype, normalize, initial, wide = case
    say("gated delta", case)
    m = DeltaMaker(T + K + V, dtype, wide)
    off = _offsets(cuts)
    seqs = 1 if cuts is None else len(cuts) - 1
    a, more = delta_inputs(m, T, KH, H, K, V, normalize, initial, seqs)
    out = torch.full((T, H, V), 7.0, dtype=dtype, device="cuda")
    final = torch.full((seqs, H, K, V), 7.0, device="cuda")
    dw.ps_gated_delta(**a, **more, offsets=off, out=out, final=final)
    torch.cuda.synchronize()
    want, bound = ref.delta(**a, **more, offsets=off, dtype=dtype)
    rows = _finite_rows(cuts, T)
    ref.close("out", out[rows], want["out"][rows], bound["out"][rows])
    ref.close("final", final, want["final"], bound["final"])
    assert (out.cpu()[_outside(cuts, T)] == 7.0).all()


@pytest.mark.parametrize("case", DELTA, ids=str)
def test_delta_gradients(dw, case):
    """From dout alone and, where there are initial states, from dfinal too."""
    T, cuts, KH, H, K, V, dtype, normalize, initial, wide = case
    say("gated delta, gradients", case)
    m = DeltaMaker(T + K + V, dtype, wide)
    off = _offsets(cuts)
    seqs = 1 if cuts is None else len(cuts) - 1
    a, more = delta_inputs(m, T, KH, H, K, V, normalize, initial, seqs)
    dout = m.act(T, H, V, packed=True)
    dfinal = m.par(seqs, H, K, V, scale=0.3) if initial else None
    kept = torch.full((dw.ps_gated_delta_checkpoint_floats(T, seqs, H, K, V),), float("nan"), device="cuda")
    out = torch.zeros(T, H, V, dtype=dtype, device="cuda")
    dw.ps_gated_delta(**a, **more, offsets=off, out=out, checkpoints=kept)
    again = torch.zeros_like(out)
    dw.ps_gated_delta(**a, **more, offsets=off, out=again)
    assert torch.equal(out, again)
    g = dw.ps_gated_delta_bwd(**a, **more, offsets=off, dout=dout, checkpoints=kept, dfinal=dfinal)
    torch.cuda.synchronize()
    want, bound = ref.delta(**a, **more, offsets=off, dout=dout, dfinal=dfinal, dtype=dtype)
    rows = _finite_rows(cuts, T)
    assert (g.dinitial is not None) == initial
    for name in g._fields:
        if name == "dinitial":
            if initial:
                ref.close(name, g.dinitial, want[name], bound[name])
        else:
            ref.close(name, getattr(g, name)[rows], want[name][rows], bound[name][rows])


STEP = [  # batch, pool, kheads, heads, key_dim, value_dim, type, normalize, slots, strided
    (1, 1, 1, 1, 1, 1, F32, False, False, False),
    (7, 9, 2, 4, 40, 36, BF16, True, True, True),
    (5, 5, 1, 3, 128, 128, BF16, True, False, False),
    (6, 8, 1, 1, 256, 256, F16, True, True, False),
    (3, 4, 2, 2, 33, 17, F32, True, True, True),
    (4, 4, 1, 1, 256, 7, F32, False, False, False),
    (4, 6, 1, 2, 8, 250, BF16, True, True, False),
    (70, 80, 4, 4, 64, 64, BF16, True, True, False),
]


@pytest.mark.parametrize("case", STEP, ids=str)
def test_delta_step(dw, case):
    B, pool, KH, H, K, V, dtype, normalize, use_slots, wide = case
    say("gated delta step", case)
    m = DeltaMaker(B + K + V, dtype, wide)
    a, _ = delta_inputs(m, B, KH, H, K, V, normalize, False, 1)
    state = m.par(pool, H, K, V)
    slots = torch.randperm(pool, generator=m.g)[:B].to(torch.int32)
    if B > 4:
        slots[2], slots[4] = -1, pool  # padding of the batch
    slots = slots.cuda() if use_slots else None
    want, bound = ref.delta_step(a["q"], a["k"], a["v"], state, a["g"], a["beta"], normalize=normalize, slots=slots, dtype=F32)
    new = state.clone()
    how = dict(normalize=normalize, slots=slots)
    args = (a["q"], a["k"], a["v"], state, a["g"], a["beta"])
    out = dw.ps_gated_delta_step(*args, **how, new_state=new)
    ref.close("out", out, want["out"], bound["out"])
    ref.close("state", new, want["state"], bound["state"])
    again = dw.ps_gated_delta_step(*args, **how)  # in place
    assert torch.equal(again, out) and torch.equal(state, new)

"""Parity of the gated delta rule by the norm over each head's rows (delta_norm):
every form that is compiled of its kernels, by type, padded keys, whole vectors or
not, and heads that share keys or not."""
import pytest
import torch

import delta_norm
import delta_ref as ref
from gpu_util import require_gpu, say
from test_gpu_block import _offsets
from test_gpu_delta import BF16, F16, F32, DeltaMaker, delta_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dw():
    return require_gpu()


# both dimensions whole vectors of 8, or not, in each of the four padded widths
DIMS = [(32, 24), (20, 17), (64, 72), (52, 60), (128, 64), (100, 33), (72, 256), (256, 40), (200, 130), (129, 24), (192, 100),
        (160, 32)]


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("shared", [1, 3])
@pytest.mark.parametrize("keys,values", DIMS)
def test_norms(dw, keys, values, shared, dtype):
    """Packed sequences of 1 to 130 rows from given states, dout and dfinal."""
    T, cuts, KH = 260, [3, 70, 71, 71, 201, 257], 2
    H, seqs, normalize = KH * shared, len(cuts) - 1, keys % 3 != 0
    m = DeltaMaker(keys + values, dtype, wide=values % 3 == 0)
    a, more = delta_inputs(m, T, KH, H, keys, values, normalize, True, seqs)
    a["g"] = m.of(delta_norm.decays(T, H, m.g), F32)
    dout, dfinal = m.act(T, H, values, packed=True), m.par(seqs, H, keys, values, scale=0.3)
    how = dict(more, offsets=_offsets(cuts))
    say("norms", keys, values, shared, dtype)
    kept = torch.empty(dw.ps_gated_delta_checkpoint_floats(T, seqs, H, keys, values), device="cuda")
    final = torch.empty(seqs, H, keys, values, device="cuda")
    out = dw.ps_gated_delta(**a, **how, final=final, checkpoints=kept)
    g = dw.ps_gated_delta_bwd(**a, **how, dout=dout, dfinal=dfinal, checkpoints=kept)
    torch.cuda.synchronize()
    want = ref.delta(**a, **how, dout=dout, dfinal=dfinal, dtype=dtype)[0]
    rows = slice(cuts[0], cuts[-1])
    for name, t in dict(out=out, final=final, **g._asdict()).items():
        if name in ("final", "dinitial"):
            delta_norm.close(name, t, want[name])
        else:
            delta_norm.close(name, t[rows], want[name][rows])


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("rows", [5, 40])
@pytest.mark.parametrize("keys,values", [(128, 128), (256, 72), (33, 17), (64, 64), (200, 256)])
def test_step_norms(dw, keys, values, rows, dtype):
    """Single tokens, few of them (a workgroup with few columns) and more."""
    KH, H = 2, 4
    m = DeltaMaker(keys + rows, dtype)
    a, _ = delta_inputs(m, rows, KH, H, keys, values, True, False, 1)
    state = m.par(rows + 3, H, keys, values)
    slots = torch.randperm(rows + 3, generator=m.g)[:rows].to(torch.int32).cuda()
    say("step norms", keys, values, rows, dtype)
    want = ref.delta_step(a["q"], a["k"], a["v"], state, a["g"], a["beta"], normalize=True, slots=slots)[0]
    out = dw.ps_gated_delta_step(a["q"], a["k"], a["v"], state, a["g"], a["beta"], normalize=True, slots=slots)
    delta_norm.close("out", out, want["out"])
    delta_norm.close("state", state, want["state"])

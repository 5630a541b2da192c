"""The gated delta rule with large states, or gradients of states, beside rows of
zeros, as padding has them: the zeros' powers of two must not take the rest past
fp32's range."""
import pytest
import torch

import delta_norm
import delta_ref as ref
from gpu_util import require_gpu, say
from test_gpu_delta import BF16, F32, DeltaMaker, delta_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dw():
    return require_gpu()


def _run(dw, a, more, dout, dfinal):
    T, H, V = a["v"].shape
    K = a["q"].shape[2]
    kept = torch.empty(dw.ps_gated_delta_checkpoint_floats(T, 1, H, K, V), device="cuda")
    final = torch.empty(1, H, K, V, device="cuda")
    out = dw.ps_gated_delta(**a, **more, final=final, checkpoints=kept)
    g = dw.ps_gated_delta_bwd(**a, **more, dout=dout, dfinal=dfinal, checkpoints=kept)
    torch.cuda.synchronize()
    return dict(out=out, final=final, **g._asdict())


@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
@pytest.mark.parametrize("size", [2.0 ** 18, 2.0 ** 24])
@pytest.mark.parametrize("zeros", ["keys and values", "queries and dout", "values and dout"])
def test_large_states_beside_zeros(dw, zeros, size, dtype):
    """All rows but the last, and a chunk of their own, are zeros in two inputs."""
    T, H, K, V = 150, 2, 48, 40
    m = DeltaMaker(70, dtype)
    a, more = delta_inputs(m, T, 1, H, K, V, True, True, 1)
    a["g"] = m.of(delta_norm.decays(T, H, m.g), F32)
    dout, dfinal = m.act(T, H, V), m.par(1, H, K, V, scale=size)
    more["initial"] *= size
    named = {"keys": a["k"], "values": a["v"], "queries": a["q"], "dout": dout}
    for name in zeros.split(" and "):
        named[name][:T - 1] = 0.0
    say("large states beside zeros", zeros, size, dtype)
    got = _run(dw, a, more, dout, dfinal)
    want = ref.delta(**a, **more, dout=dout, dfinal=dfinal, dtype=dtype)[0]
    for name, t in got.items():
        assert torch.isfinite(t).all(), name
        if bool((t.double().cpu() == want[name]).all()):
            continue
        delta_norm.close(name, t, want[name])

"""The gated delta rule with large states, or gradients of states, beside rows of
zeros, as padding has them: the zeros' powers of two must not take the rest past
fp32's range, and large numbers in one product must not take the bits of another."""
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


@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
@pytest.mark.parametrize("size", [2.0 ** 40, 2.0 ** 22, 2.0 ** -40])
@pytest.mark.parametrize("zeros", ["none", "keys and values", "queries and dout", "values and dout"])
def test_states_of_another_size(dw, zeros, size, dtype):
    """States and their gradients far from the activations in size.  Two planes hold a
    number to 2^-39 of the largest beside it in any case; delta_ref's bounds allow
    2^-12 of the columns' longest lengths a chunk, and with up to 64 rows of a chunk
    2^-39 of them is 2^-33: 2^-21 of those bounds, beside what delta_norm allows."""
    T, H, K, V = 150, 2, 48, 40
    m = DeltaMaker(70, dtype)
    a, more = delta_inputs(m, T, 1, H, K, V, True, True, 1)
    a["g"] = m.of(delta_norm.decays(T, H, m.g), F32)
    dout, dfinal = m.act(T, H, V), m.par(1, H, K, V, scale=size)
    more["initial"] *= size
    named = {"keys": a["k"], "values": a["v"], "queries": a["q"], "dout": dout}
    for name in zeros.split(" and ") if zeros != "none" else ():
        named[name][:T - 1] = 0.0
    say("states of another size", zeros, size, dtype)
    got = _run(dw, a, more, dout, dfinal)
    want, bound = ref.delta(**a, **more, dout=dout, dfinal=dfinal, dtype=dtype)
    heads = lambda t: t.transpose(0, 1).flatten(1).norm(dim=1)  # noqa: E731
    for name, t in got.items():
        assert torch.isfinite(t).all(), name
        size_of = heads(want[name])
        off = delta_norm.off_by(t, want[name]).nan_to_num(0.0, float("inf")) * size_of
        allowed = delta_norm.tolerance(name) * size_of + 2.0 ** -21 * heads(bound[name])
        assert bool((off <= allowed).all()), (name, off / size_of, allowed / size_of)

"""The gated delta rule over sequences long enough for segments side by side."""
import pytest
import torch

import block_ref
import delta_norm
import delta_ref as ref
from gpu_util import require_gpu, say
from test_gpu_block import _offsets
from test_gpu_delta import BF16, F16, F32, DeltaMaker, delta_inputs

pytestmark = pytest.mark.gpu

T, CUTS = 1500, [0, 1490, 1500]  # six segments of the first sequence


@pytest.fixture(scope="module")
def dw():
    return require_gpu()


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("keys,values", [(256, 40), (200, 24), (193, 17), (128, 40), (100, 33), (64, 72), (24, 16)])
def test_segments(dw, keys, values, dtype):
    """By norms, so that a single wrong column of the states that enter the segments
    is seen, with decays that leave much of a state after a segment."""
    H, seqs = 2, len(CUTS) - 1
    m = DeltaMaker(50 + keys, dtype)
    a, more = delta_inputs(m, T, 1, H, keys, values, True, True, seqs)
    a["g"] = m.of(delta_norm.decays(T, H, m.g), F32)
    dout, dfinal = m.act(T, H, values), m.par(seqs, H, keys, values, scale=0.3)
    how = dict(more, offsets=_offsets(CUTS))
    say("segments", keys, values, dtype)
    kept = torch.empty(dw.ps_gated_delta_checkpoint_floats(T, seqs, H, keys, values), device="cuda")
    final = torch.empty(seqs, H, keys, values, device="cuda")
    out = dw.ps_gated_delta(**a, **how, final=final, checkpoints=kept)
    g = dw.ps_gated_delta_bwd(**a, **how, dout=dout, dfinal=dfinal, checkpoints=kept)
    torch.cuda.synchronize()
    want = ref.delta(**a, **how, dout=dout, dfinal=dfinal, dtype=dtype)[0]
    for name, t in dict(out=out, final=final, **g._asdict()).items():
        delta_norm.close(name, t, want[name])


# a multiple of 32 keys and not, in each padded width; 129 to 192 keys leave the
# last 64 columns of what a segment does to a state without a walk
@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("keys", [129, 160, 192, 193, 256, 128, 72, 40, 64, 20])
def test_what_the_workspace_held_is_not_read(dw, keys, dtype):
    """On a workspace and checkpoints that hold NaN in every type, and again on zeros."""
    H, V, seqs = 2, 24, len(CUTS) - 1
    m = DeltaMaker(40 + keys, dtype)
    a, more = delta_inputs(m, T, 1, H, keys, V, True, True, seqs)
    a["g"] = m.of(delta_norm.decays(T, H, m.g), F32)
    dout, dfinal = m.act(T, H, V), m.par(seqs, H, keys, V, scale=0.3)
    how = dict(more, offsets=_offsets(CUTS))

    def run(byte):
        filled = lambda n: torch.full((n,), byte, dtype=torch.uint8, device="cuda")  # noqa: E731
        kept = filled(4 * dw.ps_gated_delta_checkpoint_floats(T, seqs, H, keys, V)).view(torch.float32)
        final = torch.empty(seqs, H, keys, V, device="cuda")
        out = dw.ps_gated_delta(**a, **how, final=final, checkpoints=kept, workspace=filled(1 << 26))
        g = dw.ps_gated_delta_bwd(**a, **how, dout=dout, dfinal=dfinal, checkpoints=kept, workspace=filled(1 << 26))
        torch.cuda.synchronize()
        return dict(out=out, final=final, **g._asdict())
    say("segments on a workspace of NaN", keys, dtype)
    got = run(0xFF)
    want = ref.delta(**a, **how, dout=dout, dfinal=dfinal, dtype=dtype)[0]
    for name, t in got.items():
        delta_norm.close(name, t, want[name])
    for name, t in run(0).items():
        assert torch.equal(t, got[name]), name


@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
def test_a_long_sequence_alone_and_among_others(dw, dtype):
    """Alone 1500 rows are cut into segments, among 29 short sequences they are walked
    whole: each is off from the formula by what delta_norm allows, so one is from the
    other by twice that (a rounding to 16 bits counts for both).  Calls alike in
    tokens and sequences give the same bits, whatever else they hold."""
    H, K, V, seqs, more_rows = 4, 48, 40, 30, 400
    m = DeltaMaker(60, dtype)
    a, more = delta_inputs(m, T + more_rows, 2, H, K, V, True, True, seqs)
    a["g"] = m.of(delta_norm.decays(T + more_rows, H, m.g), F32)
    dout = m.act(T + more_rows, H, V, packed=True)

    def run(rows, cuts, initial):
        at = {k: v[rows] for k, v in a.items()}
        n, s = at["q"].shape[0], len(cuts) - 1
        how = dict(offsets=_offsets(cuts), initial=initial, normalize=True)
        kept = torch.empty(dw.ps_gated_delta_checkpoint_floats(n, s, H, K, V), device="cuda")
        final = torch.empty_like(initial)
        out = dw.ps_gated_delta(**at, **how, checkpoints=kept, final=final)
        return out, final, dw.ps_gated_delta_bwd(**at, **how, dout=dout[rows], checkpoints=kept)
    say("a long sequence alone and among others", dtype)
    short = torch.arange(1, seqs) * more_rows // (seqs - 1)
    one, f1, g1 = run(slice(0, T), [0, T], more["initial"][:1].contiguous())
    two, f2, g2 = run(slice(0, T + more_rows), [0, T] + (T + short).tolist(), more["initial"])
    pairs = [("out", one, two), ("final", f1, f2), ("dinitial", g1.dinitial, g2.dinitial)]
    pairs += [(n, getattr(g1, n), getattr(g2, n)) for n in ("dq", "dk", "dv", "dg", "dbeta")]
    for name, x, y in pairs:
        y = y[:x.shape[0]]
        rounding = delta_norm.half_step(x.dtype, block_ref.f64(y)) * (x.dtype != F32)
        over = ((block_ref.f64(x) - block_ref.f64(y)).abs() - 2 * rounding).clamp(min=0.0)
        off = (over.norm() / block_ref.f64(y).norm()).item()
        assert off <= 2 * delta_norm.tolerance(name), (name, off)
    # the rows behind the first sequence changed and cut elsewhere
    for t in a.values():
        t[T:] = t[T:].flip(0)
    three, f3, g3 = run(slice(0, T + more_rows), [0, T] + (T + (short ** 2 // more_rows)).tolist(), more["initial"])
    assert torch.equal(two[:T], three[:T]) and torch.equal(f2[0], f3[0]) and torch.equal(g2.dinitial[0], g3.dinitial[0])
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(getattr(g2, n)[:T], getattr(g3, n)[:T]), n


@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
@pytest.mark.parametrize("where", ["q", "k", "v", "g", "initial", "dout", "dfinal"])
def test_nan_and_infinities_among_segments(dw, where, dtype):
    """In the third of six segments, of three sequences the second: other heads and
    rows before its chunk are what they are without it, from v and initial other
    columns too; other sequences keep every gradient, forwards and back."""
    H, K, V, cuts = 2, 48, 40, [0, 70, 1570, 1650]
    m = DeltaMaker(80, dtype)
    a, more = delta_inputs(m, cuts[-1], H, H, K, V, True, True, 3)
    a["g"] = m.of(delta_norm.decays(cuts[-1], H, m.g), F32)
    more.update(offsets=_offsets(cuts))
    back = dict(dout=m.act(cuts[-1], H, V, packed=True), dfinal=m.par(3, H, K, V))

    def run(a, more, back):
        kept = torch.empty(dw.ps_gated_delta_checkpoint_floats(cuts[-1], 3, H, K, V), device="cuda")
        final = torch.empty(3, H, K, V, device="cuda")
        out = dw.ps_gated_delta(**a, **more, final=final, checkpoints=kept)
        return dict(out=out, final=final, **dw.ps_gated_delta_bwd(**a, **more, **back, checkpoints=kept)._asdict())
    want = run(a, more, back)
    at = 70 + 512 + 64 + 7  # in the second chunk of that segment
    for bad in (float("nan"), float("inf")):
        say("nan and infinities among segments", where, bad, dtype)
        new = [{k: v.clone() if torch.is_tensor(v) else v for k, v in d.items()} for d in (a, more, back)]
        for d in new:
            if where in d:
                if where in ("initial", "dfinal"):
                    d[where][1, 1, 3, 5] = bad
                elif where == "g":
                    d[where][at, 1] = bad
                else:
                    d[where][at, 1, 5] = bad
        got = run(*new)
        for name, w in want.items():
            if name in ("final", "dinitial"):
                assert torch.equal(got[name][[0, 2]], w[[0, 2]]), name
            else:
                assert torch.equal(got[name][:70], w[:70]) and torch.equal(got[name][1570:], w[1570:]), name
            assert torch.equal(got[name][:, 0], w[:, 0]), name  # no heads share keys here
        if where in ("dout", "dfinal"):
            assert torch.equal(got["out"], want["out"]) and torch.equal(got["final"], want["final"])
            continue
        same = torch.ones(cuts[-1], H, V, dtype=torch.bool, device="cuda")
        first = 70 if where == "initial" else 70 + 512 + 64
        same[first:1570, 1, 5 if where in ("v", "initial") else slice(None)] = False
        assert torch.equal(got["out"][same], want["out"][same])
        after = slice(at, at + 1) if where == "q" else slice(at if where != "initial" else 70, 1570)
        cols = slice(5, 6) if where in ("v", "initial") else slice(None)
        assert not torch.isfinite(got["out"][after, 1, cols]).any()
        if where in ("v", "initial"):
            keep = [c for c in range(V) if c != 5]
            assert torch.equal(got["final"][1, 1][:, keep], want["final"][1, 1][:, keep])
            assert not torch.isfinite(got["final"][1, 1][:, 5]).any()

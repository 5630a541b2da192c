"""The state space block's operators on the CPU: the oracle's gradients
against autograd and differences, the pieces of packed sequences, and the
refusals of the C entry points and the binding (nothing is launched)."""
import ctypes
import os
import subprocess

import pytest
import torch

import block_ref as ref
import scan_bound

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000000  # a 256-byte aligned "device" address, never dereferenced
GB = 1 << 30
NULL, ALIAS, SIZE, WORKSPACE, UNSUPPORTED, ALIGNMENT = 1, 2, 3, 4, 5, 7


def _scan_inputs(T, ch, G, N, seed, seqs=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return dict(x=r(T, ch), dt=r(T, ch), A=-torch.rand(ch, N, generator=g, dtype=torch.float64) * 2, B=r(T, G, N),
                C=r(T, G, N), D=r(ch), z=r(T, ch), dt_bias=r(ch)), r


def _differences(f, t, dout, want, eps=1e-6):
    """want against central differences of sum(f * dout) at a few elements."""
    flat = t.view(-1)
    for i in range(0, flat.numel(), max(1, flat.numel() // 7)):
        old = float(flat[i])
        flat[i] = old + eps
        up = float((f() * dout).sum())
        flat[i] = old - eps
        down = float((f() * dout).sum())
        flat[i] = old
        # the difference is off by eps^2 and by 2^-53 / eps of the sum
        assert abs((up - down) / (2 * eps) - float(want.view(-1)[i])) <= 1e-6 * (1 + float(dout.abs().sum()))


def test_oracle_scan_gradients():
    off = torch.tensor([0, 3, 3, 9])
    a, r = _scan_inputs(9, 6, 2, 5, 1)
    a["initial"] = r(3, 6, 5)
    dout = r(9, 6)
    got = ref.scan(**a, offsets=off, dout=dout)
    for name, grad in (("x", "dx"), ("dt", "ddt"), ("A", "dA"), ("B", "dB"), ("C", "dC"), ("D", "dD"), ("z", "dz"),
                       ("dt_bias", "ddt_bias"), ("initial", "dinitial")):
        _differences(lambda: ref.scan(**a, offsets=off)["out"], a[name], dout, got[grad])


def test_oracle_conv_gradients():
    off = torch.tensor([0, 2, 2, 9])
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    a = dict(x=r(9, 3), weight=r(3, 4), bias=r(3), initial=r(3, 3, 3))
    dout = r(9, 3)
    got = ref.conv(**a, offsets=off, dout=dout)
    for name in a:
        _differences(lambda: ref.conv(**a, offsets=off)["out"], a[name], dout, got["d" + name])


def test_oracle_norm_gradients():
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    a = dict(y=r(4, 7), residual=r(4, 7), gate=r(4, 7), scale=r(7), post=r(7), pre=r(7))
    dout, dres = r(4, 7), r(4, 7)
    kept = ref.norm(**a)["residual"]
    got = ref.norm_bwd(a["y"], kept, dout, dres, a["gate"], a["scale"], a["post"], a["pre"])

    def both():
        v = ref.norm(**a)
        return torch.cat([v["out"], v["residual"]])
    for name in a:
        _differences(both, a[name], torch.cat([dout, dres]), got["d" + name])


def test_pieces(tmp_path):
    exe = str(tmp_path / "pieces_model")
    subprocess.run(["g++", "-O1", "-g", "-fsanitize=undefined,address", "-std=c++17", "-Wall", "-Wextra", "-Werror",
                    "-I" + os.path.join(ROOT, "device_wide_prefix_chained_amd", "csrc"),
                    os.path.join(ROOT, "tests", "c", "pieces_model.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and " 0 violations" in r.stdout, r.stdout + r.stderr


def _run_model(tmp_path, name):
    exe = str(tmp_path / name)
    subprocess.run(["g++", "-O1", "-g", "-fsanitize=undefined,address", "-std=c++17", "-Wall", "-Wextra", "-Werror",
                    "-I" + os.path.join(ROOT, "device_wide_prefix_chained_amd", "csrc"),
                    os.path.join(ROOT, "tests", "c", name + ".cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and " 0 violations" in r.stdout, r.stdout + r.stderr


def test_scan_shape(tmp_path):
    """A kernel without bounds has a state and a channel in every place, for
    all numbers of states that the scan takes."""
    _run_model(tmp_path, "scan_shape_model")


def test_launches_in_parts(tmp_path):
    """More work than one launch can count is launched in parts."""
    _run_model(tmp_path, "launch_parts_model")


def test_bounded_scan_is_the_oracle():
    """scan_bound's values are block_ref's, and its bounds are those of an
    arithmetic with 24 bits: small next to the values, and zero nowhere that
    something is computed."""
    off = torch.tensor([0, 3, 3, 40])
    a, r = _scan_inputs(40, 6, 2, 5, 4)
    a["initial"] = r(3, 6, 5)
    dout = r(40, 6)
    want = ref.scan(**a, offsets=off, dout=dout)
    got, bound = scan_bound.scan(**a, offsets=off, dout=dout)
    assert set(got) == set(want) == set(bound)
    for name in want:
        size = want[name].abs().mean()
        assert torch.allclose(got[name], want[name], rtol=1e-12, atol=1e-12 * float(size)), name
        assert 0 < float(bound[name].mean()) < 2.0 ** -10 * float(size), name


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def _mod():
    import device_wide_prefix_chained_amd as dw
    from device_wide_prefix_chained_amd import _block
    dw.lib()
    return _block, _block._lib()


def _at(i):
    return FAKE + i * GB


def _conv(b, **kw):
    a = dict(x=_at(1), x_stride=64, weight=_at(2), bias=_at(3), offsets=None, initial=None, tokens=100, channels=64,
             width=4, num_seqs=1, dtype=b.PS_BF16)
    a.update(kw)
    return b._ConvInput(**a)


CONV_BAD = [(dict(dtype=0), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(dtype=9), UNSUPPORTED),
            (dict(channels=0), SIZE), (dict(channels=(1 << 24) + 1, x_stride=1 << 25), SIZE), (dict(width=0), SIZE),
            (dict(width=9), SIZE), (dict(x_stride=63), SIZE), (dict(x_stride=-64), SIZE), (dict(tokens=1 << 31), SIZE),
            (dict(num_seqs=2), SIZE), (dict(num_seqs=1 << 24, offsets=FAKE), SIZE), (dict(x=None), NULL),
            (dict(weight=None), NULL), (dict(x=FAKE + 1), ALIGNMENT), (dict(weight=FAKE + 2), ALIGNMENT),
            (dict(bias=FAKE + 2), ALIGNMENT), (dict(offsets=FAKE + 2), ALIGNMENT), (dict(initial=FAKE + 1), ALIGNMENT)]


@pytest.mark.parametrize("bad,code", CONV_BAD)
def test_conv_refuses(bad, code):
    b, L = _mod()
    a = _conv(b, **bad)
    big = ctypes.c_size_t(GB)
    assert L.ps_causal_conv(a, _at(5), None, None) == code
    assert L.ps_causal_conv_bwd(FAKE, ctypes.byref(big), a, _at(5), _at(6), _at(7), None, None, None) == code
    if "num_seqs" not in bad and "offsets" not in bad:
        assert L.ps_causal_conv_step(a, _at(5), _at(5), None, 100, _at(6), None) == code


def test_conv_refuses_more():
    b, L = _mod()
    big, small, a = ctypes.c_size_t(GB), ctypes.c_size_t(300), _conv(b)
    assert L.ps_causal_conv(None, _at(5), None, None) == NULL
    assert L.ps_causal_conv(a, None, None, None) == NULL
    assert L.ps_causal_conv(a, _at(1) + 128, None, None) == ALIAS
    assert L.ps_causal_conv(a, _at(5), _at(5), None) == ALIAS
    assert L.ps_causal_conv(a, _at(5) + 1, None, None) == ALIGNMENT
    assert L.ps_causal_conv_bwd(FAKE, None, a, _at(5), _at(6), _at(7), None, None, None) == NULL
    assert L.ps_causal_conv_bwd(FAKE, ctypes.byref(small), a, _at(5), _at(6), _at(7), None, None, None) == WORKSPACE
    assert L.ps_causal_conv_bwd(FAKE, ctypes.byref(big), a, None, _at(6), _at(7), None, None, None) == NULL
    assert L.ps_causal_conv_bwd(FAKE, ctypes.byref(big), a, _at(5), _at(1), _at(7), None, None, None) == ALIAS
    assert L.ps_causal_conv_bwd(FAKE, ctypes.byref(big), a, _at(5), _at(6), None, None, None, None) == NULL
    assert L.ps_causal_conv_step(a, _at(5), _at(5), None, 99, _at(6), None) == SIZE   # no slots, pool too small
    assert L.ps_causal_conv_step(a, None, _at(5), None, 100, _at(6), None) == NULL
    assert L.ps_causal_conv_step(a, _at(5), _at(5) + 128, None, 100, _at(6), None) == ALIAS  # not the state itself
    assert L.ps_causal_conv_step(a, _at(5), _at(5), FAKE + 2, 100, _at(6), None) == ALIGNMENT
    assert L.ps_causal_conv_step(_conv(b, tokens=0, x=None), None, None, None, 0, None, None) == 0
    # the size query looks at no pointer
    need = ctypes.c_size_t(0)
    assert L.ps_causal_conv_bwd(None, ctypes.byref(need), _conv(b, x=None, weight=None), None, None, None, None, None,
                                None) == 0
    assert need.value > 256


def _scan(b, **kw):
    a = dict(x=_at(1), dt=_at(2), z=_at(3), B=_at(4), C=_at(5), x_stride=64, dt_stride=64, z_stride=64, b_stride=32,
             c_stride=32, A=_at(6), D=_at(7), dt_bias=_at(8), offsets=None, initial=None, tokens=100, channels=64,
             groups=2, states=16, num_seqs=1, dtype=b.PS_F16)
    a.update(kw)
    return b._ScanInput(**a)


SCAN_BAD = [(dict(dtype=0), UNSUPPORTED), (dict(dtype=7), UNSUPPORTED), (dict(channels=0), SIZE), (dict(groups=0), SIZE),
            (dict(groups=3), SIZE), (dict(groups=128), SIZE), (dict(states=0), SIZE), (dict(states=257, b_stride=999,
                                                                                            c_stride=999), SIZE),
            (dict(x_stride=63), SIZE), (dict(dt_stride=63), SIZE), (dict(z_stride=63), SIZE), (dict(b_stride=31), SIZE),
            (dict(c_stride=31), SIZE), (dict(tokens=1 << 31), SIZE), (dict(num_seqs=2), SIZE), (dict(x=None), NULL),
            (dict(dt=None), NULL), (dict(A=None), NULL), (dict(B=None), NULL), (dict(C=None), NULL),
            (dict(x=FAKE + 1), ALIGNMENT), (dict(z=FAKE + 1), ALIGNMENT), (dict(B=FAKE + 1), ALIGNMENT),
            (dict(A=FAKE + 2), ALIGNMENT), (dict(D=FAKE + 2), ALIGNMENT), (dict(initial=FAKE + 2), ALIGNMENT),
            (dict(offsets=FAKE + 2), ALIGNMENT)]


def _grads(b, **kw):
    a = dict(dx=_at(20), ddt=_at(21), dz=_at(22), dB=_at(23), dC=_at(24), dA=_at(25), dD=_at(26), ddt_bias=_at(27),
             dinitial=None)
    a.update(kw)
    return b._ScanGrads(**a)


@pytest.mark.parametrize("bad,code", SCAN_BAD)
def test_scan_refuses(bad, code):
    b, L = _mod()
    a, big = _scan(b, **bad), ctypes.c_size_t(GB)
    assert L.ps_selective_scan(FAKE, ctypes.byref(big), a, _at(10), None, None, None) == code
    assert L.ps_selective_scan_bwd(FAKE, ctypes.byref(big), a, _at(11), _at(12), _grads(b), None) == code
    if "num_seqs" not in bad:
        assert L.ps_selective_scan_step(a, _at(10), _at(10), None, 100, _at(11), None) == code


def test_scan_refuses_more():
    b, L = _mod()
    big, small, a = ctypes.c_size_t(GB), ctypes.c_size_t(300), _scan(b)
    s, ref_big = L.ps_selective_scan, ctypes.byref(big)
    assert s(FAKE, ref_big, None, _at(10), None, None, None) == NULL
    assert s(FAKE, None, a, _at(10), None, None, None) == NULL
    assert s(FAKE, ref_big, a, None, None, None, None) == NULL
    for taken in (1, 2, 3, 4, 5):
        assert s(FAKE, ref_big, a, _at(taken), None, None, None) == ALIAS
    assert s(FAKE, ref_big, a, _at(10), _at(10), None, None) == ALIAS
    assert s(FAKE, ref_big, a, _at(10), None, _at(10), None) == ALIAS
    assert s(FAKE, ref_big, a, _at(10) + 1, None, None, None) == ALIGNMENT
    assert s(FAKE, ref_big, a, _at(10), _at(11) + 2, None, None) == ALIGNMENT
    w = L.ps_selective_scan_bwd
    assert w(FAKE, ctypes.byref(small), a, _at(11), _at(12), _grads(b), None) == WORKSPACE
    assert w(FAKE, ref_big, a, None, _at(12), _grads(b), None) == NULL
    assert w(FAKE, ref_big, a, _at(11), None, _grads(b), None) == NULL
    assert w(FAKE, ref_big, a, _at(11), _at(12), None, None) == NULL
    for name in ("dx", "ddt", "dB", "dC", "dA"):
        assert w(FAKE, ref_big, a, _at(11), _at(12), _grads(b, **{name: None}), None) == NULL
    assert w(FAKE, ref_big, a, _at(11), _at(12), _grads(b, dx=_at(1)), None) == ALIAS
    assert w(FAKE, ref_big, a, _at(11), _at(12), _grads(b, ddt=_at(11)), None) == ALIAS
    assert w(FAKE, ref_big, a, _at(11), _at(12), _grads(b, dB=_at(4)), None) == ALIAS
    assert w(FAKE, ref_big, a, _at(11), _at(12), _grads(b, dA=_at(25) + 2), None) == ALIGNMENT
    st = L.ps_selective_scan_step
    assert st(a, _at(10), _at(10), None, 99, _at(11), None) == SIZE
    assert st(a, _at(10), _at(10) + 4096, None, 100, _at(11), None) == ALIAS
    assert st(a, _at(10), _at(12), None, 100, _at(10), None) == ALIAS
    assert st(a, None, _at(12), None, 100, _at(11), None) == NULL
    assert st(_scan(b, tokens=0, x=None, dt=None, B=None, C=None), None, None, None, 0, None, None) == 0
    rows = L.ps_selective_scan_checkpoint_rows
    assert [rows(t, 16) for t in (0, 1, 32, 33, 1 << 20)] == [0, 1, 1, 2, 1 << 15]
    need = ctypes.c_size_t(0)
    assert s(None, ctypes.byref(need), _scan(b, x=None, A=None), None, None, None, None) == 0 and need.value >= 256
    assert w(None, ctypes.byref(need), _scan(b, x=None, A=None), None, None, None, None) == 0 and need.value > 256


def test_scan_refuses_more_blocks_than_a_launch_holds():
    b, L = _mod()
    big = ctypes.c_size_t(1 << 60)
    wide = dict(x_stride=1 << 24, dt_stride=1 << 24, z=None, states=1, b_stride=1 << 24, c_stride=1 << 24, tokens=1)
    for channels, groups, code in ((1 << 23, 1 << 23, SIZE), (1 << 24, 1 << 23, SIZE), ((1 << 23) - 1, (1 << 23) - 1, 0)):
        a, need = _scan(b, channels=channels, groups=groups, **wide), ctypes.c_size_t(0)
        assert L.ps_selective_scan(None, ctypes.byref(need), a, None, None, None, None) == code
        assert L.ps_selective_scan_bwd(None, ctypes.byref(need), a, None, None, None, None) == code
        if code:
            assert L.ps_selective_scan(FAKE, ctypes.byref(big), a, _at(10), None, None, None) == code
            assert L.ps_selective_scan_step(a, _at(10), _at(10), None, 100, _at(11), None) == code


def test_size_queries_take_more_than_one_launch_holds():
    """Sizes inside the documented limits whose work items pass 32 bits."""
    b, L = _mod()
    need = ctypes.c_size_t(0)
    ref_need = ctypes.byref(need)
    many = dict(offsets=FAKE, num_seqs=(1 << 24) - 1, tokens=(1 << 24) - 1)
    for channels in (2048, 1 << 14):
        a = _scan(b, channels=channels, groups=1, x_stride=channels, dt_stride=channels, z_stride=channels, **many)
        assert L.ps_selective_scan(None, ref_need, a, None, None, None, None) == 0
        assert L.ps_selective_scan_bwd(None, ref_need, a, None, None, None, None) == 0
        a = _conv(b, channels=channels, x_stride=channels, **many)
        assert L.ps_causal_conv_bwd(None, ref_need, a, None, None, None, None, None, None) == 0


def _norm(b, **kw):
    a = dict(y=_at(1), gate=_at(2), residual=_at(3), y_stride=64, gate_stride=64, residual_stride=64, scale=_at(4),
             post_weight=_at(5), pre_weight=_at(6), tokens=100, channels=64, dtype=b.PS_BF16, residual_dtype=1, eps=1e-6)
    a.update(kw)
    return b._NormInput(**a)


NORM_BAD = [(dict(dtype=0), UNSUPPORTED), (dict(residual_dtype=4), UNSUPPORTED), (dict(residual_dtype=0), UNSUPPORTED),
            (dict(channels=0), SIZE), (dict(channels=16385, y_stride=1 << 15, gate_stride=1 << 15,
                                            residual_stride=1 << 15), SIZE), (dict(y_stride=63), SIZE),
            (dict(gate_stride=63), SIZE), (dict(residual_stride=63), SIZE), (dict(tokens=1 << 31), SIZE),
            (dict(y=None), NULL), (dict(residual=None), NULL), (dict(y=FAKE + 1), ALIGNMENT),
            (dict(residual=FAKE + 2), ALIGNMENT), (dict(scale=FAKE + 2), ALIGNMENT)]


@pytest.mark.parametrize("bad,code", NORM_BAD)
def test_norm_refuses(bad, code):
    b, L = _mod()
    a, big = _norm(b, **bad), ctypes.c_size_t(GB)
    g = b._NormGrads(_at(20), _at(21), _at(22), _at(23), _at(24), _at(25))
    assert L.ps_block_norm(a, _at(10), _at(11), None) == code
    assert L.ps_block_norm_bwd(FAKE, ctypes.byref(big), a, _at(12), _at(13), g, None) == code


def test_norm_refuses_more():
    b, L = _mod()
    big, small, a = ctypes.c_size_t(GB), ctypes.c_size_t(300), _norm(b)
    assert L.ps_block_norm(None, _at(10), _at(11), None) == NULL
    assert L.ps_block_norm(a, None, _at(11), None) == NULL
    assert L.ps_block_norm(a, _at(10), None, None) == NULL
    assert L.ps_block_norm(a, _at(3), _at(11), None) == ALIAS
    assert L.ps_block_norm(a, _at(10), _at(10), None) == ALIAS
    assert L.ps_block_norm(a, _at(10) + 2, _at(11), None) == ALIGNMENT
    assert L.ps_block_norm(_norm(b, tokens=0, y=None, residual=None), None, None, None) == 0
    g = b._NormGrads(_at(20), _at(21), _at(22), _at(23), _at(24), _at(25))
    w = L.ps_block_norm_bwd
    assert w(FAKE, ctypes.byref(small), a, _at(12), _at(13), g, None) == WORKSPACE
    assert w(FAKE, ctypes.byref(big), a, None, _at(13), g, None) == NULL
    assert w(FAKE, ctypes.byref(big), a, _at(12), _at(13), None, None) == NULL
    assert w(FAKE, ctypes.byref(big), a, _at(12), _at(13), b._NormGrads(None, _at(21), _at(22)), None) == NULL
    assert w(FAKE, ctypes.byref(big), a, _at(12), _at(13), b._NormGrads(_at(1), _at(21), _at(22)), None) == ALIAS


# Every output of an entry point laid over every input and every other output.
# The arrays of a call stand at places of their own (_at); a case moves one.
def _alias_calls():
    b, L = _mod()
    big = ctypes.byref(ctypes.c_size_t(GB))

    def conv(at):
        return _conv(b, x=at["x"], weight=at["weight"], bias=at["bias"], offsets=at["offsets"], initial=at["initial"],
                     num_seqs=3)

    def scan(at):
        return _scan(b, **{k: at[k] for k in ("x", "dt", "z", "B", "C", "A", "D", "dt_bias", "offsets", "initial")}, num_seqs=3)

    def norm(at):
        return _norm(b, **{k: at[k] for k in ("y", "gate", "residual", "scale", "post_weight", "pre_weight")})
    conv_in = ("x", "weight", "bias", "offsets", "initial")
    step_in = ("x", "weight", "bias", "state", "slots")
    scan_in = ("x", "dt", "z", "B", "C", "A", "D", "dt_bias", "offsets", "initial")
    scan_grads = ("dx", "ddt", "dz", "dB", "dC", "dA", "dD", "ddt_bias", "dinitial")
    norm_in = ("y", "gate", "residual", "scale", "post_weight", "pre_weight")
    norm_grads = ("dy", "dgate", "dresidual", "dscale", "dpost_weight", "dpre_weight")
    off = dict(offsets=None, initial=None)
    return {
        "conv": (conv_in, ("out", "final"), lambda at: L.ps_causal_conv(conv(at), at["out"], at["final"], None)),
        "conv_bwd": (conv_in + ("dout",), ("dx", "dweight", "dbias", "dinitial"),
                     lambda at: L.ps_causal_conv_bwd(FAKE, big, conv(at), at["dout"], at["dx"], at["dweight"], at["dbias"],
                                                     at["dinitial"], None)),
        "conv_step": (step_in, ("out", "new_state"),
                      lambda at: L.ps_causal_conv_step(conv(dict(at, **off)), at["state"], at["new_state"], at["slots"], 100,
                                                       at["out"], None)),
        "scan": (scan_in, ("out", "final", "checkpoints"),
                 lambda at: L.ps_selective_scan(FAKE, big, scan(at), at["out"], at["final"], at["checkpoints"], None)),
        "scan_bwd": (scan_in + ("dout", "checkpoints"), scan_grads,
                     lambda at: L.ps_selective_scan_bwd(FAKE, big, scan(at), at["dout"], at["checkpoints"],
                                                        b._ScanGrads(**{k: at[k] for k in scan_grads}), None)),
        "scan_step": (scan_in[:8] + ("state", "slots"), ("out", "new_state"),
                      lambda at: L.ps_selective_scan_step(scan(dict(at, **off)), at["state"], at["new_state"], at["slots"], 100,
                                                          at["out"], None)),
        "norm": (norm_in, ("residual_out", "out"), lambda at: L.ps_block_norm(norm(at), at["residual_out"], at["out"], None)),
        "norm_bwd": (norm_in + ("dout", "dresidual_out"), norm_grads,
                     lambda at: L.ps_block_norm_bwd(FAKE, big, norm(at), at["dout"], at["dresidual_out"],
                                                    b._NormGrads(**{k: at[k] for k in norm_grads}), None)),
    }


@pytest.mark.parametrize("name", ["conv", "conv_bwd", "conv_step", "scan", "scan_bwd", "scan_step", "norm", "norm_bwd"])
def test_overlaps_are_refused(name):
    ins, outs, call = _alias_calls()[name]
    place = {n: _at(1 + i) for i, n in enumerate(ins + outs)}
    for o in outs:
        for other in ins + outs:
            if other != o:
                # 8 bytes into the other array: never the state itself
                assert call(dict(place, **{o: place[other] + 8})) == ALIAS, (o, other)
                assert call(dict(place, **{other: place[o] + 8})) == ALIAS, (o, other)


def test_structs_have_the_headers_layout(tmp_path):
    """sizeof and the last member's offset of every struct, C against ctypes."""
    b, _ = _mod()
    pairs = [("ps_conv_input", "dtype", b._ConvInput), ("ps_scan_input", "dtype", b._ScanInput),
             ("ps_scan_grads", "dinitial", b._ScanGrads), ("ps_norm_input", "eps", b._NormInput),
             ("ps_norm_grads", "dpre_weight", b._NormGrads)]
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include \"dwps.h\"\nint main(void) {\n" + "".join(
        '    printf("%%zu %%zu\\n", sizeof(%s), offsetof(%s, %s));\n' % (n, n, m) for n, m, _ in pairs) + "    return 0;\n}\n")
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-std=c99", "-I" + os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    lines = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split("\n")
    for line, (n, m, s) in zip(lines, pairs):
        assert line == "%d %d" % (ctypes.sizeof(s), getattr(s, m).offset), n


def test_binding_refuses_cpu_tensors():
    import device_wide_prefix_chained_amd as dw
    x, w = torch.zeros(4, 8), torch.zeros(8, 4)
    bc, a = torch.zeros(4, 1, 2), torch.zeros(8, 2)
    for call in (lambda: dw.ps_causal_conv(x, w), lambda: dw.ps_causal_conv_bwd(x, w, x),
                 lambda: dw.ps_causal_conv_step(x, torch.zeros(4, 3, 8), w), lambda: dw.ps_selective_scan(x, x, a, bc, bc),
                 lambda: dw.ps_selective_scan_step(x, torch.zeros(4, 8, 2), x, a, bc, bc), lambda: dw.ps_block_norm(x, x)):
        with pytest.raises(ValueError):
            call()


class _AsIfOnGpu(torch.Tensor):
    """A CPU tensor that the binding takes for one of the GPU's."""
    is_cuda = True


@pytest.mark.parametrize("wrong", [None, 3.0, [1.0, 2.0]], ids=str)
def test_binding_refuses_what_is_no_tensor(wrong):
    """In every place that the binding looks into before it checks it."""
    import device_wide_prefix_chained_amd as dw
    g = lambda *s: torch.zeros(*s).as_subclass(_AsIfOnGpu)  # noqa: E731
    x, w, a, bc, s = g(4, 8), g(8, 4), g(8, 2), g(4, 1, 2), g(4, 8, 2)
    for call in (lambda: dw.ps_causal_conv(x, wrong), lambda: dw.ps_causal_conv_bwd(x, wrong, x),
                 lambda: dw.ps_causal_conv_step(x, s, wrong), lambda: dw.ps_causal_conv_step(x, wrong, w),
                 lambda: dw.ps_selective_scan(x, x, wrong, bc, bc), lambda: dw.ps_selective_scan(x, x, a, wrong, bc),
                 lambda: dw.ps_selective_scan(x, x, a, bc, wrong), lambda: dw.ps_selective_scan(x, wrong, a, bc, bc),
                 lambda: dw.ps_selective_scan_bwd(x, x, wrong, bc, bc, x, s),
                 lambda: dw.ps_selective_scan_step(x, wrong, x, a, bc, bc),
                 lambda: dw.ps_selective_scan_step(x, s, x, a, wrong, bc),
                 lambda: dw.ps_block_norm(x, wrong), lambda: dw.ps_block_norm_bwd(x, wrong, x)):
        with pytest.raises(TypeError, match="must be a torch.Tensor"):
            call()


def test_binding_refuses_wrong_dimensions():
    import device_wide_prefix_chained_amd as dw
    g = lambda *s: torch.zeros(*s).as_subclass(_AsIfOnGpu)  # noqa: E731
    x, w, a, bc, s = g(4, 8), g(8, 4), g(8, 2), g(4, 1, 2), g(4, 8, 2)
    for call in (lambda: dw.ps_causal_conv(x, g(8)), lambda: dw.ps_causal_conv_step(x, g(()), w),
                 lambda: dw.ps_causal_conv_step(x, g(4), w), lambda: dw.ps_selective_scan(x, x, g(8), bc, bc),
                 lambda: dw.ps_selective_scan(x, x, a, g(4, 2), bc), lambda: dw.ps_selective_scan(x, x, a, bc, g(4, 2)),
                 lambda: dw.ps_selective_scan_step(x, g(()), x, a, bc, bc),
                 lambda: dw.ps_selective_scan_step(x, s[0], x, a, bc, bc), lambda: dw.ps_block_norm(x, g(()))):
        with pytest.raises(ValueError):
            call()


def test_a_captured_call_does_not_use_the_streams_workspace(monkeypatch):
    """The workspace kept for a stream is replaced when a larger call comes, so
    a graph must not hold it."""
    from device_wide_prefix_chained_amd import _binding as bind
    made = []

    def new(nbytes, device="cuda", stream=None):
        made.append(torch.zeros(int(nbytes), dtype=torch.uint8))
        return made[-1]
    monkeypatch.setattr(bind, "new_workspace", new)
    monkeypatch.setattr(bind, "_raw_stream", lambda t, stream: 7)
    monkeypatch.setattr(bind, "_torch_stream", lambda device, stream: None)
    monkeypatch.setattr(bind, "_WS_CACHE", {})
    capturing = [False]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])

    def call(need):
        def size(ws, have):
            have._obj.value = need
            return 0
        return bind._workspace("ps_scan", size, torch.zeros(1), None)[0]
    kept = call(1000)
    assert call(900) is kept
    capturing[0] = True
    first, second = call(1000), call(500)
    assert first is not kept and second is not kept and second is not first
    assert first.numel() >= 1000 and second.numel() >= 500
    capturing[0] = False
    assert call(1000) is kept

"""The gated delta rule and the layer norm on the CPU: the oracles' gradients
against differences, the chunks of packed sequences, and the refusals of the C
entry points and the binding (nothing is launched)."""
import ctypes
import os
import subprocess

import pytest
import torch

import delta_ref
import layer_ref
from test_block_cpu import (ALIAS, ALIGNMENT, FAKE, GB, NULL, ROOT, SIZE, UNSUPPORTED, WORKSPACE, _AsIfOnGpu, _at,
                            _differences, _mod, _run_model)


# ---------------------------------------------------------------------------
# oracles
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("normalize", [False, True])
def test_oracle_delta_gradients(normalize):
    """Of out and of final together, with heads that share keys."""
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    off = torch.tensor([0, 3, 3, 9])
    a = dict(q=r(9, 2, 3), k=0.5 * r(9, 2, 3), v=r(9, 4, 5), g=-r(9, 4).abs(), beta=torch.sigmoid(r(9, 4)),
             initial=r(3, 4, 3, 5))
    dout, dfinal = r(9, 4, 5), r(3, 4, 3, 5)
    got = delta_ref.delta(**a, normalize=normalize, offsets=off, dout=dout, dfinal=dfinal)[0]

    def both():
        v = delta_ref.delta(**a, normalize=normalize, offsets=off)[0]
        return torch.cat([v["out"].flatten(), v["final"].flatten()])
    for name in a:
        _differences(both, a[name], torch.cat([dout.flatten(), dfinal.flatten()]), got["d" + name])


def test_oracle_delta_is_the_rule_by_chunks():
    """The token by token oracle against the formulas of a chunk: (1 + a diag(beta))
    rho = V - e K S, out = scale e Q S + P U, S' = e_C S + K^T diag(exp(G_C - G)) U."""
    g = torch.Generator().manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    T, K, V = 20, 6, 4
    q, k, v, S = r(T, K), 0.4 * r(T, K), r(T, V), r(K, V)
    gate, beta = -r(T).abs(), torch.sigmoid(r(T))
    G = gate.cumsum(0)
    apart = torch.exp(G[:, None] - G[None, :])
    a = torch.tril(apart * (k @ k.t()), -1)
    P = 0.5 * torch.tril(apart * (q @ k.t()))
    e = torch.exp(G)[:, None]
    rho = torch.linalg.solve(torch.eye(T, dtype=torch.float64) + a * beta[None, :], v - e * (k @ S))
    U = beta[:, None] * rho
    out, final = 0.5 * e * (q @ S) + P @ U, e[-1] * S + k.t() @ (torch.exp(G[-1] - G)[:, None] * U)
    one = lambda t: t.unsqueeze(1)  # noqa: E731
    want = delta_ref.delta(one(q), one(k), one(v), one(gate), one(beta), scale=0.5, initial=S[None, None])[0]
    assert torch.allclose(want["out"][:, 0], out, rtol=1e-10, atol=1e-12)
    assert torch.allclose(want["final"][0, 0], final, rtol=1e-10, atol=1e-12)


def test_oracle_delta_step_is_a_sequence_of_one():
    g = torch.Generator().manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    a = (r(2, 1, 3), r(2, 1, 3), r(2, 2, 4))
    state, gate, beta = r(3, 2, 3, 4), -r(2, 2).abs(), torch.sigmoid(r(2, 2))
    got = delta_ref.delta_step(*a, state, gate, beta, slots=torch.tensor([2, 9]))[0]
    want = delta_ref.delta(*(t[:1] for t in a), gate[:1], beta[:1], initial=state[2:])[0]
    assert torch.equal(got["out"][0], want["out"][0]) and torch.equal(got["state"][2], want["final"][0])
    assert torch.equal(got["state"][:2], state[:2])
    empty = delta_ref.delta(*(t[1:] for t in a), gate[1:], beta[1:])[0]
    assert torch.equal(got["out"][1], empty["out"][0])


def test_oracle_layer_norm_gradients():
    g = torch.Generator().manual_seed(8)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    a = dict(x=r(4, 7), weight=r(7), bias=r(7))
    dout = r(4, 7)
    got = layer_ref.layer_norm(**a, dout=dout)
    for name in a:
        _differences(lambda: layer_ref.layer_norm(**a)["out"], a[name], dout, got["d" + name])
    want = torch.nn.functional.layer_norm(a["x"], (7,), a["weight"], a["bias"], 1e-5)
    assert torch.allclose(got["out"], want, rtol=1e-12, atol=1e-12)


def test_chunks(tmp_path):
    """Every row has one chunk and every chunk a number below the number of
    slots, for all offsets, those that break their contract too."""
    _run_model(tmp_path, "chunks_model")


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def _delta(b, **kw):
    a = dict(q=_at(1), k=_at(2), v=_at(3), q_stride=64, k_stride=64, v_stride=96, g=_at(4), beta=_at(5), g_stride=4,
             beta_stride=4, offsets=None, initial=None, tokens=100, kheads=2, heads=4, key_dim=32, value_dim=24,
             num_seqs=1, dtype=b.PS_BF16, normalize=1, scale=0.2, eps=1e-6)
    a.update(kw)
    return b._DeltaInput(**a)


def _dgrads(b, **kw):
    a = dict(dq=_at(20), dk=_at(21), dv=_at(22), dg=_at(23), dbeta=_at(24), dinitial=None)
    a.update(kw)
    return b._DeltaGrads(**a)


DELTA_BAD = [(dict(dtype=0), UNSUPPORTED), (dict(dtype=9), UNSUPPORTED), (dict(key_dim=0), SIZE),
             (dict(key_dim=257, q_stride=1 << 12, k_stride=1 << 12), SIZE), (dict(value_dim=0), SIZE),
             (dict(value_dim=257, v_stride=1 << 12), SIZE), (dict(kheads=0), SIZE), (dict(heads=0), SIZE),
             (dict(kheads=3, q_stride=96, k_stride=96), SIZE), (dict(kheads=8, q_stride=256, k_stride=256), SIZE),
             (dict(heads=65538, v_stride=1 << 21, g_stride=1 << 17, beta_stride=1 << 17), SIZE),
             (dict(tokens=1 << 31), SIZE), (dict(tokens=1 << 63), SIZE), (dict(num_seqs=2), SIZE),
             (dict(num_seqs=1 << 24, offsets=FAKE), SIZE), (dict(q_stride=63), SIZE), (dict(k_stride=63), SIZE),
             (dict(v_stride=95), SIZE), (dict(g_stride=3), SIZE), (dict(beta_stride=3), SIZE), (dict(q_stride=-64), SIZE),
             (dict(k_stride=(1 << 24) + 1), SIZE), (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL),
             (dict(g=None), NULL), (dict(beta=None), NULL), (dict(q=FAKE + 1), ALIGNMENT), (dict(k=FAKE + 1), ALIGNMENT),
             (dict(v=FAKE + 1), ALIGNMENT), (dict(g=FAKE + 2), ALIGNMENT), (dict(beta=FAKE + 2), ALIGNMENT),
             (dict(offsets=FAKE + 2), ALIGNMENT), (dict(initial=FAKE + 2), ALIGNMENT)]


@pytest.mark.parametrize("bad,code", DELTA_BAD)
def test_delta_refuses(bad, code):
    b, L = _mod()
    a, big = _delta(b, **bad), ctypes.c_size_t(GB)
    assert L.ps_gated_delta(FAKE, ctypes.byref(big), a, _at(10), None, None, None) == code
    assert L.ps_gated_delta_bwd(FAKE, ctypes.byref(big), a, _at(11), None, _at(12), _dgrads(b), None) == code
    if not {"num_seqs", "offsets", "initial"} & set(bad):
        assert L.ps_gated_delta_step(a, _at(10), _at(10), None, 100, _at(11), None) == code


def test_delta_refuses_more():
    b, L = _mod()
    big, small, a = ctypes.c_size_t(GB), ctypes.c_size_t(300), _delta(b)
    f, ref_big, ref_small = L.ps_gated_delta, ctypes.byref(big), ctypes.byref(small)
    assert f(FAKE, ref_big, None, _at(10), None, None, None) == NULL
    assert f(FAKE, None, a, _at(10), None, None, None) == NULL
    assert f(FAKE, ref_small, a, _at(10), None, None, None) == WORKSPACE
    assert f(FAKE + 8, ref_big, a, _at(10), None, None, None) == ALIGNMENT
    assert f(FAKE, ref_big, a, None, None, None, None) == NULL
    assert f(FAKE, ref_big, a, _at(10) + 1, None, None, None) == ALIGNMENT
    assert f(FAKE, ref_big, a, _at(10), _at(11) + 2, None, None) == ALIGNMENT
    assert f(FAKE, ref_big, a, _at(10), None, _at(11) + 2, None) == ALIGNMENT
    w = L.ps_gated_delta_bwd
    assert w(FAKE, ref_big, None, _at(11), None, _at(12), _dgrads(b), None) == NULL
    assert w(FAKE, ref_small, a, _at(11), None, _at(12), _dgrads(b), None) == WORKSPACE
    assert w(FAKE, ref_big, a, None, None, _at(12), _dgrads(b), None) == NULL
    assert w(FAKE, ref_big, a, _at(11), None, None, _dgrads(b), None) == NULL
    assert w(FAKE, ref_big, a, _at(11), None, _at(12), None, None) == NULL
    for name in ("dq", "dk", "dv", "dg", "dbeta"):
        assert w(FAKE, ref_big, a, _at(11), None, _at(12), _dgrads(b, **{name: None}), None) == NULL
        assert w(FAKE, ref_big, a, _at(11), None, _at(12), _dgrads(b, **{name: _at(20) + 1}), None) == ALIGNMENT
    assert w(FAKE, ref_big, a, _at(11), None, _at(12), _dgrads(b, dinitial=_at(20) + 2), None) == ALIGNMENT
    assert w(FAKE, ref_big, a, _at(11) + 1, None, _at(12), _dgrads(b), None) == ALIGNMENT
    assert w(FAKE, ref_big, a, _at(11), _at(13) + 2, _at(12), _dgrads(b), None) == ALIGNMENT
    st = L.ps_gated_delta_step
    assert st(None, _at(10), _at(10), None, 100, _at(11), None) == NULL
    assert st(a, _at(10), _at(10), None, 99, _at(11), None) == SIZE  # no slots, pool too small
    assert st(a, _at(10), _at(10) + 4096, None, 100, _at(11), None) == ALIAS  # not the state itself
    assert st(a, None, _at(12), None, 100, _at(11), None) == NULL
    assert st(a, _at(10), None, None, 100, _at(11), None) == NULL
    assert st(a, _at(10), _at(10), None, 100, None, None) == NULL
    assert st(a, _at(10) + 2, _at(10) + 2, None, 100, _at(11), None) == ALIGNMENT
    assert st(a, _at(10), _at(10), FAKE + 2, 100, _at(11), None) == ALIGNMENT
    assert st(a, _at(10), _at(10), None, 100, _at(11) + 1, None) == ALIGNMENT
    none = dict(q=None, k=None, v=None, g=None, beta=None)
    assert st(_delta(b, tokens=0, **none), None, None, None, 0, None, None) == 0
    # the size queries look at no pointer
    need = ctypes.c_size_t(0)
    assert f(None, ctypes.byref(need), _delta(b, **none), None, None, None, None) == 0 and need.value > 256
    assert w(None, ctypes.byref(need), _delta(b, **none), None, None, None, None, None) == 0 and need.value > 256


def test_delta_sizes_that_a_launch_does_not_count():
    """Chunks times heads are numbered in 31 bits; rows and states in 64."""
    b, L = _mod()
    need = ctypes.c_size_t(0)

    def query(**kw):
        wide = dict(q_stride=1 << 20, k_stride=1 << 20, v_stride=1 << 24, g_stride=1 << 16, beta_stride=1 << 16)
        return L.ps_gated_delta(None, ctypes.byref(need), _delta(b, **dict(wide, **kw)), None, None, None, None)
    # (tokens / 64 + 1) * heads against 2^31
    most = ((1 << 31) // 16 - 1) * 64
    assert query(tokens=(1 << 31) - 1, heads=32, kheads=32, key_dim=16, value_dim=16) == 0 and need.value > 1 << 40
    assert query(tokens=(1 << 31) - 1, heads=64, kheads=32, key_dim=16, value_dim=16) == SIZE
    assert query(tokens=(1 << 31) - 64, heads=64, kheads=32, key_dim=16, value_dim=16) == SIZE
    assert most > 1 << 31  # 16 heads and fewer: the tokens' own limit
    one = lambda t, h: L.ps_gated_delta_step(  # noqa: E731
        _delta(b, tokens=t, heads=h, kheads=1, key_dim=1, value_dim=1, q_stride=1, k_stride=1, v_stride=1 << 16,
               g_stride=1 << 16, beta_stride=1 << 16), None, None, FAKE, 0, None, None)
    assert one(1 << 15, 1 << 16) == SIZE and one((1 << 15) - 1, 1 << 16) == NULL


def test_delta_checkpoint_floats():
    import device_wide_prefix_chained_amd as dw
    n = dw.ps_gated_delta_checkpoint_floats
    # a state, a chunk's corrections and 32 sizes for each of (tokens >> 6) + num_seqs numbers, or none
    each = 2 * ((16 + 64) * 8 + 32)
    assert [n(t, 1, 2, 16, 8) for t in (0, 1, 64, 65, 1 << 20)] == [each * c for c in (1, 1, 2, 2, (1 << 14) + 1)]
    assert n(100, 5, 2, 16, 8) == each * 6
    assert n((1 << 31) - 1, 1, 16, 256, 256) == (1 << 25) * 16 * (320 * 256 + 32)


def _layer(b, **kw):
    a = dict(x=_at(1), x_stride=64, weight=_at(2), bias=_at(3), tokens=100, channels=64, dtype=b.PS_BF16, eps=1e-5)
    a.update(kw)
    return b._LayerInput(**a)


LAYER_BAD = [(dict(dtype=0), UNSUPPORTED), (dict(dtype=7), UNSUPPORTED), (dict(channels=0), SIZE),
             (dict(channels=16385, x_stride=1 << 15), SIZE), (dict(x_stride=63), SIZE), (dict(x_stride=-64), SIZE),
             (dict(x_stride=(1 << 24) + 1), SIZE), (dict(tokens=1 << 31), SIZE), (dict(x=None), NULL),
             (dict(x=FAKE + 1), ALIGNMENT), (dict(weight=FAKE + 2), ALIGNMENT), (dict(bias=FAKE + 2), ALIGNMENT)]


@pytest.mark.parametrize("bad,code", LAYER_BAD)
def test_layer_norm_refuses(bad, code):
    b, L = _mod()
    a, big = _layer(b, **bad), ctypes.c_size_t(GB)
    assert L.ps_layer_norm(a, _at(10), None) == code
    assert L.ps_layer_norm_bwd(FAKE, ctypes.byref(big), a, _at(11), _at(12), _at(13), _at(14), None) == code


def test_layer_norm_refuses_more():
    b, L = _mod()
    big, small, a = ctypes.c_size_t(GB), ctypes.c_size_t(300), _layer(b)
    assert L.ps_layer_norm(None, _at(10), None) == NULL
    assert L.ps_layer_norm(a, None, None) == NULL
    assert L.ps_layer_norm(a, _at(10) + 1, None) == ALIGNMENT
    assert L.ps_layer_norm(_layer(b, tokens=0, x=None), None, None) == 0
    w, r = L.ps_layer_norm_bwd, ctypes.byref(big)
    assert w(FAKE, r, None, _at(11), _at(12), None, None, None) == NULL
    assert w(FAKE, None, a, _at(11), _at(12), None, None, None) == NULL
    assert w(FAKE, ctypes.byref(small), a, _at(11), _at(12), None, None, None) == WORKSPACE
    assert w(FAKE, r, a, None, _at(12), None, None, None) == NULL
    assert w(FAKE, r, a, _at(11), None, None, None, None) == NULL
    assert w(FAKE + 8, r, a, _at(11), _at(12), None, None, None) == ALIGNMENT
    for bad in ((_at(11) + 1, _at(12), _at(13), _at(14)), (_at(11), _at(12) + 1, _at(13), _at(14)),
                (_at(11), _at(12), _at(13) + 2, _at(14)), (_at(11), _at(12), _at(13), _at(14) + 2)):
        assert w(FAKE, r, a, *bad, None) == ALIGNMENT
    need = ctypes.c_size_t(0)
    assert w(None, ctypes.byref(need), _layer(b, x=None), None, None, None, None, None) == 0 and need.value > 256


# Every output of an entry point laid over every input and every other output.
def _alias_calls():
    b, L = _mod()
    big = ctypes.byref(ctypes.c_size_t(GB))
    keys = ("q", "k", "v", "g", "beta")
    packed = keys + ("offsets", "initial")
    grads = ("dq", "dk", "dv", "dg", "dbeta", "dinitial")

    def delta(at, names):
        return _delta(b, **{n: at[n] for n in names}, num_seqs=3 if "offsets" in names else 1)

    def layer(at):
        return _layer(b, **{n: at[n] for n in ("x", "weight", "bias")})
    return {
        "delta": (packed, ("out", "final", "checkpoints"),
                  lambda at: L.ps_gated_delta(FAKE, big, delta(at, packed), at["out"], at["final"], at["checkpoints"], None)),
        "delta_bwd": (packed + ("dout", "dfinal", "checkpoints"), grads,
                      lambda at: L.ps_gated_delta_bwd(FAKE, big, delta(at, packed), at["dout"], at["dfinal"], at["checkpoints"],
                                                      b._DeltaGrads(**{n: at[n] for n in grads}), None)),
        "delta_step": (keys + ("state", "slots"), ("out", "new_state"),
                       lambda at: L.ps_gated_delta_step(delta(at, keys), at["state"], at["new_state"], at["slots"], 100,
                                                        at["out"], None)),
        "layer": (("x", "weight", "bias"), ("out",), lambda at: L.ps_layer_norm(layer(at), at["out"], None)),
        "layer_bwd": (("x", "weight", "bias", "dout"), ("dx", "dweight", "dbias"),
                      lambda at: L.ps_layer_norm_bwd(FAKE, big, layer(at), at["dout"], at["dx"], at["dweight"], at["dbias"],
                                                     None)),
    }


@pytest.mark.parametrize("name", ["delta", "delta_bwd", "delta_step", "layer", "layer_bwd"])
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
    b, _ = _mod()
    src = tmp_path / "layout.c"
    pairs = [("ps_delta_input", b._DeltaInput), ("ps_delta_grads", b._DeltaGrads), ("ps_layer_input", b._LayerInput)]
    src.write_text("#include <stdio.h>\n#include \"dwps.h\"\nint main(void) {\n" + "".join(
        '    printf("%%zu\\n", sizeof(%s));\n' % n + "".join(
            '    printf("%%zu\\n", offsetof(%s, %s));\n' % (n, m) for m, _ in s._fields_) for n, s in pairs) +
        "    return 0;\n}\n")
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-std=c99", "-I" + os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for _, s in pairs:
        want += [ctypes.sizeof(s)] + [getattr(s, m).offset for m, _ in s._fields_]
    assert got == want


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
def _calls(dw, q, v, g, state, x):
    floats = torch.zeros(1)
    return (lambda: dw.ps_gated_delta(q, q, v, g, g), lambda: dw.ps_gated_delta_bwd(q, q, v, g, g, v, floats),
            lambda: dw.ps_gated_delta_step(q, q, v, state, g, g), lambda: dw.ps_layer_norm(x),
            lambda: dw.ps_layer_norm_bwd(x, x))


def test_binding_refuses_cpu_tensors():
    import device_wide_prefix_chained_amd as dw
    for call in _calls(dw, torch.zeros(4, 1, 8), torch.zeros(4, 2, 6), torch.zeros(4, 2), torch.zeros(4, 2, 8, 6),
                       torch.zeros(4, 8)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("wrong", [None, 3.0, [1.0, 2.0]], ids=str)
def test_binding_refuses_what_is_no_tensor(wrong):
    """In every place that the binding looks into before it checks it."""
    import device_wide_prefix_chained_amd as dw
    g = lambda *s: torch.zeros(*s).as_subclass(_AsIfOnGpu)  # noqa: E731
    q, v, a, s, x = g(4, 1, 8), g(4, 2, 6), g(4, 2), g(4, 2, 8, 6), g(4, 8)
    kept = g(dw.ps_gated_delta_checkpoint_floats(4, 1, 2, 8, 6))
    for i in range(5):
        args = [q, q, v, a, a]
        args[i] = wrong
        for call in (lambda: dw.ps_gated_delta(*args), lambda: dw.ps_gated_delta_bwd(*args, v, kept),
                     lambda: dw.ps_gated_delta_step(*args[:3], s, *args[3:])):
            with pytest.raises(TypeError, match="must be a torch.Tensor"):
                call()
    calls = [lambda: dw.ps_gated_delta_step(q, q, v, wrong, a, a), lambda: dw.ps_layer_norm(wrong),
             lambda: dw.ps_layer_norm_bwd(wrong, x)]
    if wrong is not None:  # None is a null pointer, which the C entry refuses
        calls += [lambda: dw.ps_gated_delta_bwd(q, q, v, a, a, wrong, kept), lambda: dw.ps_layer_norm_bwd(x, wrong)]
    for call in calls:
        with pytest.raises(TypeError, match="must be a torch.Tensor"):
            call()


def test_binding_refuses_wrong_dimensions():
    import device_wide_prefix_chained_amd as dw
    g = lambda *s: torch.zeros(*s).as_subclass(_AsIfOnGpu)  # noqa: E731
    q, v, a, s, x = g(4, 1, 8), g(4, 2, 6), g(4, 2), g(4, 2, 8, 6), g(4, 8)
    for call in (lambda: dw.ps_gated_delta(q[0], q, v, a, a), lambda: dw.ps_gated_delta(q, q[0], v, a, a),
                 lambda: dw.ps_gated_delta(q, q, v[0], a, a), lambda: dw.ps_gated_delta(q, q, v, a[0], a),
                 lambda: dw.ps_gated_delta(q, q, v, a, g(())), lambda: dw.ps_gated_delta(g(()), q, v, a, a),
                 lambda: dw.ps_gated_delta(q, g(4, 1, 9), v, a, a), lambda: dw.ps_gated_delta(q, q, v[:3], a, a),
                 lambda: dw.ps_gated_delta(q, q, v, g(4, 3), a), lambda: dw.ps_gated_delta_step(q, q, v, g(()), a, a),
                 lambda: dw.ps_gated_delta_step(q, q, v, s[0], a, a), lambda: dw.ps_layer_norm(x[0]),
                 lambda: dw.ps_layer_norm(g(())), lambda: dw.ps_layer_norm_bwd(x, x[:3])):
        with pytest.raises(ValueError):
            call()

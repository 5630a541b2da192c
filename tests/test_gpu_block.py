"""Parity of the state space block's operators (HIP, through the binding) with
their formulas in 64 bits (block_ref): causal convolution, selective scan and
the norms around a block, forwards, backwards and for single tokens.

Tolerances: half a step of the result's type, and for the fp32 arithmetic
2^-24 times the number of roundings on a term's way times the sum of the
terms' magnitudes (block_ref.close)."""
import pytest
import torch

import block_ref as ref
import scan_bound
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def dw():
    return require_gpu()


class Maker:
    """Inputs on the GPU from a seed; `wide` makes rows strided (a slice of a
    wider array, at an odd column)."""

    def __init__(self, seed, dtype, wide=False):
        self.g = torch.Generator().manual_seed(seed)
        self.dtype, self.wide = dtype, wide

    def act(self, *shape, scale=1.0, mean=0.0, packed=False, dtype=None):
        v = (torch.randn(*shape, generator=self.g) * scale + mean).to(self.dtype if dtype is None else dtype).cuda()
        if not self.wide or packed:
            return v
        row = 1
        for n in shape[1:]:
            row *= n
        big = torch.full((shape[0], row + 13), float("nan"), dtype=v.dtype, device="cuda")
        big[:, 3:3 + row] = v.reshape(shape[0], row)
        return big[:, 3:3 + row].unflatten(1, shape[1:]) if len(shape) > 2 else big[:, 3:3 + row]

    def par(self, *shape, scale=1.0, mean=0.0):
        return (torch.randn(*shape, generator=self.g) * scale + mean).cuda()


def _offsets(cuts):
    return None if cuts is None else torch.tensor(cuts, dtype=torch.int32, device="cuda")


def _finite_rows(cuts, tokens):
    return slice(0, tokens) if cuts is None else slice(cuts[0], cuts[-1])


# ---------------------------------------------------------------------------
# causal convolution
# ---------------------------------------------------------------------------
CONV = [  # tokens, cuts, channels, width, type, initial, bias, strided
    (1, None, 1, 4, F32, False, True, False),
    (0, [0, 0], 8, 3, BF16, True, True, False),
    (70, None, 8, 1, F32, False, False, False),
    (70, [0, 1, 1, 3, 40, 70], 24, 4, BF16, True, True, False),
    (70, [0, 1, 1, 3, 40, 70], 37, 3, F16, True, True, True),
    (97, [0, 31, 32, 33, 64, 96, 97], 130, 2, F32, True, False, True),
    (200, [5, 60, 60, 190], 515, 5, BF16, False, True, False),
    (64, [0, 64], 513, 8, F16, True, True, True),
    (333, [0, 333], 1024, 4, BF16, False, True, False),
    (50, list(range(51)), 40, 4, F32, True, True, False),
]


@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv(dw, case):
    T, cuts, ch, W, dtype, initial, bias, wide = case
    say("conv", case)
    m = Maker(T + ch, dtype, wide)
    off = _offsets(cuts)
    seqs = 1 if cuts is None else len(cuts) - 1
    x, w = m.act(T, ch), m.par(ch, W, scale=0.5)
    b = m.par(ch, scale=0.3) if bias else None
    init = m.act(seqs, W - 1, ch, packed=True) if initial else None
    dout = m.act(T, ch, packed=True)
    out = torch.full((T, ch), 7.0, dtype=dtype, device="cuda")
    final = torch.full((seqs, W - 1, ch), 7.0, dtype=dtype, device="cuda")
    dw.ps_causal_conv(x, w, b, offsets=off, initial=init, out=out, final=final)
    g = dw.ps_causal_conv_bwd(x, w, dout, b, offsets=off, initial=init)
    torch.cuda.synchronize()
    want = ref.conv(x, w, b, off, init, dout)
    mag = ref.conv(x, w, b, off, init, dout, bound=True)
    rows, K = _finite_rows(cuts, T), 2 * W + 64
    ref.close("out", out[rows], want["out"][rows], mag["out"][rows], K)
    assert torch.equal(ref.f64(final), want["final"])
    outside = torch.ones(T, dtype=torch.bool)
    outside[rows] = False
    assert (out.cpu()[outside] == 7.0).all()
    K += T
    ref.close("dx", g.dx[rows], want["dx"][rows], mag["dx"][rows], K)
    ref.close("dweight", g.dweight, want["dweight"], mag["dweight"], K)
    assert (g.dbias is None) == (b is None) and (g.dinitial is None) == (init is None)
    if bias:
        ref.close("dbias", g.dbias, want["dbias"], mag["dbias"], K)
    if initial:
        ref.close("dinitial", g.dinitial, want["dinitial"], mag["dinitial"], K)


@pytest.mark.parametrize("case", [(1, 1, 8, 4, BF16, False, False), (7, 9, 40, 3, F32, True, True),
                                  (33, 40, 515, 4, F16, True, False), (5, 5, 130, 1, F32, True, False)], ids=str)
def test_conv_step(dw, case):
    batch, pool, ch, W, dtype, use_slots, wide = case
    say("conv step", case)
    m = Maker(batch + ch, dtype, wide)
    x, w, b = m.act(batch, ch), m.par(ch, W, scale=0.5), m.par(ch, scale=0.3)
    state = m.act(pool, W - 1, ch, packed=True)
    slots = torch.randperm(pool, generator=m.g)[:batch].to(torch.int32)
    if use_slots and batch > 4:
        slots[2], slots[4] = -1, pool  # padding of the batch
    slots = slots.cuda() if use_slots else None
    want, mag = (ref.conv_step(x, state, w, b, slots, bound=v) for v in (False, True))
    new = state.clone()
    out = dw.ps_causal_conv_step(x, state, w, b, slots=slots, new_state=new)
    ref.close("out", out, want["out"], mag["out"], 2 * W + 64)
    assert torch.equal(ref.f64(new), want["state"])
    again = dw.ps_causal_conv_step(x, state, w, b, slots=slots)  # in place
    assert torch.equal(again, out) and torch.equal(state, new)


# ---------------------------------------------------------------------------
# selective scan
# ---------------------------------------------------------------------------
SCAN = [  # tokens, cuts, channels, groups, states, type, initial, optional inputs, strided
    (1, None, 1, 1, 1, F32, False, "", False),
    (0, [0, 0, 0], 16, 1, 16, BF16, True, "Dzb", False),
    (33, None, 16, 1, 16, F32, False, "Dzb", False),
    (32, [0, 32], 20, 1, 16, BF16, True, "zb", False),
    (70, [0, 1, 1, 3, 40, 70], 40, 2, 16, BF16, True, "Dzb", True),
    (70, [0, 1, 1, 3, 40, 70], 33, 1, 4, F16, True, "Dz", False),
    (130, [0, 31, 32, 33, 64, 96, 96, 130], 36, 4, 24, F32, True, "Dzb", True),
    (100, [7, 50, 50, 95], 18, 1, 64, F16, False, "b", False),
    (64, None, 17, 1, 17, BF16, False, "D", True),
    (40, [0, 23, 40], 5, 1, 256, F32, True, "Dzb", False),
    (50, list(range(51)), 24, 2, 8, F32, True, "Dzb", False),
    (700, [0, 650, 700], 64, 1, 16, BF16, True, "Dzb", False),
    (900, None, 80, 1, 16, F32, False, "Dzb", False),
    # few channels and long sequences: cells of sequences side by side
    (2500, None, 16, 1, 16, F32, True, "Dzb", False),
    (3001, [0, 2, 1500, 1500, 1531, 3001], 20, 1, 24, BF16, True, "Dzb", True),
    (4096, [0, 4096], 24, 2, 4, F16, False, "z", False),
]


def _scan_inputs(m, T, ch, G, N, seqs, initial, extra):
    a = dict(x=m.act(T, ch), dt=m.act(T, ch), A=-m.par(ch, N).abs() * 2 - 0.01, B=m.act(T, G, N), C=m.act(T, G, N))
    more = dict(D=m.par(ch) if "D" in extra else None, z=m.act(T, ch) if "z" in extra else None,
                dt_bias=m.par(ch, mean=-2.0) if "b" in extra else None)
    if initial:
        more["initial"] = m.par(seqs, ch, N)
    return a, more


@pytest.mark.parametrize("case", SCAN, ids=str)
def test_scan(dw, case):
    T, cuts, ch, G, N, dtype, initial, extra, wide = case
    say("scan", case)
    m = Maker(T + ch + N, dtype, wide)
    off = _offsets(cuts)
    seqs = 1 if cuts is None else len(cuts) - 1
    a, more = _scan_inputs(m, T, ch, G, N, seqs, initial, extra)
    dout = m.act(T, ch, packed=True)
    out = torch.full((T, ch), 7.0, dtype=dtype, device="cuda")
    final = torch.full((seqs, ch, N), 7.0, device="cuda")
    kept = torch.full((dw.ps_selective_scan_checkpoint_rows(T, N), ch, N), float("nan"), device="cuda")
    dw.ps_selective_scan(**a, **more, offsets=off, out=out, final=final, checkpoints=kept)
    want = ref.scan(**a, **more, offsets=off, dout=dout)
    mag = ref.scan(**a, **more, offsets=off, dout=dout, bound=True)
    K = ref.scan_roundings(a["dt"], a["A"], more["dt_bias"], T, ch, N)
    rows = _finite_rows(cuts, T)
    ref.close("out", out[rows], want["out"][rows], mag["out"][rows], K)
    ref.close("final", final, want["final"], mag["final"], K)
    outside = torch.ones(T, dtype=torch.bool)
    outside[rows] = False
    assert (out.cpu()[outside] == 7.0).all()
    say("scan backwards", case)
    g = dw.ps_selective_scan_bwd(*a.values(), dout, kept, **more, offsets=off)
    for name in ("dx", "ddt", "dz", "dB", "dC"):
        if name != "dz" or "z" in extra:
            ref.close(name, getattr(g, name)[rows], want[name][rows], mag[name][rows], K)
    ref.close("dA", g.dA, want["dA"], mag["dA"], K)
    for name, there in (("dD", "D" in extra), ("ddt_bias", "b" in extra), ("dinitial", initial), ("dz", "z" in extra)):
        assert (getattr(g, name) is not None) == there
        if there and name != "dz":
            ref.close(name, getattr(g, name), want[name], mag[name], K)


# Groups of whole blocks of 16 channels.  Numbers of states that are a multiple
# of 16 and no power of two leave places of a lane without a state; those that
# are 16 times a power of two run the kernels without bounds.  The strided
# cases' rows lie between NaN, so a state past the last shows.
SCAN_WHOLE = [  # as SCAN
    (100, [0, 1, 1, 40, 100], 32, 1, 48, BF16, True, "Dzb", True),
    (100, None, 64, 2, 80, F32, True, "Dzb", True),
    (97, [0, 31, 32, 97], 64, 2, 96, F16, False, "Dz", False),
    (100, [0, 65, 100], 16, 1, 112, F32, True, "b", True),
    (70, [0, 33, 33, 70], 32, 2, 144, F32, False, "Dzb", False),
    (70, [0, 33, 70], 32, 2, 240, BF16, True, "Dzb", True),
    (70, [5, 33, 66], 16, 1, 240, F32, True, "zb", True),
    (100, [0, 1, 1, 40, 100], 64, 2, 16, F32, True, "Dzb", True),
    (100, [0, 1, 1, 40, 100], 64, 4, 32, F32, True, "Dzb", True),
    (130, [0, 31, 32, 96, 96, 130], 128, 2, 64, BF16, True, "Dzb", True),
    (70, [0, 33, 70], 64, 4, 128, F32, True, "Dzb", False),
    (70, None, 32, 2, 256, F16, True, "Dzb", True),
    # cells of sequences side by side
    (2500, [0, 2, 1500, 1500, 2500], 16, 1, 48, F32, True, "Dzb", True),
    (2500, None, 32, 2, 80, BF16, False, "Dzb", True),
    (2500, [0, 2, 1500, 1500, 2500], 32, 2, 16, F32, True, "Dzb", True),
    (2500, None, 32, 2, 32, BF16, True, "zb", True),
    (2500, [0, 700, 2500], 16, 1, 64, F32, True, "Dzb", True),
    (2500, [0, 700, 2500], 16, 1, 128, F16, True, "Dzb", False),
]


@pytest.mark.parametrize("case", SCAN_WHOLE, ids=str)
def test_scan_whole_channel_blocks(dw, case):
    """Every result against 64 bits, within a bound carried along with the
    values (scan_bound)."""
    T, cuts, ch, G, N, dtype, initial, extra, wide = case
    say("scan, whole channel blocks", case)
    m = Maker(T + ch + N, dtype, wide)
    off = _offsets(cuts)
    seqs = 1 if cuts is None else len(cuts) - 1
    a, more = _scan_inputs(m, T, ch, G, N, seqs, initial, extra)
    dout = m.act(T, ch, packed=True)
    out = torch.full((T, ch), 7.0, dtype=dtype, device="cuda")
    final = torch.full((seqs, ch, N), 7.0, device="cuda")
    kept = torch.full((dw.ps_selective_scan_checkpoint_rows(T, N), ch, N), float("nan"), device="cuda")
    dw.ps_selective_scan(**a, **more, offsets=off, out=out, final=final, checkpoints=kept)
    g = dw.ps_selective_scan_bwd(*a.values(), dout, kept, **more, offsets=off)
    torch.cuda.synchronize()
    want, bound = scan_bound.scan(**a, **more, offsets=off, dout=dout)
    rows = _finite_rows(cuts, T)
    outside = torch.ones(T, dtype=torch.bool)
    outside[rows] = False
    assert (out.cpu()[outside] == 7.0).all()
    scan_bound.close("out", out[rows], want["out"][rows], bound["out"][rows])
    scan_bound.close("final", final, want["final"], bound["final"])
    for name in g._fields:
        got, by_row = getattr(g, name), name in ("dx", "ddt", "dz", "dB", "dC")
        given = {"dD": "D" in extra, "dz": "z" in extra, "ddt_bias": "b" in extra, "dinitial": initial}
        assert (got is not None) == given.get(name, True)
        if got is None:
            continue
        if by_row:
            scan_bound.close(name, got[rows], want[name][rows], bound[name][rows])
        else:
            scan_bound.close(name, got, want[name], bound[name])


@pytest.mark.parametrize("case", [(1, 1, 16, 1, 16, BF16, False, False), (7, 9, 40, 2, 24, F32, True, True),
                                  (33, 40, 130, 1, 4, F16, True, False), (5, 5, 66, 1, 64, BF16, True, False),
                                  (6, 8, 9, 3, 7, F32, True, True), (5, 6, 3, 1, 256, F32, False, False)], ids=str)
def test_scan_step(dw, case):
    batch, pool, ch, G, N, dtype, use_slots, wide = case
    say("scan step", case)
    m = Maker(batch + ch + N, dtype, wide)
    a, more = _scan_inputs(m, batch, ch, G, N, 0, False, "Dzb")
    state = m.par(pool, ch, N)
    slots = torch.randperm(pool, generator=m.g)[:batch].to(torch.int32)
    if use_slots and batch > 4:
        slots[2], slots[4] = -1, pool  # padding of the batch
    slots = slots.cuda() if use_slots else None
    x = a.pop("x")
    want, mag = (ref.scan_step(x, state, **a, **more, slots=slots, bound=v) for v in (False, True))
    K = ref.scan_roundings(a["dt"], a["A"], more["dt_bias"], 1, 1, N)
    new = state.clone()
    out = dw.ps_selective_scan_step(x, state, **a, **more, slots=slots, new_state=new)
    ref.close("out", out, want["out"], mag["out"], K)
    ref.close("state", new, want["state"], mag["state"], K)
    again = dw.ps_selective_scan_step(x, state, **a, **more, slots=slots)  # in place
    assert torch.equal(again, out) and torch.equal(state, new)


def test_steps_go_on_from_a_prompt(dw):
    """A prompt in one call equals a part of it, then single tokens: the same
    states within rounding, for the convolution and the scan."""
    m = Maker(5, F32)
    T, cut, ch, N, W = 45, 38, 48, 16, 4
    a, more = _scan_inputs(m, T, ch, 1, N, 1, False, "Dzb")
    w, b = m.par(ch, W, scale=0.5), m.par(ch)
    say("steps after a prompt")
    whole_c = dw.ps_causal_conv(a["x"], w, b)
    rows = torch.empty(1, W - 1, ch, device="cuda")
    part = dw.ps_causal_conv(a["x"][:cut], w, b, final=rows)
    steps = [dw.ps_causal_conv_step(a["x"][t:t + 1], rows, w, b) for t in range(cut, T)]
    assert torch.equal(torch.cat([part, *steps]), whole_c)
    final, state = torch.empty(1, ch, N, device="cuda"), torch.empty(1, ch, N, device="cuda")
    whole = dw.ps_selective_scan(**a, **more, final=final)
    at = lambda d, r: {k: v[r] if v is not None and v.shape[0] == T and k not in ("A", "D", "dt_bias") else v  # noqa: E731
                       for k, v in d.items()}
    part = dw.ps_selective_scan(**at(a, slice(0, cut)), **at(more, slice(0, cut)), final=state)
    steps = []
    for t in range(cut, T):
        s = at(a, slice(t, t + 1))
        x = s.pop("x")
        steps.append(dw.ps_selective_scan_step(x, state, **s, **at(more, slice(t, t + 1))))
    mag = ref.scan(**a, **more, bound=True)
    K = 2 * ref.scan_roundings(a["dt"], a["A"], more["dt_bias"], T, ch, N)
    ref.close("out", torch.cat([part, *steps]), ref.f64(whole), mag["out"], K)
    ref.close("state", state, ref.f64(final), mag["final"], K)


def test_sequences_do_not_touch(dw):
    """NaN, infinities and the lowest values in one sequence leave the bits of
    the others as they were."""
    m = Maker(6, F32)
    T, ch, N, cuts = 80, 24, 16, [0, 21, 45, 80]
    a, more = _scan_inputs(m, T, ch, 1, N, 3, True, "Dzb")
    w, b = m.par(ch, 4, scale=0.5), m.par(ch)
    off, dout = _offsets(cuts), m.act(T, ch)
    rows = [t for t in range(T) if not 21 <= t < 45]

    def run():
        kept = torch.empty(dw.ps_selective_scan_checkpoint_rows(T, N), ch, N, device="cuda")
        o = dw.ps_selective_scan(**a, **more, offsets=off, checkpoints=kept)
        g = dw.ps_selective_scan_bwd(*a.values(), dout, kept, **more, offsets=off)
        c = dw.ps_causal_conv(a["x"], w, b, offsets=off)
        cg = dw.ps_causal_conv_bwd(a["x"], w, dout, b, offsets=off)
        return [t[rows].clone() for t in (o, g.dx, g.ddt, g.dz, g.dB, g.dC, c, cg.dx)]
    say("sequences apart")
    before = run()
    low = torch.finfo(F32).min
    for i, v in enumerate((float("nan"), float("inf"), float("-inf"), low)):
        a["x"][21 + i], a["dt"][25 + i], a["B"][29 + i], a["C"][33 + i] = v, v, v, v
        more["z"][37 + i], dout[40 + i] = v, v
    more["initial"][1] = float("nan")
    for x, y in zip(before, run()):
        assert torch.equal(x, y)


def test_offsets_out_of_contract_stay_in_bounds(dw):
    """Offsets that go down or past the rows: no promise on the values, but
    memory beside the results stays as it is (the pieces themselves are
    checked on the CPU)."""
    m = Maker(7, F32)
    T, ch, N = 75, 20, 16
    a, more = _scan_inputs(m, T, ch, 1, N, 3, True, "Dzb")
    big = torch.full((T + 20, ch), 7.0, device="cuda")
    for cuts in ([60, 10, 2000000000, 5], [0, -1, -5, 75], [90, 90, 90, 90]):
        say("offsets", cuts)
        off = _offsets(cuts)
        kept = torch.zeros(dw.ps_selective_scan_checkpoint_rows(T, N), ch, N, device="cuda")
        out = dw.ps_selective_scan(**a, **more, offsets=off, out=big[10:10 + T], checkpoints=kept)
        dw.ps_selective_scan_bwd(*a.values(), m.act(T, ch), kept, **more, offsets=off)
        dw.ps_causal_conv(a["x"], m.par(ch, 4), offsets=off, out=out)
        dw.ps_causal_conv_bwd(a["x"], m.par(ch, 4), m.act(T, ch), offsets=off)
        torch.cuda.synchronize()
        assert (big[:10] == 7.0).all() and (big[10 + T:] == 7.0).all()


# ---------------------------------------------------------------------------
# norms around a block
# ---------------------------------------------------------------------------
NORM = [  # tokens, channels, type, residual type, optional inputs, strided
    (1, 1, F32, F32, "gsop", False),
    (3, 40, BF16, BF16, "gsop", False),
    (5, 515, F16, F32, "gsop", True),
    (9, 512, BF16, F32, "so", False),
    (700, 513, F32, F32, "gp", False),
    (6, 2048, BF16, BF16, "", True),
    (4, 4099, F16, F16, "gsop", True),
    (3, 5120, BF16, F32, "gsop", False),
    (3, 9000, F32, F32, "gsop", False),
    (2, 16384, BF16, BF16, "gsop", False),
    (2, 12289, BF16, F32, "gsop", True),
]


@pytest.mark.parametrize("case", NORM, ids=str)
def test_norm(dw, case):
    T, ch, dtype, rt, extra, wide = case
    say("norm", case)
    m = Maker(T + ch, dtype, wide)
    y, res = m.act(T, ch), m.act(T, ch, scale=2.0, dtype=rt)
    kw = dict(gate=m.act(T, ch) if "g" in extra else None, scale=m.par(ch, mean=0.5) if "s" in extra else None,
              post_weight=m.par(ch, mean=1.0) if "o" in extra else None,
              pre_weight=m.par(ch, mean=1.0) if "p" in extra else None)
    if T > 2:
        y[1] = 0.0  # a row with nothing to norm
    r, o = dw.ps_block_norm(y, res, **kw)
    args = (y, res, kw["gate"], kw["scale"], kw["post_weight"], kw["pre_weight"])
    want, mag = (ref.norm(*args, bound=v) for v in (False, True))
    ref.close("residual", r, want["residual"], mag["residual"], 200)
    ref.close("out", o, want["out"], mag["out"], 200)
    say("norm backwards", case)
    dout, dres = m.act(T, ch, packed=True), m.act(T, ch, packed=True, dtype=rt)
    for given in (dres, None):
        g = dw.ps_block_norm_bwd(y, r, dout, given, **kw)
        args = (y, r, dout, given, kw["gate"], kw["scale"], kw["post_weight"], kw["pre_weight"])
        want, mag = (ref.norm_bwd(*args, bound=v) for v in (False, True))
        for name, key, there in (("dy", "dy", 1), ("dresidual", "dresidual", 1), ("dgate", "dgate", "g" in extra),
                                 ("dscale", "dscale", "s" in extra), ("dpost_weight", "dpost", "o" in extra),
                                 ("dpre_weight", "dpre", "p" in extra)):
            assert (getattr(g, name) is not None) == bool(there)
            if there:
                ref.close(name, getattr(g, name), want[key], mag[key], 200 + T)


NORM_WIDE = [  # as NORM: rows next to where the gradients change from one vector a thread to two
    (400, 5128, BF16, F32, "gsop", False),
    (5, 5127, BF16, BF16, "gsop", True),
    (600, 6144, F16, F32, "gsop", True),
    (300, 6144, F32, F32, "so", False),
    (4, 6143, F32, F32, "gsop", False),
    (3, 6152, BF16, F32, "gsop", False),
]


@pytest.mark.parametrize("case", NORM_WIDE, ids=str)
def test_norm_wide_rows(dw, case):
    test_norm(dw, case)


# ---------------------------------------------------------------------------
# streams, workspaces, graphs
# ---------------------------------------------------------------------------
def _train_step(dw, a, more, off, w, b, dout, ws=None):
    kept = torch.empty(dw.ps_selective_scan_checkpoint_rows(a["x"].shape[0], a["A"].shape[1]), *a["A"].shape,
                       device="cuda")
    c = dw.ps_causal_conv(a["x"], w, b, offsets=off)
    s = dict(a, x=c)
    o = dw.ps_selective_scan(**s, **more, offsets=off, checkpoints=kept, workspace=ws)
    r, n = dw.ps_block_norm(o, a["x"], gate=more["z"])
    gn = dw.ps_block_norm_bwd(o, r, dout, gate=more["z"], workspace=ws)
    g = dw.ps_selective_scan_bwd(*s.values(), gn.dy, kept, **more, offsets=off, workspace=ws)
    gc = dw.ps_causal_conv_bwd(a["x"], w, g.dx, b, offsets=off, workspace=ws)
    return [c, o, r, n, *(t for t in (*gn, *g, *gc) if t is not None)]


def _train_inputs(seed, T=150, ch=40, N=16, cuts=(0, 60, 60, 150)):
    m = Maker(seed, BF16)
    a, more = _scan_inputs(m, T, ch, 1, N, len(cuts) - 1, True, "Dzb")
    return a, more, _offsets(list(cuts)), m.par(ch, 4, scale=0.5), m.par(ch), m.act(T, ch)


def test_same_bits_again_and_on_another_stream(dw):
    args = _train_inputs(8)
    say("same bits")
    first = _train_step(dw, *args)
    second = _train_step(dw, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        third = _train_step(dw, *args)
    side.synchronize()
    for x, y, z in zip(first, second, third):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_stream_argument(dw):
    a, more, off, w, b, _ = _train_inputs(9)
    want = dw.ps_causal_conv(a["x"], w, b, offsets=off)
    scan = dw.ps_selective_scan(**a, **more, offsets=off)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    say("stream argument")
    got = dw.ps_causal_conv(a["x"], w, b, offsets=off, stream=side)
    got2 = dw.ps_selective_scan(**a, **more, offsets=off, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(got2, scan)


def test_workspace_shared_with_the_scans(dw, orc):
    """One prepared workspace serves the block's calls and the chained scans
    in turn; the scans' descriptors are cleaned of what the block left."""
    import numpy as np
    import workloads as wl
    from gpu_util import dev, host
    args = _train_inputs(10)
    want = _train_step(dw, *args)
    n = 40 * dw.ps_tile_elements(0) + 5
    x = wl.full_range_u32(n, seed=77)
    total = orc.scan_u32(x, "sum", True)[0]
    ws = dw.new_workspace(1 << 26)
    d_in, d_out = dev(x), torch.empty(n, dtype=torch.int32, device="cuda")
    for _ in range(3):
        say("workspace in turn")
        dw.ps_scan_single_pass("sum", True, d_in, d_out, workspace=ws)
        assert np.array_equal(host(d_out), total)
        for got, w in zip(_train_step(dw, *args, ws=ws), want):
            assert torch.equal(got, w)
    assert dw.workspace_header(ws)[dw.PS_WS_ERROR] == 0


def test_small_workspace_refused(dw):
    a, more, off, w, b, dout = _train_inputs(11)
    ws = dw.new_workspace(256)
    with pytest.raises(dw.DwpsError) as e:
        dw.ps_causal_conv_bwd(a["x"], w, dout, b, offsets=off, workspace=ws)
    assert e.value.status == 4


def test_graph(dw):
    """A training step and a decoding step in one graph, replayed with eager
    calls between."""
    args = _train_inputs(12)
    a, more, off, w, b, dout = args
    ws = dw.new_workspace(1 << 24)
    state = torch.zeros(4, *a["A"].shape, device="cuda")
    rows = torch.zeros(4, 3, a["x"].shape[1], dtype=BF16, device="cuda")
    slots = torch.tensor([2, 0], dtype=torch.int32, device="cuda")

    def decode(state, rows):
        two = {k: v[:2] if v.shape[0] == 150 else v for k, v in a.items()}
        x = dw.ps_causal_conv_step(two.pop("x"), rows, w, b, slots=slots)
        return dw.ps_selective_scan_step(x, state, **two, D=more["D"], z=more["z"][:2], dt_bias=more["dt_bias"],
                                         slots=slots)
    say("graph")
    want = _train_step(dw, *args, ws=ws)
    s2, r2 = state.clone(), rows.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _train_step(dw, *args, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _train_step(dw, *args, ws=ws)
        token = decode(state, rows)
    for k in range(4):
        say("graph replay", k)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        eager = decode(s2, r2)
        assert torch.equal(token, eager) and torch.equal(state, s2) and torch.equal(rows, r2)
        for x, y in zip(_train_step(dw, *args, ws=ws), want):
            assert torch.equal(x, y)


def test_graph_without_a_workspace(dw, orc):
    """Calls captured without a workspace have one of the graph's own: larger
    eager calls on the capture's stream, which replace the stream's workspace,
    and tensors that take its memory change no replay."""
    import numpy as np
    import workloads as wl
    from gpu_util import dev, host
    args = _train_inputs(15)
    n = 3 * dw.ps_tile_elements(0) + 7
    x = wl.full_range_u32(n, seed=78)
    total = orc.scan_u32(x, "sum", True)[0]
    d_in, d_out = dev(x), torch.empty(n, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    say("graph without a workspace")
    want = _train_step(dw, *args)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # the stream has a workspace that would do
        _train_step(dw, *args)
        dw.ps_scan_single_pass("sum", True, d_in, d_out)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = _train_step(dw, *args)
        dw.ps_scan_single_pass("sum", True, d_in, d_out)
    large = [torch.ones(k << 16, dtype=torch.int32, device="cuda") for k in (64, 256, 1024)]
    torch.cuda.synchronize()
    for k, big in enumerate(large):
        say("graph without a workspace, replay", k)
        with torch.cuda.stream(side):
            dw.ps_scan_single_pass("sum", True, big, torch.empty_like(big))
            junk = [torch.full((1 << 16,), -1, dtype=torch.int32, device="cuda") for _ in range(16)]
        d_out.fill_(0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(d_out), total)
        for g, w in zip(got, want):
            assert torch.equal(g, w)
        for g, w in zip(_train_step(dw, *args), want):
            assert torch.equal(g, w)
        del junk


# ---------------------------------------------------------------------------
# what the binding refuses
# ---------------------------------------------------------------------------
def test_binding_refuses(dw):
    m = Maker(13, BF16)
    T, ch, N = 10, 8, 4
    a, more = _scan_inputs(m, T, ch, 2, N, 1, False, "Dzb")
    w = m.par(ch, 4)
    x = a["x"]
    bad = lambda **kw: dict(dict(a, **more), **kw)  # noqa: E731
    for call in (
        lambda: dw.ps_causal_conv(x, w.half()), lambda: dw.ps_causal_conv(x.double(), w), lambda: dw.ps_causal_conv(x.int(), w),
        lambda: dw.ps_causal_conv(x, w[:4]), lambda: dw.ps_causal_conv(x, w, out=torch.empty_like(x, dtype=F32)),
        lambda: dw.ps_causal_conv(x, w, out=torch.empty(T, ch + 1, dtype=BF16, device="cuda")),
        lambda: dw.ps_causal_conv(x.t().contiguous().t(), w), lambda: dw.ps_causal_conv(x[0], w),
        lambda: dw.ps_causal_conv(x, w.cpu()), lambda: dw.ps_causal_conv(x.expand(T, ch)[:1].expand(T, ch), w),
        lambda: dw.ps_causal_conv(x, w, offsets=torch.zeros(2, device="cuda")),
        lambda: dw.ps_causal_conv(x, w, final=torch.empty(2, 3, ch, dtype=BF16, device="cuda")),
        lambda: dw.ps_selective_scan(**bad(dt=a["dt"].float())), lambda: dw.ps_selective_scan(**bad(dt=a["dt"][:5])),
        lambda: dw.ps_selective_scan(**bad(B=a["B"][:, :1])), lambda: dw.ps_selective_scan(**bad(A=a["A"][:, :2])),
        lambda: dw.ps_selective_scan(**bad(A=a["A"].to(BF16))), lambda: dw.ps_selective_scan(**bad(D=more["D"][:4])),
        lambda: dw.ps_selective_scan(**bad(initial=torch.zeros(2, ch, N, device="cuda"))),
        lambda: dw.ps_selective_scan(**bad(checkpoints=torch.zeros(2, ch, N, device="cuda"))),
        lambda: dw.ps_selective_scan_bwd(*a.values(), x, torch.zeros(2, ch, N, device="cuda"), **more),
        lambda: dw.ps_selective_scan_step(x, torch.zeros(4, ch, N, device="cuda"), *list(a.values())[1:], **more),
        lambda: dw.ps_selective_scan_step(x, torch.zeros(20, ch, N, device="cuda"), *list(a.values())[1:], **more,
                                          slots=torch.zeros(T, dtype=torch.int64, device="cuda")),
        lambda: dw.ps_block_norm(x, x.half()), lambda: dw.ps_block_norm(x, x[:4]), lambda: dw.ps_block_norm(x, x, gate=x[:4]),
        lambda: dw.ps_block_norm(x, x, scale=w), lambda: dw.ps_block_norm_bwd(x, x, x[:4]),
    ):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(dw.DwpsError):
        dw.ps_causal_conv(x, m.par(ch, 9))
    with pytest.raises(dw.DwpsError):
        dw.ps_causal_conv(x, w, out=x)


def test_a_sequence_alone_and_among_others(dw):
    """Many states, few channels and long sequences: the gradients' largest
    workgroups (four channel blocks, their sums over states in shared memory).
    A sequence gives what it gives by itself; only where its states come from
    (cells or the walk itself) may round differently."""
    m = Maker(14, F32)
    T, cut, ch, N = 16448, 320, 64, 64
    a, more = _scan_inputs(m, T, ch, 1, N, 2, False, "Dzb")
    dout = m.act(T, ch)

    def run(rows, off):
        at = {k: v[rows] if v.shape[0] == T else v for k, v in a.items()}
        opt = dict(more, z=more["z"][rows])
        kept = torch.empty(dw.ps_selective_scan_checkpoint_rows(at["x"].shape[0], N), ch, N, device="cuda")
        out = dw.ps_selective_scan(**at, **opt, offsets=off, checkpoints=kept)
        g = dw.ps_selective_scan_bwd(*at.values(), dout[rows], kept, **opt, offsets=off)
        return at, opt, [out, g.dx, g.ddt, g.dz, g.dB, g.dC]
    say("alone and among others")
    _, _, among = run(slice(0, T), _offsets([0, cut, T]))
    at, opt, alone = run(slice(0, cut), None)
    mag = ref.scan(**at, **opt, dout=dout[:cut], bound=True)
    K = 2 * ref.scan_roundings(at["dt"], at["A"], opt["dt_bias"], cut, ch, N)
    for name, x, y in zip(("out", "dx", "ddt", "dz", "dB", "dC"), among, alone):
        ref.close(name, x[:cut], ref.f64(y), mag[name], K)

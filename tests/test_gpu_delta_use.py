"""The gated delta rule and the layer norm as they are used: together in a
block, on other streams, side by side, in graphs that are replayed, with a
workspace that others use too, and at the edges of what the calls allow."""
import os
import sys

import pytest
import torch

import block_ref
import delta_ref as ref
import layer_ref
from gpu_util import require_gpu, say
from test_gpu_block import Maker, _offsets
from test_gpu_delta import BF16, F16, F32, DeltaMaker, delta_inputs

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def dw():
    return require_gpu()


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import delta_block
    finally:
        sys.path.pop(0)
    return delta_block


# ---------------------------------------------------------------------------
# the block
# ---------------------------------------------------------------------------
def test_the_example_runs(dw, example, capsys):
    say("example")
    example.main(["--channels", "128", "--heads", "4", "--kheads", "2", "--tokens", "300", "--decode", "3"])
    assert "training: loss" in capsys.readouterr().out


def _plain_block(block, x, offsets):
    """The example's block from plain products in 64 bits, token by token, with
    autograd; leaves: the block's parameters."""
    p = [t.detach().double().cpu().requires_grad_(True) for t in block.parameters]
    w_in, w_out, conv_w, conv_b, rate, rate_bias, in_w, in_b, head_w, head_b = p
    x = x.double().cpu()
    norm = torch.nn.functional.layer_norm
    h = norm(x, (x.shape[1],), in_w, in_b, 1e-5)
    c, g, beta = (h @ w_in).split(block.cuts, dim=1)
    g, beta = -torch.exp(rate) * torch.nn.functional.softplus(g + rate_bias), torch.sigmoid(beta)
    rows = []
    for lo, hi in block_ref.sequences(offsets, x.shape[0]):
        past = torch.cat([torch.zeros(block.width - 1, c.shape[1], dtype=c.dtype), c[lo:hi]])
        pre = sum(past[i:i + hi - lo] * conv_w[:, i] for i in range(block.width)) + conv_b
        q, k, v = block._heads(pre * torch.sigmoid(pre))
        q, k = (t / torch.sqrt(t.square().sum(-1, keepdim=True) + 1e-6) for t in (q, k))
        q, k = (t.repeat_interleave(block.heads // block.kheads, 1) for t in (q, k))
        S = torch.zeros(block.heads, block.key_dim, block.value_dim, dtype=c.dtype)
        for t in range(hi - lo):
            S = torch.exp(g[lo + t])[:, None, None] * S
            u = beta[lo + t][:, None] * (v[t] - torch.einsum("hkv,hk->hv", S, k[t]))
            S = S + k[t][:, :, None] * u[:, None, :]
            rows.append(block.key_dim ** -0.5 * torch.einsum("hkv,hk->hv", S, q[t]))
    o = norm(torch.stack(rows), (block.value_dim,), head_w, head_b, 1e-5).reshape(x.shape[0], -1)
    return x + o @ w_out, p


def test_the_examples_gradients(dw, example):
    """In fp32 against 64 bits.  A gradient is a sum whose terms pass at most 2^11
    roundings one after another (products over up to 96 channels and 150 rows, the
    rule's over 64 + 24 terms a chunk, twice for there and back), and the norms
    and the division by |k| make an error at most 8 times as large: 2^-24 * 2^14
    of a gradient's length."""
    block = example.Block(48, 4, 2, key_dim=24, value_dim=16, dtype=F32)
    off = _offsets([0, 70, 70, 150])
    x = Maker(3, F32).act(150, 48)
    for p in block.parameters:
        p.requires_grad_(True)
    say("the example's gradients")
    out = block.train(x, off)
    dout = Maker(4, F32).act(150, 48)
    out.backward(dout)
    want, leaves = _plain_block(block, x, off)
    want.backward(dout.double().cpu())
    assert (out.detach().double().cpu() - want.detach()).norm() <= 2.0 ** -10 * want.detach().norm()
    for i, (p, w) in enumerate(zip(block.parameters, leaves)):
        off_by = float((p.grad.double().cpu() - w.grad).norm() / w.grad.norm())
        assert off_by <= 2.0 ** -10, (i, off_by)


def test_prompts_then_tokens_are_one_prompt(dw, example):
    """Prompts of two sequences and 70 tokens one at a time from the pools give
    what longer prompts give, rows and pools (fp32; tolerance as above)."""
    block = example.Block(40, 6, 2, key_dim=32, value_dim=20, dtype=F32)
    n, more = (130, 5), 70
    x = [Maker(5 + i, F32).act(c + more, 40) for i, c in enumerate(n)]

    def pools(count):
        return (torch.zeros(count, block.width - 1, block.inner, device="cuda"),
                torch.zeros(count, block.heads, block.key_dim, block.value_dim, device="cuda"))
    say("prompts then tokens")
    rows, states = pools(2)
    block.prompts(torch.cat([x[0][:n[0]], x[1][:n[1]]]), _offsets([0, n[0], sum(n)]), rows, states)
    slots = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    got = [[], []]
    for t in range(more):
        out = block.token(torch.stack([x[1][n[1] + t], x[0][n[0] + t]]), slots, rows, states)
        got[1].append(out[0])
        got[0].append(out[1])
    all_rows, all_states = pools(2)
    want = block.prompts(torch.cat(x), _offsets([0, n[0] + more, sum(n) + 2 * more]), all_rows, all_states)
    for g, w in ((torch.stack(got[0]), want[n[0]:n[0] + more]), (torch.stack(got[1]), want[n[0] + more + n[1]:]),
                 (rows, all_rows), (states, all_states)):
        assert float((g - w).norm()) <= 2.0 ** -10 * float(w.norm())


# ---------------------------------------------------------------------------
# streams, graphs, workspaces
# ---------------------------------------------------------------------------
def _inputs(seed, dtype=BF16, T=700, KH=2, H=4, K=40, V=24, cuts=(0, 600, 600, 700), initial=True):
    m = DeltaMaker(seed, dtype)
    a, more = delta_inputs(m, T, KH, H, K, V, True, initial, len(cuts) - 1)
    return a, dict(more, offsets=_offsets(list(cuts))), m.act(T, H, V), m.par(H * V, mean=1.0), m.par(H * V)


def _train_step(dw, a, more, dout, w, b, ws=None):
    T, H, V = a["v"].shape
    seqs = more["offsets"].numel() - 1
    kept = torch.empty(dw.ps_gated_delta_checkpoint_floats(T, seqs, H, a["q"].shape[2], V), device="cuda")
    final = torch.empty_like(more["initial"])
    o = dw.ps_gated_delta(**a, **more, checkpoints=kept, final=final, workspace=ws)
    n = dw.ps_layer_norm(o.reshape(T, -1), w, b)
    gn = dw.ps_layer_norm_bwd(o.reshape(T, -1), dout.reshape(T, -1), w, b, workspace=ws)
    g = dw.ps_gated_delta_bwd(**a, **more, dout=gn.dx.view_as(o), checkpoints=kept, dfinal=final, workspace=ws)
    return [o, final, n, *gn, *g]


def test_same_bits_again_and_on_another_stream(dw):
    args = _inputs(20)
    say("same bits")
    first, second = _train_step(dw, *args), _train_step(dw, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        third = _train_step(dw, *args)
    side.synchronize()
    for x, y, z in zip(first, second, third):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_stream_argument(dw):
    a, more, dout, w, b = _inputs(21)
    x = dout.reshape(dout.shape[0], -1)
    state = more["initial"].clone()
    want = dw.ps_gated_delta(**a, **more), dw.ps_layer_norm(x, w, b), dw.ps_layer_norm_bwd(x, x, w, b).dx
    step = {k: v[:3] for k, v in a.items()}
    want += (dw.ps_gated_delta_step(**step, state=state.clone()),)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    say("stream argument")
    got = (dw.ps_gated_delta(**a, **more, stream=side), dw.ps_layer_norm(x, w, b, stream=side),
           dw.ps_layer_norm_bwd(x, x, w, b, stream=side).dx, dw.ps_gated_delta_step(**step, state=state, stream=side))
    side.synchronize()
    for g, t in zip(got, want):
        assert torch.equal(g, t)


def test_two_calls_at_once(dw):
    """Two streams with calls of their own in flight together."""
    one, two = _inputs(22), _inputs(23, F16, T=1500, cuts=(0, 1400, 1450, 1500))
    say("two calls at once")
    want = [_train_step(dw, *one), _train_step(dw, *two)]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for k in range(3):
        for i, args in enumerate((one, two)):
            with torch.cuda.stream(sides[i]):
                got[i].append(_train_step(dw, *args))
    for s in sides:
        s.synchronize()
    for i in range(2):
        for run in got[i]:
            for x, y in zip(run, want[i]):
                assert torch.equal(x, y)


def test_workspace_shared_with_the_scans(dw, orc):
    """One prepared workspace serves these calls and the chained scans in turn."""
    import numpy as np
    import workloads as wl
    from gpu_util import dev, host
    args = _inputs(24)
    want = _train_step(dw, *args)
    n = 40 * dw.ps_tile_elements(0) + 5
    x = wl.full_range_u32(n, seed=79)
    total = orc.scan_u32(x, "sum", True)[0]
    ws = dw.new_workspace(1 << 27)
    d_in, d_out = dev(x), torch.empty(n, dtype=torch.int32, device="cuda")
    for _ in range(3):
        say("workspace in turn")
        dw.ps_scan_single_pass("sum", True, d_in, d_out, workspace=ws)
        assert np.array_equal(host(d_out), total)
        for got, w in zip(_train_step(dw, *args, ws=ws), want):
            assert torch.equal(got, w)
    assert dw.workspace_header(ws)[dw.PS_WS_ERROR] == 0


def test_small_workspace_refused(dw):
    a, more, dout, w, b = _inputs(25)
    ws = dw.new_workspace(256)
    for call in (lambda: dw.ps_gated_delta(**a, **more, workspace=ws),
                 lambda: dw.ps_layer_norm_bwd(dout.reshape(700, -1), dout.reshape(700, -1), w, b, workspace=ws)):
        with pytest.raises(dw.DwpsError) as e:
            call()
        assert e.value.status == 4


@pytest.mark.parametrize("given", [True, False], ids=["workspace", "none"])
def test_graphs(dw, given):
    """A training step and decoding in one graph and another training step in a
    second one, which shares the first's workspace, replayed in turn with eager
    calls between."""
    args, other = _inputs(26), _inputs(27, T=300, cuts=(0, 10, 300))
    ws = dw.new_workspace(1 << 27) if given else None
    slots = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    two = {k: v[:2] for k, v in args[0].items()}
    state = torch.rand(4, 4, 40, 24, device="cuda")
    s2 = state.clone()
    decode = lambda s: dw.ps_gated_delta_step(**two, state=s, slots=slots, normalize=True)  # noqa: E731
    say("graph")
    want, want2 = _train_step(dw, *args, ws=ws), _train_step(dw, *other, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _train_step(dw, *args, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        got = _train_step(dw, *args, ws=ws)
        token = decode(state)
    with torch.cuda.graph(second):
        got2 = _train_step(dw, *other, ws=ws)
    for k in range(4):
        say("graph replay", k)
        first.replay()
        second.replay()
        torch.cuda.synchronize()
        eager = decode(s2)
        assert torch.equal(token, eager) and torch.equal(state, s2)
        for x, y in zip(got + got2, want + want2):
            assert torch.equal(x, y)
        for x, y in zip(_train_step(dw, *args, ws=ws), want):
            assert torch.equal(x, y)


# ---------------------------------------------------------------------------
# edges
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
def test_a_sequence_alone_and_among_others(dw, dtype):
    """Chunks begin at a sequence's first row: a short sequence gives the same bits
    by itself and packed with others, gradients included."""
    m = DeltaMaker(28, dtype)
    T, lo, hi = 400, 37, 230
    a, more = delta_inputs(m, T, 1, 2, 48, 32, True, True, 3)
    dout = m.act(T, 2, 32, packed=True)

    def run(rows, initial, off, seqs):
        at = {k: v[rows] for k, v in a.items()}
        n = at["q"].shape[0]
        kept = torch.empty(dw.ps_gated_delta_checkpoint_floats(n, seqs, 2, 48, 32), device="cuda")
        how = dict(initial=initial, normalize=True, offsets=off)
        final = torch.empty_like(initial)
        out = dw.ps_gated_delta(**at, **how, checkpoints=kept, final=final)
        g = dw.ps_gated_delta_bwd(**at, **how, dout=dout[rows], checkpoints=kept)
        return out, g.dq, g.dk, g.dv, g.dg, g.dbeta, final, g.dinitial
    say("alone and among others")
    among = run(slice(0, T), more["initial"], _offsets([0, lo, hi, T]), 3)
    alone = run(slice(lo, hi), more["initial"][1:2].contiguous(), None, 1)
    for x, y in zip(among[:6], alone[:6]):
        assert torch.equal(x[lo:hi], y)
    for x, y in zip(among[6:], alone[6:]):
        assert torch.equal(x[1:2], y)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("where", ["q", "k", "v", "g", "beta", "initial"])
def test_nan_and_infinities_stay_in_their_head_and_sequence(dw, dtype, where):
    """Heads, other sequences, and rows of chunks before are what they are without
    them; one in a value or in a state's column stays in its column."""
    m = DeltaMaker(29, dtype)
    T, H, K, V = 500, 2, 32, 40
    cuts = [0, 100, 400, 500]
    off = _offsets(cuts)
    a, more = delta_inputs(m, T, 2, H, K, V, True, True, 3)
    want, wfin = dw.ps_gated_delta(**a, **more, offsets=off), torch.empty_like(more["initial"])
    dw.ps_gated_delta(**a, **more, offsets=off, final=wfin)
    for bad in (float("nan"), float("inf"), float("-inf")):
        if where == "g" and bad == float("-inf"):
            continue  # a state that starts again
        say("nan and infinities", where, bad, dtype)
        b, opt = {k: v.clone() for k, v in a.items()}, dict(more)
        at = 100 + 64 * 2 + 7  # in the third chunk of the second sequence
        if where == "initial":
            opt["initial"] = more["initial"].clone()
            opt["initial"][1, 1, 3, 5] = bad
        elif where in ("g", "beta"):
            b[where][at, 1] = bad
        else:
            b[where][at, 1, 5] = bad
        final = torch.empty_like(wfin)
        out = dw.ps_gated_delta(**b, **opt, offsets=off, final=final)
        same = torch.ones(T, H, V, dtype=torch.bool)
        first = 100 if where == "initial" else 100 + 64 * 2
        if where in ("v", "initial"):
            same[first:400, 1, 5] = False
        else:
            same[first:400, 1] = False
        assert torch.equal(out.cpu()[same], want.cpu()[same])
        bad_rows = {"initial": slice(100, 400), "q": slice(at, at + 1)}.get(where, slice(at, 400))
        cols = slice(5, 6) if where in ("v", "initial") else slice(0, V)
        assert not torch.isfinite(out[bad_rows, 1, cols]).any()
        others = [0, 2]
        assert torch.equal(final[others], wfin[others]) and torch.equal(final[1, 0], wfin[1, 0])
        if where == "q":
            assert torch.equal(final, wfin)
        elif where in ("v", "initial"):
            keep = [c for c in range(V) if c != 5]
            assert torch.equal(final[1, 1][:, keep], wfin[1, 1][:, keep])
            assert not torch.isfinite(final[1, 1][:, 5]).any()
        else:
            assert not torch.isfinite(final[1, 1]).any()


def test_minus_infinity_starts_a_state_again(dw):
    """Where g is minus infinity nothing of the rows before is left: rows from there
    on are a sequence of their own (fp32: to the roundings of 130 rows)."""
    m = DeltaMaker(30, F32)
    T, at = 200, 70
    a, _ = delta_inputs(m, T, 1, 2, 16, 8, True, False, 1)
    for bad in (float("-inf"), -1e30, -600.0):
        b = dict(a, g=a["g"].clone())
        b["g"][at] = bad
        say("a state that starts again", bad)
        out = dw.ps_gated_delta(**b, normalize=True)
        tail = {k: v[at:] for k, v in a.items()}
        want, bound = ref.delta(**tail, normalize=True)
        ref.close("out", out[at:], want["out"], 2 * bound["out"])
        state = torch.ones(1, 2, 16, 8, device="cuda")
        one = dw.ps_gated_delta_step(**{k: v[at:at + 1] for k, v in b.items()}, state=state, normalize=True)
        ref.close("step", one, want["out"][:1], bound["out"][:1])


def test_strong_and_no_corrections(dw):
    """beta 0 writes nothing, beta up to 2 overshoots; no decay at all."""
    m = DeltaMaker(31, F32)
    T, H, K, V = 150, 2, 24, 16
    a, more = delta_inputs(m, T, 1, H, K, V, True, True, 1)
    a["g"].zero_()
    say("no corrections")
    final = torch.empty_like(more["initial"])
    dw.ps_gated_delta(**dict(a, beta=torch.zeros_like(a["beta"])), **more, final=final)
    assert torch.equal(final, more["initial"])
    a["beta"].mul_(2.0)
    out = dw.ps_gated_delta(**a, **more, final=final)
    want, bound = ref.delta(**a, **more)
    ref.close("out", out, want["out"], bound["out"])
    ref.close("final", final, want["final"], bound["final"])


def test_equal_keys(dw):
    """The same key in every row, beta 1: a chunk's triangle is all ones, its
    inverse two diagonals, and every row replaces what the one before wrote."""
    for dtype in (BF16, F32):
        T, K, V = 200, 16, 8
        m = DeltaMaker(32, dtype)
        key = torch.zeros(T, 1, K, dtype=dtype, device="cuda")
        key[:, :, 3] = 1.0
        v = m.act(T, 1, V)
        say("equal keys", dtype)
        out = dw.ps_gated_delta(key, key, v, torch.zeros(T, 1, device="cuda"), torch.ones(T, 1, device="cuda"), scale=1.0)
        # a term's roundings as delta_ref counts them, of the value replaced and the new one
        bound = torch.full(v.shape, 4.0 * ref.PER_CHUNK * ref.step_of(dtype, K) * 4 * float(v.abs().max()), dtype=torch.float64)
        ref.close("out", out, block_ref.f64(v), bound)


def test_offsets_out_of_contract_stay_in_bounds(dw):
    """Falling offsets and ones past the last row: some results, within the arrays."""
    m = DeltaMaker(33, BF16)
    T, H, K, V = 200, 2, 16, 24
    a, more = delta_inputs(m, T, 1, H, K, V, True, True, 4)
    dout = m.act(T, H, V)
    for cuts in ([0, 150, 30, 180, 200], [50, 20, 10, 5, 0], [0, 500, 700, 100, 1 << 30], [-1, -1, -1, -1, -1],
                 [190, 250, 20, 300, 60]):
        say("offsets out of contract", cuts)
        off = _offsets(cuts)
        big = torch.full((T + 200, H, V), 7.0, dtype=BF16, device="cuda")
        kept = torch.zeros(dw.ps_gated_delta_checkpoint_floats(T, 4, H, K, V), device="cuda")
        dw.ps_gated_delta(**a, **more, offsets=off, out=big[100:100 + T], checkpoints=kept)
        dw.ps_gated_delta_bwd(**a, **more, offsets=off, dout=dout, checkpoints=kept)
        torch.cuda.synchronize()
        assert (big[:100] == 7.0).all() and (big[100 + T:] == 7.0).all()


def test_the_same_slot_twice_and_slots_outside(dw):
    """The same slot twice is outside the contract (rows race for it) and stays
    within the pool: the slots that no row names keep their bits.  Slots outside
    read zeros and write nothing."""
    m = DeltaMaker(34, BF16)
    a, _ = delta_inputs(m, 6, 1, 2, 32, 16, True, False, 1)
    state = m.par(5, 2, 32, 16)
    before = state.clone()
    slots = torch.tensor([1, 1, -7, 2 ** 31 - 1, 5, 3], dtype=torch.int32, device="cuda")
    say("the same slot twice")
    out = dw.ps_gated_delta_step(**a, state=state, slots=slots, normalize=True)
    assert torch.equal(state[[0, 2, 4]], before[[0, 2, 4]]) and torch.isfinite(out).all() and torch.isfinite(state).all()
    want, bound = ref.delta_step(a["q"], a["k"], a["v"], before, a["g"], a["beta"], normalize=True, slots=slots)
    ref.close("out", out[2:], want["out"][2:], bound["out"][2:])
    ref.close("state", state[3], want["state"][3], bound["state"][3])
    none = dw.ps_gated_delta_step(**a, state=before[:0], slots=slots, normalize=True)  # an empty pool
    ref.close("out", none[2:5], want["out"][2:5], bound["out"][2:5])


def test_a_pool_past_32_bits(dw):
    """States whose elements' numbers pass 2^32: the last slot's are read and
    written in place, the others stay."""
    H, K, V = 32, 256, 256
    pool = (1 << 32) // (H * K * V) + 3
    state = torch.zeros(pool, H, K, V, device="cuda")
    m = DeltaMaker(35, BF16)
    a, _ = delta_inputs(m, 2, 1, H, K, V, True, False, 1)
    last = m.par(1, H, K, V)
    state[pool - 1] = last[0]
    slots = torch.tensor([pool - 1, 1], dtype=torch.int32, device="cuda")
    say("a pool past 32 bits", pool)
    out = dw.ps_gated_delta_step(**a, state=state, slots=slots, normalize=True)
    small = torch.cat([last, torch.zeros_like(last)])
    want = dw.ps_gated_delta_step(**a, state=small, normalize=True)
    assert torch.equal(out, want) and torch.equal(state[pool - 1], small[0]) and torch.equal(state[1], small[1])
    assert not state[0].any() and not state[2:pool - 1].any()


def test_rows_past_32_bits(dw):
    """Activations whose elements' numbers pass 2^32: a sequence at the end of
    them gives what it gives by itself."""
    T, H, V = 66000, 256, 256
    m = DeltaMaker(36, BF16)
    a, _ = delta_inputs(m, 100, 1, H, 8, V, True, False, 1)
    big = {k: torch.zeros(T, *v.shape[1:], dtype=v.dtype, device="cuda") for k, v in a.items()}
    for k, v in a.items():
        big[k][-100:] = v
    say("rows past 32 bits")
    out = dw.ps_gated_delta(**big, normalize=True, offsets=_offsets([T - 100, T]))
    want = dw.ps_gated_delta(**a, normalize=True, offsets=_offsets([0, 100]))
    assert torch.equal(out[-100:], want)
    x = out.view(T * 16, -1)
    assert torch.equal(dw.ps_layer_norm(x)[-1600:], dw.ps_layer_norm(x[-1600:].contiguous()))


@pytest.mark.parametrize("heads", [80, 160])
def test_many_workgroups_of_sequences_that_differ(dw, heads):
    """More walks than run at once, of lengths that differ: every sequence gives
    the same bits as by itself, empty and equally long ones too."""
    m = DeltaMaker(37 + heads, BF16)
    cuts = [3, 3, 20, 60, 60, 190, 207, 247, 247]
    T = 260
    a, more = delta_inputs(m, T, heads // 4, heads, 16, 8, True, True, len(cuts) - 1)
    dout = m.act(T, heads, 8, packed=True)
    kept = lambda n, s: torch.empty(dw.ps_gated_delta_checkpoint_floats(n, s, heads, 16, 8), device="cuda")  # noqa: E731
    say("sequences that differ", heads)
    c, final = kept(T, len(cuts) - 1), torch.empty_like(more["initial"])
    out = dw.ps_gated_delta(**a, **more, offsets=_offsets(cuts), checkpoints=c, final=final)
    g = dw.ps_gated_delta_bwd(**a, **more, offsets=_offsets(cuts), dout=dout, checkpoints=c, dfinal=final)
    for s, (lo, hi) in enumerate(zip(cuts, cuts[1:])):
        if lo == hi:
            assert torch.equal(final[s], more["initial"][s]) and torch.equal(g.dinitial[s], final[s])
            continue
        one = {k: v[lo:hi] for k, v in a.items()}
        how = dict(normalize=True, initial=more["initial"][s:s + 1].contiguous())
        c1, f1 = kept(hi - lo, 1), torch.empty(1, heads, 16, 8, device="cuda")
        assert torch.equal(dw.ps_gated_delta(**one, **how, checkpoints=c1, final=f1), out[lo:hi])
        g1 = dw.ps_gated_delta_bwd(**one, **how, dout=dout[lo:hi], checkpoints=c1, dfinal=f1)
        assert torch.equal(f1[0], final[s]) and torch.equal(g1.dinitial[0], g.dinitial[s])
        for name in ("dq", "dk", "dv", "dg", "dbeta"):
            assert torch.equal(getattr(g1, name), getattr(g, name)[lo:hi]), name


@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
def test_nan_outside_all_sequences_is_not_read(dw, dtype):
    """Rows before the first sequence and behind the last hold NaN, gates and
    gradients too; the sequences' results have none."""
    m = DeltaMaker(38, dtype)
    T, lo, hi = 150, 5, 140
    a, more = delta_inputs(m, T, 1, 2, 24, 12, True, True, 2)
    dout = m.act(T, 2, 12, packed=True)
    for t in (*a.values(), dout):
        t[:lo], t[hi:] = float("nan"), float("nan")
    off = _offsets([lo, 75, hi])
    say("NaN outside all sequences", dtype)
    kept = torch.empty(dw.ps_gated_delta_checkpoint_floats(T, 2, 2, 24, 12), device="cuda")
    out, final = torch.full((T, 2, 12), 7.0, dtype=dtype, device="cuda"), torch.empty_like(more["initial"])
    dw.ps_gated_delta(**a, **more, offsets=off, checkpoints=kept, out=out, final=final)
    g = dw.ps_gated_delta_bwd(**a, **more, offsets=off, dout=dout, checkpoints=kept, dfinal=final)
    assert (out[:lo] == 7.0).all() and (out[hi:] == 7.0).all()
    for t in (out[lo:hi], final, g.dinitial, *(t[lo:hi] for t in g[:5])):
        assert torch.isfinite(t).all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
def test_eps_zero(dw, dtype):
    """eps 0 with rows that are no zeros: chunks and sets of rows that are partly
    filled divide nothing by the lengths of rows that are not there."""
    m = DeltaMaker(39, dtype)
    T, cuts = 90, [0, 3, 90]
    a, more = delta_inputs(m, T, 1, 2, 24, 12, True, True, 2)
    dout = m.act(T, 2, 12, packed=True)
    say("eps zero", dtype)
    off = _offsets(cuts)
    kept = torch.empty(dw.ps_gated_delta_checkpoint_floats(T, 2, 2, 24, 12), device="cuda")
    out, final = torch.empty_like(dout), torch.empty_like(more["initial"])
    dw.ps_gated_delta(**a, **more, eps=0.0, offsets=off, checkpoints=kept, out=out, final=final)
    g = dw.ps_gated_delta_bwd(**a, **more, eps=0.0, offsets=off, dout=dout, checkpoints=kept)
    want, bound = ref.delta(**a, **more, eps=0.0, offsets=off, dout=dout, dtype=dtype)
    ref.close("out", out, want["out"], bound["out"])
    ref.close("final", final, want["final"], bound["final"])
    for name in g._fields:
        ref.close(name, getattr(g, name), want[name], bound[name])
    for ch in (100, 300, 600):
        x, d, w = m.act(21, ch), m.act(21, ch), m.par(ch)
        got = dw.ps_layer_norm_bwd(x, d, w, w, eps=0.0)
        want, mag = (layer_ref.layer_norm(x, w, w, eps=0.0, dout=d, bound=v) for v in (False, True))
        for name, t in (("out", dw.ps_layer_norm(x, w, w, eps=0.0)), ("dx", got.dx), ("dweight", got.dweight),
                        ("dbias", got.dbias)):
            block_ref.close(name, t, want[name], mag[name], 2 * (ch + 64) + 21)

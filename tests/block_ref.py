"""The state space block's operators from their formulas in 64 bits, one token
after another, on the CPU.

Every function also takes ``bound=True``: the same sums with every term's
magnitude in place of the term, which is what a rounding error can grow
with.  A term is a product of factors each a few roundings off; a decay
exp(step A) is off by |step A| times its argument's relative error, and a run
of decays with arguments summing to -S by S e^-S <= 0.74 e^(-S/2), so the
bound's decays are those of A / 2."""
from __future__ import annotations

import torch

F64 = torch.float64
U32 = 2.0 ** -24


def f64(t):
    return None if t is None else t.detach().cpu().to(F64)


def _mag(t, bound):
    return t.abs() if bound and t is not None else t


def sequences(offsets, tokens):
    off = [0, tokens] if offsets is None else offsets.cpu().to(torch.int64).tolist()
    return list(zip(off[:-1], off[1:]))


def _silu(v, bound):
    return _mag(v * torch.sigmoid(v), bound)


def _dsilu(v, bound):
    s = torch.sigmoid(v)
    return s * (1.0 + _mag(v, bound) * (1.0 - s))


def conv(x, weight, bias=None, offsets=None, initial=None, dout=None, bound=False):
    """out, final and, with dout, the gradients."""
    x, weight, bias, initial, dout = (f64(t) for t in (x, weight, bias, initial, dout))
    T, D = x.shape
    W = weight.shape[1]
    seqs = sequences(offsets, T)
    out = torch.zeros_like(x)
    final = torch.zeros(len(seqs), W - 1, D, dtype=F64)
    r = dict(dx=torch.zeros_like(x), dweight=torch.zeros_like(weight), dbias=torch.zeros(D, dtype=F64),
             dinitial=torch.zeros_like(final))
    b = torch.zeros(D, dtype=F64) if bias is None else bias
    for q, (lo, hi) in enumerate(seqs):
        before = torch.zeros(W - 1, D, dtype=F64) if initial is None else initial[q]
        rows = torch.cat([before, x[lo:hi]])
        drows = torch.zeros_like(rows)
        final[q] = rows[len(rows) - (W - 1):] if W > 1 else final[q]
        for t in range(lo, hi):
            win = rows[t - lo:t - lo + W]                       # [W, D]
            pre = b + (win * weight.t()).sum(0)
            mag = _mag(b, bound) + _mag(win * weight.t(), bound).sum(0)
            out[t] = 1.1 * mag if bound else _silu(pre, False)  # |silu'| <= 1.1
            if dout is not None:
                g = dout[t] * _dsilu(pre, False)
                if bound:  # |silu''| <= 0.5
                    g = dout[t].abs() * (_dsilu(pre, True) + 0.5 * mag)
                drows[t - lo:t - lo + W] += g * _mag(weight.t(), bound)
                r["dweight"] += (g * _mag(win, bound)).t()
                r["dbias"] += g
        r["dx"][lo:hi] = drows[W - 1:]
        r["dinitial"][q] = drows[:W - 1]
    return dict(out=out, final=final, **(r if dout is not None else {}))


def scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, offsets=None, initial=None, dout=None, bound=False):
    """out, final and, with dout, the gradients."""
    x, dt, A, B, C, D, z, dt_bias, initial, dout = (f64(t) for t in (x, dt, A, B, C, D, z, dt_bias, initial, dout))
    T, ch = x.shape
    G, N = B.shape[1:]
    raw = dt if dt_bias is None else dt + dt_bias
    step = torch.logaddexp(raw, torch.zeros_like(raw))
    sig = torch.sigmoid(raw)
    sg = torch.ones_like(x) if z is None else _silu(z, bound)
    dsg = torch.zeros_like(x) if z is None else _dsilu(z, bound)
    x, B, C, initial, dout = (_mag(t, bound) for t in (x, B, C, initial, dout))
    Am = A.abs() if bound else A
    Ad = A / 2 if bound else A
    D_ = torch.zeros(ch, dtype=F64) if D is None else _mag(D, bound)
    wide = lambda v: v.repeat_interleave(ch // G, 0)  # noqa: E731
    seqs = sequences(offsets, T)
    inner = torch.zeros_like(x)
    final = torch.zeros(len(seqs), ch, N, dtype=F64)
    hs = torch.zeros(T, ch, N, dtype=F64)
    for q, (lo, hi) in enumerate(seqs):
        h = torch.zeros(ch, N, dtype=F64) if initial is None else initial[q]
        for t in range(lo, hi):
            h = torch.exp(step[t][:, None] * Ad) * h + (step[t] * x[t])[:, None] * wide(B[t])
            hs[t] = h
            inner[t] = (h * wide(C[t])).sum(1) + D_ * x[t]
        final[q] = h
    r = dict(out=inner * sg, final=final)
    if dout is None:
        return r
    gy = dout * sg
    r.update(dz=dout * inner * dsg, dD=(gy * x).sum(0), dx=gy * D_, ddt=torch.zeros_like(x), dA=torch.zeros_like(A),
             dB=torch.zeros_like(B), dC=torch.zeros_like(C), dinitial=torch.zeros_like(final))
    for q, (lo, hi) in enumerate(seqs):
        back = torch.zeros(ch, N, dtype=F64)
        for t in reversed(range(lo, hi)):
            dh = back + gy[t][:, None] * wide(C[t])
            r["dC"][t] = (gy[t][:, None] * hs[t]).view(G, ch // G, N).sum(1)
            r["dB"][t] = (dh * (step[t] * x[t])[:, None]).view(G, ch // G, N).sum(1)
            back = torch.exp(step[t][:, None] * Ad) * dh
            before = hs[t - 1] if t > lo else torch.zeros(ch, N, dtype=F64) if initial is None else initial[q]
            flow = back * before
            along = (dh * wide(B[t])).sum(1)
            r["dA"] += flow * step[t][:, None]
            r["dx"][t] += step[t] * along
            r["ddt"][t] = ((flow * Am).sum(1) + x[t] * along) * sig[t]
        r["dinitial"][q] = back
    r["ddt_bias"] = r["ddt"].sum(0)
    return r


def scan_roundings(dt, A, dt_bias, T, ch, N):
    """How many half-ulps of fp32 a term of the scan's sums can be off by: 3
    for each of up to T decays and 2 for each sum along the way, the softplus
    (its series and e^-|v|, off by 2 |v|), products and sums over states,
    channels and tokens (forwards, backwards and the sum over tokens)."""
    raw = f64(dt) if dt_bias is None else f64(dt) + f64(dt_bias)
    v = float(raw.abs().max()) if raw.numel() else 0.0
    return 5.0 * 2 * T + N + ch + T + 2 * (12 + 4 * v) + 32


def scan_step(x, state, dt, A, B, C, D=None, z=None, dt_bias=None, slots=None, bound=False):
    """out and the whole new state; a slot outside the pool reads zeros."""
    pool = state.shape[0]
    at = list(range(x.shape[0])) if slots is None else slots.cpu().tolist()
    out, new = torch.zeros(x.shape, dtype=F64), f64(state).clone()
    if bound:
        new = new.abs()
    for i, slot in enumerate(at):
        held = 0 <= slot < pool
        init = f64(state)[slot:slot + 1] if held else None
        row = lambda t: None if t is None else t[i:i + 1]  # noqa: E731
        r = scan(row(x), row(dt), A, row(B), row(C), D, row(z), dt_bias, None, init, bound=bound)
        out[i] = r["out"][0]
        if held:
            new[slot] = r["final"][0]
    return dict(out=out, state=new)


def conv_step(x, state, weight, bias=None, slots=None, bound=False):
    pool = state.shape[0]
    at = list(range(x.shape[0])) if slots is None else slots.cpu().tolist()
    out, new = torch.zeros(x.shape, dtype=F64), f64(state).clone()
    for i, slot in enumerate(at):
        held = 0 <= slot < pool
        r = conv(x[i:i + 1], weight, bias, None, f64(state)[slot:slot + 1] if held else None, bound=bound)
        out[i] = r["out"][0]
        if held:
            new[slot] = r["final"][0]
    return dict(out=out, state=new)


def norm(y, residual, gate=None, scale=None, post=None, pre=None, eps=1e-6, bound=False):
    y, residual, gate, scale, post, pre = (f64(t) for t in (y, residual, gate, scale, post, pre))
    d = y.shape[1]
    one = torch.ones(d, dtype=F64)
    scale, post, pre = (one if p is None else p for p in (scale, post, pre))
    ny = torch.rsqrt(y.square().sum(1, keepdim=True) / d + eps)
    sg = torch.ones_like(y) if gate is None else torch.sigmoid(gate)
    add = scale * sg * (y * ny * post)
    r = residual + add
    nr = torch.rsqrt(r.square().sum(1, keepdim=True) / d + eps)
    if bound:  # residual_out's error reaches out through the element and the row's norm
        mag = residual.abs() + add.abs()
        lean = (mag * r.abs()).sum(1, keepdim=True) / d
        return dict(residual=mag, out=(mag * nr + r.abs() * nr ** 3 * lean) * pre.abs())
    return dict(residual=r, out=r * nr * pre)


def norm_bwd(y, residual_out, dout, dres=None, gate=None, scale=None, post=None, pre=None, eps=1e-6, bound=False):
    y, r, dout, dres, gate, scale, post, pre = (f64(t) for t in (y, residual_out, dout, dres, gate, scale, post, pre))
    d = y.shape[1]
    one = torch.ones(d, dtype=F64)
    scale, post, pre = (one if p is None else p for p in (scale, post, pre))
    ny = torch.rsqrt(y.square().sum(1, keepdim=True) / d + eps)
    nr = torch.rsqrt(r.square().sum(1, keepdim=True) / d + eps)
    sg = torch.ones_like(y) if gate is None else torch.sigmoid(gate)
    y, r, dout, dres, scale, post, pre = (_mag(t, bound) for t in (y, r, dout, dres, scale, post, pre))
    minus = 1.0 if bound else -1.0
    unit, inner, g = y * ny, r * nr, dout * pre
    dr = nr * (g + minus * inner * (g * inner).sum(1, keepdim=True) / d)
    if dres is not None:
        dr = dr + dres
    dp = dr * scale * sg
    u = dp * post
    along = dr * sg * unit
    return dict(dy=ny * (u + minus * unit * (u * unit).sum(1, keepdim=True) / d), dresidual=dr,
                dgate=along * scale * post * (1.0 - sg), dscale=(along * post).sum(0), dpost=(along * scale).sum(0),
                dpre=(dout * inner).sum(0))


def close(name, got, want, mag, roundings):
    """|got - want| <= half a step of got's type + roundings * 2^-24 * mag,
    element by element; NaN and infinities in the same places."""
    got_type, got = got.dtype, f64(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine), "%s: finite in other places" % name
    half = torch.finfo(got_type).eps / 2
    tol = half * want.abs() + roundings * U32 * (1 + half) * mag + torch.finfo(got_type).tiny
    err = (got - want).abs()
    bad = fine & ~(err <= tol)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError("%s: %d of %d out of tolerance, first %s: got %r want %r tolerance %r"
                             % (name, int(bad.sum()), bad.numel(), i, float(got[i]), float(want[i]), float(tol[i])))

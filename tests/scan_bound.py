"""The selective scan and its gradients in 64 bits with, for every result, a
bound on how far the fp32 kernels may be from it.

The bound is carried along with the values (a running error analysis to first
order): every operation adds its own rounding, at most u = 2^-24 of its result
(exp2, reciprocal and square root instructions: 2 u), and hands on the errors
of its operands, so an error decays with the state that it sits in.  With
|v| the size of an argument:

  exp(-|v|)    v log2(e) is off by 2 u |v| (constant, product), exp2 by 2 u:
               (2 |v| + 2) u relative
  softplus(v)  log1p(e) = 2 (q + q^3/3 + ...), q = e / (2 + e): e's error, 6
               operations and the terms left out (below u): (2 |v| + 12) u of
               log1p(e), u of the sum, and dt + bias' own u |v| times sigmoid
  sigmoid(v)   e's error, 1 + e, reciprocal: (2 |v| + 6) u relative
  exp(step A)  the argument is off by 3 u |step A| (A log2(e), the product),
               by A times the step's error; exp2 adds 2 u.  Where cells are
               linked, the argument is A times a cell's sum of steps, formed
               with up to 36 roundings: 40 u |step A| instead of 3 u |step A|
"""
from __future__ import annotations

import torch

from block_ref import F64, U32, f64, sequences


def scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, offsets=None, initial=None, dout=None):
    """(values, bounds): dicts of out, final and, with dout, the gradients."""
    u = U32
    x, dt, A, B, C, D, z, dt_bias, initial, dout = (f64(t) for t in (x, dt, A, B, C, D, z, dt_bias, initial, dout))
    T, ch = x.shape
    G, N = B.shape[1:]
    per = (N + 15) // 16
    pieces = T // 32 + 1 + (1 if offsets is None else offsets.numel() - 1)
    zero = torch.zeros(ch, N, dtype=F64)
    D = torch.zeros(ch, dtype=F64) if D is None else D
    raw = dt if dt_bias is None else dt + dt_bias
    step, sig = torch.logaddexp(raw, torch.zeros_like(raw)), torch.sigmoid(raw)
    tail = torch.log1p(torch.exp(-raw.abs()))
    e_step = u * (tail * (2 * raw.abs() + 12) + step + sig * raw.abs())
    if z is None:
        gate, e_gate = torch.ones_like(x), torch.zeros_like(x)
    else:
        sz = torch.sigmoid(z)
        gate = z * sz
        e_gate = gate.abs() * (2 * z.abs() + 7) * u
    drive = step * x
    e_drive = x.abs() * e_step + u * drive.abs()
    wide = lambda v: v.repeat_interleave(ch // G, 0)  # noqa: E731
    group = lambda v: v.view(G, ch // G, N).sum(1)  # noqa: E731
    seqs = sequences(offsets, T)

    def decay(t):
        arg = step[t][:, None] * A
        a = torch.exp(arg)
        return a, a * (arg.abs() * 40 * u + A.abs() * e_step[t][:, None] + 2 * u)

    inner, e_inner = torch.zeros_like(x), torch.zeros_like(x)
    final, e_final = torch.zeros(len(seqs), ch, N, dtype=F64), torch.zeros(len(seqs), ch, N, dtype=F64)
    hs, e_hs = torch.zeros(T, ch, N, dtype=F64), torch.zeros(T, ch, N, dtype=F64)
    for q, (lo, hi) in enumerate(seqs):
        h, e = (zero if initial is None else initial[q]), zero
        for t in range(lo, hi):
            a, e_a = decay(t)
            b, c = wide(B[t]), wide(C[t])
            add = drive[t][:, None] * b
            e = a * e + e_a * h.abs() + b.abs() * e_drive[t][:, None] + u * add.abs()
            h = a * h + add
            e = e + u * h.abs()
            hs[t], e_hs[t] = h, e
            inner[t] = (h * c).sum(1) + D * x[t]
            e_inner[t] = (c.abs() * e).sum(1) + (per + 6) * u * (h * c).abs().sum(1) + u * (D * x[t]).abs()
        final[q], e_final[q] = h, e
    out = inner * gate
    v = dict(out=out, final=final)
    b_ = dict(out=gate.abs() * e_inner + inner.abs() * e_gate + u * out.abs(), final=e_final)
    if dout is None:
        return v, b_
    gy = dout * gate
    e_gy = dout.abs() * e_gate + u * gy.abs()
    keys = ("dx", "ddt", "dB", "dC", "dA")
    for d in (v, b_):
        d.update(zip(keys, (torch.zeros_like(t) for t in (x, x, B, C, A))), dinitial=torch.zeros_like(final))
    size_A, size_ddt = torch.zeros_like(A), torch.zeros(ch, dtype=F64)
    for q, (lo, hi) in enumerate(seqs):
        back, e_back = zero, zero
        for t in reversed(range(lo, hi)):
            b, c = wide(B[t]), wide(C[t])
            st, e_st, g, e_g = (s[t][:, None] for s in (step, e_step, gy, e_gy))
            dh = back + g * c
            e_dh = e_back + c.abs() * e_g + u * dh.abs()
            v["dC"][t] = group(g * hs[t])
            b_["dC"][t] = group(g.abs() * e_hs[t] + e_g * hs[t].abs() + (ch // G + 16) * u * (g * hs[t]).abs())
            dr, e_dr = drive[t][:, None], e_drive[t][:, None]
            v["dB"][t] = group(dh * dr)
            b_["dB"][t] = group(dr.abs() * e_dh + e_dr * dh.abs() + (ch // G + 16) * u * (dh * dr).abs())
            a, e_a = decay(t)
            back = a * dh
            e_back = a * e_dh + e_a * dh.abs() + u * back.abs()
            if t > lo:
                before, e_before = hs[t - 1], e_hs[t - 1]
            else:
                before, e_before = (zero if initial is None else initial[q]), zero
            flow = back * before
            e_flow = back.abs() * e_before + e_back * before.abs() + u * flow.abs()
            v["dA"] += flow * st
            b_["dA"] += st * e_flow + e_st * flow.abs()
            size_A += (flow * st).abs()
            along, flow_a = (dh * b).sum(1), (flow * A).sum(1)
            e_along = (b.abs() * e_dh).sum(1) + (2 * per + 6) * u * (dh * b).abs().sum(1)
            e_flow_a = (A.abs() * e_flow).sum(1) + (2 * per + 6) * u * (flow * A).abs().sum(1)
            v["dx"][t] = D * gy[t] + step[t] * along
            b_["dx"][t] = (D.abs() * e_gy[t] + e_step[t] * along.abs() + step[t] * e_along
                           + 2 * u * ((D * gy[t]).abs() + (step[t] * along).abs()))
            dstep = flow_a + x[t] * along
            v["ddt"][t] = dstep * sig[t]
            b_["ddt"][t] = (sig[t] * (x[t].abs() * e_along + e_flow_a + u * dstep.abs())
                            + v["ddt"][t].abs() * (3 * raw[t].abs() + 8) * u)
        v["dinitial"][q], b_["dinitial"][q] = back, e_back
    b_["dA"] += (32 + pieces + 8) * u * size_A
    many = (24 + pieces) * u
    v["ddt_bias"] = v["ddt"].sum(0)
    b_["ddt_bias"] = b_["ddt"].sum(0) + many * v["ddt"].abs().sum(0)
    v["dD"] = (gy * x).sum(0)
    b_["dD"] = (e_gy * x.abs()).sum(0) + many * (gy * x).abs().sum(0)
    if z is not None:
        slope = sz * (1 + z * (1 - sz))
        e_slope = sz * (z.abs() * (sz * (2 * z.abs() + 6) + 1) + 1 + z.abs()) * u + slope.abs() * (2 * z.abs() + 7) * u
        v["dz"] = dout * inner * slope
        b_["dz"] = dout.abs() * (slope.abs() * e_inner + inner.abs() * e_slope) + 3 * u * v["dz"].abs()
    return v, b_


def close(name, got, want, bound):
    """|got - want| <= half a step of got's type + bound (to second order, 1 +
    2^-6), element by element."""
    kind, got = got.dtype, f64(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    half = torch.finfo(kind).eps / 2
    # below the smallest normal number a result may be rounded to a step of that
    tol = half * want.abs() + (1 + half) * (1 + 2.0 ** -6) * bound + torch.finfo(kind).tiny
    err = (got - want).abs()
    bad = ~(err <= tol)
    if bad.any():
        i = tuple(int(k) for k in bad.nonzero()[0])
        raise AssertionError("%s: %d of %d out of tolerance, first %s: got %r want %r tolerance %r, worst %.3g of its tolerance"
                             % (name, int(bad.sum()), bad.numel(), i, float(got[i]), float(want[i]), float(tol[i]),
                                float((err / tol).nan_to_num(nan=float("inf")).max())))

"""The gated delta rule from its formula in 64 bits, one token after another, on
the CPU, with the sizes that its errors are measured by.

A column c of a head's state goes its own way: S'[:, c] = exp(g) S[:, c], then
(1 - beta k k^T) S' + beta v_c k.  With exp(g) <= 1 and beta |k|^2 <= 2 no step
makes a column's error longer, so what a chunk of 64 rows adds to it stays as
it is or shrinks: after n chunks it is at most n times what one adds, a few
roundings eps of the column's longest length so far, M_c = max |S[:, c]| + max
|v_c|.  Backwards the same holds of the columns of the state's gradient, N_c.
Results are sums of such columns: their bounds below are those sums with M_c
and N_c in the columns' place.

Roundings of a chunk: eight products on the way of a value (k S, the inverse
and its blocks, its product with what is left, beta, the scores' two products,
k^T u), each off by `eps` of its terms' lengths, times up to 4 for the length of
the inverse (1 + a diag(beta))^-1.  eps is 2^-17 where products take two fp16
planes of a number, which hold it to 2^-22 if it is 2^-17 or more of the largest
of its tiles and to 2^-39 of that largest otherwise: 64 and more such terms of a
column are off by less than 2^-17 of its length.  In fp32 products sum up to
key_dim + 64 terms, each off by 2^-24."""
from __future__ import annotations

import torch

from block_ref import F64, U32, f64, sequences

PER_CHUNK = 32.0


def step_of(dtype, key_dim):
    return (key_dim + 64) * U32 if dtype == torch.float32 else 2.0 ** -17


def unit(v, normalize, eps):
    return v / torch.sqrt(v.square().sum(-1, keepdim=True) + eps) if normalize else v


def unit_grad(v, d, normalize, eps):
    if not normalize:
        return d
    m = v.square().sum(-1, keepdim=True) + eps
    return d / m.sqrt() - v * (v * d).sum(-1, keepdim=True) / m ** 1.5


def delta(q, k, v, g, beta, scale=None, normalize=False, eps=1e-6, offsets=None, initial=None, dout=None, dfinal=None,
          dtype=torch.float32, chunk=64):
    """(results, bounds): out, final and, with dout, the gradients."""
    q_in, k_in, v, g, beta, initial, dout, dfinal = (f64(t) for t in (q, k, v, g, beta, initial, dout, dfinal))
    T, KH, dk = q_in.shape
    _, H, dv = v.shape
    scale = dk ** -0.5 if scale is None else scale
    g = torch.where(g < -512.0, torch.full_like(g, -512.0), g)
    q, k = (unit(t, normalize, eps).repeat_interleave(H // KH, 1) for t in (q_in, k_in))
    seqs = sequences(offsets, T)
    out, out_b = torch.zeros_like(v), torch.zeros_like(v)
    final = torch.zeros(len(seqs), H, dk, dv, dtype=F64) if initial is None else initial.clone()
    final_b = torch.zeros_like(final)
    step = PER_CHUNK * step_of(dtype, dk)
    names = ("dq", "dk", "dv", "dg", "dbeta")
    like = (q, k, v, g, beta)
    r, b = ({n: torch.zeros_like(t) for n, t in zip(names, like)} for _ in range(2))
    r["dinitial"], b["dinitial"] = torch.zeros_like(final), torch.zeros_like(final)
    for i, (lo, hi) in enumerate(seqs):
        S = final[i]
        M = S.norm(dim=1)
        if hi > lo:
            M = M + v[lo:hi].abs().amax(0)
        held, us = [], []
        for t in range(lo, hi):
            S = torch.exp(g[t])[:, None, None] * S
            held.append(S)
            u = v[t] - torch.einsum("hkv,hk->hv", S, k[t])
            us.append(u)
            S = S + torch.einsum("hk,hv->hkv", k[t], beta[t][:, None] * u)
            M = torch.maximum(M, S.norm(dim=1))
            out[t] = scale * torch.einsum("hkv,hk->hv", S, q[t])
        final[i] = S
        n = -(-(hi - lo) // chunk) + 1
        out_b[lo:hi] = step * n * scale * q[lo:hi].norm(dim=2)[..., None] * M
        final_b[i] = (step * n if hi > lo else 0.0) * M[:, None, :]
        if dout is None:
            continue
        D = torch.zeros_like(S) if dfinal is None else dfinal[i]
        N = D.norm(dim=1)
        if hi > lo:
            N = N + scale * (q[lo:hi].norm(dim=2)[..., None] * dout[lo:hi].abs()).amax(0)
        for t in reversed(range(lo, hi)):
            before, u = held[t - lo], us[t - lo]
            bu = beta[t][:, None] * u
            r["dq"][t] = scale * torch.einsum("hkv,hv->hk", before + torch.einsum("hk,hv->hkv", k[t], bu), dout[t])
            D = D + scale * torch.einsum("hk,hv->hkv", q[t], dout[t])
            N = torch.maximum(N, D.norm(dim=1))
            du = torch.einsum("hkv,hk->hv", D, k[t])
            r["dbeta"][t] = (du * u).sum(1)
            r["dv"][t] = beta[t][:, None] * du
            r["dk"][t] = torch.einsum("hkv,hv->hk", D, bu) - torch.einsum("hkv,hv->hk", before, r["dv"][t])
            D = D - torch.einsum("hk,hv->hkv", k[t], r["dv"][t])
            r["dg"][t] = (D * before).sum((1, 2))
            D = torch.exp(g[t])[:, None, None] * D
        r["dinitial"][i] = D
        if hi == lo:
            continue
        # u is at most |v| + |k| |S|, and so 2 M; every term has an error of a state's
        # and of a gradient's column
        both = (N * M).sum(1)
        b["dinitial"][i] = step * n * N[:, None, :]
        b["dv"][lo:hi] = step * n * N
        b["dq"][lo:hi] = step * n * scale * ((dout[lo:hi].abs() * M).sum(2))[..., None]
        b["dk"][lo:hi] = (8.0 * step * n * both)[:, None]
        b["dbeta"][lo:hi] = 4.0 * step * n * both
        b["dg"][lo:hi] = 2.0 * step * n * both
    res, bound = dict(out=out, final=final), dict(out=out_b, final=final_b)
    if dout is None:
        return res, bound
    for name, raw in (("dq", q_in), ("dk", k_in)):
        per = lambda t: t.view(T, KH, H // KH, dk).sum(2)  # noqa: E731
        r[name], b[name] = unit_grad(raw, per(r[name]), normalize, eps), per(b[name])
        if normalize:  # the projection adds its own products; both by the length of the input
            b[name] = b[name] * (1.0 + dk ** 0.5) / torch.sqrt(raw.square().sum(-1, keepdim=True) + eps)
    res.update(r)
    bound.update(b)
    return res, bound


def delta_step(q, k, v, state, g, beta, scale=None, normalize=False, eps=1e-6, slots=None, dtype=torch.float32):
    """out and the whole new state; a slot outside the pool reads zeros."""
    pool = state.shape[0]
    at = list(range(q.shape[0])) if slots is None else slots.cpu().tolist()
    new = f64(state).clone()
    out, out_b, new_b = torch.zeros(v.shape, dtype=F64), torch.zeros(v.shape, dtype=F64), torch.zeros_like(new)
    for i, slot in enumerate(at):
        held = 0 <= slot < pool
        row = slice(i, i + 1)
        r, b = delta(q[row], k[row], v[row], g[row], beta[row], scale, normalize, eps, None,
                     f64(state)[slot:slot + 1] if held else None, dtype=dtype)
        out[i], out_b[i] = r["out"][0], b["out"][0]
        if held:
            new[slot], new_b[slot] = r["final"][0], b["final"][0]
    return dict(out=out, state=new), dict(out=out_b, state=new_b)


def close(name, got, want, bound):
    """|got - want| <= half a step of got's type + bound, element by element;
    NaN and infinities in the same places."""
    kind, got = got.dtype, f64(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine), "%s: finite in other places" % name
    half = torch.finfo(kind).eps / 2
    tol = half * want.abs() + (1 + half) * bound + torch.finfo(kind).tiny
    bad = fine & ~((got - want).abs() <= tol)
    if bad.any():
        at = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError("%s: %d of %d out of tolerance, first %s: got %r want %r tolerance %r"
                             % (name, int(bad.sum()), bad.numel(), at, float(got[at]), float(want[at]), float(tol[at])))

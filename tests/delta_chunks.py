"""The gated delta rule by chunks of 64 rows, in 64 bits on the CPU: the formulas that
the kernels work by (csrc/delta_block.hpp, delta_back.hpp), one term at a time.

`drop` leaves a term out and `planes` holds what a chunk computes (states, their
gradients, corrections, inverses, scores, triangles) in so many fp16 planes of a
common power of two: mistakes that a test of the kernels has to see."""
from __future__ import annotations

import torch

from block_ref import F64, f64, sequences
from delta_ref import unit, unit_grad

CHUNK = 64
# a result and the terms of its formula
TERMS = {
    "out": ("out_state", "out_scores"),
    "final": ("state_decayed", "state_new"),
    "dq": ("dq_state", "dq_pairs"),
    "dk": ("dk_state", "dk_end", "dk_row", "dk_query", "dk_column"),
    "dv": ("du_state", "du_scores"),
    "dbeta": ("dbeta",),
    "dg": ("dg_pairs", "dg_query", "dg_key", "dg_end", "dg_whole"),
    "dinitial": ("d_decayed", "d_query", "d_key"),
}


def hold(t, planes):
    if planes is None:
        return t
    most = t.abs().amax(dim=(-2, -1), keepdim=True).clamp(min=2.0 ** -60)
    by = torch.ldexp(torch.ones_like(most), 15 - torch.frexp(most)[1])
    kept, rest = torch.zeros_like(t), t * by
    for _ in range(planes):
        plane = rest.to(torch.float16).to(F64)
        kept, rest = kept + plane, rest - plane
    return kept / by


def delta(q, k, v, g, beta, scale=None, normalize=False, eps=1e-6, offsets=None, initial=None, dout=None, dfinal=None,
          drop=None, planes=None):
    """out, final and the gradients."""
    q_in, k_in, v, g, beta, initial, dout, dfinal = (f64(t) for t in (q, k, v, g, beta, initial, dout, dfinal))
    T, KH, K = q_in.shape
    _, H, V = v.shape
    scale = K ** -0.5 if scale is None else scale
    g = torch.clamp(g, min=-512.0)
    q, k = (unit(t, normalize, eps).repeat_interleave(H // KH, 1) for t in (q_in, k_in))
    is_ = lambda name: 0.0 if name == drop else 1.0  # noqa: E731
    h = lambda t: hold(t, planes)  # noqa: E731
    mT = lambda t: t.transpose(-1, -2)  # noqa: E731
    seqs = sequences(offsets, T)
    r = dict(out=torch.zeros_like(v), final=torch.zeros(len(seqs), H, K, V, dtype=F64), dq=torch.zeros_like(q),
             dk=torch.zeros_like(k), dv=torch.zeros_like(v), dg=torch.zeros_like(g), dbeta=torch.zeros_like(g),
             dinitial=torch.zeros(len(seqs), H, K, V, dtype=F64))
    for i, (lo, hi) in enumerate(seqs):
        S = torch.zeros(H, K, V, dtype=F64) if initial is None else initial[i]
        kept = []
        for at in range(lo, hi, CHUNK):
            rows = slice(at, min(at + CHUNK, hi))
            Q, Kc, Vc = (t[rows].transpose(0, 1) for t in (q, k, v))
            b, G = beta[rows].t()[..., None], g[rows].t().cumsum(-1)
            e, tail, whole = torch.exp(G)[..., None], torch.exp(G[..., -1:] - G)[..., None], torch.exp(G[..., -1:])[..., None]
            between = torch.tril(torch.exp(torch.tril(G[..., :, None] - G[..., None, :])))
            a = torch.tril(between * (Kc @ mT(Kc)), -1)
            P = scale * between * (Q @ mT(Kc))
            one = torch.eye(Q.shape[1], dtype=F64)
            rho = h(torch.linalg.inv(one + a * mT(b))) @ h(Vc - e * (Kc @ h(S)))
            U = b * rho
            r["out"][rows] = (is_("out_state") * scale * e * (Q @ h(S)) + is_("out_scores") * (h(P) @ h(U))).transpose(0, 1)
            kept.append((rows, Q, Kc, b, e, tail, whole, between, a, P, S, rho, U))
            S = is_("state_decayed") * whole * S + is_("state_new") * (mT(Kc) @ h(tail * U))
        r["final"][i] = S
        if dout is None:
            continue
        D = torch.zeros_like(S) if dfinal is None else dfinal[i]
        for rows, Q, Kc, b, e, tail, whole, between, a, P, S, rho, U in reversed(kept):
            dO = dout[rows].transpose(0, 1)
            dU = is_("du_scores") * (mT(h(P)) @ dO) + is_("du_state") * tail * (Kc @ h(D))
            one = torch.eye(Q.shape[1], dtype=F64)
            omega = mT(h(torch.linalg.inv(one + b * a))) @ h(dU)
            dR = b * omega
            r["dv"][rows] = dR.transpose(0, 1)
            r["dbeta"][rows] = is_("dbeta") * (rho * omega).sum(-1).t()
            dqk = scale * between * (dO @ mT(h(rho) * b))
            dkk = -torch.tril(between, -1) * ((b * h(omega)) @ mT(h(rho) * b))
            query, key = scale * e * (dO @ mT(h(S))), e * (b * (h(omega) @ mT(h(S))))
            end = tail * (b * (h(rho) @ mT(h(D))))
            r["dq"][rows] = (is_("dq_state") * query + is_("dq_pairs") * (h(dqk) @ Kc)).transpose(0, 1)
            r["dk"][rows] = (-is_("dk_state") * key + is_("dk_end") * end + is_("dk_row") * (h(dkk) @ Kc)
                             + is_("dk_query") * (mT(h(dqk)) @ Q) + is_("dk_column") * (mT(h(dkk)) @ Kc)).transpose(0, 1)
            # z_ij holds the g of the rows t with j < t <= i
            z = dqk * (Q @ mT(Kc)) + dkk * (Kc @ mT(Kc))
            n = z.shape[-1]
            before = torch.cat([torch.zeros_like(z[..., :1]), z.cumsum(-1)[..., :-1]], -1)
            dg = is_("dg_pairs") * torch.tril(before).sum(-2)
            after = is_("dg_query") * (Q * query).sum(-1) - is_("dg_key") * (Kc * key).sum(-1)
            dg = dg + after.flip(-1).cumsum(-1).flip(-1)
            ends = (Kc * end).sum(-1).cumsum(-1)
            dg = dg + is_("dg_end") * torch.cat([torch.zeros_like(ends[..., :1]), ends[..., :n - 1]], -1)
            r["dg"][rows] = (dg + is_("dg_whole") * whole[..., 0] * (S * D).sum((1, 2))[:, None]).t()
            D = (is_("d_decayed") * whole * D + is_("d_query") * (mT(Q) @ (scale * e * dO))
                 - is_("d_key") * (mT(Kc) @ h(e * dR)))
        r["dinitial"][i] = D
    if dout is None:
        return dict(out=r["out"], final=r["final"])
    for name, raw in (("dq", q_in), ("dk", k_in)):
        r[name] = unit_grad(raw, r[name].view(T, KH, H // KH, K).sum(2), normalize, eps)
    return r

"""Layer norm and its gradients from their formulas in 64 bits, on the CPU.

`bound=True` gives the sizes that rounding errors grow with: a difference from
the mean is off by a rounding of x and of the mean, which is a sum of all
channels (`lift`), and the reciprocal deviation by the mean of what its squares
are off by (`tilt`, relative to it)."""
from __future__ import annotations

import torch

from block_ref import f64


def layer_norm(x, weight=None, bias=None, eps=1e-5, dout=None, bound=False):
    """out and, with dout, dx, dweight and dbias."""
    x, weight, bias, dout = (f64(t) for t in (x, weight, bias, dout))
    d = x.shape[1]
    w = torch.ones(d, dtype=x.dtype) if weight is None else weight
    b = torch.zeros(d, dtype=x.dtype) if bias is None else bias
    c = x - x.sum(1, keepdim=True) / d
    r = torch.rsqrt(c.square().sum(1, keepdim=True) / d + eps)
    n = c * r
    if bound:
        lift = x.abs() + x.abs().sum(1, keepdim=True) / d + c.abs()
        tilt = (c.abs() * lift).sum(1, keepdim=True) / d * r * r
        n, w, b = lift * r + n.abs() * tilt, w.abs(), b.abs()
    res = dict(out=n * w + b)
    if dout is None:
        return res
    if not bound:
        g = dout * w
        res["dx"] = r * (g - g.sum(1, keepdim=True) / d - n * (g * n).sum(1, keepdim=True) / d)
        res["dweight"] = (dout * n).sum(0)
    else:
        g, size = dout.abs() * w, (c * r).abs()
        along = lambda v: (g * v).sum(1, keepdim=True) / d  # noqa: E731
        res["dx"] = r * (1.0 + tilt) * (g + g.sum(1, keepdim=True) / d + n * along(size) + size * along(n))
        res["dweight"] = (dout.abs() * n).sum(0)
    res["dbias"] = (dout.abs() if bound else dout).sum(0)
    return res

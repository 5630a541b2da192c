"""The operators of a state space block, in their plain form and through the library.

Three operators work on tokens packed one sequence after another (row t is
a token, offsets[s] .. offsets[s + 1] are the rows of sequence s), for
prompts, for training and for single tokens:

  conv   a short causal convolution over each channel's own past
  scan   the selective scan h[t] = exp(dt[t] A) h[t-1] + dt[t] B[t] x[t],
         y[t] = C[t] h[t] + D x[t], gated by silu(z)
  norm   the norm after a block, its gate, the residual scale and sum, and
         the norm before the next block

``run`` computes a case with elementary torch operations in 32 bits, or
through the library where ``own`` is set; ``exact`` computes it from the
definition in 64 bits, one token after another.
"""
import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a serving step's prompts of mixed lengths, before they are scanned
        dict(name="conv_prompts", op="conv", tokens=16384, seqs=13, channels=4096, width=4, dtype="bf16", state=True),
        # training on documents packed into one row; channels that are no multiple of a vector
        dict(name="conv_train_odd", op="conv_train", tokens=6001, seqs=5, channels=1537, width=3, dtype="fp32", state=False),
        # one new token for each of many sequences in flight
        dict(name="conv_step_many", op="conv_step", batch=384, pool=512, channels=8192, width=4, dtype="bf16"),
        # one long prompt, the case with the fewest rows to work on
        dict(name="scan_prompt_long", op="scan", tokens=8191, seqs=1, channels=4096, states=16, groups=1, dtype="bf16", state=False),
        # prompts that go on from earlier states, of lengths from zero up
        dict(name="scan_prompts_ragged", op="scan", tokens=16384, seqs=41, channels=2048, states=16, groups=1, dtype="fp16", state=True),
        # a training step: forward, then every gradient
        dict(name="scan_train", op="scan_train", tokens=8192, seqs=4, channels=2048, states=16, groups=1, dtype="bf16", state=False),
        # the same with many states, grouped B and C, 32 bits and an odd number of tokens
        dict(name="scan_train_states", op="scan_train", tokens=1023, seqs=3, channels=768, states=64, groups=4, dtype="fp32", state=True),
        # one token of one sequence: latency
        dict(name="scan_step_one", op="scan_step", batch=1, pool=4, channels=1536, states=16, groups=1, dtype="bf16"),
        # one token for each of many sequences: the states' traffic
        dict(name="scan_step_many", op="scan_step", batch=384, pool=512, channels=4096, states=16, groups=1, dtype="bf16"),
        # prompts through the norms around a block
        dict(name="norm_prompts", op="norm", tokens=16384, channels=4096, dtype="bf16", residual="bf16"),
        # their gradients, the residual stream in 32 bits
        dict(name="norm_train", op="norm_train", tokens=8192, channels=5120, dtype="bf16", residual="fp32"),
        # a few decoded tokens: latency
        dict(name="norm_step", op="norm", tokens=3, channels=2048, dtype="fp16", residual="fp16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["conv", "conv_train", "conv_step", "scan", "scan_train", "scan_step", "norm", "norm_train"])
        d = _log_int(rng, 40, 8192)
        if rng.random() < 0.6:
            d = max(8, d // 8 * 8)
        t = _log_int(rng, 1, 16384)
        case = dict(op=op, channels=d, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
        if op.endswith("_step"):
            b = _log_int(rng, 1, 512)
            case.update(batch=b, pool=b + rng.randrange(0, 9))
        else:
            case.update(tokens=t)
        if op.startswith("conv"):
            case.update(width=rng.choice([2, 3, 4, 4, 5]))
        elif op.startswith("scan"):
            groups = rng.choice([1, 1, 2, 4])
            case.update(channels=d // groups * groups, states=rng.choice([4, 8, 16, 16, 16, 24, 32, 64]), groups=groups)
        else:
            case.update(residual=rng.choice([case["dtype"], "fp32"]))
        if op in ("conv", "conv_train", "scan", "scan_train"):
            case.update(seqs=_log_int(rng, 1, 64), state=rng.random() < 0.5)
        if _cost(case) <= most and case.get("states", 1) * d * case.get("tokens", 1) <= (1 << 29) // (2 if "train" in op else 1):
            return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _offsets(tokens, seqs, seed):
    """Random cuts of the packed rows: lengths differ, some are zero or one."""
    g = torch.Generator().manual_seed(seed * 7919 + 17)
    cuts = torch.randint(0, tokens + 1, (seqs - 1,), generator=g).tolist()
    if seqs > 8 and tokens > 8:
        cuts[0], cuts[1] = cuts[2], min(cuts[2] + 1, tokens)  # an empty sequence and one of a single token, as a rule
    return torch.tensor([0] + sorted(cuts) + [tokens], dtype=torch.int32, device=DEVICE)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, mean=0.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=DEVICE) * scale + mean).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=g, device=DEVICE) * (hi - lo) + lo

    op, d, f32 = case["op"], case["channels"], torch.float32
    s = dict(case=case)
    if op.endswith("_step"):
        order = torch.randperm(case["pool"], generator=g, device=DEVICE)
        rows = (case["batch"],)
        s["slots"] = order[:case["batch"]].to(torch.int32)
    else:
        rows = (case["tokens"],)
    if "seqs" in case:
        s["offsets"] = _offsets(case["tokens"], case["seqs"], seed)
    if op.startswith("conv"):
        w = case["width"]
        s.update(x=normal(*rows, d), weight=normal(d, w, scale=w ** -0.5, dtype=f32), bias=normal(d, scale=0.1, dtype=f32))
        if op == "conv_step":
            s["state"] = normal(case["pool"], w - 1, d)
            s["new_state"] = s["state"].clone()
        elif case["state"]:
            s["initial"] = normal(case["seqs"], w - 1, d)
        if op == "conv_train":
            s["dout"] = normal(*rows, d)
    elif op.startswith("scan"):
        n, groups = case["states"], case["groups"]
        step = torch.exp(uniform(d, lo=math.log(1e-3), hi=math.log(1e-1)))
        s.update(x=normal(*rows, d), dt=normal(*rows, d), z=normal(*rows, d),
                 B=normal(*rows, groups, n), C=normal(*rows, groups, n),
                 A=-(torch.arange(1, n + 1, device=DEVICE, dtype=f32) * uniform(d, 1, lo=0.8, hi=1.2)).contiguous(),
                 D=normal(d, scale=0.1, mean=1.0, dtype=f32),
                 dt_bias=step + torch.log(-torch.expm1(-step)))
        if op == "scan_step":
            s["state"] = normal(case["pool"], d, n, dtype=f32)
            s["new_state"] = s["state"].clone()
        elif case["state"]:
            s["initial"] = normal(case["seqs"], d, n, dtype=f32)
        if op == "scan_train":
            s["dout"] = normal(*rows, d)
    else:
        rt = TYPES[case["residual"]]
        s.update(y=normal(*rows, d) * torch.exp(uniform(rows[0], 1, lo=-1.0, hi=1.0)).to(dt), gate=normal(*rows, d),
                 residual=normal(*rows, d, scale=2.0, dtype=rt), scale=normal(d, scale=0.1, mean=0.5, dtype=f32),
                 post=normal(d, scale=0.1, mean=1.0, dtype=f32), pre=normal(d, scale=0.1, mean=1.0, dtype=f32))
        if op == "norm_train":
            s.update(dresidual=normal(*rows, d, dtype=rt), dout=normal(*rows, d))
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _dsilu(v):
    s = _sigmoid(v)
    return s * (1.0 + v * (1.0 - s))


def _softplus(v):
    return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-torch.abs(v)))


def _places(offsets, tokens):
    """The sequence of each packed row and the row's place in it."""
    t = torch.arange(tokens, device=offsets.device)
    seq = torch.searchsorted(offsets[1:].long(), t, right=True)
    return seq, t - offsets.long()[seq]


def _past(x, shift, seq, pos, initial):
    """x[t - shift] within the row's sequence, from `initial` (the rows
    before the sequence, oldest first) or zero where that lies before it."""
    t = torch.arange(x.shape[0], device=x.device)
    inside = pos >= shift
    got = x[torch.clamp(t - shift, min=0)]
    before = torch.zeros_like(got)
    if initial is not None and initial.shape[1] > 0:
        at = torch.clamp(initial.shape[1] + pos - shift, 0, initial.shape[1] - 1)
        before = initial[seq, at]
    return torch.where(inside[:, None], got, before)


def _conv_pre(s):
    x, w = s["x"].float(), s["weight"]
    initial = s["initial"].float() if "initial" in s else None
    seq, pos = _places(s["offsets"], x.shape[0])
    width = w.shape[1]
    taps = [_past(x, width - 1 - k, seq, pos, initial) for k in range(width)]
    pre = s["bias"] + sum(w[:, k] * taps[k] for k in range(width))
    return pre, taps, seq, pos


def _conv_final(s):
    x, width = s["x"], s["weight"].shape[1]
    off = s["offsets"].long()
    lens = off[1:] - off[:-1]
    rows = []
    for j in range(width - 1):
        p = lens - (width - 1) + j
        got = x[torch.clamp(off[:-1] + p, 0, x.shape[0] - 1)]
        before = torch.zeros_like(got)
        if "initial" in s:
            before = s["initial"][torch.arange(len(lens), device=x.device), torch.clamp(width - 1 + p, 0, width - 2)]
        rows.append(torch.where((p >= 0)[:, None], got, before))
    return torch.stack(rows, 1)


def _plain_conv(s):
    pre = _conv_pre(s)[0]
    return dict(out=_silu(pre).to(s["x"].dtype), final=_conv_final(s))


def _plain_conv_train(s):
    x, w = s["x"], s["weight"]
    pre, taps, seq, pos = _conv_pre(s)
    width, tokens = w.shape[1], x.shape[0]
    off = s["offsets"].long()
    g = s["dout"].float() * _dsilu(pre)
    dx = torch.zeros_like(g)
    t = torch.arange(tokens, device=x.device)
    left = off[1:][seq] - t  # rows from t to the end of its sequence
    for k in range(width):
        shift = width - 1 - k
        dx += torch.where((left > shift)[:, None], w[:, k] * g[torch.clamp(t + shift, max=tokens - 1)], torch.zeros_like(g))
    r = dict(out=_silu(pre).to(x.dtype), dx=dx.to(x.dtype), dweight=torch.stack([(g * taps[k]).sum(0) for k in range(width)], 1), dbias=g.sum(0))
    if "initial" in s:
        d = torch.zeros(len(off) - 1, width - 1, x.shape[1], device=x.device)
        for k in range(width):
            shift = width - 1 - k
            for p in range(min(shift, tokens)):
                has = (off[1:] - off[:-1]) > p
                at = torch.clamp(off[:-1] + p, max=tokens - 1)
                d[:, width - 1 + p - shift] += torch.where(has[:, None], w[:, k] * g[at], torch.zeros_like(g[at]))
        r["dinitial"] = d.to(x.dtype)
    return r


def _plain_conv_step(s):
    at = s["slots"].long()
    window = torch.cat([s["state"][at], s["x"][:, None]], 1)
    pre = s["bias"] + (window.float() * s["weight"].t()[None]).sum(1)
    s["new_state"][at] = window[:, 1:]
    return dict(out=_silu(pre).to(s["x"].dtype), state=s["new_state"])


def _recur(a, b):
    """h[t] = a[t] h[t-1] + b[t] along the first axis, h[-1] = 0: pieces of
    rows side by side, then from piece to piece.  Works in b's memory."""
    t = b.shape[0]
    q = max(1, int(t ** 0.5))
    m = -(-t // q)
    if m * q > t:
        pad = torch.zeros((m * q - t,) + b.shape[1:], dtype=b.dtype, device=b.device)
        a, b = torch.cat([a, pad]), torch.cat([b, pad])
    else:
        a = a.clone()
    A, H = a.view((m, q) + a.shape[1:]), b.view((m, q) + b.shape[1:])
    for i in range(1, q):
        H[:, i] += A[:, i] * H[:, i - 1]
        A[:, i] *= A[:, i - 1]
    for j in range(1, m):
        H[j] += A[j] * H[j - 1, -1]
    return H.view((m * q,) + b.shape[1:])[:t]


def _channels(v, d):
    """[T, G, N] as one row of states for each of the d channels."""
    t, groups, n = v.shape
    return v.float()[:, :, None, :].expand(t, groups, d // groups, n).reshape(t, d, n)


def _scan_parts(s):
    x = s["x"].float()
    tokens, d = x.shape
    raw = s["dt"].float() + s["dt_bias"]
    step = _softplus(raw)
    decay = torch.exp(step[:, :, None] * s["A"])
    drive = (step * x)[:, :, None] * _channels(s["B"], d)
    off = s["offsets"].long()
    begins = off[:-1][off[1:] > off[:-1]]
    seqs = torch.nonzero(off[1:] > off[:-1])[:, 0]
    if "initial" in s:
        drive[begins] += decay[begins] * s["initial"][seqs]
    keep = decay.clone()
    keep[begins] = 0.0
    h = _recur(keep, drive)
    return x, raw, step, decay, h, begins, seqs, off


def _scan_out(s, h, x):
    inner = (h * _channels(s["C"], x.shape[1])).sum(-1) + s["D"] * x
    return inner, (inner * _silu(s["z"].float())).to(s["x"].dtype)


def _scan_final(s, h, off, seqs):
    final = s["initial"].clone() if "initial" in s else torch.zeros((len(off) - 1,) + h.shape[1:], device=h.device)
    final[seqs] = h[off[1:][seqs] - 1]
    return final


def _plain_scan(s):
    x, _, _, _, h, _, seqs, off = _scan_parts(s)
    return dict(out=_scan_out(s, h, x)[1], final=_scan_final(s, h, off, seqs))


def _plain_scan_train(s):
    x, raw, step, decay, h, begins, seqs, off = _scan_parts(s)
    d, groups = x.shape[1], s["B"].shape[1]
    inner, out = _scan_out(s, h, x)
    z, dout = s["z"].float(), s["dout"].float()
    gy = dout * _silu(z)
    r = dict(out=out, dz=(dout * inner * _dsilu(z)).to(out.dtype), dD=(gy * x).sum(0))
    r["dC"] = (gy[:, :, None] * h).view(h.shape[0], groups, d // groups, -1).sum(2).to(out.dtype)
    # dh[t] = C[t] gy[t] + decay[t + 1] dh[t + 1], backwards through each sequence
    follow = torch.zeros_like(decay)
    follow[:-1] = decay[1:]
    follow[off[1:][seqs] - 1] = 0.0
    dh = _recur(follow.flip(0), (gy[:, :, None] * _channels(s["C"], d)).flip(0)).flip(0)
    del follow
    before = torch.zeros_like(h)
    before[1:] = h[:-1]
    before[begins] = s["initial"][seqs] if "initial" in s else 0.0
    flow = dh * before * decay
    r["dA"] = (flow * step[:, :, None]).sum(0)
    along = (dh * _channels(s["B"], d)).sum(-1)
    r["dx"] = (s["D"] * gy + step * along).to(out.dtype)
    ddt = ((flow * s["A"]).sum(-1) + x * along) * _sigmoid(raw)
    r["ddt"], r["ddt_bias"] = ddt.to(out.dtype), ddt.sum(0)
    r["dB"] = (dh * (step * x)[:, :, None]).view(h.shape[0], groups, d // groups, -1).sum(2).to(out.dtype)
    if "initial" in s:
        r["dinitial"] = torch.zeros_like(s["initial"])
        r["dinitial"][seqs] = (decay * dh)[begins]
    return r


def _plain_scan_step(s):
    at = s["slots"].long()
    x = s["x"].float()
    step = _softplus(s["dt"].float() + s["dt_bias"])
    h = torch.exp(step[:, :, None] * s["A"]) * s["state"][at] + (step * x)[:, :, None] * _channels(s["B"], x.shape[1])
    s["new_state"][at] = h
    return dict(out=_scan_out(s, h, x)[1], state=s["new_state"])


def _norm_parts(s):
    y, z = s["y"].float(), s["gate"].float()
    ry = 1.0 / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS)
    return y, z, ry, y * ry * s["post"]


def _plain_norm(s):
    y, z, ry, p = _norm_parts(s)
    r = s["residual"].float() + s["scale"] * _sigmoid(z) * p
    rr = 1.0 / torch.sqrt((r * r).mean(-1, keepdim=True) + EPS)
    return dict(residual=r.to(s["residual"].dtype), out=(r * rr * s["pre"]).to(s["y"].dtype))


def _plain_norm_train(s):
    # s["residual"] is the sum that the forward pass gave
    y, z, ry, p = _norm_parts(s)
    r, dout = s["residual"].float(), s["dout"].float()
    rr = 1.0 / torch.sqrt((r * r).mean(-1, keepdim=True) + EPS)
    wd = s["pre"] * dout
    dr = s["dresidual"].float() + rr * (wd - r * rr * rr * (wd * r).mean(-1, keepdim=True))
    sg = _sigmoid(z)
    q = s["scale"] * dr
    dp = q * sg
    wp = s["post"] * dp
    dy = ry * (wp - y * ry * ry * (wp * y).mean(-1, keepdim=True))
    t = s["y"].dtype
    return dict(dy=dy.to(t), dresidual=dr.to(s["residual"].dtype), dgate=(q * p * sg * (1.0 - sg)).to(t), dscale=(dr * sg * p).sum(0),
                dpost=(dp * y * ry).sum(0), dpre=(dout * r * rr).sum(0))


PLAIN = dict(conv=_plain_conv, conv_train=_plain_conv_train, conv_step=_plain_conv_step, scan=_plain_scan, scan_train=_plain_scan_train,
             scan_step=_plain_scan_step, norm=_plain_norm, norm_train=_plain_norm_train)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own(s):
    import device_wide_prefix_chained_amd as dw
    op, x, offsets, initial = s["case"]["op"], s.get("x"), s.get("offsets"), s.get("initial")
    if op == "conv":
        final = torch.empty(s["case"]["seqs"], s["case"]["width"] - 1, x.shape[1], dtype=x.dtype, device=x.device)
        out = dw.ps_causal_conv(x, s["weight"], s["bias"], offsets=offsets, initial=initial, final=final)
        return dict(out=out, final=final)
    if op == "conv_train":
        out = dw.ps_causal_conv(x, s["weight"], s["bias"], offsets=offsets, initial=initial)
        g = dw.ps_causal_conv_bwd(x, s["weight"], s["dout"], s["bias"], offsets=offsets, initial=initial)
        r = dict(out=out, dx=g.dx, dweight=g.dweight, dbias=g.dbias)
        if initial is not None:
            r["dinitial"] = g.dinitial
        return r
    if op == "conv_step":
        out = dw.ps_causal_conv_step(x, s["state"], s["weight"], s["bias"], slots=s["slots"], new_state=s["new_state"])
        return dict(out=out, state=s["new_state"])
    if op.startswith("scan"):
        block = (x, s["dt"], s["A"], s["B"], s["C"])
        more = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
    if op == "scan":
        final = torch.empty(s["case"]["seqs"], x.shape[1], s["case"]["states"], dtype=torch.float32, device=x.device)
        out = dw.ps_selective_scan(*block, **more, offsets=offsets, initial=initial, final=final)
        return dict(out=out, final=final)
    if op == "scan_train":
        rows = dw.ps_selective_scan_checkpoint_rows(x.shape[0], s["case"]["states"])
        kept = torch.empty(rows, x.shape[1], s["case"]["states"], dtype=torch.float32, device=x.device)
        out = dw.ps_selective_scan(*block, **more, offsets=offsets, initial=initial, checkpoints=kept)
        g = dw.ps_selective_scan_bwd(*block, s["dout"], kept, **more, offsets=offsets, initial=initial)
        r = dict(out=out, dz=g.dz, dD=g.dD, dC=g.dC, dA=g.dA, dx=g.dx, ddt=g.ddt, ddt_bias=g.ddt_bias, dB=g.dB)
        if initial is not None:
            r["dinitial"] = g.dinitial
        return r
    if op == "scan_step":
        out = dw.ps_selective_scan_step(s["x"], s["state"], *block[1:], **more, slots=s["slots"], new_state=s["new_state"])
        return dict(out=out, state=s["new_state"])
    weights = dict(gate=s["gate"], scale=s["scale"], post_weight=s["post"], pre_weight=s["pre"], eps=EPS)
    if op == "norm":
        residual, out = dw.ps_block_norm(s["y"], s["residual"], **weights)
        return dict(residual=residual, out=out)
    g = dw.ps_block_norm_bwd(s["y"], s["residual"], s["dout"], s["dresidual"], **weights)
    return dict(dy=g.dy, dresidual=g.dresidual, dgate=g.dgate, dscale=g.dscale, dpost=g.dpost_weight, dpre=g.dpre_weight)


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass has to move and to compute
# ---------------------------------------------------------------------------
def work(case):
    op, d = case["op"], case["channels"]
    e = TYPES[case["dtype"]].itemsize
    rows = case["batch"] if op.endswith("_step") else case["tokens"]
    cells, seqs = rows * d, case.get("seqs", 0)
    if op.startswith("conv"):
        w = case["width"]
        tail = (w - 1) * d * e
        weights = d * (w + 1) * 4
        per = 2 * w + 5  # products and sums, the bias, silu
        if op == "conv":
            return dict(bytes=2 * cells * e + weights + 4 * (seqs + 1) + seqs * tail * (2 if case["state"] else 1), flops=cells * per)
        if op == "conv_train":
            return dict(bytes=4 * cells * e + 2 * weights + 4 * (seqs + 1) + (2 * seqs * tail if case["state"] else 0), flops=cells * (per + 4 * w + 8))
        return dict(bytes=2 * cells * e + weights + 2 * rows * tail + 4 * rows, flops=cells * per)
    if op.startswith("scan"):
        n, groups = case["states"], case["groups"]
        states, bc = d * n * 4, 2 * rows * groups * n * e
        weights = states + 2 * d * 4
        per = 8 * n + 14  # exp, its argument, the recurrence, C h; softplus, D x and the gate
        if op == "scan":
            return dict(bytes=4 * cells * e + bc + weights + 4 * (seqs + 1) + seqs * states * (2 if case["state"] else 1), flops=cells * per)
        if op == "scan_train":
            return dict(bytes=8 * cells * e + 2 * bc + 2 * weights + 4 * (seqs + 1) + (2 * seqs * states if case["state"] else 0),
                        flops=cells * (per + 18 * n + 30))
        return dict(bytes=4 * cells * e + bc + weights + 2 * rows * states + 4 * rows, flops=cells * per)
    re = TYPES[case["residual"]].itemsize
    if op == "norm":
        return dict(bytes=cells * (3 * e + 2 * re) + 3 * d * 4, flops=cells * 16)
    return dict(bytes=cells * (5 * e + 3 * re) + 6 * d * 4, flops=cells * 45)


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _f(s, *names):
    return [s[k].double() if k in s else None for k in names]


def _exact_conv(s, train):
    x, w, bias, initial, dout = _f(s, "x", "weight", "bias", "initial", "dout")
    t, d = x.shape
    width, off = w.shape[1], s["offsets"].tolist()
    out, final = torch.zeros_like(x), x.new_zeros(len(off) - 1, width - 1, d)
    dx, dw, db, di = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(bias), torch.zeros_like(final)
    for q, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        before = initial[q] if initial is not None else final[q] * 0.0
        row = torch.cat([before, x[lo:hi]])
        n = hi - lo
        final[q] = row[n:]
        pre = torch.zeros(n, d, dtype=row.dtype, device=row.device) + bias
        for k in range(width):
            pre = pre + row[k:k + n] * w[:, k]
        gate = torch.sigmoid(pre)
        out[lo:hi] = pre * gate
        if train:
            g = dout[lo:hi] * (gate + pre * gate * (1 - gate))
            drow = torch.zeros_like(row)
            for k in range(width):
                drow[k:k + n] += g * w[:, k]
                dw[:, k] += (g * row[k:k + n]).sum(0)
            db += g.sum(0)
            dx[lo:hi], di[q] = drow[width - 1:], drow[:width - 1]
    if not train:
        return dict(out=out, final=final)
    r = dict(out=out, dx=dx, dweight=dw, dbias=db)
    if initial is not None:
        r["dinitial"] = di
    return r


def _exact_conv_step(s):
    x, w, bias, state = _f(s, "x", "weight", "bias", "state")
    out, new = torch.zeros_like(x), state.clone()
    for i, slot in enumerate(s["slots"].tolist()):
        row = torch.cat([state[slot], x[i:i + 1]])
        pre = bias + (row.t() * w).sum(1)
        out[i], new[slot] = pre * torch.sigmoid(pre), row[1:]
    return dict(out=out, state=new)


def _exact_scan(s, train):
    x, dt, A, B, C, D, z, bias, initial, dout = _f(s, "x", "dt", "A", "B", "C", "D", "z", "dt_bias", "initial", "dout")
    tokens, d = x.shape
    groups, n = B.shape[1], B.shape[2]
    off = s["offsets"].tolist()
    raw = dt + bias
    step = torch.logaddexp(raw, torch.zeros_like(raw))

    def wide(v):  # one token's [G, N] for each channel
        return v.repeat_interleave(d // groups, 0)

    inner = torch.zeros_like(x)
    final = initial.clone() if initial is not None else x.new_zeros(len(off) - 1, d, n)
    hs = x.new_zeros(tokens, d, n) if train else None
    for q, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        h = final[q]
        for t in range(lo, hi):
            h = torch.exp(step[t][:, None] * A) * h + (step[t] * x[t])[:, None] * wide(B[t])
            inner[t] = (h * wide(C[t])).sum(1) + D * x[t]
            if train:
                hs[t] = h
        final[q] = h
    gate = z * torch.sigmoid(z)
    if not train:
        return dict(out=inner * gate, final=final)
    gy = dout * gate
    sg = torch.sigmoid(z)
    r = dict(out=inner * gate, dz=dout * inner * (sg + z * sg * (1 - sg)), dD=(gy * x).sum(0), dC=torch.zeros_like(C), dA=torch.zeros_like(A),
             dx=gy * D, ddt=torch.zeros_like(x), ddt_bias=None, dB=torch.zeros_like(B))
    dinitial = x.new_zeros(len(off) - 1, d, n)
    for q, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        back = x.new_zeros(d, n)  # decay[t + 1] dh[t + 1]
        for t in range(hi - 1, lo - 1, -1):
            dh = back + gy[t][:, None] * wide(C[t])
            r["dC"][t] = (gy[t][:, None] * hs[t]).view(groups, d // groups, n).sum(1)
            r["dB"][t] = (dh * (step[t] * x[t])[:, None]).view(groups, d // groups, n).sum(1)
            back = torch.exp(step[t][:, None] * A) * dh
            before = hs[t - 1] if t > lo else initial[q] if initial is not None else torch.zeros_like(back)
            flow = back * before
            r["dA"] += flow * step[t][:, None]
            along = (dh * wide(B[t])).sum(1)
            r["dx"][t] += step[t] * along
            r["ddt"][t] = (flow * A).sum(1) + x[t] * along
        dinitial[q] = back
    r["ddt"] = r["ddt"] * torch.sigmoid(raw)
    r["ddt_bias"] = r["ddt"].sum(0)
    if initial is not None:
        r["dinitial"] = dinitial
    return r


def _exact_scan_step(s):
    x, state, dt, A, B, C, D, z, bias = _f(s, "x", "state", "dt", "A", "B", "C", "D", "z", "dt_bias")
    d, groups = x.shape[1], B.shape[1]
    out, new = torch.zeros_like(x), state.clone()
    for i, slot in enumerate(s["slots"].tolist()):
        step = torch.logaddexp(dt[i] + bias, torch.zeros_like(bias))
        wide_b, wide_c = (v[i].repeat_interleave(d // groups, 0) for v in (B, C))
        h = torch.exp(step[:, None] * A) * state[slot] + (step * x[i])[:, None] * wide_b
        out[i] = ((h * wide_c).sum(1) + D * x[i]) * z[i] * torch.sigmoid(z[i])
        new[slot] = h
    return dict(out=out, state=new)


def _exact_norm(s, train):
    y, z, r, scale, post, pre, dres, dout = _f(s, "y", "gate", "residual", "scale", "post", "pre", "dresidual", "dout")
    d = y.shape[1]
    ny = torch.rsqrt(y.square().sum(1, keepdim=True) / d + EPS)
    gate = torch.sigmoid(z)
    if not train:
        r = r + scale * gate * (y * ny * post)
        return dict(residual=r, out=r * torch.rsqrt(r.square().sum(1, keepdim=True) / d + EPS) * pre)
    nr = torch.rsqrt(r.square().sum(1, keepdim=True) / d + EPS)
    unit, inner = y * ny, r * nr
    g = dout * pre
    total = dres + nr * (g - inner * (g * inner).sum(1, keepdim=True) / d)
    dp = total * scale * gate
    h = dp * post
    return dict(dy=ny * (h - unit * (h * unit).sum(1, keepdim=True) / d), dresidual=total, dgate=total * scale * unit * post * gate * (1 - gate),
                dscale=(total * gate * unit * post).sum(0), dpost=(dp * unit).sum(0), dpre=(dout * inner).sum(0))


def exact(case, seed):
    op = case["op"]
    if op == "scan_train" and case["tokens"] * case["channels"] * case["states"] > 1 << 29:
        return None
    s = prepare(case, seed)
    if op.startswith("conv"):
        return _exact_conv_step(s) if op == "conv_step" else _exact_conv(s, op == "conv_train")
    if op.startswith("scan"):
        return _exact_scan_step(s) if op == "scan_step" else _exact_scan(s, op == "scan_train")
    return _exact_norm(s, op == "norm_train")

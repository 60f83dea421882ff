"""Cases of the linear-attention and group-norm operators, with their plain forms.

Five kinds of case, each one call of the library:

  attend       linear attention with a decay for each head over whole
               sequences, dense or packed: S_t = gamma_h S_{t-1} + k_t v_t^T,
               o_t = S_t^T q_t, from an initial state or from zeros; returns
               the outputs and the final state (fp32)
  step         the same for one token on a carried state, updated in place
  attend_grad  its gradients for q, k, v and the initial state
  norm         group norm, channels last ([N, S, C], statistics over S and
               the C / groups channels of a group), an affine map and an
               activation; S = 1 is the per-token norm of each head's output
  norm_grad    its gradients for x, weight and bias
"""
import math

import torch

own = False
_LIB = None


def _dp():
    """The library, imported only where its kernels run."""
    global _LIB
    if _LIB is None:
        import deltaproduct_householder_product_gb300 as dp
        _LIB = dp
    return _LIB


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # the smallest prompt: the fp32 parity workload, launch latency
        {"name": "attend-tiny-f32", "kind": "attend", "dtype": "f32", "B": 1, "T": 64, "H": 2, "Dk": 32, "Dv": 32,
         "h0": False, "lengths": ""},
        # an ordinary training or prompt batch (the base workload's sizes)
        {"name": "attend-base", "kind": "attend", "dtype": "bf16", "B": 4, "T": 2048, "H": 8, "Dk": 128, "Dv": 128,
         "h0": False, "lengths": ""},
        # one long prompt with a carried state: few heads, many tokens
        {"name": "attend-long", "kind": "attend", "dtype": "bf16", "B": 1, "T": 32768, "H": 16, "Dk": 128, "Dv": 128,
         "h0": True, "lengths": ""},
        # a serving batch of prompts of different lengths packed back to back,
        # an empty one and one-token ones among them, at half the head size
        {"name": "attend-packed", "kind": "attend", "dtype": "bf16", "B": 12, "T": 15410, "H": 16, "Dk": 64, "Dv": 64,
         "h0": True, "lengths": "1,4096,37,0,2500,129,1000,1,3777,128,715,3026"},
        # one token of one sequence: launch latency
        {"name": "step-one", "kind": "step", "dtype": "bf16", "B": 1, "H": 16, "Dk": 128, "Dv": 128},
        # one token of a serving batch: the states' traffic
        {"name": "step-batch", "kind": "step", "dtype": "bf16", "B": 64, "H": 16, "Dk": 128, "Dv": 128},
        # the gradients of the ordinary batch
        {"name": "grad-base", "kind": "attend_grad", "dtype": "bf16", "B": 4, "T": 2048, "H": 8, "Dk": 128, "Dv": 128,
         "h0": False, "lengths": ""},
        # the gradients of the largest batch, with a carried state
        {"name": "grad-large", "kind": "attend_grad", "dtype": "bf16", "B": 4, "T": 8192, "H": 16, "Dk": 128,
         "Dv": 128, "h0": True, "lengths": ""},
        # the norm of each head's output in a long batch (16 heads of 128)
        {"name": "norm-heads", "kind": "norm", "dtype": "bf16", "N": 32768, "S": 1, "C": 2048, "groups": 16,
         "act": "silu", "affine": True},
        # few images or clips of many positions, groups of 20 channels
        {"name": "norm-positions", "kind": "norm", "dtype": "bf16", "N": 4, "S": 4099, "C": 640, "groups": 32,
         "act": "silu", "affine": True},
        # the gradients of the ordinary batch's output norm (8 heads of 128)
        {"name": "norm-grad-heads", "kind": "norm_grad", "dtype": "bf16", "N": 8192, "S": 1, "C": 1024, "groups": 8,
         "act": "silu", "affine": True},
        # the gradients over many positions
        {"name": "norm-grad-positions", "kind": "norm_grad", "dtype": "bf16", "N": 4, "S": 4099, "C": 640,
         "groups": 32, "act": "silu", "affine": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "step", "attend_grad", "norm", "norm_grad"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if kind in ("attend", "attend_grad"):
        # token-heads in all; fp32 and gradients cost more for each
        most = (1 << 19 if kind == "attend" else 1 << 18) >> (2 if dtype == "f32" else 0)
        H = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
        Dk = rng.choice([32, 64, 64, 128, 128, 128])
        Dv = Dk if rng.random() < 0.7 else rng.choice([32, 64, 128])
        case = {"kind": kind, "dtype": dtype, "H": H, "Dk": Dk, "Dv": Dv, "h0": rng.random() < 0.5, "lengths": ""}
        T = _log_int(rng, 1, min(32768, most // H))
        if rng.random() < 0.35:   # packed: lengths from one token (some empty) to T
            B = rng.randint(2, 24)
            lengths = [0 if rng.random() < 0.06 else _log_int(rng, 1, T) for _ in range(B)]
            while sum(lengths) * H > most:
                lengths[lengths.index(max(lengths))] //= 2
            if sum(lengths) == 0:
                lengths[0] = 1
            case.update(B=B, T=sum(lengths), lengths=",".join(str(n) for n in lengths))
        else:
            case.update(B=rng.randint(1, max(1, min(32, most // (T * H)))), T=T)
        return case
    if kind == "step":
        Dk = rng.choice([32, 64, 128, 128])
        return {"kind": kind, "dtype": dtype, "B": _log_int(rng, 1, 128), "H": rng.choice([1, 2, 3, 4, 8, 12, 16]),
                "Dk": Dk, "Dv": Dk if rng.random() < 0.7 else rng.choice([32, 64, 128])}
    # norms: at most 2^26 elements (2^24 in fp32 or for gradients)
    most = 1 << (26 if kind == "norm" and dtype == "bf16" else 24)
    groups = rng.choice([1, 2, 4, 8, 16, 32])
    wide = rng.choice([8, 10, 16, 20, 32, 33, 40, 64, 80, 128, 128, 256])
    C = groups * wide
    if rng.random() < 0.5:
        N, S = _log_int(rng, 1, max(1, min(65536, most // C))), 1
    else:
        S = _log_int(rng, 2, max(2, min(16384, most // C)))
        N = rng.randint(1, max(1, min(16, most // (S * C))))
    return {"kind": kind, "dtype": dtype, "N": N, "S": S, "C": C, "groups": groups,
            "act": rng.choice(["silu", "silu", "none"]), "affine": rng.random() < 0.8}


# ---------------------------------------------------------------- the inputs
def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _lengths(case):
    return [int(n) for n in case["lengths"].split(",")] if case.get("lengths") else None


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True).clamp_min(1e-12)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    dt, s = _dtype(case), {"case": case}
    if case["kind"] in ("norm", "norm_grad"):
        N, S, C, G = case["N"], case["S"], case["C"], case["groups"]
        # values of a head's outputs or of a feature map: a mean of its own for each group
        mid = 0.5 * randn(N, 1, G, 1)
        s["x"] = (1.5 * randn(N, S, G, C // G) + mid).reshape(N, S, C).to(dt)
        s["weight"] = (1 + 0.2 * randn(C)).to(dt) if case["affine"] else None
        s["bias"] = (0.2 * randn(C)).to(dt) if case["affine"] else None
        if case["kind"] == "norm_grad":
            s["dy"] = randn(N, S, C).to(dt)
            # the statistics that the forward pass left
            var, mean = torch.var_mean(s["x"].float().view(N, S, G, C // G), dim=(1, 3), unbiased=False)
            s["mean"], s["rstd"] = mean.contiguous(), torch.rsqrt(var + 1e-5).contiguous()
        return s
    B, H, Dk, Dv = case["B"], case["H"], case["Dk"], case["Dv"]
    # decays spaced over the heads, from a memory of 32 tokens to one of 4096
    s["log_decay"] = torch.log1p(-torch.exp2(-5 - 7 * torch.arange(H, device="cuda") / max(1, H - 1))).float()
    lengths = _lengths(case)
    if case["kind"] == "step":
        lead, states = (B, H), B
    elif lengths:
        lead, states = (case["T"], H), B
        s["cu_seqlens"] = torch.tensor([sum(lengths[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
        s["max_seqlen"] = max(lengths)
    else:
        lead, states = (B, case["T"], H), B
    s["q"] = _unit(randn(*lead, Dk)).to(dt)
    s["k"] = _unit(torch.nn.functional.silu(randn(*lead, Dk))).to(dt)
    s["v"] = randn(*lead, Dv).to(dt)
    if case["kind"] == "step":
        s["state"] = randn(B, H, Dk, Dv)
        s["out"] = torch.empty(B, H, Dv, dtype=dt, device="cuda")
        return s
    s["h0"] = randn(states, H, Dk, Dv) if case["h0"] else None
    if case["kind"] == "attend":
        s["out"] = torch.empty(*lead, Dv, dtype=dt, device="cuda")
        s["h_final"] = torch.empty(states, H, Dk, Dv, device="cuda")
    else:
        s["d_o"] = randn(*lead, Dv).to(dt)
        s["dh_final"] = 0.1 * randn(states, H, Dk, Dv)
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    kind = state["case"]["kind"]
    if own:
        return _OWN[kind](state)
    return _PLAIN[kind](state)


def _workspace(s, backward):
    """The device workspace that a program keeps for its calls of one shape."""
    if "workspace" not in s:
        c = s["case"]
        n = _dp().linear_attention_workspace_size(c["B"], c["T"], c["H"], c["Dk"], c["Dv"], dtype=_dtype(c),
                                                  max_seqlen=s.get("max_seqlen"), backward=backward)
        s["workspace"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own_attend(s):
    if "cu_seqlens" in s:
        return _dp().linear_attention_varlen(s["q"], s["k"], s["v"], s["log_decay"], s["h0"],
                                             cu_seqlens=s["cu_seqlens"], max_seqlen=s["max_seqlen"], out=s["out"],
                                             h_final=s["h_final"], workspace=_workspace(s, False))
    return _dp().linear_attention(s["q"], s["k"], s["v"], s["log_decay"], s["h0"], out=s["out"],
                                  h_final=s["h_final"], workspace=_workspace(s, False))


def _own_step(s):
    o = _dp().linear_attention_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], out=s["out"])
    return o, s["state"]


def _own_attend_grad(s):
    if "cu_seqlens" in s:
        g = _dp().linear_attention_backward_varlen(s["q"], s["k"], s["v"], s["log_decay"], s["h0"],
                                                   cu_seqlens=s["cu_seqlens"], max_seqlen=s["max_seqlen"],
                                                   d_o=s["d_o"], dh_final=s["dh_final"],
                                                   workspace=_workspace(s, True))
    else:
        g = _dp().linear_attention_backward(s["q"], s["k"], s["v"], s["log_decay"], s["h0"], d_o=s["d_o"],
                                            dh_final=s["dh_final"], workspace=_workspace(s, True))
    return g["dq"], g["dk"], g["dv"], g["dh0"]


def _own_norm(s):
    c = s["case"]
    return _dp().group_norm(s["x"], s["weight"], s["bias"], groups=c["groups"], eps=1e-5, act=c["act"])


def _own_norm_grad(s):
    c = s["case"]
    g = _dp().group_norm_backward(s["dy"], s["x"], s["weight"], s["bias"], s["mean"], s["rstd"],
                                  groups=c["groups"], act=c["act"])
    return (g["dx"], g["dweight"], g["dbias"]) if c["affine"] else (g["dx"],)


_OWN = {"attend": _own_attend, "step": _own_step, "attend_grad": _own_attend_grad, "norm": _own_norm,
        "norm_grad": _own_norm_grad}


# ---------------------------------------------------------------- the plain forms
def _spread(s, names):
    """The named tensors as fp32 [B, H, T, D] with every sequence ending at the
    last row (zero rows before it), and the place of each row: its index in
    the packed or dense layout, and its token number (negative in the padding)."""
    c, C = s["case"], 128
    if "cu_seqlens" in s:
        cu = s["cu_seqlens"].long()
        lens = cu[1:] - cu[:-1]
        T = max(C, -(-s["max_seqlen"] // C) * C)
        tok = torch.arange(T, device="cuda")[None, :] - (T - lens)[:, None]          # [B, T]
        row = (cu[:-1, None] + tok).clamp(0, max(0, c["T"] - 1))
        flat = {n: s[n] for n in names}
    else:
        T = max(C, -(-c["T"] // C) * C)
        lens = torch.full((c["B"],), c["T"], device="cuda")
        tok = (torch.arange(T, device="cuda") - (T - c["T"]))[None, :].expand(c["B"], T)
        row = torch.arange(c["B"], device="cuda")[:, None] * c["T"] + tok.clamp_min(0)
        flat = {n: s[n].reshape(-1, *s[n].shape[2:]) for n in names}
    live = (tok >= 0)[:, None, :, None]
    out = {n: torch.where(live, t[row].float().transpose(1, 2), 0.0) for n, t in flat.items()}
    return out, row, tok, lens


def _gather(x, s, row, tok):
    """[B, H, T, D] rows back to the layout of the inputs."""
    c = s["case"]
    x = x.transpose(1, 2)
    if "cu_seqlens" in s:
        out = x.new_empty(c["T"], *x.shape[2:])
        live = tok >= 0
        out[row[live]] = x[live]
        return out.to(_dtype(c))
    return x[:, x.shape[1] - c["T"]:].to(_dtype(c))


def _weighted_sums(x, y, z, ld, C=128):
    """For [B, H, T, D] rows, T a multiple of C: out_t = sum_{s <= t} gamma^(t-s)
    (x_t . y_s) z_s, and sum_s gamma^(T-1-s) y_s z_s^T, chunk by chunk."""
    B, H, T, _ = x.shape
    n = T // C
    xc, yc, zc = (t.reshape(B, H, n, C, t.shape[-1]) for t in (x, y, z))
    i = torch.arange(C, device="cuda", dtype=torch.float32)
    far = i[:, None] - i[None, :]
    decay = torch.where(far >= 0, torch.exp(far.clamp_min(0) * ld[:, None, None]), 0.0)      # [H, C, C]
    inside = (xc @ yc.transpose(-1, -2) * decay[:, None]) @ zc
    last = torch.exp((C - 1 - i) * ld[:, None])                                              # [H, C]
    sums = (yc * last[:, None, :, None]).transpose(-1, -2) @ zc                              # [B, H, n, Dy, Dz]
    j = torch.arange(n + 1, device="cuda", dtype=torch.float32)
    steps = j[:, None] - 1 - j[None, :n]
    carry = torch.where(steps >= 0, torch.exp(steps.clamp_min(0) * C * ld[:, None, None]), 0.0)   # [H, n+1, n]
    states = (carry @ sums.reshape(B, H, n, -1)).reshape(B, H, n + 1, x.shape[-1], z.shape[-1])
    first = torch.exp((i + 1) * ld[:, None])
    before = (xc * first[:, None, :, None]) @ states[:, :, :n]
    return (inside + before).reshape(B, H, T, -1), states[:, :, n]


def _powers(ld, n):
    """gamma_h^n for token counts n [B, T] or [B], 0 for negative ones."""
    p = torch.exp(n.clamp_min(0).float()[:, None] * ld.reshape(1, -1, *([1] * (n.dim() - 1))))
    return torch.where(n[:, None] >= 0, p, 0.0)


def _plain_attend(s):
    t, row, tok, lens = _spread(s, ("q", "k", "v"))
    ld = s["log_decay"]
    o, h = _weighted_sums(t["q"], t["k"], t["v"], ld)
    if s["h0"] is not None:
        o = o + _powers(ld, torch.where(tok >= 0, tok + 1, -1))[..., None] * (t["q"] @ s["h0"])
        h = h + _powers(ld, lens)[..., None, None] * s["h0"]
    return _gather(o, s, row, tok), h


def _plain_step(s):
    gamma = torch.exp(s["log_decay"])[:, None, None]
    q, k, v = (s[n].float() for n in "qkv")
    s["state"].mul_(gamma).add_(k[..., :, None] * v[..., None, :])
    return (s["state"] * q[..., :, None]).sum(-2).to(s["q"].dtype), s["state"]


def _plain_attend_grad(s):
    t, row, tok, lens = _spread(s, ("q", "k", "v", "d_o"))
    q, k, v, d, ld = t["q"], t["k"], t["v"], t["d_o"], s["log_decay"]
    dq, _ = _weighted_sums(d, v, k, ld)
    if s["h0"] is not None:
        dq = dq + _powers(ld, torch.where(tok >= 0, tok + 1, -1))[..., None] * (d @ s["h0"].transpose(-1, -2))
    # the state's gradient runs from the last token to the first: sums over the flipped rows
    qr, kr, vr, dr = (x.flip(2) for x in (q, k, v, d))
    dv, _ = _weighted_sums(kr, qr, dr, ld)
    dk, _ = _weighted_sums(vr, dr, qr, ld)
    back = torch.where(tok >= 0, lens[:, None] - 1 - tok, -1)
    far = _powers(ld, back)[..., None]
    dk = dk.flip(2) + far * (v @ s["dh_final"].transpose(-1, -2))
    dv = dv.flip(2) + far * (k @ s["dh_final"])
    first = _powers(ld, torch.where(tok >= 0, tok + 1, -1))[..., None]
    dh0 = (q * first).transpose(-1, -2) @ d + _powers(ld, lens)[..., None, None] * s["dh_final"]
    return _gather(dq, s, row, tok), _gather(dk, s, row, tok), _gather(dv, s, row, tok), dh0


def _plain_norm(s):
    c, x = s["case"], s["x"]
    N, S, C, G = c["N"], c["S"], c["C"], c["groups"]
    f = x.float().view(N, S, G, C // G)
    mean = f.mean((1, 3), keepdim=True)
    mid = f - mean
    rstd = 1 / torch.sqrt((mid * mid).mean((1, 3), keepdim=True) + 1e-5)
    z = (mid * rstd).view(N, S, C)
    if c["affine"]:
        z = z * s["weight"].float() + s["bias"].float()
    if c["act"] == "silu":
        z = z / (1 + torch.exp(-z))
    return z.to(x.dtype), mean.view(N, G), rstd.view(N, G)


def _plain_norm_grad(s):
    c, x = s["case"], s["x"]
    N, S, C, G = c["N"], c["S"], c["C"], c["groups"]
    mean, rstd = s["mean"].view(N, 1, G, 1), s["rstd"].view(N, 1, G, 1)
    hat = ((x.float().view(N, S, G, C // G) - mean) * rstd).view(N, S, C)
    d = s["dy"].float()
    z = hat * s["weight"].float() + s["bias"].float() if c["affine"] else hat
    if c["act"] == "silu":
        p = 1 / (1 + torch.exp(-z))
        d = d * p * (1 + z * (1 - p))
    u = d * s["weight"].float() if c["affine"] else d
    ug, hg = u.view(N, S, G, C // G), hat.view(N, S, G, C // G)
    dx = rstd * (ug - ug.mean((1, 3), keepdim=True) - hg * (ug * hg).mean((1, 3), keepdim=True))
    dx = dx.view(N, S, C).to(x.dtype)
    return (dx, (d * hat).sum((0, 1)), d.sum((0, 1))) if c["affine"] else (dx,)


_PLAIN = {"attend": _plain_attend, "step": _plain_step, "attend_grad": _plain_attend_grad, "norm": _plain_norm,
          "norm_grad": _plain_norm_grad}


# ---------------------------------------------------------------- the least work
def work(case):
    el = 4 if case["dtype"] == "f32" else 2
    if case["kind"] in ("norm", "norm_grad"):
        n, stats = case["N"] * case["S"] * case["C"], 8 * case["N"] * case["groups"]
        affine = 2 * case["C"] if case["affine"] else 0
        if case["kind"] == "norm":
            return {"bytes": 2 * n * el + stats + affine * el, "flops": 12 * n}
        return {"bytes": 3 * n * el + stats + affine * (el + 4), "flops": 25 * n}
    B, H, Dk, Dv = case["B"], case["H"], case["Dk"], case["Dv"]
    state, cell = 4 * B * H * Dk * Dv, Dk * Dv
    if case["kind"] == "step":
        return {"bytes": 2 * state + B * H * (2 * Dk + 2 * Dv) * el, "flops": 5 * B * H * cell}
    rows = (case["T"] if case["lengths"] else B * case["T"]) * H
    if case["kind"] == "attend":
        return {"bytes": rows * (2 * Dk + 2 * Dv) * el + state * (2 if case["h0"] else 1), "flops": 4 * rows * cell}
    return {"bytes": rows * (4 * Dk + 3 * Dv) * el + state * (3 if case["h0"] else 2), "flops": 10 * rows * cell}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The recurrences token by token, the norms by their definition, in 64 bits."""
    s = prepare(case, seed)
    for name, t in list(s.items()):
        if torch.is_tensor(t) and t.is_floating_point():
            s[name] = t.double()
    if case["kind"] in ("norm", "norm_grad"):
        return _exact_norm(case, s)
    if case["kind"] == "step":
        h = torch.exp(s["log_decay"])[None, :, None, None] * s["state"] + torch.einsum("bhi,bhj->bhij", s["k"], s["v"])
        return torch.einsum("bhij,bhi->bhj", h, s["q"]), h
    return _exact_attend(case, s)


def _exact_attend(case, s):
    lengths = _lengths(case)
    B, H, Dk, Dv = case["B"], case["H"], case["Dk"], case["Dv"]
    if not lengths:
        lengths = [case["T"]] * B
    starts = [sum(lengths[:i]) for i in range(B)]
    order = sorted(range(B), key=lambda b: -lengths[b])          # the longest first
    start = torch.tensor([starts[b] for b in order], device="cuda")
    perm = torch.tensor(order, device="cuda")
    counts = [sum(1 for n in lengths if n > t) for t in range(max(lengths))]
    rows = {n: s[n].reshape(-1, H, s[n].shape[-1]) for n in ("q", "k", "v", "d_o") if n in s}
    gamma = torch.exp(s["log_decay"])[None, :, None, None]
    zeros = torch.zeros(B, H, Dk, Dv, dtype=torch.float64, device="cuda")
    h = (zeros if s["h0"] is None else s["h0"])[perm].clone()
    grad = case["kind"] == "attend_grad"
    out = {n: torch.empty_like(rows[n]) for n in (("q", "k", "v") if grad else ("v",))}
    for t, n in enumerate(counts):
        at = start[:n] + t
        k, v = rows["k"][at], rows["v"][at]
        h[:n] = h[:n] * gamma + k[..., :, None] * v[..., None, :]
        if grad:
            out["q"][at] = (h[:n] * rows["d_o"][at][..., None, :]).sum(-1)
        else:
            out["v"][at] = (h[:n] * rows["q"][at][..., :, None]).sum(-2)
    back = torch.empty_like(perm)
    back[perm] = torch.arange(B, device="cuda")
    if not grad:
        return out["v"].view(s["v"].shape), h[back]
    g = s["dh_final"][perm].clone()
    for t in reversed(range(len(counts))):
        n = counts[t]
        at = start[:n] + t
        q, d = rows["q"][at], rows["d_o"][at]
        g[:n] += q[..., :, None] * d[..., None, :]
        out["k"][at] = (g[:n] * rows["v"][at][..., None, :]).sum(-1)
        out["v"][at] = (g[:n] * rows["k"][at][..., :, None]).sum(-2)
        g[:n] *= gamma
    return out["q"].view(s["q"].shape), out["k"].view(s["k"].shape), out["v"].view(s["v"].shape), g[back]


def _exact_norm(case, s):
    N, S, C, G = case["N"], case["S"], case["C"], case["groups"]
    x = s["x"].view(N, S, G, C // G)
    w = s["weight"].view(G, C // G) if case["affine"] else torch.ones((), dtype=torch.float64, device="cuda")
    b = s["bias"].view(G, C // G) if case["affine"] else torch.zeros((), dtype=torch.float64, device="cuda")
    if case["kind"] == "norm":
        mean = x.sum((1, 3)) / (S * (C // G))
        var = (x - mean[:, None, :, None]).square().sum((1, 3)) / (S * (C // G))
        rstd = (var + 1e-5) ** -0.5
        z = (x - mean[:, None, :, None]) * rstd[:, None, :, None] * w + b
        y = z * torch.sigmoid(z) if case["act"] == "silu" else z
        return y.reshape(N, S, C), mean, rstd
    rstd = s["rstd"][:, None, :, None]
    hat = (x - s["mean"][:, None, :, None]) * rstd
    d = s["dy"].view(N, S, G, C // G)
    if case["act"] == "silu":
        z = hat * w + b
        p = torch.sigmoid(z)
        d = d * (p + z * p * (1 - p))
    u = d * w
    m = S * (C // G)
    dx = rstd * (u - u.sum((1, 3), keepdim=True) / m - hat * ((u * hat).sum((1, 3), keepdim=True) / m))
    dx = dx.reshape(N, S, C)
    return (dx, (d * hat).sum((0, 1)).reshape(C), d.sum((0, 1)).reshape(C)) if case["affine"] else (dx,)

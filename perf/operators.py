"""Cases of the group norm with an activation and of the rotary positions.

``listed()`` and ``draw()`` give cases, ``prepare()`` makes what a program has
in hand before the call, ``run()`` makes one pass: in plain torch operations,
or, where ``own`` is true, through this package. ``exact()`` computes the same
outputs in 64 bits.

Four operators: ``gn_fwd`` and ``gn_bwd`` (group norm over channels-last
activations [samples, rows, channels] with SiLU, GELU or nothing behind it)
and ``rope_fwd`` and ``rope_bwd`` (rotary positions of the queries and keys,
[batch, tokens, heads, head_dim], with the RMSNorm of each head before the
rotation where the case has one).
"""

from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ---- cases ------------------------------------------------------------------

def _gn(name, op, dtype, samples, rows, channels, groups, act, affine="channel", wide=0, eps=1e-5):
    """affine: "channel" (gamma and beta of the channels) or "sample" (a scale
    and shift of each sample); wide: channels of the tensor that x is a slice
    of (0: x is whole)."""
    return {"name": name, "op": op, "dtype": dtype, "samples": samples, "rows": rows,
            "channels": channels, "groups": groups, "act": act, "affine": affine, "wide": wide,
            "eps": eps}


def _rope(name, op, dtype, batch, tokens, heads, kv_heads, dim, rot, layout, norm, storage,
          axes=1, scaling="none", start=0, eps=1e-6):
    """layout: "half" or "interleaved"; storage: "packed" (slices of one
    projection's [batch, tokens, (heads + 2 kv_heads) dim]), "separate", or
    "heads" ([batch, heads, tokens, dim] in memory); start: the first
    position of the sequences (each has its own where they are single tokens)."""
    return {"name": name, "op": op, "dtype": dtype, "batch": batch, "tokens": tokens,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot, "layout": layout,
            "norm": norm, "storage": storage, "axes": axes, "scaling": scaling, "start": start,
            "eps": eps}


def listed():
    return [
        # a diffusion UNet's first level at inference, two samples of 64 x 64: a few MB, where latency counts
        _gn("gn_fwd_f16_2x4096x320", "gn_fwd", "f16", 2, 4096, 320, 32, "silu"),
        # its deepest level with a training batch: many channels, few rows
        _gn("gn_fwd_bf16_16x1024x1280", "gn_fwd", "bf16", 16, 1024, 1280, 32, "silu"),
        # an image decoder's last level, 512 x 512: the longest rows, the largest case
        _gn("gn_fwd_bf16_2x262144x256", "gn_fwd", "bf16", 2, 262144, 256, 32, "silu"),
        # odd sizes: rows of 330 bytes, 33 channels a group, a ragged image
        _gn("gn_fwd_bf16_3x2867x165", "gn_fwd", "bf16", 3, 2867, 165, 5, "gelu"),
        # the training step of a UNet level of 64 x 64 with two samples
        _gn("gn_bwd_f16_2x4096x640", "gn_bwd", "f16", 2, 4096, 640, 32, "silu"),
        # the training step of a level of 128 x 128 with a batch
        _gn("gn_bwd_bf16_8x16384x320", "gn_bwd", "bf16", 8, 16384, 320, 32, "silu"),
        # a scale and shift of each sample; x is the first channels of a joined skip connection
        _gn("gn_bwd_f32_5x957x96", "gn_bwd", "f32", 5, 957, 96, 8, "none", affine="sample", wide=144),
        # serving: one token of each of 64 sequences, far positions of a scaled context, q and k out of one projection
        _rope("rope_fwd_bf16_64x1", "rope_fwd", "bf16", 64, 1, 32, 8, 128, 128, "half", True,
              "packed", scaling="yarn", start=120000),
        # a prompt of 16384 tokens
        _rope("rope_fwd_bf16_1x16384", "rope_fwd", "bf16", 1, 16384, 32, 8, 128, 128, "half", True,
              "packed"),
        # part of the head, neighbouring pairs, heads before tokens in memory, no norm, odd lengths
        _rope("rope_fwd_f16_3x1023", "rope_fwd", "f16", 3, 1023, 20, 20, 80, 32, "interleaved",
              False, "heads", scaling="linear"),
        # a training step's backward with shared key heads
        _rope("rope_bwd_bf16_4x4096", "rope_bwd", "bf16", 4, 4096, 16, 4, 64, 64, "half", True,
              "packed", scaling="ntk"),
        # image tokens of 64 x 64 with two position axes, heads of 40 (320 channels in 8 heads)
        _rope("rope_bwd_f16_2x4096_axes", "rope_bwd", "f16", 2, 4096, 8, 8, 40, 40, "half", True,
              "separate", axes=2),
    ]


MOST_BYTES = 2 * 2 * 262144 * 256 * 2   # what the largest listed case moves


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gn_fwd", "gn_bwd", "rope_fwd", "rope_bwd"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op.startswith("gn"):
        per_group = _log(rng, 1, 64)
        groups = rng.choice([1, 2, 4, 5, 8, 16, 32])
        if per_group * groups > 2048:
            groups = 8
        channels = per_group * groups
        samples = _log(rng, 1, 16)
        most = MOST_BYTES // (3 * SIZE[dtype] * samples * channels)
        # from 32 values a group on: the gradient of a group of two or three is what is left of
        # terms that all but cancel, and says nothing of either side
        rows = max(-(-32 // per_group), min(_log(rng, 1, 262144), most))
        wide = rng.choice([0, 0, channels + rng.choice([8, 16, 33])])
        case = _gn("", op, dtype, samples, rows, channels, groups,
                   rng.choice(["none", "silu", "silu", "gelu"]),
                   affine=rng.choice(["channel", "channel", "sample"]), wide=wide)
    else:
        dim = rng.choice([16, 32, 40, 64, 64, 80, 96, 128, 128, 160, 256, 2 * rng.randint(4, 120)])
        axes = rng.choice([1, 1, 1, 2, 3])
        rot = dim if rng.random() < 0.6 else 2 * rng.randint(1, dim // 2)
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 1, 3, 4, 8])
        batch = _log(rng, 1, 64)
        most = MOST_BYTES // (3 * SIZE[dtype] * batch * (heads + kv_heads) * dim)
        tokens = max(1, min(_log(rng, 1, 32768), most))
        case = _rope("", op, dtype, batch, tokens, heads, kv_heads, dim, rot,
                     rng.choice(["half", "interleaved"]), rng.random() < 0.6,
                     rng.choice(["packed", "separate", "heads"]), axes=axes,
                     scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                     start=rng.choice([0, 0, _log(rng, 1, 1000000)]))
    del case["name"]
    return case


# ---- inputs -----------------------------------------------------------------

def _normal(gen, shape, dtype, std=1.0, mean=0.0):
    t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return t.mul_(std).add_(mean).to(DTYPES[dtype])


def _frequencies(rot, scaling):
    """Radians a position for each pair, 64 bits, and the scale of cos and
    sin. The scaled forms stretch an original context of 16384 eight times."""
    base, factor, original = 10000.0, 8.0, 16384
    pairs = rot // 2
    j = torch.arange(pairs, dtype=torch.float64)
    if scaling == "ntk" and rot > 2:
        base *= factor ** (rot / (rot - 2))
    f = base ** (-2.0 * j / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        # pairs that make over 32 turns in the original context keep their
        # frequency, those that make less than one have it divided by factor,
        # and the share runs linearly with the pair's number between the two
        at = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        share = ((j - low) / max(high - low, 1e-3)).clamp(0, 1)
        return f / factor * share + f * (1 - share), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _prepare_gn(case, gen):
    N, R, C, G = case["samples"], case["rows"], case["channels"], case["groups"]
    dt = case["dtype"]
    offset = _normal(gen, (N, 1, C), "f32", 0.5)
    whole = torch.randn((N, R, case["wide"] or C), generator=gen, device="cuda")
    whole[..., :C].mul_(1.5).add_(offset)
    x = whole.to(DTYPES[dt])[..., :C]
    per = (N, C) if case["affine"] == "sample" else (C,)
    state = {"case": case, "x": x, "gamma": _normal(gen, per, dt, 0.05, 1.0),
             "beta": _normal(gen, per, dt, 0.05)}
    del whole
    if case["op"] == "gn_bwd":
        state["dy"] = _normal(gen, (N, R, C), dt)
        # the statistics that the forward left
        mean = torch.empty((N, G), device="cuda")
        rstd = torch.empty((N, G), device="cuda")
        for n in range(N):
            s = x[n].reshape(R, G, C // G).double()
            mean[n] = s.mean(dim=(0, 2))
            rstd[n] = (s.var(dim=(0, 2), correction=0) + case["eps"]).rsqrt()
        state["mean"], state["rstd"] = mean, rstd
    return state


def _prepare_rope(case, gen):
    B, T, H, K, D = (case[k] for k in ("batch", "tokens", "heads", "kv_heads", "dim"))
    dt = case["dtype"]

    def heads_of(n):
        if case["storage"] == "heads":
            return _normal(gen, (B, n, T, D), dt).transpose(1, 2)
        return _normal(gen, (B, T, n, D), dt)

    def both():
        if case["storage"] == "packed":
            p = _normal(gen, (B, T, H + 2 * K, D), dt)
            return p[:, :, :H], p[:, :, H:H + K]
        return heads_of(H), heads_of(K)

    state = {"case": case}
    state["q"], state["k"] = both()
    if case["op"] == "rope_bwd":
        state["dq"], state["dk"] = (heads_of(H), heads_of(K))
    state["q_gamma"] = _normal(gen, (D,), dt, 0.05, 1.0) if case["norm"] else None
    state["k_gamma"] = _normal(gen, (D,), dt, 0.05, 1.0) if case["norm"] else None
    # positions: [batch, tokens], or [axes, batch, tokens] of a grid
    t = torch.arange(T, device="cuda", dtype=torch.int64)
    if case["axes"] == 1:
        first = torch.full((B, 1), case["start"], device="cuda", dtype=torch.int64)
        if T == 1:   # single tokens: each sequence has a length of its own
            first = first - torch.randint(0, case["start"] // 2 + 1, (B, 1), generator=gen, device="cuda")
        state["positions"] = first + t
    else:
        side = max(1, math.isqrt(T))
        grid = [t // side, t % side, torch.full_like(t, case["start"])][:case["axes"]]
        state["positions"] = torch.stack(grid)[:, None].expand(-1, B, -1).contiguous()
    pairs = case["rot"] // 2
    if case["axes"] == 1:
        f, scale = _frequencies(case["rot"], case["scaling"])
    else:
        # the pairs are shared out to the axes in order, each with a range of its own
        f = torch.zeros((case["axes"], pairs), dtype=torch.float64)
        at, scale = 0, 1.0
        for a in range(case["axes"]):
            n = pairs // case["axes"] + (a < pairs % case["axes"])
            if n:
                f[a, at:at + n], scale = _frequencies(2 * n, case["scaling"])
            at += n
    state["freqs"], state["scale"] = f.cuda(), scale
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    return (_prepare_gn if case["op"].startswith("gn") else _prepare_rope)(case, gen)


# ---- the plain forms --------------------------------------------------------

def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return z * 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_grad(z, act):
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    return torch.ones_like(z)


def _params(p, N, G):
    """gamma or beta as [N or 1, 1, G, channels of a group], 32 bits."""
    return p.float().reshape(N if p.dim() == 2 else 1, 1, G, -1)


def _plain_gn_fwd(s):
    c = s["case"]
    N, R, C, G = c["samples"], c["rows"], c["channels"], c["groups"]
    x = s["x"].float().reshape(N, R, G, C // G)
    mean = x.mean(dim=(1, 3), keepdim=True)
    d = x - mean
    rstd = 1 / torch.sqrt((d * d).mean(dim=(1, 3), keepdim=True) + c["eps"])
    z = d * rstd * _params(s["gamma"], N, G) + _params(s["beta"], N, G)
    y = _act(z, c["act"]).reshape(N, R, C).to(s["x"].dtype)
    return {"y": y, "mean": mean.reshape(N, G), "rstd": rstd.reshape(N, G)}


def _plain_gn_bwd(s):
    c = s["case"]
    N, R, C, G = c["samples"], c["rows"], c["channels"], c["groups"]
    per = C // G
    rstd = s["rstd"].reshape(N, 1, G, 1)
    xhat = (s["x"].float().reshape(N, R, G, per) - s["mean"].reshape(N, 1, G, 1)) * rstd
    w = _params(s["gamma"], N, G)
    dz = s["dy"].float().reshape(N, R, G, per) * _act_grad(xhat * w + _params(s["beta"], N, G), c["act"])
    a, b = dz.sum(dim=1, keepdim=True), (dz * xhat).sum(dim=1, keepdim=True)
    c1 = (w * a).sum(dim=3, keepdim=True) / (R * per)
    c2 = (w * b).sum(dim=3, keepdim=True) / (R * per)
    dx = (rstd * (w * dz - c1 - xhat * c2)).reshape(N, R, C).to(s["x"].dtype)
    a, b = a.reshape(N, C), b.reshape(N, C)
    if c["affine"] == "channel":
        a, b = a.sum(dim=0), b.sum(dim=0)
    return {"dx": dx, "dgamma": b, "dbeta": a}


def _cos_sin(s):
    """cos and sin of the angles, [batch, tokens, 1, pairs], from 64 bits."""
    pos = s["positions"].double()
    f = s["freqs"]
    angle = pos[..., None] * f if f.dim() == 1 else (pos[..., None] * f[:, None, None]).sum(dim=0)
    angle = angle[:, :, None]
    return (angle.cos() * s["scale"]).float(), (angle.sin() * s["scale"]).float()


def _rotate(u, cos, sin, c):
    """The rotation of the first `rot` elements of the heads; the others stay."""
    rot = c["rot"]
    if c["layout"] == "half":
        a, b = u[..., :rot // 2], u[..., rot // 2:rot]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    else:
        a, b = u[..., 0:rot:2], u[..., 1:rot:2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    return torch.cat((r, u[..., rot:]), dim=-1) if rot < c["dim"] else r


def _plain_rope_fwd(s):
    c = s["case"]
    cos, sin = _cos_sin(s)
    out = {}
    for name in ("q", "k"):
        u = s[name].float()
        if c["norm"]:
            u = u / torch.sqrt((u * u).mean(dim=-1, keepdim=True) + c["eps"]) * s[name + "_gamma"].float()
        out[name] = _rotate(u, cos, sin, c).to(s[name].dtype)
    return out


def _plain_rope_bwd(s):
    c = s["case"]
    cos, sin = _cos_sin(s)
    out = {}
    for name in ("q", "k"):
        g = _rotate(s["d" + name].float(), cos, -sin, c)
        if c["norm"]:
            x = s[name].float()
            rstd = 1 / torch.sqrt((x * x).mean(dim=-1, keepdim=True) + c["eps"])
            xhat = x * rstd
            out["d%s_gamma" % name] = (g * xhat).sum(dim=(0, 1, 2))
            g = g * s[name + "_gamma"].float()
            g = rstd * (g - xhat * (g * xhat).mean(dim=-1, keepdim=True))
        out["d" + name] = g.to(s[name].dtype)
    return out


# ---- through the package ----------------------------------------------------

def _own(s):
    import normalization_fwd_gb300 as nf
    c = s["case"]
    if c["op"] == "gn_fwd":
        return nf.fused_group_norm_fwd(s["x"], c["groups"], s["gamma"], s["beta"], eps=c["eps"],
                                       activation=c["act"])
    if c["op"] == "gn_bwd":
        return nf.fused_group_norm_bwd(s["dy"], s["x"], c["groups"], s["gamma"], s["beta"],
                                       s["mean"], s["rstd"], activation=c["act"])
    kw = dict(q_gamma=s["q_gamma"], k_gamma=s["k_gamma"], eps=c["eps"], scale=s["scale"],
              interleaved=c["layout"] == "interleaved")
    if c["op"] == "rope_fwd":
        return nf.fused_rope_fwd(s["q"], s["k"], s["positions"], s["freqs"], **kw)
    q, k = (s["q"], s["k"]) if c["norm"] else (None, None)
    out = nf.fused_rope_bwd(s["dq"], s["dk"], s["positions"], s["freqs"], q=q, k=k, **kw)
    return {name: t for name, t in out.items() if t is not None}


def run(state):
    if own:
        return _own(state)
    return {"gn_fwd": _plain_gn_fwd, "gn_bwd": _plain_gn_bwd, "rope_fwd": _plain_rope_fwd,
            "rope_bwd": _plain_rope_bwd}[state["case"]["op"]](state)


def work(case):
    es = SIZE[case["dtype"]]
    if case["op"].startswith("gn"):
        N, C = case["samples"], case["channels"]
        n = N * case["rows"] * C
        small = 8 * N * case["groups"] + 2 * es * C * (N if case["affine"] == "sample" else 1)
        if case["op"] == "gn_fwd":
            return {"bytes": 2 * n * es + small, "flops": 10 * n}
        return {"bytes": 3 * n * es + small + 8 * C * (N if case["affine"] == "sample" else 1),
                "flops": 25 * n}
    tokens = case["batch"] * case["tokens"]
    n = tokens * (case["heads"] + case["kv_heads"]) * case["dim"]
    small = 8 * tokens * case["axes"] + 4 * case["axes"] * case["rot"]
    passes = 3 if case["op"] == "rope_bwd" and case["norm"] else 2
    return {"bytes": passes * n * es + small, "flops": 8 * n}


# ---- 64 bits ----------------------------------------------------------------

def _phi(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def _exact_gn(s):
    c = s["case"]
    N, R, C, G = c["samples"], c["rows"], c["channels"], c["groups"]
    per_channel = lambda t: t.double().repeat_interleave(C // G, dim=-1)  # noqa: E731
    rows = []
    for n in range(N):
        x = s["x"][n].double()
        w = (s["gamma"][n] if s["gamma"].dim() == 2 else s["gamma"]).double()
        b = (s["beta"][n] if s["beta"].dim() == 2 else s["beta"]).double()
        if c["op"] == "gn_fwd":
            m = x.mean(dim=0).reshape(G, -1).mean(dim=1)
            x.sub_(per_channel(m))
            v = x.square().mean(dim=0).reshape(G, -1).mean(dim=1)
            r = (v + c["eps"]).pow(-0.5)
            z = x.mul_(per_channel(r) * w).add_(b)
        else:
            m, r = s["mean"][n].double(), s["rstd"][n].double()
            x.sub_(per_channel(m)).mul_(per_channel(r))
            z = x * w + b
        if c["op"] == "gn_fwd":
            y = z * torch.sigmoid(z) if c["act"] == "silu" else z * _phi(z) if c["act"] == "gelu" else z
            rows.append((y, m, r))
            continue
        if c["act"] == "silu":
            sig = torch.sigmoid(z)
            slope = sig + z * sig * torch.sigmoid(-z)
        elif c["act"] == "gelu":
            slope = _phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        else:
            slope = torch.ones_like(z)
        g = s["dy"][n].double() * slope
        a, bb = g.sum(dim=0), (g * x).sum(dim=0)
        mean_of = lambda t: per_channel((t * w).reshape(G, -1).sum(dim=1) / (R * (C // G)))  # noqa: E731
        dx = per_channel(r) * (g * w - mean_of(a) - x * mean_of(bb))
        rows.append((dx, bb, a))
    first, second, third = (torch.stack(t) for t in zip(*rows))
    if c["op"] == "gn_fwd":
        return {"y": first, "mean": second, "rstd": third}
    if c["affine"] == "channel":
        second, third = second.sum(dim=0), third.sum(dim=0)
    return {"dx": first, "dgamma": second, "dbeta": third}


def _exact_rope(s):
    c = s["case"]
    f = s["freqs"] if s["freqs"].dim() == 2 else s["freqs"][None]
    pos = s["positions"] if s["positions"].dim() == 3 else s["positions"][None]
    angle = torch.einsum("abt,aj->btj", pos.double(), f)
    turn = torch.polar(torch.full_like(angle, s["scale"]), angle)[:, :, None]   # s e^(i angle)
    rot, out = c["rot"], {}
    for name in ("q", "k"):
        x = s[name].double()
        w = s[name + "_gamma"].double() if c["norm"] else None
        rstd = (x.square().sum(dim=-1, keepdim=True) / c["dim"] + c["eps"]).pow(-0.5) if c["norm"] else 1.0
        v = (x * rstd * w if c["norm"] else x) if c["op"] == "rope_fwd" else s["d" + name].double()
        pair = v[..., :rot].unflatten(-1, (2, -1)).transpose(-1, -2) if c["layout"] == "half" else v[..., :rot].unflatten(-1, (-1, 2))
        r = torch.complex(pair[..., 0].contiguous(), pair[..., 1].contiguous())
        r = torch.view_as_real(r * (turn if c["op"] == "rope_fwd" else turn.conj()))
        r = r.transpose(-1, -2) if c["layout"] == "half" else r
        v = torch.cat((r.flatten(-2), v[..., rot:]), dim=-1)
        if c["op"] == "rope_fwd":
            out[name] = v
            continue
        if c["norm"]:
            xhat = x * rstd
            out["d%s_gamma" % name] = torch.einsum("bthd,bthd->d", v, xhat)
            g = v * w
            v = rstd * (g - xhat * ((g * xhat).sum(dim=-1, keepdim=True) / c["dim"]))
        out["d" + name] = v
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_gn(s) if case["op"].startswith("gn") else _exact_rope(s)

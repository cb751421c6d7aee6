"""Cases of the experts' own products and of what feeds them: linear layers of
rows sorted by expert with the activation and the gate's product in the same
pass, and their gradients; the same with 4-bit weights and group scales, for
decode batches; and the norm before the layer with its output in 8 bits.

``run`` computes an operator in its plain form (elementary torch operations
in 32 bits, rounded once at the end) or, where ``own`` is true, through the
library's calls.  ``exact`` gives the same outputs from the definitions in 64
bits.
"""
import math

import torch

own = False

_DEV = "cuda"
_GATED = ("silu", "gelu", "gelu_tanh", "swigluoai", "swiglustep")
_SINGLE = ("silu_no_mul", "gelu_no_mul", "gelu_tanh_no_mul", "relu2_no_mul")


def listed():
    return [
        # one sequence's token through a shared expert's gated half: a call's latency and
        # one pass over the weights
        dict(name="linear one token", op="linear", R=1, E=1, K=7168, N=2048,
             dtype="bfloat16", act="silu", limit=0.0, pad=0.0, keep=False, grad=False),
        # the rows of a decode batch of 32 tokens, sorted by expert: few rows for each
        dict(name="linear decode", op="linear", R=256, E=64, K=4096, N=1024,
             dtype="bfloat16", act="silu", limit=0.0, pad=0.0, keep=False, grad=False),
        # the largest: a training batch's gated half forward, pre-activations kept
        dict(name="linear training", op="linear", R=32768, E=32, K=7168, N=2048,
             dtype="bfloat16", act="silu", limit=0.0, pad=0.05, keep=True, grad=False),
        # the same half's gradients: rows and weights
        dict(name="linear gradients", op="linear", R=16384, E=32, K=4096, N=2048,
             dtype="bfloat16", act="silu", limit=0.0, pad=0.05, keep=True, grad=True),
        # odd sizes all round, a down projection's gradients
        dict(name="linear odd", op="linear", R=8191, E=60, K=1001, N=2047,
             dtype="float16", act="none", limit=0.0, pad=0.1, keep=False, grad=True),
        # 32-bit rows, as a master-precision run or a check of one has them
        dict(name="linear float32", op="linear", R=2051, E=8, K=2048, N=1408,
             dtype="float32", act="gelu_tanh", limit=0.0, pad=0.0, keep=False, grad=False),
        # one token through a shared expert's projection with 4-bit weights
        dict(name="w4 one token", op="w4", R=1, E=1, K=7168, N=4096, dtype="bfloat16",
             act="none", limit=0.0, pad=0.0, format="int4", group=128, scales="bfloat16"),
        # a decode batch of 64 tokens, 8 experts each, through the gated half of MXFP4 experts
        dict(name="w4 decode", op="w4", R=512, E=128, K=4096, N=2048, dtype="bfloat16",
             act="silu", limit=0.0, pad=0.0, format="mxfp4", group=32, scales="uint8"),
        # an odd batch of sequences, zero points, 16-bit scales for groups of 64
        dict(name="w4 batch", op="w4", R=37, E=1, K=14336, N=4096, dtype="float16",
             act="none", limit=0.0, pad=0.0, format="int4_zero", group=64,
             scales="float16"),
        # between two blocks of a decode batch: the next layer's input leaves the norm staged
        dict(name="norm quant decode", op="norm", T=32, H=7168, dtype="bfloat16",
             weights="bfloat16", y=True, post=True, gate="token", sigmoid=True, scale=1.0,
             offset=0.0, keep=True, quant="ue8m0"),
        # the same behind a long prefill, which keeps no 16-bit copy
        dict(name="norm quant prefill", op="norm", T=16381, H=7168, dtype="bfloat16",
             weights="bfloat16", y=True, post=False, gate="none", sigmoid=False, scale=1.0,
             offset=0.0, keep=False, quant="fp32"),
        # a first norm without a block before it, groups of 32, 16-bit floats
        dict(name="norm quant mx", op="norm", T=4099, H=4096, dtype="float16",
             weights="float32", y=False, post=False, gate="none", sigmoid=False, scale=1.0,
             offset=1.0, keep=True, quant="mxfp8"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "w4", "norm"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
    if op == "norm":
        H = 128 * _log_uniform(rng, 1, 64)
        T = min(_log_uniform(rng, 1, 16384), 16381 * 7168 // H)
        return dict(op=op, T=T, H=H, dtype=dtype, weights=rng.choice([dtype, "float32"]),
                    y=rng.random() < 0.8, post=rng.random() < 0.6,
                    gate=rng.choice(["none", "token", "channel", "full"]),
                    sigmoid=rng.random() < 0.5, scale=rng.choice([1.0, 0.22]),
                    offset=rng.choice([0.0, 1.0]), keep=rng.random() < 0.5,
                    quant=rng.choice(["ue8m0", "fp32", "mxfp8"]))
    act = rng.choice(["none", "silu", "silu", rng.choice(_GATED), rng.choice(_SINGLE)])
    limit = rng.choice([0.0, 1.5]) if act in ("silu", "swigluoai", "swiglustep") else 0.0
    E = rng.choice([1, 1, 4, 8, 16, 60, 64, 128])
    gates = 2 if act in _GATED else 1
    N = _log_uniform(rng, 64, 8192)
    if rng.random() < 0.6:
        N = (N + 63) // 64 * 64
    if op == "w4":
        K = 128 * _log_uniform(rng, 2, 112)
        N = max(1, min(N, (1 << 31) // (E * gates * K)))
        R = _log_uniform(rng, 1, 64) if E == 1 else _log_uniform(rng, 8, 1024)
        form = rng.choice(["int4", "int4_zero", "mxfp4"])
        group = 32 if form == "mxfp4" else rng.choice([32, 64, 128])
        scales = "uint8" if form == "mxfp4" else rng.choice([dtype, "float32"])
        return dict(op=op, R=R, E=E, K=K, N=N, dtype=dtype, act=act, limit=limit,
                    pad=rng.choice([0.0, 0.1]), format=form, group=group, scales=scales)
    K = _log_uniform(rng, 64, 8192)
    if rng.random() < 0.7:
        K = (K + 63) // 64 * 64
    # no more weights and products than the largest listed case has
    grad = rng.random() < 0.5
    N = max(1, min(N, (1 << 29) // ((4 if dtype == "float32" else 1) * (1 + grad) *
                                    E * gates * K)))
    most = 32768 * 7168 * 4096 // 4 // (10 if dtype == "float32" else 1)
    R = min(_log_uniform(rng, 1, 32768), max(8, most // (gates * K * N)))
    return dict(op=op, R=R, E=E, K=K, N=N, dtype=dtype, act=act, limit=limit,
                pad=rng.choice([0.0, 0.1]), keep=grad and act != "none" or
                act != "none" and rng.random() < 0.3, grad=grad)


def _routed(c):
    return c["R"] - int(c["pad"] * c["R"])


def _wide(c):
    """Columns of the product before the activation."""
    return c["N"] * (2 if c["act"] in _GATED else 1)


def _size(name):
    return {"float32": 4, "uint8": 1}.get(name, 2)


def work(c):
    size = _size(c["dtype"])
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        gates = {"none": 0, "token": T, "channel": H, "full": T * H}[c["gate"]] if c["y"] else 0
        vecs = (1 + (c["y"] and c["post"])) * H * _size(c["weights"]) + gates * size
        groups = T * (H // (32 if c["quant"] == "mxfp8" else 128))
        out = T * H + groups * (4 if c["quant"] == "fp32" else 1)
        streams = (3 if c["y"] else 1) + bool(c["keep"])
        return {"bytes": streams * T * H * size + vecs + out, "flops": 14 * T * H}
    rows, K, N, wide = _routed(c), c["K"], c["N"], _wide(c)
    experts = min(c["E"], rows)
    if c["op"] == "w4":
        groups = wide * (K // c["group"])
        zeros = groups if c["format"] == "int4_zero" else 0
        weights = wide * K // 2 + groups * _size(c["scales"]) + zeros
        return {"bytes": experts * weights + rows * (K + N) * size, "flops": 2 * rows * wide * K}
    weights = wide * K * size
    if not c["grad"]:
        kept = wide if c["keep"] else 0
        return {"bytes": experts * weights + rows * (K + N + kept) * size,
                "flops": 2 * rows * wide * K}
    kept = wide if c["act"] != "none" else 0
    return {"bytes": (experts + c["E"]) * weights + rows * (2 * K + N + kept) * size,
            "flops": 4 * rows * wide * K}


def _normal(g, dtype, *shape, std=1.0, mean=0.0):
    t = torch.empty(shape, dtype=torch.float32, device=_DEV)
    return t.normal_(mean, std, generator=g).to(dtype)


def _offsets(c, g):
    """Rows per expert of uneven popularity, as offsets, and the most that one has."""
    if c["E"] == 1 and not c["pad"]:
        return None, c["R"]
    E, n = c["E"], _routed(c)
    like = torch.softmax(0.7 * torch.randn(E, generator=g, device=_DEV), 0)
    pick = torch.multinomial(like, max(n, 1), replacement=True, generator=g)[:n]
    counts = torch.bincount(pick, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=_DEV)
    offsets[1:] = counts.cumsum(0)
    return offsets, int(counts.max())


def prepare(c, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    dt = getattr(torch, c["dtype"])
    s = {"c": c}
    if c["op"] == "norm":
        T, H, wt = c["T"], c["H"], getattr(torch, c["weights"])
        # a residual stream has a few channels far above the others
        loud = torch.exp(0.8 * torch.randn(H, generator=g, device=_DEV))
        s["residual"] = (_normal(g, torch.float32, T, H) * loud).to(dt)
        s["y"] = _normal(g, dt, T, H, std=0.7) if c["y"] else None
        s["pre_weight"] = _normal(g, wt, H, std=0.1, mean=1.0 - c["offset"])
        s["post_weight"] = (_normal(g, wt, H, std=0.1, mean=1.0 - c["offset"])
                            if c["y"] and c["post"] else None)
        shape = {"none": None, "token": (T,), "channel": (H,), "full": (T, H)}[c["gate"]]
        s["gate"] = _normal(g, dt, *shape) if shape and c["y"] else None
        G = H // (32 if c["quant"] == "mxfp8" else 128)
        width = {"ue8m0": (G + 3) // 4 * 4, "fp32": G, "mxfp8": G}[c["quant"]]
        s["codes"] = torch.empty((T, H), dtype=torch.uint8, device=_DEV)
        s["scales"] = torch.empty((T, width), device=_DEV,
                                  dtype=torch.float32 if c["quant"] == "fp32" else torch.uint8)
        s["out"] = {"x_q": s["codes"].view(torch.float8_e4m3fn),
                    "x_sf": s["scales"] if c["quant"] == "fp32"
                    else s["scales"].view(torch.float8_e8m0fnu)}
        if c["y"]:
            s["out"]["residual_out"] = torch.empty_like(s["residual"])
        if c["keep"]:
            s["out"]["normed"] = torch.empty_like(s["residual"])
    else:
        R, E, K, N, wide = c["R"], c["E"], c["K"], c["N"], _wide(c)
        s["offsets"], s["most"] = _offsets(c, g)
        s["x"] = _normal(g, dt, R, K)
        std = 1.0 / math.sqrt(K)
        # rows behind the last routed one stay as they are: zeros here
        if c["op"] == "w4":
            G = K // c["group"]
            s["codes"] = torch.randint(0, 256, (E, wide, K // 2), generator=g, device=_DEV,
                                       dtype=torch.uint8)
            if c["format"] == "mxfp4":
                mid = 127 + int(round(math.log2(std / 2.6)))
                s["scales"] = torch.randint(mid - 2, mid + 2, (E, wide, G), generator=g,
                                            device=_DEV, dtype=torch.uint8)
            else:
                spread = torch.exp(0.4 * torch.randn((E, wide, G), generator=g, device=_DEV))
                s["scales"] = (spread * (std / 4.6)).to(getattr(torch, c["scales"]))
            s["zeros"] = (torch.randint(0, 16, (E, wide, G), generator=g, device=_DEV,
                                        dtype=torch.uint8)
                          if c["format"] == "int4_zero" else None)
            s["out"] = {"out": torch.zeros((R, N), dtype=dt, device=_DEV)}
        else:
            s["weight"] = _normal(g, dt, E, wide, K, std=std)
            if c["grad"]:
                s["pre_act"] = _normal(g, dt, R, wide, std=1.2) if c["act"] != "none" else None
                s["grad_out"] = _normal(g, dt, R, N)
                s["out"] = {"grad_x": torch.zeros_like(s["x"]),
                            "grad_weight": torch.empty_like(s["weight"])}
            else:
                s["out"] = {"out": torch.zeros((R, N), dtype=dt, device=_DEV)}
                if c["keep"]:
                    s["out"]["pre_act"] = torch.zeros((R, wide), dtype=dt, device=_DEV)
    if own:
        s["plan"], s["ws"] = _plan(c)
    return s


def _plan(c):
    """The descriptor and the workspace a program keeps beside its buffers."""
    import fp8_block_quantized_group_amd as moe
    dt = getattr(torch, c["dtype"])
    if c["op"] == "norm":
        return moe.BlockNorm(c["T"], c["H"], dtype=dt, weight_dtype=getattr(torch, c["weights"]),
                             post_norm=c["y"] and c["post"], gate=c["gate"] if c["y"] else "none",
                             gate_sigmoid=c["sigmoid"], eps=1e-6, residual_scale=c["scale"],
                             weight_offset=c["offset"]), None
    if c["op"] == "w4":
        return moe.ExpertLinearW4(c["R"], c["K"], c["N"], c["E"], dtype=dt, activation=c["act"],
                                  act_limit=c["limit"], format=c["format"],
                                  group_size=c["group"],
                                  scale_dtype=getattr(torch, c["scales"])), None
    p = moe.ExpertLinear(c["R"], c["K"], c["N"], c["E"], dtype=dt, activation=c["act"],
                         act_limit=c["limit"])
    return p, moe.alloc_expert_linear_workspace(p, _DEV) if c["grad"] else None


def run(s):
    if own:
        return _run_own(s)
    c = s["c"]
    if c["op"] == "norm":
        return _plain_norm(s)
    if c["op"] == "w4":
        return {"out": _plain_linear(s, _plain_dequant(s))[0]}
    if c["grad"]:
        return _plain_linear_grad(s)
    out, pre = _plain_linear(s, s["weight"].float())
    return {"out": out, "pre_act": pre} if c["keep"] else {"out": out}


def _run_own(s):
    import fp8_block_quantized_group_amd as moe
    c, p, out = s["c"], s["plan"], s["out"]
    if c["op"] == "norm":
        moe.block_norm_quant(p, s["residual"], s["codes"], s["scales"], quant=c["quant"],
                             normed=out.get("normed"), y=s["y"],
                             residual_out=out.get("residual_out"), pre_weight=s["pre_weight"],
                             post_weight=s["post_weight"], gate=s["gate"])
    elif c["op"] == "w4":
        moe.expert_linear_w4(p, s["x"], s["codes"], s["scales"], out["out"],
                             expert_offsets=s["offsets"], zeros=s["zeros"])
    elif c["grad"]:
        moe.expert_linear_backward(p, s["x"], s["weight"], s["grad_out"], out["grad_x"],
                                   out["grad_weight"], expert_offsets=s["offsets"],
                                   pre_act=s["pre_act"], ws=s["ws"])
    else:
        moe.expert_linear(p, s["x"], s["weight"], out["out"], expert_offsets=s["offsets"],
                          pre_act=out.get("pre_act"))
    return out


# ---- plain forms ------------------------------------------------------------

def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _limit(c):
    """The clamp limit, 0 for none."""
    if c["act"] in ("swigluoai", "swiglustep"):
        return c["limit"] or 7.0
    return c["limit"] if c["act"] == "silu" else 0.0


def _half(act, x):
    """f(x) and f'(x) of an activation without its clamps."""
    if act.startswith("silu") or act == "swiglustep":
        p = _sigmoid(x)
        return x * p, p * (1.0 + x * _sigmoid(-x))
    if act == "swigluoai":
        p = _sigmoid(1.702 * x)
        return x * p, p * (1.0 + 1.702 * x * _sigmoid(-1.702 * x))
    if act.startswith("gelu_tanh"):
        a, b = 2.0 * math.sqrt(2.0 / math.pi), 0.044715
        p = _sigmoid(a * (x + b * x * x * x))
        q = _sigmoid(-a * (x + b * x * x * x))
        return x * p, p * (1.0 + x * q * a * (1.0 + 3.0 * b * x * x))
    if act.startswith("gelu"):
        p = 0.5 * torch.special.erfc(x * -math.sqrt(0.5))
        return x * p, p + x * torch.exp(-0.5 * x * x) * (1.0 / math.sqrt(2.0 * math.pi))
    r = x.clamp_min(0.0)
    return r * r, 2.0 * r


def _activate(c, v):
    act, L = c["act"], _limit(c)
    if act == "none":
        return v
    if act not in _GATED:
        return _half(act, v)[0]
    x, u = v[..., :c["N"]], v[..., c["N"]:]
    if L > 0.0:
        u = u.clamp(-L, L)
        if act != "swiglustep":
            x = x.clamp_max(L)
    f = _half(act, x)[0]
    if act == "swiglustep":
        f = f.clamp_max(L)
    return f * (u + 1.0 if act == "swigluoai" else u)


def _activate_grad(c, v, dh):
    act, L = c["act"], _limit(c)
    if act == "none":
        return dh
    if act not in _GATED:
        return _half(act, v)[1] * dh
    x, u = v[..., :c["N"]], v[..., c["N"]:]
    live_x = live_u = torch.ones((), device=v.device)
    if L > 0.0:
        live_u = (u.abs() <= L).float()
        u = u.clamp(-L, L)
        if act != "swiglustep":
            live_x = (x <= L).float()
            x = x.clamp_max(L)
    f, df = _half(act, x)
    if act == "swiglustep":
        live_x = (f <= L).float()
        f = f.clamp_max(L)
    if act == "swigluoai":
        u = u + 1.0
    return torch.cat([dh * u * df * live_x, dh * f * live_u], dim=-1)


def _places(s):
    """Rows of every expert, [E, most], and which of them there are; None for all rows of one."""
    if s["offsets"] is None:
        return None
    o = s["offsets"].long()
    at = o[:-1, None] + torch.arange(s["most"], device=o.device)
    live = at < o[1:, None]
    return torch.where(live, at, s["c"]["R"]), live


def _spread(rows, places):
    """Rows as [E, most, width], zeros where an expert has fewer."""
    if places is None:
        return rows.float()[None]
    at, live = places
    if not rows.shape[0] or not at.numel():
        return rows.new_zeros((*at.shape, rows.shape[1]), dtype=torch.float32)
    return rows[at.clamp_max(rows.shape[0] - 1)].float() * live[:, :, None]


def _gather(v, places, R, dtype):
    """[E, most, width] back to rows, zeros behind the last routed one."""
    if places is None:
        return v[0].to(dtype)
    out = torch.zeros((R + 1, v.shape[2]), dtype=dtype, device=v.device)
    out[places[0].view(-1)] = v.to(dtype).view(-1, v.shape[2])
    return out[:R]


def _plain_linear(s, w):
    c, dt = s["c"], s["x"].dtype
    places = _places(s)
    pre = torch.bmm(_spread(s["x"], places), w.transpose(1, 2))
    out = _gather(_activate(c, pre), places, c["R"], dt)
    return out, _gather(pre, places, c["R"], dt) if c.get("keep") else None


def _plain_linear_grad(s):
    c, dt = s["c"], s["x"].dtype
    places = _places(s)
    dh = _spread(s["grad_out"], places)
    pre = _spread(s["pre_act"], places) if s["pre_act"] is not None else None
    d = _activate_grad(c, pre, dh)
    return {"grad_x": _gather(torch.bmm(d, s["weight"].float()), places, c["R"], dt),
            "grad_weight": torch.bmm(d.transpose(1, 2), _spread(s["x"], places)).to(dt)}


def _plain_dequant(s):
    c = s["c"]
    codes = torch.stack([s["codes"] & 15, s["codes"] >> 4], dim=-1)
    E, wide = codes.shape[:2]
    codes = codes.view(E, wide, -1, c["group"])
    if c["format"] == "mxfp4":
        table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6],
                             dtype=torch.float32, device=codes.device)
        q = table[codes.int()]
        scale = torch.exp2(s["scales"].float() - 127.0)
    else:
        zero = 8.0 if s["zeros"] is None else s["zeros"].float()[..., None]
        q = codes.float() - zero
        scale = s["scales"].float()
    return (q * scale[..., None]).view(E, wide, -1)


def _plain_norm(s):
    c, r = s["c"], s["residual"].float()
    out = {}
    if s["y"] is not None:
        n = s["y"].float()
        if s["post_weight"] is not None:
            n = n * torch.rsqrt((n * n).mean(1, keepdim=True) + 1e-6)
            n = n * (s["post_weight"].float() + c["offset"])
        if s["gate"] is not None:
            g = s["gate"].float()
            g = _sigmoid(g) if c["sigmoid"] else g
            n = n * (g[:, None] if c["gate"] == "token" else g)
        r = r + c["scale"] * n
        out["residual_out"] = r.to(s["residual"].dtype)
    h = r * torch.rsqrt((r * r).mean(1, keepdim=True) + 1e-6)
    h = h * (s["pre_weight"].float() + c["offset"])
    if c["keep"]:
        out["normed"] = h.to(s["residual"].dtype)
    T, H = h.shape
    v = h.view(T, -1, 32 if c["quant"] == "mxfp8" else 128)
    scale = v.abs().amax(2).clamp_min(1e-4) / 448.0
    if c["quant"] == "fp32":
        out["x_sf"] = scale
    else:
        bits = scale.view(torch.int32)
        e = ((bits >> 23) + ((bits & 0x7FFFFF) != 0).int()).clamp(1, 254)
        scale = (e << 23).view(torch.float32)
        more = s["scales"].shape[1] - e.shape[1]
        out["x_sf"] = torch.nn.functional.pad(e.to(torch.uint8), (0, more)).view(
            torch.float8_e8m0fnu)
    q = (v * (1.0 / scale)[:, :, None]).clamp(-448.0, 448.0)
    out["x_q"] = q.view(T, H).to(torch.float8_e4m3fn)
    return out


# ---- definitions in 64 bits -------------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    return {"norm": _exact_norm, "w4": _exact_w4, "linear": _exact_linear}[c["op"]](s)


def _define(c, pre):
    """The activation from its definition."""
    act, N, L = c["act"], c["N"], _limit(c)
    if act == "none":
        return pre
    gate, up = (pre[:, :N], pre[:, N:]) if act in _GATED else (pre, None)
    if L > 0.0:
        up = torch.clamp(up, -L, L)
        if act != "swiglustep":
            gate = torch.clamp(gate, max=L)
    kind = act.replace("_no_mul", "")
    if kind in ("silu", "swiglustep"):
        f = gate * torch.sigmoid(gate)
        if act == "swiglustep":
            f = torch.clamp(f, max=L)
    elif kind == "swigluoai":
        f = gate * torch.sigmoid(1.702 * gate)
        up = up + 1.0
    elif kind == "gelu":
        f = 0.5 * gate * (1.0 + torch.erf(gate / math.sqrt(2.0)))
    elif kind == "gelu_tanh":
        inner = math.sqrt(2.0 / math.pi) * (gate + 0.044715 * gate ** 3)
        f = 0.5 * gate * (1.0 + torch.tanh(inner))
    else:
        f = torch.relu(gate) ** 2
    return f if up is None else f * up


def _experts(s):
    if s["offsets"] is None:
        return [(0, 0, s["c"]["R"])]
    o = s["offsets"].tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1)]


def _exact_linear(s):
    c, x = s["c"], s["x"].double()
    if not c["grad"]:
        out = {k: torch.zeros(v.shape, dtype=torch.float64, device=_DEV)
               for k, v in s["out"].items()}
        for e, a, b in _experts(s):
            pre = x[a:b] @ s["weight"][e].double().t()
            out["out"][a:b] = _define(c, pre)
            if c["keep"]:
                out["pre_act"][a:b] = pre
        return out
    gx = torch.zeros(x.shape, dtype=torch.float64, device=_DEV)
    gw = torch.zeros(s["weight"].shape, dtype=torch.float64, device=_DEV)
    for e, a, b in _experts(s):
        d = s["grad_out"][a:b].double()
        if c["act"] != "none":
            pre = s["pre_act"][a:b].double().requires_grad_()
            d, = torch.autograd.grad(_define(c, pre), pre, d)
        gx[a:b] = d @ s["weight"][e].double()
        gw[e] = d.t() @ x[a:b]
    return {"grad_x": gx, "grad_weight": gw}


def _exact_w4(s):
    c, x = s["c"], s["x"].double()
    out = torch.zeros(s["out"]["out"].shape, dtype=torch.float64, device=_DEV)
    for e, a, b in _experts(s):
        byte = s["codes"][e].long()
        q = torch.empty((byte.shape[0], c["K"]), dtype=torch.long, device=_DEV)
        q[:, 0::2], q[:, 1::2] = byte % 16, byte // 16
        if c["format"] == "mxfp4":          # sign, two exponent bits, one mantissa bit
            sign, ex, m = 1 - 2 * (q // 8), q // 2 % 4, q % 2
            v = torch.where(ex > 0, 2.0 ** (ex - 1).double() * (1.0 + 0.5 * m), 0.5 * m) * sign
            scale = 2.0 ** (s["scales"][e].double() - 127.0)
        else:
            zero = 8 if s["zeros"] is None else s["zeros"][e].long().repeat_interleave(
                c["group"], dim=1)
            v = (q - zero).double()
            scale = s["scales"][e].double()
        w = v * scale.repeat_interleave(c["group"], dim=1)
        out[a:b] = _define(c, x[a:b] @ w.t())
    return {"out": out}


def _exact_norm(s):
    c = s["c"]
    r = s["residual"].double()

    def norm(v, weight):
        n = v / torch.sqrt(torch.mean(v ** 2, dim=1, keepdim=True) + 1e-6)
        return n * (c["offset"] + weight.double())

    out = {}
    if s["y"] is not None:
        n = s["y"].double()
        if s["post_weight"] is not None:
            n = norm(n, s["post_weight"])
        if s["gate"] is not None:
            g = s["gate"].double()
            g = torch.sigmoid(g) if c["sigmoid"] else g
            n = n * (g.unsqueeze(1) if c["gate"] == "token" else g)
        r = out["residual_out"] = r + c["scale"] * n
    h = norm(r, s["pre_weight"])
    if c["keep"]:
        out["normed"] = h
    wide = 32 if c["quant"] == "mxfp8" else 128
    groups = h.reshape(h.shape[0], -1, wide)
    # the floor is a 32-bit number
    scale = groups.abs().amax(dim=2).clamp_min(
        float(torch.tensor(1e-4, dtype=torch.float32))) / 448.0
    sf = scale
    if c["quant"] != "fp32":
        scale = 2.0 ** torch.ceil(torch.log2(scale))
        sf = torch.full(s["scales"].shape, 2.0 ** -127, dtype=torch.float64, device=_DEV)
        sf[:, :scale.shape[1]] = scale
    v = (groups / scale.unsqueeze(2)).clamp(-448.0, 448.0)
    # e4m3: three bits after the leading one, steps of 2^-9 below 2^-6
    step = 2.0 ** (torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3.0)
    out["x_q"] = (torch.round(v / step) * step).reshape(h.shape)
    out["x_sf"] = sf
    return out

"""Cases of the operators around the expert layer: the router's choice of
experts, tokens sorted by expert and combined back, and the norms before and
after the block, each with its gradient.

``run`` computes an operator in its plain form (elementary torch operations
in 32 bits, rounded once at the end) or, where ``own`` is true, through the
library's calls.  ``exact`` gives the same outputs from the definitions in 64
bits.
"""
import math

import torch

own = False

_DEV = "cuda"
_FLT_MAX = torch.finfo(torch.float32).max


def listed():
    return [
        # one decode step of a few sequences: the call's own latency
        dict(name="router decode", op="router", T=4, E=256, k=8, dtype="float32",
             score="sigmoid", bias=True, groups=8, topk_groups=4, group_top=2,
             renormalize=True, scale=2.5, masked=0, pad=0.0, grad=False),
        # a long prefill batch with padding tokens, group-limited sigmoid routing
        dict(name="router prefill", op="router", T=16384, E=256, k=8, dtype="float32",
             score="sigmoid", bias=True, groups=8, topk_groups=4, group_top=2,
             renormalize=True, scale=2.5, masked=0, pad=0.05, grad=False),
        # a training step with an odd batch, softmax over all experts, three of
        # them out of service; the gradient is dense over the experts
        dict(name="router training", op="router", T=8191, E=128, k=8, dtype="bfloat16",
             score="softmax", bias=False, groups=1, topk_groups=1, group_top=1,
             renormalize=False, scale=1.0, masked=3, pad=0.0, grad=True),
        # a decode batch sorted by expert
        dict(name="sort decode", op="sort", T=64, E=256, k=8, H=7168, dtype="bfloat16",
             pad=0.0, grad=False),
        # ragged everything: odd hidden size, odd batch, experts not a power of two
        dict(name="sort odd", op="sort", T=2049, E=60, k=6, H=1001, dtype="float16",
             pad=0.1, grad=True),
        # a training batch: rows out, and the gradient of the rows back to the tokens
        dict(name="sort training", op="sort", T=4096, E=256, k=8, H=7168, dtype="bfloat16",
             pad=0.05, grad=True),
        # the experts' rows of a decode batch back to its tokens
        dict(name="combine decode", op="combine", T=64, E=256, k=8, H=7168, dtype="bfloat16",
             pad=0.0, grad=False),
        # 32-bit rows, as a master-precision run or a check of one has them
        dict(name="combine float32", op="combine", T=4099, E=60, k=6, H=2048, dtype="float32",
             pad=0.0, grad=True),
        # the largest: a training batch of 131072 rows, forward and both gradients
        dict(name="combine training", op="combine", T=16384, E=128, k=8, H=4096,
             dtype="bfloat16", pad=0.05, grad=True),
        # a decode batch between two blocks: post-norm, per-token gate, residual, pre-norm
        dict(name="norm decode", op="norm", T=32, H=7168, dtype="bfloat16",
             weights="bfloat16", y=True, post=True, pre=True, gate="token", sigmoid=True,
             scale=1.0, offset=0.0, grad=False),
        # the same between two blocks of a long prefill, weights kept around one
        dict(name="norm prefill", op="norm", T=16381, H=4096, dtype="bfloat16",
             weights="bfloat16", y=True, post=True, pre=True, gate="none", sigmoid=False,
             scale=0.22, offset=1.0, grad=False),
        # a training step: gradients of the stream, the block's output, a per-channel gate
        # and both 32-bit weights
        dict(name="norm training", op="norm", T=4095, H=7168, dtype="bfloat16",
             weights="float32", y=True, post=True, pre=True, gate="channel", sigmoid=False,
             scale=0.5, offset=0.0, grad=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["router", "sort", "combine", "norm"])
    T = _log_uniform(rng, 1, 16384)
    dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
    size = 4 if dtype == "float32" else 2
    if op == "router":
        E = rng.choice([8, 16, 60, 64, 128, 160, 256, 384, 512])
        k = rng.randint(1, min(E, 10))
        score = rng.choice(["softmax", "sigmoid"])
        groups, topk_groups, group_top = 1, 1, 1
        if E % 8 == 0 and E >= 64 and rng.random() < 0.5:
            groups = rng.choice([4, 8])
            topk_groups = rng.randint(2, groups)
            group_top = rng.choice([1, 2])
        k = min(k, topk_groups * (E // groups))
        return dict(op=op, T=T, E=E, k=k, dtype=dtype, score=score,
                    bias=rng.random() < 0.5, groups=groups, topk_groups=topk_groups,
                    group_top=group_top, renormalize=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5]), masked=rng.choice([0, 0, E // 8]),
                    pad=rng.choice([0.0, 0.1]), grad=rng.random() < 0.5)
    H = _log_uniform(rng, 64, 8192)
    if rng.random() < 0.7:
        H = (H + 7) // 8 * 8
    if op == "norm":
        c = dict(op=op, T=min(T, 4095 * 7168 // H), H=H, dtype=dtype,
                 weights=rng.choice([dtype, "float32"]), y=rng.random() < 0.8,
                 post=rng.random() < 0.6, pre=True,
                 gate=rng.choice(["none", "token", "channel", "full"]),
                 sigmoid=rng.random() < 0.5, scale=rng.choice([1.0, 0.22]),
                 offset=rng.choice([0.0, 1.0]), grad=rng.random() < 0.5)
        # a token's gate gradient is one sum that may cancel: not of a single token
        if c["grad"] and c["gate"] == "token":
            c["T"] = max(c["T"], 8)
        return c
    E = rng.choice([4, 8, 60, 64, 128, 256, 512])
    k = rng.randint(1, min(E, 9))
    T = max(1, min(T, 16384 * 4096 * 9 * 2 // (H * (k + 1) * size)))
    grad = rng.random() < 0.6
    if grad and op == "combine":    # likewise the weights' gradients
        T = max(T, 8)
    return dict(op=op, T=T, E=E, k=k, H=H, dtype=dtype, pad=rng.choice([0.0, 0.05]), grad=grad)


def _pads(c):
    return int(c["pad"] * c["T"])


def work(c):
    size = 4 if c["dtype"] == "float32" else 2
    T = c["T"]
    if c["op"] == "router":
        logits = T * c["E"] * size
        byts = logits + T * c["k"] * 8 + (4 * c["E"] if c["bias"] else 0) + (T if c["pad"] else 0)
        flops = 8 * T * c["E"]
        if c["grad"]:
            byts += logits + T * c["k"] * 4
            flops += 6 * T * (c["k"] if c["renormalize"] else c["E"])
        return {"bytes": byts, "flops": flops}
    H = c["H"]
    if c["op"] == "norm":
        w = 4 if c["weights"] == "float32" else 2
        gates = {"none": 0, "token": T, "channel": H, "full": T * H}[c["gate"]] if c["y"] else 0
        vecs = (1 + (c["y"] and c["post"])) * H * w + gates * size
        if not c["grad"]:
            streams = 4 if c["y"] else 2
            return {"bytes": streams * T * H * size + vecs, "flops": 12 * T * H}
        streams = 6 if c["y"] else 3
        grads = (1 + (c["y"] and c["post"])) * H * 4 + (
            H * 4 if c["gate"] == "channel" and c["y"] else
            T * 4 if c["gate"] == "token" and c["y"] else gates * size)
        return {"bytes": streams * T * H * size + vecs + grads, "flops": 30 * T * H}
    rows = (T - _pads(c)) * c["k"]
    move = (rows + T) * H * size
    slots = T * c["k"] * 4
    if c["op"] == "sort":
        byts = move + 2 * slots + rows * 4 + (c["E"] + 1) * 4
        return {"bytes": byts * (2 if c["grad"] else 1), "flops": rows * H * c["grad"] + slots}
    byts, flops = move + 2 * slots, 2 * rows * H
    if c["grad"]:   # the rows are read once for both directions
        byts += T * H * size + rows * H * size + slots
        flops += 3 * rows * H
    return {"bytes": byts, "flops": flops}


def _routing(c, g):
    """Top-k ids over experts of uneven popularity, and the padding tokens."""
    T, E, k = c["T"], c["E"], c["k"]
    like = torch.randn(E, generator=g, device=_DEV)
    ids = (torch.randn((T, E), generator=g, device=_DEV) + like).topk(k, dim=1).indices
    pad = None
    if c["pad"]:
        pad = torch.zeros(T, dtype=torch.uint8, device=_DEV)
        pad[torch.randperm(T, generator=g, device=_DEV)[:_pads(c)]] = 1
    return ids.to(torch.int32).contiguous(), pad


def _normal(g, dtype, *shape, std=1.0, mean=0.0):
    t = torch.empty(shape, dtype=torch.float32, device=_DEV)
    return t.normal_(mean, std, generator=g).to(dtype)


def prepare(c, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    dt, T = getattr(torch, c["dtype"]), c["T"]
    s = {"c": c}
    if c["op"] == "router":
        E, k = c["E"], c["k"]
        x = _normal(g, torch.float32, T, E, std=1.3) + _normal(g, torch.float32, E, std=0.5)
        s["logits"] = x.to(dt)
        if c["masked"]:
            out = torch.randperm(E, generator=g, device=_DEV)[:c["masked"]]
            s["logits"][:, out] = -math.inf
        s["bias"] = _normal(g, torch.float32, E, std=0.05) if c["bias"] else None
        s["pad"] = _routing(dict(c, k=1), g)[1]
        s["grad_weights"] = _normal(g, torch.float32, T, k) if c["grad"] else None
        s["out"] = {"topk_ids": torch.empty((T, k), dtype=torch.int32, device=_DEV),
                    "topk_weights": torch.empty((T, k), dtype=torch.float32, device=_DEV)}
        if c["grad"]:
            s["out"]["grad_logits"] = torch.empty_like(s["logits"])
    elif c["op"] == "norm":
        H, wt = c["H"], getattr(torch, c["weights"])
        std = 0.1
        s["residual"] = _normal(g, dt, T, H, std=3.0)
        s["y"] = _normal(g, dt, T, H, std=0.7) if c["y"] else None
        s["pre_weight"] = _normal(g, wt, H, std=std, mean=1.0 - c["offset"])
        s["post_weight"] = (_normal(g, wt, H, std=std, mean=1.0 - c["offset"])
                            if c["y"] and c["post"] else None)
        shape = {"none": None, "token": (T,), "channel": (H,), "full": (T, H)}[c["gate"]]
        s["gate"] = _normal(g, dt, *shape) if shape and c["y"] else None
        if c["grad"]:
            s["grad_normed"] = _normal(g, dt, T, H)
            s["grad_residual_out"] = _normal(g, dt, T, H) if c["y"] else None
            s["out"] = {"grad_residual": torch.empty_like(s["residual"]),
                        "grad_pre_weight": torch.empty(H, dtype=torch.float32, device=_DEV)}
            if c["y"]:
                s["out"]["grad_y"] = torch.empty_like(s["residual"])
            if s["post_weight"] is not None:
                s["out"]["grad_post_weight"] = torch.empty(H, dtype=torch.float32, device=_DEV)
            if s["gate"] is not None:
                s["out"]["grad_gate"] = torch.empty(
                    shape, dtype=dt if c["gate"] == "full" else torch.float32, device=_DEV)
        else:
            s["out"] = {"normed": torch.empty_like(s["residual"])}
            if c["y"]:
                s["out"]["residual_out"] = torch.empty_like(s["residual"])
    else:
        E, k, H = c["E"], c["k"], c["H"]
        s["ids"], s["pad"] = _routing(c, g)
        n = T * k
        if c["op"] == "sort":
            s["x"] = _normal(g, dt, T, H)
            # rows behind the routed ones stay as they are: zeros and -1 here
            s["out"] = {"rows": torch.zeros((n, H), dtype=dt, device=_DEV),
                        "expert_offsets": torch.empty(E + 1, dtype=torch.int32, device=_DEV),
                        "slot_row": torch.empty((T, k), dtype=torch.int32, device=_DEV),
                        "row_slot": torch.full((n,), -1, dtype=torch.int32, device=_DEV)}
            if c["grad"]:
                s["grad_rows"] = _normal(g, dt, n, H)
                s["out"]["grad_x"] = torch.empty_like(s["x"])
        else:
            s["slot_row"] = _sorted_slots(s["ids"], s["pad"], E)[0]
            s["rows"] = _normal(g, dt, n, H)
            s["weights"] = torch.softmax(_normal(g, torch.float32, T, k), dim=1)
            s["out"] = {"out": torch.empty((T, H), dtype=dt, device=_DEV)}
            if c["grad"]:
                s["grad_out"] = _normal(g, dt, T, H)
                s["out"]["grad_rows"] = torch.zeros_like(s["rows"])
                s["out"]["grad_weights"] = torch.empty((T, k), dtype=torch.float32,
                                                       device=_DEV)
    if own:
        s["plan"], s["ws"] = _plan(c)
    return s


def _plan(c):
    """The descriptor and the workspace a program keeps beside its buffers."""
    import fp8_block_quantized_group_amd as moe
    dt = getattr(torch, c["dtype"])
    if c["op"] == "router":
        return moe.Router(c["T"], c["E"], c["k"], score=c["score"], num_groups=c["groups"],
                          topk_groups=c["topk_groups"], group_top=c["group_top"],
                          renormalize=c["renormalize"], scale=c["scale"], dtype=dt), None
    if c["op"] == "norm":
        p = moe.BlockNorm(c["T"], c["H"], dtype=dt, weight_dtype=getattr(torch, c["weights"]),
                          post_norm=c["y"] and c["post"], gate=c["gate"] if c["y"] else "none",
                          gate_sigmoid=c["sigmoid"], eps=1e-6, residual_scale=c["scale"],
                          weight_offset=c["offset"])
        return p, moe.alloc_block_norm_workspace(p, _DEV) if c["grad"] else None
    p = moe.ExpertRows(c["T"], c["H"], c["E"], c["k"], dtype=dt)
    return p, moe.alloc_permute_workspace(p, _DEV) if c["op"] == "sort" else None


def run(s):
    if own:
        return _run_own(s)
    op = s["c"]["op"]
    if op == "router":
        return _plain_router(s)
    if op == "sort":
        return _plain_sort(s)
    if op == "combine":
        return _plain_combine(s)
    return _plain_norm_grad(s) if s["c"]["grad"] else _plain_norm(s)


def _run_own(s):
    import fp8_block_quantized_group_amd as moe
    c, p, out = s["c"], s["plan"], s["out"]
    if c["op"] == "router":
        moe.router_topk(p, s["logits"], out["topk_ids"], out["topk_weights"], bias=s["bias"],
                        is_padding=s["pad"])
        if c["grad"]:
            moe.router_topk_backward(p, s["logits"], out["topk_ids"], s["grad_weights"],
                                     out["grad_logits"])
    elif c["op"] == "sort":
        moe.permute(p, s["x"], s["ids"], out["rows"], out["expert_offsets"], out["slot_row"],
                    out["row_slot"], ws=s["ws"], is_padding=s["pad"])
        if c["grad"]:
            moe.permute_backward(p, s["grad_rows"], out["slot_row"], out["grad_x"])
    elif c["op"] == "combine":
        moe.unpermute(p, s["rows"], s["slot_row"], s["weights"], out["out"])
        if c["grad"]:
            moe.unpermute_backward(p, s["grad_out"], s["rows"], s["slot_row"], s["weights"],
                                   out["grad_rows"], out["grad_weights"])
    elif c["grad"]:
        moe.block_norm_backward(p, s["residual"], s["grad_normed"], out["grad_residual"],
                                y=s["y"], grad_residual_out=s["grad_residual_out"],
                                pre_weight=s["pre_weight"], post_weight=s["post_weight"],
                                gate=s["gate"], grad_y=out.get("grad_y"),
                                grad_pre_weight=out["grad_pre_weight"],
                                grad_post_weight=out.get("grad_post_weight"),
                                grad_gate=out.get("grad_gate"), ws=s["ws"])
    else:
        moe.block_norm(p, s["residual"], out["normed"], y=s["y"],
                       residual_out=out.get("residual_out"), pre_weight=s["pre_weight"],
                       post_weight=s["post_weight"], gate=s["gate"])
    return out


# ---- plain forms ------------------------------------------------------------

def _plain_router(s):
    c, x = s["c"], s["logits"].float()
    E, k, G = c["E"], c["k"], c["groups"]
    x = torch.where(x.isnan(), -math.inf, x).clamp_max(_FLT_MAX)
    live = x > -math.inf
    if s["pad"] is not None:
        live = live & (s["pad"] == 0)[:, None]
    x = torch.where(live, x, -math.inf)
    # 64 bits where two experts' keys may lie next to each other
    if s["bias"] is None and c["group_top"] == 1:
        key = x.double()
    else:
        xd = x.double()
        if c["score"] == "sigmoid":
            key = 1.0 / (1.0 + torch.exp(-xd))
        else:
            e = torch.exp(xd - xd.amax(1, keepdim=True).clamp_min(-1e300))
            key = e / e.sum(1, keepdim=True).clamp_min(1e-300)
        if s["bias"] is not None:
            key = key + s["bias"].double()
        key = torch.where(live, key, -math.inf)
    if G > 1:
        best = key.view(-1, G, E // G).sort(dim=2, descending=True).values[:, :, :c["group_top"]]
        rest = best[:, :, 1:]
        value = best[:, :, 0] + torch.where(rest > -math.inf, rest, 0.0).sum(2)
        order = value.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        kept = torch.zeros_like(value, dtype=torch.bool).scatter(1, order, True)
        key = torch.where(kept.repeat_interleave(E // G, dim=1), key, -math.inf)
    val, ids = key.sort(dim=1, descending=True, stable=True)
    val, ids = val[:, :k], ids[:, :k]
    chosen = val > -math.inf
    xs = torch.where(chosen, x.gather(1, ids), -math.inf)
    m = x.amax(1, keepdim=True).clamp_min(-_FLT_MAX)
    p = torch.exp(x - m)
    total = p.sum(1, keepdim=True).clamp_min(1e-30)
    if c["score"] == "sigmoid":
        sc = 1.0 / (1.0 + torch.exp(-xs))
        denom = sc.sum(1, keepdim=True) + 1e-20
    else:
        ms = xs.amax(1, keepdim=True).clamp_min(-_FLT_MAX)
        sc = torch.exp(xs - ms)
        denom = sc.sum(1, keepdim=True).clamp_min(1e-30)
        if not c["renormalize"]:
            sc = torch.exp(xs - m) / total
    w = sc / denom if c["renormalize"] else sc
    out = {"topk_ids": torch.where(chosen, ids, -1).to(torch.int32),
           "topk_weights": w * c["scale"]}
    if c["grad"]:
        gw = torch.where(chosen, s["grad_weights"], 0.0)
        a = gw - (gw * w).sum(1, keepdim=True) if c["renormalize"] or c["score"] == "softmax" \
            else gw
        if c["score"] == "sigmoid":
            d = a * sc * (1.0 - sc) / (denom if c["renormalize"] else 1.0)
            dx = torch.zeros_like(x)
        elif c["renormalize"]:
            d = a * w
            dx = torch.zeros_like(x)
        else:
            d = a * w
            dx = -(gw * w).sum(1, keepdim=True) * p / total
        # a place without an expert keeps what the dense part has there
        dx = dx.scatter(1, ids, torch.where(chosen, d, dx.gather(1, ids))) * c["scale"]
        out["grad_logits"] = dx.to(s["logits"].dtype)
    return out


def _sorted_slots(ids, pad, E):
    """slot_row [T, k], row_slot [T*k] (-1 behind the routed rows), offsets [E+1]."""
    T, k = ids.shape
    e = ids.long()
    routed = (e >= 0) & (e < E)
    if pad is not None:
        routed = routed & (pad == 0)[:, None]
    e = torch.where(routed, e, E).view(-1)
    order = torch.sort(e, stable=True).indices
    slot_row = torch.empty_like(order)
    slot_row[order] = torch.arange(T * k, device=ids.device)
    counts = (e[:, None] == torch.arange(E, device=ids.device)).sum(0)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = counts.cumsum(0)
    behind = e[order] == E
    return (torch.where(routed.view(-1), slot_row, -1).view(T, k).to(torch.int32),
            torch.where(behind, -1, order).to(torch.int32), offsets)


def _plain_sort(s):
    c = s["c"]
    slot_row, row_slot, offsets = _sorted_slots(s["ids"], s["pad"], c["E"])
    src = row_slot.long()
    rows = s["x"][src.clamp_min(0) // c["k"]]
    rows = torch.where((src >= 0)[:, None], rows, 0)
    out = {"rows": rows, "expert_offsets": offsets, "slot_row": slot_row, "row_slot": row_slot}
    if c["grad"]:
        at = slot_row.long()
        g = s["grad_rows"][at.clamp_min(0)].float() * (at >= 0)[:, :, None]
        out["grad_x"] = g.sum(1).to(s["x"].dtype)
    return out


def _plain_combine(s):
    c, at = s["c"], s["slot_row"].long()
    routed = at >= 0
    y = s["rows"][at.clamp_min(0)].float()
    w = torch.where(routed, s["weights"], 0.0)
    out = {"out": (y * w[:, :, None]).sum(1).to(s["rows"].dtype)}
    if c["grad"]:
        g = s["grad_out"].float()
        out["grad_weights"] = torch.where(routed, (y * g[:, None, :]).sum(2), 0.0)
        gr = (g[:, None, :] * w[:, :, None]).to(s["rows"].dtype)
        n = at.numel()      # slots without a row write to one behind the last
        grad_rows = s["rows"].new_zeros((n + 1, c["H"]))
        grad_rows[torch.where(routed, at, n)] = gr
        out["grad_rows"] = grad_rows[:n]
    return out


def _gate(s, dtype):
    """The gate's value as it enters the product, broadcast to [T, H]."""
    if s["gate"] is None:
        return None
    g = s["gate"].to(dtype)
    if s["c"]["sigmoid"]:
        g = 1.0 / (1.0 + torch.exp(-g))
    return g[:, None] if s["c"]["gate"] == "token" else g


def _plain_norm(s):
    c, r = s["c"], s["residual"].float()
    out = {}
    if s["y"] is not None:
        n = s["y"].float()
        if s["post_weight"] is not None:
            n = n * torch.rsqrt((n * n).mean(1, keepdim=True) + 1e-6)
            n = n * (s["post_weight"].float() + c["offset"])
        g = _gate(s, torch.float32)
        r = r + c["scale"] * (n if g is None else n * g)
        out["residual_out"] = r.to(s["residual"].dtype)
    h = r * torch.rsqrt((r * r).mean(1, keepdim=True) + 1e-6)
    out["normed"] = (h * (s["pre_weight"].float() + c["offset"])).to(s["residual"].dtype)
    return out


def _plain_norm_grad(s):
    """The gradients at the stored residual stream (what the forward pass wrote)."""
    c, r, dh = s["c"], s["residual"].float(), s["grad_normed"].float()
    dt = s["residual"].dtype
    rs = torch.rsqrt((r * r).mean(1, keepdim=True) + 1e-6)
    xh = r * rs
    dxh = dh * (s["pre_weight"].float() + c["offset"])
    d = rs * (dxh - xh * (dxh * xh).mean(1, keepdim=True))
    out = {"grad_pre_weight": (dh * xh).sum(0)}
    if s["y"] is None:
        out["grad_residual"] = d.to(dt)
        return out
    d = d + s["grad_residual_out"].float()
    out["grad_residual"] = d.to(dt)
    y = s["y"].float()
    n = y
    if s["post_weight"] is not None:
        ys = torch.rsqrt((y * y).mean(1, keepdim=True) + 1e-6)
        yh = y * ys
        wp = s["post_weight"].float() + c["offset"]
        n = yh * wp
    g = _gate(s, torch.float32)
    dn = c["scale"] * (d if g is None else d * g)
    if g is not None:
        dg = c["scale"] * d * n
        if c["sigmoid"]:
            dg = dg * g * (1.0 - g)
        out["grad_gate"] = dg.sum(1) if c["gate"] == "token" else \
            dg.sum(0) if c["gate"] == "channel" else dg.to(dt)
    if s["post_weight"] is not None:
        out["grad_post_weight"] = (dn * yh).sum(0)
        dyh = dn * wp
        dn = ys * (dyh - yh * (dyh * yh).mean(1, keepdim=True))
    out["grad_y"] = dn.to(dt)
    return out


# ---- the definitions in 64 bits ---------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "router":
        return _exact_router(s)
    if c["op"] == "sort":
        return _exact_sort(s)
    if c["op"] == "combine":
        return _exact_combine(s)
    return _exact_norm_grad(s) if c["grad"] else _exact_norm(s)


def _take_best(key, count):
    """The `count` largest of each row, one after the other, each time the lowest
    index among the largest; -1 where nothing but -inf is left."""
    key, n = key.clone(), key.shape[1]
    at = torch.arange(n, device=key.device)
    found = []
    for _ in range(count):
        top = key.amax(1, keepdim=True)
        first = torch.where(key == top, at, n).amin(1)
        found.append(torch.where(top[:, 0] > -math.inf, first, -1))
        key.scatter_(1, first[:, None], -math.inf)
    return torch.stack(found, 1)


def _exact_router(s):
    c = s["c"]
    x = s["logits"].double()
    x = torch.nan_to_num(x, nan=-math.inf, posinf=_FLT_MAX, neginf=-math.inf)
    if s["pad"] is not None:
        x[s["pad"] != 0] = -math.inf
    live = x > -math.inf
    if c["score"] == "sigmoid":
        score = torch.sigmoid(x)
    else:
        score = torch.softmax(x, 1).nan_to_num(0.0)
    key = x
    if c["bias"] or c["group_top"] > 1:
        key = score + (s["bias"].double() if c["bias"] else 0.0)
        key = key.masked_fill(~live, -math.inf)
    if c["groups"] > 1:
        size = c["E"] // c["groups"]
        value = []
        for j in range(c["groups"]):
            part = key[:, j * size:(j + 1) * size].topk(min(size, c["group_top"]), dim=1).values
            none = part[:, 0] == -math.inf
            value.append(part.masked_fill(part == -math.inf, 0.0).sum(1)
                         .masked_fill(none, -math.inf))
        best = _take_best(torch.stack(value, 1), c["topk_groups"])
        of = torch.arange(c["E"], device=x.device) // size
        key = key.masked_fill(~(best[:, :, None] == of).any(1), -math.inf)
    ids = _take_best(key, c["k"])
    chosen = ids >= 0
    at = ids.clamp_min(0)
    sc = score.gather(1, at) * chosen
    if not c["renormalize"]:
        w = sc
    elif c["score"] == "sigmoid":
        w = sc / (sc.sum(1, keepdim=True) + 1e-20)
    else:
        w = torch.softmax(x.gather(1, at).masked_fill(~chosen, -math.inf), 1).nan_to_num(0.0)
    out = {"topk_ids": ids.to(torch.int32), "topk_weights": w * c["scale"]}
    if c["grad"]:
        g = s["grad_weights"].double() * chosen * c["scale"]
        one = torch.zeros_like(x).scatter_add(1, at, g)     # dL/dw spread over the experts
        wd = torch.zeros_like(x).scatter_add(1, at, w)
        mine = torch.zeros_like(x).scatter_add(1, at, chosen.double())
        if c["score"] == "softmax":
            pr = wd if c["renormalize"] else score
            dx = pr * (one - (one * wd).sum(1, keepdim=True))
        else:
            ds = one
            if c["renormalize"]:
                total = (sc.sum(1, keepdim=True) + 1e-20)
                ds = mine * (one - (one * wd).sum(1, keepdim=True)) / total
            dx = ds * score * (1.0 - score)
        out["grad_logits"] = dx.masked_fill(~live, 0.0)
    return out


def _exact_sort(s):
    c, ids = s["c"], s["ids"].long()
    E, k, n = c["E"], c["k"], ids.numel()
    if s["pad"] is not None:
        ids = ids.masked_fill((s["pad"] != 0)[:, None], -1)
    flat = ids.reshape(-1)
    hot = flat[None, :] == torch.arange(E, device=flat.device)[:, None]     # [E, slots]
    count = hot.sum(1)
    first = torch.cat([count.new_zeros(1), count.cumsum(0)])
    rank = hot.cumsum(1, dtype=torch.int32).sub_(1)
    row = (torch.where(hot, rank, 0).sum(0) + first[flat.clamp_min(0)])
    row = torch.where(flat >= 0, row, -1)
    row_slot = torch.full((n,), -1, dtype=torch.int64, device=flat.device)
    routed = (flat >= 0).nonzero()[:, 0]
    row_slot[row[routed]] = routed
    rows = torch.zeros((n, c["H"]), dtype=torch.float64, device=flat.device)
    rows[row[routed]] = s["x"].double()[routed // k]
    out = {"rows": rows, "expert_offsets": first.to(torch.int32),
           "slot_row": row.view(-1, k).to(torch.int32), "row_slot": row_slot.to(torch.int32)}
    if c["grad"]:
        dx = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device=flat.device)
        for j in range(k):
            r = row.view(-1, k)[:, j]
            t = (r >= 0).nonzero()[:, 0]
            dx[t] += s["grad_rows"][r[t]].double()
        out["grad_x"] = dx
    return out


def _exact_combine(s):
    c, at, w = s["c"], s["slot_row"].long(), s["weights"].double()
    dev = at.device
    total = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device=dev)
    out = {"out": total}
    if c["grad"]:
        out["grad_rows"] = torch.zeros((at.numel(), c["H"]), dtype=torch.float64, device=dev)
        out["grad_weights"] = torch.zeros_like(w)
    for j in range(c["k"]):
        t = (at[:, j] >= 0).nonzero()[:, 0]
        r = at[t, j]
        y = s["rows"][r].double()
        total[t] += w[t, j, None] * y
        if c["grad"]:
            g = s["grad_out"][t].double()
            out["grad_rows"][r] = w[t, j, None] * g
            out["grad_weights"][t, j] = torch.linalg.vecdot(g, y)
    return out


def _exact_norm(s):
    c, r = s["c"], s["residual"].double()
    out = {}
    if s["y"] is not None:
        n = s["y"].double()
        if s["post_weight"] is not None:
            n = n / (n.square().mean(1, keepdim=True) + 1e-6).sqrt()
            n = n * (c["offset"] + s["post_weight"].double())
        if s["gate"] is not None:
            g = s["gate"].double()
            g = torch.sigmoid(g) if c["sigmoid"] else g
            n = n * (g.unsqueeze(1) if c["gate"] == "token" else g)
        r = r + c["scale"] * n
        out["residual_out"] = r
    h = r / (r.square().mean(1, keepdim=True) + 1e-6).sqrt()
    out["normed"] = h * (c["offset"] + s["pre_weight"].double())
    return out


def _exact_norm_grad(s):
    """By torch's own differentiation of the definition in 64 bits; the stored
    stream r' is a leaf, and what follows from it (r' = r + scale gate n) hands
    its gradient on to the gate, the block's output and its weight."""
    c = s["c"]
    r = s["residual"].double().requires_grad_()
    pre = s["pre_weight"].double().requires_grad_()
    h = r / (r.square().mean(1, keepdim=True) + 1e-6).sqrt() * (c["offset"] + pre)
    into_r, into_pre = torch.autograd.grad(h, (r, pre), s["grad_normed"].double())
    out = {"grad_pre_weight": into_pre}
    if s["y"] is None:
        out["grad_residual"] = into_r
        return out
    into_r = into_r + s["grad_residual_out"].double()
    out["grad_residual"] = into_r
    names, leaves = ["grad_y"], [s["y"].double().requires_grad_()]
    n = leaves[0]
    if s["post_weight"] is not None:
        wp = s["post_weight"].double().requires_grad_()
        names, leaves = names + ["grad_post_weight"], leaves + [wp]
        n = n / (n.square().mean(1, keepdim=True) + 1e-6).sqrt() * (c["offset"] + wp)
    if s["gate"] is not None:
        gate = s["gate"].double().requires_grad_()
        names, leaves = names + ["grad_gate"], leaves + [gate]
        g = torch.sigmoid(gate) if c["sigmoid"] else gate
        n = n * (g.unsqueeze(1) if c["gate"] == "token" else g)
    out.update(zip(names, torch.autograd.grad(c["scale"] * n, leaves, into_r)))
    return out

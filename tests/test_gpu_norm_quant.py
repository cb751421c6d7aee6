"""The norms around a block with the normed row in 8 bits, against the oracle:
bit for bit from fp32 rows (whose stored norm is what was quantized), within a
code's half step of the 64-bit norm from 16-bit ones; the layer on rows staged
this way; the block that uses both."""
import numpy as np
import pytest
import torch

import fp8_block_quantized_group_amd as moe
from expert_util import close, f64, marked, rand, untouched
from oracle import block_oracle as B
from oracle import moe_oracle as O

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
QUANTS = ["ue8m0", "fp32", "mxfp8"]
REL = 2.0 ** -16        # two norms of at most 2^-17 each, as tests/test_gpu_block.py derives


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    moe.load_library()


def make(seed, T, H, dtype, wdtype, gate="none", y=True, post=True, std=1.0):
    rng = np.random.default_rng(seed)
    t = {"residual": rand(rng, (T, H), dtype, std), "pre_weight": rand(rng, (H,), wdtype)}
    if y:
        t["y"] = rand(rng, (T, H), dtype)
        if post:
            t["post_weight"] = rand(rng, (H,), wdtype)
        shape = {"none": None, "token": (T,), "channel": (H,), "full": (T, H)}[gate]
        if shape:
            t["gate"] = rand(rng, shape, dtype)
    p = moe.BlockNorm(T, H, dtype=dtype, weight_dtype=wdtype, post_norm=y and post,
                      gate=gate if y else "none", gate_sigmoid=True, eps=1e-5,
                      residual_scale=0.37, weight_offset=float(seed & 1))
    return p, t


def run(p, t, quant, keep=True):
    d = {k: v.cuda() for k, v in t.items()}
    shape = (p.num_tokens, p.hidden)
    dt, sshape = moe.quant_shape(*shape, quant)
    o = {"x_q": marked(shape, torch.uint8), "x_sf": marked(sshape, dt)}
    if keep:
        o["normed"] = marked(shape, p.dtype)
    if "y" in t:
        o["residual_out"] = marked(shape, p.dtype)
    moe.block_norm_quant(p, quant=quant, **d, **o)
    return o


def plain(p, t):
    d = {k: v.cuda() for k, v in t.items()}
    o = {"normed": marked(t["residual"].shape, p.dtype)}
    if "y" in t:
        o["residual_out"] = marked(t["residual"].shape, p.dtype)
    moe.block_norm(p, **d, **o)
    return o


def check(p, t, quant, keep=True):
    o, want = run(p, t, quant, keep), plain(p, t)
    n = lambda k: None if t.get(k) is None else f64(t[k])              # noqa: E731
    exact = B.block_norm(f64(t["residual"]), y=n("y"), post_norm=p.post_norm,
                         w_post=n("post_weight"), gate=n("gate"), kind=p.gate, sigmoid=True,
                         w_pre=n("pre_weight"), eps=float(np.float32(p.eps)),
                         scale=float(np.float32(p.residual_scale)), offset=p.weight_offset)
    for k in want:
        if k in o:
            close(o[k], exact[k][0], REL * exact[k][1], k)
            # block_norm's bits, but for fp16: a product that only goes to fp16 is
            # rounded once (v_fma_mixlo_f16), one that the codes take too is
            # rounded to fp32 first, and 2^-24 beside a tie decides the other way
            assert p.dtype == torch.float16 or torch.equal(o[k], want[k]), k
    T, H = p.num_tokens, p.hidden
    group = 32 if quant == "mxfp8" else 128
    G = H // group
    codes, sf = o["x_q"].cpu().numpy(), o["x_sf"].cpu().numpy()
    if p.dtype == torch.float32:
        cw, sw = O.quantize_groups(want["normed"].cpu().numpy(), quant != "fp32", group)
        assert np.array_equal(codes, cw)
        if quant == "ue8m0":
            sw = O.pack_ue8m0_rows(sw)
        assert np.array_equal(sf, sw)
        return o
    v, mag = exact["normed"]
    err = REL * mag
    if quant == "ue8m0":
        assert not sf[:, G:].any()          # pad bytes
        sf = sf[:, :G]
    v, err = v.reshape(T, G, group), err.reshape(T, G, group)
    floor = float(np.float32(1e-4))
    lo = np.maximum((np.abs(v) - err).max(2), floor) / 448 * (1 - 2.0 ** -23)
    hi = np.maximum((np.abs(v) + err).max(2), floor) / 448 * (1 + 2.0 ** -23)
    if quant == "fp32":
        s = sf.astype(np.float64)
        assert ((s >= lo) & (s <= hi)).all()
    else:
        s = 2.0 ** (sf.astype(np.float64) - 127)
        assert ((s >= lo) & (s / 2 < hi)).all()
    s = s[:, :, None]
    got = O.e4m3_decode(codes).reshape(v.shape) * s
    # half a code's step (2^-4 of the value, 2^-10 below the normal codes), two
    # roundings of the quotient, and 448 for what lies at most err above
    tol = np.maximum(np.abs(v) * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -20) + 2 * err
    assert (np.abs(got - v) <= tol).all()
    return o


WIDTHS = [128, 256, 384, 512, 640, 1024, 1536, 2048, 4096, 5120, 7168, 8192, 12288, 32768]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("H", WIDTHS)
def test_widths(H, dtype):
    for i, (quant, gate) in enumerate(zip(QUANTS * 2, ("none", "token", "channel", "full",
                                                       "none", "token"))):
        p, t = make(H + i, (1, 3, 6, 13)[(i + H // 128) % 4], H, dtype,
                    (dtype, torch.float32)[i & 1], gate, y=i != 4, post=i != 1)
        check(p, t, quant, keep=i % 2 == 0)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("quant", QUANTS)
@pytest.mark.parametrize("T,H", [(700, 128), (515, 384), (520, 1408), (600, 2048), (530, 2688),
                                 (514, 3584), (513, 5120), (515, 6144), (514, 7168),
                                 (513, 12288), (513, 16384)])
def test_many_rows(T, H, quant, dtype):
    p, t = make(T + H, T, H, dtype, torch.float32, "token")
    check(p, t, quant)


@pytest.mark.parametrize("quant", QUANTS)
def test_floor_infinities_and_nan(quant):
    """Groups of zeros and of values below the quantizer's floor; a row with an
    infinity or a NaN leaves the others alone."""
    p, t = make(3, 9, 512, torch.float32, torch.float32, y=False)
    t["pre_weight"][:160] = 0
    t["pre_weight"][160:256] = 1e-8
    clean = check(p, t, quant)
    t["residual"][4, 7] = float("nan")
    t["residual"][6, 300] = float("inf")
    o = run(p, t, quant)
    rest = [r for r in range(9) if r not in (4, 6)]
    for k in ("x_q", "x_sf"):
        assert torch.equal(o[k][rest], clean[k][rest])


def test_no_tokens_and_host_rows():
    p = moe.BlockNorm(0, 256)
    e = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    moe.block_norm_quant(p, e, **moe.alloc_quant_outputs(p))
    p, t = make(1, 2, 256, torch.bfloat16, torch.bfloat16, y=False)
    o = moe.alloc_quant_outputs(p, "fp32")
    with pytest.raises(ValueError, match="x_sf"):
        moe.block_norm_quant(p, t["residual"].cuda(), **o)
    with pytest.raises(ValueError, match="quant"):
        moe.block_norm_quant(p, t["residual"].cuda(), **o, quant="bf16")


def test_in_place_and_replayed():
    p, t = make(5, 40, 768, torch.bfloat16, torch.float32, "channel")
    d = {k: v.cuda() for k, v in t.items()}
    o = moe.alloc_quant_outputs(p)
    x = d.pop("residual")
    start = x.clone()

    def call():
        moe.block_norm_quant(p, x, residual_out=x, **d, **o)

    want = run(p, t, "ue8m0")
    call()
    assert torch.equal(x, want["residual_out"])
    assert torch.equal(o["x_q"], want["x_q"]) and torch.equal(o["x_sf"], want["x_sf"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    for _ in range(3):
        x.copy_(start)
        for v in o.values():
            v.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want["residual_out"])
        assert torch.equal(o["x_q"], want["x_q"]) and torch.equal(o["x_sf"], want["x_sf"])


# ---- the layer on staged rows ------------------------------------------------------

def layer_of(act_quant, weight_quant, layout="contiguous", T=40, **kw):
    import moe_synth
    cfg = moe_synth.custom(name="staged", T=T, E=8, top_k=2, K=256, N=256, seed=91,
                           act_quant=act_quant, weight_quant=weight_quant, layout=layout, **kw)
    inp = moe_synth.make_inputs(cfg, "cuda")
    p = moe.Problem.from_config(cfg)
    return p, moe.MoeLayer(p, inp["w13"], inp["w13_sf"], inp["w2"], inp["w2_sf"]), inp


PAIRS = [("ue8m0", "fp8_block128"), ("fp32", "fp8_block128"), ("mxfp8", "mxfp8"),
         ("mxfp8", "mxfp4")]


@pytest.mark.parametrize("layout", ["contiguous", "indexed"])
@pytest.mark.parametrize("act,weight", PAIRS)
def test_layer_on_staged_rows(act, weight, layout):
    """moe_stage's own rows give moe_forward's bits, and are left as they were;
    the routing alone is the stage's."""
    p, layer, inp = layer_of(act, weight, layout)
    want = layer(inp["hidden"], inp["topk_ids"], inp["topk_weights"])
    bufs, only = moe.alloc_stage_outputs(p), moe.alloc_stage_outputs(p)
    moe.stage(p, inp["hidden"], inp["topk_ids"], inp["topk_weights"], bufs)
    x_q, x_sf = bufs["x_q"].clone(), bufs["x_sf"].clone()
    out = layer.quantized(bufs["x_q"], bufs["x_sf"], inp["topk_ids"], inp["topk_weights"])
    assert torch.equal(out, want)
    assert torch.equal(x_q, bufs["x_q"]) and torch.equal(x_sf, bufs["x_sf"])
    for k in ("x_q", "x_sf"):
        only[k].view(torch.uint8).fill_(0x5A)
    moe.stage_routing(p, inp["topk_ids"], inp["topk_weights"], only)
    for k in ("topk_idx", "topk_w", "expert_num_tokens", "expert_offsets", "slot_row"):
        assert torch.equal(only[k], bufs[k]), k
    n = int(bufs["expert_offsets"][-1])
    assert torch.equal(only["row_src"][:n], bufs["row_src"][:n])
    assert untouched(only["x_q"]) and untouched(only["x_sf"])
    # the tile list too: the GEMM step by step
    a = moe.alloc_act_outputs(p)
    b = moe.alloc_act_outputs(p)
    for r, o in ((bufs, a), (only, b)):
        moe.grouped_gemm_w13_act(p, x_q, x_sf, r, layer.w13, layer.w13_sf, *o)
    assert all(torch.equal(u[:n], v[:n]) for u, v in zip(a, b))


def make_block(act, weight, staged, T=40):
    p, layer, inp = layer_of(act, weight, T=T)
    rng = np.random.default_rng(17)
    norm = moe.BlockNorm(T, 256, weight_dtype=torch.float32, post_norm=True, gate="token",
                         gate_sigmoid=True, residual_scale=0.4)
    w = {n: rand(rng, (256,), torch.float32).cuda() for n in ("pre", "post", "next")}
    block = moe.MoeBlock(layer, moe.Router(T, 8, 2, score="sigmoid", scale=2.0),
                         rand(rng, (8, 256), torch.float32, 0.1).cuda(), norm, w["pre"],
                         w["post"], staged=staged)
    x = rand(rng, (T, 256), torch.bfloat16, 2.0).cuda()
    return block, w, x, rand(rng, (T,), torch.bfloat16).cuda()


@pytest.mark.parametrize("act,weight", PAIRS)
def test_block_with_a_staging_norm(act, weight):
    block, w, x, g = make_block(act, weight, True)
    out = block(x, gate=g)
    q = moe.alloc_quant_outputs(block.norm, act)
    h = torch.empty_like(x)
    moe.block_norm_quant(block.pre, x, **q, quant=act, normed=h, pre_weight=w["pre"])
    assert torch.equal(h, block.hidden)
    logits = torch.matmul(h.float(), block.router_weight.t())
    ids, wt = torch.empty_like(block.topk_ids), torch.empty_like(block.topk_weights)
    moe.router_topk(block.router, logits, ids, wt)
    y = block.layer.quantized(q["x_q"], q["x_sf"], ids, wt)
    want, nxt, nq = torch.empty_like(x), torch.empty_like(x), moe.alloc_quant_outputs(
        block.norm, act)
    moe.block_norm_quant(block.norm, x, **nq, quant=act, normed=nxt, y=y, residual_out=want,
                         pre_weight=w["next"], post_weight=w["post"], gate=g)
    assert torch.equal(out, want)
    # the next block's input leaves this one staged, and is taken as given
    n2, q2 = torch.empty_like(x), moe.alloc_quant_outputs(block.norm, act)
    assert torch.equal(block(x, gate=g, next_normed=n2, next_weight=w["next"], next_staged=q2),
                       out)
    assert torch.equal(n2, nxt) and all(torch.equal(q2[k], nq[k]) for k in nq)
    assert torch.equal(block(x, normed=h, staged=q, gate=g), out)
    # near the block that stages the 16-bit rows: codes a step apart at most,
    # 2^-3 of a few of them, where each layer output sums 256 products
    plain = make_block(act, weight, False)[0]
    ref = plain(x, gate=g).float()
    assert float((out.float() - ref).norm()) <= 2.0 ** -5 * float(ref.norm())


def test_block_refuses_staged_rows_it_cannot_use():
    block, w, x, g = make_block("ue8m0", "fp8_block128", False)
    q = moe.alloc_quant_outputs(block.norm)
    with pytest.raises(ValueError, match="normed"):
        block(x, gate=g, staged=q)
    with pytest.raises(ValueError, match="x_sf"):
        block(x, gate=g, normed=x, staged=moe.alloc_quant_outputs(block.norm, "fp32"))
    p, layer, inp = layer_of("bf16", "fp8_block128")
    with pytest.raises(ValueError, match="bf16"):
        moe.MoeBlock(layer, block.router, block.router_weight, block.norm, staged=True)


@pytest.mark.parametrize("act,weight", PAIRS)
def test_layer_on_staged_slabs(act, weight):
    """The batched layout: slabs of staged rows, counts from the dispatch."""
    p, layer, inp = layer_of(act, weight, "batched", T=250, max_tokens=160, pad_frac=0.0)
    n = inp["expert_num_tokens"]
    bufs = moe.alloc_stage_outputs(p)
    moe.stage(p, inp["hidden"], inp["topk_ids"], inp["topk_weights"], bufs, expert_num_tokens=n)
    want = layer(inp["hidden"], inp["topk_ids"], inp["topk_weights"], expert_num_tokens=n)
    out = layer.quantized(bufs["x_q"], bufs["x_sf"], inp["topk_ids"], inp["topk_weights"],
                          expert_num_tokens=n)
    assert torch.equal(out, want)


def test_layer_on_staged_rows_of_two_lists_with_padding():
    """More than 128 rows of an expert, a quarter of the tokens padding."""
    p, layer, inp = layer_of("ue8m0", "fp8_block128", T=2500)
    pad = (torch.arange(2500, device="cuda") % 4 == 1).to(torch.uint8)
    bufs = moe.alloc_stage_outputs(p)
    moe.stage(p, inp["hidden"], inp["topk_ids"], inp["topk_weights"], bufs, is_padding=pad)
    want = layer(inp["hidden"], inp["topk_ids"], inp["topk_weights"], is_padding=pad)
    out = layer.quantized(bufs["x_q"], bufs["x_sf"], inp["topk_ids"], inp["topk_weights"],
                          is_padding=pad)
    assert torch.equal(out, want)

"""The experts' own products on the GPU against the 64-bit oracle, whose
bounds (oracle/expert_oracle.py) are the tolerances, plus half a step of the
type that leaves; d is rounded by half a step of its type too."""
import threading

import numpy as np
import pytest
import torch

import fp8_block_quantized_group_amd as moe
from expert_util import close, f64, marked, rand, shifted, spread, untouched
from oracle import expert_oracle as X

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    moe.load_library()


def make(seed, R, E, K, N, dtype, act, offsets="spread", behind=0):
    """Host tensors; the rows from the last offset on are NaN."""
    rng = np.random.default_rng(seed)
    wide = N * (2 if act in X.GATED else 1)
    off = None
    if offsets == "spread":
        off = spread(rng, R - behind, E)
    elif offsets is not None:
        off = np.asarray(offsets)
    t = {"x": rand(rng, (R, K), dtype), "w": rand(rng, (E, wide, K), dtype, K ** -0.5),
         "gout": rand(rng, (R, N), dtype), "pre": rand(rng, (R, wide), dtype, 1.5), "off": off}
    last = R if off is None else int(off[-1])
    for k in ("x", "gout", "pre"):
        t[k][last:] = float("nan")
    return t, last


def device_offsets(t):
    return None if t["off"] is None else torch.from_numpy(t["off"]).to(torch.int32).cuda()


def problem(t, dtype, act, limit=0.0):
    R, K = t["x"].shape
    return moe.ExpertLinear(R, K, t["gout"].shape[1], t["w"].shape[0], dtype=dtype,
                            activation=act, act_limit=limit)


def check_forward(t, last, dtype, act, limit=0.0, put=lambda v: v.cuda(), keep=True):
    p = problem(t, dtype, act, limit)
    out = put(marked((p.num_rows, p.out_features), dtype))
    pre = put(marked((p.num_rows, p.wide), dtype)) if keep else None
    moe.expert_linear(p, put(t["x"]), put(t["w"]), out, expert_offsets=device_offsets(t),
                      pre_act=pre)
    want = X.linear(f64(t["x"]), f64(t["w"]), t["off"], act, limit)
    close(out[:last], *(v[:last] for v in want["out"]), "out")
    assert untouched(out[last:])
    if keep:
        close(pre[:last], *(v[:last] for v in want["pre_act"]), "pre_act")
        assert untouched(pre[last:])
    return out


def check_backward(t, last, dtype, act, limit=0.0, put=lambda v: v.cuda()):
    p = problem(t, dtype, act, limit)
    gx = put(marked(t["x"].shape, dtype))
    gw = put(marked(t["w"].shape, dtype))
    moe.expert_linear_backward(p, put(t["x"]), put(t["w"]), put(t["gout"]), gx, gw,
                               expert_offsets=device_offsets(t),
                               pre_act=None if act == "none" else put(t["pre"]))
    step = 0.0 if act == "none" else torch.finfo(dtype).eps / 2
    want = X.linear_grad(f64(t["x"]), f64(t["w"]), t["off"], f64(t["gout"]), f64(t["pre"]), act,
                         limit, step)
    close(gx[:last], *(v[:last] for v in want["grad_x"]), "grad_x")
    close(gw, *want["grad_weight"], "grad_weight")
    assert untouched(gx[last:])
    return gx, gw


SHAPES = [
    # R, E, K, N, rows behind the last expert's
    (1, 1, 64, 64, 0), (1, 1, 1, 1, 0), (3, 1, 7, 5, 0), (5, 3, 9, 17, 2),
    (64, 1, 128, 128, 0), (65, 2, 136, 72, 1), (130, 5, 255, 129, 7), (200, 9, 320, 260, 0),
    (17, 64, 96, 40, 3), (300, 3, 1001, 33, 0), (257, 2, 64, 513, 30), (700, 1, 200, 300, 100),
    (40, 1024, 32, 24, 4), (9, 5, 72, 8, 9)]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_shapes(i, act, dtype):
    R, E, K, N, behind = SHAPES[i]
    t, last = make(i, R, E, K, N, dtype, act, behind=behind)
    check_forward(t, last, dtype, act)
    check_backward(t, last, dtype, act)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("act,limit", [(a, 0.0) for a in X.GATED + X.SINGLE] + [
    ("silu", 1.0), ("swigluoai", 0.75), ("swiglustep", 0.5)])
def test_activations(act, limit, dtype):
    t, last = make(7, 150, 3, 88, 52, dtype, act, behind=3)
    check_forward(t, last, dtype, act, limit)
    check_backward(t, last, dtype, act, limit)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("by", [1, 3, 4])
def test_addresses(by, dtype):
    """Data at an element's address, 16-byte rows or not."""
    for i, (R, E, K, N) in enumerate([(70, 2, 64, 48), (33, 1, 65, 30), (300, 2, 128, 128)]):
        t, last = make(20 + i, R, E, K, N, dtype, "silu")
        put = lambda v: shifted(v, by)                               # noqa: E731
        check_forward(t, last, dtype, "silu", put=put)
        check_backward(t, last, dtype, "silu", put=put)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_one_expert_without_offsets(dtype):
    for R in (1, 2, 15, 16, 17, 31, 33, 48, 63, 64, 127, 129, 256, 300):
        t, last = make(R, R, 1, 264, 136, dtype, "silu", offsets=None)
        a = check_forward(t, last, dtype, "silu")
        t["off"] = np.array([0, R])
        assert torch.equal(a, check_forward(t, last, dtype, "silu"))
        check_backward(t, last, dtype, "silu")


def test_offsets_that_do_not_ascend_stay_inside():
    """Rows are cut to [0, R]: what surrounds the outputs stays as it was."""
    R, E, K, N = 40, 4, 64, 48
    t, _ = make(1, R, E, K, N, torch.bfloat16, "silu", offsets=[0, 1, 2, 3, 4])
    for name in ("x", "gout", "pre"):
        t[name] = torch.nan_to_num(t[name])
    p = problem(t, torch.bfloat16, "silu")
    for off in ([5, 1 << 30, -7, 12, 2000], [-9, -8, -7, -6, -5], [40, 30, 20, 10, 0],
                [0, 100, 100, 100, 100]):
        off = torch.tensor(off, dtype=torch.int32, device="cuda")
        room = {k: marked((3 * R, w), torch.bfloat16) for k, w in
                (("out", N), ("pre", 2 * N), ("gx", K))}
        mid = {k: v[R:2 * R] for k, v in room.items()}
        gw = marked((3 * E, 2 * N, K), torch.bfloat16)
        x, w, gout, pre = (t[k].cuda() for k in ("x", "w", "gout", "pre"))
        moe.expert_linear(p, x, w, mid["out"], expert_offsets=off, pre_act=mid["pre"])
        moe.expert_linear_backward(p, x, w, gout, mid["gx"], gw[E:2 * E], expert_offsets=off,
                                   pre_act=pre)
        torch.cuda.synchronize()
        for v in room.values():
            assert untouched(v[:R]) and untouched(v[2 * R:])
        assert untouched(gw[:E]) and untouched(gw[2 * E:])


@pytest.mark.parametrize("act", ["none", "silu"])
def test_no_rows(act):
    t, _ = make(1, 4, 3, 16, 8, torch.bfloat16, act, offsets=[0, 0, 0, 0])
    out, gx, gw = check_forward(t, 0, torch.bfloat16, act), *check_backward(t, 0, torch.bfloat16,
                                                                         act)
    assert untouched(out) and untouched(gx) and not gw.any()
    p = moe.ExpertLinear(0, 16, 8, 3, activation=act)
    empty = torch.empty((0, 16), dtype=torch.bfloat16, device="cuda")
    eo = torch.empty((0, 8), dtype=torch.bfloat16, device="cuda")
    gw = marked((3, p.wide, 16), torch.bfloat16)
    moe.expert_linear(p, empty, t["w"].cuda(), eo)
    moe.expert_linear_backward(p, empty, t["w"].cuda(), eo, empty, gw)
    assert not gw.any()


def test_either_gradient_alone():
    t, last = make(3, 90, 3, 72, 40, torch.bfloat16, "silu")
    gx, gw = check_backward(t, last, torch.bfloat16, "silu")
    p = problem(t, torch.bfloat16, "silu")
    a, b = marked(gx.shape, gx.dtype), marked(gw.shape, gw.dtype)
    d = {k: t[k].cuda() for k in ("x", "w", "gout", "pre")}
    off = device_offsets(t)
    moe.expert_linear_backward(p, None, d["w"], d["gout"], a, None, expert_offsets=off,
                               pre_act=d["pre"])
    moe.expert_linear_backward(p, d["x"], None, d["gout"], None, b, expert_offsets=off,
                               pre_act=d["pre"])
    assert torch.equal(a, gx) and torch.equal(b, gw)


def test_infinities_stay_in_their_rows():
    """A row or an expert with infinities or NaN does not reach the others."""
    t, last = make(4, 70, 4, 80, 48, torch.bfloat16, "silu", offsets=[0, 20, 20, 45, 70])
    clean = check_forward(t, last, torch.bfloat16, "silu")
    cgx, cgw = check_backward(t, last, torch.bfloat16, "silu")
    bad = {k: v.clone() if torch.is_tensor(v) else v for k, v in t.items()}
    for k in ("x", "gout", "pre"):
        bad[k][20:45] = float("inf")
        bad[k][21] = float("nan")
    bad["w"][2] = float("nan")
    bad["w"][1] = float("inf")             # the expert without rows
    p = problem(t, torch.bfloat16, "silu")
    out, gx, gw = (marked(v.shape, v.dtype) for v in (clean, cgx, cgw))
    moe.expert_linear(p, bad["x"].cuda(), bad["w"].cuda(), out, expert_offsets=device_offsets(t))
    moe.expert_linear_backward(p, bad["x"].cuda(), bad["w"].cuda(), bad["gout"].cuda(), gx, gw,
                               expert_offsets=device_offsets(t), pre_act=bad["pre"].cuda())
    rest = [*range(20), *range(45, 70)]
    assert torch.equal(out[rest], clean[rest]) and torch.equal(gx[rest], cgx[rest])
    assert torch.equal(gw[[0, 1, 3]], cgw[[0, 1, 3]])


def test_replayed_graph_and_other_stream():
    t, last = make(9, 150, 4, 136, 72, torch.bfloat16, "silu", behind=5)
    p = problem(t, torch.bfloat16, "silu")
    d = {k: t[k].cuda() for k in ("x", "w", "gout", "pre")}
    off, ws = device_offsets(t), moe.alloc_expert_linear_workspace(p)
    shapes = {"out": (150, 72), "act": (150, 144), "gx": (150, 136), "gw": t["w"].shape}
    o = {k: marked(s, torch.bfloat16) for k, s in shapes.items()}

    def calls():
        moe.expert_linear(p, d["x"], d["w"], o["out"], expert_offsets=off, pre_act=o["act"])
        moe.expert_linear_backward(p, d["x"], d["w"], d["gout"], o["gx"], o["gw"],
                                   expert_offsets=off, pre_act=o["act"], ws=ws)

    calls()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    eager = {k: v.clone() for k, v in o.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        calls()
    for turn in range(3):
        d["x"].mul_(-1.0)                  # other work, and other inputs, in between
        for v in o.values():
            v.fill_(float(turn))
        ws.fill_(0xAB)
        if turn == 1:                      # out and pre change with x's sign
            graph.replay()
            for k in o:
                assert torch.equal(o[k][:last] if k != "gw" else o[k],
                                   eager[k][:last] if k != "gw" else eager[k]), k
        else:
            graph.replay()
            torch.cuda.synchronize()
            got = {k: v.clone() for k, v in o.items()}
            calls()
            for k in o:
                assert torch.equal(got[k], o[k]), k


def test_two_threads():
    ts = [make(30 + i, 120, 3, 96, 64, torch.float16, "silu") for i in range(2)]
    want = [check_backward(t, last, torch.float16, "silu") for t, last in ts]
    got, fail = [None, None], []

    def work(i):
        try:
            t, last = ts[i]
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    got[i] = check_backward(t, last, torch.float16, "silu")
                torch.cuda.current_stream().synchronize()
        except BaseException as e:         # noqa: BLE001 -- handed to the test
            fail.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not fail, fail
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))


def test_large_tiles_and_repeats():
    """Experts of several tiles of rows and columns; the same bits every time."""
    t, last = make(11, 1500, 3, 520, 392, torch.bfloat16, "silu", behind=20)
    a = check_forward(t, last, torch.bfloat16, "silu")
    b = check_backward(t, last, torch.bfloat16, "silu")
    for _ in range(3):
        assert torch.equal(a, check_forward(t, last, torch.bfloat16, "silu"))
        assert all(torch.equal(u, v) for u, v in
                   zip(b, check_backward(t, last, torch.bfloat16, "silu")))


# ---- the kernels that sizes choose --------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("act", ["none", "silu", "gelu_no_mul"])
@pytest.mark.parametrize("R,E,K,N,behind", [
    (1, 1, 4096, 24, 0), (5, 1, 4104, 33, 0), (16, 1, 136, 700, 0), (17, 1, 1000, 40, 0),
    (70, 1, 264, 50, 0), (128, 1, 72, 24, 0), (12, 6, 4160, 21, 2), (3, 40, 4096, 16, 1),
    (60, 2, 520, 64, 3), (9, 300, 4096, 8, 0)])
def test_few_rows_forward(R, E, K, N, behind, act, dtype):
    t, last = make(R + K, R, E, K, N, dtype, act, behind=behind)
    check_forward(t, last, dtype, act)
    check_forward(t, last, dtype, act, keep=False)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_whole_cards_of_large_tiles(dtype):
    """More than 256 tiles of 256 x 256, ragged on every side: out, grad_x (many
    columns of the weights) and grad_weight (many experts)."""
    t, last = make(41, 9000, 3, 72, 2000, dtype, "none", behind=5)
    check_forward(t, last, dtype, "none")
    t, last = make(42, 9000, 3, 2072, 40, dtype, "silu", behind=5)
    check_backward(t, last, dtype, "silu")
    t, last = make(43, 600, 64, 520, 264, dtype, "silu", behind=5)
    check_backward(t, last, dtype, "silu")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_whole_cards_of_large_unaligned_tiles(dtype):
    t, last = make(44, 4500, 2, 77, 4001, dtype, "none", behind=5)
    check_forward(t, last, dtype, "none")
    t, last = make(45, 4500, 2, 4001, 27, dtype, "silu", behind=5)
    check_backward(t, last, dtype, "silu")
    t, last = make(46, 600, 64, 519, 263, dtype, "silu", behind=5)
    check_backward(t, last, dtype, "silu")


@pytest.mark.parametrize("rows", [1, 40, 65, 129, 200, 256, 257])
def test_large_tiles_of_few_rows(rows):
    """Tiles with a quarter, half and all of their rows."""
    E, N = 40, 2048
    off = np.minimum(np.arange(E + 1) * 77, 2990)
    off = np.concatenate([off[:20], off[20:] - off[20] + off[19] + rows])
    t, last = make(rows, 40 * 77 + 400, E, 64, N, torch.bfloat16, "none",
                   offsets=off.tolist())
    check_forward(t, last, torch.bfloat16, "none")


@pytest.mark.parametrize("K,N,E,R", [(1, 32768, 2, 9), (32768, 1, 2, 9), (8, 3, 1024, 1),
                                     (32768, 24, 1, 3)])
def test_the_ends_of_the_sizes(K, N, E, R):
    for dtype in (torch.bfloat16, torch.float32):
        t, last = make(K + N, R, E, K, N, dtype, "none")
        check_forward(t, last, dtype, "none")
        check_backward(t, last, dtype, "none")


def test_weights_past_four_gib():
    """All experts' weights are more than 32-bit offsets reach; each alone is not."""
    E, K, N = 40, 8192, 8192                                   # 5.4 GB of bf16
    w = torch.zeros((E, N, K), dtype=torch.bfloat16, device="cuda")
    w[E - 1, N - 1, K - 1] = 3.0
    x = torch.zeros((80, K), dtype=torch.bfloat16, device="cuda")
    x[:, K - 1] = torch.arange(80, device="cuda").to(torch.bfloat16)
    off = (torch.arange(E + 1, device="cuda") * 2).to(torch.int32)
    p = moe.ExpertLinear(80, K, N, E)
    out = torch.empty((80, N), dtype=torch.bfloat16, device="cuda")
    moe.expert_linear(p, x, w, out, expert_offsets=off)
    want = torch.zeros_like(out)
    want[78:, N - 1] = 3.0 * x[78:, K - 1]
    assert torch.equal(out, want)
    gx = torch.empty_like(x)
    gw = torch.empty_like(w)
    moe.expert_linear_backward(p, x, w, out, gx, gw, expert_offsets=off)
    assert torch.equal(gx[:78], torch.zeros_like(gx[:78]))
    assert torch.equal(gx[78:, K - 1], 3.0 * out[78:, N - 1])
    total = (out[78:, N - 1].double() * x[78:, K - 1].double()).sum().to(torch.bfloat16)
    assert gw[E - 1, N - 1, K - 1] == total and int((gw != 0).sum()) == 1


# ---- as they are used together ------------------------------------------------------

def test_a_training_step_around_the_experts():
    """Router, sorted rows, both linear layers, the weighted combine and every
    gradient, in fp32, against torch's differentiation in 64 bits.

    Each step is off by a few sums' roundings of its terms; six of them in a chain,
    of at most 96 terms: 6 * 2 * (96 + 8) * 2^-24 of the gradient's norm, times 8
    for what cancels: terms of random signs are sqrt(96) / 2 to sqrt(96) times their
    sum, taken as norms, and errors of random signs add up the same way."""
    T, H, F, E, k = 50, 96, 64, 6, 2
    g = torch.Generator().manual_seed(5)
    x, w1, w2, gy = (torch.randn(s, generator=g) for s in
                     ((T, H), (E, 2 * F, H), (E, H, F), (T, H)))
    w1, w2 = w1 * H ** -0.5, w2 * F ** -0.5
    logits = torch.randn((T, E), generator=g)
    f32 = torch.float32
    r = moe.Router(T, E, k)
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    wt = torch.empty((T, k), dtype=f32, device="cuda")
    moe.router_topk(r, logits.cuda(), ids, wt)
    rows = moe.ExpertRows(T, H, E, k, dtype=f32)
    s = moe.alloc_permute_outputs(rows)
    moe.permute(rows, x.cuda(), ids, **s)
    up = moe.ExpertLinear(T * k, H, F, E, dtype=f32, activation="silu")
    down = moe.ExpertLinear(T * k, F, H, E, dtype=f32)
    e = lambda *shape: torch.empty(shape, device="cuda")                # noqa: E731
    h, pre, yr, y = e(T * k, F), e(T * k, 2 * F), e(T * k, H), e(T, H)
    W1, W2, off = w1.cuda(), w2.cuda(), s["expert_offsets"]
    moe.expert_linear(up, s["rows"], W1, h, expert_offsets=off, pre_act=pre)
    moe.expert_linear(down, h, W2, yr, expert_offsets=off)
    moe.unpermute(rows, yr, s["slot_row"], wt, y)
    gr, gw, gh, gx_rows, gx = e(T * k, H), e(T, k), e(T * k, F), e(T * k, H), e(T, H)
    g1, g2, glog = e(*w1.shape), e(*w2.shape), e(T, E)
    moe.unpermute_backward(rows, gy.cuda(), yr, s["slot_row"], wt, gr, gw)
    moe.expert_linear_backward(down, h, W2, gr, gh, g2, expert_offsets=off)
    moe.expert_linear_backward(up, s["rows"], W1, gh, gx_rows, g1, expert_offsets=off,
                               pre_act=pre)
    moe.permute_backward(rows, gx_rows, s["slot_row"], gx)
    moe.router_topk_backward(r, logits.cuda(), ids, gw, glog)

    d = {n: v.double().requires_grad_() for n, v in
         dict(x=x, w1=w1, w2=w2, logits=logits).items()}
    p = torch.softmax(d["logits"], 1).gather(1, ids.cpu().long())
    p = p / p.sum(1, keepdim=True)
    at = ids.cpu().long()
    both = torch.einsum("th,tkfh->tkf", d["x"], d["w1"][at])
    hd = torch.nn.functional.silu(both[..., :F]) * both[..., F:]
    yd = (p[:, :, None] * torch.einsum("tkf,tkhf->tkh", hd, d["w2"][at])).sum(1)
    (yd * gy.double()).sum().backward()
    yd = yd.detach()
    bound = 6 * 2 * (96 + 8) * X.U * 8
    assert float((y.cpu().double() - yd).norm()) <= bound * float(yd.norm())
    for name, got in (("x", gx), ("w1", g1), ("w2", g2), ("logits", glog)):
        want = d[name].grad
        assert float((got.cpu().double() - want).norm()) <= bound * float(want.norm()), name


def test_a_decode_step_with_4_bit_experts():
    """Sorted rows through both 4-bit layers and back, as one captured graph, bit for
    bit the calls one by one; the same weights as the layer's MXFP4 ones."""
    T, H, F, E, k = 9, 256, 128, 8, 2
    rng = np.random.default_rng(2)
    byte = lambda *s: torch.from_numpy(rng.integers(0, 256, s, dtype=np.uint8)).cuda()  # noqa: E731,E501
    exps = lambda *s: torch.from_numpy(rng.integers(117, 122, s, dtype=np.uint8)).cuda()  # noqa: E731,E501
    x = rand(rng, (T, H), torch.bfloat16).cuda()
    ids = torch.from_numpy(np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int32)).cuda()
    wt = torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda()
    rows = moe.ExpertRows(T, H, E, k)
    s = moe.alloc_permute_outputs(rows)
    up = moe.ExpertLinearW4(T * k, H, F, E, activation="silu", format="mxfp4", group_size=32)
    down = moe.ExpertLinearW4(T * k, F, H, E, format="int4", group_size=64)
    c1, s1 = byte(E, 2 * F, H // 2), exps(E, 2 * F, H // 32)
    c2 = byte(E, H, F // 2)
    s2 = rand(rng, (E, H, F // 64), torch.bfloat16, 0.02).cuda()
    h = torch.empty((T * k, F), dtype=torch.bfloat16, device="cuda")
    yr = torch.empty((T * k, H), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")

    def step():
        moe.permute(rows, x, ids, **s)
        moe.expert_linear_w4(up, s["rows"], c1, s1, h, expert_offsets=s["expert_offsets"])
        moe.expert_linear_w4(down, h, c2, s2, yr, expert_offsets=s["expert_offsets"])
        moe.unpermute(rows, yr, s["slot_row"], wt, y)

    step()
    v1 = X.dequant_w4(c1.cpu().numpy(), s1.cpu().numpy(), "mxfp4")
    v2 = X.dequant_w4(c2.cpu().numpy(), f64(s2), "int4")
    off = s["expert_offsets"].cpu().numpy()
    close(h, *X.linear_w4(f64(s["rows"]), *v1, off, "silu"), "h")
    close(yr, *X.linear_w4(f64(h), *v2, off), "y rows")
    want = y.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        step()
    for turn in range(3):
        for v in (h, yr, y, s["rows"]):
            v.fill_(float(turn))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


# ---- gradients whose reduction is split -----------------------------------------------

@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("R,E,K,N,behind", [
    (6300, 1, 136, 200, 0), (6999, 1, 77, 131, 0), (9000, 2, 264, 72, 3), (5, 1, 72, 4400, 0),
    (70, 3, 40, 3500, 1), (33, 1, 129, 4047, 0), (9500, 3, 8, 8, 7)])
def test_split_gradients(R, E, K, N, behind, dtype, act):
    p = moe.ExpertLinear(R, K, N, E, dtype=dtype, activation=act)
    d = 0 if act == "none" else R * p.wide * dtype.itemsize
    assert moe.expert_linear_workspace_size(p) > d + 512            # there are parts
    t, last = make(R + K, R, E, K, N, dtype, act, behind=behind)
    check_backward(t, last, dtype, act)


def test_split_gradients_of_one_expert_with_all_rows():
    off = [0, 0, 0, 12990, 12990]
    t, last = make(8, 13000, 4, 136, 100, torch.bfloat16, "silu", offsets=off)
    check_backward(t, last, torch.bfloat16, "silu")


def test_split_gradients_replayed():
    """One captured graph, its workspace dirty before every replay, with other rows per
    expert in each."""
    R, K, N, E = 6500, 264, 72, 2
    p = moe.ExpertLinear(R, K, N, E, activation="silu")
    rng = np.random.default_rng(4)
    dev = lambda *s: rand(rng, s, torch.bfloat16).cuda()               # noqa: E731
    x, w, g, pre = dev(R, K), dev(E, 2 * N, K), dev(R, N), dev(R, 2 * N)
    off = torch.tensor([0, 100, R], dtype=torch.int32, device="cuda")
    gx, gw = torch.empty_like(x), torch.empty_like(w)
    ws = moe.alloc_expert_linear_workspace(p)
    call = lambda a, b, s: moe.expert_linear_backward(                  # noqa: E731
        p, x, w, g, a, b, expert_offsets=off, pre_act=pre, ws=s)
    call(gx, gw, ws)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        call(gx, gw, ws)
    for first in (0, 1700, 6500):
        off[1] = first
        for v in (gx, gw):
            v.fill_(7.0)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        ax, aw = torch.empty_like(x), torch.empty_like(w)
        call(ax, aw, "auto")
        assert torch.equal(gx, ax) and torch.equal(gw, aw)


def test_long_sums_of_fp32():
    """32768 terms: parts of 256 are summed first, so the error is that of 256 + 128
    additions in a chain at most, not of 32768."""
    g = torch.Generator().manual_seed(3)
    x, w = torch.rand((40, 32768), generator=g), torch.rand((1, 24, 32768), generator=g)
    p = moe.ExpertLinear(40, 32768, 24, 1, dtype=torch.float32)
    out = torch.empty((40, 24), device="cuda")
    moe.expert_linear(p, x.cuda(), w.cuda(), out)
    want = x.double() @ w[0].double().T
    assert float(((out.cpu().double() - want) / want).abs().max()) <= (256 + 128) * X.U

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

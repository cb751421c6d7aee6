"""Rows sorted by expert times 4-bit weights on the GPU against the 64-bit
oracle, whose bounds (oracle/expert_oracle.py) are the tolerances, plus half
a step of the type that leaves.  Integer codes may be carried as 128 + q,
corrected by the sum of x: the bound counts |s| (144 + |z|) per column."""
import numpy as np
import pytest
import torch

import fp8_block_quantized_group_amd as moe
from expert_util import close, f64, marked, rand, shifted, spread, untouched
from oracle import expert_oracle as X

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
FORMS = [("int4", 32), ("int4", 64), ("int4", 128), ("int4_zero", 32), ("int4_zero", 64),
         ("int4_zero", 128), ("mxfp4", 32)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    moe.load_library()


def make(seed, R, E, K, N, dtype, form, group, act="none", scale_dtype=None, offsets="spread",
         behind=0, top=16):
    rng = np.random.default_rng(seed)
    wide = N * (2 if act in X.GATED else 1)
    off = None
    if offsets == "spread":
        off = spread(rng, R - behind, E)
    elif offsets is not None:
        off = np.asarray(offsets)
    t = {"x": rand(rng, (R, K), dtype), "off": off, "zeros": None,
         "codes": torch.from_numpy(rng.integers(0, 256, (E, wide, K // 2), dtype=np.uint8))}
    G = K // group
    if form == "mxfp4":
        t["scales"] = torch.from_numpy(rng.integers(118, 124, (E, wide, G), dtype=np.uint8))
    else:
        t["scales"] = torch.from_numpy(
            (np.exp(rng.normal(0, 0.5, (E, wide, G))) * 0.2 * K ** -0.5).astype(
                np.float32)).to(scale_dtype or dtype)
        if form == "int4_zero":
            t["zeros"] = torch.from_numpy(rng.integers(0, top, (E, wide, G), dtype=np.uint8))
    last = R if off is None else int(off[-1])
    t["x"][last:] = float("nan")
    p = moe.ExpertLinearW4(R, K, N, E, dtype=dtype, activation=act, format=form,
                           group_size=group,
                           scale_dtype=None if form == "mxfp4" else scale_dtype)
    return t, last, p


def run(t, p, put=lambda v: v.cuda()):
    out = put(marked((p.num_rows, p.out_features), p.dtype))
    off = None if t["off"] is None else torch.from_numpy(t["off"]).to(torch.int32).cuda()
    moe.expert_linear_w4(p, put(t["x"]), put(t["codes"]), put(t["scales"]), out,
                         expert_offsets=off,
                         zeros=None if t["zeros"] is None else put(t["zeros"]))
    return out


def check(t, last, p, put=lambda v: v.cuda()):
    out = run(t, p, put)
    sc = t["scales"].numpy() if p.format == "mxfp4" else f64(t["scales"])
    w, mag = X.dequant_w4(t["codes"].numpy(), sc, p.format,
                          None if t["zeros"] is None else t["zeros"].numpy())
    want = X.linear_w4(f64(t["x"]), w, mag, t["off"], p.activation)
    close(out[:last], *(v[:last] for v in want), "out")
    assert untouched(out[last:])
    return out


SHAPES = [
    # R, E, K, N, rows behind the last expert's
    (1, 1, 128, 16, 0), (1, 1, 128, 1, 0), (3, 1, 384, 33, 0), (16, 1, 1152, 64, 0),
    (17, 2, 256, 40, 1), (33, 1, 2304, 24, 0), (65, 1, 128, 17, 0), (200, 3, 640, 50, 9),
    (24, 64, 256, 31, 4), (40, 1024, 128, 20, 3)]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("form,group", FORMS)
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_shapes(i, form, group, dtype):
    R, E, K, N, behind = SHAPES[i]
    check(*make(i, R, E, K, N, dtype, form, group, behind=behind))
    check(*make(i, R, E, K, N, dtype, form, group, act="silu", behind=behind))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("group,K", [(32, 32), (32, 96), (32, 1312), (64, 64), (64, 192),
                                     (64, 1088)])
def test_columns_that_end_inside_a_run(group, K, dtype):
    for form in ("int4", "int4_zero") + (("mxfp4",) if group == 32 else ()):
        check(*make(K, 5, 2, K, 37, dtype, form, group, offsets=[0, 2, 5]))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("act", X.GATED + X.SINGLE)
def test_activations(act, dtype):
    check(*make(5, 20, 2, 256, 40, dtype, "int4", 64, act=act))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_scale_types_zero_points_and_addresses(dtype):
    for form in ("int4", "int4_zero"):
        check(*make(6, 7, 2, 256, 40, dtype, form, 32, scale_dtype=torch.float32))
    check(*make(6, 7, 2, 256, 40, dtype, "int4_zero", 64, top=256))
    for by in (1, 3):
        put = lambda v: shifted(v, by)                               # noqa: E731
        for form, group in FORMS:
            check(*make(6, 19, 2, 256, 23, dtype, form, group, act="silu"), put=put)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_extreme_codes_and_scales(dtype):
    """All-equal codes (sums that only the zero point cancels), scales of every
    sign, the ends of E8M0."""
    for code in (0x00, 0x88, 0xFF):
        for form in ("int4", "int4_zero"):
            t, last, p = make(8, 9, 1, 512, 18, dtype, form, 128, offsets=None)
            t["codes"].fill_(code)
            t["scales"][:, ::2] *= -1
            t["scales"][:, 3] = 0
            check(t, last, p)
    t, last, p = make(9, 9, 1, 256, 16, dtype, "mxfp4", 32, offsets=None)
    t["x"] *= 2.0 ** -9
    for i, e in enumerate((0, 1, 60, 100, 126, 127, 128, 130, 133)):
        t["scales"][0, i] = e
    check(t, last, p)
    t["scales"][0, 11, 3] = 255
    out = run(t, p)
    assert out[:, 11].isnan().all() and not out[:, :11].isnan().any()


def test_rows_with_nan_stay_alone():
    t, last, p = make(4, 30, 2, 256, 40, torch.bfloat16, "int4", 32, offsets=[0, 12, 30])
    clean = check(t, last, p)
    t["x"][3] = float("nan")
    t["x"][20] = float("inf")
    out = run(t, p)
    keep = [r for r in range(30) if r not in (3, 20)]
    assert torch.equal(out[keep], clean[keep])
    assert not out[[3, 20]].isfinite().any()


def test_no_rows_and_offsets_that_do_not_ascend():
    t, last, p = make(1, 6, 3, 128, 24, torch.bfloat16, "int4", 64, offsets=[0, 0, 0, 0])
    assert untouched(run(t, p))
    t["x"] = torch.zeros_like(t["x"])
    for off in ([5, 1 << 30, -7, 12], [-9, -8, -7, -6], [6, 4, 2, 0], [0, 100, 100, 100]):
        t["off"] = np.array(off)
        room = marked((18, 24), torch.bfloat16)
        moe.expert_linear_w4(p, t["x"].cuda(), t["codes"].cuda(), t["scales"].cuda(), room[6:12],
                             expert_offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
        assert untouched(room[:6]) and untouched(room[12:])


def test_replayed_graph():
    t, last, p = make(2, 40, 8, 512, 72, torch.bfloat16, "mxfp4", 32, act="silu", behind=3)
    d = {k: t[k].cuda() for k in ("x", "codes", "scales")}
    off = torch.from_numpy(t["off"]).to(torch.int32).cuda()
    out = marked((40, 72), torch.bfloat16)

    def call():
        moe.expert_linear_w4(p, d["x"], d["codes"], d["scales"], out, expert_offsets=off)

    call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    for turn in range(3):
        d["x"].mul_(0.5)
        out.fill_(float(turn))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        call()
        assert torch.equal(got, out)


@pytest.mark.parametrize("form,group", FORMS)
@pytest.mark.parametrize("R,E,K,N", [
    (4, 3, 1024, 40), (4, 3, 3968, 40), (4, 3, 4224, 24), (4, 2, 8192, 24), (4, 2, 8320, 24),
    (3, 2, 4224, 16500), (20, 1, 1024, 24), (40, 1, 1024, 24), (64, 1, 1152, 24),
    (100, 1, 512, 20)])
def test_kernels_that_sizes_choose(R, E, K, N, form, group):
    """x in registers with 8 x 2, 8 x 4 and 16 x 4 runs (the last of many tiles), and
    streamed, in row tiles of 16 to 64; wholes and parts of the waves' runs."""
    for act in ("none", "silu"):
        if N > 10000 and (form != "int4" or group == 32):
            act = "none"
        check(*make(R + K, R, E, K, N if act == "none" or N < 10000 else 8300, torch.bfloat16,
                    form, group, act=act, behind=1 if E > 1 else 0))


def test_other_stream_and_two_threads():
    import threading
    made = [make(30 + i, 40, 4, 512, 64, torch.float16, "int4_zero", 64, act="silu")
            for i in range(2)]
    want = [check(*m) for m in made]
    got, fail = [None, None], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    got[i] = run(made[i][0], made[i][2])
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
        last = made[i][1]
        assert torch.equal(got[i][:last], want[i][:last])

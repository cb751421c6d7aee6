"""NaN, infinities and the far ends of the types through the experts' own products: a
row that went wrong shows, whatever the activation, and the others stay as they were."""
import numpy as np
import pytest
import torch

import fp8_block_quantized_group_amd as moe
from expert_util import marked, rand
from oracle import expert_oracle as X

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
NAN = float("nan")
ACTS = [("none", 0.0)] + [(a, 0.0) for a in X.GATED + X.SINGLE] + [
    ("silu", 1.0), ("swigluoai", 0.75), ("swiglustep", 0.5)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    moe.load_library()


def check_rows(clean, got, bad):
    rest = [r for r in range(clean.shape[0]) if r not in bad]
    assert got[bad].isnan().all()
    assert torch.equal(got[rest], clean[rest])


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("act,limit", ACTS)
@pytest.mark.parametrize("R,K,N", [(5, 72, 40), (150, 65, 33), (300, 128, 264)])
def test_linear(R, K, N, act, limit, dtype):
    rng = np.random.default_rng(R)
    p = moe.ExpertLinear(R, K, N, dtype=dtype, activation=act, act_limit=limit)
    x, w = rand(rng, (R, K), dtype).cuda(), rand(rng, (1, p.wide, K), dtype, K ** -0.5).cuda()

    def run():
        out, pre = marked((R, N), dtype), marked((R, p.wide), dtype)
        moe.expert_linear(p, x, w, out, pre_act=pre)
        return out, pre

    clean = run()
    bad = [1, R - 1]
    x[bad, [3, K - 1]] = NAN
    for a, b in zip(clean, run()):
        check_rows(a, b, bad)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("act,limit", ACTS[1:])
def test_linear_gradients(act, limit, dtype):
    """NaN in a gate or an only column, and in an up column, of pre_act; in grad_out.
    grad_weight: the column's own rows of it (of the up column at a clamp)."""
    rng, R, K, N = np.random.default_rng(3), 20, 72, 40
    p = moe.ExpertLinear(R, K, N, dtype=dtype, activation=act, act_limit=limit)
    x, w = rand(rng, (R, K), dtype).cuda(), rand(rng, (1, p.wide, K), dtype, K ** -0.5).cuda()
    gout, pre = rand(rng, (R, N), dtype).cuda(), rand(rng, (R, p.wide), dtype, 0.2).cuda()

    def run(gout, pre):
        gx, gw = marked((R, K), dtype), marked(w.shape, dtype)
        moe.expert_linear_backward(p, x, w, gout, gx, gw, pre_act=pre)
        return gx, gw[0]

    clean = run(gout, pre)
    for col in (7,) if p.wide == N else (7, N + 7):
        bad = pre.clone()
        bad[4, col] = NAN
        gx, gw = run(gout, bad)
        check_rows(clean[0], gx, [4])
        rest = [c for c in range(p.wide) if c % N != 7]
        assert gw[7].isnan().all() and torch.equal(gw[rest], clean[1][rest])
    bad = gout.clone()
    bad[4, 7] = NAN
    check_rows(clean[0], run(bad, pre)[0], [4])


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("act,limit", ACTS)
@pytest.mark.parametrize("R,K,form,group", [(5, 256, "int4", 64), (40, 512, "int4_zero", 128),
                                            (9, 96, "int4", 32), (20, 256, "mxfp4", 32)])
def test_4_bit_weights(R, K, form, group, act, limit, dtype):
    rng, N = np.random.default_rng(R), 40
    p = moe.ExpertLinearW4(R, K, N, dtype=dtype, activation=act, act_limit=limit, format=form,
                           group_size=group)
    codes = torch.from_numpy(rng.integers(0, 256, (1, p.wide, K // 2), dtype=np.uint8)).cuda()
    groups = (1, p.wide, K // group)
    scales = (torch.full(groups, 124, dtype=torch.uint8) if form == "mxfp4" else
              rand(rng, groups, dtype, 0.1)).cuda()
    zeros = torch.full(groups, 7, dtype=torch.uint8).cuda() if form == "int4_zero" else None
    x = rand(rng, (R, K), dtype).cuda()

    def run():
        out = marked((R, N), dtype)
        moe.expert_linear_w4(p, x, codes, scales, out, zeros=zeros)
        return out

    clean = run()
    bad = [1, R - 1]
    x[bad, [3, K - 1]] = NAN
    check_rows(clean, run(), bad)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("act,limit", ACTS[1:])
def test_gradients_of_large_pre_activations(act, limit, dtype):
    """One row and one column per expert, x = 1: grad_weight is d.  The roundings are the
    oracle's at 20; from 100 on a sigmoid and its slope are 0 or 1, in 64 bits to 1e-40 and
    in 32 exactly, so that nothing rounds with the argument.  An infinity has the slopes
    and, below, the value of the largest numbers."""
    top = torch.finfo(dtype).max
    far = [v for v in (20.0, 100.0, 300.0, 1e4, 1e19, 1e20, 1e30) if v < top] + [top]
    at = [s * v for v in far + [float("inf")] for s in (1, -1)]
    E, gated = len(at), act in X.GATED
    dh, up = 0.5, 0.5
    p = moe.ExpertLinear(E, 1, 1, E, dtype=dtype, activation=act, act_limit=limit)
    pre = torch.tensor([[g, up][:p.wide] for g in at], dtype=dtype)
    ones = torch.ones((E, 1), dtype=dtype, device="cuda")
    gw = marked((E, p.wide, 1), dtype)
    moe.expert_linear_backward(p, ones, None, ones * dh, None, gw, pre_act=pre.cuda(),
                               expert_offsets=torch.arange(E + 1, dtype=torch.int32).cuda())
    got = gw[:, :, 0].cpu().double().numpy()
    pre = pre.double().numpy()
    g = np.clip(pre[:, :1], -1e38, 1e38)       # the slopes of infinities
    f, dg, du = X.activate(act, np.concatenate([g, pre[:, 1:]], 1), limit)
    if act == "relu2_no_mul":
        dg = 2.0 * np.maximum(pre, 0.0)
    want = np.concatenate([dg, du], 1) * dh if gated else dg * dh
    if gated and limit == 0.0 and act in ("silu", "gelu", "gelu_tanh"):
        want[:, 1:] = np.where(pre[:, :1] > 0, pre[:, :1] * dh, want[:, 1:])
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine])
    rel = X.act_rel(20.0) + 3.0 * torch.finfo(dtype).eps / 2     # d, the product, 1 + X
    tiny = float(torch.finfo(dtype).smallest_normal)
    assert (np.abs(got - want)[fine] <= rel * np.abs(want[fine]) * 1.01 + tiny).all(), (got, want)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("quant", ["ue8m0", "fp32", "mxfp8"])
@pytest.mark.parametrize("T,H", [(9, 512), (600, 128), (40, 7168), (600, 5120)])
def test_norm_that_leaves_staged(T, H, quant, dtype):
    """A row with a NaN has NaN codes alone, one with an infinity where it was; the e4m3
    NaN is 0x7F with either sign."""
    x = rand(np.random.default_rng(H), (T, H), dtype)
    p = moe.BlockNorm(T, H, dtype=dtype)

    def run():
        o = moe.alloc_quant_outputs(p, quant)
        o["x_q"].fill_(0x5A)
        moe.block_norm_quant(p, x.cuda(), quant=quant, **o)
        return o["x_q"], o["x_sf"]

    q, sf = run()
    x[1, 7] = NAN
    x[4, 100] = float("inf")
    got, gsf = run()
    rest = [r for r in range(T) if r not in (1, 4)]
    assert torch.equal(got[rest], q[rest]) and torch.equal(gsf[rest], sf[rest])
    nan = (got & 0x7F) == 0x7F
    assert nan[1].all() and nan[4].nonzero().flatten().tolist() == [100]
    assert not nan[rest].any()

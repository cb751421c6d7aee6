"""The operators around the layer on the GPU against the 64-bit oracle:
router, sorted rows, block norms and their gradients, over types, odd widths,
empty rows, masks and the smallest and largest sizes.

Tolerances, each times the oracle's magnitude (the sum of the absolute values
of the terms a result is made of), with u = 2^-24 the half step of fp32:
  * a result rounded to type t on the way out: eps(t) / 2 of its value, and
    half the smallest subnormal of t;
  * exp and the quotients made of it: an argument x - m rounded to half a
    step moves exp by |x - m| u, here at most 64 u; exp, the sum and the
    division add at most 16 u: REL_EXP = 2^-17 = 128 u;
  * a row's mean square: a lane adds at most 64 squares, 6 steps cross the
    wave, 16 waves follow: 86 u, half of it after the square root, and 4 more
    roundings: REL_NORM = 2^-17; a gradient uses its cube and one more such
    sum: REL_GRAD = 2^-15;
  * a sum over n rows: n u at the most, in any order.
"""
import ctypes

import numpy as np
import pytest
import torch

import fp8_block_quantized_group_amd as moe
from oracle import block_oracle as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
REL_EXP, REL_NORM, REL_GRAD = 2.0 ** -17, 2.0 ** -17, 2.0 ** -15
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
MARK = 0x5A                                # byte of buffers that must stay as they were


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    moe.load_library()
    return torch.device("cuda:0")


def f64(t):
    return t.detach().to("cpu").double().numpy()


def close(got, want, mag, rel, what):
    """|got - want| <= rel * mag + the rounding of got's type."""
    eps, tiny = torch.finfo(got.dtype).eps, torch.finfo(got.dtype).smallest_normal
    if got.dtype != torch.float32:
        tiny *= eps                        # half a step below the normal numbers
    tol = rel * mag + 1.01 * (np.abs(want) * eps / 2 + tiny)
    d = np.abs(f64(got) - want)
    bad = ~(d <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst "
                           f"{np.nanmax(d[bad] / tol[bad]):.3g} of the bound")


def rand(rng, shape, dtype, std=1.0):
    return torch.from_numpy(rng.normal(0, std, shape).astype(np.float32)).to(dtype)


def marked(shape, dtype):
    """A device buffer of a byte pattern no kernel writes by chance."""
    t = torch.empty(shape, dtype=dtype, device="cuda")
    t.view(torch.uint8).fill_(MARK) if t.numel() else None
    return t


def shifted(t):
    """The same values at an address that only the element's size divides."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    out = buf[1:].view(t.shape)
    out.copy_(t)
    return out


# ---- router -------------------------------------------------------------------

def run_router(x, k, bias=None, pad=None, grad_w=None, dtype=None, **kw):
    T, E = x.shape
    r = moe.Router(T, E, k, score=kw["score"], num_groups=kw.get("groups", 1),
                   topk_groups=kw.get("topk_groups", 1), group_top=kw.get("group_top", 1),
                   renormalize=kw.get("renormalize", True), scale=kw.get("scale", 1.0),
                   dtype=x.dtype)
    xd = x.cuda()
    ids, w = marked((T, k), torch.int32), marked((T, k), torch.float32)
    moe.router_topk(r, xd, ids, w, bias=None if bias is None else bias.cuda(),
                    is_padding=None if pad is None else pad.cuda())
    if grad_w is None:
        return ids, w, None
    gx = marked((T, E), x.dtype)
    moe.router_topk_backward(r, xd, ids, grad_w.cuda(), gx)
    return ids, w, gx


def check_router(x, k, bias=None, pad=None, seed=0, tokens=None, **kw):
    """tokens: a batch of that many, the rows of x over and over; every copy of
    a row has to give the same bits."""
    rng = np.random.default_rng(seed + 1000)
    n = x.shape[0]
    gw = torch.from_numpy(rng.normal(size=(n, k)).astype(np.float32))
    at = torch.arange(tokens or n) % n
    ids, w, gx = run_router(x[at], k, bias, None if pad is None else pad[at], gw[at], **kw)
    if tokens:
        for t in (ids, w, gx):
            assert torch.equal(t, t[at.cuda()])
        ids, w, gx = ids[:n], w[:n], gx[:n]
    bn, pn = None if bias is None else bias.numpy(), None if pad is None else pad.numpy()
    want_ids, want_w = B.router_topk(f64(x), k, bias=bn, pad=pn, **kw)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    close(w, want_w, np.abs(want_w), REL_EXP, "weights")
    g, mag = B.router_topk_grad(f64(x), want_ids, gw.numpy(), kw["score"],
                                kw.get("renormalize", True), kw.get("scale", 1.0))
    close(gx, g, mag, 2 * REL_EXP, "grad_logits")


GROUPED = dict(groups=8, topk_groups=4, group_top=2)
ROUTERS = [
    # T, E, k, settings
    (1, 256, 8, dict(score="sigmoid", bias=True, scale=2.5, **GROUPED)),
    (131, 256, 8, dict(score="sigmoid", bias=True, scale=2.5, **GROUPED)),
    (67, 128, 8, dict(score="softmax")),
    (67, 128, 8, dict(score="softmax", renormalize=False)),
    (33, 60, 4, dict(score="softmax", renormalize=False, bias=True)),
    (33, 160, 6, dict(score="softmax", renormalize=False, groups=8, topk_groups=3, scale=16.0)),
    (33, 72, 5, dict(score="softmax", groups=9, topk_groups=2, group_top=2)),
    (9, 8, 2, dict(score="softmax")),
    (5, 1, 1, dict(score="sigmoid")),
    (5, 7, 7, dict(score="sigmoid", renormalize=False)),
    (17, 64, 64, dict(score="sigmoid", bias=True)),
    (17, 64, 3, dict(score="sigmoid", groups=64, topk_groups=9)),
    (9, 1024, 64, dict(score="softmax", renormalize=False)),
    (9, 1000, 10, dict(score="sigmoid", bias=True, groups=4, topk_groups=1, group_top=2)),
    (13, 384, 8, dict(score="sigmoid", bias=True, renormalize=False)),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("i", range(len(ROUTERS)))
def test_router(gpu, i, dtype):
    T, E, k, kw = ROUTERS[i]
    kw = dict(kw)
    rng = np.random.default_rng(i)
    bias = torch.from_numpy(rng.normal(0, 0.1, E).astype(np.float32)) if kw.pop("bias", False) \
        else None
    x = rand(rng, (T, E), dtype, 2.0)
    pad = torch.from_numpy((rng.random(T) < 0.2).astype(np.uint8))
    check_router(x, k, bias, pad, i, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("grouped", [False, True])
def test_router_masks_and_special_values(gpu, score, renormalize, grouped):
    """Masked experts, rows with fewer experts than slots or none, NaN and
    both infinities, the type's lowest and largest values, padding tokens full
    of NaN, equal logits."""
    rng = np.random.default_rng(4)
    x = rand(rng, (12, 32), torch.float32)
    x[0] = -np.inf
    x[1, 3:] = -np.inf
    x[2, ::2] = np.nan
    x[3] = np.nan
    x[4, 5] = np.inf
    x[5, 7:] = torch.finfo(torch.float32).min
    x[6] = torch.finfo(torch.float32).min
    x[7] = np.nan                            # padding
    x[8] = 0.25
    x[9, 16:] = x[9, :16]
    x[10, 4] = torch.finfo(torch.float32).max
    x[11, 1:] = -80.0
    x[11, 0] = -88.0
    pad = torch.zeros(12, dtype=torch.uint8)
    pad[7] = 1
    bias = torch.zeros(32)
    bias[9] = 0.5
    kw = dict(score=score, renormalize=renormalize)
    if grouped:
        kw.update(groups=4, topk_groups=2, group_top=2)
    check_router(x, 6, bias if grouped else None, pad, **kw)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("E,k,kw", [
    (256, 8, dict(score="sigmoid", bias=True, scale=2.5, **GROUPED)),
    (128, 8, dict(score="softmax", renormalize=False)),
    (60, 4, dict(score="softmax", bias=True)),
    (160, 6, dict(score="softmax", renormalize=False, groups=10, topk_groups=3, scale=16.0)),
    (17, 15, dict(score="sigmoid")), (100, 15, dict(score="sigmoid", renormalize=False)),
    (64, 5, dict(score="softmax", groups=16, topk_groups=5, group_top=2)),
    (128, 1, dict(score="softmax", bias=True, groups=2, topk_groups=1)),
    (256, 9, dict(score="softmax", bias=True, groups=4, topk_groups=2, group_top=2)),
    (250, 3, dict(score="sigmoid", bias=True)), (24, 16, dict(score="sigmoid")),
    (256, 4, dict(score="sigmoid", groups=32, topk_groups=9))])
def test_router_many_tokens(gpu, E, k, kw, dtype):
    """Batches that share a wave among four tokens, with a last wave of three."""
    kw = dict(kw)
    rng = np.random.default_rng(E + k)
    T = 701
    bias = torch.from_numpy(rng.normal(0, 0.1, E).astype(np.float32)) if kw.pop("bias", False) \
        else None
    x = rand(rng, (T, E), dtype, 2.0)
    x[rng.random(T) < 0.05, 2::3] = -np.inf
    x[rng.random((T, E)) < 1e-3] = np.nan
    x[rng.random((T, E)) < 1e-3] = np.inf
    pad = torch.from_numpy((rng.random(T) < 0.1).astype(np.uint8))
    check_router(x, k, bias, pad, E, tokens=20003, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,group_top", [(1, 1), (8, 1), (8, 2)])
def test_router_many_tokens_hard_to_tell(gpu, score, groups, group_top):
    """The same, with equal keys, keys few steps of fp32 apart, group values
    that cancel, masked rows: tokens that need the choice of 64 bits lie beside
    others in a wave."""
    rng = np.random.default_rng(18)
    T, E, many = 701, 128, 20002
    x = rand(rng, (T, E), torch.float32, 1.0)
    x[0::7] = torch.round(x[0::7])
    x[1::7] *= 2.0 ** -20
    x[2::7, 64:] = x[2::7, :64]
    x[3::7, 5:] = -np.inf
    x[4::35] = -np.inf
    x[5::35] = torch.finfo(torch.float32).min
    kw = dict(score=score, groups=groups, topk_groups=max(1, groups // 2), group_top=group_top)
    check_router(x, 8, None, None, tokens=many, **kw)
    check_router(x, 8, torch.zeros(E), None, tokens=many, **kw)
    check_router(x, 8, rand(rng, (E,), torch.float32, 2.0 ** -10), None, tokens=many, **kw)
    bias = torch.full((E,), -2000.0)
    bias[::16], bias[15::16] = 1000.0, -1000.0
    bias[40:44] = torch.tensor([np.inf, -np.inf, np.nan, 1e30])
    with np.errstate(invalid="ignore"):
        check_router(x, 8, bias, None, tokens=many, **kw)
    check_router(x.bfloat16(), 8, None, None, tokens=many, **kw)


@pytest.mark.parametrize("tokens", [None, 20003])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(64, 16), (128, 8), (256, 8), (256, 16)])
def test_router_groups_of_subnormal_logits(gpu, E, groups, score, tokens):
    """Logits a few steps of 2^-149 apart, or zero: groups are told apart by
    them, in batches of any size."""
    rng = np.random.default_rng(21)
    steps = rng.integers(-40, 41, (200, E))
    steps[0::5] *= 1 << 10
    steps[1::5] //= 16
    x = torch.from_numpy((steps * 2.0 ** -149).astype(np.float32))
    assert (x.double() * 2.0 ** 149 == torch.from_numpy(steps)).all()
    check_router(x, 5, None, None, tokens=tokens, score=score, groups=groups,
                 topk_groups=groups // 4 + 1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(256, 2), (128, 2), (64, 2)])
def test_router_open_tokens_of_one_wave(gpu, E, groups, score):
    """All four tokens of a wave need the choice of 64 bits, one after the other
    through the same LDS, groups and experts alike."""
    rng = np.random.default_rng(25)
    x = rand(rng, (701, E), torch.float32, 2.0 ** -21)
    for top in (1, 2):
        check_router(x, 8, torch.zeros(E), None, tokens=12007, score=score, groups=groups,
                     topk_groups=1, group_top=top)


def test_router_ties_go_to_the_lower_index(gpu):
    """bf16 logits from a few values and a zero bias: most keys are equal."""
    rng = np.random.default_rng(6)
    x = torch.from_numpy(rng.integers(-2, 3, (200, 96)).astype(np.float32)).bfloat16()
    check_router(x, 8, None, None, score="softmax")
    check_router(x, 8, torch.zeros(96), None, score="sigmoid")
    check_router(x, 8, torch.zeros(96), None, score="sigmoid", groups=8, topk_groups=3,
                 group_top=2)


def test_router_keys_closer_than_32_bits(gpu):
    """Biases that make two experts' keys differ by less than fp32 resolves:
    the choice is the one of 64 bits."""
    rng = np.random.default_rng(8)
    x = rand(rng, (256, 16), torch.float32)
    s = 1.0 / (1.0 + np.exp(-x.double().numpy()))
    # the bias that makes experts 0 and 1 meet at token 0's scores, to fp32
    bias = torch.zeros(16)
    bias[0] = 4.0
    for t in range(256):
        x[t, 1] = x[t, 0] + float(rng.integers(-2, 3)) * 2.0 ** -23
    bias[1] = 4.0
    assert s.shape == (256, 16)
    check_router(x, 2, bias, None, score="sigmoid")
    check_router(x, 2, bias, None, score="softmax", renormalize=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,group_top", [(1, 1), (8, 1), (8, 2), (64, 2)])
@pytest.mark.parametrize("spread", [2.0 ** -21, 2.0 ** -14, 0.5])
def test_router_scores_close_together(gpu, score, groups, group_top, spread):
    """Logits that differ by a few to many steps of fp32, with a bias of the
    scores' size: the order of 64 bits among experts and among groups."""
    rng = np.random.default_rng(15)
    x = rand(rng, (300, 128), torch.float32, spread)
    bias = rand(rng, (128,), torch.float32, spread / 128)
    check_router(x, 5, bias, None, score=score, groups=groups,
                 topk_groups=max(1, 3 * groups // 8), group_top=group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [2, 8, 13])
def test_router_group_values_that_cancel(gpu, score, size):
    """A group's two keys of opposite signs and nearly the same magnitude: in
    fp32 their sum is off by steps of the keys, not of the sum."""
    rng = np.random.default_rng(16)
    x = rand(rng, (200, 8 * size), torch.float32, 2.0 ** -10)
    bias = torch.full((8 * size,), -2000.0)
    bias[::size], bias[size - 1::size] = 1000.0, -1000.0
    check_router(x, 4, bias, None, score=score, groups=8, topk_groups=4, group_top=2)


@pytest.mark.parametrize("tokens", [None, 12001])
@pytest.mark.parametrize("groups,group_top", [(1, 1), (1, 2), (4, 1), (4, 2)])
@pytest.mark.parametrize("E", [128, 256, 1024])
def test_router_more_equal_keys_than_lanes(gpu, E, groups, group_top, tokens):
    """More experts with one and the same key of 32 bits than a wave has lanes:
    the largest in 64 bits is chosen, wherever it stands."""
    at = (E - 1, E // 2 + 40, 3 * E // 4)
    kw = dict(groups=groups, topk_groups=max(1, groups - 1), group_top=group_top)
    # 1 / (1 + e^-30) and e^-31 are both 1 in fp32, 6e-14 apart
    x = torch.full((4, E), 30.0)
    x[torch.arange(3), torch.tensor(at)] = 31.0
    check_router(x, 8, torch.zeros(E), None, tokens=tokens, score="sigmoid", **kw)
    # a bias of 2^20 has steps of 1 / 8, the scores differ by 1 / E at most
    x = torch.zeros((4, E))
    x[torch.arange(3), torch.tensor(at)] = 1.0
    x[0, 5], x[1, 64:] = 0.5, -1.0
    bias = torch.full((E,), 2.0 ** 20)
    check_router(x, 8, bias, None, tokens=tokens, score="softmax", **kw)
    check_router(x.bfloat16(), 3, bias, None, tokens=tokens, score="sigmoid", **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [128, 300])
def test_router_last_of_64_places(gpu, E, score):
    """The last of 64 places goes to the larger of two experts that only 64
    bits tell apart; with one place less, to the lower of two equal ones."""
    x = torch.zeros((3, E))
    bias = torch.full((E,), -10.0)
    bias[:63] = 5000.0 - 10.0 * torch.arange(63)
    bias[100] = bias[E - 3] = 1024.0             # steps of 2^-13
    x[0, 100], x[0, E - 3] = 30.0, 31.0
    x[1, 100], x[1, E - 3] = 2.0 ** -20, 2.0 ** -19
    if score == "softmax":
        x *= 2.0 ** -8
    check_router(x, 64, bias, None, score=score)
    check_router(x, 63, bias, None, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_router_special_biases(gpu, score, groups):
    """Infinite, NaN and large biases (the score drowns in them, in 64 bits
    too: ties by the index)."""
    rng = np.random.default_rng(14)
    x = rand(rng, (40, 64), torch.float32, 2.0)
    x[3, ::3] = -np.inf
    bias = rand(rng, (64,), torch.float32, 0.1)
    for i, v in enumerate((np.inf, -np.inf, np.nan, 1e30, 1e30, -1e30, 1e9, 1e9, 3e38)):
        bias[7 * i % 64] = v
    with np.errstate(invalid="ignore"):
        check_router(x, 7, bias, None, score=score, groups=groups,
                     topk_groups=min(3, groups), group_top=2)
        check_router(x, 64, bias, None, score=score)


def test_router_gradient_of_repeated_and_foreign_ids(gpu):
    """Ids the forward call never returns: repeated ones add up, ids outside
    the experts and masked experts contribute nothing."""
    rng = np.random.default_rng(9)
    x = rand(rng, (4, 10), torch.float32)
    x[2, 5] = -np.inf
    ids = np.array([[3, 3, 3], [-1, 10, 4], [5, 2, 2], [-7, 2 ** 30, -1]])
    gw = rng.normal(size=(4, 3)).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            r = moe.Router(4, 10, 3, score=score, renormalize=renorm)
            gx = marked((4, 10), torch.float32)
            moe.router_topk_backward(r, x.cuda(), torch.from_numpy(ids).int().cuda(),
                                     torch.from_numpy(gw).cuda(), gx)
            g, mag = B.router_topk_grad(f64(x), ids, gw, score, renorm)
            close(gx, g, mag, 4 * REL_EXP, f"{score} {renorm}")


def test_router_unaligned(gpu):
    rng = np.random.default_rng(10)
    x = shifted(rand(rng, (21, 128), torch.bfloat16))
    r = moe.Router(21, 128, 4, dtype=torch.bfloat16)
    ids, w = marked((21, 4), torch.int32), marked((21, 4), torch.float32)
    moe.router_topk(r, x, ids, w)
    want, ww = B.router_topk(f64(x), 4, "softmax")
    assert np.array_equal(ids.cpu().numpy(), want)
    close(w, ww, np.abs(ww), REL_EXP, "weights")
    gx = shifted(marked((21, 128), torch.bfloat16))
    gw = torch.ones((21, 4), device="cuda")
    gw[:, 0] = -1
    moe.router_topk_backward(r, x, ids, gw, gx)
    g, mag = B.router_topk_grad(f64(x), want, f64(gw), "softmax")
    close(gx, g, mag, 2 * REL_EXP, "grad")


# ---- sorted rows ----------------------------------------------------------------

ROWS = [
    # T, E, k, H
    (1, 1, 1, 1), (1, 8, 2, 7), (3, 4, 4, 33), (64, 256, 8, 512), (129, 60, 6, 1001),
    (700, 16, 3, 264), (1300, 1024, 8, 40), (2100, 5, 2, 9), (17, 8, 9, 2056), (9, 4, 20, 4100),
    (6, 3, 2, 32768), (1025, 128, 4, 64),
]


def make_ids(rng, T, E, k):
    ids = rng.integers(-1, E + 1, (T, k)).astype(np.int32)
    if T > 2:
        ids[1] = ids[1, 0]                   # one expert in every slot
        ids[2] = -1                          # an unrouted token
        ids[0, 0] = 2 ** 31 - 1
    pad = (rng.random(T) < 0.1).astype(np.uint8)
    return ids, pad


def run_permute(p, x, ids, pad):
    out = moe.alloc_permute_outputs(p)
    for t in (out["rows"], out["row_slot"], out["slot_row"], out["expert_offsets"], out["ws"]):
        t.view(torch.uint8).fill_(MARK) if t.numel() else None
    moe.permute(p, x, ids, is_padding=pad, **out)
    return out


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("T,E,k,H", ROWS)
def test_permute(gpu, T, E, k, H, dtype):
    rng = np.random.default_rng(T + H)
    ids, pad = make_ids(rng, T, E, k)
    x = rand(rng, (T, H), dtype)
    p = moe.ExpertRows(T, H, E, k, dtype=dtype)
    out = run_permute(p, x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(pad).cuda())
    off, slot_row, row_slot = B.sort_slots(ids, E, pad)
    R = len(row_slot)
    assert np.array_equal(out["expert_offsets"].cpu().numpy(), off)
    assert np.array_equal(out["slot_row"].cpu().numpy(), slot_row)
    assert np.array_equal(out["row_slot"][:R].cpu().numpy(), row_slot)
    assert torch.equal(out["rows"][:R].cpu(), x[torch.from_numpy(row_slot // k)])
    # behind the last routed row nothing was written
    assert (out["rows"][R:].contiguous().view(torch.uint8) == MARK).all()
    assert (out["row_slot"][R:].contiguous().view(torch.uint8) == MARK).all()
    # the gradient: unrouted rows hold NaN and are not read
    g = rand(rng, (T * k, H), dtype)
    g[R:] = np.nan
    gx = marked((T, H), dtype)
    moe.permute_backward(p, g.cuda(), out["slot_row"], gx)
    want, mag = B.combine(np.nan_to_num(f64(g)), slot_row)
    close(gx, want, mag, k * U, "grad_x")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("T,E,k,H", ROWS)
def test_unpermute(gpu, T, E, k, H, dtype):
    rng = np.random.default_rng(T * 3 + H)
    ids, pad = make_ids(rng, T, E, k)
    _, slot_row, row_slot = B.sort_slots(ids, E, pad)
    R = len(row_slot)
    rows = rand(rng, (T * k, H), dtype)
    rows[R:] = np.nan
    w = torch.from_numpy(rng.normal(size=(T, k)).astype(np.float32))
    w[torch.from_numpy(slot_row < 0)] = np.nan          # weights of unrouted slots
    sr = torch.from_numpy(slot_row).int()
    far = sr.clone()
    far[sr < 0] = T * k                                  # also unrouted
    p = moe.ExpertRows(T, H, E, k, dtype=dtype)
    clean = np.nan_to_num(f64(rows))
    for weights in (w, None):
        for s in (sr, far):
            out = marked((T, H), dtype)
            moe.unpermute(p, rows.cuda(), s.cuda(), None if weights is None else w.cuda(), out)
            want, mag = B.combine(clean, slot_row, None if weights is None else f64(w))
            close(out, want, mag, k * U, "out")
            g = rand(rng, (T, H), dtype)
            gr, gw = marked((T * k, H), dtype), marked((T, k), torch.float32)
            moe.unpermute_backward(p, g.cuda(), rows.cuda(), s.cuda(),
                                   None if weights is None else w.cuda(), gr, gw)
            want_r, want_w, mag_w = B.combine_grad(f64(g), clean, slot_row,
                                                   None if weights is None else f64(w))
            assert sorted(want_r) == list(range(R))
            if R:
                value = np.stack([want_r[r] for r in range(R)])
                close(gr[:R], value, np.abs(value), U, "grad_rows")
            assert (gr[R:].contiguous().view(torch.uint8) == MARK).all()
            # a lane adds at most H / 64 products (128 columns in flight), then 10 steps
            close(gw, want_w, mag_w, (H / 64 + 24) * U, "grad_weights")


def test_unpermute_backward_in_place(gpu):
    rng = np.random.default_rng(2)
    T, E, k, H = 50, 8, 3, 136
    ids, pad = make_ids(rng, T, E, k)
    _, slot_row, _ = B.sort_slots(ids, E, pad)
    sr = torch.from_numpy(slot_row).int().cuda()
    rows, g = rand(rng, (T * k, H), torch.bfloat16).cuda(), rand(rng, (T, H), torch.bfloat16).cuda()
    w = torch.rand((T, k), device="cuda")
    p = moe.ExpertRows(T, H, E, k)
    gr, gw, gw2 = rows.clone(), torch.zeros_like(w), torch.zeros_like(w)
    moe.unpermute_backward(p, g, rows, sr, w, gr, gw)
    moe.unpermute_backward(p, g, rows, sr, w, rows, gw2)
    assert torch.equal(gr, rows) and torch.equal(gw, gw2)


@pytest.mark.parametrize("dtype,H", [(torch.bfloat16, 2049), (torch.bfloat16, 2563),
                                     (torch.float16, 4103), (torch.bfloat16, 4101),
                                     (torch.float32, 1025), (torch.float32, 1283)])
def test_unpermute_backward_in_place_of_ragged_rows(gpu, dtype, H):
    """A row's last, partial vector is another wave's, or the next turn's: it
    must not write columns that the vector before it still reads."""
    rng = np.random.default_rng(H)
    T, E, k = 700, 8, 9
    ids, pad = make_ids(rng, T, E, k)
    _, slot_row, _ = B.sort_slots(ids, E, pad)
    sr = torch.from_numpy(slot_row).int().cuda()
    rows, g = rand(rng, (T * k, H), dtype).cuda(), rand(rng, (T, H), dtype).cuda()
    w = torch.rand((T, k), device="cuda")
    p = moe.ExpertRows(T, H, E, k, dtype=dtype)
    gr, gw, gw2 = rows.clone(), torch.zeros_like(w), torch.zeros_like(w)
    moe.unpermute_backward(p, g, rows, sr, w, gr, gw)
    moe.unpermute_backward(p, g, rows, sr, w, rows, gw2)
    assert torch.equal(gr, rows) and torch.equal(gw, gw2)


def test_rows_unaligned(gpu):
    rng = np.random.default_rng(12)
    T, E, k, H = 40, 8, 2, 264
    ids, pad = make_ids(rng, T, E, k)
    off, slot_row, row_slot = B.sort_slots(ids, E, pad)
    p = moe.ExpertRows(T, H, E, k)
    x = shifted(rand(rng, (T, H), torch.bfloat16))
    out = moe.alloc_permute_outputs(p)
    out["rows"] = shifted(out["rows"])
    moe.permute(p, x, torch.from_numpy(ids).cuda(), is_padding=torch.from_numpy(pad).cuda(), **out)
    assert torch.equal(out["rows"][:off[-1]].cpu(), x.cpu()[torch.from_numpy(row_slot // k)])
    w = torch.rand((T, k), device="cuda")
    y = shifted(marked((T, H), torch.bfloat16))
    moe.unpermute(p, out["rows"], out["slot_row"], w, y)
    rows = np.zeros((T * k, H))
    rows[:off[-1]] = f64(out["rows"][:off[-1]])
    want, mag = B.combine(rows, slot_row, f64(w))
    close(y, want, mag, k * U, "out")
    gr, gw = shifted(marked((T * k, H), torch.bfloat16)), marked((T, k), torch.float32)
    moe.unpermute_backward(p, x, out["rows"], out["slot_row"], w, gr, gw)
    want_r, want_w, mag_w = B.combine_grad(f64(x), rows, slot_row, f64(w))
    value = np.stack([want_r[r] for r in range(off[-1])])
    close(gr[:off[-1]], value, np.abs(value), U, "grad_rows")
    close(gw, want_w, mag_w, (H / 64 + 24) * U, "grad_weights")


@pytest.mark.parametrize("T,E,k", [(2000, 400, 2), (30000, 300, 3), (9000, 1024, 8),
                                   (70000, 7, 1), (700, 33, 3), (683, 256, 3)])
def test_sort_of_many_slots(gpu, T, E, k):
    """Every way the sort takes, by its number of slots and experts, against a
    stable sort."""
    rng = np.random.default_rng(T)
    ids, pad = make_ids(rng, T, E, k)
    p = moe.ExpertRows(T, 8, E, k, dtype=torch.float32)
    x = rand(rng, (T, 8), torch.float32)
    out = run_permute(p, x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(pad).cuda())
    e = np.where((ids < 0) | (ids >= E) | (pad[:, None] != 0), E, ids).reshape(-1)
    order = np.argsort(e, kind="stable")
    off = np.searchsorted(e[order], np.arange(E + 1))
    R = off[E]
    slot_row = np.full(T * k, -1)
    slot_row[order[:R]] = np.arange(R)
    assert np.array_equal(out["expert_offsets"].cpu().numpy(), off)
    assert np.array_equal(out["slot_row"].cpu().numpy().reshape(-1), slot_row)
    assert np.array_equal(out["row_slot"][:R].cpu().numpy(), order[:R])
    assert torch.equal(out["rows"][:R].cpu(), x[torch.from_numpy(order[:R] // k)])


def test_sort_of_no_tokens(gpu):
    p = moe.ExpertRows(0, 64, 9, 4)
    out = run_permute(p, torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"),
                      torch.empty((0, 4), dtype=torch.int32, device="cuda"), None)
    assert out["expert_offsets"].tolist() == [0] * 10


def test_sort_agrees_with_stage(gpu):
    """The rows' order is moe_stage's contiguous one."""
    T, E, k, H = 333, 24, 4, 256
    g = torch.Generator().manual_seed(3)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32).cuda()
    x = torch.randn((T, H), generator=g).bfloat16().cuda()
    pad = (torch.rand(T, generator=g) < 0.1).to(torch.uint8).cuda()
    prob = moe.Problem(T, H, 128, E, k)
    bufs = moe.alloc_stage_outputs(prob)
    moe.stage(prob, x, ids, torch.ones((T, k), device="cuda"), bufs, is_padding=pad)
    out = run_permute(moe.ExpertRows(T, H, E, k), x, ids, pad)
    R = int(out["expert_offsets"][-1])
    assert torch.equal(out["expert_offsets"], bufs["expert_offsets"])
    assert torch.equal(out["slot_row"].view(-1), bufs["slot_row"])
    assert torch.equal(out["row_slot"][:R] // k, bufs["row_src"][:R])


def test_unpermute_agrees_with_topk_reduce(gpu):
    T, E, k, H = 100, 8, 2, 512
    g = torch.Generator().manual_seed(4)
    sr = torch.randperm(T * k, generator=g).view(T, k).int()
    sr[5, 1] = -1
    down = torch.randn((T * k, H), generator=g).bfloat16().cuda()
    w = torch.rand((T, k), generator=g).cuda()
    a, b = (torch.empty((T, H), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    moe.topk_reduce(moe.Problem(T, H, 128, E, k), down, sr.cuda(), w, a)
    moe.unpermute(moe.ExpertRows(T, H, E, k), down, sr.cuda(), w, b)
    assert torch.equal(a, b)


def test_rows_past_four_gib(gpu):
    """Row offsets that pass 32 bits: 4.9 GiB of rows, checked at both ends."""
    T, E, k, H = 80000, 4, 4, 8200
    ids = torch.arange(T * k, dtype=torch.int32, device="cuda").view(T, k) % E
    x = torch.randn((T, H), device="cuda", dtype=torch.bfloat16)
    p = moe.ExpertRows(T, H, E, k)
    out = moe.alloc_permute_outputs(p)
    moe.permute(p, x, ids, **out)
    assert out["rows"].numel() * 2 > 1 << 32
    for e in range(E):
        for a in (0, T // 2, T - 1):
            assert torch.equal(out["rows"][e * T + a], x[a]), (e, a)
    y = torch.empty_like(x)
    moe.unpermute(p, out["rows"], out["slot_row"], torch.full((T, k), 0.25, device="cuda"), y)
    assert torch.equal(x, y)
    gw = torch.empty((T, k), device="cuda")
    moe.unpermute_backward(p, x, out["rows"], out["slot_row"],
                           torch.ones((T, k), device="cuda"), out["rows"], gw)
    at = torch.tensor([0, 1, T // 2, T - 1], device="cuda")
    assert torch.equal(out["rows"][3 * T + at], x[at])
    want = x[at].double().square().sum(1, keepdim=True).expand(4, k)
    assert ((gw[at].double() - want).abs() <= want * (H / 64 + 24) * U).all()


def test_more_tokens_than_a_grid_dimension_holds(gpu):
    """64 lanes per token and 2^26 tokens: 2^32 lanes."""
    T, H, E = (1 << 26) + 5, 8, 2
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn((T, E), generator=g, device="cuda", dtype=torch.bfloat16)
    ids = torch.empty((T, 1), dtype=torch.int32, device="cuda")
    w = torch.empty((T, 1), device="cuda")
    r = moe.Router(T, E, 1, dtype=torch.bfloat16)
    moe.router_topk(r, x, ids, w)
    assert torch.equal(ids[:, 0], (x[:, 1] > x[:, 0]).int()) and (w == 1).all()
    gx = torch.full_like(x, 7)
    moe.router_topk_backward(r, x, ids, w, gx)             # of a constant weight
    assert (gx == 0).all()
    del gx, x
    # rows in their tokens' order, twice the token, weights of 2
    w.fill_(2.0)
    tokens = torch.randn((T, H), generator=g, device="cuda", dtype=torch.bfloat16)
    p = moe.ExpertRows(T, H, 1, 1)
    out = moe.alloc_permute_outputs(p)
    moe.permute(p, tokens, ids.zero_(), **out)
    assert torch.equal(out["rows"], tokens)
    y = torch.empty_like(tokens)
    moe.unpermute(p, out["rows"], out["slot_row"], w, y)
    assert torch.equal(y, tokens * 2)
    gw = torch.empty_like(w)
    moe.unpermute_backward(p, tokens, out["rows"], out["slot_row"], w, y.zero_(), gw)
    assert torch.equal(y, tokens * 2)
    # eight products, each exact in fp32, and seven or more additions
    want = torch.cat([(c.float() ** 2).sum(1) for c in tokens.split(1 << 24)])
    assert ((gw[:, 0] - want).abs() <= 16 * U * want).all()
    del out, gw, want, w, ids
    n = moe.BlockNorm(T, H)
    moe.block_norm(n, tokens, y)
    for c, d in zip(tokens.split(1 << 24), y.split(1 << 24)):
        f = c.float()
        f = f * torch.rsqrt((f * f).mean(1, keepdim=True) + 1e-6)
        # both within REL_NORM of the norm in 64 bits, then half a step
        assert ((d.float() - f).abs() <= (2 * REL_NORM + 2 ** -8) * f.abs()).all()


# ---- block norms ------------------------------------------------------------------

WIDTHS = [1, 5, 64, 511, 520, 1001, 2048, 3000, 4104, 7168, 8200, 16400, 32768]


def make_norm(rng, T, H, dtype, wdtype, gate, y=True, post=True):
    t = {"residual": rand(rng, (T, H), dtype, 2.0), "pre_weight": rand(rng, (H,), wdtype)}
    if y:
        t["y"] = rand(rng, (T, H), dtype)
        if post:
            t["post_weight"] = rand(rng, (H,), wdtype)
        shape = {"none": None, "token": (T,), "channel": (H,), "full": (T, H)}[gate]
        if shape:
            t["gate"] = rand(rng, shape, dtype)
    return t


def oracle_args(p, t):
    n = lambda k: None if t.get(k) is None else f64(t[k])              # noqa: E731
    return dict(y=n("y"), post_norm=p.post_norm, w_post=n("post_weight"), gate=n("gate"),
                kind=p.gate, sigmoid=p.gate_sigmoid, w_pre=n("pre_weight"),
                eps=float(np.float32(p.eps)), scale=float(np.float32(p.residual_scale)),
                offset=float(np.float32(p.weight_offset)))


def check_norm(p, t, with_normed=True):
    d = {k: v.cuda() for k, v in t.items()}
    shape = (p.num_tokens, p.hidden)
    normed = marked(shape, p.dtype) if with_normed else None
    ro = marked(shape, p.dtype) if "y" in t else None
    moe.block_norm(p, normed=normed, residual_out=ro, **d)
    want = B.block_norm(f64(t["residual"]), **oracle_args(p, t))
    if ro is not None:
        close(ro, *want["residual_out"], REL_NORM, "residual_out")
    if with_normed:
        close(normed, *want["normed"], 2 * REL_NORM, "normed")
    return ro, normed


def check_norm_grad(p, t, rng, skip=()):
    T, H = p.num_tokens, p.hidden
    d = {k: v.cuda() for k, v in t.items()}
    x = d.pop("residual")
    dh = None if "grad_normed" in skip else rand(rng, (T, H), p.dtype)
    dr = None if "grad_residual_out" in skip else rand(rng, (T, H), p.dtype)
    outs = {"grad_residual": marked((T, H), p.dtype),
            "grad_pre_weight": marked((H,), torch.float32)}
    if "y" in t:
        outs["grad_y"] = marked((T, H), p.dtype)
        if p.post_norm:
            outs["grad_post_weight"] = marked((H,), torch.float32)
        if p.gate != "none":
            outs["grad_gate"] = marked(p.gate_shape,
                                       p.dtype if p.gate == "full" else torch.float32)
    for k in skip:
        outs.pop(k, None)
    moe.block_norm_backward(p, x, None if dh is None else dh.cuda(),
                            grad_residual_out=None if dr is None else dr.cuda(), **d, **outs)
    want = B.block_norm_grad(f64(x), None if dh is None else f64(dh),
                             None if dr is None else f64(dr), **oracle_args(p, t))
    for k, got in outs.items():
        value, mag = want[k]
        n = T if k in ("grad_pre_weight", "grad_post_weight") or (
            k == "grad_gate" and p.gate == "channel") else 64
        close(got, value, mag, REL_GRAD + n * U, k)
    return outs


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("H", WIDTHS)
def test_block_norm(gpu, H, dtype):
    """Every width class, with each kind of gate at one of them."""
    rng = np.random.default_rng(H)
    for i, gate in enumerate(("none", "token", "channel", "full")):
        T = (1, 3, 6, 13)[(i + H) % 4]
        p = moe.BlockNorm(T, H, dtype=dtype, weight_dtype=(dtype, torch.float32)[i & 1],
                          post_norm=i != 1, gate=gate, gate_sigmoid=(i + H) % 3 == 0, eps=1e-5,
                          residual_scale=0.37, weight_offset=float(i & 1))
        t = make_norm(rng, T, H, dtype, p.weight_dtype, gate, post=p.post_norm)
        check_norm(p, t, with_normed=i != 2)
        check_norm_grad(p, t, rng)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("T,H", [(1, 96), (700, 40), (2100, 200), (1030, 4096), (600, 7168),
                                 (530, 1800), (514, 12000)])
def test_block_norm_many_rows(gpu, T, H, dtype):
    """More rows than blocks: every block walks several."""
    rng = np.random.default_rng(T)
    p = moe.BlockNorm(T, H, dtype=dtype, weight_dtype=torch.float32, post_norm=True,
                      gate="channel", residual_scale=0.5)
    t = make_norm(rng, T, H, dtype, torch.float32, "channel")
    check_norm(p, t)
    a = check_norm_grad(p, t, rng)
    rng2 = np.random.default_rng(T)
    make_norm(rng2, T, H, dtype, torch.float32, "channel")
    b = check_norm_grad(p, t, rng2)
    for k in a:                              # the same bits every time
        assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("H", [1300, 2600, 4700, 6000, 7000, 8001])
def test_block_norm_many_rows_of_every_shape(gpu, H, dtype):
    rng = np.random.default_rng(H)
    gate = "channel" if H % 8 else "token"
    p = moe.BlockNorm(515, H, dtype=dtype, weight_dtype=torch.float32, post_norm=True, gate=gate)
    check_norm(p, make_norm(rng, 515, H, dtype, torch.float32, gate))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("H", [7, 264, 5000])
def test_norm_without_a_block(gpu, H, dtype):
    rng = np.random.default_rng(H)
    p = moe.BlockNorm(11, H, dtype=dtype, post_norm=True, gate="token", weight_offset=1.0)
    t = make_norm(rng, 11, H, dtype, dtype, "none", y=False)
    check_norm(p, t)
    check_norm_grad(p, t, rng, skip=("grad_residual_out",))
    check_norm_grad(p, t, rng, skip=("grad_pre_weight",))


@pytest.mark.parametrize("skip", [("grad_normed",), ("grad_residual_out",),
                                  ("grad_pre_weight", "grad_post_weight", "grad_gate"),
                                  ("grad_post_weight",), ("grad_pre_weight", "grad_gate")])
@pytest.mark.parametrize("gate", ["token", "channel", "full"])
def test_norm_optional_gradients(gpu, gate, skip):
    rng = np.random.default_rng(5)
    p = moe.BlockNorm(40, 272, post_norm=True, gate=gate, gate_sigmoid=True)
    check_norm_grad(p, make_norm(rng, 40, 272, torch.bfloat16, torch.bfloat16, gate), rng, skip)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("H", [5, 200, 2056, 9000])
@pytest.mark.parametrize("gate", ["token", "channel", "full"])
def test_norm_saturated_gates(gpu, gate, H, dtype):
    """Gates whose sigmoid is next to 0 or 1: their gradient is its slope s (1 -
    s), 2e-9 at 20, where fp32 has no step between s and 1."""
    rng = np.random.default_rng(H)
    T = 17
    p = moe.BlockNorm(T, H, dtype=dtype, weight_dtype=torch.float32, post_norm=True, gate=gate,
                      gate_sigmoid=True, residual_scale=0.7)
    t = make_norm(rng, T, H, dtype, torch.float32, gate)
    at = torch.arange(t["gate"].numel()) % 7
    t["gate"] = torch.tensor([12.0, -12.0, 20.0, -20.0, 0.0, 17.0, 3.5])[at].view(
        t["gate"].shape).to(dtype)
    check_norm(p, t)
    check_norm_grad(p, t, rng)
    check_norm_grad(p, t, rng, skip=("grad_normed", "grad_post_weight"))


def test_norm_without_weights(gpu):
    rng = np.random.default_rng(6)
    p = moe.BlockNorm(9, 300, post_norm=True, weight_offset=1.0)
    t = make_norm(rng, 9, 300, torch.bfloat16, torch.bfloat16, "none")
    del t["pre_weight"], t["post_weight"]
    check_norm(p, t)
    check_norm_grad(p, t, rng)


def test_norm_zero_rows_and_large_values(gpu):
    """Rows of zeros (eps alone holds the quotient), rows up to 1e18 and down
    to 1e-18, whose squares fp32 still holds or flushes below eps."""
    rng = np.random.default_rng(7)
    p = moe.BlockNorm(6, 128, dtype=torch.float32, post_norm=True)
    t = make_norm(rng, 6, 128, torch.float32, torch.float32, "none")
    for i, s in enumerate((0.0, 1e18, 1e-18, 1.0, 0.0, 1e15)):
        t["residual"][i] *= s
        t["y"][i] *= (1.0, 1.0, 0.0, 1e18, 0.0, 1e-18)[i]
    check_norm(p, t)
    check_norm_grad(p, t, rng)


@pytest.mark.parametrize("block", [True, False])
@pytest.mark.parametrize("dtype,T,H", [
    (torch.float32, 2100, 128), (torch.float32, 2100, 400), (torch.float32, 700, 900),
    (torch.float32, 530, 2000), (torch.float32, 530, 4000), (torch.float32, 270, 8000),
    (torch.float32, 270, 9000), (torch.float32, 40, 1500), (torch.bfloat16, 1100, 1030),
    (torch.bfloat16, 530, 7168), (torch.bfloat16, 270, 12001), (torch.bfloat16, 40, 32768)])
def test_norm_large_rows_among_others(gpu, dtype, T, H, block):
    """Rows whose squares pass fp32's range beside rows that a block, or lanes
    side by side in one, take with them or next: in every shape a row can have,
    with several rows per block."""
    rng = np.random.default_rng(H)
    gate = "channel" if block else "none"
    p = moe.BlockNorm(T, H, dtype=dtype, weight_dtype=torch.float32, post_norm=True, gate=gate)
    t = make_norm(rng, T, H, dtype, torch.float32, gate, y=block)
    size = torch.ones((2, T, 1))
    size[0, T // 2::53], size[0, 3::37] = 3e30, 1e22
    size[1, 5::41], size[1, 3::74] = 1e25, 1e20
    t["residual"] = (t["residual"] * size[0]).to(dtype)
    if block:
        t["y"] = (t["y"] * size[1]).to(dtype)
    check_norm(p, t)
    check_norm_grad(p, t, rng)


def test_norm_in_place_and_unaligned(gpu):
    rng = np.random.default_rng(8)
    p = moe.BlockNorm(70, 2056, post_norm=True, gate="full")
    t = make_norm(rng, 70, 2056, torch.bfloat16, torch.bfloat16, "full")
    ro, h = check_norm(p, t)
    d = {k: shifted(v) for k, v in t.items()}
    moe.block_norm(p, normed=d["y"], residual_out=d["residual"], **d)
    assert torch.equal(d["residual"], ro) and torch.equal(d["y"], h)
    dh, dr = (rand(rng, (70, 2056), torch.bfloat16).cuda() for _ in range(2))
    c = {k: v.cuda() for k, v in t.items() if k != "residual"}
    gr, gy = torch.empty_like(dh), torch.empty_like(dh)
    gw = [torch.empty(2056, device="cuda") for _ in range(2)]
    moe.block_norm_backward(p, ro, dh, gr, grad_residual_out=dr, grad_y=gy,
                            grad_pre_weight=gw[0], **c)
    moe.block_norm_backward(p, ro, dh, dr, grad_residual_out=dr, grad_y=dh,
                            grad_pre_weight=gw[1], **c)
    assert torch.equal(gr, dr) and torch.equal(gy, dh) and torch.equal(*gw)


def test_norm_of_no_tokens(gpu):
    p = moe.BlockNorm(0, 300, post_norm=True, gate="channel")
    e = torch.empty((0, 300), dtype=torch.bfloat16, device="cuda")
    g = [marked((300,), torch.float32) for _ in range(3)]
    w = torch.ones(300, dtype=torch.bfloat16, device="cuda")
    moe.block_norm(p, e, e.clone(), y=e, residual_out=e, gate=w)
    moe.block_norm_backward(p, e, e, e.clone(), y=e, grad_y=e.clone(), gate=w, post_weight=w,
                            grad_pre_weight=g[0], grad_post_weight=g[1], grad_gate=g[2])
    for t in g:
        assert (t == 0).all()


# ---- streams, graphs, threads -------------------------------------------------------

def chain(rng, T=70, E=16, k=4, H=520):
    """Buffers and one pass of every call, forward and backward."""
    bf, f32 = torch.bfloat16, torch.float32
    pre = moe.BlockNorm(T, H)
    post = moe.BlockNorm(T, H, post_norm=True, gate="channel")
    r = moe.Router(T, E, k, score="sigmoid", num_groups=4, topk_groups=2, group_top=2)
    p = moe.ExpertRows(T, H, E, k)
    c = {n: rand(rng, s, d).cuda() for n, s, d in [
        ("x", (T, H), bf), ("wr", (E,), f32), ("w1", (H,), bf), ("w2", (H,), bf),
        ("w3", (H,), bf), ("gate", (H,), bf), ("dh", (T, H), bf), ("dr", (T, H), bf),
        ("bias", (E,), f32)]}
    o = {n: torch.empty(s, dtype=d, device="cuda") for n, s, d in [
        ("h", (T, H), bf), ("ids", (T, k), torch.int32), ("w", (T, k), f32), ("y", (T, H), bf),
        ("r2", (T, H), bf), ("h2", (T, H), bf), ("gr", (T, H), bf), ("gy", (T, H), bf),
        ("g1", (H,), f32), ("g2", (H,), f32), ("gg", (H,), f32), ("grows", (T * k, H), bf),
        ("gw", (T, k), f32), ("glogits", (T, E), f32), ("gx", (T, H), bf)]}
    o.update(moe.alloc_permute_outputs(p))
    ws = moe.alloc_block_norm_workspace(post)
    ps = o.pop("ws")
    logits = o["logits"] = torch.empty((T, E), device="cuda")
    o["rows"].zero_(), o["row_slot"].zero_(), o["grows"].zero_()

    def step():
        moe.block_norm(pre, c["x"], o["h"], pre_weight=c["w1"])
        # (no product of torch's here: its reductions clear memory in ways that a
        # captured graph does not repeat)
        torch.mul(o["h"][:, :E], c["wr"], out=logits)
        moe.router_topk(r, logits, o["ids"], o["w"], bias=c["bias"])
        moe.permute(p, o["h"], o["ids"], o["rows"], o["expert_offsets"], o["slot_row"],
                    o["row_slot"], ps)
        moe.unpermute(p, o["rows"], o["slot_row"], o["w"], o["y"])
        moe.block_norm(post, c["x"], o["h2"], y=o["y"], residual_out=o["r2"],
                       pre_weight=c["w3"], post_weight=c["w2"], gate=c["gate"])
        moe.block_norm_backward(post, o["r2"], c["dh"], o["gr"], y=o["y"],
                                grad_residual_out=c["dr"], pre_weight=c["w3"],
                                post_weight=c["w2"], gate=c["gate"], grad_y=o["gy"],
                                grad_pre_weight=o["g1"], grad_post_weight=o["g2"],
                                grad_gate=o["gg"], ws=ws)
        moe.unpermute_backward(p, o["gy"], o["rows"], o["slot_row"], o["w"], o["grows"],
                               o["gw"])
        moe.router_topk_backward(r, logits, o["ids"], o["gw"], o["glogits"])
        moe.permute_backward(p, o["grows"], o["slot_row"], o["gx"])

    return c, o, step


def snapshot(o):
    return {k: v.clone() for k, v in o.items()}


def same(a, b):
    for k in a:
        assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k


def test_graph_replays(gpu):
    """All calls captured into one graph: every replay gives the eager bits,
    with other inputs, eager work and cleared outputs in between."""
    rng = np.random.default_rng(11)
    c, o, step = chain(rng)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        c["x"].copy_(rand(rng, tuple(c["x"].shape), torch.bfloat16))
        step()
        want = snapshot(o)
        for v in o.values():
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        same(o, want)


def test_another_stream_and_threads(gpu):
    """Two host threads on streams of their own, at once, against the default
    stream's results."""
    import threading
    rng = np.random.default_rng(12)
    runs = [chain(np.random.default_rng(13 + i)) for i in range(2)]
    want = []
    for c, o, step in runs:
        step()
        want.append(snapshot(o))
    torch.cuda.synchronize()
    errors = []

    def work(i):
        try:
            c, o, step = runs[i]
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(5):
                    for v in o.values():
                        v.zero_()
                    step()
            s.synchronize()
            same(o, want[i])
        except Exception as exc:
            errors.append(repr(exc))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=100)
    assert not errors, errors
    assert rng is not None


def test_chain_of_gradients_against_autograd(gpu):
    """The calls of a block run together, forward and backward, as a training
    step does, against torch's differentiation of the same block in 64 bits
    (float32 data; the experts scale their rows)."""
    torch.manual_seed(5)
    T, E, k, H = 37, 12, 3, 72
    f, dev = torch.float32, "cuda"
    pre = moe.BlockNorm(T, H, dtype=f)
    post = moe.BlockNorm(T, H, dtype=f, post_norm=True, gate="token", gate_sigmoid=True,
                         residual_scale=0.5)
    r = moe.Router(T, E, k, score="sigmoid", renormalize=True, scale=1.5)
    p = moe.ExpertRows(T, H, E, k, dtype=f)
    x, w1, w2, w3 = torch.randn(T, H), torch.randn(H), torch.randn(H), torch.randn(H)
    wr, gate, scale = torch.randn(H, E) / 8, torch.randn(T), torch.randn(E)
    dh, dr = torch.randn(T, H), torch.randn(T, H)
    a = {n: t.to(dev) for n, t in dict(x=x, w1=w1, w2=w2, w3=w3, wr=wr, gate=gate, scale=scale,
                                       dh=dh, dr=dr).items()}
    e = lambda *s: torch.empty(s, device=dev)                           # noqa: E731
    h, y, r2, h2 = e(T, H), e(T, H), e(T, H), e(T, H)
    ids, w = torch.empty((T, k), dtype=torch.int32, device=dev), e(T, k)
    moe.block_norm(pre, a["x"], h, pre_weight=a["w1"])
    logits = h @ a["wr"]
    moe.router_topk(r, logits, ids, w)
    out = moe.alloc_permute_outputs(p)
    moe.permute(p, h, ids, **out)
    expert = torch.repeat_interleave(torch.arange(E, device=dev),
                                     out["expert_offsets"].diff().long())
    rows = out["rows"] * a["scale"][expert][:, None]
    moe.unpermute(p, rows, out["slot_row"], w, y)
    moe.block_norm(post, a["x"], h2, y=y, residual_out=r2, pre_weight=a["w3"],
                   post_weight=a["w2"], gate=a["gate"])
    # backward
    g = {n: e(H) for n in ("w1", "w2", "w3")}
    g["gate"], gr, gy = e(T), e(T, H), e(T, H)
    moe.block_norm_backward(post, r2, a["dh"], gr, y=y, grad_residual_out=a["dr"],
                            pre_weight=a["w3"], post_weight=a["w2"], gate=a["gate"], grad_y=gy,
                            grad_pre_weight=g["w3"], grad_post_weight=g["w2"],
                            grad_gate=g["gate"])
    grows, gw, glog, gh, gx = e(T * k, H), e(T, k), e(T, E), e(T, H), e(T, H)
    moe.unpermute_backward(p, gy, rows, out["slot_row"], w, grows, gw)
    g["scale"] = torch.zeros(E, device=dev).index_add_(0, expert, (grows * out["rows"]).sum(1))
    moe.router_topk_backward(r, logits, ids, gw, glog)
    g["wr"] = h.t() @ glog
    moe.permute_backward(p, grows * a["scale"][expert][:, None], out["slot_row"], gh)
    moe.block_norm_backward(pre, a["x"], gh + glog @ a["wr"].t(), gx, grad_residual_out=gr,
                            pre_weight=a["w1"], grad_pre_weight=g["w1"])
    g["x"] = gx

    d = {n: t.double().requires_grad_() for n, t in dict(
        x=x, w1=w1, w2=w2, w3=w3, wr=wr, gate=gate, scale=scale).items()}
    norm = lambda v: v / (v.square().mean(1, keepdim=True) + float(np.float32(1e-6))).sqrt()  # noqa: E731,E501
    hd = norm(d["x"]) * d["w1"]
    s = torch.sigmoid(hd @ d["wr"]).gather(1, ids.cpu().long())
    wd = 1.5 * s / (s.sum(1, keepdim=True) + 1e-20)
    yd = (wd[:, :, None] * d["scale"][ids.cpu().long()][:, :, None] * hd[:, None, :]).sum(1)
    r2d = d["x"] + 0.5 * torch.sigmoid(d["gate"])[:, None] * norm(yd) * d["w2"]
    loss = (norm(r2d) * d["w3"] * dh.double()).sum() + (r2d * dr.double()).sum()
    loss.backward()
    # A chain of eight fp32 steps over sums of up to 72 terms, each off by at
    # most 2^-24 of its terms' absolute sum: 8 * 72 * 2^-24 of the result's norm
    # where terms do not cancel.  They do on the way to the experts' scales and
    # the router: every row of a token is a multiple of its h, so y is one too,
    # the post norm takes the factor out again, and dL/dw = <grad_y, row> is 0
    # but for eps: grad_y is orthogonal to y, hence to the row.  What these two
    # sums are off by is therefore relative to their terms' absolute values,
    # sum |grad_y row|, carried on linearly: |dlogits| by the router's own
    # magnitudes, then |h|^T of it for the router's matrix.
    mag = {n: float(t.grad.norm()) for n, t in d.items()}
    terms = (grows * out["rows"]).abs().sum(1)
    mag["scale"] = float(torch.zeros(E, device=dev).index_add_(0, expert, terms).norm())
    gw_terms = torch.zeros((T, k), device=dev)
    moe.unpermute_backward(p, gy.abs(), rows.abs(), out["slot_row"], w, torch.empty_like(rows),
                           gw_terms)
    m = B.router_topk_grad(f64(logits), ids.cpu().numpy(), f64(gw_terms), "sigmoid", True, 1.5)[1]
    mag["wr"] = float(np.linalg.norm(np.abs(f64(h)).T @ m))
    for n, t in d.items():
        err = float((g[n].cpu().double() - t.grad).norm())
        assert err <= 8 * 72 * U * mag[n], (n, err, mag[n])


# ---- a block around the layer ---------------------------------------------------------

def make_block(T=40, layout=moe.LAYOUT_CONTIGUOUS, post=True, gate="token"):
    import moe_synth
    cfg = moe_synth.custom(name="block", T=T, E=8, top_k=2, K=256, N=256, seed=91)
    inp = moe_synth.make_inputs(cfg, "cuda")
    p = moe.Problem(T, 256, 256, 8, 2, layout)
    layer = moe.MoeLayer(p, inp["w13"], inp["w13_sf"], inp["w2"], inp["w2_sf"])
    rng = np.random.default_rng(17)
    norm = moe.BlockNorm(T, 256, weight_dtype=torch.float32, post_norm=post, gate=gate,
                         gate_sigmoid=True, residual_scale=0.4)
    w = {n: rand(rng, (256,), torch.float32).cuda() for n in ("pre", "post", "next")}
    block = moe.MoeBlock(layer, moe.Router(T, 8, 2, score="sigmoid", scale=2.0),
                         rand(rng, (8, 256), torch.float32, 0.1).cuda(), norm, w["pre"],
                         w["post"] if post else None, rand(rng, (8,), torch.float32, 0.1).cuda())
    x = rand(rng, (T, 256), torch.bfloat16, 2.0).cuda()
    g = rand(rng, (T,), torch.bfloat16).cuda()
    pad = torch.from_numpy((rng.random(T) < 0.1).astype(np.uint8)).cuda()
    return block, layer, norm, w, x, g, pad


@pytest.mark.parametrize("layout", [moe.LAYOUT_CONTIGUOUS, moe.LAYOUT_INDEXED])
def test_block_runs_its_steps(gpu, layout):
    """Every step's result inside the block against the oracle (the layer
    itself against its own direct call, bit for bit)."""
    block, layer, norm, w, x, g, pad = make_block(layout=layout)
    nxt = torch.empty_like(x)
    out = block(x, gate=g, is_padding=pad, next_normed=nxt, next_weight=w["next"])
    h = B.block_norm(f64(x), w_pre=f64(w["pre"]), eps=float(np.float32(1e-6)))["normed"]
    close(block.hidden, *h, 2 * REL_NORM, "hidden")
    logits = torch.matmul(block.hidden.float(), block.router_weight.t())
    ids, wt = B.router_topk(f64(logits), 2, "sigmoid", bias=f64(block.bias), scale=2.0,
                            pad=pad.cpu().numpy())
    assert np.array_equal(block.topk_ids.cpu().numpy(), ids)
    close(block.topk_weights, wt, np.abs(wt), REL_EXP, "weights")
    y = layer(block.hidden, block.topk_ids, block.topk_weights, is_padding=pad)
    assert torch.equal(y, block.y)
    assert (block.y[pad.bool()] == 0).all() and block.y.abs().sum() > 0
    want = B.block_norm(f64(x), f64(y), True, f64(w["post"]), f64(g), "token", True,
                        f64(w["next"]), float(np.float32(1e-6)), float(np.float32(0.4)))
    close(out, *want["residual_out"], REL_NORM, "residual_out")
    close(nxt, *want["normed"], 2 * REL_NORM, "next_normed")
    # the norm that the block before left, and the stream updated in place
    again = x.clone()
    assert block(again, normed=block.hidden.clone(), gate=g, is_padding=pad,
                 residual_out=again) is again
    assert torch.equal(again, out)


def test_block_in_a_graph(gpu):
    """Router and norms captured with the layer between them (the logits'
    product, a library call, is made outside)."""
    block, layer, norm, w, x, g, pad = make_block()
    out = block(x, gate=g, is_padding=pad)
    logits = torch.matmul(block.hidden.float(), block.router_weight.t())
    got = torch.empty_like(x)
    torch.cuda.synchronize()

    def rest():
        moe.block_norm(block.pre, x, block.hidden, pre_weight=w["pre"])
        moe.router_topk(block.router, logits, block.topk_ids, block.topk_weights,
                        bias=block.bias, is_padding=pad)
        layer(block.hidden, block.topk_ids, block.topk_weights, out=block.y, is_padding=pad)
        moe.block_norm(norm, x, y=block.y, residual_out=got, post_weight=w["post"], gate=g)

    rest()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rest()
    for _ in range(3):
        got.zero_()
        block.y.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, out)


@pytest.mark.parametrize("layout", [moe.LAYOUT_CONTIGUOUS, moe.LAYOUT_INDEXED])
def test_block_captured_whole(gpu, layout):
    """One call, the logits' product in it: every replay gives the eager bits, of
    other inputs, with eager work and cleared buffers in between."""
    block, layer, norm, w, x, g, pad = make_block(T=200, layout=layout)
    got, nxt = torch.empty_like(x), torch.empty_like(x)

    def run():
        block(x, gate=g, is_padding=pad, residual_out=got, next_normed=nxt,
              next_weight=w["next"])

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    rng = np.random.default_rng(23)
    bufs = (got, nxt, block.hidden, block.y, block.topk_ids, block.topk_weights)
    for _ in range(4):
        x.copy_(rand(rng, tuple(x.shape), torch.bfloat16, 2.0))
        run()
        want = [t.clone() for t in bufs]
        for t in bufs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(bufs, want):
            assert torch.equal(a, b)


def test_block_of_no_tokens(gpu):
    block, layer, norm, w, x, g, pad = make_block(T=0)
    assert block(x, gate=g, is_padding=pad).shape == (0, 256)


def test_block_refusals(gpu):
    block, layer, norm, w, x, g, pad = make_block()
    r, rw = block.router, block.router_weight
    for kw, word in [(dict(router=moe.Router(41, 8, 2)), "router"),
                     (dict(router=moe.Router(40, 8, 1)), "router"),
                     (dict(norm=moe.BlockNorm(40, 128)), "norm"),
                     (dict(norm=moe.BlockNorm(40, 256, dtype=torch.float16)), "bfloat16"),
                     (dict(router_weight=rw[:7]), "router_weight"),
                     (dict(router_weight=rw.half()), "router_weight")]:
        with pytest.raises(ValueError, match=word):
            moe.MoeBlock(**{**dict(layer=layer, router=r, router_weight=rw, norm=norm), **kw})
    batched = moe.MoeLayer(moe.Problem(40, 256, 256, 8, 2, moe.LAYOUT_BATCHED, 80), layer.w13,
                           layer.w13_sf, layer.w2, layer.w2_sf)
    with pytest.raises(ValueError, match="layout"):
        moe.MoeBlock(batched, r, rw, norm)
    with pytest.raises(ValueError, match="gate"):
        block(x, gate=g[:-1])
    with pytest.raises(moe.MoeError, match="gate is NULL"):
        block(x)

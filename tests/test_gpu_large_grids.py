"""The experts' products and the staged norm in grids of more than 2^20 blocks, thin
enough to be quick: every result is there, nothing behind the last one is written."""
import pytest
import torch

import fp8_block_quantized_group_amd as moe
from expert_util import marked, untouched

pytestmark = pytest.mark.gpu
GRID = 1 << 20                             # blocks of a row of the grid


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    moe.load_library()
    yield
    torch.cuda.empty_cache()


def normal(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)


def test_weights_gradient():
    """1 050 624 blocks of tiles: 1024 experts, three with rows, against the three alone."""
    E, K, N = 1024, 257, 21825
    x, gout, pre = normal(1, 6, K), normal(2, 6, N), normal(3, 6, 2 * N)

    def gradient(experts, counts, room):
        p = moe.ExpertLinear(6, K, N, experts, dtype=torch.float32, activation="silu")
        off = torch.zeros(experts + 1, dtype=torch.int32)
        off[1:] = torch.tensor([counts.get(e, 0) for e in range(experts)]).cumsum(0)
        gw = torch.empty((experts + room, 2 * N, K), device="cuda")
        gw[experts:].view(torch.uint8).fill_(0x5A)
        moe.expert_linear_backward(p, x, None, gout, None, gw[:experts],
                                   expert_offsets=off.cuda(), pre_act=pre)
        torch.cuda.synchronize()
        return gw

    few = gradient(3, {0: 1, 1: 2, 2: 3}, 0)
    gw = gradient(E, {0: 1, 700: 2, E - 1: 3}, 3)
    for i, e in enumerate((0, 700, E - 1)):
        assert torch.equal(gw[e], few[i])
    assert untouched(gw[E:])
    for a, b in ((1, 350), (350, 700), (701, E - 1)):
        assert not gw[a:b].any()


def test_rows():
    R = (GRID + 5) * 128 + 1
    x, w = normal(1, R, 1), torch.tensor([2.0, -0.5, 4.0], device="cuda").view(1, 3, 1)
    p = moe.ExpertLinear(R, 1, 3, dtype=torch.float32)
    room = marked((R + 300, 3), torch.float32)
    moe.expert_linear(p, x, w, room[:R])
    assert torch.equal(room[:R], x * w[0].T) and untouched(room[R:])


def test_rows_gradient():
    """Of the rows, through an activation: one weight of three counts."""
    R = (GRID + 5) * 128 + 1
    gout, pre = normal(1, R, 3), normal(2, R, 3)
    w = torch.tensor([0.0, 2.0, 0.0], device="cuda").view(1, 3, 1)
    p = moe.ExpertLinear(R, 1, 3, dtype=torch.float32, activation="relu2_no_mul")
    room = marked((R + 300, 1), torch.float32)
    moe.expert_linear_backward(p, None, w, gout, room[:R], pre_act=pre)
    want = gout[:, 1] * pre[:, 1].clamp_min(0.0) * 4.0
    assert torch.equal(room[:R, 0], want) and untouched(room[R:])


def test_4_bit_rows():
    """fp16 and one code that is not the zero: the products are exact."""
    R = (GRID + 3) * 16 + 5
    x = normal(1, R, 32, dtype=torch.float16)
    codes = torch.full((1, 1, 16), 0x88, dtype=torch.uint8, device="cuda")
    codes[0, 0, 2] = 0x98                                   # column 5: 1
    scales = torch.ones((1, 1, 1), dtype=torch.float16, device="cuda")
    p = moe.ExpertLinearW4(R, 32, 1, dtype=torch.float16, group_size=32)
    room = marked((R + 300, 1), torch.float16)
    moe.expert_linear_w4(p, x, codes, scales, room[:R])
    assert torch.equal(room[:R, 0], x[:, 5]) and untouched(room[R:])


def test_norm_that_leaves_staged():
    """Rows in the second row of the grid leave what the same rows leave alone."""
    T, H, tail = 4 * GRID + 9, 128, 4 * 100 + 1
    x = normal(1, T, H, dtype=torch.bfloat16)

    def run(rows):
        n = rows.shape[0]
        q = marked((n + 8, H), torch.uint8)
        sf = marked((n + 8, 4), torch.uint8)
        moe.block_norm_quant(moe.BlockNorm(n, H), rows, q[:n], sf[:n])
        assert untouched(q[n:]) and untouched(sf[n:])
        return q[:n], sf[:n]

    q, sf = run(x)
    for rows in (slice(0, tail), slice(T - tail, T)):
        a, b = run(x[rows])
        assert torch.equal(q[rows], a) and torch.equal(sf[rows], b)


def test_as_many_rows_as_32_bits_hold():
    """Rows and a tile less one are more than 31 bits."""
    R = (1 << 31) - 1
    x = torch.empty((R, 1), dtype=torch.bfloat16, device="cuda")
    for a in range(0, R, 1 << 28):
        x[a:a + (1 << 28)].normal_()
    w = torch.full((1, 1, 1), 2.0, dtype=torch.bfloat16, device="cuda")
    out = marked((R + 300, 1), torch.bfloat16)
    moe.expert_linear(moe.ExpertLinear(R, 1, 1), x, w, out[:R])
    assert untouched(out[R:])
    for a in range(0, R, 1 << 28):
        b = min(R, a + (1 << 28))
        assert torch.equal(out[a:b], 2.0 * x[a:b])


def test_offsets_whose_tiles_pass_32_bits():
    """512 of 1024 experts with all rows each, 2^32 + 1536 tiles of 128: nothing around
    the rows is written."""
    R, E = (1 << 30) + 384, 1024
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1::2] = R
    off = off.cuda()
    x = torch.ones((R, 1), device="cuda")
    w = torch.ones((E, 1, 1), device="cuda")
    room = marked((R + 600, 1), torch.float32)
    p = moe.ExpertLinear(R, 1, 1, E, dtype=torch.float32)
    moe.expert_linear(p, x, w, room[300:R + 300], expert_offsets=off)
    torch.cuda.synchronize()
    assert untouched(room[:300]) and untouched(room[R + 300:])
    moe.expert_linear_backward(p, None, w, x, room[300:R + 300], expert_offsets=off)
    torch.cuda.synchronize()
    assert untouched(room[:300]) and untouched(room[R + 300:])

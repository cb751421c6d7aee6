"""Refusals of the calls around the layer, without a GPU: the C ABI checks
every argument before anything is enqueued (the pointers here are not
addresses of anything), the Python binding the shapes, types and devices."""
import ctypes
import os

import pytest
import torch

import fp8_block_quantized_group_amd as moe

V = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 1)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        from fp8_block_quantized_group_amd import build
        build.build()
    return moe.load_library()


def refused(lib, status, want, word):
    assert status == want, (status, lib.moe_last_error())
    assert word in lib.moe_last_error().decode(), lib.moe_last_error()


@pytest.mark.parametrize("kw,status,word", [
    (dict(num_tokens=-1), -1, "num_tokens"), (dict(num_experts=0), -2, "num_experts"),
    (dict(num_experts=1025), -2, "num_experts"), (dict(top_k=0), -1, "top_k"),
    (dict(top_k=65), -1, "top_k"), (dict(num_experts=128, top_k=65), -2, "top_k"),
    (dict(num_groups=0), -1, "num_groups"), (dict(num_groups=7), -1, "num_groups"),
    (dict(num_experts=256, num_groups=128), -1, "num_groups"),
    (dict(num_groups=8, topk_groups=0), -1, "topk_groups"),
    (dict(num_groups=8, topk_groups=9), -1, "topk_groups"),
    (dict(num_groups=32, topk_groups=3, top_k=7), -1, "top_k 7"),
    (dict(group_top=3), -1, "group_top"), (dict(scale=float("inf")), -1, "scale"),
    (dict(scale=float("nan")), -1, "scale")])
def test_router_problems(lib, kw, status, word):
    r = moe.Router(**{**dict(num_tokens=4, num_experts=64, top_k=8), **kw})
    refused(lib, lib.moe_router_topk(r._ref, V, None, None, V, V, None), status, word)
    refused(lib, lib.moe_router_topk_backward(r._ref, V, V, V, V, None), status, word)


def test_router_arguments(lib):
    r = moe.Router(4, 64, 8)
    call = lib.moe_router_topk
    refused(lib, call(None, V, None, None, V, V, None), -1, "router")
    refused(lib, call(r._ref, None, None, None, V, V, None), -1, "logits")
    refused(lib, call(r._ref, ODD, None, None, V, V, None), -1, "aligned")
    refused(lib, call(r._ref, V, ODD, None, V, V, None), -1, "bias")
    refused(lib, call(r._ref, V, None, None, None, V, None), -1, "topk_ids")
    refused(lib, call(r._ref, V, None, None, V, ODD, None), -1, "topk_weights")
    call = lib.moe_router_topk_backward
    for i, word in enumerate(("logits", "topk_ids", "grad_topk_weights", "grad_logits")):
        args = [V] * 4
        args[i] = None
        refused(lib, call(r._ref, *args, None), -1, word)
    bad = moe._Router(4, 64, 8, 5, 0, 1, 1, 1, 1, 1.0)
    refused(lib, call(ctypes.byref(bad), V, V, V, V, None), -1, "dtype")
    bad = moe._Router(4, 64, 8, 0, 2, 1, 1, 1, 1, 1.0)
    refused(lib, call(ctypes.byref(bad), V, V, V, V, None), -1, "score")
    empty = moe.Router(0, 64, 8)
    assert lib.moe_router_topk(empty._ref, None, None, None, None, None, None) == 0
    assert call(empty._ref, None, None, None, None, None) == 0


@pytest.mark.parametrize("kw,status,word", [
    (dict(num_tokens=-1), -1, "num_tokens"), (dict(hidden=0), -2, "hidden"),
    (dict(hidden=32769), -2, "hidden"), (dict(num_experts=0), -2, "num_experts"),
    (dict(num_experts=1025), -2, "num_experts"), (dict(top_k=0), -1, "top_k"),
    (dict(num_tokens=1 << 30, top_k=2), -2, "2^31"),
    (dict(num_tokens=1 << 27, top_k=1, hidden=32768), -2, "2^31")])
def test_rows_problems(lib, kw, status, word):
    p = moe.ExpertRows(**{**dict(num_tokens=4, hidden=100, num_experts=8, top_k=2), **kw})
    with pytest.raises(moe.MoeError) as e:
        moe.permute_workspace_size(p)
    assert e.value.status == status and word in str(e.value)
    refused(lib, lib.moe_permute(p._ref, V, V, None, V, V, V, V, V, 1 << 40, None), status, word)
    refused(lib, lib.moe_permute_backward(p._ref, V, V, V, None), status, word)
    refused(lib, lib.moe_unpermute(p._ref, V, V, V, V, None), status, word)
    refused(lib, lib.moe_unpermute_backward(p._ref, V, V, V, V, V, V, None), status, word)


def test_rows_arguments(lib):
    p = moe.ExpertRows(4, 100, 8, 2)
    n = moe.permute_workspace_size(p)
    for i, word in [(0, "x"), (1, "topk_ids"), (3, "rows"), (4, "expert_offsets"),
                    (5, "slot_row"), (6, "row_slot"), (7, "ws")]:
        args = [V, V, None, V, V, V, V, V]
        args[i] = None
        refused(lib, lib.moe_permute(p._ref, *args, n, None), -1, word + " is NULL")
    args = [V, V, None, V, V, V, V, V]
    refused(lib, lib.moe_permute(p._ref, *args, n - 1, None), -3, "workspace")
    for i, word in enumerate(("grad_rows", "slot_row", "grad_x")):
        args = [V] * 3
        args[i] = None
        refused(lib, lib.moe_permute_backward(p._ref, *args, None), -1, word)
    for i, word in [(0, "rows"), (1, "slot_row"), (3, "out")]:
        args = [V] * 4
        args[i] = ODD
        refused(lib, lib.moe_unpermute(p._ref, *args, None), -1, word)
    for i, word in enumerate(("grad_out", "rows", "slot_row", "topk_weights", "grad_rows",
                              "grad_topk_weights")):
        args = [V] * 6
        args[i] = ODD
        refused(lib, lib.moe_unpermute_backward(p._ref, *args, None), -1, word)
    empty = moe.ExpertRows(0, 100, 8, 2)
    assert lib.moe_permute_backward(empty._ref, None, None, None, None) == 0
    assert lib.moe_unpermute(empty._ref, None, None, None, None, None) == 0
    assert lib.moe_unpermute_backward(empty._ref, *[None] * 7) == 0
    # the offsets of no rows are still written
    refused(lib, lib.moe_permute(empty._ref, *[None] * 8, 0, None), -1, "expert_offsets")


@pytest.mark.parametrize("kw,status,word", [
    (dict(num_tokens=-1), -1, "num_tokens"), (dict(hidden=0), -2, "hidden"),
    (dict(hidden=32769), -2, "hidden"), (dict(eps=-1.0), -1, "eps"),
    (dict(eps=float("nan")), -1, "eps"), (dict(residual_scale=float("inf")), -1, "scale"),
    (dict(weight_offset=float("nan")), -1, "offset"),
    (dict(weight_dtype=torch.float16), -2, "weight_dtype")])
def test_norm_problems(lib, kw, status, word):
    p = moe.BlockNorm(**{**dict(num_tokens=4, hidden=100), **kw})
    with pytest.raises(moe.MoeError) as e:
        moe.block_norm_workspace_size(p)
    assert e.value.status == status and word in str(e.value)
    refused(lib, lib.moe_block_norm(p._ref, V, V, None, None, V, V, V, None), status, word)
    refused(lib, lib.moe_block_norm_backward(p._ref, *[V] * 13, 1 << 40, None), status, word)


def test_norm_arguments(lib):
    p = moe.BlockNorm(4, 100, post_norm=True, gate="token")
    fwd = lib.moe_block_norm
    # residual, y, post_weight, gate, pre_weight, residual_out, normed
    good = [V] * 7
    for at, value, word in [(0, None, "residual"), (1, ODD, "y must"), (2, ODD, "post_weight"),
                            (3, None, "gate"), (4, ODD, "pre_weight"), (5, None, "residual_out"),
                            (6, ODD, "normed")]:
        args = list(good)
        args[at] = value
        refused(lib, fwd(p._ref, *args, None), -1, word)
    # without y: no weight, gate or stream of its own, and a norm to write
    for args, word in [([V, None, V, None, V, None, V], "post_weight"),
                       ([V, None, None, V, V, None, V], "gate"),
                       ([V, None, None, None, V, V, V], "residual_out"),
                       ([V, None, None, None, V, None, None], "normed")]:
        refused(lib, fwd(p._ref, *args, None), -1, word)
    plain = moe.BlockNorm(4, 100)
    refused(lib, fwd(plain._ref, V, V, V, None, V, V, V, None), -1, "post_weight")
    refused(lib, fwd(plain._ref, V, V, None, V, V, V, V, None), -1, "gate")

    bwd, n = lib.moe_block_norm_backward, moe.block_norm_workspace_size(p)
    # residual_out, y, post_weight, gate, pre_weight, grad_normed, grad_residual_out,
    # grad_residual, grad_y, grad_pre_weight, grad_post_weight, grad_gate, ws
    good = [V] * 13
    for at, value, word in [(0, None, "residual_out"), (3, None, "gate"), (5, ODD, "grad_normed"),
                            (6, ODD, "grad_residual_out"), (7, None, "grad_residual"),
                            (8, None, "grad_y"), (9, ODD, "grad_pre_weight"),
                            (10, ODD, "grad_post_weight"), (11, ODD, "grad_gate"),
                            (12, None, "ws")]:
        args = list(good)
        args[at] = value
        refused(lib, bwd(p._ref, *args, n, None), -1, word)
    refused(lib, bwd(p._ref, *good, n - 1, None), -3, "workspace")
    none = [V, None, None, None, V, V, V, V, None, V, None, None, V]
    for at, word in [(8, "grad_y"), (10, "grad_post_weight"), (11, "grad_gate")]:
        args = list(none)
        args[at] = V
        refused(lib, bwd(p._ref, *args, n, None), -1, word)
    refused(lib, bwd(plain._ref, V, V, None, None, V, V, V, V, V, V, None, V, V, n, None), -1,
            "grad_gate")
    empty = moe.BlockNorm(0, 100)
    assert fwd(empty._ref, *[None] * 7, None) == 0
    assert bwd(empty._ref, *[None] * 13, 0, None) == 0


def test_descriptor_choices():
    for kw in (dict(score="relu"), dict(dtype=torch.float64)):
        with pytest.raises(ValueError):
            moe.Router(4, 8, 2, **kw)
    with pytest.raises(ValueError):
        moe.ExpertRows(4, 8, 2, 1, dtype=torch.int32)
    for kw in (dict(gate="row"), dict(dtype=torch.float64), dict(weight_dtype=torch.int8)):
        with pytest.raises(ValueError):
            moe.BlockNorm(4, 8, **kw)


def test_binding_refuses_host_tensors():
    x = torch.zeros((4, 8), dtype=torch.bfloat16)
    i = torch.zeros((4, 2), dtype=torch.int32)
    w = torch.zeros((4, 2))
    with pytest.raises(ValueError, match="GPU"):
        moe.router_topk(moe.Router(4, 8, 2, dtype=torch.bfloat16), x, i, w)
    p = moe.ExpertRows(4, 8, 2, 2)
    with pytest.raises(ValueError, match="GPU"):
        moe.unpermute(p, torch.zeros((8, 8), dtype=torch.bfloat16), i, w, x)
    with pytest.raises(ValueError, match="GPU"):
        moe.block_norm(moe.BlockNorm(4, 8), x, x)


def test_argument_checks():
    d = torch.device("cpu")
    x = torch.zeros((4, 8))
    assert moe._arg(x, "x", torch.float32, (4, 8), d) == x.data_ptr()
    assert moe._arg(None, "x", torch.float32, (4, 8), d) is None
    for t, word in [(x.half(), "float32"), (x[:3], "4, 8"), (x.t().contiguous().t(), "contiguous"),
                    (x.to("meta"), "meta")]:
        with pytest.raises(ValueError, match=word):
            moe._arg(t, "x", torch.float32, (4, 8), d)


def small_block(experts=8):
    """A block on the host: what it refuses, it refuses before anything runs."""
    from types import SimpleNamespace
    layer = SimpleNamespace(p=moe.Problem(4, 128, 128, 8, 2))
    return moe.MoeBlock(layer, moe.Router(4, experts, 2), torch.zeros((experts, 128)),
                        moe.BlockNorm(4, 128))


def test_block_refuses_a_pre_norm_its_layer_would_misread():
    """One of another type or shape: the layer would read its bytes as bfloat16."""
    x, block = torch.zeros((4, 128), dtype=torch.bfloat16), small_block()
    for bad, word in [(x.half(), "normed must be torch.bfloat16"),
                      (x.float(), "normed must be torch.bfloat16"),
                      (x[:, :64].contiguous(), "normed must be"),
                      (x.t().contiguous().t(), "normed must be contiguous"),
                      (x.to("meta"), "normed is on meta")]:
        with pytest.raises(ValueError, match=word):
            block(x, normed=bad)
    with pytest.raises(ValueError, match="GPU"):
        block(x, normed=x)


def test_block_refuses_a_router_of_other_experts():
    """The layer would drop the ids past its own experts."""
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    maps = [dict(l2p=torch.zeros((n, 2), dtype=torch.int64)) for n in (7, 8, 9)]
    for n in (7, 9):
        with pytest.raises(ValueError, match=f"{n} experts, the layer has 8$"):
            small_block(n)(x)
    with pytest.raises(ValueError, match="8 experts, the layer has 7 logical ones"):
        small_block(8)(x, eplb=maps[0])
    for n, eplb in ((8, None), (9, maps[2]), (7, maps[0])):
        with pytest.raises(ValueError, match="GPU"):
            small_block(n)(x, eplb=eplb)


def test_descriptors_refuse_sizes_past_32_bits():
    """ctypes would keep their low 32 bits: 2^32 + 3 tokens would run as 3."""
    for make in (lambda n: moe.Router(n, 8, 2), lambda n: moe.Router(4, n, 2),
                 lambda n: moe.ExpertRows(n, 8, 8, 2), lambda n: moe.ExpertRows(4, n, 8, 2),
                 lambda n: moe.BlockNorm(n, 8), lambda n: moe.BlockNorm(4, n)):
        for n in (2 ** 31, 2 ** 32 + 3, -2 ** 31 - 1):
            with pytest.raises(ValueError, match="32 bits"):
                make(n)
        make(2 ** 31 - 1)


def test_descriptors_refuse_numpy_sizes_past_32_bits():
    import numpy as np
    for n in (np.int64(2 ** 32 + 3), np.uint32(2 ** 31), torch.tensor(2 ** 32 + 3)):
        with pytest.raises(ValueError, match="32 bits"):
            moe.BlockNorm(n, 8)
    assert moe.BlockNorm(np.int64(4), 8)._c.num_tokens == 4


def test_descriptors_can_be_copied_and_pickled():
    """As part of a model or of a worker's arguments."""
    import copy
    import pickle
    for p in (moe.Router(4, 8, 2, score="sigmoid", dtype=torch.float16),
              moe.ExpertRows(4, 8, 8, 2), moe.BlockNorm(4, 8, gate="token", post_norm=True)):
        for other in (copy.copy(p), copy.deepcopy(p), pickle.loads(pickle.dumps(p))):
            assert other == p and bytes(other._c) == bytes(p._c)
            assert getattr(other, "gate_shape", None) == getattr(p, "gate_shape", None)

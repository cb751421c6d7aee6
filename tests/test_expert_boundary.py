"""Refusals of the experts' own products, of the norm that leaves in 8 bits and
of the layer on staged rows, without a GPU: the C ABI checks
every argument before anything is enqueued (the pointers here are not
addresses of anything), the Python binding the shapes, types and devices."""
import copy
import ctypes
import os
import pickle

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


SIZES = [
    (dict(num_rows=-1), -1, "num_rows"), (dict(in_features=0), -2, "in_features"),
    (dict(in_features=32769), -2, "in_features"), (dict(out_features=0), -2, "out_features"),
    (dict(out_features=32769), -2, "out_features"), (dict(num_experts=0), -2, "num_experts"),
    (dict(num_experts=1025), -2, "num_experts"), (dict(act_limit=-1.0), -1, "act_limit"),
    (dict(act_limit=float("nan")), -1, "act_limit"),
    (dict(act_limit=float("inf")), -1, "act_limit"),
    (dict(activation="none", act_limit=1.0), -2, "clamp"),
    (dict(activation="gelu", act_limit=1.0), -2, "clamp"),
    (dict(num_rows=(1 << 31) - 1, in_features=32768), -2, "tiles")]


@pytest.mark.parametrize("kw,status,word", SIZES + [
    (dict(in_features=32768, out_features=32768, dtype=torch.float32), -2, "3.75 GiB"),
    (dict(in_features=32768, out_features=32768, activation="silu"), -2, "3.75 GiB")])
def test_linear_problems(lib, kw, status, word):
    p = moe.ExpertLinear(**{**dict(num_rows=4, in_features=64, out_features=32, num_experts=2,
                                   activation="silu"), **kw})
    refused(lib, lib.moe_expert_linear(p._ref, V, V, V, V, V, None), status, word)
    refused(lib, lib.moe_expert_linear_backward(p._ref, *[V] * 8, 1 << 40, None), status, word)
    n = ctypes.c_size_t()
    refused(lib, lib.moe_expert_linear_workspace_size(p._ref, ctypes.byref(n)), status, word)


def test_linear_arguments(lib):
    p = moe.ExpertLinear(4, 64, 32, 2, activation="silu")
    fwd, bwd = lib.moe_expert_linear, lib.moe_expert_linear_backward
    refused(lib, fwd(None, V, V, V, V, V, None), -1, "expert linear")
    for i, word in enumerate(("x", "expert_offsets", "weight", "out")):
        args = [V] * 5
        args[i] = None
        refused(lib, fwd(p._ref, *args, None), -1, word + " is NULL")
        args[i] = ODD
        refused(lib, fwd(p._ref, *args, None), -1, word)
    refused(lib, fwd(p._ref, V, V, V, V, ODD, None), -1, "pre_act")
    n = moe.expert_linear_workspace_size(p)
    assert n >= 4 * 64 * 2
    refused(lib, bwd(None, *[V] * 8, n, None), -1, "expert linear")
    # x, offsets, weight, pre_act, grad_out, grad_x, grad_weight, ws
    for i, word in ((0, "x"), (1, "expert_offsets"), (2, "weight"), (3, "pre_act"),
                    (4, "grad_out"), (7, "ws")):
        args = [V] * 8
        args[i] = None
        refused(lib, bwd(p._ref, *args, n, None), -1, word + " is NULL")
    for i, word in ((5, "grad_x"), (6, "grad_weight"), (7, "ws")):
        args = [V] * 8
        args[i] = ODD
        refused(lib, bwd(p._ref, *args, n, None), -1, word)
    refused(lib, bwd(p._ref, *[V] * 8, n - 1, None), -3, "workspace")
    plain = moe.ExpertLinear(4, 64, 32, 2)
    assert moe.expert_linear_workspace_size(plain) == 0
    refused(lib, bwd(plain._ref, *[V] * 8, 0, None), -1, "pre_act")
    refused(lib, lib.moe_expert_linear_workspace_size(p._ref, None), -1, "bytes")
    empty = moe.ExpertLinear(0, 64, 32, 2, activation="silu")
    assert fwd(empty._ref, *[None] * 6) == 0
    assert bwd(empty._ref, *[None] * 8, 0, None) == 0
    refused(lib, bwd(empty._ref, *[None] * 6, ODD, None, 0, None), -1, "grad_weight")
    bad = moe._ExpertLinear(4, 64, 32, 2, 3, 0, 0.0)
    refused(lib, fwd(ctypes.byref(bad), V, V, V, V, V, None), -1, "dtype")
    for act in (-2, 9):
        bad = moe._ExpertLinear(4, 64, 32, 2, 0, act, 0.0)
        refused(lib, fwd(ctypes.byref(bad), V, V, V, V, V, None), -1, "activation")


def test_the_layer_still_needs_an_activation(lib):
    """MOE_ACT_NONE belongs to the linear layers alone."""
    p = moe.Problem(16, 256, 512, 4, 2, activation=-1)
    with pytest.raises(moe.MoeError, match="activation"):
        moe.workspace_size(p)


def test_linear_binding():
    with pytest.raises(ValueError, match="activation"):
        moe.ExpertLinear(4, 64, 32, activation="relu")
    with pytest.raises(ValueError, match="dtype"):
        moe.ExpertLinear(4, 64, 32, dtype=torch.float64)
    with pytest.raises(ValueError, match="32 bits"):
        moe.ExpertLinear(1 << 32, 64, 32)
    p = moe.ExpertLinear(4, 64, 32, 2, activation="swiglustep", act_limit=2.0)
    assert p.wide == 64 and moe.ExpertLinear(4, 64, 32, activation="gelu_no_mul").wide == 32
    for q in (copy.deepcopy(p), pickle.loads(pickle.dumps(p))):
        assert q == p and q.wide == 64
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        moe.expert_linear(p, x, x, x)
    with pytest.raises(ValueError, match="GPU"):
        moe.expert_linear_backward(p, x, x, x)


@pytest.mark.parametrize("kw,status,word", SIZES + [
    (dict(group_size=16), -2, "group_size"), (dict(group_size=0), -2, "group_size"),
    (dict(format="mxfp4", group_size=64), -2, "MXFP4"),
    (dict(in_features=96, group_size=64), -2, "does not divide"),
    (dict(scale_dtype=torch.float16), -2, "scale_dtype")])
def test_w4_problems(lib, kw, status, word):
    p = moe.ExpertLinearW4(**{**dict(num_rows=4, in_features=64, out_features=32, num_experts=2,
                                     activation="silu", group_size=32), **kw})
    refused(lib, lib.moe_expert_linear_w4(p._ref, V, V, V, V, None, V, None), status, word)


def test_w4_arguments(lib):
    p = moe.ExpertLinearW4(4, 64, 32, 2, format="int4_zero", group_size=32)
    call = lib.moe_expert_linear_w4
    refused(lib, call(None, V, V, V, V, V, V, None), -1, "expert linear")
    for i, word in enumerate(("x", "expert_offsets", "codes", "scales", "zeros", "out")):
        args = [V] * 6
        args[i] = None
        refused(lib, call(p._ref, *args, None), -1, word + " is NULL")
        if word not in ("codes", "zeros"):              # bytes lie at any address
            args[i] = ODD
            refused(lib, call(p._ref, *args, None), -1, word)
    plain = moe.ExpertLinearW4(4, 64, 32, 2, group_size=32)
    refused(lib, call(plain._ref, V, V, V, V, V, V, None), -1, "zeros")
    empty = moe.ExpertLinearW4(0, 64, 32, 2, group_size=32)
    assert call(empty._ref, *[None] * 7) == 0
    bad = moe._ExpertLinearW4(4, 64, 32, 2, 0, -1, 0.0, 3, 32, 0)
    refused(lib, call(ctypes.byref(bad), V, V, V, V, None, V, None), -1, "format")


def test_w4_binding():
    with pytest.raises(ValueError, match="format"):
        moe.ExpertLinearW4(4, 64, 32, format="nf4")
    with pytest.raises(ValueError, match="uint8"):
        moe.ExpertLinearW4(4, 64, 32, format="mxfp4", group_size=32, scale_dtype=torch.float32)
    with pytest.raises(ValueError, match="scale_dtype"):
        moe.ExpertLinearW4(4, 64, 32, scale_dtype=torch.uint8)
    p = moe.ExpertLinearW4(4, 64, 32, 2, activation="silu", format="mxfp4", group_size=32)
    assert p.wide == 64 and p.scales == torch.uint8
    assert pickle.loads(pickle.dumps(p)) == p
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        moe.expert_linear_w4(p, x, x, x, x)


# ---- the norm in 8 bits and the layer on staged rows --------------------------------

@pytest.mark.parametrize("kw,status,word", [
    (dict(num_tokens=-1), -1, "num_tokens"), (dict(hidden=0), -2, "hidden"),
    (dict(hidden=32896), -2, "hidden"), (dict(hidden=200), -2, "multiple of 128"),
    (dict(eps=0.0), -1, "eps")])
def test_norm_quant_problems(lib, kw, status, word):
    p = moe.BlockNorm(**{**dict(num_tokens=4, hidden=256), **kw})
    refused(lib, lib.moe_block_norm_quant(p._ref, 0, V, V, None, None, V, V, V, V, V, None),
            status, word)


def test_norm_quant_arguments(lib):
    p = moe.BlockNorm(4, 256, post_norm=True, gate="token")
    call = lib.moe_block_norm_quant
    # residual, y, post_weight, gate, pre_weight, residual_out, normed, x_q, x_sf
    for i, word in ((0, "residual"), (3, "gate"), (5, "residual_out"), (7, "x_q"), (8, "x_sf")):
        args = [V] * 9
        args[i] = None
        refused(lib, call(p._ref, 0, *args, None), -1, word + " is NULL")
        args[i] = ODD
        refused(lib, call(p._ref, 0, *args, None), -1, word)
    refused(lib, call(p._ref, 0, *[V] * 7, ctypes.c_void_p((1 << 20) + 8), V, None), -1, "x_q")
    for kind in (-1, 2, 4):
        refused(lib, call(p._ref, kind, *[V] * 9, None), -1, "quantization")
    refused(lib, call(p._ref, 0, V, None, None, None, V, V, V, V, V, None), -1, "residual_out")
    refused(lib, call(None, 0, *[V] * 9, None), -1, "block norm")
    empty = moe.BlockNorm(0, 256)
    assert call(empty._ref, 0, *[None] * 10) == 0


def test_staged_rows_arguments(lib):
    p = moe.Problem(16, 256, 256, 4, 2)
    ref = ctypes.byref(p.c())
    call = lib.moe_forward_quantized
    # x_q, x_sf, counts, ids, weights, padding | eplb | w13, w13_sf, w2, w2_sf, out, ws
    good = [V, V, None, V, V, None, None, V, V, V, V, V, V]
    n = moe.workspace_size(p)
    for i, word in ((0, "x_q"), (1, "x_sf"), (3, "topk_ids"), (4, "topk_weights"), (7, "w13"),
                    (8, "w13_sf"), (9, "w2"), (10, "w2_sf"), (11, "out"), (12, "ws")):
        args = list(good)
        args[i] = None
        refused(lib, call(ref, *args, n, None), -1, word + " is NULL")
    refused(lib, call(ref, ODD, *good[1:], n, None), -1, "x_q")
    refused(lib, call(ref, *good, n - 1, None), -3, "workspace")
    half = moe.Problem(16, 256, 256, 4, 2, act_quant=moe.Q_BF16)
    refused(lib, call(ctypes.byref(half.c()), *good, 1 << 40, None), -2, "staged")
    call = lib.moe_stage_routing
    r = moe._Routing(*[V] * 5)
    good = [None, V, V, None, None, V, V, ctypes.byref(r), V]
    n = moe.stage_workspace_size(p)
    for i, word in ((1, "topk_ids"), (2, "topk_weights"), (5, "topk_idx_out"), (6, "topk_w_out"),
                    (7, "routing"), (8, "ws")):
        args = list(good)
        args[i] = None
        refused(lib, call(ref, *args, n, None), -1, word)
    refused(lib, call(ref, *good, n - 1, None), -3, "workspace")
    empty = moe.Problem(0, 256, 256, 4, 2)
    assert call(ctypes.byref(empty.c()), *[None] * 9, 0, None) == 0
    assert lib.moe_forward_quantized(ctypes.byref(empty.c()), *[None] * 13, 0, None) == 0


def test_linear_workspace_of_split_gradients(lib):
    """No activation, but few results of long sums: their parts need a workspace."""
    p = moe.ExpertLinear(6300, 136, 200, 1)
    n = moe.expert_linear_workspace_size(p)
    assert 0 < n <= 32 << 20
    bwd = lib.moe_expert_linear_backward
    args = [V, None, V, None, V, V, V]
    refused(lib, bwd(p._ref, *args, None, n, None), -1, "ws is NULL")
    refused(lib, bwd(p._ref, *args, ODD, n, None), -1, "ws")
    refused(lib, bwd(p._ref, *args, V, n - 1, None), -3, "workspace")
    for R in (1, 100, 6000, 32768, 1 << 20):
        for K, N, E in ((64, 64, 1), (4096, 4096, 1), (32768, 64, 1), (64, 32768, 3),
                        (7168, 2048, 32), (8, 8, 1024)):
            p = moe.ExpertLinear(R, K, N, E)
            assert moe.expert_linear_workspace_size(p) <= 32 << 20
            p = moe.ExpertLinear(R, K, N, E, activation="silu")
            assert moe.expert_linear_workspace_size(p) <= (32 << 20) + 512 + R * p.wide * 2

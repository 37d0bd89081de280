"""Argument checks of the backward entry points on the host (CPU only, no launches)."""
import ctypes

import pytest

import sparse_moe_layer_smoe_b200 as smoe

WS = 1 << 40   # bytes claimed for a workspace that no call here reaches

# entry point -> its arguments after the config: "p" a required pointer, "o" an optional one, "T", ws, bytes, stream
CALLS = {
    "smoe_expert_ffn_save": "p o o p T p p p p ws bytes stream",
    "smoe_checkpoint_values": "p p T p stream",
    "smoe_combine_backward": "p p p p T p p ws bytes stream",
    "smoe_route_backward": "p T p p p p p p p p p ws bytes stream",
    "smoe_expert_ffn_backward": "p p p T p p p p p p p p p p p p ws bytes stream",
    "smoe_permute_backward": "p p p p p T p ws bytes stream",
}


def _args(spec, T=4, change=None):
    given = {"p": 16, "o": 16, "T": T, "ws": 256, "bytes": WS, "stream": None}
    a = [given[s] for s in spec.split()]
    for i, v in (change or {}).items():
        a[i] = v
    return a


@pytest.mark.parametrize("fn", CALLS)
def test_pointers_are_checked(fn):
    f, c = getattr(smoe.lib(), fn), smoe.config()
    kinds = CALLS[fn].split()
    for i, kind in enumerate(kinds):
        if kind in ("p", "o"):
            assert f(ctypes.byref(c), *_args(CALLS[fn], change={i: 24})) == smoe.SMOE_ERR_INVALID_ARG, i
        if kind == "p":
            # dlogits NULL leaves the router's term of smoe_permute_backward out: an allowed call
            if fn == "smoe_permute_backward" and i == 3:
                continue
            assert f(ctypes.byref(c), *_args(CALLS[fn], change={i: None})) == smoe.SMOE_ERR_INVALID_ARG, i
        if kind == "ws":
            for bad in (None, 272):
                assert f(ctypes.byref(c), *_args(CALLS[fn], change={i: bad})) == smoe.SMOE_ERR_INVALID_ARG
    if fn == "smoe_expert_ffn_save":
        assert f(ctypes.byref(c), *_args(CALLS[fn], change={1: None, 2: None})) == smoe.SMOE_ERR_INVALID_ARG


@pytest.mark.parametrize("fn", CALLS)
def test_sizes_are_checked(fn):
    f, c = getattr(smoe.lib(), fn), smoe.config()
    assert f(ctypes.byref(c), *_args(CALLS[fn], T=-1)) == smoe.SMOE_ERR_INVALID_ARG
    assert f(ctypes.byref(c), *_args(CALLS[fn], T=1 << 40)) == smoe.SMOE_ERR_UNSUPPORTED
    assert f(None, *_args(CALLS[fn])) == smoe.SMOE_ERR_INVALID_ARG
    assert f(ctypes.byref(smoe.config(hidden=100)), *_args(CALLS[fn])) == smoe.SMOE_ERR_UNSUPPORTED
    kinds = CALLS[fn].split()
    if "bytes" in kinds:
        need = (smoe.smoe_scratch_bytes if fn.endswith("save") else smoe.smoe_backward_bytes)(c, 4)
        a = _args(CALLS[fn], change={kinds.index("bytes"): need - 1})
        assert f(ctypes.byref(c), *a) == smoe.SMOE_ERR_WORKSPACE


@pytest.mark.parametrize("fn", ["smoe_expert_ffn_save", "smoe_checkpoint_values", "smoe_combine_backward",
                                "smoe_permute_backward"])
def test_no_tokens_is_a_no_op(fn):
    a = [None if s in ("p", "o", "ws") else (0 if s == "bytes" else v)
         for s, v in zip(CALLS[fn].split(), _args(CALLS[fn], T=0))]
    c = smoe.config()
    assert getattr(smoe.lib(), fn)(ctypes.byref(c), *a) == smoe.SMOE_OK


def test_no_tokens_still_needs_the_gradients_to_clear():
    L, c = smoe.lib(), smoe.config()
    a = _args(CALLS["smoe_route_backward"], T=0, change={10: None})
    assert L.smoe_route_backward(ctypes.byref(c), *a) == smoe.SMOE_ERR_INVALID_ARG
    for i in range(10, 16):
        a = _args(CALLS["smoe_expert_ffn_backward"], T=0, change={i: None})
        assert L.smoe_expert_ffn_backward(ctypes.byref(c), *a) == smoe.SMOE_ERR_INVALID_ARG


def test_workspace_bytes():
    c = smoe.config()
    one, many = smoe.smoe_backward_bytes(c, 1), smoe.smoe_backward_bytes(c, 8192)
    assert 0 < one < many and smoe.smoe_backward_bytes(c, 0) > 0
    # h, dg and du of every row
    assert many >= 8192 * 9 * 3 * 1280 * 2
    assert smoe.lib().smoe_backward_bytes(ctypes.byref(c), 4, None) == smoe.SMOE_ERR_INVALID_ARG


@pytest.mark.parametrize("shape", [(4, 64), (4, 2, 512), (512,)])
def test_layer_training_methods_check_shapes(shape):
    import torch
    layer = smoe.MoELayer(smoe.config(hidden=512), None, None, None)
    good, bad = torch.zeros(4, 512, dtype=torch.bfloat16), torch.zeros(shape, dtype=torch.bfloat16)
    with pytest.raises(smoe.SmoeError, match="x is") as e:
        layer.forward_train(bad)
    assert e.value.status == smoe.SMOE_ERR_INVALID_ARG
    for dout in (bad, good[:3]):
        with pytest.raises(smoe.SmoeError, match="dout is") as e:
            layer.backward({"x": good}, dout)
        assert e.value.status == smoe.SMOE_ERR_INVALID_ARG

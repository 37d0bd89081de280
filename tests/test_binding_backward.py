"""What the Python form of the training calls refuses, on the host: CPU tensors on a pretended device, and a library
that must not be reached."""
import sys
import warnings

import pytest
import torch

import sparse_moe_layer_smoe_b200 as smoe

T, H, E, k, I = 4, 128, 4, 2, 128
R = T * k


class _NothingNative:
    """Stands in for the native module and leaves every call to Python."""
    def __getattr__(self, name):
        return lambda *args: None


class _Library:
    """Records the calls that would have reached the library."""
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append(name) or smoe.SMOE_OK


@pytest.fixture
def library(monkeypatch):
    """The current device is the CPU's index, -1: CPU tensors are on it."""
    fake = _Library()
    monkeypatch.setattr(smoe, "lib", lambda: fake)
    monkeypatch.setattr(smoe, "_native", _NothingNative())
    monkeypatch.setattr(smoe, "_cuda", (lambda: -1, lambda device: 0))
    return fake


def _cfg():
    return smoe.config(H, E, k, I, I)


def _new(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def _calls():
    """entry point -> its arguments by name, in order (the config left out)."""
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    x, x_perm, y, rows = _new(T, H), _new(R, H), _new(R + T, H), _new(R + T, H)
    offsets, perm_row, row_token = _new(E + 1, dtype=i32), _new(R, dtype=i32), _new(R, dtype=i32)
    idx, w = _new(T, k, dtype=i32), _new(T, k, dtype=f32)
    q, sc = _new(R + T, 2 * I, dtype=u8), _new(2 * I // 32, R + T, dtype=u8)
    packed, ws = _new(_packed_bytes(), dtype=u8), _new(256, dtype=u8)
    wr = _new(E, H, dtype=f32)
    return {
        "smoe_expert_ffn_save": dict(x=x, x_perm=x_perm, row_token=row_token, offsets=offsets, T=T, packed=packed, y=y,
                                     gu_q=q, gu_scale=sc, ws=ws),
        "smoe_expert_ffn_backward": dict(
            x=x, x_perm=x_perm, offsets=offsets, T=T, packed=packed, gu_q=q, gu_scale=sc, dy=_new(R, H), dout=_new(T, H),
            dx_rows=rows, dw_gate=_new(E, I, H), dw_up=_new(E, I, H), dw_down=_new(E, H, I), dws_gate=_new(I, H),
            dws_up=_new(I, H), dws_down=_new(H, I), ws=ws),
        "smoe_combine_backward": dict(dout=_new(T, H), y=y, perm_row=perm_row, topk_w=w, T=T, dy=_new(R, H),
                                      dtopk_w=_new(T, k, dtype=f32), ws=ws),
        "smoe_route_backward": dict(x=x, T=T, logits=_new(T, E, dtype=f32), topk_idx=idx, topk_w=w,
                                    dtopk_w=_new(T, k, dtype=f32), offsets=offsets, perm_row=perm_row, row_token=row_token,
                                    dlogits=_new(T, k, dtype=f32), dw_router=wr, ws=ws),
        "smoe_permute_backward": dict(dx_rows=rows, perm_row=perm_row, topk_idx=idx, dlogits=_new(T, k, dtype=f32),
                                      w_router=wr, T=T, dx=_new(T, H), ws=ws),
        "smoe_checkpoint_values": dict(gu_q=q, gu_scale=sc, T=T, gu=_new(R + T, 2 * I)),
    }


def _packed_bytes():
    return (E + 1) * 3 * I * H * 2


def _refused(fn, args, name):
    with pytest.raises(smoe.SmoeError, match=rf"\b{name} ") as e:
        getattr(smoe, fn)(_cfg(), **args)
    assert e.value.status == smoe.SMOE_ERR_INVALID_ARG


@pytest.mark.parametrize("fn", ["smoe_expert_ffn_save", "smoe_expert_ffn_backward"])
def test_packed_weights_are_checked(fn, library, monkeypatch):
    """The tensor maps span the whole of them: too few bytes, gaps or another device are refused before any launch."""
    good = _calls()[fn]
    getattr(smoe, fn)(_cfg(), **good)
    # any type will do: the bytes count
    getattr(smoe, fn)(_cfg(), **{**good, "packed": good["packed"].view(torch.bfloat16)})
    assert library.calls == [fn, fn]
    for bad in (good["packed"][:-1], good["packed"][:_packed_bytes() // 2].view(torch.bfloat16),
                _new(2 * _packed_bytes(), dtype=torch.uint8)[::2]):
        _refused(fn, {**good, "packed": bad}, "packed")
    monkeypatch.setattr(smoe, "_cuda", (lambda: 0, lambda device: 0))
    pointers = {a: v if a == "packed" or not isinstance(v, torch.Tensor) else v.data_ptr() for a, v in good.items()}
    _refused(fn, pointers, "packed")
    assert library.calls == [fn, fn]


def test_packed_bytes_are_the_librarys():
    for c in (_cfg(), smoe.config()):
        assert smoe._packed_bytes(c) == smoe.smoe_packed_weight_bytes(c)


def test_forward_train_checks_the_packed_weights(library):
    packed = _new(_packed_bytes() - 1, dtype=torch.uint8)
    layer = smoe.MoELayer(_cfg(), _new(E, H, dtype=torch.float32), _new(E, dtype=torch.float32), packed)
    with pytest.raises(smoe.SmoeError, match="packed has"):
        layer.forward_train(_new(T, H), ws=_new(256, dtype=torch.uint8))
    assert library.calls == []


def test_calls_without_the_native_module(monkeypatch):
    """Built for another Python or torch it does not load: one warning, and the Python form makes every call."""
    monkeypatch.setattr(smoe, "_native", None)
    monkeypatch.setitem(sys.modules, "sparse_moe_layer_smoe_b200._pyargs", None)
    monkeypatch.delattr(smoe, "_pyargs", raising=False)
    c = _cfg()
    with pytest.warns(RuntimeWarning, match="native training calls"):
        smoe.smoe_combine_backward(c, None, None, None, None, 0, None, None)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        smoe.smoe_permute_backward(c, None, None, None, None, None, 0, None)
        smoe.smoe_expert_ffn_save(c, None, None, None, None, 0, None, None, None, None)
        smoe.smoe_checkpoint_values(c, None, None, 0, None)
        with pytest.raises(smoe.SmoeError, match="smoe_route_backward"):
            smoe.smoe_route_backward(c, *[None] * 1, 0, *[None] * 9)
        with pytest.raises(smoe.SmoeError, match="smoe_expert_ffn_backward"):
            smoe.smoe_expert_ffn_backward(c, *[None] * 3, 0, *[None] * 12)

"""The native form of the training calls: what it leaves to Python, and how it calls the library."""
import ctypes

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import sparse_moe_layer_smoe_b200 as smoe  # noqa: E402
import test_binding_backward as host  # noqa: E402


def _calls():
    """The host tests' calls on the GPU, with a workspace."""
    n = max(smoe.smoe_scratch_bytes(host._cfg(), host.T), smoe.smoe_backward_bytes(host._cfg(), host.T))
    out = {}
    for fn, args in host._calls().items():
        out[fn] = {a: v.cuda() if isinstance(v, torch.Tensor) else v for a, v in args.items()}
        if "ws" in args:
            out[fn]["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    return out


def _native(fn, args, native=None):
    """The native call's answer: a status, or None where it leaves the call to Python."""
    rest = (None, None) if "ws" in args else (None,)      # ws_bytes, stream
    return getattr(native or smoe._load_native(), fn.removeprefix("smoe_"))(host._cfg(), *args.values(), *rest)


@pytest.mark.parametrize("fn", ["smoe_expert_ffn_save", "smoe_expert_ffn_backward"])
def test_packed_weights_are_checked(fn):
    """Too few bytes, gaps or another device: left to Python, which refuses them before any launch."""
    good = _calls()[fn]
    assert _native(fn, good) == smoe.SMOE_OK
    assert _native(fn, {**good, "packed": good["packed"].view(torch.bfloat16)}) == smoe.SMOE_OK
    torch.cuda.synchronize()
    half = good["packed"][:good["packed"].numel() // 2]
    for bad in (good["packed"][:-1], half.view(torch.bfloat16), good["packed"].repeat(2)[::2], good["packed"].cpu()):
        args = {**good, "packed": bad}
        assert _native(fn, args) is None
        with pytest.raises(smoe.SmoeError, match=r"\bpacked ") as e:
            getattr(smoe, fn)(host._cfg(), **args)
        assert e.value.status == smoe.SMOE_ERR_INVALID_ARG
    torch.cuda.synchronize()


def test_the_library_is_called_without_the_interpreter_lock():
    """A launch may block (a full queue, a host callback that needs the lock): other Python threads go on meanwhile.
    PyGILState_Check stands in for the library: it answers 1 where the caller holds the lock, and launches nothing."""
    calls, native = _calls(), smoe._load_native()
    check = ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value
    try:
        native.use(*[check] * 6)
        answers = {fn: _native(fn, args, native) for fn, args in calls.items()}
    finally:
        smoe._load_native()
    assert answers == dict.fromkeys(calls, 0)

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


def _arguments():
    for fn, args in host._calls().items():
        for a, v in args.items():
            if isinstance(v, torch.Tensor):
                yield fn, a


@pytest.mark.parametrize("fn,name", list(_arguments()))
def test_both_forms_refuse_the_same(fn, name):
    """Every tensor of every call: of one element fewer, with gaps, on the host or (but for the packed weights and
    the workspace) of another type the native form leaves the call, and the Python form refuses it."""
    good = _calls()[fn]
    t = good[name].reshape(-1)
    bad = {"short": t[:-1], "gaps": t.repeat(2)[::2], "host": t.cpu()}
    if name not in ("packed", "ws"):
        bad["type"] = t.to(torch.float64)
    if name == "ws":    # the library's own check: SMOE_ERR_WORKSPACE
        del bad["short"]
    for kind, b in bad.items():
        args = {**good, name: b}
        assert _native(fn, args) is None, kind
        with pytest.raises(smoe.SmoeError, match=rf"\b{name} ") as e:
            getattr(smoe, fn)(host._cfg(), **args)
        assert e.value.status == smoe.SMOE_ERR_INVALID_ARG, kind

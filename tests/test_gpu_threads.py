"""Host threads that use the library at the same time, each on its own stream with its own workspace."""
import ctypes
import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import sparse_moe_layer_smoe_b200 as smoe  # noqa: E402


class _NothingNative:
    """Stands in for the native module and leaves every call to Python."""
    def __getattr__(self, name):
        return lambda *args: None


def _layer(E, H, I, k, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    new = lambda *s, std=0.05: torch.empty(s, device="cuda").normal_(0, std, generator=gen)
    w = [new(*s).bfloat16() for s in ((E, I, H), (E, I, H), (E, H, I), (I, H), (I, H), (H, I))]
    cfg = smoe.config(H, E, k, I, I)
    return smoe.MoELayer(cfg, new(E, H), new(E), smoe.pack_weights(cfg, *w)), gen


def _together(jobs):
    errors = []

    def guarded(job):
        try:
            job()
        except Exception as e:   # noqa: BLE001  (reported below)
            errors.append(repr(e))
    threads = [threading.Thread(target=guarded, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[:2]


# E, H, I, k, T of the two threads: different shared-memory sizes of the same kernels, on single CTAs and on pairs
SHAPES = [((8, 128, 128, 2, 40), (1024, 128, 128, 4, 40)), ((4, 256, 256, 2, 300), (16, 256, 256, 4, 900))]


@pytest.mark.parametrize("shapes", SHAPES)
def test_launches_of_two_threads(shapes):
    """A kernel's shared-memory limit is the process's: one thread's call must not lower it between another's check
    and its launch. Calls of the C-ABI with nothing of Python between them."""
    f, work = smoe.lib().smoe_expert_ffn_backward, []
    for n, (E, H, I, k, T) in enumerate(shapes):
        layer, gen = _layer(E, H, I, k, n)
        cfg, R = layer.cfg, T * k
        new = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")
        offsets = torch.linspace(0, R, E + 1, device="cuda").int()
        ws = smoe.workspace(cfg, T, backward=True)
        tensors = [new(T, H), new(R, H), offsets, layer.packed, new(R + T, 2 * I, dt=torch.uint8),
                   new(2 * I // 32, R + T, dt=torch.uint8), new(R, H), new(T, H), new(R + T, H), new(E, I, H), new(E, I, H),
                   new(E, H, I), new(I, H), new(I, H), new(H, I)]
        p = [t.data_ptr() for t in tensors]
        stream = torch.cuda.Stream()
        work.append((f, (ctypes.byref(cfg), *p[:3], T, *p[3:], ws.data_ptr(), ws.numel(), stream.cuda_stream), tensors, ws))
    torch.cuda.synchronize()

    def job(f, args, tensors, ws):
        torch.cuda.set_device(0)
        bad = [s for s in (f(*args) for _ in range(5000)) if s != smoe.SMOE_OK]
        assert not bad, f"{len(bad)} of 5000 calls failed, the first with {smoe.STATUS[bad[0]]}"
    _together([lambda w=w: job(*w) for w in work])
    torch.cuda.synchronize()
    assert [smoe.smoe_get_device_error(w[3]) for w in work] == [0, 0]


@pytest.mark.parametrize("shapes", SHAPES)
@pytest.mark.parametrize("native", [True, False])
def test_training_steps_of_two_threads(shapes, native, monkeypatch):
    """A kernel's shared-memory limit is the process's: one thread's call must not lower it under another's launch."""
    if native:
        smoe._load_native()
    else:
        monkeypatch.setattr(smoe, "_native", _NothingNative())
    work = []
    for n, (E, H, I, k, T) in enumerate(shapes):
        layer, gen = _layer(E, H, I, k, n)
        x, dout = (torch.empty(T, H, device="cuda").normal_(generator=gen).bfloat16() for _ in range(2))
        ws = smoe.workspace(layer.cfg, T, backward=True)

        def step(layer=layer, x=x, dout=dout, ws=ws):
            out, saved = layer.forward_train(x, ws)
            return dict(layer.backward(saved, dout, ws), out=out)
        want = step()
        torch.cuda.synchronize()
        work.append((step, want))

    def job(step, want):
        with torch.cuda.stream(torch.cuda.Stream()):
            for i in range(150):
                got = step()
                if i % 50 == 0:
                    for key, v in want.items():
                        assert torch.equal(got[key].view(torch.uint8), v.view(torch.uint8)), key
            torch.cuda.current_stream().synchronize()
    _together([lambda w=w: job(*w) for w in work])

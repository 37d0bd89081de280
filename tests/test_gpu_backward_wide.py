"""GPU tests of the backward entry points on widths like the layer's: every CTA pair takes several units, each of
several stages with a row tail, and rows take several turns of the feature loops. Helpers, oracle and error
bounds are those of test_gpu_backward.py."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import numpy as np  # noqa: E402

import test_gpu_backward as base  # noqa: E402

# T, H, E, k, I, clamp, skew
TAILS = (600, 1024, 9, 2, 512, False, 0.0)     # 240 units of the weight gradients on 74 pairs, 2 to 3 stages and 10


@pytest.fixture
def shape(monkeypatch):
    def use(name, values):
        monkeypatch.setitem(base.SHAPES, name, values)
        return values
    return use


def test_row_tails_are_cleared_before_the_products_read_them(shape):
    """The neighbours' rows in every last stage are NaN and infinite; the second CTA clears its own and the first
    one's products read both. Twenty runs, each with the clean one's bits."""
    T, H, E, k, I, _, _ = shape("tails", TAILS)
    p = base._backward_inputs("tails", np.random.default_rng(72))
    off = p["r"]["offsets"]
    assert all((off[e + 1] - off[e]) % 16 for e in range(E)), "every expert has a tail"
    clean, ws = base._outputs(p["cfg"], T), base._ws(p["cfg"], T)
    base._ffn_backward(p, T, clean, ws)
    assert base.smoe.smoe_get_device_error(ws) == 0
    base._check_ffn_backward("tails", p, clean)
    for e in range(1, E, 2):
        p["dy"][off[e]:off[e + 1]] = float("nan")
        p["x_perm"][off[e]:off[e + 1]] = float("inf")
        p["q"][off[e]:off[e + 1]] = 0x7F
    p["q"][T * k:T * k + 16] = 0x7F       # the shared expert's first rows, behind the last expert's
    good = list(range(0, E, 2))
    for _ in range(20):
        out = base._outputs(p["cfg"], T)
        base._ffn_backward(p, T, out, ws)
        for key in ("dw_gate", "dw_up", "dw_down"):
            assert torch.equal(out[key][good].view(torch.int16), clean[key][good].view(torch.int16)), key


WIDE = {
    # the layer's widths: 256 threads a row and several turns of the feature loops, two slices of router features, partial
    # sums joined in eight column blocks, an odd number of 256-feature blocks, thirteen weight-gradient units a pair
    "layer": (200, 4096, 3, 2, 1280, False, 0.0),
    # odd multiples of 128 with a last slice, column block and turn that are partly empty; single CTAs on large tiles
    "partial_slices": (150, 2176, 5, 2, 384, True, 1.5),
    # 45 token tiles of two blocks each: a second unit for the CTA pairs of every product, with one accumulator
    # set (gate/up with the checkpoint) and two (dh, dx)
    "second_units": (1100, 512, 40, 4, 512, True, 0.0),
}
TESTS = {
    "combine": base.test_combine_backward,
    "permute": lambda name: base.test_permute_backward(name, True),
    "permute_without_router": lambda name: base.test_permute_backward(name, False),
    "route": base.test_route_backward,
    "ffn_save": lambda name: base.test_expert_ffn_save(name, False),
    "ffn_save_gathered": lambda name: base.test_expert_ffn_save(name, True),
    "ffn_backward": base.test_expert_ffn_backward,
    "training_step": base.test_training_step_against_the_oracle,
}


@pytest.mark.parametrize("test", TESTS)
@pytest.mark.parametrize("name", WIDE)
def test_wide(name, test, shape):
    """The small shapes' tests, their bounds among them."""
    shape(name, WIDE[name])
    TESTS[test](name)

"""The fp64 gradient oracle against differences of the forward oracle (CPU).

A central difference of step d has error of order d^2 times a third derivative plus 2^-52 / d of the
value: with d = 1e-5 and values of order 1 to 100 that is below 1e-8, and 1e-6 relative to the largest
gradient leaves two orders."""
import numpy as np
import pytest

from oracle import backward as ob
from oracle import moe
from oracle.fp8 import e4m3_code, e4m3_round

STEP, TOL = 1e-5, 1e-6


def _diff(f, a):
    """Central differences of the scalar f() in every entry of a (changed in place)."""
    g = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        v = a[i]
        a[i] = v + STEP
        hi = f()
        a[i] = v - STEP
        lo = f()
        a[i] = v
        g[i] = (hi - lo) / (2 * STEP)
    return g


def _close(got, want):
    assert np.abs(got - want).max() <= TOL * max(1.0, np.abs(want).max())


@pytest.mark.parametrize("k,limit,limit_shared", [(1, 0.0, 0.0), (3, 0.0, 0.0), (3, 0.5, 0.8)])
def test_the_whole_backward_pass_against_differences(k, limit, limit_shared):
    """Chained as a training step chains them, the oracle's gradients are those of <dout, layer(x)>."""
    rng = np.random.default_rng(7 + k)
    T, H, E, I, c = 5, 6, 4, 3, 3.0
    x, wr = rng.normal(size=(T, H)), rng.normal(size=(E, H))
    W = [tuple(rng.normal(size=s) for s in ((I, H), (I, H), (H, I))) for _ in range(E + 1)]
    dout = rng.normal(size=(T, H))
    bias = np.zeros(E)
    r = moe.route(x, wr, bias, k, c)
    # no selection flips within the difference step: a step moves a logit by STEP * max(|x|, |w|) < 1e-4
    # and a score by a quarter of that
    assert r.gap.min() > 1e-3 and max(np.abs(x).max(), np.abs(wr).max()) < 10
    lim = lambda e: limit_shared if e == E else limit

    def loss():
        q = moe.route(x, wr, bias, k, c)
        return float((dout * moe.moe_sparse(x, q, lambda e: W[e], E, limit, limit_shared)).sum())

    counts, offsets, perm_row, row_token = moe.permute(r.idx, E)
    xr = np.concatenate([x[row_token], x])
    bounds = list(offsets) + [T * k + T]
    g, u, y = np.zeros((T * k + T, I)), np.zeros((T * k + T, I)), np.zeros((T * k + T, H))
    for e in range(E + 1):
        a, b = bounds[e], bounds[e + 1]
        g[a:b], u[a:b] = xr[a:b] @ W[e][0].T, xr[a:b] @ W[e][1].T
        y[a:b] = moe.swiglu_ffn(xr[a:b], *W[e], limit=lim(e))
    if limit:
        for v, L in ((g, lim(0)), (u, lim(0))):   # both sides of the clamp, none near it
            assert (np.abs(np.abs(v) - L) > 1e-4).all() and (np.abs(v) > L).any()
    dy, dw = ob.combine_backward(dout, y, perm_row, r.w)
    dl, dwr = ob.route_backward(x, r.logits, r.idx, dw, c)
    dy = np.concatenate([dy, dout])
    dxr = np.zeros((T * k + T, H))
    dW = []
    for e in range(E + 1):
        a, b = bounds[e], bounds[e + 1]
        dxr[a:b], *d = ob.expert_backward(xr[a:b], g[a:b], u[a:b], dy[a:b], *W[e], limit=lim(e))
        dW.append(d)
    _close(ob.permute_backward(dxr, perm_row, r.idx, dl, wr), _diff(loss, x))
    _close(dwr, _diff(loss, wr))
    for e in range(E + 1):
        for got, w in zip(dW[e], W[e]):
            _close(got, _diff(loss, w))


def test_route_gradient_with_one_expert_is_zero():
    rng = np.random.default_rng(3)
    dl, dwr = ob.route_backward(rng.normal(size=(4, 6)), rng.normal(size=(4, 3)), np.zeros((4, 1), np.int32),
                                rng.normal(size=(4, 1)), 3.0)
    assert np.abs(dl).max() <= 1e-15 and np.abs(dwr).max() <= 1e-14


def test_checkpoint_holds_values_to_half_a_step():
    """Half a step of e4m3 is 2^-4 of the value, and 2^-10 of the scale under 2^-6 of it; the scale is the
    least power of two with no magnitude above 448."""
    rng = np.random.default_rng(5)
    v = (rng.normal(size=(64, 128)) * np.exp(rng.normal(size=(64, 1)) * 4)).astype(np.float32).astype(np.float64)
    v[3, :32] = 0.0
    v[4, 0], v[4, 1:32] = 448.0 * 2.0 ** 9, 1.0
    v[5, 0], v[5, 1:32] = np.nextafter(np.float32(448.0), np.float32(1e9)), 1.0
    held, exps = ob.checkpoint(v)
    scale = np.repeat(np.exp2(exps.T.astype(float) - 127), 32, axis=1)
    assert (np.abs(held - v) <= np.maximum(np.abs(v) * 2.0 ** -4, scale * 2.0 ** -10)).all()
    assert exps[0, 3] == 1 and exps[0, 4] == 127 + 9 and exps[0, 5] == 128
    top = np.abs(v).reshape(64, 4, 32).max(axis=2).T
    some = top > 0
    assert (top <= 448.0 * np.exp2(exps.astype(float) - 127)).all()
    assert (top[some] > 448.0 * np.exp2(exps.astype(float) - 128)[some]).all()
    assert np.array_equal(ob.checkpoint_values(e4m3_code(e4m3_round((held / scale).astype(np.float32))), exps), held)

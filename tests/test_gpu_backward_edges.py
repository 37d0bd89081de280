"""GPU tests of the backward entry points on the data that they are least often given: entries that smoe_permute
skipped, NaN under the SwiGLU clamp, experts of more rows than an item. Helpers, oracle and the error bounds of
single operations are those of test_gpu_backward.py."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import oracle.backward as ob  # noqa: E402
import sparse_moe_layer_smoe_b200 as smoe  # noqa: E402
import test_gpu_backward as base  # noqa: E402
from oracle import moe  # noqa: E402
from test_gpu_backward import F, U, _bf16, _f32, _i32, _np, _within, _ws  # noqa: E402


def test_skipped_entries_have_no_gradient():
    """A repeated or invalid expert of a token gets no row (smoe_permute): its weight, its logit, the router's row and
    dx see none of it, and what remains is consistent: dw_router is the sum of dl x, dx has the sum of dl W_r."""
    T, H, E, k = 70, 256, 8, 4
    rng = np.random.default_rng(61)
    cfg = smoe.config(H, E, k, 128, 128, 3.0)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    idx[3, 1] = idx[3, 0]
    idx[8, 2], idx[9, 0], idx[9, 3] = -1, E, -7
    new = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")
    counts, offsets, perm_row, row_token = new(E), new(E + 1), new(T * k), new(T * k)
    smoe.smoe_permute(cfg, _i32(idx), T, None, counts, offsets, perm_row, row_token, None,
                      smoe.workspace(cfg, T, forward=False))
    skipped = (perm_row < 0).cpu().numpy().reshape(T, k)
    assert skipped.sum() == 4 and skipped[3, 1] and skipped[8, 2] and skipped[9, 0] and skipped[9, 3]
    x, x64 = _bf16(rng.normal(size=(T, H)))
    logits, l64 = _f32(rng.normal(size=(T, E)))
    w, w64 = _f32(rng.uniform(0.2, 1.0, size=(T, k)))
    dw, dw64 = _f32(np.where(skipped, 0.0, rng.normal(size=(T, k))))     # as smoe_combine_backward gives them
    dl, dwr = torch.full((T, k), 7.0, device="cuda"), torch.full((E, H), 7.0, device="cuda")
    ws = _ws(cfg, T)
    smoe.smoe_route_backward(cfg, x, T, logits, _i32(idx), w, dw, offsets, perm_row, row_token, dl, dwr, ws)
    assert smoe.smoe_get_device_error(ws) == smoe.SMOE_ERR_DEVICE
    e = np.clip(idx, 0, E - 1).astype(np.int64)
    rest = 1.0 - moe.sigmoid(np.take_along_axis(l64, e, 1))
    diff = dw64[:, :, None] - dw64[:, None, :]
    ref = np.where(skipped, 0.0, w64 * rest * ((w64 / 3.0)[:, None, :] * diff).sum(2))
    size = w64 * rest * ((w64 / 3.0)[:, None, :] * np.abs(diff)).sum(2)
    # the exponential is good to 2 F, the sum has k terms, and six more operations round
    _within(_np(dl), ref, np.where(skipped, 0.0, (k + 12) * F * size), "dlogits")
    dl64 = _np(dl)
    want, terms = np.zeros((E, H)), np.zeros((E, H))
    for j in range(k):
        np.add.at(want, e[:, j], dl64[:, j:j + 1] * x64)
        np.add.at(terms, e[:, j], np.abs(dl64[:, j:j + 1] * x64))
    _within(_np(dwr), want, (T + 2) * F * terms, "dw_router")
    # dx: no row and no router term of theirs
    dxr, dxr64 = _bf16(rng.normal(size=(T * k + T, H)))
    wr, wr64 = _f32(rng.normal(size=(E, H)))
    dx = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    ws = _ws(cfg, T)
    smoe.smoe_permute_backward(cfg, dxr, perm_row, _i32(idx), dl, wr, T, dx, ws)
    assert smoe.smoe_get_device_error(ws) == smoe.SMOE_ERR_DEVICE
    rows = np.where(skipped, 0, perm_row.cpu().numpy().reshape(T, k))
    got = np.where(skipped[:, :, None], 0.0, dxr64[rows])
    router = dl64[:, :, None] * wr64[e]
    ref = dxr64[T * k:] + got.sum(1) + router.sum(1)
    terms = np.abs(dxr64[T * k:]) + np.abs(got).sum(1) + np.abs(router).sum(1)
    _within(_np(dx), ref, np.abs(ref) * U + (2 * k + 2) * F * (1 + U) * terms, "dx")


@pytest.mark.parametrize("T,k", [(1, 32), (3, 32), (20, 4), (64, 8), (65, 4)])
def test_route_backward_of_one_expert_in_every_slot(T, k):
    """A caller's own permutation may give an expert more rows than there are tokens; every gradient is written."""
    H, E = 128, 40
    rng = np.random.default_rng(62)
    cfg = smoe.config(H, E, k, 128, 128, 3.0)
    idx = np.full((T, k), 5, dtype=np.int32)
    perm_row = rng.permutation(T * k).astype(np.int32)
    row_token = np.empty(T * k, dtype=np.int32)
    row_token[perm_row] = np.arange(T * k) // k
    offsets = np.where(np.arange(E + 1) > 5, T * k, 0)
    x, x64 = _bf16(rng.normal(size=(T, H)))
    logits, l64 = _f32(rng.normal(size=(T, E)))
    w, w64 = _f32(rng.uniform(0.2, 1.0, size=(T, k)))
    dw, dw64 = _f32(rng.normal(size=(T, k)))
    dl, dwr = torch.full((T, k), 7.0, device="cuda"), torch.full((E, H), 7.0, device="cuda")
    ws = _ws(cfg, T)
    smoe.smoe_route_backward(cfg, x, T, logits, _i32(idx), w, dw, _i32(offsets), _i32(perm_row), _i32(row_token), dl, dwr,
                             ws)
    assert smoe.smoe_get_device_error(ws) == 0
    rest = 1.0 - moe.sigmoid(l64[:, 5:6])
    diff = dw64[:, :, None] - dw64[:, None, :]
    size = w64 * rest * ((w64 / 3.0)[:, None, :] * np.abs(diff)).sum(2)
    _within(_np(dl), w64 * rest * ((w64 / 3.0)[:, None, :] * diff).sum(2), (k + 12) * F * size, "dlogits")
    dl64, got = _np(dl), _np(dwr)
    assert not np.delete(got, 5, axis=0).any()
    _within(got[5], dl64.sum(1) @ x64, (T * k + 2) * F * (np.abs(dl64).sum(1) @ np.abs(x64)), "dw_router")


# ------------------------------------------------------------------------------ NaN under the SwiGLU clamp
@pytest.mark.parametrize("name", ["clamp", "pairs_64"])
def test_a_nan_token_stays_nan_under_the_clamp(name):
    """The clamp of a NaN product is NaN, as the oracle's: the token's rows of y are NaN, the others' bits the same."""
    T, H, E, k, I, _, _ = base.SHAPES[name]
    rng = np.random.default_rng(63)
    r, cfg = base._routing(name, rng), base._cfg(name)
    packed, g64, u64, d64 = base._weights(name, rng)
    x, x_perm, _ = base._x(name, r, rng)

    def run(x, x_perm):
        n = T * k + T
        y, y2 = (torch.full((n, H), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        q = torch.empty(n, 2 * I, dtype=torch.uint8, device="cuda")
        sc = torch.empty(2 * I // 32, n, dtype=torch.uint8, device="cuda")
        args = (cfg, x, x_perm, _i32(r["row_token"]), _i32(r["offsets"]), T, packed)
        smoe.smoe_expert_ffn_save(*args, y, q, sc, _ws(cfg, T))
        smoe.smoe_expert_ffn(*args, y2, smoe.workspace(cfg, T, forward=False))
        assert torch.equal(y.view(torch.int16), y2.view(torch.int16))
        return y
    clean = run(x, x_perm)
    t = T // 2
    x[t] = float("nan")
    rows = torch.from_numpy(np.concatenate([r["row_token"], np.arange(T)]) == t).cuda()
    x_perm[rows[:T * k]] = float("nan")
    for given in (x_perm, None):
        y = run(x, given)
        assert torch.isnan(y[rows].float()).all()
        assert torch.equal(y[~rows].view(torch.int16), clean[~rows].view(torch.int16))


def test_a_nan_token_stays_nan_under_the_clamp_with_e4m3_experts():
    T, H, E, k, I, _, _ = base.SHAPES["clamp"]
    rng = np.random.default_rng(64)
    cfg = base._cfg("clamp")
    w = [_bf16(rng.normal(size=s) * 0.05)[0] for s in ((E, I, H), (E, I, H), (E, H, I), (I, H), (I, H), (H, I))]
    w[0][:, 7] = w[3][7] = float("nan")      # one gate feature of every expert
    packed = smoe.pack_weights_fp8(cfg, *w)
    x, (wr, _), (bias, _) = _bf16(rng.normal(size=(T, H)))[0], _f32(rng.normal(size=(E, H))), _f32(np.zeros(E))
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    smoe.smoe_forward_fp8(cfg, x, T, wr, bias, packed, out, smoe.workspace(cfg, T, fp8=True))
    assert torch.isnan(out.float()).all()


@pytest.mark.parametrize("name", ["clamp", "pairs_64"])
def test_nan_products_under_the_clamp_in_the_backward_pass(name):
    """Where the checkpoint holds NaN, h and the gradients that take it in are NaN as in the oracle: a NaN gate reaches
    h and du (and its own gradient is cut off: 0), a NaN up product h and dg. All others keep their bits."""
    T, H, E, k, I, _, _ = base.SHAPES[name]
    p = base._backward_inputs(name, np.random.default_rng(65))
    clean, ws = base._outputs(p["cfg"], T), _ws(p["cfg"], T)
    base._ffn_backward(p, T, clean, ws)
    b = base._bounds(p["r"], T, k)
    e = int(np.argmax(p["r"]["counts"]))
    at = [(b[e], 3), (b[e], I + 40), (b[E] + 1, 64), (b[E] + 2, I + 1)]     # row, column of (g, u)
    for row, col in at:
        p["q"][row, col] = 0x7F
        p["held"][row, col] = np.nan
    out = base._outputs(p["cfg"], T)
    base._ffn_backward(p, T, out, ws)
    g64, u64, d64 = p["W"]
    for grp, keys in ((e, "dw_"), (E, "dws_")):
        a, z = b[grp], b[grp + 1]
        dx, *dW = ob.expert_backward(p["rows64"][a:z], p["held"][a:z, :I], p["held"][a:z, I:], p["dy64"][a:z], g64[grp],
                                     u64[grp], d64[grp], base._limit(name, grp))
        got = [out["dx_rows"][a:z]] + [out[keys + q] if grp == E else out[keys + q][grp] for q in ("gate", "up", "down")]
        was = [clean["dx_rows"][a:z]] + [clean[keys + q] if grp == E else clean[keys + q][grp] for q in ("gate", "up", "down")]
        for key, v, old, ref in zip(("dx", "gate", "up", "down"), got, was, (dx, *dW)):
            nan = torch.from_numpy(np.isnan(ref)).cuda()
            # (a NaN up product reaches no gate gradient where the gate itself is cut off)
            assert nan.any() or key == "gate", key
            assert torch.equal(torch.isnan(v.float()), nan), (grp, key)
            if key == "dx":     # the rows without a NaN product are the same
                same = torch.tensor([i not in [row for row, _ in at] for i in range(a, z)], device="cuda")
                assert not nan[same].any()
                assert torch.equal(v[same].view(torch.int16), old[same].view(torch.int16)), (grp, key)
    others = [i for i in range(E) if i != e]
    for key in ("dw_gate", "dw_up", "dw_down"):
        assert torch.equal(out[key][others].view(torch.int16), clean[key][others].view(torch.int16)), key


@pytest.mark.parametrize("k", [1, 3, 5, 8])
def test_permute_backward_with_an_infinite_router_weight(k):
    """Slots past k (and skipped entries) add nothing: an infinite weight of a token's own expert stays infinite."""
    T, H, E = 20, 256, 24
    rng = np.random.default_rng(66)
    cfg = smoe.config(H, E, k, 128, 128, 3.0)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    perm_row = moe.permute(idx, E)[2]
    wr = rng.normal(size=(E, H))
    wr[:, 5], wr[:, 9] = np.inf, -np.inf
    (wr, wr64), (dl, dl64) = _f32(wr), _f32(np.abs(rng.normal(size=(T, k))) + 0.1)
    dxr, dxr64 = _bf16(rng.normal(size=(T * k + T, H)))
    dx = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    smoe.smoe_permute_backward(cfg, dxr, _i32(perm_row), _i32(idx), dl, wr, T, dx, _ws(cfg, T))
    got, ref = _np(dx), ob.permute_backward(dxr64, perm_row, idx, dl64, wr64)
    assert (got[:, 5] == np.inf).all() and (got[:, 9] == -np.inf).all()
    rest = np.isfinite(wr64[0])
    assert np.isfinite(got[:, rest]).all() and np.isfinite(ref[:, rest]).all()

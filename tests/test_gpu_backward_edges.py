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

"""GPU tests of the backward entry points and the 8-bit checkpoint against the fp64 oracle.

Tolerances. A rounding is off by at most half a step: U = 2^-8 of the value for bf16, F = 2^-24 for fp32.
A sum of n fp32 terms in any order is off by at most n F sum|terms|; the tensor cores may cut instead of
round, so their sums count 2 F a term. What is rounded to bf16 between two products (h, dg, du) carries U
of its value into the next one. Each bound below adds these terms up, computed in fp64 from the inputs.
Where the bound sums worst cases over many terms, the Frobenius norm is held too: independent roundings
to bf16 have an rms of at most U / sqrt(3), so two in a row stay under sqrt(2/3) U = 3.2e-3 of the norm;
5e-3 leaves half as much again for the oracle's operands not being independent."""
import ctypes

import numpy as np
import pytest

import oracle.backward as ob
from oracle import moe
from oracle.fp8 import e4m3_code, e4m3_decode, e4m3_round

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import sparse_moe_layer_smoe_b200 as smoe  # noqa: E402

U, F = 2.0 ** -8, 2.0 ** -24
FRO = 5e-3

# T, H, E, k, I, clamp, skew
SHAPES = {
    "one_token": (1, 512, 32, 4, 128, False, 0.0),
    "narrow": (17, 128, 8, 2, 128, False, 0.0),
    "tiny": (64, 512, 32, 4, 128, False, 0.0),
    "clamp": (64, 512, 32, 4, 128, True, 0.0),
    "all_experts": (33, 256, 4, 4, 256, False, 0.0),
    "one_slot": (50, 256, 6, 1, 128, False, 0.0),
    "many_slots": (40, 256, 40, 20, 128, False, 0.0),
    "largest_counts": (70, 128, 1024, 32, 128, False, 0.0),   # the most experts and slots
    "odd_widths": (257, 384, 5, 3, 384, False, 0.0),      # H, I odd multiples of 128, large token tiles
    "pairs": (600, 512, 4, 2, 256, False, 0.0),           # CTA pairs, 256-row tiles
    "pairs_64": (300, 256, 16, 3, 512, True, 0.0),        # CTA pairs, 64-row tiles
    "skewed": (700, 256, 24, 4, 256, False, 2.5),         # hot experts of several items, dead ones
}
LIMITS = (1.0, 1.5)


def _bf16(a):
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(torch.bfloat16)
    return t, t.double().cpu().numpy()


def _f32(a):
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()
    return t, t.double().cpu().numpy()


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _np(t):
    return t.double().cpu().numpy()


def _cfg(name):
    T, H, E, k, I, clamp, _ = SHAPES[name]
    return smoe.config(H, E, k, I, I, 3.0, *(LIMITS if clamp else (0.0, 0.0)))


def _limit(name, e):
    T, H, E, k, I, clamp, _ = SHAPES[name]
    return (LIMITS[1] if e == E else LIMITS[0]) if clamp else 0.0


def _routing(name, rng):
    T, H, E, k, I, _, skew = SHAPES[name]
    pop = -skew * np.log(np.arange(1, E + 1))
    noise = -np.log(-np.log(rng.uniform(1e-9, 1 - 1e-9, size=(T, E))))
    idx = np.argsort(-(pop + noise), axis=1, kind="stable")[:, :k].astype(np.int32)
    counts, offsets, perm_row, row_token = moe.permute(idx, E)
    logits = rng.normal(size=(T, E)).astype(np.float32).astype(np.float64)
    w = moe.normalise(np.take_along_axis(moe.sigmoid(logits), idx.astype(np.int64), 1), 3.0)
    return dict(idx=idx, offsets=offsets, perm_row=perm_row, row_token=row_token, logits=logits,
                w=w.astype(np.float32).astype(np.float64), counts=counts)


def _weights(name, rng):
    T, H, E, k, I, _, _ = SHAPES[name]
    (g, g64), (u, u64) = _bf16(rng.normal(size=(E + 1, I, H)) * 0.05), _bf16(rng.normal(size=(E + 1, I, H)) * 0.05)
    d, d64 = _bf16(rng.normal(size=(E + 1, H, I)) * 0.05)
    packed = smoe.pack_weights(_cfg(name), g[:E].contiguous(), u[:E].contiguous(), d[:E].contiguous(), g[E].contiguous(),
                               u[E].contiguous(), d[E].contiguous())
    return packed, g64, u64, d64


def _ws(cfg, T):
    return smoe.workspace(cfg, T, backward=True)


def _within(got, want, bound, what):
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - want) / bound):.3g} x its bound"


def _fro(got, want, what):
    n = np.linalg.norm(want)
    rel = np.linalg.norm(got - want) / n if n else np.abs(got).max(initial=0.0)
    assert rel <= FRO, f"{what}: relative Frobenius error {rel:.3e}"


# ------------------------------------------------------------------------------ combine, permute, route
@pytest.mark.parametrize("name", SHAPES)
def test_combine_backward(name):
    T, H, E, k, I, _, _ = SHAPES[name]
    rng = np.random.default_rng(11)
    r, cfg = _routing(name, rng), _cfg(name)
    dout, dout64 = _bf16(rng.normal(size=(T, H)) * 1e-3)
    y, y64 = _bf16(rng.normal(size=(T * k + T, H)))
    w, w64 = _f32(r["w"])
    dy = torch.full((T * k, H), 7.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((T, k), 7.0, device="cuda")
    ws = _ws(cfg, T)
    smoe.smoe_combine_backward(cfg, dout, y, _i32(r["perm_row"]), w, T, dy, dw, ws)
    assert smoe.smoe_get_device_error(ws) == 0
    dy_ref, dw_ref = ob.combine_backward(dout64, y64, r["perm_row"], w64)
    _within(_np(dy), dy_ref, np.abs(dy_ref) * (U + 2 * F), "dy")
    terms = np.einsum("th,tjh->tj", np.abs(dout64), np.abs(y64[r["perm_row"].reshape(T, k)]))
    _within(_np(dw), dw_ref, H * F * terms, "dtopk_w")


@pytest.mark.parametrize("router", [True, False])
@pytest.mark.parametrize("name", SHAPES)
def test_permute_backward(name, router):
    T, H, E, k, I, _, _ = SHAPES[name]
    rng = np.random.default_rng(12)
    r, cfg = _routing(name, rng), _cfg(name)
    dxr, dxr64 = _bf16(rng.normal(size=(T * k + T, H)))
    dl, dl64 = _f32(rng.normal(size=(T, k)))
    wr, wr64 = _f32(rng.normal(size=(E, H)))
    dx = torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = _ws(cfg, T)
    if router:
        smoe.smoe_permute_backward(cfg, dxr, _i32(r["perm_row"]), _i32(r["idx"]), dl, wr, T, dx, ws)
    else:
        smoe.smoe_permute_backward(cfg, dxr, _i32(r["perm_row"]), None, None, None, T, dx, ws)
    assert smoe.smoe_get_device_error(ws) == 0
    ref = ob.permute_backward(dxr64, r["perm_row"], r["idx"], dl64 if router else None, wr64)
    terms = ob.permute_backward(np.abs(dxr64), r["perm_row"], r["idx"], np.abs(dl64) if router else None, np.abs(wr64))
    _within(_np(dx), ref, np.abs(ref) * U + (2 * k + 2) * F * (1 + U) * terms, "dx")


@pytest.mark.parametrize("k", [1, 3, 5, 20])
def test_permute_backward_reads_no_other_experts_weights(k):
    """Experts that a token did not choose may hold anything, expert 0 too."""
    T, H, E = 20, 128, 24
    cfg = smoe.config(H, E, k, 128, 128, 3.0)
    rng = np.random.default_rng(15)
    idx = np.stack([1 + rng.permutation(E - 2)[:k] for _ in range(T)]).astype(np.int32)   # never 0 or E - 1
    perm_row = moe.permute(idx, E)[2]
    wr, wr64 = _f32(rng.normal(size=(E, H)))
    wr[0], wr[E - 1] = float("inf"), float("nan")
    dxr, dxr64 = _bf16(rng.normal(size=(T * k + T, H)))
    dl, dl64 = _f32(rng.normal(size=(T, k)))
    dx = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    smoe.smoe_permute_backward(cfg, dxr, _i32(perm_row), _i32(idx), dl, wr, T, dx, _ws(cfg, T))
    ref = ob.permute_backward(dxr64, perm_row, idx, dl64, wr64)
    terms = ob.permute_backward(np.abs(dxr64), perm_row, idx, np.abs(dl64), np.abs(wr64))
    _within(_np(dx), ref, np.abs(ref) * U + (2 * k + 2) * F * (1 + U) * terms, "dx")


def _route_backward(name, rng, r=None):
    T, H, E, k, I, _, _ = SHAPES[name]
    r, cfg = r or _routing(name, rng), _cfg(name)
    x, x64 = _bf16(rng.normal(size=(T, H)))
    logits, logits64 = _f32(r["logits"])
    w, _ = _f32(r["w"])
    dw, dw64 = _f32(rng.normal(size=(T, k)))
    dl = torch.full((T, k), 7.0, device="cuda")
    dwr = torch.full((E, H), 7.0, device="cuda")
    ws = _ws(cfg, T)
    smoe.smoe_route_backward(cfg, x, T, logits, _i32(r["idx"]), w, dw, _i32(r["offsets"]), _i32(r["perm_row"]),
                             _i32(r["row_token"]), dl, dwr, ws)
    return r, x64, logits64, dw64, dl, dwr, ws


@pytest.mark.parametrize("name", SHAPES)
def test_route_backward(name):
    T, H, E, k, I, _, _ = SHAPES[name]
    r, x64, logits64, dw64, dl, dwr, ws = _route_backward(name, np.random.default_rng(13))
    assert smoe.smoe_get_device_error(ws) == 0
    dl_ref, dwr_ref = ob.route_backward(x64, logits64, r["idx"], dw64, 3.0)
    # the given w are fp32 roundings of the oracle's (F each, in w_j and under the sum), the exponential is good
    # to 2 F, the sum has k terms, and six more operations round
    w = r["w"]
    rest = 1.0 - moe.sigmoid(np.take_along_axis(logits64, r["idx"].astype(np.int64), 1))
    size = w * rest * ((w / 3.0)[:, None, :] * np.abs(dw64[:, :, None] - dw64[:, None, :])).sum(2)
    # (the oracle's quotient rule subtracts terms of size w |dw| in fp64: 8 roundings of 2^-53 of those are its own)
    e_dl = (k + 12) * F * size + 2.0 ** -50 * w * np.abs(dw64).max(axis=1, keepdims=True)
    _within(_np(dl), dl_ref, e_dl, "dlogits")
    # a sum over an expert's rows: at most counts terms, each with dl's own error
    terms, carried = np.zeros((E, H)), np.zeros((E, H))
    for j in range(k):
        np.add.at(terms, r["idx"][:, j], np.abs(dl_ref[:, j:j + 1] * x64))
        np.add.at(carried, r["idx"][:, j], e_dl[:, j:j + 1] * np.abs(x64))
    _within(_np(dwr), dwr_ref, (r["counts"][:, None] + 2) * F * (terms + carried) + carried + 1e-300,
            "dw_router")
    if k == 1:
        assert not _np(dl).any() and not _np(dwr).any()
    assert not _np(dwr)[r["counts"] == 0].any()


def test_route_backward_with_far_logits():
    """Scores next to 0 and 1: 1 - s keeps its relative precision, exp(88) and above give gradients of 0."""
    name = "tiny"
    T, H, E, k, I, _, _ = SHAPES[name]
    rng = np.random.default_rng(14)
    r = _routing(name, rng)
    r["logits"] = (rng.uniform(-30, 30, size=(T, E))).astype(np.float32).astype(np.float64)
    r["logits"][0] = 95.0
    w = moe.normalise(np.take_along_axis(moe.sigmoid(r["logits"]), r["idx"].astype(np.int64), 1), 3.0)
    r["w"] = w.astype(np.float32).astype(np.float64)
    r, x64, logits64, dw64, dl, dwr, ws = _route_backward(name, rng, r)
    dl_ref, _ = ob.route_backward(x64, logits64, r["idx"], dw64, 3.0)
    with np.errstate(over="ignore"):
        rest = 1.0 / (1.0 + np.exp(np.take_along_axis(logits64, r["idx"].astype(np.int64), 1)))
    ref = r["w"] * rest * ((r["w"] / 3.0)[:, None, :] * (dw64[:, :, None] - dw64[:, None, :])).sum(2)
    size = r["w"] * rest * ((r["w"] / 3.0)[:, None, :] * np.abs(dw64[:, :, None] - dw64[:, None, :])).sum(2)
    _within(_np(dl), ref, (k + 12) * F * size + 2.0 ** -126, "dlogits")   # 2^-126: the least normal fp32
    assert not _np(dl)[0].any() and np.isfinite(_np(dwr)).all()
    # the oracle's own form agrees where 1 - s is not lost to cancellation
    near = np.abs(np.take_along_axis(logits64, r["idx"].astype(np.int64), 1)) < 10
    assert np.allclose(ref[near], dl_ref[near], rtol=1e-6, atol=1e-9)


# ------------------------------------------------------------------------------ experts
def _x(name, r, rng):
    T, H, E, k, I, _, _ = SHAPES[name]
    x, x64 = _bf16(rng.normal(size=(T, H)))
    return x, x[torch.from_numpy(r["row_token"]).long().cuda()].contiguous(), np.concatenate([x64[r["row_token"]], x64])


def _bounds(r, T, k):
    return list(r["offsets"]) + [T * k + T]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("name", SHAPES)
def test_expert_ffn_save(name, gather):
    T, H, E, k, I, _, _ = SHAPES[name]
    rng = np.random.default_rng(21)
    r, cfg = _routing(name, rng), _cfg(name)
    packed, g64, u64, _ = _weights(name, rng)
    x, x_perm, rows64 = _x(name, r, rng)
    n = T * k + T
    y, y2 = (torch.full((n, H), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.full((n, 2 * I), 0x55, dtype=torch.uint8, device="cuda")
    sc = torch.full((2 * I // 32, n), 0x55, dtype=torch.uint8, device="cuda")
    gu = torch.empty(n, 2 * I, dtype=torch.bfloat16, device="cuda")
    ws = _ws(cfg, T)
    args = (cfg, x, None if gather else x_perm, _i32(r["row_token"]), _i32(r["offsets"]), T, packed)
    smoe.smoe_expert_ffn_save(*args, y, q, sc, ws)
    smoe.smoe_expert_ffn(*args, y2, smoe.workspace(cfg, T, forward=False))
    smoe.smoe_checkpoint_values(cfg, q, sc, T, gu)
    assert smoe.smoe_get_device_error(ws) == 0
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16))
    exps = sc.cpu().numpy()
    held = ob.checkpoint_values(q.cpu().numpy(), exps)
    assert np.array_equal(_np(gu), held)          # bf16 holds them exactly
    scale = np.repeat(np.exp2(exps.T.astype(float) - 127), 32, axis=1)
    b = _bounds(r, T, k)
    ref, err = np.zeros((n, 2 * I)), np.zeros((n, 2 * I))
    for e in range(E + 1):
        X = rows64[b[e]:b[e + 1]]
        W = np.concatenate([g64[e], u64[e]])
        ref[b[e]:b[e + 1]] = X @ W.T
        err[b[e]:b[e + 1]] = 2 * H * F * (np.abs(X) @ np.abs(W).T)
    _within(held, ref, err + np.maximum((np.abs(ref) + err) * 2.0 ** -4, scale * 2.0 ** -10), "checkpoint")
    # the scale is the oracle's wherever the largest magnitude is not within the sum's error of a power's edge
    blocks = lambda v: v.reshape(n, -1, 32)
    top, te = np.abs(blocks(ref)).max(2).T, blocks(err).max(2).T
    assert (top - te <= 448.0 * np.exp2(exps.astype(float) - 127)).all()
    assert ((top + te > 448.0 * np.exp2(exps.astype(float) - 128)) | (exps <= 1)).all()


def test_checkpoint_of_extreme_products():
    """Products that are 0, infinite or NaN in one feature: infinite and NaN products are held as such in a
    block of scale 2^120, the row's other blocks are unaffected."""
    name = "tiny"
    T, H, E, k, I, _, _ = SHAPES[name]
    rng = np.random.default_rng(22)
    r, cfg = _routing(name, rng), _cfg(name)
    x, x_perm, rows64 = _x(name, r, rng)
    g, u, d = (rng.normal(size=s) * 0.05 for s in ((E + 1, I, H), (E + 1, I, H), (E + 1, H, I)))
    g[:, 32:64] = 0.0                 # a block of zeros
    g[:, 5], u[:, 70] = np.inf, np.nan
    g[:, 96:128] *= 1e30              # a large scale
    u[:, 0:32] *= 1e-30               # a small one
    (tg, g64), (tu, u64), (td, _) = _bf16(g), _bf16(u), _bf16(d)
    packed = smoe.pack_weights(cfg, tg[:E].contiguous(), tu[:E].contiguous(), td[:E].contiguous(), tg[E].contiguous(),
                               tu[E].contiguous(), td[E].contiguous())
    n = T * k + T
    y = torch.empty(n, H, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(n, 2 * I, dtype=torch.uint8, device="cuda")
    sc = torch.empty(2 * I // 32, n, dtype=torch.uint8, device="cuda")
    smoe.smoe_expert_ffn_save(cfg, x, x_perm, _i32(r["row_token"]), _i32(r["offsets"]), T, packed, y, q, sc, _ws(cfg, T))
    exps = sc.cpu().numpy()
    held = ob.checkpoint_values(q.cpu().numpy(), exps)
    # an infinity has the exponent of 448 * 2^120, NaN's all-ones mantissa carries into the next; 448 * 2^120 is
    # infinite in fp32, which is what the values are read as (as is inf - inf = NaN)
    assert not np.isfinite(held[:, 5].astype(np.float32)).any() and np.isnan(held[:, I + 70]).all()
    assert np.isin(exps[[0, I // 32 + 2]], (247, 248)).all()
    assert (exps[1] == 1).all() and not held[:, 32:64].any()
    b = _bounds(r, T, k)
    for e in range(E + 1):
        X = rows64[b[e]:b[e + 1]]
        W = np.concatenate([g64[e], u64[e]])
        fine = np.isfinite(W).all(1)
        fine[0:32] = fine[I + 64:I + 96] = False      # the blocks of the infinite and the NaN feature
        ref = X @ np.where(fine[:, None], W, 0.0).T
        err = 2 * H * F * (np.abs(X) @ np.abs(np.where(fine[:, None], W, 0.0)).T)
        scale = np.repeat(np.exp2(exps.T[b[e]:b[e + 1]].astype(float) - 127), 32, axis=1)
        bound = err + np.maximum((np.abs(ref) + err) * 2.0 ** -4, scale * 2.0 ** -10)
        _within(held[b[e]:b[e + 1]][:, fine], ref[:, fine], bound[:, fine], f"group {e}")


def _backward_inputs(name, rng, r=None):
    T, H, E, k, I, _, _ = SHAPES[name]
    r, cfg = r or _routing(name, rng), _cfg(name)
    packed, g64, u64, d64 = _weights(name, rng)
    x, x_perm, rows64 = _x(name, r, rng)
    n = T * k + T
    held, exps = ob.checkpoint(rng.normal(size=(n, 2 * I)).astype(np.float32))
    scale = np.repeat(np.exp2(exps.T.astype(float) - 127), 32, axis=1)
    q = torch.from_numpy(e4m3_code(e4m3_round((held / scale).astype(np.float32)))).cuda()
    dy, dy64 = _bf16(rng.normal(size=(T * k, H)) * 1e-2)
    dout, dout64 = _bf16(rng.normal(size=(T, H)) * 1e-2)
    return dict(r=r, cfg=cfg, packed=packed, W=(g64, u64, d64), x=x, x_perm=x_perm, rows64=rows64, held=held, q=q,
                sc=torch.from_numpy(np.ascontiguousarray(exps)).cuda(), dy=dy, dout=dout,
                dy64=np.concatenate([dy64, dout64]), offsets=_i32(r["offsets"]))


def _outputs(cfg, T, fill=7.0):
    H, E, I, n = cfg.hidden, cfg.n_experts, cfg.inter, T * cfg.top_k + T
    shapes = dict(dx_rows=(n, H), dw_gate=(E, I, H), dw_up=(E, I, H), dw_down=(E, H, I), dws_gate=(I, H), dws_up=(I, H),
                  dws_down=(H, I))
    return {a: torch.full(s, fill, dtype=torch.bfloat16, device="cuda") for a, s in shapes.items()}


def _ffn_backward(p, T, out, ws, stream=None):
    smoe.smoe_expert_ffn_backward(p["cfg"], p["x"], p["x_perm"], p["offsets"], T, p["packed"], p["q"], p["sc"], p["dy"],
                                  p["dout"], *out.values(), ws, stream=stream)


def _check_ffn_backward(name, p, out):
    T, H, E, k, I, _, _ = SHAPES[name]
    b = _bounds(p["r"], T, k)
    g64, u64, d64 = p["W"]
    o = {a: _np(t) for a, t in out.items()}
    refs = {a: np.zeros_like(v) for a, v in o.items()}
    ends = {a: np.zeros_like(v) for a, v in o.items()}
    for e in range(E + 1):
        a, z = b[e], b[e + 1]
        g, u = p["held"][a:z, :I], p["held"][a:z, I:]
        X, dy = p["rows64"][a:z], p["dy64"][a:z]
        lim = _limit(name, e)
        dx, *dW = ob.expert_backward(X, g, u, dy, g64[e], u64[e], d64[e], lim)
        h, dg, du = ob.swiglu_backward(g, u, dy @ d64[e], lim)
        # dh's own sum (H terms), carried by the slopes of dg and du in dh; 16 F for the exponential, the
        # quotient and the products; then the rounding to bf16
        e_dh = 2 * H * F * (np.abs(dy) @ np.abs(d64[e]))
        _, slope_g, slope_u = ob.swiglu_backward(g, u, np.ones_like(g), lim)
        sg = np.abs(slope_g) + 16 * F * (1 + np.abs(g)) * np.abs(u)
        e_dg = sg * e_dh + (1 + np.abs(g)) * np.abs(u) * np.abs(dy @ d64[e]) * 16 * F + np.abs(dg) * U * (1 + U)
        e_du = np.abs(slope_u) * e_dh + np.abs(du) * (16 * F + U)
        e_h = np.abs(h) * (16 * F + U)
        n = z - a

        def product(A, eA, B, terms):   # error of A^T B, A off by eA, B exact
            return (eA + 2 * terms * F * (np.abs(A) + eA)).T @ np.abs(B)
        bound = {"dx": product(dg.T, e_dg.T, g64[e], 2 * I) + product(du.T, e_du.T, u64[e], 2 * I),
                 "dw_gate": product(dg, e_dg, X, n), "dw_up": product(du, e_du, X, n),
                 "dw_down": product(h, e_h, dy, n).T}
        refs["dx_rows"][a:z], ends["dx_rows"][a:z] = dx, bound["dx"]
        for w, key in zip(dW, ("gate", "up", "down")):
            if e == E:
                refs["dws_" + key], ends["dws_" + key] = w, bound["dw_" + key]
            else:
                refs["dw_" + key][e], ends["dw_" + key][e] = w, bound["dw_" + key]
    for key in o:
        _within(o[key], refs[key], ends[key] + U * (np.abs(refs[key]) + ends[key]) + 1e-300, key)
        _fro(o[key], refs[key], key)
    dead = p["r"]["counts"] == 0
    for key in ("dw_gate", "dw_up", "dw_down"):
        assert not o[key][dead].any()


@pytest.mark.parametrize("name", SHAPES)
def test_expert_ffn_backward(name):
    T = SHAPES[name][0]
    p = _backward_inputs(name, np.random.default_rng(31))
    out, ws = _outputs(p["cfg"], T), _ws(p["cfg"], T)
    _ffn_backward(p, T, out, ws)
    assert smoe.smoe_get_device_error(ws) == 0
    _check_ffn_backward(name, p, out)
    again = _outputs(p["cfg"], T, fill=-3.0)
    _ffn_backward(p, T, again, ws)
    for a in out:
        assert torch.equal(out[a].view(torch.int16), again[a].view(torch.int16)), a


@pytest.mark.parametrize("name", ["tiny", "pairs", "odd_widths"])
def test_infinite_and_nan_rows_stay_with_their_expert(name):
    """Tiles and row steps of one expert reach into the next expert's rows: those may hold anything."""
    T, H, E, k, I, _, _ = SHAPES[name]
    p = _backward_inputs(name, np.random.default_rng(32))
    clean, ws = _outputs(p["cfg"], T), _ws(p["cfg"], T)
    _ffn_backward(p, T, clean, ws)
    off = p["r"]["offsets"]
    bad = [e for e in range(E) if off[e + 1] > off[e]][1::2]
    for e in bad:
        p["dy"][off[e]:off[e + 1]] = float("nan")
        p["x_perm"][off[e]:off[e + 1]] = float("inf")
        p["q"][off[e]:off[e + 1]] = 0x7F
    p["dout"][T - 1] = float("inf")      # behind all routed rows
    out = _outputs(p["cfg"], T)
    _ffn_backward(p, T, out, ws)
    good = [e for e in range(E) if e not in bad]
    for key in ("dw_gate", "dw_up", "dw_down"):
        assert torch.equal(out[key][good].view(torch.int16), clean[key][good].view(torch.int16)), key
        assert not torch.isfinite(out[key][bad].float()).any(), key
    rows = [i for e in good for i in range(off[e], off[e + 1])]
    assert torch.equal(out["dx_rows"][rows].view(torch.int16), clean["dx_rows"][rows].view(torch.int16))


# ------------------------------------------------------------------------------ the chain, as a training step runs it
def _chain(cfg, x, wr, bias, packed, dout, ws, stream=None):
    T, H, E, k, I = x.shape[0], cfg.hidden, cfg.n_experts, cfg.top_k, cfg.inter
    n, R = T * k + T, T * k
    new = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device="cuda")
    f, i32 = torch.float32, torch.int32
    idx, w, logits = new(T, k, dt=i32), new(T, k, dt=f), new(T, E, dt=f)
    counts, offsets, perm_row, row_token = new(E, dt=i32), new(E + 1, dt=i32), new(R, dt=i32), new(R, dt=i32)
    x_perm, y, q, sc, out = new(R, H), new(n, H), new(n, 2 * I, dt=torch.uint8), new(2 * I // 32, n, dt=torch.uint8), new(T, H)
    s = dict(ws=ws, stream=stream)
    smoe.smoe_route(cfg, x, T, wr, bias, idx, w, logits, **s)
    smoe.smoe_permute(cfg, idx, T, x, counts, offsets, perm_row, row_token, x_perm, **s)
    smoe.smoe_expert_ffn_save(cfg, x, x_perm, row_token, offsets, T, packed, y, q, sc, **s)
    smoe.smoe_combine(cfg, y, perm_row, w, T, out, **s)
    dy, dw, dl, dwr, dx = new(R, H), new(T, k, dt=f), new(T, k, dt=f), new(E, H, dt=f), new(T, H)
    grads = _outputs(cfg, T)
    smoe.smoe_combine_backward(cfg, dout, y, perm_row, w, T, dy, dw, **s)
    smoe.smoe_expert_ffn_backward(cfg, x, x_perm, offsets, T, packed, q, sc, dy, dout, *grads.values(), **s)
    smoe.smoe_route_backward(cfg, x, T, logits, idx, w, dw, offsets, perm_row, row_token, dl, dwr, **s)
    smoe.smoe_permute_backward(cfg, grads["dx_rows"], perm_row, idx, dl, wr, T, dx, **s)
    return dict(out=out, dx=dx, dwr=dwr, idx=idx, q=q, sc=sc, **grads)


def _chain_inputs(name, seed):
    T, H, E, k, I, _, _ = SHAPES[name]
    rng = np.random.default_rng(seed)
    packed, g64, u64, d64 = _weights(name, rng)
    x, x64 = _bf16(rng.normal(size=(T, H)))
    wr, wr64 = _f32(rng.normal(size=(E, H)) * 0.05)
    dout, dout64 = _bf16(rng.normal(size=(T, H)))
    bias, bias64 = _f32(rng.normal(size=E) * 0.1)
    return packed, (g64, u64, d64), x, x64, wr, wr64, dout, dout64, bias, bias64


@pytest.mark.parametrize("name", ["tiny", "clamp", "pairs", "one_slot"])
def test_training_step_against_the_oracle(name):
    """All gradients of <dout, layer(x)>, with the checkpoint's values in the experts' backward pass. y, dy and
    the rows of dx are rounded to bf16 on the way, each within U of its value: three roundings in a row
    have an rms of at most U, and the norms are held to 1.5 U."""
    T, H, E, k, I, _, _ = SHAPES[name]
    packed, W, x, x64, wr, wr64, dout, dout64, bias, bias64 = _chain_inputs(name, 41)
    cfg = _cfg(name)
    ws = _ws(cfg, T)
    o = _chain(cfg, x, wr, bias, packed, dout, ws)
    assert smoe.smoe_get_device_error(ws) == 0
    r = moe.route(x64, wr64, bias64, k, 3.0)
    assert not r.near_tie.any() and np.array_equal(np.sort(_np(o["idx"]), 1), np.sort(r.idx, 1))
    lim = lambda e: _limit(name, e)
    idx = _np(o["idx"]).astype(np.int32)
    _, offsets, perm_row, row_token = moe.permute(idx, E)
    w = moe.normalise(np.take_along_axis(r.s, idx.astype(np.int64), 1), 3.0)
    xr = np.concatenate([x64[row_token], x64])
    b = list(offsets) + [T * k + T]
    held = ob.checkpoint_values(o["q"].cpu().numpy(), o["sc"].cpu().numpy())
    y = np.zeros((T * k + T, H))
    for e in range(E + 1):
        y[b[e]:b[e + 1]] = moe.swiglu_ffn(xr[b[e]:b[e + 1]], *(m[e] for m in W), limit=lim(e))
    dy, dw = ob.combine_backward(dout64, y, perm_row, w)
    dl, dwr = ob.route_backward(x64, r.logits, idx, dw, 3.0)
    dy = np.concatenate([dy, dout64])
    dxr = np.zeros((T * k + T, H))
    dW = [np.zeros((E + 1,) + m.shape[1:]) for m in W]
    for e in range(E + 1):
        a, z = b[e], b[e + 1]
        dxr[a:z], *d = ob.expert_backward(xr[a:z], held[a:z, :I], held[a:z, I:], dy[a:z], *(m[e] for m in W), limit=lim(e))
        for at, v in zip(dW, d):
            at[e] = v
    dx = ob.permute_backward(dxr, perm_row, idx, dl, wr64)

    def norm(got, want, what):
        n = np.linalg.norm(want)
        rel = np.linalg.norm(got - want) / n if n > 1e-12 else np.abs(got - want).max()
        assert rel <= 1.5 * U, f"{what}: {rel:.3e}"
    norm(_np(o["dx"]), dx, "dx")
    norm(_np(o["dwr"]), dwr, "dw_router")
    for key, at in zip(("gate", "up", "down"), dW):
        norm(_np(o["dw_" + key]), at[:E], key)
        norm(_np(o["dws_" + key]), at[E], "shared " + key)


def test_kernel_times_and_launch_counts():
    name = "tiny"
    T = SHAPES[name][0]
    packed, W, x, x64, wr, wr64, dout, dout64, bias, _ = _chain_inputs(name, 45)
    cfg = _cfg(name)
    layer = smoe.MoELayer(cfg, wr, bias, packed)
    ws = _ws(cfg, T)
    smoe.smoe_timing_begin(100)
    _, saved = layer.forward_train(x, ws)
    layer.backward(saved, dout, ws)
    assert smoe.smoe_last_launch_count() == 1      # permute_backward
    smoe.smoe_checkpoint_values(cfg, saved["gu_q"], saved["gu_scale"], T,
                                torch.empty(T * cfg.top_k + T, 2 * cfg.inter, dtype=torch.bfloat16, device="cuda"))
    times = smoe.smoe_timing_end()
    for kernel in ("expert_gateup_save", "expert_down", "combine_backward", "expert_dh", "expert_dx", "expert_wgrad",
                   "router_backward", "permute_backward", "checkpoint_values"):
        launches, ms = times[kernel]
        assert launches == 1 and 0 < ms < 1000, kernel


def test_layer_training_methods_are_the_chain():
    name = "tiny"
    T = SHAPES[name][0]
    packed, W, x, x64, wr, wr64, dout, dout64, bias, _ = _chain_inputs(name, 44)
    cfg = _cfg(name)
    want = _chain(cfg, x, wr, bias, packed, dout, _ws(cfg, T))
    layer = smoe.MoELayer(cfg, wr, bias, packed)
    out, saved = layer.forward_train(x)
    got = dict(layer.backward(saved, dout), out=out)
    got["dwr"] = got.pop("dw_router")
    for key, v in got.items():
        assert torch.equal(v.view(torch.uint8), want[key].view(torch.uint8)), key
    for t in (0, 1):      # no tokens, and one
        o, s = layer.forward_train(x[:t].contiguous())
        g = layer.backward(s, dout[:t].contiguous())
        assert o.shape == (t, cfg.hidden) and g["dx"].shape == (t, cfg.hidden)
        assert all(torch.isfinite(v.float()).all() for v in g.values())
        assert t or not any(g[key].any() for key in g if key.startswith("dw"))


@pytest.mark.parametrize("name", ["tiny", "pairs"])
def test_training_step_captured_and_on_another_stream(name):
    """The chain captured into a graph and replayed twice, and run on a side stream, gives the eager bits."""
    T = SHAPES[name][0]
    packed, W, x, x64, wr, wr64, dout, dout64, bias, _ = _chain_inputs(name, 42)
    cfg = _cfg(name)
    ws = _ws(cfg, T)
    eager = _chain(cfg, x, wr, bias, packed, dout, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = _chain(cfg, x, wr, bias, packed, dout, ws)
    given = _chain(cfg, x, wr, bias, packed, dout, ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = _chain(cfg, x, wr, bias, packed, dout, ws)
    for _ in range(2):
        for v in captured.values():
            v.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for key in eager:
        for got in (other, given, captured):
            assert torch.equal(eager[key].view(torch.uint8), got[key].view(torch.uint8)), key
    # other inputs in the captured tensors
    x.copy_(_bf16(np.random.default_rng(43).normal(size=x.shape))[0])
    graph.replay()
    want = _chain(cfg, x, wr, bias, packed, dout, ws)
    torch.cuda.synchronize()
    for key in want:
        assert torch.equal(want[key].view(torch.uint8), captured[key].view(torch.uint8)), key


@pytest.mark.parametrize("raw", [False, True])
def test_layer_training_methods_own_memory_on_the_given_stream(raw):
    """While the given stream is busy, the current one allocates and fills as much memory as the methods used: it
    gets none of theirs, which work queued on the given stream still needs."""
    name = "tiny"
    T = SHAPES[name][0]
    packed, W, x, x64, wr, wr64, dout, dout64, bias, _ = _chain_inputs(name, 45)
    cfg = _cfg(name)
    layer = smoe.MoELayer(cfg, wr, bias, packed)
    out, saved = layer.forward_train(x)
    want = dict(layer.backward(saved, dout), out=out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    given = side.cuda_stream if raw else side

    def fill():
        return [torch.zeros(n, dtype=torch.uint8, device="cuda")
                for n in (4 * cfg.n_experts, _ws(cfg, T).numel(), *(v.numel() * v.element_size() for v in want.values()))
                for _ in range(4)]

    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    out, saved = layer.forward_train(x, stream=given)
    kept = fill()
    got = dict(layer.backward(saved, dout, stream=given), out=out)
    kept += fill()
    torch.cuda.current_stream().wait_stream(side)
    for key, v in got.items():
        assert torch.equal(v.view(torch.uint8), want[key].view(torch.uint8)), key
    assert not any(v.any() for v in kept)


# ------------------------------------------------------------------------------ bad data, edges
def test_bad_rows_are_skipped_and_recorded():
    name = "tiny"
    T, H, E, k, I, _, _ = SHAPES[name]
    rng = np.random.default_rng(51)
    r, cfg = _routing(name, rng), _cfg(name)
    bad = r["perm_row"].copy()
    bad[5], bad[9] = T * k + 3, -1
    skipped = {int(r["perm_row"][5]), int(r["perm_row"][9])}
    dout, dout64 = _bf16(rng.normal(size=(T, H)))
    y, y64 = _bf16(rng.normal(size=(T * k + T, H)))
    w, w64 = _f32(r["w"])
    dy = torch.full((T * k, H), 7.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((T, k), 7.0, device="cuda")
    ws = _ws(cfg, T)
    smoe.smoe_combine_backward(cfg, dout, y, _i32(bad), w, T, dy, dw, ws)
    assert smoe.smoe_get_device_error(ws) == smoe.SMOE_ERR_DEVICE
    dy_ref, dw_ref = ob.combine_backward(dout64, y64, r["perm_row"], w64)
    got = _np(dy)
    for i in skipped:
        assert (got[i] == 7.0).all()
    keep = [i for i in range(T * k) if i not in skipped]
    assert (np.abs(got[keep] - dy_ref[keep]) <= np.abs(dy_ref[keep]) * (U + 2 * F)).all()
    flat = _np(dw).reshape(-1)
    assert flat[5] == 0 and flat[9] == 0 and np.allclose(np.delete(flat, [5, 9]), np.delete(dw_ref.reshape(-1), [5, 9]),
                                                         rtol=1e-4, atol=1e-4)
    # permute: the skipped entries' rows and an expert out of range add nothing
    idx = r["idx"].copy()
    idx[7, 0] = E
    dxr, dxr64 = _bf16(rng.normal(size=(T * k + T, H)))
    dl, dl64 = _f32(rng.normal(size=(T, k)))
    wr, wr64 = _f32(rng.normal(size=(E, H)))
    dx = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    ws = _ws(cfg, T)
    smoe.smoe_permute_backward(cfg, dxr, _i32(bad), _i32(idx), dl, wr, T, dx, ws)
    assert smoe.smoe_get_device_error(ws) == smoe.SMOE_ERR_DEVICE
    dl64[7, 0], idx[7, 0] = 0.0, 0
    ref = ob.permute_backward(dxr64, r["perm_row"], idx, dl64, wr64)
    for e in (5, 9):
        ref[e // k] -= dxr64[r["perm_row"][e]]
    terms = ob.permute_backward(np.abs(dxr64), r["perm_row"], idx, np.abs(dl64), np.abs(wr64))
    _within(_np(dx), ref, np.abs(ref) * U + (2 * k + 2) * F * (1 + U) * terms, "dx")


def test_corrupt_offsets_give_no_routed_work():
    name = "tiny"
    T, H, E, k, I, _, _ = SHAPES[name]
    p = _backward_inputs(name, np.random.default_rng(52))
    good, ws = _outputs(p["cfg"], T), _ws(p["cfg"], T)
    _ffn_backward(p, T, good, ws)
    bad = p["r"]["offsets"].copy()
    bad[3], bad[4] = bad[4] + 5, bad[3]
    for off in (bad, bad * 0 + 2 ** 30, -p["r"]["offsets"]):
        p["offsets"] = _i32(off)
        out, ws2 = _outputs(p["cfg"], T), _ws(p["cfg"], T)
        _ffn_backward(p, T, out, ws2)
        assert smoe.smoe_get_device_error(ws2) == smoe.SMOE_ERR_DEVICE
        for key in ("dw_gate", "dw_up", "dw_down"):
            assert not out[key].any()
        for key in ("dws_gate", "dws_up", "dws_down"):
            assert torch.equal(out[key], good[key])
        assert (out["dx_rows"][:T * k] == 7.0).all() and torch.equal(out["dx_rows"][T * k:], good["dx_rows"][T * k:])
    r = _routing(name, np.random.default_rng(53))
    keep = r["offsets"].copy()
    for off in (bad, -keep):
        r["offsets"] = off
        *_, dl, dwr, ws3 = _route_backward(name, np.random.default_rng(54), r)
        assert smoe.smoe_get_device_error(ws3) == smoe.SMOE_ERR_DEVICE
        assert not dwr.any()


def test_rows_behind_the_last_entry_stay_as_they_were():
    """With skipped entries offsets[E] < T*k: the rows behind are neither read nor written."""
    name = "tiny"
    T, H, E, k, I, _, _ = SHAPES[name]
    rng = np.random.default_rng(55)
    idx = _routing(name, rng)["idx"]
    idx[3, 1] = idx[3, 0]
    idx[8, 2] = -1
    cfg = _cfg(name)
    new = lambda n: torch.full((n,), -5, dtype=torch.int32, device="cuda")
    counts, offsets, perm_row, row_token = new(E), new(E + 1), new(T * k), new(T * k)
    smoe.smoe_permute(cfg, _i32(idx), T, None, counts, offsets, perm_row, row_token, None,
                      smoe.workspace(cfg, T, forward=False))
    end = int(offsets[E])
    assert end == T * k - 2
    p = _backward_inputs(name, rng)
    p["offsets"] = offsets
    for t in (p["dy"], p["x_perm"]):
        t[end:] = float("nan")
    p["q"][end:T * k] = 0x7F
    out, ws = _outputs(cfg, T), _ws(cfg, T)
    _ffn_backward(p, T, out, ws)
    assert (out["dx_rows"][end:T * k] == 7.0).all()
    for key, v in out.items():
        assert torch.isfinite(v.float()).all(), key
    y = torch.full((T * k + T, H), 7.0, dtype=torch.bfloat16, device="cuda")
    q = torch.full((T * k + T, 2 * I), 0x55, dtype=torch.uint8, device="cuda")
    sc = torch.full((2 * I // 32, T * k + T), 0x55, dtype=torch.uint8, device="cuda")
    smoe.smoe_expert_ffn_save(cfg, p["x"], p["x_perm"], row_token, offsets, T, p["packed"], y, q, sc, _ws(cfg, T))
    assert (y[end:T * k] == 7.0).all() and (q[end:T * k] == 0x55).all() and (sc[:, end:T * k] == 0x55).all()
    assert torch.isfinite(y.float()).all()


def test_no_tokens_give_zero_weight_gradients():
    cfg = _cfg("tiny")
    E, H, I = cfg.n_experts, cfg.hidden, cfg.inter
    out = _outputs(cfg, 0)
    empty = torch.empty(0, dtype=torch.bfloat16, device="cuda")
    smoe.smoe_expert_ffn_backward(cfg, empty, empty, None, 0, None, None, None, empty, empty, *out.values())
    dwr = torch.full((E, H), 7.0, device="cuda")
    smoe.smoe_route_backward(cfg, empty, 0, None, None, None, None, None, None, None, None, dwr)
    torch.cuda.synchronize()
    assert not any(v.any() for v in out.values()) and not dwr.any()
    smoe.smoe_combine_backward(cfg, None, None, None, None, 0, None, None)
    smoe.smoe_permute_backward(cfg, None, None, None, None, None, 0, None)
    smoe.smoe_expert_ffn_save(cfg, None, None, None, None, 0, None, None, None, None)
    smoe.smoe_checkpoint_values(cfg, None, None, 0, None)


class _NothingNative:
    """Stands in for the native module and leaves every call to Python."""
    def __getattr__(self, name):
        return lambda *args: None


def test_native_and_python_calls_agree(monkeypatch):
    """The native calls and the Python ones behind them (taken for whatever is not plain) give the same bits."""
    name = "tiny"
    T = SHAPES[name][0]
    packed, W, x, x64, wr, wr64, dout, dout64, bias, _ = _chain_inputs(name, 46)
    cfg = _cfg(name)
    ws = _ws(cfg, T)
    native = _chain(cfg, x, wr, bias, packed, dout, ws)
    assert smoe._native is not None
    monkeypatch.setattr(smoe, "_native", _NothingNative())
    python = _chain(cfg, x, wr, bias, packed, dout, ws)
    torch.cuda.synchronize()
    for key in native:
        assert torch.equal(native[key].view(torch.uint8), python[key].view(torch.uint8)), key


def test_native_calls_leave_what_is_not_plain():
    T, H, k, E, I = 4, 128, 2, 4, 128
    cfg = smoe.config(H, E, k, I, I)
    R = T * k
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    ws = _ws(cfg, T)
    good = [cfg, bf(T, H), bf(R + T, H), i32(R), torch.zeros(T, k, device="cuda"), T, bf(R, H),
            torch.zeros(T, k, device="cuda"), ws, None, None]
    f = smoe._load_native().combine_backward
    assert f(*good) == smoe.SMOE_OK
    for at, bad in ((0, 7), (1, bf(T, H).float()), (1, bf(T, H).cpu()), (2, bf(R + T - 1, H)), (3, i32(R).long()),
                    (4, [1.0]), (5, 0), (5, -1), (5, 1 << 40), (5, 4.0), (6, bf(H, R).t()), (7, bf(T, k)), (8, ws.cpu()),
                    (9, ws.numel()), (10, torch.cuda.current_stream())):
        assert f(*good[:at], bad, *good[at + 1:]) is None, at
    assert f(*good[:-1]) is None
    # raw pointers and None are plain: the library's own checks answer
    raw = [a.data_ptr() if isinstance(a, torch.Tensor) and i < 8 else a for i, a in enumerate(good)]
    assert f(*raw) == smoe.SMOE_OK
    assert f(*good[:1], None, *good[2:]) == smoe.SMOE_ERR_INVALID_ARG
    assert f(*good[:8], None, None, None) == smoe.SMOE_ERR_INVALID_ARG
    assert f(*good[:8], ws[:256], None, None) == smoe.SMOE_ERR_WORKSPACE
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert f(*good) == smoe.SMOE_OK
    torch.cuda.synchronize()


def test_tensor_checks_of_the_binding():
    name = "tiny"
    T, H, E, k, I, _, _ = SHAPES[name]
    cfg = _cfg(name)
    ws = _ws(cfg, T)
    i32 = torch.zeros(T * k, dtype=torch.int32, device="cuda")
    dout, y = (torch.zeros(n, H, dtype=torch.bfloat16, device="cuda") for n in (T, T * k + T))
    w, dw = torch.zeros(T, k, device="cuda"), torch.zeros(T, k, device="cuda")
    dy = torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda")
    bad = [dict(dout=dout.float()), dict(y=y[:-1]), dict(dy=dy.t()), dict(topk_w=w.cpu()), dict(perm_row=i32.long())]
    for b in bad:
        a = {**dict(dout=dout, y=y, perm_row=i32, topk_w=w, T=T, dy=dy, dtopk_w=dw, ws=ws), **b}
        with pytest.raises(smoe.SmoeError) as ei:
            smoe.smoe_combine_backward(cfg, **a)
        assert ei.value.status == smoe.SMOE_ERR_INVALID_ARG and next(iter(b)) in str(ei.value)
    with pytest.raises(smoe.SmoeError) as ei:
        smoe.smoe_combine_backward(cfg, dout, y, i32, w, T, dy, dw, ws, ws_bytes=smoe.smoe_backward_bytes(cfg, T) - 1)
    assert ei.value.status == smoe.SMOE_ERR_WORKSPACE

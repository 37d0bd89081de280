"""Measured cases of the layer's training operators: what runs between a step's loss and its gradients.

A training step of one sparse MoE layer runs the forward pass with an 8-bit checkpoint of the experts'
gate and up products, then the backward pass in four calls: the way back from the rows of the experts
to the tokens (combine), the experts themselves, the router, and the way from the tokens to the rows
(permute). Rows are those of the layer: R = T * k routed rows in expert order, then T rows of the
shared expert.

    combine_backward   dy[r(t,j)] = w[t,j] dout[t],  dw[t,j] = <dout[t], y[r(t,j)]>
    route_backward     w_j = c s_j / sum s over the selected j, s = sigmoid(l):
                       dl_j = w_j (1 - s_j) sum_i (w_i / c) (dw_j - dw_i),  dW_r[e] = sum dl[t,j] x[t]
    permute_backward   dx[t] = dx_rows[R + t] + sum_j dx_rows[r(t,j)] + sum_j dl[t,j] W_r[e(t,j)]
    ffn_save           g = x W_g^T, u = x W_u^T, h = SiLU(g) u, y = h W_d^T, and (g, u) as e4m3 codes
                       with one power-of-two scale for each row and 32 features
    ffn_backward       from the held (g, u): h, dh = dy W_d, dg = dh u s (1 + g (1 - s)), du = dh g s,
                       dx = dg W_g + du W_u, dW_g = dg^T x, dW_u = du^T x, dW_d = dy^T h

Inputs are bf16 (the router's fp32); sums are held in 32 bits.
"""
import math

import torch

own = False

#: Width, routed experts, experts a token, expert width: the layer's own shape, the share of it that one
#: of eight expert-parallel ranks holds, and the small shape of the tests.
STEP, SHARE, TINY = (4096, 288, 8, 1280), (4096, 36, 8, 1280), (512, 32, 4, 128)
SCALE = 3.0          # the router's factor on the normalised weights
LIMITS = (7.0, 16.0)  # SwiGLU clamps of the deepest layers: routed, shared


def _case(name, op, T, shape, skew=0.0, clamp=False):
    H, E, k, I = shape
    return {"name": name, "op": op, "T": T, "H": H, "E": E, "k": k, "I": I, "skew": skew, "clamp": clamp}


def listed():
    return [
        # one decode-sized batch (64 sequences) of the layer's shape: online fine-tuning, where latency counts
        _case("combine_backward_64", "combine_backward", 64, STEP),
        # a full micro-batch of training
        _case("combine_backward_8192", "combine_backward", 8192, STEP),
        # a handful of ragged tokens: the last, short micro-batch of a document
        _case("permute_backward_17", "permute_backward", 17, STEP),
        # a full micro-batch of training
        _case("permute_backward_8192", "permute_backward", 8192, STEP),
        # a short prompt, odd in length
        _case("route_backward_257", "route_backward", 257, STEP),
        # half a micro-batch early in training, when a few experts draw most tokens
        _case("route_backward_skewed_4096", "route_backward", 4096, STEP, skew=1.2),
        # the tests' small layer: nothing but launches
        _case("ffn_save_tiny_64", "ffn_save", 64, TINY),
        # one expert-parallel rank's experts, an odd number of tokens, the clamp of the deepest layers
        _case("ffn_save_share_777", "ffn_save", 777, SHARE, clamp=True),
        # a full micro-batch on the whole layer
        _case("ffn_save_8192", "ffn_save", 8192, STEP),
        # the tests' small layer
        _case("ffn_backward_tiny_64", "ffn_backward", 64, TINY),
        # one expert-parallel rank's experts, an odd number of tokens, skewed, with the clamp
        _case("ffn_backward_share_1501", "ffn_backward", 1501, SHARE, skew=1.2, clamp=True),
        # a full micro-batch on the whole layer
        _case("ffn_backward_8192", "ffn_backward", 8192, STEP),
    ]


def draw(rng):
    """A batch of 1 to 8192 tokens on a layer up to the full one: widths in steps of 128, any experts and top-k."""
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["combine_backward", "permute_backward", "route_backward", "ffn_save", "ffn_backward"])
    E = log(8, 288)
    return {"op": op, "T": log(1, 8192), "H": 128 * log(2, 32), "E": E, "k": rng.randint(2, min(8, E)),
            "I": 128 * log(1, 10), "skew": rng.choice([0.0, 0.6, 1.2]), "clamp": rng.random() < 0.3}


# ------------------------------------------------------------------------------ inputs
def _normal(gen, shape, std, dtype=torch.bfloat16):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for a in range(0, flat.numel(), 1 << 28):   # in pieces: weights of the whole layer are 9 GB
        flat[a:a + (1 << 28)].normal_(0.0, std, generator=gen)
    return out


def _routing(gen, c):
    """A selection of k distinct experts a token, popular ones more often under skew, its scores and rows."""
    T, E, k = c["T"], c["E"], c["k"]
    popular = -c["skew"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    popular = popular[torch.randperm(E, generator=gen, device="cuda")]
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=gen, device="cuda").clamp(1e-7, 1 - 1e-7)))
    idx = (popular + noise).topk(k, dim=1).indices.to(torch.int32)
    logits = _normal(gen, (T, E), 1.28, torch.float32)
    s = torch.sigmoid(logits.gather(1, idx.long()))
    w = SCALE * s / s.sum(1, keepdim=True)
    order = torch.sort(idx.reshape(-1).long(), stable=True).indices
    perm_row = torch.empty(T * k, dtype=torch.int32, device="cuda")
    perm_row[order] = torch.arange(T * k, dtype=torch.int32, device="cuda")
    counts = torch.bincount(idx.reshape(-1).long(), minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return {"topk_idx": idx, "topk_w": w, "logits": logits, "perm_row": perm_row,
            "row_token": (order // k).to(torch.int32), "offsets": offsets, "counts": counts.tolist() + [T]}


def _experts(gen, c):
    """The experts' weights, and the tile-major form of them that the layer keeps (shared expert last)."""
    H, E, I = c["H"], c["E"], c["I"]
    gu = _normal(gen, (E + 1, 2, I, H), 0.02)
    down = _normal(gen, (E + 1, H, I), 0.02)
    tiles = torch.empty(gu.numel() + down.numel(), dtype=torch.bfloat16, device="cuda")
    tiles[:gu.numel()].view(E + 1, I // 128, H // 64, 2, 128, 64).copy_(
        gu.view(E + 1, 2, I // 128, 128, H // 64, 64).permute(0, 2, 4, 1, 3, 5))
    tiles[gu.numel():].view(E + 1, H // 128, I // 64, 128, 64).copy_(
        down.view(E + 1, H // 128, 128, I // 64, 64).permute(0, 1, 3, 2, 4))
    return {"gu": gu, "down": down, "packed": tiles.view(torch.uint8)}


def _quantise(v):
    """e4m3 codes and power-of-two scales of each 32 neighbours: the least 2^e that brings them to 448 or less."""
    b = v.view(v.shape[0], -1, 32)
    m, e = torch.frexp(b.abs().amax(2))            # amax = m 2^e with 0.5 <= m < 1
    e = e - 9 + (m > 0.875).to(e.dtype)            # 448 = 0.875 * 2^9
    e = torch.where(m == 0, torch.zeros_like(e), e).clamp(-126, 127)
    codes = torch.ldexp(b, -e.unsqueeze(2)).to(torch.float32).to(torch.float8_e4m3fn)
    return codes.view(v.shape), e


def _held(codes, e):
    """The values that codes and exponents stand for."""
    return torch.ldexp(codes.to(torch.float32).view(*e.shape, 32), e.unsqueeze(2)).view(codes.shape)


def prepare(case, seed):
    c = dict(case)
    T, H, E, k, I, op = c["T"], c["H"], c["E"], c["k"], c["I"], c["op"]
    R = T * k
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 17)
    s = {"case": c, **_routing(gen, c)}
    if op == "combine_backward":
        s["dout"] = _normal(gen, (T, H), 1e-3)
        s["y"] = _normal(gen, (R + T, H), 0.5)
    elif op == "permute_backward":
        s["dx_rows"] = _normal(gen, (R + T, H), 1e-3)
        s["dlogits"] = _normal(gen, (T, k), 1e-2, torch.float32)
        s["w_router"] = _normal(gen, (E, H), 0.02, torch.float32)
    elif op == "route_backward":
        s["x"] = _normal(gen, (T, H), 1.0)
        s["dtopk_w"] = _normal(gen, (T, k), 1e-2, torch.float32)
    else:
        s |= _experts(gen, c)
        s["x"] = _normal(gen, (T, H), 1.0)
        s["x_perm"] = s["x"][s["row_token"].long()]
        if op == "ffn_backward":
            s["dout"] = _normal(gen, (T, H), 1e-3)
            s["dy"] = _normal(gen, (R, H), 1e-3)
            s["gu_q"] = torch.empty(R + T, 2 * I, dtype=torch.uint8, device="cuda")
            s["gu_scale"] = torch.empty(2 * I // 32, R + T, dtype=torch.uint8, device="cuda")
            for a in range(0, R + T, 16384):
                codes, e = _quantise(_normal(gen, (min(16384, R + T - a), 2 * I), 0.02 * math.sqrt(H), torch.float32))
                s["gu_q"][a:a + 16384] = codes.view(torch.uint8)
                s["gu_scale"][:, a:a + 16384] = (e + 127).to(torch.uint8).t()
    if own:   # the workspace that a training program keeps for all its steps
        import sparse_moe_layer_smoe_b200 as smoe
        s["cfg"] = smoe.config(H, E, k, I, I, SCALE, *(LIMITS if c["clamp"] else (0.0, 0.0)))
        s["ws"] = smoe.workspace(s["cfg"], T, backward=True)
    return s


# ------------------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)(s, s["case"])


def _run_own(s, c):
    import sparse_moe_layer_smoe_b200 as smoe
    T, H, E, k, I, op = c["T"], c["H"], c["E"], c["k"], c["I"], c["op"]
    R, cfg, ws = T * k, s["cfg"], s["ws"]

    def new(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if op == "combine_backward":
        dy, dw = new(R, H), new(T, k, dtype=torch.float32)
        smoe.smoe_combine_backward(cfg, s["dout"], s["y"], s["perm_row"], s["topk_w"], T, dy, dw, ws)
        return {"dy": dy, "dtopk_w": dw}
    if op == "permute_backward":
        dx = new(T, H)
        smoe.smoe_permute_backward(cfg, s["dx_rows"], s["perm_row"], s["topk_idx"], s["dlogits"], s["w_router"], T, dx, ws)
        return {"dx": dx}
    if op == "route_backward":
        dl, dwr = new(T, k, dtype=torch.float32), new(E, H, dtype=torch.float32)
        smoe.smoe_route_backward(cfg, s["x"], T, s["logits"], s["topk_idx"], s["topk_w"], s["dtopk_w"], s["offsets"],
                                 s["perm_row"], s["row_token"], dl, dwr, ws)
        return {"dlogits": dl, "dw_router": dwr}
    if op == "ffn_save":
        y, q = new(R + T, H), new(R + T, 2 * I, dtype=torch.uint8)
        scale, gu = new(2 * I // 32, R + T, dtype=torch.uint8), new(R + T, 2 * I)
        smoe.smoe_expert_ffn_save(cfg, s["x"], s["x_perm"], s["row_token"], s["offsets"], T, s["packed"], y, q, scale, ws)
        smoe.smoe_checkpoint_values(cfg, q, scale, T, gu)
        return {"y": y, "gu": gu}
    dx_rows = new(R + T, H)
    dg, du, dd = new(E, I, H), new(E, I, H), new(E, H, I)
    sg, su, sd = new(I, H), new(I, H), new(H, I)
    smoe.smoe_expert_ffn_backward(cfg, s["x"], s["x_perm"], s["offsets"], T, s["packed"], s["gu_q"], s["gu_scale"],
                                  s["dy"], s["dout"], dx_rows, dg, du, dd, sg, su, sd, ws)
    return {"dx_rows": dx_rows, "dw_gate": dg, "dw_up": du, "dw_down": dd, "dws_gate": sg, "dws_up": su, "dws_down": sd}


def _groups(s, c):
    """(group, first row, last row + 1, clamp limit) of every expert with rows, the shared one last."""
    a = 0
    for g, n in enumerate(s["counts"]):
        limit = LIMITS[g == c["E"]] if c["clamp"] else math.inf
        if n:
            yield g, a, a + n, limit
        a += n


def _run_plain(s, c):
    T, H, E, k, I, op = c["T"], c["H"], c["E"], c["k"], c["I"], c["op"]
    R = T * k
    rows = s["perm_row"].long()
    if op == "combine_backward":
        dout = s["dout"].float().unsqueeze(1)
        dy = torch.empty(R, H, dtype=torch.bfloat16, device="cuda")
        dy[rows] = (dout * s["topk_w"].unsqueeze(2)).to(torch.bfloat16).view(R, H)
        return {"dy": dy, "dtopk_w": (dout * s["y"][rows].float().view(T, k, H)).sum(2)}
    if op == "permute_backward":
        dx = s["dx_rows"][rows].float().view(T, k, H).sum(1) + s["dx_rows"][R:].float()
        dx += (s["dlogits"].unsqueeze(2) * s["w_router"][s["topk_idx"].long()]).sum(1)
        return {"dx": dx.to(torch.bfloat16)}
    if op == "route_backward":
        w, dw = s["topk_w"], s["dtopk_w"]
        rest = torch.sigmoid(-s["logits"].gather(1, s["topk_idx"].long()))
        dl = w * rest * ((w / SCALE).unsqueeze(1) * (dw.unsqueeze(2) - dw.unsqueeze(1))).sum(2)
        dense = torch.zeros(T, E, device="cuda").scatter_(1, s["topk_idx"].long(), dl)
        return {"dlogits": dl, "dw_router": dense.t() @ s["x"].float()}
    if op == "ffn_save":
        y = torch.empty(R + T, H, dtype=torch.bfloat16, device="cuda")
        gu = torch.empty(R + T, 2 * I, dtype=torch.bfloat16, device="cuda")
        for g, a, b, limit in _groups(s, c):
            x = (s["x"] if g == E else s["x_perm"][a:b]).float()
            v = x @ s["gu"][g].view(2 * I, H).float().t()
            gu[a:b] = _held(*_quantise(v)).to(torch.bfloat16)
            gate, up = v[:, :I].clamp(max=limit), v[:, I:].clamp(-limit, limit)
            y[a:b] = ((gate / (1 + torch.exp(-gate)) * up) @ s["down"][g].float().t()).to(torch.bfloat16)
        return {"y": y, "gu": gu}
    dx_rows = torch.empty(R + T, H, dtype=torch.bfloat16, device="cuda")
    dgu = torch.zeros(2, E + 1, I, H, dtype=torch.bfloat16, device="cuda")
    dd = torch.zeros(E + 1, H, I, dtype=torch.bfloat16, device="cuda")
    for g, a, b, limit in _groups(s, c):
        v = _held(s["gu_q"][a:b].view(torch.float8_e4m3fn), s["gu_scale"][:, a:b].t().to(torch.int32) - 127)
        gate, up = v[:, :I].clamp(max=limit), v[:, I:].clamp(-limit, limit)
        sig = 1 / (1 + torch.exp(-gate))
        dy = (s["dout"] if g == E else s["dy"][a:b]).float()
        dh = dy @ s["down"][g].float()
        d = torch.cat([dh * up * sig * (1 + gate * (1 - sig)) * (v[:, :I] <= limit),
                       dh * gate * sig * (v[:, I:].abs() <= limit)], 1)
        x = (s["x"] if g == E else s["x_perm"][a:b]).float()
        dx_rows[a:b] = (d @ s["gu"][g].view(2 * I, H).float()).to(torch.bfloat16)
        dgu[:, g] = (d.t() @ x).to(torch.bfloat16).view(2, I, H)
        dd[g] = (dy.t() @ (gate * sig * up)).to(torch.bfloat16)
    return {"dx_rows": dx_rows, "dw_gate": dgu[0, :E], "dw_up": dgu[1, :E], "dw_down": dd[:E], "dws_gate": dgu[0, E],
            "dws_up": dgu[1, E], "dws_down": dd[E]}


# ------------------------------------------------------------------------------ the work, and 64 bits
def work(case):
    T, H, E, k, I, op = (case[n] for n in ("T", "H", "E", "k", "I", "op"))
    R = T * k
    # experts that some token chose; under skew fewer, by the chance of each under the drawn popularity
    p = [(e + 1.0) ** -case["skew"] for e in range(E)]
    total = sum(p)
    touched = sum(1 - (1 - min(1.0, k * q / total)) ** T for q in p)
    index = 4 * R
    if op == "combine_backward":
        return {"bytes": 2 * H * (T + 2 * R) + 3 * index, "flops": 3 * R * H}
    if op == "permute_backward":
        return {"bytes": 2 * H * (R + 2 * T) + 3 * index + 4 * H * touched, "flops": 3 * R * H}
    if op == "route_backward":
        return {"bytes": 2 * H * T + 7 * index + 4 * H * E, "flops": 2 * R * H}
    weights = 6 * H * I * (touched + 1)
    held = 2 * I * (R + T) * 33 / 32
    if op == "ffn_save":
        # the values that the codes stand for are read back once: that is how they are looked at here
        return {"bytes": weights + 2 * H * (R + T) * 2 + 2 * held + 4 * I * (R + T), "flops": 6 * (R + T) * H * I}
    return {"bytes": weights + 2 * H * (R + T) * 3 + held + 6 * H * I * (E + 1), "flops": 12 * (R + T) * H * I}


def exact(case, seed):
    """The operators' definitions in 64 bits: token by token or expert by expert, from the inputs alone."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    T, H, E, k, I, op = (case[n] for n in ("T", "H", "E", "k", "I", "op"))
    R, d = T * k, torch.float64
    row = s["perm_row"].long().view(T, k)
    if op == "combine_backward":
        dy, dw = torch.empty(R, H, dtype=d, device="cuda"), torch.empty(T, k, dtype=d, device="cuda")
        for j in range(k):
            dy[row[:, j]] = s["topk_w"][:, j:j + 1].to(d) * s["dout"].to(d)
            dw[:, j] = torch.einsum("th,th->t", s["dout"].to(d), s["y"][row[:, j]].to(d))
        return {"dy": dy, "dtopk_w": dw}
    if op == "permute_backward":
        dx = s["dx_rows"][R:].to(d)
        for j in range(k):
            dx = dx + s["dx_rows"][row[:, j]].to(d) + s["dlogits"][:, j:j + 1].to(d) * s["w_router"].to(d)[s["topk_idx"][:, j].long()]
        return {"dx": dx}
    if op == "route_backward":
        # through the scores: w = c s / S, so dL/ds_j = c (dw_j - sum_i dw_i s_i / S) / S, with the given w for s / S
        l = s["logits"].to(d).gather(1, s["topk_idx"].long())
        w, dw = s["topk_w"].to(d), s["dtopk_w"].to(d)
        p = w / SCALE
        dl = w * (dw * p.sum(1, keepdim=True) - (dw * p).sum(1, keepdim=True)) / (1 + torch.exp(l))
        dwr = torch.zeros(E, H, dtype=d, device="cuda")
        for j in range(k):
            dwr.index_add_(0, s["topk_idx"][:, j].long(), dl[:, j:j + 1] * s["x"].to(d))
        return {"dlogits": dl, "dw_router": dwr}
    bounds = [0] + s["offsets"].tolist()[1:] + [R + T]
    out = {}
    if op == "ffn_save":
        y, gu = torch.empty(R + T, H, dtype=d, device="cuda"), torch.empty(R + T, 2 * I, dtype=d, device="cuda")
    else:
        dx_rows = torch.empty(R + T, H, dtype=d, device="cuda")
        dwg, dwu = (torch.zeros(E + 1, I, H, dtype=d, device="cuda") for _ in range(2))
        dwd = torch.zeros(E + 1, H, I, dtype=d, device="cuda")
    for e in range(E + 1):
        a, b = bounds[e], bounds[e + 1]
        if a == b:
            continue
        limit = math.inf if not case["clamp"] else LIMITS[1] if e == E else LIMITS[0]
        wg, wu, wd = s["gu"][e, 0].to(d), s["gu"][e, 1].to(d), s["down"][e].to(d)
        x = (s["x"] if e == E else s["x"][s["row_token"][a:b].long()]).to(d)
        if op == "ffn_save":
            g, u = x @ wg.t(), x @ wu.t()
            for at, v in ((0, g), (I, u)):
                block = v.view(b - a, I // 32, 32)
                top = block.abs().amax(2, keepdim=True)
                step = torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(-126, 127))
                step = torch.where(top == 0, torch.ones_like(step), step)
                gu[a:b, at:at + I] = ((block / step).to(torch.float32).to(torch.float8_e4m3fn).to(d) * step).view(b - a, I)
            g, u = torch.minimum(g, torch.tensor(limit, device="cuda", dtype=d)), u.clamp(-limit, limit)
            y[a:b] = (g * torch.sigmoid(g) * u) @ wd.t()
            continue
        scale = torch.exp2(s["gu_scale"][:, a:b].t().to(d) - 127).repeat_interleave(32, 1)
        v = s["gu_q"][a:b].view(torch.float8_e4m3fn).to(d) * scale
        g, u = v[:, :I], v[:, I:]
        gc, uc = g.clamp(max=limit), u.clamp(-limit, limit)
        sig = torch.sigmoid(gc)
        dy = (s["dout"] if e == E else s["dy"][a:b]).to(d)
        dh = dy @ wd
        dg = torch.where(g <= limit, dh * uc * (sig + gc * sig * torch.sigmoid(-gc)), 0.0)
        du = torch.where(u.abs() <= limit, dh * gc * sig, 0.0)
        dx_rows[a:b] = dg @ wg + du @ wu
        dwg[e], dwu[e], dwd[e] = dg.t() @ x, du.t() @ x, dy.t() @ (gc * sig * uc)
    if op == "ffn_save":
        return {"y": y, "gu": gu}
    return {"dx_rows": dx_rows, "dw_gate": dwg[:E], "dw_up": dwu[:E], "dw_down": dwd[:E], "dws_gate": dwg[E],
            "dws_up": dwu[E], "dws_down": dwd[E]}

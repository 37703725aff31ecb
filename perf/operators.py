"""Measured cases of the operators that answer with NVFP4 weights and route tokens to experts.

Each case is one call (or the calls of one step) of the package's binding; with
own false the same result is computed by elementary torch operations."""
import math

import torch

own = False

GROUP = 16          # weights per block scale
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decoded token through the key projection of the 70B-shaped decoder layer
        dict(name="kv-1", op="gemv", tokens=1, d_out=1024, d_in=8192, dtype="bf16"),
        # eight sequences' next tokens through its down projection
        dict(name="down-8", op="gemv", tokens=8, d_out=8192, d_in=28672, dtype="bf16"),
        # a few fp32 tokens through a layer of odd sizes (257 blocks a row)
        dict(name="odd-f32-5", op="gemv", tokens=5, d_out=4001, d_in=4112, dtype="f32"),
        # 64 sequences' next tokens through the down projections of 128 experts, 8 a token
        dict(name="experts-down-64", op="gemv_experts", tokens=64, top_k=8, experts=128,
             d_out=4096, d_in=1536, dtype="bf16"),
        # one decoded token, and a batch of 32, through the gate and up projections of the decoder layer
        dict(name="gateup-1", op="swiglu", tokens=1, d_out=28672, d_in=8192, dtype="bf16"),
        dict(name="gateup-32", op="swiglu", tokens=32, d_out=28672, d_in=8192, dtype="bf16"),
        # one decoded token, and a batch of 64, through the gate and up projections of 128 experts
        dict(name="experts-up-1", op="swiglu_experts", tokens=1, top_k=8, experts=128,
             d_out=1536, d_in=4096, dtype="bf16"),
        dict(name="experts-up-64", op="swiglu_experts", tokens=64, top_k=8, experts=128,
             d_out=1536, d_in=4096, dtype="bf16"),
        # routing of a decoded batch, and of 8192 calibration tokens with padding among them
        dict(name="route-64", op="route", tokens=64, top_k=8, experts=128, d=4096, dtype="bf16",
             padded=0.0),
        dict(name="route-8192", op="route", tokens=8192, top_k=8, experts=128, d=4096,
             dtype="bf16", padded=0.03),
        # the experts' rows of a decoded batch back to its tokens
        dict(name="combine-64", op="combine", tokens=64, top_k=8, experts=128, d=4096,
             dtype="f32", padded=0.0),
        # a step that trains: the way back, its gradient and the gradient of the way there
        dict(name="combine-train-8192", op="combine_train", tokens=8192, top_k=8, experts=128,
             d=4096, dtype="bf16", padded=0.03),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemv", "gemv", "swiglu", "gemv_experts", "swiglu_experts", "route",
                     "combine", "combine_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("gemv", "swiglu"):
        d_in = GROUP * _log(rng, 16, 1792)
        d_out = min(_log(rng, 64, 28672), 28672 * 8192 // d_in)
        return dict(op=op, tokens=_log(rng, 1, 32), d_out=d_out, d_in=d_in, dtype=dtype)
    experts = _log(rng, 4, 160)
    c = dict(op=op, tokens=_log(rng, 1, 64), top_k=rng.randint(1, min(8, experts)),
             experts=experts, dtype=dtype)
    if op in ("gemv_experts", "swiglu_experts"):
        c.update(d_out=_log(rng, 64, 2048), d_in=GROUP * _log(rng, 16, 160))
        return c
    c.update(tokens=_log(rng, 1, 4096), d=_log(rng, 64, 4096),
             padded=rng.choice([0.0, 0.0, 0.05, 0.3]))
    return c


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _weights(g, shape, d_in):
    """Codes, scales and global scale as a solve of N(0, 0.02^2) weights leaves
    them: a block's largest weight sits at E2M1's 6 (sixteen equally likely
    quantiles of the rest) and the scales in the upper octaves of E4M3."""
    levels = 6.0 / 1.9 * 2.0 ** 0.5 * torch.special.erfinv(
        (2.0 * torch.arange(16, device="cuda") + 1.0) / 16.0 - 1.0)
    grid = torch.tensor(MAGNITUDES, device="cuda")
    code = (levels.abs()[:, None] - grid[None, :]).abs().argmin(1)
    code = torch.where((levels < 0) & (code > 0), code + 8, code).to(torch.uint8)
    pairs = (code[None, :] + 16 * code[:, None]).reshape(256).to(torch.uint8)
    lead = shape[:-1]
    raw = torch.randint(0, 256, (*shape, d_in // 2), generator=g, device="cuda", dtype=torch.uint8)
    codes = torch.empty_like(raw)
    torch.index_select(pairs, 0, raw.reshape(-1).int(), out=codes.view(-1))
    scales = torch.randint(104, 127, (*shape, d_in // GROUP), generator=g, device="cuda",
                           dtype=torch.uint8)
    s_g = torch.rand(lead or (1,), generator=g, device="cuda") * 2e-5 + 3e-5
    return codes, scales, s_g


def _acts(g, rows, d, dtype, spread=1.0):
    x = torch.randn((rows, d), generator=g, device="cuda")
    return (x * torch.exp(spread * torch.randn(d, generator=g, device="cuda"))).to(dtype)


def _routing(case, seed):
    """Distinct experts of every token by a skewed popularity (int32), their
    weights (fp32), a padded token's experts -1."""
    g = torch.Generator()
    g.manual_seed(seed)
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    logits = torch.randn(E, generator=g) * 0.7 + torch.randn((T, E), generator=g)
    w, ids = torch.topk(logits, k, dim=1)
    gone = torch.rand(T, generator=g) < case.get("padded", 0.0)
    ids[gone] = -1
    return ids.to(torch.int32), torch.softmax(w, 1)


def _sorted(ids, experts):
    """(offsets, rows, position) of the slots sorted by expert."""
    k = ids.shape[1]
    flat = ids.reshape(-1).long()
    key = torch.where((flat < 0) | (flat >= experts), experts, flat)
    order = torch.argsort(key, stable=True)
    ranks = torch.arange(key.numel(), device=ids.device)
    place = torch.empty_like(order)
    place[order] = ranks
    offsets = (key[None, :] < torch.arange(experts + 1, device=ids.device)[:, None]).sum(1)
    rows = torch.where(ranks < offsets[-1], order // k, -1)
    position = torch.where(key < experts, place, -1).view(ids.shape)
    return offsets.int(), rows.int(), position.int()


def prepare(case, seed):
    g = _generator(seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    s = dict(op=op)
    if op in ("gemv", "swiglu"):
        s["x"] = _acts(g, case["tokens"], case["d_in"], dtype, 1.5)
        s["w"] = [_weights(g, (case["d_out"],), case["d_in"])
                  for _ in range(1 if op == "gemv" else 2)]
        s["y"] = torch.empty((case["tokens"], case["d_out"]), dtype=dtype, device="cuda")
        return s
    ids, weights = _routing(case, seed)
    ids, weights = ids.cuda(), weights.cuda()
    E, T, k = case["experts"], case["tokens"], case["top_k"]
    if op in ("gemv_experts", "swiglu_experts"):
        offsets, rows, _ = _sorted(ids, E)
        s["offsets"] = offsets
        s["w"] = [_weights(g, (E, case["d_out"]), case["d_in"])
                  for _ in range(1 if op == "gemv_experts" else 2)]
        # the down projections read the experts' own rows, gate and up the tokens' rows
        s["rows"] = rows if op == "swiglu_experts" else None
        s["x"] = _acts(g, T if op == "swiglu_experts" else T * k, case["d_in"], dtype)
        s["y"] = torch.empty((T * k, case["d_out"]), dtype=dtype if op == "swiglu_experts" else
                             torch.float32, device="cuda")
        s["cap"] = T
        return s
    d = case["d"]
    s.update(experts=E, ids=ids, weights=weights)
    if op == "route":
        s["x"] = _acts(g, T, d, dtype)
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        s["rows"] = torch.empty(T * k, dtype=torch.int32, device="cuda")
        s["position"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        s["xs"] = torch.zeros((T * k, d), dtype=dtype, device="cuda")
        return s
    s["position"] = _sorted(ids, E)[2]
    s["ys"] = _acts(g, T * k, d, dtype)
    s["y"] = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    if op == "combine_train":
        s["dy"] = _acts(g, T, d, dtype)
        s["dxs"] = _acts(g, T * k, d, dtype)
        s["dys"] = torch.zeros((T * k, d), dtype=dtype, device="cuda")
        s["dw"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
        s["dx"] = torch.empty((T, d), dtype=dtype, device="cuda")
    return s


def _dequantised(codes, scales, s_g):
    """fp32 weights of the last two dimensions."""
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=codes.device)
    nib = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    values = table[nib.int()]
    code = (scales & 127).int()
    e, m = code >> 3, (code & 7).float()
    block = torch.where(e > 0, torch.exp2((e - 7).float()) * (1 + m / 8), m / 512)
    values = values.unflatten(-1, (-1, GROUP)) * block[..., None]
    return values.flatten(-2) * s_g.view(*([-1] + [1, 1] if codes.dim() == 3 else [1, 1]))


def _by_expert(x, offsets, w, n, cap):
    """Products of sorted rows with their expert's weights.  Fewer rows than
    experts: each row with the weights taken for it; else the rows are laid
    out as (expert, place), multiplied as a batch, and taken back."""
    E = offsets.numel() - 1
    r = torch.arange(n, device=x.device)
    e = (r[:, None] >= offsets[None, 1:]).sum(1).clamp(max=E - 1)
    if n < E:
        mine = _dequantised(*(t[e] for t in w))
        return torch.bmm(mine, x[:, :, None])[:, :, 0]
    place = (r - offsets[e]).clamp(max=cap - 1)
    pad = torch.zeros((E, cap, x.shape[1]), device=x.device)
    pad[e, place] = x
    return torch.bmm(pad, _dequantised(*w).transpose(1, 2))[e, place]


def _summed(values, position, weights, dtype):
    v = values.float()[position.clamp(min=0).long()]
    if weights is not None:
        v = v * weights[..., None]
    return torch.where(position[..., None] < 0, 0.0, v).sum(1).to(dtype)


def _plain(s):
    op = s["op"]
    if op in ("gemv", "swiglu", "gemv_experts", "swiglu_experts"):
        x = s["x"].float()
        if op in ("gemv", "swiglu"):
            out = [x @ _dequantised(*w).T for w in s["w"]]
        else:
            if s["rows"] is not None:
                x = x[s["rows"].long()]
            out = [_by_expert(x, s["offsets"], w, s["y"].shape[0], s["cap"])
                   for w in s["w"]]
        y = out[0] if len(out) == 1 else out[0] / (1 + torch.exp(-out[0])) * out[1]
        return y.to(s["y"].dtype)
    if op == "route":
        offsets, rows, position = _sorted(s["ids"], s["experts"])
        n, k = s["xs"].shape[0], position.shape[1]
        xs = torch.zeros((n + 1, s["x"].shape[1]), dtype=s["x"].dtype, device="cuda")
        to = torch.where(position < 0, n, position).reshape(-1).long()
        xs[to] = s["x"].repeat_interleave(k, 0)
        xs = torch.where(torch.arange(n, device="cuda")[:, None] < offsets[-1], xs[:n], 0)
        return offsets, rows, position, xs
    w, position = s["weights"], s["position"]
    y = _summed(s["ys"], position, w, s["y"].dtype)
    if op == "combine":
        return y
    n = s["ys"].shape[0]
    dy = s["dy"].float()
    dys = torch.zeros((n + 1, dy.shape[1]), dtype=s["dys"].dtype, device="cuda")
    to = torch.where(position < 0, n, position).long()
    dys[to] = (w[..., None] * dy[:, None, :]).to(dys.dtype)
    dys[n] = 0
    dw = (dy[:, None, :] * s["ys"].float()[position.clamp(min=0).long()]).sum(-1)
    dw = torch.where(position < 0, 0.0, dw)
    return y, dys[:n], dw, _summed(s["dxs"], position, None, s["dx"].dtype)


def run(state):
    if not own:
        return _plain(state)
    from nvfp4_post_weight_b200 import binding as B
    s, op = state, state["op"]
    if op == "gemv":
        B.nvfp4_gemv(s["x"], *s["w"][0], s["y"])
        return s["y"]
    if op == "swiglu":
        B.nvfp4_gemv_swiglu(s["x"], s["w"][0], s["w"][1], s["y"])
        return s["y"]
    if op == "gemv_experts":
        B.nvfp4_gemv_experts(s["x"], s["offsets"], *s["w"][0], s["y"])
        return s["y"]
    if op == "swiglu_experts":
        B.nvfp4_gemv_swiglu_experts(s["x"], s["offsets"], s["w"][0], s["w"][1], s["y"], s["rows"])
        return s["y"]
    if op == "route":
        B.nvfp4_moe_sort(s["ids"], s["offsets"], s["rows"], s["position"])
        B.nvfp4_moe_gather(s["x"], s["position"], s["xs"])
        return s["offsets"], s["rows"], s["position"], s["xs"]
    B.nvfp4_moe_combine(s["ys"], s["position"], s["y"], s["weights"])
    if op == "combine":
        return s["y"]
    B.nvfp4_moe_combine_backward(s["dy"], s["ys"], s["position"], s["weights"], s["dys"], s["dw"])
    B.nvfp4_moe_combine(s["dxs"], s["position"], s["dx"])
    return s["y"], s["dys"], s["dw"], s["dx"]


def work(case):
    op, T = case["op"], case["tokens"]
    size = 4 if case["dtype"] == "f32" else 2
    if op in ("gemv", "swiglu"):
        n = case["d_out"] * case["d_in"] * (1 if op == "gemv" else 2)
        return {"bytes": n * 9 / 16 + T * (case["d_in"] + case["d_out"]) * size,
                "flops": 2 * n * T}
    k, E = case["top_k"], case["experts"]
    ids = _routing(case, 0)[0]
    kept = int((ids >= 0).sum())
    if op in ("gemv_experts", "swiglu_experts"):
        one = case["d_out"] * case["d_in"] * (1 if op == "gemv_experts" else 2)
        active = int(torch.unique(ids[ids >= 0]).numel())
        x = (T if op == "swiglu_experts" else kept) * case["d_in"] * size
        y = kept * case["d_out"] * (size if op == "swiglu_experts" else 4)
        return {"bytes": active * one * 9 / 16 + x + y + 4 * (E + 1), "flops": 2 * one * kept}
    d = case["d"]
    if op == "route":
        return {"bytes": T * k * 12 + 4 * (E + 1) + (T + kept) * d * size, "flops": 0}
    if op == "combine":
        return {"bytes": T * k * 8 + kept * d * size + T * d * 2, "flops": 2 * kept * d}
    return {"bytes": T * k * 12 + 3 * kept * d * size + T * d * (2 + 2 * size),
            "flops": 6 * kept * d}


def _exact_weights(codes, scales, s_g):
    """fp64 weights of one matrix, by the formats' definitions."""
    c = codes.long()
    nib = torch.empty((c.shape[0], 2 * c.shape[1]), dtype=torch.long, device=c.device)
    nib[:, 0::2], nib[:, 1::2] = c % 16, c // 16
    e, m = (nib % 8) // 2, (nib % 2).double()
    mag = torch.where(e == 0, m * 0.5, (1 + 0.5 * m) * 2.0 ** (e - 1).double())
    mag = torch.where(nib >= 8, -mag, mag)
    s = scales.long() % 128
    es, ms = s // 8, (s % 8).double()
    block = torch.where(es == 0, ms * 2.0 ** -9, (8 + ms) * 2.0 ** (es - 10).double())
    return mag * torch.repeat_interleave(block, GROUP, 1) * s_g.double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("gemv", "swiglu", "gemv_experts", "swiglu_experts"):
        x = s["x"].double()
        if op in ("gemv", "swiglu"):
            out = [torch.matmul(x, _exact_weights(*w).t()) for w in s["w"]]
        else:
            x = x if s["rows"] is None else x[s["rows"].long()]
            ends = s["offsets"].tolist()
            out = [torch.cat([x[a:b] @ _exact_weights(w[0][e], w[1][e], w[2][e]).t()
                              for e, (a, b) in enumerate(zip(ends, ends[1:])) if b > a])
                   for w in s["w"]]
        return out[0] if len(out) == 1 else out[0] * torch.sigmoid(out[0]) * out[1]
    if op == "route":
        xs = torch.zeros(s["xs"].shape, dtype=torch.float64, device="cuda")
        ids = s["ids"].cpu().reshape(-1).tolist()
        k = case["top_k"]
        slots = sorted((e, i) for i, e in enumerate(ids) if 0 <= e < case["experts"])
        if slots:
            xs[:len(slots)] = s["x"].double()[torch.tensor([i // k for _, i in slots]).cuda()]
        return None, None, None, xs
    pos, w = s["position"].long(), s["weights"].double()
    keep = (pos >= 0).double()
    ys = s["ys"].double()
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    dx = torch.zeros_like(y)
    dw = torch.zeros(pos.shape, dtype=torch.float64, device="cuda")
    dys = torch.zeros(ys.shape, dtype=torch.float64, device="cuda")
    train = op == "combine_train"
    for j in range(pos.shape[1]):
        p, kj = pos[:, j].clamp(min=0), keep[:, j]
        y += (w[:, j] * kj)[:, None] * ys[p]
        if train:
            dy = s["dy"].double()
            dx += kj[:, None] * s["dxs"].double()[p]
            dw[:, j] = kj * (dy * ys[p]).sum(1)
            live = pos[:, j] >= 0
            dys[p[live]] = (w[:, j, None] * dy)[live]
    return (y, dys, dw, dx) if train else y

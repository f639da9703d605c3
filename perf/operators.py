"""The mixture-of-experts operators around the grouped 4-bit matmul, as cases
that can be timed and compared: their inputs, their plain form in elementary
torch operations, the calls a user makes of this package, and their values in
64 bits.

  route    router logits -> the k experts of each token, their weights and the
           expert-sorted plan the grouped calls read; with its gradient
  combine  the routed rows of each token back into one, weighted; with its
           gradient
  layer    a whole mixture-of-experts layer for a few tokens: router, gate_up,
           SwiGLU, down, combine, on NF4 or MXFP4 expert weights
  product  activations to MXFP4, then MXFP4 x MXFP4 grouped product (W4A4)

Sizes are those of the package's own workloads (128 experts of 2048 x 768,
32 experts of 2880 x 2880, the tiny configuration of 8 experts) and odd ones
around them."""
import math

import torch

own = False

NF4 = (-1.0, -0.6961928009986877, -0.5250730514526367, -0.39491748809814453,
       -0.28444138169288635, -0.18477343022823334, -0.09105003625154495, 0.0,
       0.07958029955625534, 0.16093020141124725, 0.24611230194568634, 0.33791524171829224,
       0.44070982933044434, 0.5626170039176941, 0.7229568362236023, 1.0)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _route(name, T, E, k, dtype, renorm, grad):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "dtype": dtype,
            "renorm": renorm, "grad": grad}


def _combine(name, T, H, k, grad):
    return {"name": name, "op": "combine", "T": T, "H": H, "k": k, "grad": grad}


def _layer(name, fmt, T, E, k, H, I, renorm, bias):
    return {"name": name, "op": "layer", "fmt": fmt, "T": T, "E": E, "k": k, "H": H, "I": I,
            "renorm": renorm, "bias": bias}


def _product(name, T, E, k, N, K, swiglu):
    return {"name": name, "op": "product", "T": T, "E": E, "k": k, "N": N, "K": K,
            "swiglu": swiglu}


def listed():
    return [
        # routing of a decode batch of four requests
        _route("route decode 4", 4, 128, 8, "bf16", True, False),
        # routing of a prompt, logits kept in fp32 by the router
        _route("route prompt 4096", 4096, 128, 8, "fp32", True, False),
        # a training step's routing, forward and backward, odd number of tokens,
        # weights left as the softmax over all experts gives them
        _route("route train 16411", 16411, 32, 4, "bf16", False, True),
        # the combine behind the down projection of a prompt
        _combine("combine prompt 2048", 2048, 2880, 4, False),
        # a training step's combine, forward and backward
        _combine("combine train 4096", 4096, 2048, 8, True),
        # single-request decode on NF4 experts: latency counts
        _layer("layer nf4 1", "nf4", 1, 128, 8, 2048, 768, True, False),
        # a small decode batch: experts shared by few tokens
        _layer("layer nf4 8", "nf4", 8, 128, 8, 2048, 768, True, False),
        # single-request decode on MXFP4 experts, a router with a bias
        _layer("layer mxfp4 1", "mxfp4", 1, 32, 4, 2880, 2880, True, True),
        # the largest decode batch: nearly every expert is read
        _layer("layer mxfp4 32", "mxfp4", 32, 32, 4, 2880, 2880, True, True),
        # the tiny configuration: latency of the two launches
        _product("product tiny", 64, 8, 2, 256, 512, False),
        # gate_up of a prompt, rows gathered from its tokens
        _product("product gate_up 2048", 2048, 32, 4, 5760, 2880, False),
        # down behind SwiGLU, a ragged number of rows
        _product("product down 1001", 1001, 32, 4, 2880, 2880, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "combine", "layer", "layer", "product", "product"))
    if op == "route":
        E = rng.choice((8, 32, 60, 64, 128, 256))
        return _drawn(_route("", _log(rng, 1, 16384), E, rng.randint(1, 8),
                             rng.choice(("bf16", "fp32")), rng.random() < 0.5,
                             rng.random() < 0.5))
    if op == "combine":
        return _drawn(_combine("", _log(rng, 1, 4096), 8 * _log(rng, 8, 360), rng.randint(1, 8),
                               rng.random() < 0.5))
    if op == "layer":
        E = rng.choice((8, 16, 32, 64, 128))
        fmt = rng.choice(("nf4", "mxfp4"))
        most = 2880 * 2880 * 32
        while True:
            H, I = 64 * rng.randint(2, 45), 64 * rng.randint(2, 45)
            if E * H * I <= most:
                break
        return _drawn(_layer("", fmt, _log(rng, 1, 32), E, rng.randint(1, min(8, E)), H, I,
                             rng.random() < 0.5, rng.random() < 0.5))
    E = rng.choice((1, 4, 8, 16, 32))
    return _drawn(_product("", _log(rng, 1, 2048), E, rng.randint(1, min(4, E)),
                           8 * rng.randint(8, 720), 32 * rng.randint(2, 90),
                           rng.random() < 0.4))


def _drawn(c):
    return {k: v for k, v in c.items() if k != "name"}


# ---------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _nf4_weights(g, E, N, K):
    """Codes and absmax of normal weights: the NF4 levels are quantiles of the
    normal distribution, so their codes are nearly uniform."""
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    absmax = 0.02 * (2.4 + 0.35 * torch.randn((E, N, K // 64), generator=g, device="cuda"))
    return codes, absmax.clamp_(min=0.02)


def _mxfp4_weights(g, E, N, K):
    """N(0, 0.02) weights in MXFP4, packed low nibble first."""
    codes = torch.empty((E, N, K // 32, 16), device="cuda", dtype=torch.uint8)
    scales = torch.empty((E, N, K // 32), device="cuda", dtype=torch.uint8)
    edges = torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), device="cuda")
    step = max(1, 8 * (1 << 20) // (N * K))
    for e in range(0, E, step):
        w = torch.randn((min(step, E - e), N, K // 32, 32), generator=g, device="cuda") * 0.02
        x = torch.frexp(w.abs().amax(-1))[1] - 3
        v = w * _pow2(-x)[..., None]
        q = (torch.bucketize(v.abs(), edges) + 8 * (v < 0)).to(torch.uint8)
        codes[e:e + step] = q[..., 0::2] | (q[..., 1::2] << 4)
        scales[e:e + step] = (x + 127).to(torch.uint8)
    return codes, scales


def _pow2(x):
    """2^x in fp32 for whole x in [-126, 127]."""
    return ((x.to(torch.int32) + 127) << 23).view(torch.float32)


def _topk_of(seed, T, E, k):
    """k different experts for each token, some experts asked for more."""
    g = _gen(seed)
    pull = torch.randn((E,), generator=g, device="cuda") * 0.5
    return (torch.randn((T, E), generator=g, device="cuda") + pull).topk(k, dim=1).indices


def _sorted_plan(ids, E):
    """What the grouped calls read for the expert choices `ids` [T, k]."""
    k = ids.shape[1]
    flat = ids.reshape(-1)
    slot_of_row = torch.sort(flat, stable=True).indices
    n = torch.zeros(E, dtype=torch.int64, device=ids.device)
    n.scatter_add_(0, flat.long(), torch.ones_like(flat, dtype=torch.int64))
    offsets = torch.cat([n.new_zeros(1), n.cumsum(0)])
    rows = torch.arange(flat.numel(), device=ids.device)
    row_of_slot = torch.empty_like(rows).scatter_(0, slot_of_row, rows).reshape(ids.shape)
    i = torch.int32
    return offsets.to(i), (slot_of_row // k).to(i), row_of_slot.to(i), slot_of_row.to(i)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op, T, k = case["op"], case["T"], case["k"]
    if op == "route":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["logits"] = _normal(g, (T, case["E"]), 1.5, dt)
        if case["grad"]:
            s["dw"] = _normal(g, (T, k))
        return s
    if op == "combine":
        P, H = T * k, case["H"]
        ids = _topk_of(seed + 1, T, 64, k)
        _, _, s["row_of_slot"], s["slot_of_row"] = _sorted_plan(ids, 64)
        s["y"] = _normal(g, (P, H), 1.0, torch.bfloat16)
        w = torch.rand((T, k), generator=g, device="cuda") + 0.05
        s["w"] = w / w.sum(1, keepdim=True)
        if case["grad"]:
            s["dout"] = _normal(g, (T, H), 0.1, torch.bfloat16)
        return s
    E = case["E"]
    if op == "layer":
        H, I = case["H"], case["I"]
        s["x"] = _normal(g, (T, H), 1.0, torch.bfloat16)
        s["rw"] = _normal(g, (E, H), 1.5 / math.sqrt(H), torch.bfloat16)
        s["rb"] = _normal(g, (E,), 0.2) if case["bias"] else None
        make = _nf4_weights if case["fmt"] == "nf4" else _mxfp4_weights
        s["gu"] = make(g, E, 2 * I, H)
        s["dn"] = make(g, E, H, I)
        return s
    N, K = case["N"], case["K"]
    s["w"], s["ws"] = _mxfp4_weights(g, E, N, K)
    off, r2t, _, _ = _sorted_plan(_topk_of(seed + 1, T, E, k), E)
    s["off"] = off
    n = off.cpu()
    s["most_rows"] = int((n[1:] - n[:-1]).max())  # the plan's largest expert
    if case["swiglu"]:
        s["x"] = _normal(g, (T * k, 2 * K), 1.0, torch.bfloat16)
        s["r2t"] = None
    else:
        s["x"] = _normal(g, (T, K), 1.0, torch.bfloat16)
        s["r2t"] = r2t
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    return (_OWN if own else _PLAIN)[s["op"]](s)


def _own_route(s):
    import grouped_bit_weight_b200 as gbw
    r = gbw.gmoe_route(s["logits"], s["k"], renormalize=s["renorm"])
    out = dict(r._asdict())
    if s["grad"]:
        out["dlogits"] = gbw.gmoe_route_bwd(s["logits"], r.topk_ids, r.topk_weights, s["dw"],
                                            renormalize=s["renorm"])
    return out


def _own_combine(s):
    import grouped_bit_weight_b200 as gbw
    out = {"out": gbw.gmoe_combine(s["y"], s["row_of_slot"], s["w"])}
    if s["grad"]:
        out["dy"], out["dw"] = gbw.gmoe_combine_bwd(s["dout"], s["y"], s["row_of_slot"],
                                                    s["slot_of_row"], s["w"])
    return out


def _own_layer(s):
    import grouped_bit_weight_b200 as gbw
    f = gbw.gnf4_moe_layer if s["fmt"] == "nf4" else gbw.gmxfp4_moe_layer
    return f(s["x"], s["rw"], *s["gu"], *s["dn"], k=s["k"], renormalize=s["renorm"],
             router_bias=s["rb"])


def _own_product(s):
    import grouped_bit_weight_b200 as gbw
    xq, xs = gbw.gmxfp4_quantize_rows(s["x"], row_to_token=s["r2t"], swiglu=s["swiglu"])
    return gbw.gmxfp4_grouped_gemm_a4(xq, xs, s["w"], s["ws"], s["off"])


_OWN = {"route": _own_route, "combine": _own_combine, "layer": _own_layer,
        "product": _own_product}


def _choose(logits, k, renorm):
    """The k largest of each row (ties: the lowest index) and their softmax
    weights, over all experts or over the chosen ones."""
    v, i = torch.sort(logits, dim=1, descending=True, stable=True)
    ids, top = i[:, :k], v[:, :k]
    p = (top - v[:, :1]).exp()
    total = p if renorm else (v - v[:, :1]).exp()
    return ids, p / total.sum(1, keepdim=True)


def _plain_route(s):
    x = s["logits"].float()
    ids, w = _choose(x, s["k"], s["renorm"])
    off, r2t, row_of_slot, slot_of_row = _sorted_plan(ids, s["E"])
    out = {"topk_ids": ids.to(torch.int32), "topk_weights": w, "expert_offsets": off,
           "row_to_token": r2t, "row_of_slot": row_of_slot, "slot_of_row": slot_of_row}
    if s["grad"]:
        # w_s = p_s / sum: dlogits_e = [e chosen] w dw - w_or_p_e * sum_s w_s dw_s
        t = (w * s["dw"]).sum(1, keepdim=True)
        if s["renorm"]:
            d = torch.zeros_like(x).scatter_(1, ids, w * (s["dw"] - t))
        else:
            p = (x - x.amax(1, keepdim=True)).exp()
            d = -(p / p.sum(1, keepdim=True)) * t
            d = d.scatter_add(1, ids, w * s["dw"])
        out["dlogits"] = d.to(s["logits"].dtype)
    return out


def _plain_combine(s):
    rows = s["row_of_slot"].long()
    y = s["y"].float()[rows]  # [T, k, H]
    w = s["w"]
    out = {"out": (y * w[..., None]).sum(1).to(torch.bfloat16)}
    if s["grad"]:
        d = s["dout"].float()[:, None]
        out["dy"] = torch.empty_like(s["y"]).index_copy_(
            0, rows.reshape(-1), (d * w[..., None]).to(torch.bfloat16).flatten(0, 1))
        out["dw"] = (y * d).sum(-1)
    return out


def _nibbles(b, high_first):
    lo, hi = b & 15, b >> 4
    return torch.stack((hi, lo) if high_first else (lo, hi), -1).flatten(-2).int()


def _weights(fmt, codes, scale):
    """fp32 weights of packed ones [..., K/2] (MXFP4: [..., K/32, 16])."""
    if fmt == "nf4":
        q = torch.tensor(NF4, device=codes.device)[_nibbles(codes, True)]
        return (q.unflatten(-1, (-1, 64)) * scale[..., None]).flatten(-2)
    q = torch.tensor(E2M1, device=codes.device)[_nibbles(codes, False)]
    return (q * _pow2(scale.int() - 127)[..., None]).flatten(-2)


def _silu(v):
    return v / (1 + (-v).exp())


def _plain_layer(s):
    x, k, E, I = s["x"].float(), s["k"], s["E"], s["I"]
    T = x.shape[0]
    # the choice of experts lies next to a border: logits in 64 bits
    logits = s["x"].double() @ s["rw"].double().T
    if s["rb"] is not None:
        logits = logits + s["rb"].double()
    ids, w = _choose(logits, k, s["renorm"])
    w = w.float()
    if T * k < E:  # the rows' own experts
        e = ids.reshape(-1)
        gu = _weights(s["fmt"], *(v[e] for v in s["gu"]))
        h = torch.bmm(gu, x.repeat_interleave(k, 0)[..., None])[..., 0]
        h = _silu(h[:, :I]) * h[:, I:]
        dn = _weights(s["fmt"], *(v[e] for v in s["dn"]))
        y = torch.bmm(dn, h[..., None])[..., 0].unflatten(0, (T, k))
    else:  # every expert on every token, then the rows' own
        h = torch.matmul(x, _weights(s["fmt"], *s["gu"]).mT)  # [E, T, 2I]
        h = _silu(h[..., :I]) * h[..., I:]
        y = torch.bmm(h, _weights(s["fmt"], *s["dn"]).mT)  # [E, T, H]
        y = y[ids, torch.arange(T, device=x.device)[:, None]]
    return (y * w[..., None]).sum(1).to(torch.bfloat16)


def _to_mxfp4(v):
    """The values that MXFP4 holds for v [..., K]: blocks of 32 with the scale
    2^(floor(log2 max) - 2), elements to the nearest (ties to even), at most 6."""
    b = v.unflatten(-1, (-1, 32))
    m = b.abs().amax(-1, keepdim=True)
    x = (torch.frexp(m)[1] - 3).clamp(-126, 127)
    x = torch.where(m == 0, torch.full_like(x, -126), x)
    a = b * _pow2(-x)
    t = a.abs()
    step = torch.where(t < 2, 0.5, torch.where(t < 4, 1.0, 2.0))
    q = (torch.round(t / step) * step).clamp(max=6.0)
    return (torch.copysign(q, a) * _pow2(x)).flatten(-2).float()


def _plain_product(s):
    x = s["x"].float()
    if s["swiglu"]:  # next to a border of the rounding: in 64 bits
        v = s["x"].double()
        x = (_silu(v[:, :s["K"]]) * v[:, s["K"]:]).float()
    x = _to_mxfp4(x)
    if s["r2t"] is not None:
        x = x[s["r2t"].long()]
    P, E = x.shape[0], s["E"]
    off = s["off"].long()
    # each expert's rows, filled up to those of the largest expert
    at = off[:-1, None] + torch.arange(s["most_rows"], device=x.device)
    y = torch.bmm(x[at.clamp(max=P - 1)], _weights("mxfp4", s["w"], s["ws"]).mT)
    p = torch.arange(P, device=x.device)
    e = torch.searchsorted(off[1:], p, right=True)
    return y[e, p - off[e]].to(torch.bfloat16)


_PLAIN = {"route": _plain_route, "combine": _plain_combine, "layer": _plain_layer,
          "product": _plain_product}


# ---------------------------------------------------------------- work


def work(case):
    op, T, k = case["op"], case["T"], case["k"]
    P = T * k
    if op == "route":
        size = 2 if case["dtype"] == "bf16" else 4
        b = T * case["E"] * size + 20 * P + 4 * (case["E"] + 1)
        f = 4 * T * case["E"]
        if case["grad"]:
            b, f = b + 2 * T * case["E"] * size + 12 * P, f + 6 * T * case["E"]
        return {"bytes": b, "flops": f}
    if op == "combine":
        H = case["H"]
        b = 2 * P * H + 2 * T * H + 8 * P
        f = 2 * P * H
        if case["grad"]:  # y is read again: the forward pass's copy is gone
            b, f = b + 4 * P * H + 2 * T * H + 16 * P, f + 3 * P * H
        return {"bytes": b, "flops": f}
    E = case["E"]
    if op == "layer":
        H, I = case["H"], case["I"]
        experts = E * (1 - (1 - k / E) ** T)  # expected number of experts read
        bits = 4 + (0.5 if case["fmt"] == "nf4" else 0.25)
        return {"bytes": experts * 3 * H * I * bits / 8 + 2 * E * H + 4 * T * H,
                "flops": 6 * P * H * I + 2 * T * E * H}
    N, K = case["N"], case["K"]
    rows = P if case["swiglu"] else T
    experts = E * (1 - (1 - k / E) ** T)
    return {"bytes": 2 * rows * K * (2 if case["swiglu"] else 1) + 4 * P
            + experts * N * K * 4.25 / 8 + 2 * P * N,
            "flops": 2 * P * N * K}


# ---------------------------------------------------------------- 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "combine": _exact_combine, "layer": _exact_layer,
            "product": _exact_product}[case["op"]](s)


def _largest(v, k):
    """Indices of the k largest of each row, one after the other."""
    left, ids = v.clone(), []
    for _ in range(k):
        i = (left == left.amax(1, keepdim=True)).to(torch.int8).argmax(1, keepdim=True)
        ids.append(i)
        left.scatter_(1, i, -math.inf)
    return torch.cat(ids, 1)


def _share(v, ids, renorm):
    c = v.gather(1, ids)
    return c.softmax(1) if renorm else v.softmax(1).gather(1, ids)


def _exact_route(s):
    v = s["logits"].double()
    ids = _largest(v, s["k"])
    out = {"topk_ids": None, "topk_weights": _share(v, ids, s["renorm"]), "expert_offsets": None,
           "row_to_token": None, "row_of_slot": None, "slot_of_row": None}
    if s["grad"]:
        with torch.enable_grad():
            a = v.requires_grad_(True)
            _share(a, ids, s["renorm"]).backward(s["dw"].double())
        out["dlogits"] = a.grad
    return out


def _exact_combine(s):
    T, k = s["row_of_slot"].shape
    o = torch.zeros((T, s["H"]), dtype=torch.float64, device="cuda")
    out = {"out": o}
    dy = torch.zeros((T * k, s["H"]), dtype=torch.float64, device="cuda")
    dw = torch.zeros((T, k), dtype=torch.float64, device="cuda")
    for j in range(k):
        r, w = s["row_of_slot"][:, j].long(), s["w"][:, j:j + 1].double()
        o += w * s["y"][r].double()
        if s["grad"]:
            dy[r] = w * s["dout"].double()
            dw[:, j] = torch.einsum("th,th->t", s["y"][r].double(), s["dout"].double())
    if s["grad"]:
        out.update(dy=dy, dw=dw)
    return out


def _weight64(fmt, codes, scale, e):
    """Expert e's weights in 64 bits, [N, K]."""
    c = codes[e].flatten(1).long()
    even, odd = (c // 16, c % 16) if fmt == "nf4" else (c % 16, c // 16)
    q = torch.empty((c.shape[0], 2 * c.shape[1]), dtype=torch.int64, device="cuda")
    q[:, 0::2], q[:, 1::2] = even, odd
    if fmt == "nf4":
        v = torch.tensor(NF4, dtype=torch.float64, device="cuda").take(q)
        return v * scale[e].double().repeat_interleave(64, 1)
    m, x = q % 2, (q // 2) % 4
    v = torch.where(x == 0, 0.5 * m, (1 + 0.5 * m) * torch.pow(2.0, (x - 1).double()))
    v = torch.where(q >= 8, -v, v).double()
    return v * torch.pow(2.0, scale[e].double() - 127).repeat_interleave(32, 1)


def _exact_layer(s):
    x = s["x"].double()
    v = torch.einsum("th,eh->te", x, s["rw"].double())
    if s["rb"] is not None:
        v = v + s["rb"].double()
    ids = _largest(v, s["k"])
    w = _share(v, ids, s["renorm"])
    out = torch.zeros_like(x)
    for e in sorted(set(ids.flatten().tolist())):
        t, j = (ids == e).nonzero(as_tuple=True)
        a = x[t] @ _weight64(s["fmt"], *s["gu"], e).T
        h = torch.nn.functional.silu(a[:, :s["I"]]) * a[:, s["I"]:]
        out[t] += w[t, j][:, None] * (h @ _weight64(s["fmt"], *s["dn"], e).T)
    return out


def _exact_product(s):
    x = s["x"].double()
    if s["swiglu"]:
        x = torch.sigmoid(x[:, :s["K"]]) * x[:, :s["K"]] * x[:, s["K"]:]
    b = x.reshape(x.shape[0], -1, 32)
    m = b.abs().amax(2, keepdim=True)
    scale = torch.pow(2.0, torch.floor(torch.log2(torch.where(m > 0, m, 1.0))) - 2)
    levels = torch.tensor(E2M1[:8], dtype=torch.float64, device="cuda")
    t = (b / scale).abs()
    # the nearer of the two levels around it; halfway, the one of even code
    hi = torch.searchsorted(levels, t).clamp(1, 7)
    a, c = t - levels[hi - 1], levels[hi] - t
    up = (a > c) | ((a == c) & (hi % 2 == 0))
    q = levels[torch.where(up, hi, hi - 1)]
    x = (torch.where(b < 0, -q, q) * scale).reshape(x.shape)
    if s["r2t"] is not None:
        x = x[s["r2t"].long()]
    off = s["off"].tolist()
    out = torch.empty((off[-1], s["N"]), dtype=torch.float64, device="cuda")
    for e in range(s["E"]):
        if off[e + 1] > off[e]:
            out[off[e]:off[e + 1]] = x[off[e]:off[e + 1]] @ _weight64("mxfp4", s["w"], s["ws"], e).T
    return out

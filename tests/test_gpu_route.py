"""Routing and combine against plain 64-bit implementations: choices and plans
exactly, weights and gradients within bounds counted from their roundings."""
import numpy as np
import pytest
import torch

import moe_plain as mp

gbw = pytest.importorskip("grouped_bit_weight_b200")
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _logits(T, E, dtype, seed, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, E), generator=g) * std).to(DT[dtype])


def _check_route(l, k, renorm):
    T, E = l.shape
    r = gbw.gmoe_route(l.to(DEV), k, renormalize=renorm)
    torch.cuda.synchronize()
    ids, w = mp.route(l.double().numpy(), k, renorm)
    off, r2t, ros, sor = mp.plan(ids, E)
    assert (r.topk_ids.cpu().numpy() == ids).all()
    assert (r.expert_offsets.cpu().numpy() == off).all()
    assert (r.row_to_token.cpu().numpy() == r2t).all()
    assert (r.row_of_slot.cpu().numpy() == ros).all()
    assert (r.slot_of_row.cpu().numpy() == sor).all()
    # exp's argument l - m rounds by 2^-24 |l - m| (absolute, so relative in
    # the exponential), exp itself by 2 ulp, the sum of n terms by (5 + n / 32)
    # 2^-24 (a lane's chain, then five shuffle steps), the division by 2^-24
    v = np.where(np.isfinite(l.double().numpy()), l.double().numpy(), 0.0)
    spread = 2 * np.abs(v).max(initial=0.0)
    rel = 2.0 ** -24 * (2 * spread + 4 + 4 + 6 + E / 32 + 2)
    got = r.topk_weights.cpu().double().numpy()
    assert (np.abs(got - w) <= rel * w + 1e-37).all(), np.abs(got - w).max()
    assert gbw.device_status() == 0
    return r, ids, w


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (3, 8, 2), (5, 33, 32), (127, 60, 6),
                                   (128, 128, 8), (129, 128, 8), (601, 1024, 5), (1000, 32, 4),
                                   (4099, 257, 9), (10007, 8, 8)])
def test_route_matches_plain(T, E, k, renorm, dtype):
    l = _logits(T, E, dtype, T + E)
    r, ids, w = _check_route(l, k, renorm)
    g = torch.Generator().manual_seed(7)
    dw = torch.randn((T, k), generator=g)
    d = gbw.gmoe_route_bwd(l.to(DEV), r.topk_ids, r.topk_weights, dw.to(DEV), renormalize=renorm)
    ref = mp.route_bwd(l.double().numpy(), ids, w, dw.double().numpy(), renorm)
    # every term is w dw or q * sum(w dw), each rounded a few times: 40 roundings
    # of the largest term cover the chain (weights' own error included)
    big = (w * np.abs(dw.numpy())).sum(1, keepdims=True) + (w * np.abs(dw.numpy())).max(1, keepdims=True)
    spread = 2 * np.abs(l.double().numpy()).max()
    tol = 2.0 ** -24 * (40 + 4 * spread + E / 16) * big
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * np.abs(ref)
    assert d.dtype == l.dtype
    assert (np.abs(d.cpu().double().numpy() - ref) <= tol + 1e-38).all()
    assert gbw.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 300])
def test_route_ties_go_to_the_lowest_index(T):
    l = torch.zeros((T, 64))
    l[:, 10] = -0.0
    l[1::2] = torch.tensor([1.0, 2.0]).repeat(32)
    _check_route(l.to(torch.bfloat16), 6, True)
    _check_route(_logits(T, 128, "bf16", 3, std=0.02).round(decimals=2), 8, True)


@pytest.mark.gpu
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T", [9, 400])
def test_route_masked_rows_infinities_and_nan(T, renorm):
    l = _logits(T, 40, "fp32", 5)
    inf, low = float("inf"), torch.finfo(torch.float32).min
    l[0] = -inf                      # nothing left
    l[1] = -inf
    l[1, 17] = 0.25                  # one expert left, k = 4 asked
    l[2, 3] = inf                    # an infinite maximum
    l[3, 5] = l[3, 30] = inf         # two of them share
    l[4, :20] = float("nan")         # NaN is never chosen before a number
    l[5] = float("nan")
    l[6] = low                       # a mask of the type's lowest value: equal logits
    l[7, 1:] = low
    l[8, ::2] = -inf
    r, ids, w = _check_route(l, 4, renorm)
    assert (r.topk_weights[[0, 5]] == 0).all()
    dw = torch.full((T, 4), 2.0)
    dw[1, 1:] = float("nan")         # at slots of weight 0: passes nothing on
    dw[0] = inf
    d = gbw.gmoe_route_bwd(l.to(DEV), r.topk_ids, r.topk_weights, dw.to(DEV), renormalize=renorm)
    ref = mp.route_bwd(l.double().numpy(), ids, w, dw.double().numpy(), renorm)
    got = d.cpu().double().numpy()
    assert np.isfinite(got).all() and (np.abs(got - ref) <= 1e-5).all()


@pytest.mark.gpu
def test_route_without_tokens_and_repeats_bit_for_bit():
    r = gbw.gmoe_route(torch.empty((0, 16), device=DEV), 2)
    assert r.expert_offsets.tolist() == [0] * 17 and r.row_to_token.numel() == 0
    assert gbw.gmoe_route_bwd(torch.empty((0, 16), device=DEV), r.topk_ids, r.topk_weights,
                              r.topk_weights).shape == (0, 16)
    l = _logits(3000, 128, "bf16", 9).to(DEV)
    a, b = gbw.gmoe_route(l, 8), gbw.gmoe_route(l, 8)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
def test_route_gradient_against_differences():
    """dlogits against central differences of the weighted sum, in 64 bits on
    the plain implementation's side, for logits far from ties."""
    g = torch.Generator().manual_seed(3)
    l = torch.stack([torch.randperm(12, generator=g) for _ in range(6)]).float() * 0.5
    dw = torch.randn((6, 3), generator=g)
    for renorm in (True, False):
        r = gbw.gmoe_route(l.to(DEV), 3, renormalize=renorm)
        d = gbw.gmoe_route_bwd(l.to(DEV), r.topk_ids, r.topk_weights, dw.to(DEV),
                               renormalize=renorm).cpu().numpy()
        f = lambda v: (mp.route(v, 3, renorm)[1] * dw.double().numpy()).sum(1)
        for e in range(12):
            h = np.zeros((1, 12))
            h[0, e] = 1e-4
            diff = (f(l.double().numpy() + h) - f(l.double().numpy() - h)) / 2e-4
            assert np.abs(diff - d[:, e]).max() < 1e-6


def _combine_inputs(T, H, k, seed, P=None):
    g = torch.Generator().manual_seed(seed)
    P = T * k if P is None else P
    y = torch.randn((P, H), generator=g).to(torch.bfloat16)
    slot_of_row = torch.full((P,), -1, dtype=torch.int32)
    rows = torch.randperm(P, generator=g)[:T * k].to(torch.int32)
    slot_of_row[rows.long()] = torch.arange(T * k, dtype=torch.int32)
    w = torch.rand((T, k), generator=g)
    dout = torch.randn((T, H), generator=g).to(torch.bfloat16)
    return y, rows.reshape(T, k), slot_of_row, w, dout


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,k", [(1, 8, 1), (1, 2048, 8), (3, 264, 5), (64, 512, 2),
                                   (601, 2880, 4), (33, 1000, 32), (2, 100000, 3)])
def test_combine_and_its_gradient_match_plain(T, H, k):
    y, rows, slots, w, dout = _combine_inputs(T, H, k, T + H)
    yd, rd, sd, wd, dd = (t.to(DEV) for t in (y, rows, slots, w, dout))
    y64, d64, w64 = y.double().numpy(), dout.double().numpy(), w.double().numpy()
    out = gbw.gmoe_combine(yd, rd, wd).cpu().double().numpy()
    # k products summed in fp32: (k + 1) roundings of the sum of magnitudes
    extra = (k + 1) * 2.0 ** -24 * mp.combine(np.abs(y64), rows.numpy(), w64)
    mp.bf16_close(out, mp.combine(y64, rows.numpy(), w64), extra)
    ones = gbw.gmoe_combine(yd, rd).cpu().double().numpy()
    mp.bf16_close(ones, mp.combine(y64, rows.numpy(), np.ones_like(w64)),
                  (k + 1) * 2.0 ** -24 * mp.combine(np.abs(y64), rows.numpy(), np.ones_like(w64)))
    dy, dw = gbw.gmoe_combine_bwd(dd, yd, rd, sd, wd)
    ref = np.empty_like(y64)
    ref[rows.numpy().reshape(-1)] = (w64[..., None] * d64[:, None]).reshape(-1, H)
    mp.bf16_close(dy.cpu().double().numpy(), ref, 2.0 ** -24 * np.abs(ref))
    # a lane sums H / 32 products one after the other, then five steps
    mag = np.einsum("tkh,th->tk", np.abs(y64[rows.numpy()]), np.abs(d64))
    dref = np.einsum("tkh,th->tk", y64[rows.numpy()], d64)
    assert (np.abs(dw.cpu().numpy() - dref) <= 2.0 ** -24 * (H / 32 + 14) * mag).all()
    assert gbw.device_status() == 0


@pytest.mark.gpu
def test_combine_leaves_unnamed_rows_and_masked_slots_alone():
    T, H, k, P = 5, 64, 3, 20
    y, rows, slots, w, dout = _combine_inputs(T, H, k, 1, P)
    w[2] = 0.0                       # a token that is masked out
    y[rows[2].long()] = float("nan")
    y[rows[3, 1].long()] = float("inf")
    w[3, 1] = 0.0
    out = gbw.gmoe_combine(y.to(DEV), rows.to(DEV), w.to(DEV))
    assert torch.isfinite(out).all() and (out[2] == 0).all()
    dy = torch.full((P, H), 7.0, dtype=torch.bfloat16, device=DEV)
    gbw.gmoe_combine_bwd(dout.to(DEV), y.to(DEV), rows.to(DEV), slots.to(DEV), w.to(DEV), dy=dy)
    unnamed = (slots < 0).nonzero().flatten().to(DEV)
    assert len(unnamed) == 5 and (dy[unnamed] == 7.0).all()
    assert (dy[rows[2].long().to(DEV)] == 0).all()
    dy2, _ = gbw.gmoe_combine_bwd(dout.to(DEV), y.to(DEV), rows.to(DEV), slots.to(DEV), w.to(DEV))
    assert (dy2[unnamed] == 0).all()
    assert gbw.device_status() == 0


@pytest.mark.gpu
def test_combine_reports_bad_rows_and_writes_each_row_once():
    """Rows outside [0, P) add nothing; the same row in two slots is summed
    forward, and in the backward pass written by the slot that slot_of_row
    names.  All are checked in the kernel before any access."""
    T, H, k = 4, 64, 2
    y, rows, slots, w, dout = _combine_inputs(T, H, k, 2)
    args = lambda: (t.to(DEV) for t in (dout, y, rows, slots, w))
    good = rows.clone()
    rows[0, 0], rows[1, 1] = -1, T * k
    out = gbw.gmoe_combine(y.to(DEV), rows.to(DEV), w.to(DEV)).cpu().double().numpy()
    assert gbw.device_status() == gbw.DEVERR_ROUTE
    w64 = w.double().numpy().copy()
    w64[0, 0] = w64[1, 1] = 0
    mp.bf16_close(out, mp.combine(y.double().numpy(), good.numpy(), w64), 1e-6)
    d, *rest = args()
    dy, dw = gbw.gmoe_combine_bwd(d, *rest)
    assert gbw.device_status() == gbw.DEVERR_ROUTE
    assert dw[0, 0] == 0 and dw[1, 1] == 0
    rows = good.clone()
    rows[3, 1] = rows[0, 0]
    d, *rest = args()
    dy, dw = gbw.gmoe_combine_bwd(d, *rest)
    assert gbw.device_status() == gbw.DEVERR_ROUTE
    assert dw[3, 1] == 0
    want = (w[0, 0] * dout[0].float()).to(torch.bfloat16)
    assert torch.equal(dy[rows[0, 0].long()].cpu(), want)


@pytest.mark.gpu
def test_route_bwd_reports_bad_ids():
    l = _logits(4, 16, "fp32", 1).to(DEV)
    r = gbw.gmoe_route(l, 2)
    ids = r.topk_ids.clone()
    ids[1, 0], ids[2, 1] = 16, -3
    d = gbw.gmoe_route_bwd(l, ids, r.topk_weights, torch.ones_like(r.topk_weights))
    assert torch.isfinite(d).all()
    assert gbw.device_status() == gbw.DEVERR_ROUTE


@pytest.mark.gpu
@pytest.mark.parametrize("renorm", [True, False])
def test_route_bwd_leaves_a_slot_with_a_bad_id_out(renorm):
    """The gradient is that of the same call with the slot's weight zero, and
    other tokens' rows are those of good ids."""
    l = _logits(4, 16, "fp32", 1).to(DEV)
    r = gbw.gmoe_route(l, 3, renormalize=renorm)
    dw = _logits(4, 3, "fp32", 2).to(DEV)
    good = gbw.gmoe_route_bwd(l, r.topk_ids, r.topk_weights, dw, renormalize=renorm)
    assert gbw.device_status() == 0
    ids, w = r.topk_ids.clone(), r.topk_weights.clone()
    ids[1, 0], ids[2, 2] = 16, -3
    got = gbw.gmoe_route_bwd(l, ids, w, dw, renormalize=renorm)
    assert gbw.device_status() == gbw.DEVERR_ROUTE
    w[1, 0] = w[2, 2] = 0.0
    want = gbw.gmoe_route_bwd(l, r.topk_ids, w, dw, renormalize=renorm)
    assert torch.equal(got, want) and gbw.device_status() == 0
    assert torch.equal(got[[0, 3]], good[[0, 3]]) and not torch.equal(got[1], good[1])
    w64, dw64 = w.cpu().double().numpy(), dw.cpu().double().numpy()
    ref = mp.route_bwd(l.cpu().double().numpy(), r.topk_ids.cpu().numpy(), w64, dw64, renorm)
    # 3 products and sums, 16 exponentials, each within 2^-21 of a share of at most 1
    assert (np.abs(got.cpu().double().numpy() - ref) <= 2.0 ** -19 * np.abs(dw64).sum(1, keepdims=True)).all()


@pytest.mark.gpu
def test_route_then_grouped_then_combine_on_a_side_stream_and_in_a_graph():
    """Route -> fused expert pass -> combine: eager on a side stream, then
    captured once and replayed on other inputs, equals the plain chain."""
    T, E, k, H, I = 48, 8, 2, 128, 64
    g = torch.Generator(device=DEV).manual_seed(1)
    gu = gbw.gnf4_quantize(torch.randn((E, 2 * I, H), generator=g, device=DEV) * 0.05)
    dn = gbw.gnf4_quantize(torch.randn((E, H, I), generator=g, device=DEV) * 0.05)
    x = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
    l = torch.randn((T, E), generator=g, device=DEV)

    def chain():
        r = gbw.gmoe_route(l, k)
        y, _ = gbw.gnf4_grouped_expert_mlp(x, *gu, *dn, r.expert_offsets, r.row_to_token)
        return gbw.gmoe_combine(y, r.row_of_slot, r.topk_weights), y

    def check(out, y):
        ids, w = mp.route(l.cpu().double().numpy(), k, True)
        rows = mp.plan(ids, E)[2]
        y64 = y.cpu().double().numpy()
        mag = mp.combine(np.abs(y64), rows, w)
        mp.bf16_close(out.cpu().double().numpy(), mp.combine(y64, rows, w), 2.0 ** -18 * mag)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = chain()
    torch.cuda.current_stream().wait_stream(side)
    check(*got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, y = chain()
    for seed in (5, 6):
        g.manual_seed(seed)
        l.copy_(torch.randn((T, E), generator=g, device=DEV))
        x.copy_(torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        check(out, y)
    assert gbw.device_status() == 0


# ---------------------------------------------------------------- refusals


def test_route_refusals():
    with pytest.raises(TypeError, match="logits"):
        gbw.gmoe_route(torch.zeros((2, 8), dtype=torch.float16), 2)
    with pytest.raises(ValueError, match="contiguous"):
        gbw.gmoe_route(torch.zeros((8, 2)).t(), 2)
    with pytest.raises(ValueError, match="T, E"):
        gbw.gmoe_route(torch.zeros(8), 2)
    for k in (0, 9, 33):
        with pytest.raises(ValueError, match="k="):
            gbw.gmoe_route(torch.zeros((2, 8 if k < 33 else 64)), k)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gbw.gmoe_route(torch.zeros((2, 8)), 2)
    ids = torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="dweights"):
        gbw.gmoe_route_bwd(torch.zeros((2, 8)), ids, torch.zeros((2, 2)), torch.zeros((2, 3)))
    with pytest.raises(TypeError, match="topk_ids"):
        gbw.gmoe_route_bwd(torch.zeros((2, 8)), ids.long(), torch.zeros((2, 2)), torch.zeros((2, 2)))


def test_combine_refusals():
    y, rows, slots, w, dout = _combine_inputs(4, 64, 2, 1)
    with pytest.raises(TypeError, match="y must"):
        gbw.gmoe_combine(y.float(), rows, w)
    with pytest.raises(ValueError, match="weights"):
        gbw.gmoe_combine(y, rows, w[:, :1].contiguous())
    with pytest.raises(ValueError, match="out must"):
        gbw.gmoe_combine(y, rows, w, out=torch.empty((4, 72), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="slot_of_row"):
        gbw.gmoe_combine_bwd(dout, y, rows, slots[:-1].contiguous(), w)
    with pytest.raises(ValueError, match="weights are needed"):
        gbw.gmoe_combine_bwd(dout, y, rows, slots, None)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gbw.gmoe_combine(y, rows, w)


def test_route_and_combine_host_validation():
    import ctypes as C
    L, p, NULL, SHAPE, ALIGN = gbw.lib, C.c_void_p(16), 1, 2, 3

    def route(T=4, E=8, k=2, typ=0, logits=p, off=p, ws=p, n=1 << 20):
        return L.gmoe_route(logits, typ, T, E, k, 1, p, p, off, p, p, p, ws, n, None)
    assert route(typ=2) == SHAPE and route(T=-1) == SHAPE and route(E=1025) == SHAPE
    assert route(k=9) == SHAPE and route(E=64, k=33) == SHAPE and route(T=1 << 30, k=4) == SHAPE
    assert route(logits=None) == NULL and route(off=None) == NULL
    assert route(T=200, ws=None) == NULL and route(T=200, n=0) == SHAPE
    assert route(logits=C.c_void_p(18), typ=1) == ALIGN and route(off=C.c_void_p(18)) == ALIGN
    assert L.gmoe_route_workspace(128, 64) == 0
    assert L.gmoe_route_workspace(129, 64) == 5 * 64 * 4
    assert L.gmoe_combine(p, 8, 60, p, p, 4, 2, p, None) == SHAPE
    assert L.gmoe_combine(p, 8, 64, p, p, 4, 33, p, None) == SHAPE
    assert L.gmoe_combine(p, 8, 64, None, p, 4, 2, p, None) == NULL
    assert L.gmoe_combine(C.c_void_p(8), 8, 64, p, p, 4, 2, p, None) == ALIGN
    assert L.gmoe_combine_bwd(p, p, 8, 64, p, p, None, 4, 2, p, p, None) == NULL
    assert L.gmoe_combine_bwd(p, p, 8, 64, p, p, p, 4, 2, C.c_void_p(24), p, None) == ALIGN
    assert L.gmoe_route_bwd(None, 0, 4, 8, 2, 0, p, p, p, p, None) == NULL


@pytest.mark.gpu
def test_a_routing_can_be_saved(tmp_path):
    r = gbw.gmoe_route(torch.randn((200, 16), generator=torch.Generator().manual_seed(0)).to(DEV), 4)
    torch.save(tuple(r), tmp_path / "r.pt")
    for a, b in zip(r, torch.load(tmp_path / "r.pt")):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_a_routing_can_be_copied_and_changed_in_inference_mode():
    import copy
    l = torch.randn((7, 16), generator=torch.Generator().manual_seed(0)).to(DEV)
    ref = gbw.gmoe_route(l, 4)
    with torch.inference_mode():
        r = copy.deepcopy(gbw.gmoe_route(l, 4))
        for a, b in zip(r, ref):
            assert torch.equal(a, b)
        r.topk_ids.add_(1)
        r.topk_weights.mul_(2.0)
        assert torch.equal(r.row_to_token, ref.row_to_token) and torch.equal(r.topk_ids, ref.topk_ids + 1)

"""Tensors whose elements or bytes pass 2^31 and 2^32, at whose far end an offset
held in 32 bits would go wrong; and the library's refusals through the binding."""
import numpy as np
import pytest
import torch

import moe_plain as mp

gbw = pytest.importorskip("grouped_bit_weight_b200")
DEV = "cuda:0"


def _nf4(codes, absmax):
    q = torch.stack([codes >> 4, codes & 15], -1).flatten(-2).long()
    return torch.from_numpy(mp.NF4).to(DEV)[q] * absmax.double().repeat_interleave(64, -1)


def _mxfp4(codes, scales):
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-3 if codes.dim() > scales.dim() else -2).long()
    v = torch.from_numpy(mp.E2M1).to(DEV)[q & 7] * torch.where(q & 8 > 0, -1.0, 1.0).double()
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,T", [("nf4", 2), ("mxfp4", 1), ("mxfp4", 32)])
def test_layer_with_weights_beyond_2_32_bytes(fmt, T):
    """1024 experts of 2048 x 2048, 4.3 GB of gate_up codes; the bias chooses the
    last ones.  (MXFP4: 16 experts of 50 MB a token, so 32 tokens take rows in
    pieces; the layer of one token has fewer than 100 MB.)"""
    E, H, I, k = 1024, 2048, 2048, 16 if T == 32 else 3
    g = torch.Generator(device=DEV).manual_seed(T)
    u8 = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, dtype=torch.uint8, device=DEV)
    if fmt == "nf4":
        gu, dn = u8(0, 256, E, 2 * I, H // 2), u8(0, 256, E, H, I // 2)
        gs, ds = (0.02 * (1 + torch.rand((E, n, K // 64), generator=g, device=DEV)) for n, K in ((2 * I, H), (H, I)))
        call, values = gbw.gnf4_moe_layer, _nf4
    else:
        gu, dn = u8(0, 256, E, 2 * I, H // 32, 16), u8(0, 256, E, H, I // 32, 16)
        gs, ds = u8(118, 122, E, 2 * I, H // 32), u8(118, 122, E, H, I // 32)
        call, values = gbw.gmxfp4_moe_layer, _mxfp4
    assert gu.numel() >= 2 ** 32
    bias = torch.zeros(E, device=DEV)
    last = torch.arange(E - k + 1, E, device=DEV)
    chosen = torch.cat([last, torch.tensor([1], device=DEV)])
    bias[chosen] = 40.0
    rw = torch.zeros((E, H), dtype=torch.bfloat16, device=DEV)  # k equal weights
    x = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
    got = call(x, rw, gu, gs, dn, ds, k=k, router_bias=bias).double()
    assert gbw.device_status() == 0
    ref = torch.zeros((T, H), dtype=torch.float64, device=DEV)
    for e in chosen.tolist():
        a = x.double() @ values(gu[e], gs[e]).T
        ref += torch.nn.functional.silu(a[:, :I]) * a[:, I:] @ values(dn[e], ds[e]).T / k
    # one rounding to bf16, 2^-8 / sqrt(3) at most, and the NF4 levels' 7.5e-4 in
    # gate (times 1.1), up and down; a tenth for the spread
    levels = 7.5e-4 if fmt == "nf4" else 0.0
    assert (got - ref).norm() / ref.norm() < 1.1 * ((1.1 ** 2 + 2) * levels ** 2 + 2.0 ** -16 / 3) ** 0.5


@pytest.mark.gpu
def test_quantise_and_product_beyond_2_31_elements():
    """300011 rows: an output of 2.4e9 elements, and rows of 2.2e9 values."""
    P, E, N, K = 300011, 3, 8136, 64
    g = torch.Generator(device=DEV).manual_seed(1)
    w = torch.randint(0, 256, (E, N, K // 32, 16), generator=g, dtype=torch.uint8, device=DEV)
    ws = torch.randint(118, 122, (E, N, K // 32), generator=g, dtype=torch.uint8, device=DEV)
    off = torch.tensor([0, 5, 150000, P], dtype=torch.int32, device=DEV)
    x = torch.randn((P, K), generator=g, device=DEV).to(torch.bfloat16)
    xq, xs = gbw.gmxfp4_quantize_rows(x)
    out = gbw.gmxfp4_grouped_gemm_a4(xq, xs, w, ws, off)
    assert out.numel() > 2 ** 31 and gbw.device_status() == 0
    rows = torch.tensor([0, 4, 5, 149999, 150000, 263000, 263957, P - 200, P - 1], device=DEV)
    for r in rows.tolist():
        c, s, v = mp.mxfp4(x[r].cpu().double().numpy())
        ref = _mxfp4(w[(r >= 5) + (r >= 150000)], ws[(r >= 5) + (r >= 150000)]).cpu().numpy()
        mp.bf16_close(out[r].cpu().double().numpy(), ref @ v, K * 2.0 ** -24 * (np.abs(ref) @ np.abs(v)))
    del out
    K = 2 ** 13
    rows = torch.randint(0, 100, (270000,), generator=g, dtype=torch.int32, device=DEV)
    x = torch.randn((100, K), generator=g, device=DEV).to(torch.bfloat16)
    assert rows.numel() * K > 2 ** 31
    codes, scales = gbw.gmxfp4_quantize_rows(x, rows)
    c, s = gbw.gmxfp4_quantize_rows(x)
    for part in (slice(0, 1000), slice(261000, 263000), slice(269000, 270000)):
        assert torch.equal(codes[part], c[rows[part].long()])
        assert torch.equal(scales[:, part], s[:, rows[part].long()])
    assert gbw.device_status() == 0


@pytest.mark.gpu
def test_combine_and_its_gradient_beyond_2_31_elements():
    T, k, H = 100003, 8, 2880
    g = torch.Generator(device=DEV).manual_seed(1)
    P = T * k
    slots = torch.randperm(P, generator=g, device=DEV)
    rows = torch.empty_like(slots)
    rows[slots] = torch.arange(P, device=DEV)
    rows, slots = rows.reshape(T, k).int(), slots.int()
    y = torch.empty((P, H), dtype=torch.bfloat16, device=DEV)
    for part in y.split(1 << 17):
        part.copy_(torch.randn(part.shape, generator=g, device=DEV))
    assert y.numel() > 2 ** 31
    w = torch.rand((T, k), generator=g, device=DEV)
    dout = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
    out = gbw.gmoe_combine(y, rows, w)
    dy, dw = gbw.gmoe_combine_bwd(dout, y, rows, slots, w)
    assert gbw.device_status() == 0
    for t in (slice(0, 50), slice(T // 2, T // 2 + 50), slice(T - 50, T)):
        r, w64, d64 = rows[t].long(), w[t].double(), dout[t].double()
        y64 = y[r].double()
        mag = (w64[..., None] * y64.abs()).sum(1)
        mp.bf16_close(out[t].cpu().double().numpy(), (w64[..., None] * y64).sum(1).cpu().numpy(),
                      9 * 2.0 ** -24 * mag.cpu().numpy())
        ref = w64[..., None] * d64[:, None]
        mp.bf16_close(dy[r].cpu().double().numpy(), ref.cpu().numpy(), 2.0 ** -24 * ref.abs().cpu().numpy())
        tol = 2.0 ** -24 * (H / 32 + 14) * (y64.abs() * d64[:, None].abs()).sum(-1)
        assert ((dw[t].double() - (y64 * d64[:, None]).sum(-1)).abs() <= tol).all()
    last = y.flatten()[2 ** 31 - 8:2 ** 31 + 8].clone()
    del y, dy
    assert torch.isfinite(last).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(1 << 21, 1024, 1), (3000017, 8, 4)])
def test_route_of_millions_of_tokens(T, E, k):
    g = torch.Generator(device=DEV).manual_seed(2)
    l = torch.empty((T, E), dtype=torch.bfloat16, device=DEV)
    for part in l.split(1 << 18):
        part.copy_(torch.randn(part.shape, generator=g, device=DEV))
    r = gbw.gmoe_route(l, k)
    assert gbw.device_status() == 0
    flat = r.topk_ids.flatten().long()
    order = torch.sort(flat, stable=True).indices
    assert torch.equal(r.slot_of_row.long(), order)
    assert torch.equal(r.row_to_token.long(), order // k)
    assert torch.equal(r.row_of_slot.flatten().long()[order], torch.arange(T * k, device=DEV))
    n = torch.bincount(flat, minlength=E)
    assert torch.equal(r.expert_offsets[1:].long(), n.cumsum(0))
    for t in (slice(0, 100), slice(T - 100, T)):
        ids, w = mp.route(l[t].cpu().double().numpy(), k, True)
        assert (r.topk_ids[t].cpu().numpy() == ids).all()
        assert np.abs(r.topk_weights[t].cpu().numpy() - w).max() < 2.0 ** -20


@pytest.mark.gpu
def test_refusals_of_the_library_raise_its_error():
    """What the library refuses itself, through the C++ half of the binding."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)
    f32 = lambda *s: torch.zeros(s, device=DEV)
    layer = lambda E, x, **kw: gbw.gnf4_moe_layer(x, bf(E, 64), u8(E, 128, 32), f32(E, 128, 1), u8(E, 64, 32),
                                                  f32(E, 64, 1), 1, **kw)
    for call, status in (
            (lambda: gbw.gmoe_route(bf(2, 1025), 1), 2),
            (lambda: gbw.gmoe_combine(bf(4, 12), i32(2, 2)), 2),
            (lambda: gbw.gmoe_combine(bf(8 * 8 + 1)[1:].view(8, 8), i32(4, 2)), 3),
            (lambda: gbw.gmoe_combine_bwd(bf(2, 12), bf(4, 12), i32(2, 2), i32(4), f32(2, 2)), 2),
            (lambda: gbw.gmxfp4_quantize_rows(bf(64 + 1)[1:].view(1, 64)), 3),
            (lambda: gbw.gmxfp4_grouped_gemm_a4(u8(4, 1, 16), u8(1, 4, 4), u8(2, 12, 1, 16), u8(2, 12, 1), i32(3)), 2),
            (lambda: layer(1025, bf(1, 64)), 2),
            (lambda: layer(4, bf(64 + 1)[1:].view(1, 64)), 3),
            (lambda: layer(4, bf(1, 64), workspace=u8(1 << 20)[1:]), 3)):
        with pytest.raises(gbw.GbwError) as e:
            call()
        assert e.value.status == status
    assert layer(4, bf(1, 64)).shape == (1, 64) and gbw.device_status() == 0

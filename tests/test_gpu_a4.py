"""MXFP4 activations: the row quantiser byte for byte against the 64-bit
definition, and the W4A4 grouped product against the 64-bit sum of the same
4-bit values."""
import ctypes as C

import numpy as np
import pytest
import torch

import moe_plain as mp

gbw = pytest.importorskip("grouped_bit_weight_b200")
DEV = "cuda:0"


def _bf16(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16)


def _codes(t):
    """codes [P, K/32, 16] uint8 -> [P, K] values 0..15, low nibble first."""
    c = t.cpu().numpy().reshape(t.shape[0], -1)
    return np.stack([c & 15, c >> 4], -1).reshape(t.shape[0], -1)


def _scales(t, K):
    """scales [ceil(K/128), P, 4] uint8 -> [P, K/32]; past K they are 127."""
    s = t.cpu().numpy().transpose(1, 0, 2).reshape(t.shape[1], -1)
    assert (s[:, K // 32:] == 127).all()
    return s[:, :K // 32]


def _values(codes, scales):
    q = codes.astype(np.int64)
    v = mp.E2M1[q & 7] * np.where(q & 8, -1.0, 1.0)
    s = scales.astype(np.float64)
    f = np.where(s == 255, np.nan, 2.0 ** (s - 127))
    return v * np.repeat(f, 32, axis=-1)


def _weights(E, N, K, seed, lo=117, hi=122):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    scales = rng.integers(lo, hi, (E, N, K // 32), dtype=np.uint8)
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(E, N, K)
    return codes, scales, _values(nib, scales)


def _offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K", [(1, 32), (3, 96), (64, 512), (7, 2880), (257, 160), (1000, 64)])
def test_quantize_rows_bytes(T, K):
    x = _bf16((T, K), T + K) * (2.0 ** torch.arange(-8, 8).repeat((T + 15) // 16)[:T, None])
    x = x.to(torch.bfloat16)
    codes, scales = gbw.gmxfp4_quantize_rows(x.to(DEV))
    c, s, _ = mp.mxfp4(x.double().numpy())
    assert codes.shape == (T, K // 32, 16) and scales.shape == ((K + 127) // 128, T, 4)
    assert (_scales(scales, K) == s).all() and (_codes(codes) == c).all()
    perm = torch.randint(0, T, (2 * T + 1,), generator=torch.Generator().manual_seed(1))
    codes, scales = gbw.gmxfp4_quantize_rows(x.to(DEV), perm.to(torch.int32).to(DEV))
    assert (_scales(scales, K) == s[perm]).all() and (_codes(codes) == c[perm]).all()
    assert gbw.device_status() == 0


@pytest.mark.gpu
def test_quantize_rows_special_values():
    """Halfway values, saturation, zeros of both signs, subnormals, the largest
    bf16, and blocks that hold NaN or an infinity."""
    x = torch.zeros((10, 64))
    x[0, :16] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25,
                              -1.75, -2.5, -3.5, -5.0, 7.0])
    x[1, :4] = torch.tensor([7.9, -7.9, 4.0, -0.0])
    x[2, 32] = -0.0
    x[3, :3] = torch.tensor([1e-38, -1e-39, 9e-41])
    x[4, 5] = 3.3e38
    x[5, 7] = float("nan")
    x[6, 40] = float("inf")
    x[7, 1], x[7, 2] = float("-inf"), float("nan")
    x[8] = 1.1754944e-38 * torch.arange(64)
    x[9, :2] = torch.tensor([2.0 ** -126, 2.0 ** -133])
    x = x.to(torch.bfloat16)
    codes, scales = gbw.gmxfp4_quantize_rows(x.to(DEV))
    c, s, _ = mp.mxfp4(x.double().numpy())
    assert (_scales(scales, 64) == s).all() and (_codes(codes) == c).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,K", [(1, 32), (33, 288), (130, 2880)])
def test_quantize_rows_swiglu(T, K):
    """silu(gate) * up in fp32 and then rounded to 4 bits: the 64-bit value may
    lie on the other side of a rounding border only when it is nearer to it
    than fp32's own error, 8 roundings of 2^-24."""
    x = _bf16((T, 2 * K), T)
    x[0, :4] = torch.tensor([100.0, -100.0, 0.0, -3e38])
    h = mp.silu(x[:, :K].double().numpy()) * x[:, K:].double().numpy()
    codes, scales = gbw.gmxfp4_quantize_rows(x.to(DEV), swiglu=True)
    got = _values(_codes(codes), _scales(scales, K))
    lo, hi = (mp.mxfp4(h * (1 + s * 2.0 ** -21))[2] for s in (-1, 1))
    mid = mp.mxfp4(h)[2]
    near = (got == lo) | (got == hi) | (got == mid)
    assert near.all() and (got != mid).mean() < 1e-3
    perm = torch.randint(0, T, (T + 3,), dtype=torch.int32)
    c2, s2 = gbw.gmxfp4_quantize_rows(x.to(DEV), perm.to(DEV), swiglu=True)
    assert torch.equal(c2, codes[perm.long().to(DEV)]) and torch.equal(s2, scales[:, perm.long().to(DEV)])


@pytest.mark.gpu
def test_quantize_rows_swiglu_of_gates_far_below_zero():
    """Blocks of gates down to -91, whose silu is about 1e-37: fp32 and the scale
    byte hold it.  Error: __expf's bound, 2 + 1.173 * 91 = 109 steps of 2^-23 or
    2^-16.2, a subnormal e^-91 rounded by 2^-149 or 2^-18.7 of it, 4 roundings."""
    gates = torch.tensor([-80.0, -86.0, -87.0, -87.5, -88.0, -88.5, -89.0, -90.0, -91.0])
    x = torch.empty((4 * len(gates), 128))
    x[:, :64] = gates.repeat(4)[:, None]
    x[:, 64:] = _bf16((len(x), 64), 7).float() * 10.0 ** torch.arange(4).repeat_interleave(len(gates))[:, None]
    x = x.to(torch.bfloat16)
    codes, scales = gbw.gmxfp4_quantize_rows(x.to(DEV), swiglu=True)
    got = _values(_codes(codes), _scales(scales, 64))
    h = mp.silu(x[:, :64].double().numpy()) * x[:, 64:].double().numpy()
    lo, hi = (mp.mxfp4(h * (1 + s * 2.0 ** -15))[2] for s in (-1, 1))
    assert ((got == lo) | (got == hi)).all() and (got != 0).any(1).all()


def _check_product(counts, N, K, seed, rows_pad=0, xstd=None):
    E, P = len(counts), int(sum(counts))
    w, ws, wv = _weights(E, N, K, seed)
    x = _bf16((P + rows_pad, K), seed + 1)
    if xstd is not None:
        x = (x.float() * xstd[:, None]).to(torch.bfloat16)
    xq, xs = gbw.gmxfp4_quantize_rows(x.to(DEV))
    xv = _values(_codes(xq), _scales(xs, K))
    off = _offsets(counts)
    t = lambda a: torch.from_numpy(a).to(DEV)
    out = torch.full((P + rows_pad, N), 7.0, dtype=torch.bfloat16, device=DEV)
    if rows_pad:
        off[-1] = P + rows_pad  # the last expert takes the padding too
    got = gbw.gmxfp4_grouped_gemm_a4(xq, xs, t(w), t(ws), t(off), out=out)
    assert got is out
    got = got.cpu().double().numpy()
    assert gbw.device_status() == 0
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        ref = xv[a:b] @ wv[e].T
        mag = np.abs(xv[a:b]) @ np.abs(wv[e]).T
        # the products are exact; K of them summed in fp32 may each drop what
        # lies below 2^-24 of the sum of magnitudes
        mp.bf16_close(got[a:b], ref, K * 2.0 ** -24 * mag)
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("counts,N,K", [
    ([16], 128, 256), ([1], 8, 32), ([5, 0, 3], 136, 64), ([17, 31], 200, 96),
    ([16] * 8, 256, 512), ([0, 0, 40, 0], 264, 352), ([128, 129, 130], 128, 128),
    ([191, 192, 193], 320, 288), ([383, 384, 385], 128, 544), ([601, 2, 0, 77], 192, 320),
    ([1000], 72, 1024), ([33], 1000, 2912), ([250, 256, 262, 20], 640, 2880), ([255, 256, 257, 319, 320], 136, 640),
    ([3] * 64, 64, 160), ([2, 1] * 20, 2056, 768), ([0, 1] * 500, 64, 64), ([0] * 1023 + [70], 72, 96),
    ([3000], 136, 128)])
def test_product_matches_plain(counts, N, K):
    _check_product(counts, N, K, sum(counts) + N + K)


@pytest.mark.gpu
@pytest.mark.parametrize("counts,pad", [
    ([16], 1), ([0], 5), ([5, 0, 3], 56), ([0, 0, 0], 64), ([17, 31, 0], 300), ([255, 1], 1),
    ([250, 256], 262), ([383, 2, 0], 1000)], ids=str)
def test_product_leaves_rows_behind_the_last_expert_as_they_were(counts, pad):
    """A buffer padded to a fixed number of rows: the last offset is below P, the
    rows behind it hold NaN scales, and no error is raised."""
    E, N, K, P = len(counts), 136, 288, sum(counts)
    w, ws, wv = _weights(E, N, K, P)
    xq, xs = gbw.gmxfp4_quantize_rows(_bf16((P + pad, K), 1).to(DEV))
    xs[:, P:, 0] = 255  # NaN
    xv = _values(_codes(xq), _scales(xs, K))[:P]
    off = _offsets(counts)
    t = lambda a: torch.from_numpy(a).to(DEV)
    out = torch.full((P + pad, N), 7.0, dtype=torch.bfloat16, device=DEV)
    gbw.gmxfp4_grouped_gemm_a4(xq, xs, t(w), t(ws), t(off), out=out)
    assert gbw.device_status() == 0
    assert (out[P:] == 7.0).all()
    got = out[:P].cpu().double().numpy()
    for e in range(E):
        s = slice(off[e], off[e + 1])
        mp.bf16_close(got[s], xv[s] @ wv[e].T, K * 2.0 ** -24 * (np.abs(xv[s]) @ np.abs(wv[e]).T))


@pytest.mark.gpu
@pytest.mark.parametrize("off", [[1, 20, 30, 40], [0, 20, 10, 40], [0, 60, 70, 80], [0, -5, -5, -1],
                                 [0, 10, 20, 51], [0, 2 ** 31 - 1, -2 ** 31, 30]], ids=str)
def test_product_reports_bad_offsets_and_stays_inside_its_rows(off):
    E, N, K, P = 3, 64, 128, 50
    w, ws, _ = _weights(E, N, K, 3)
    t = lambda a: torch.from_numpy(a).to(DEV)
    xq, xs = gbw.gmxfp4_quantize_rows(_bf16((P, K), 1).to(DEV))
    buf = torch.full((P + 60, N), 7.0, dtype=torch.bfloat16, device=DEV)
    gbw.gmxfp4_grouped_gemm_a4(xq, xs, t(w), t(ws), t(np.array(off, np.int32)), out=buf[20:20 + P])
    assert gbw.device_status() == gbw.DEVERR_OFFSETS
    assert (buf[:20] == 7.0).all() and (buf[20 + P:] == 7.0).all()


@pytest.mark.gpu
def test_product_scales_over_a_wide_range():
    """Every row has a magnitude of its own, 2^-60 to 2^60."""
    P = 300
    _check_product([100, 200], 136, 416, 5, xstd=2.0 ** torch.linspace(-60, 60, P))


@pytest.mark.gpu
def test_product_scales_at_every_alignment():
    """Scale arrays that start at odd addresses."""
    E, N, K, P = 3, 136, 512, 60
    w, ws, _ = _weights(E, N, K, 3)
    x = _bf16((P, K), 4).to(DEV)
    xq, xs = gbw.gmxfp4_quantize_rows(x)
    off = torch.from_numpy(_offsets([20, 30, 10])).to(DEV)
    t = lambda a: torch.from_numpy(a).to(DEV)
    ref = gbw.gmxfp4_grouped_gemm_a4(xq, xs, t(w), t(ws), off)

    def shifted(a, n):
        b = torch.empty(a.numel() + 16, dtype=torch.uint8, device=DEV)
        b[n:n + a.numel()] = a.flatten()
        return b[n:n + a.numel()].view(a.shape)

    for n in (1, 2, 4, 6):
        got = gbw.gmxfp4_grouped_gemm_a4(xq, shifted(xs, 4), t(w), shifted(t(ws), n), off)
        assert torch.equal(got, ref)
    assert gbw.device_status() == 0


@pytest.mark.gpu
def test_product_nan_scale_marks_its_rows_and_columns_only():
    E, N, K, P = 2, 136, 256, 40
    w, ws, _ = _weights(E, N, K, 3)
    ws[0, 9, 3] = 255
    x = _bf16((P, K), 4)
    x[7, 100] = float("inf")
    x[30, 0] = float("nan")
    off = _offsets([20, 20])
    t = lambda a: torch.from_numpy(a).to(DEV)
    xq, xs = gbw.gmxfp4_quantize_rows(x.to(DEV))
    got = gbw.gmxfp4_grouped_gemm_a4(xq, xs, t(w), t(ws), t(off)).cpu()
    bad = torch.isnan(got)
    want = torch.zeros_like(bad)
    want[7] = want[30] = True
    want[:20, 9] = True
    assert torch.equal(bad, want)


@pytest.mark.gpu
def test_quantise_and_product_on_two_streams_and_in_inference_mode():
    E, N, K = 4, 264, 416
    w, ws, _ = _weights(E, N, K, 3)
    t = lambda a: torch.from_numpy(a).to(DEV)
    w, ws, calls = t(w), t(ws), []
    for i, counts in enumerate(([100, 0, 30, 7], [1, 290, 3, 64])):
        x, off = _bf16((sum(counts), K), i).to(DEV), t(_offsets(counts))
        calls.append((x, off, gbw.gmxfp4_grouped_gemm_a4(*gbw.gmxfp4_quantize_rows(x), w, ws, off)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    with torch.inference_mode():
        for _ in range(20):
            for s, (x, off, ref) in zip(streams, calls):
                with torch.cuda.stream(s):
                    q = gbw.gmxfp4_quantize_rows(x)
                    got.append((gbw.gmxfp4_grouped_gemm_a4(*q, w, ws, off), ref))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in got) and gbw.device_status() == 0


@pytest.mark.gpu
def test_product_in_a_graph_behind_every_kind_of_node():
    """First in the graph; behind a copy, a fill, and two streams that join."""
    E, N, K = 4, 264, 416
    w, ws, _ = _weights(E, N, K, 3)
    t = lambda a: torch.from_numpy(a).to(DEV)
    w, ws, off = t(w), t(ws), t(_offsets([100, 0, 30, 7]))
    x = [_bf16((137, K), i).to(DEV) for i in range(2)]
    q = [gbw.gmxfp4_quantize_rows(v) for v in x]
    ref = [gbw.gmxfp4_grouped_gemm_a4(*v, w, ws, off) for v in q]
    codes, scales = (v.clone() for v in q[0])
    call = lambda out: gbw.gmxfp4_grouped_gemm_a4(codes, scales, w, ws, off, out=out)
    outs = [torch.empty_like(ref[0]) for _ in range(4)]
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(outs[0])
        codes.copy_(q[1][0])
        scales.copy_(q[1][1])
        call(outs[1])
        outs[2].zero_()
        call(outs[2])
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            codes.copy_(q[0][0])
        scales.copy_(q[0][1])
        main.wait_stream(side)
        call(outs[3])
    for _ in range(3):
        for o in outs:
            o.fill_(float("nan"))
        g.replay()
        for o, r in zip(outs, (ref[0], ref[1], ref[1], ref[0])):
            assert torch.equal(o, r)
    assert gbw.device_status() == 0


@pytest.mark.gpu
def test_product_without_rows_bad_offsets_and_repeats():
    E, N, K = 3, 64, 128
    w, ws, _ = _weights(E, N, K, 3)
    t = lambda a: torch.from_numpy(a).to(DEV)
    xq, xs = gbw.gmxfp4_quantize_rows(_bf16((0, K), 1).to(DEV))
    assert gbw.gmxfp4_grouped_gemm_a4(xq, xs, t(w), t(ws), t(_offsets([0, 0, 0]))).shape == (0, N)
    xq, xs = gbw.gmxfp4_quantize_rows(_bf16((50, K), 1).to(DEV))
    a = gbw.gmxfp4_grouped_gemm_a4(xq, xs, t(w), t(ws), t(_offsets([20, 0, 30])))
    b = gbw.gmxfp4_grouped_gemm_a4(xq, xs, t(w), t(ws), t(_offsets([20, 0, 30])))
    assert torch.equal(a, b) and gbw.device_status() == 0
    gbw.gmxfp4_grouped_gemm_a4(xq, xs, t(w), t(ws), t(np.array([0, 60, 30, 50], np.int32)))
    assert gbw.device_status() == gbw.DEVERR_OFFSETS
    bad = torch.tensor([0, 50, -1], dtype=torch.int32, device=DEV)
    gbw.gmxfp4_quantize_rows(_bf16((50, K), 1).to(DEV), bad)
    assert gbw.device_status() == gbw.DEVERR_TOKEN


@pytest.mark.gpu
def test_prompt_layer_in_mxfp4_from_routing_to_combine_in_a_graph():
    """route -> quantise -> gate_up -> SwiGLU + quantise -> down -> combine, as
    a prompt runs it, captured and replayed on other inputs, each step against
    the 64-bit value of what went into it."""
    T, E, k, H, I = 200, 8, 2, 256, 192
    gw, gs, gv = _weights(E, 2 * I, H, 1)
    dw, ds, dv = _weights(E, H, I, 2)
    d = [torch.from_numpy(a).to(DEV) for a in (gw, gs, dw, ds)]
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
    l = torch.randn((T, E), generator=g, device=DEV)

    def layer():
        r = gbw.gmoe_route(l, k)
        q = gbw.gmxfp4_quantize_rows(x, r.row_to_token)
        a = gbw.gmxfp4_grouped_gemm_a4(*q, d[0], d[1], r.expert_offsets)
        h = gbw.gmxfp4_quantize_rows(a, swiglu=True)
        y = gbw.gmxfp4_grouped_gemm_a4(*h, d[2], d[3], r.expert_offsets)
        return r, q, a, h, y, gbw.gmoe_combine(y, r.row_of_slot, r.topk_weights)

    def check(r, q, a, h, y, out):
        ids, w = mp.route(l.cpu().double().numpy(), k, True)
        off, r2t, ros, _ = mp.plan(ids, E)
        assert (r.row_to_token.cpu().numpy() == r2t).all()
        xv = mp.mxfp4(x.cpu().double().numpy())[2][r2t]
        hv = _values(_codes(h[0]), _scales(h[1], I))
        a64, y64 = a.cpu().double().numpy(), y.cpu().double().numpy()
        for e in range(E):
            s = slice(off[e], off[e + 1])
            mp.bf16_close(a64[s], xv[s] @ gv[e].T, H * 2.0 ** -24 * (np.abs(xv[s]) @ np.abs(gv[e]).T))
            mp.bf16_close(y64[s], hv[s] @ dv[e].T, I * 2.0 ** -24 * (np.abs(hv[s]) @ np.abs(dv[e]).T))
        want = mp.mxfp4(mp.silu(a64[:, :I]) * a64[:, I:])[2]
        assert (hv != want).mean() < 1e-3
        mp.bf16_close(out.cpu().double().numpy(), mp.combine(y64, ros, w),
                      2.0 ** -18 * mp.combine(np.abs(y64), ros, w))

    check(*layer())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer()
    for seed in (5, 6):
        g.manual_seed(seed)
        l.copy_(torch.randn((T, E), generator=g, device=DEV))
        x.copy_(torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        check(*got)
    assert gbw.device_status() == 0


# ---------------------------------------------------------------- refusals


def test_a4_refusals():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="x must"):
        gbw.gmxfp4_quantize_rows(x.float())
    with pytest.raises(ValueError, match="multiple of 32"):
        gbw.gmxfp4_quantize_rows(x[:, :48].contiguous())
    with pytest.raises(ValueError, match="multiple of 32"):
        gbw.gmxfp4_quantize_rows(x[:, :32].contiguous(), swiglu=True)
    with pytest.raises(ValueError, match="contiguous"):
        gbw.gmxfp4_quantize_rows(x[:, ::2])
    with pytest.raises(ValueError, match="no rows"):
        gbw.gmxfp4_quantize_rows(x[:0], torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA tensor"):
        gbw.gmxfp4_quantize_rows(x)
    a = dict(x_codes=u8(4, 2, 16), x_scales=u8(1, 4, 4), blocks=u8(3, 8, 2, 16), scales=u8(3, 8, 2),
             expert_offsets=torch.zeros(4, dtype=torch.int32))
    for name, bad, text in (("x_codes", u8(4, 32), "x_codes"), ("x_codes", u8(5, 2, 16), "x_scales"),
                            ("scales", u8(3, 8, 3), "scales"),
                            ("blocks", u8(3, 8, 3, 16), "packed weights"),
                            ("expert_offsets", torch.zeros(3, dtype=torch.int32), "expert_offsets"),
                            ("x_scales", u8(4, 2), "x_scales")):
        with pytest.raises(ValueError, match=text):
            gbw.gmxfp4_grouped_gemm_a4(**{**a, name: bad})
    with pytest.raises(ValueError, match="out must"):
        gbw.gmxfp4_grouped_gemm_a4(**a, out=torch.zeros((4, 16), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA tensor"):
        gbw.gmxfp4_grouped_gemm_a4(**a)


def test_a4_host_validation():
    L, p, NULL, SHAPE, ALIGN = gbw.lib, C.c_void_p(16), 1, 2, 3

    def q(x=p, T=4, K=64, r2t=None, P=4, codes=p, scales=p):
        return L.gmxfp4_quantize_rows(x, T, K, r2t, P, 0, codes, scales, None)
    assert q(K=48) == SHAPE and q(K=(1 << 24) + 32) == SHAPE and q(T=3) == SHAPE and q(P=-1) == SHAPE and q(T=0, r2t=p) == SHAPE
    assert q(x=None) == NULL and q(scales=None) == NULL
    assert q(x=C.c_void_p(24)) == ALIGN and q(codes=C.c_void_p(18)) == ALIGN

    def g(xc=p, P=4, K=64, w=p, ws=p, E=2, N=64, off=p, out=p):
        return L.gmxfp4_grouped_gemm_a4(xc, p, P, K, w, ws, E, N, off, out, None)
    assert g(K=48) == SHAPE and g(N=60) == SHAPE and g(E=1025) == SHAPE and g(P=-1) == SHAPE
    assert g(E=1000, N=1 << 24) == SHAPE
    assert g(w=None) == NULL and g(off=None) == NULL and g(out=None) == NULL
    assert g(xc=C.c_void_p(24)) == ALIGN and g(w=C.c_void_p(8)) == ALIGN
    assert g(off=C.c_void_p(18)) == ALIGN

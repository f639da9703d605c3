"""The whole mixture-of-experts layer for a few tokens against a plain 64-bit
layer: every format, token count, split and mask, on streams, in graphs and
with two calls at once."""
import ctypes as C

import numpy as np
import pytest
import torch

import moe_plain as mp

gbw = pytest.importorskip("grouped_bit_weight_b200")
DEV = "cuda:0"


def _levels_error():
    """Largest relative error of an NF4 level in the kernel's table: 1.437
    times the level, rounded to bf16."""
    v = torch.from_numpy(mp.NF4) * float(np.float32(1.437))
    r = v.to(torch.bfloat16).double()
    nz = v != 0
    return float(((r - v)[nz] / v[nz]).abs().max())


def _pack(fmt, E, N, K, rng, std):
    """(codes, scales, 64-bit weights) of random 4-bit weights."""
    codes = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    lo, hi = codes & 15, codes >> 4
    if fmt == "nf4":
        q = np.stack([hi, lo], -1).reshape(E, N, K)
        s = (std * (2 + rng.random((E, N, K // 64)))).astype(np.float32)
        return codes, s, mp.NF4[q] * np.repeat(s.astype(np.float64), 64, -1)
    q = np.stack([lo, hi], -1).reshape(E, N, K)
    s = rng.integers(118, 122, (E, N, K // 32), dtype=np.uint8)
    v = mp.E2M1[q & 7] * np.where(q & 8, -1.0, 1.0)
    return (codes.reshape(E, N, K // 32, 16), s,
            v * np.repeat(2.0 ** (s.astype(np.float64) - 127), 32, -1))


class Layer:
    def __init__(self, fmt, E, k, H, I, seed=0, renorm=True, bias=False):
        rng = np.random.default_rng(seed)
        self.fmt, self.E, self.k, self.H, self.I, self.renorm = fmt, E, k, H, I, renorm
        self.gu = _pack(fmt, E, 2 * I, H, rng, 1 / np.sqrt(H))
        self.dn = _pack(fmt, E, H, I, rng, 1 / np.sqrt(I))
        self.rw = torch.from_numpy(rng.standard_normal((E, H)) * 1.5 / np.sqrt(H)).to(torch.bfloat16)
        self.rb = torch.from_numpy(rng.standard_normal(E) * 0.5).float() if bias else None
        t = lambda a: torch.from_numpy(a).to(DEV)
        self.args = (self.rw.to(DEV), t(self.gu[0]), t(self.gu[1]), t(self.dn[0]), t(self.dn[1]))
        self.kw = dict(k=k, renormalize=renorm, router_bias=None if self.rb is None else self.rb.to(DEV))
        self.fn = gbw.gnf4_moe_layer if fmt == "nf4" else gbw.gmxfp4_moe_layer

    def __call__(self, x, **kw):
        return self.fn(x, *self.args, **self.kw, **kw)

    def plain(self, x):
        """(out, allowed error, tokens whose choice is not near a tie)."""
        x = x.cpu().double().numpy()
        l = x @ self.rw.double().numpy().T
        mag = np.abs(x) @ np.abs(self.rw.double().numpy()).T
        if self.rb is not None:
            l = l + self.rb.double().numpy()
        ids, w = mp.route(l, self.k, self.renorm)
        # logits: products of bf16 exact, fp32 chains of at most H / 256 and
        # then 13 steps, each 2^-24 of the magnitudes: an absolute error dl,
        # and a relative one of 2 dl (+ 16 roundings) in the weights
        dl = 2.0 ** -24 * (self.H / 256 * 8 + 16) * mag.max(1)
        s = -np.sort(-l, 1)
        far = np.ones(len(l), bool)
        if self.k < self.E:
            far = s[:, self.k - 1] - s[:, self.k] > 2 * dl
        dw = 4 * dl + 16 * 2.0 ** -24
        # gate and up: each weight off by `lev`, sums of H products in fp32
        lev = _levels_error() + 2.0 ** -22 if self.fmt == "nf4" else 0.0
        e1, e2 = (lev + (n + 8) * 2.0 ** -24 for n in (self.H, self.I))
        out, tol = np.zeros_like(x), np.zeros_like(x)
        for t in range(len(x)):
            for e, we in zip(ids[t], w[t]):
                if we == 0:
                    continue
                a = self.gu[2][e] @ x[t]
                m = np.abs(self.gu[2][e]) @ np.abs(x[t])
                g, u, dg, du = a[:self.I], a[self.I:], e1 * m[:self.I], e1 * m[self.I:]
                h = mp.silu(g) * u
                # |silu'| <= 1.1; h is kept to 2^-16, silu to 8 roundings
                dh = 1.1 * dg * (np.abs(u) + du) + np.abs(mp.silu(g)) * du + 2.0 ** -16 * np.abs(h)
                y = self.dn[2][e] @ h
                dy = np.abs(self.dn[2][e]) @ (dh + e2 * np.abs(h))
                out[t] += we * y
                tol[t] += we * (dy + dw[t] * np.abs(y)) + (self.k + 1) * 2.0 ** -24 * we * np.abs(y)
        return out, tol, far

    def check(self, x, got):
        ref, tol, far = self.plain(x)
        assert far.all(), "the inputs have a choice next to a tie: choose another seed"
        mp.bf16_close(got.cpu().double().numpy(), ref, tol)
        # the bound above is for the worst signs: most errors are far inside
        err = np.linalg.norm(got.cpu().double().numpy() - ref) / max(np.linalg.norm(ref), 1e-30)
        assert err < 4e-3, err
        assert gbw.device_status() == 0


def _x(T, H, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, H), generator=g) * std).to(torch.bfloat16).to(DEV)


SHAPES = [  # T, E, k, H, I
    (1, 1, 1, 64, 64), (1, 8, 2, 128, 64), (2, 4, 4, 192, 320), (3, 16, 8, 512, 128),
    (7, 8, 1, 320, 192), (8, 32, 8, 256, 448), (9, 2, 2, 576, 64), (31, 6, 3, 128, 704),
    (32, 8, 4, 256, 256), (32, 1, 1, 448, 128), (32, 40, 16, 128, 64), (17, 300, 5, 64, 64),
    (5, 1024, 3, 64, 64), (1, 8, 8, 2048, 768), (4, 4, 2, 704, 1472)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_layer_matches_plain(shape, fmt):
    T, E, k, H, I = shape
    n = sum(shape)
    m = Layer(fmt, E, k, H, I, seed=n, renorm=n % 2 == 0, bias=n % 3 == 0)
    x = _x(T, H, n)
    m.check(x, m(x))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
@pytest.mark.parametrize("T", [1, 32])
def test_layer_all_tokens_on_the_same_experts(T, fmt):
    """The bias sends every token to the same experts: one of them gets all
    rows, and most experts none."""
    m = Layer(fmt, 16, 3, 512, 320, seed=T)
    m.kw["router_bias"] = torch.zeros(16, device=DEV)
    m.kw["router_bias"][[2, 7, 15]] = 50.0
    m.rb = m.kw["router_bias"].cpu()
    x = _x(T, 512, 5)
    m.check(x, m(x))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
def test_layer_inputs_far_from_one(fmt):
    """Rows of very different magnitude, a row of zeros among them."""
    m = Layer(fmt, 8, 2, 256, 128, seed=3)
    scale = torch.tensor([1e-12, 1e-4, 0.0, 30.0, 1.0, 1e-30])[:, None].to(DEV)
    x = (_x(6, 256, 4).float() * scale).to(torch.bfloat16)
    ref, tol, far = m.plain(x)
    keep = far.copy()
    keep[[0, 2, 5]] = True  # logits of (nearly) zero: the tie goes to the lowest index
    got = m(x).cpu().double().numpy()
    assert (got[2] == 0).all()
    for t in (1, 3, 4):
        assert far[t]
        mp.bf16_close(got[t], ref[t], tol[t])
    assert np.isfinite(got).all() and gbw.device_status() == 0


@pytest.mark.gpu
def test_layer_ties_masked_experts_and_bad_rows():
    """Equal logits choose the lowest experts; a bias of -inf or of the lowest
    value masks an expert; a token of NaN or infinity stays in its own row."""
    m = Layer("nf4", 12, 4, 128, 64, seed=9)
    m.rw.zero_()
    m.args[0].zero_()
    x = _x(5, 128, 1)
    m.kw["router_bias"] = torch.zeros(12, device=DEV)
    m.kw["router_bias"][0] = float("-inf")
    m.kw["router_bias"][1] = torch.finfo(torch.float32).min
    m.rb = m.kw["router_bias"].cpu()
    ref, tol, _ = m.plain(x)
    mp.bf16_close(m(x).cpu().double().numpy(), ref, tol)  # experts 2, 3, 4, 5, a quarter each
    m.kw["router_bias"] = torch.full((12,), float("-inf"), device=DEV)
    m.rb = m.kw["router_bias"].cpu()
    assert (m(x) == 0).all()                              # nothing left: weights of zero
    m.kw["router_bias"][7] = 1.0                          # one expert left of the four asked for
    m.rb = m.kw["router_bias"].cpu()
    ref, tol, _ = m.plain(x)
    mp.bf16_close(m(x).cpu().double().numpy(), ref, tol)
    good = m(x)
    x[1, 3] = float("nan")
    x[3, 0] = float("inf")
    got = m(x)
    assert torch.equal(got[[0, 2, 4]], good[[0, 2, 4]])
    # (a row of NaN logits has no expert at all: its output is zero)
    assert gbw.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
def test_layer_rows_do_not_depend_on_the_batch(fmt):
    """A token's output is bit for bit the same alone and in a batch whenever
    the split of its sums is the same; and repeats are identical."""
    m = Layer(fmt, 16, 4, 256, 192, seed=6)
    x = _x(24, 256, 8)
    a = m(x)
    for _ in range(3):
        assert torch.equal(m(x), a)
    perm = torch.randperm(24, generator=torch.Generator().manual_seed(2)).to(DEV)
    assert torch.equal(m(x[perm].contiguous()), a[perm])


@pytest.mark.gpu
def test_layer_workspaces_streams_graphs_and_two_calls_at_once():
    m, n = Layer("nf4", 16, 4, 256, 128, seed=1), Layer("mxfp4", 8, 2, 512, 256, seed=2)
    x, z = _x(5, 256, 1), _x(9, 512, 2)
    a, b = m(x), n(z)
    m.check(x, a)
    n.check(z, b)
    # a workspace and an output of the caller's, full of garbage
    need = gbw.lib.gmoe_layer_workspace(5, 16, 4, 256, 128)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    out = torch.full((5, 256), float("nan"), dtype=torch.bfloat16, device=DEV)
    for _ in range(2):
        assert m(x, out=out, workspace=ws) is out and torch.equal(out, a)
    # two streams at once, many calls each
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(40):
        with torch.cuda.stream(s1):
            got.append((m(x), a))
        with torch.cuda.stream(s2):
            got.append((n(z), b))
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in got)
    # two graphs, replayed on two streams at once, on other inputs
    graphs = []
    for layer, inp in ((m, x), (n, z)):
        layer(inp)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = layer(inp)
        graphs.append((g, o))
    x.copy_(_x(5, 256, 11))
    z.copy_(_x(9, 512, 12))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (g, _) in zip((s1, s2), graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    m.check(x, graphs[0][1])
    n.check(z, graphs[1][1])
    assert torch.equal(graphs[0][1], m(x)) and torch.equal(graphs[1][1], n(z))


@pytest.mark.gpu
def test_layer_equals_route_experts_combine():
    """The layer against the calls a larger batch makes, within the roundings
    of the intermediate tensors those store in bf16."""
    m = Layer("nf4", 8, 2, 256, 128, seed=4)
    x = _x(32, 256, 3)
    l = (x.float() @ m.args[0].float().T).contiguous()
    r = gbw.gmoe_route(l, 2)
    y, _ = gbw.gnf4_grouped_expert_mlp(x, *m.args[1:], r.expert_offsets, r.row_to_token)
    z = gbw.gmoe_combine(y, r.row_of_slot, r.topk_weights).float()
    d = (m(x).float() - z).norm() / z.norm()
    assert d < 1.5e-2  # gate, up, h, y and out each rounded to 2^-8, weights too


@pytest.mark.gpu
def test_layer_without_tokens():
    m = Layer("nf4", 4, 2, 64, 64)
    assert m(torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)).shape == (0, 64)


# ---------------------------------------------------------------- many weights


def _blocks_max(a):
    """The largest magnitude of each 32 columns, at every one of them."""
    m = a.abs().reshape(*a.shape[:-1], -1, 32).amax(-1, keepdim=True)
    return m.expand(*m.shape[:-1], 32).reshape(a.shape)


class Large:
    """An MXFP4 layer whose active experts hold more than 100 MB, which takes
    rows in eight 4-bit pieces; its 64-bit values are computed on the GPU."""

    def __init__(self, E, k, H, I, seed, renorm=True):
        g = torch.Generator(device=DEV).manual_seed(seed)
        u8 = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, dtype=torch.uint8, device=DEV)
        self.E, self.k, self.H, self.I, self.renorm = E, k, H, I, renorm
        self.gu, self.gs = u8(0, 256, E, 2 * I, H // 32, 16), u8(117, 122, E, 2 * I, H // 32)
        self.dn, self.ds = u8(0, 256, E, H, I // 32, 16), u8(117, 122, E, H, I // 32)
        self.rw = (torch.randn((E, H), generator=g, device=DEV) * 1.5 / H ** 0.5).to(torch.bfloat16)
        self.rb = torch.zeros(E, device=DEV)

    def __call__(self, x, **kw):
        return gbw.gmxfp4_moe_layer(x, self.rw, self.gu, self.gs, self.dn, self.ds, k=self.k,
                                    renormalize=self.renorm, router_bias=self.rb, **kw)

    def weight(self, codes, scales, e):
        q = torch.stack([codes[e] & 15, codes[e] >> 4], -1).reshape(codes.shape[1], -1, 32).long()
        v = torch.from_numpy(mp.E2M1).to(DEV)[q & 7] * torch.where(q & 8 > 0, -1.0, 1.0).double()
        return (v * torch.exp2(scales[e].double() - 127)[..., None]).reshape(codes.shape[1], -1)

    def check(self, x, got):
        xd = x.double()
        l = (xd @ self.rw.double().T + self.rb.double()).cpu().numpy()
        mag = (xd.abs() @ self.rw.double().abs().T).cpu().numpy()
        ids, w = mp.route(l, self.k, self.renorm)
        dl = 2.0 ** -24 * (self.H / 256 * 8 + 16) * mag.max(1)
        s = -np.sort(-l, 1)
        if self.k < self.E:
            assert (s[:, self.k - 1] - s[:, self.k] > 2 * dl).all(), "a choice next to a tie"
        ref, tol = torch.zeros_like(xd), torch.zeros_like(xd)
        # a row is kept to 2^-16 of the largest of each 32 values m (each piece
        # leaves a quarter of it); the pieces' magnitudes are at most
        # m (1 + 1/4 + 1/16 + ..), of whose sum each of the n products and 8 sums
        # may drop 2^-24
        keep = lambda n: 2.0 ** -16 + 4 / 3 * (n + 8) * 2.0 ** -24
        for e in np.unique(ids):
            t, j = np.nonzero((ids == e) & (w != 0))
            if not len(t):
                continue
            gw, dw = self.weight(self.gu, self.gs, e), self.weight(self.dn, self.ds, e)
            t = torch.from_numpy(t).to(DEV)
            a, da = xd[t] @ gw.T, keep(self.H) * (_blocks_max(xd[t]) @ gw.abs().T)
            (g, u), (dg, du) = a.split(self.I, 1), da.split(self.I, 1)
            h = torch.nn.functional.silu(g) * u
            # |silu'| <= 1.1, silu to 8 roundings
            dh = 1.1 * dg * (u.abs() + du) + torch.nn.functional.silu(g).abs() * du + 8 * 2.0 ** -24 * h.abs()
            y = h @ dw.T
            dy = dh @ dw.abs().T + keep(self.I) * (_blocks_max(h.abs() + dh) @ dw.abs().T)
            we = torch.from_numpy(w[t.cpu().numpy(), j]).to(DEV)[:, None]
            rel = torch.from_numpy(4 * dl + (16 + self.k) * 2.0 ** -24).to(DEV)[t][:, None]
            ref.index_add_(0, t, we * y)
            tol.index_add_(0, t, we * (dy + rel * y.abs()))
        got, ref, tol = (v.cpu().double().numpy() for v in (got, ref, tol))
        mp.bf16_close(got, ref, tol)
        err = np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-30)
        assert err < 2.0 ** -8 / 3 ** 0.5 * 1.1, err  # one rounding to bf16, evenly spread, and little else
        assert gbw.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [  # T, E, k, H, I
    (4, 32, 4, 2880, 2880), (1, 8, 8, 2880, 3648), (5, 16, 4, 2112, 4160), (17, 1024, 16, 704, 576),
    (32, 10, 2, 4032, 2112), (31, 6, 6, 64, 217024)], ids=str)
def test_large_layer_matches_plain(shape):
    T, E, k, H, I = shape
    m = Large(E, k, H, I, sum(shape), renorm=T % 2 == 0)
    x = _x(T, H, T)
    m.check(x, m(x))


@pytest.mark.gpu
def test_large_layer_rows_streams_and_graphs():
    """All tokens on the same experts; rows of every magnitude, zero, infinite
    and NaN; any order of the batch; two streams and a replayed graph."""
    T, E, k, H, I = 32, 12, 3, 2112, 3456
    m = Large(E, k, H, I, 5)
    x = _x(T, H, 6)
    a = m(x)
    m.check(x, a)
    perm = torch.randperm(T, generator=torch.Generator().manual_seed(2)).to(DEV)
    assert torch.equal(m(x), a) and torch.equal(m(x[perm].contiguous()), a[perm])
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s, v, ref in ((s1, x, a), (s2, x[perm].contiguous(), a[perm])):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append((m(v), ref, v))
    torch.cuda.synchronize()
    assert all(torch.equal(u, r) for u, r, _ in got)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = m(x)
    m.rb[[1, 4, 9]] = 50.0
    x.copy_(_x(T, H, 7) * torch.logspace(-6, 1, T, base=10.0).to(DEV)[:, None])
    x[3] = 0
    g.replay()
    m.check(x, o)
    good = m(x)
    assert torch.equal(good, o) and (good[3] == 0).all()
    x[8, 5], x[20, 700] = float("inf"), float("nan")
    got = m(x)
    rest = [t for t in range(T) if t not in (8, 20)]
    assert torch.equal(got[rest], good[rest]) and gbw.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("ratio", [10, 17, 21])
@pytest.mark.parametrize("where", ["x", "h"])
def test_large_layer_with_a_large_value_in_every_block(where, ratio):
    """Of each 32 values of h one is 2^ratio times the others, of x three are 2^ratio,
    2^(2 ratio / 3) and 2^(ratio / 3) times them, and their weights are zero: the
    others make the result, at full precision."""
    E, H, I = 32, 2880, 2880
    m = Large(E, 4, H, I, ratio)
    x = _x(4, H, 4)
    if where == "x":
        for i, c in enumerate((4, 6, 8)):
            x[:, c::32] *= 2.0 ** (ratio * (i + 1) // 3)
            m.rw[:, c::32] = 0
            m.gu[..., c // 2] &= 0xF0  # column c of each block: a byte's low nibble
    else:
        m.gs[:, I + 6::32] += ratio    # the up rows of columns 6
        m.dn[..., 3] &= 0xF0
    m.check(x, m(x))


@pytest.mark.gpu
def test_layers_in_graphs_behind_copies_and_one_another():
    """Layers of both kinds one behind the other in a graph, in between copies,
    fills and a join of two streams, sharing one workspace."""
    small, nf4, large = Layer("mxfp4", 8, 2, 512, 256, seed=2), Layer("nf4", 16, 4, 512, 128, seed=1), \
        Large(6, 3, 512, 44032, 3)
    x = [_x(9, 512, i) for i in range(2)]
    layers = (large, nf4, large, small, large)
    need = max(gbw.lib.gmoe_layer_workspace(9, m.E, m.k, m.H, m.I) for m in layers)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    refs = [[m(v) for m in layers] for v in x]
    buf, side, g = x[0].clone(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    outs = [torch.empty_like(buf) for _ in range(10)]
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        for i in range(2):
            for j, m in enumerate(layers):
                m(buf, out=outs[5 * i + j], workspace=ws)
            if i == 0:
                ws.fill_(255)
                side.wait_stream(main)
                with torch.cuda.stream(side):
                    buf.copy_(x[1])
                main.wait_stream(side)
        buf.copy_(x[0])
    for _ in range(5):
        for o in outs:
            o.fill_(float("nan"))
        g.replay()
        for o, r in zip(outs, refs[0] + refs[1]):
            assert torch.equal(o, r)
    assert gbw.device_status() == 0


def _check_bad_tokens(m, x, nan, inf):
    """A token that holds a NaN gives NaN throughout, one that holds an infinity
    nothing finite, a masked one zeros, the others what they gave before."""
    good = m(x)
    x[nan, 3] = float("nan")
    x[inf, 5] = float("inf")
    got = m(x)
    rest = [t for t in range(len(x)) if t not in (nan, inf)]
    assert torch.equal(got[rest], good[rest]) and torch.isfinite(good).all()
    assert torch.isnan(got[nan]).all() and not torch.isfinite(got[inf]).any()
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
def test_layer_of_a_token_with_nan_is_nan(fmt, renorm):
    m = Layer(fmt, 12, 4, 256, 128, seed=9, renorm=renorm)
    x = _x(5, 256, 1)
    _check_bad_tokens(m, x, 1, 3)
    # an expert of NaN logits is masked, as gmoe_route masks it
    m.kw["router_bias"] = torch.zeros(12, device=DEV)
    m.kw["router_bias"][7] = float("nan")
    a = m(x)
    m.kw["router_bias"][7] = float("-inf")
    b = m(x)
    assert torch.equal(a[[0, 2, 4]], b[[0, 2, 4]])
    # without any expert: zeros, but for the token of NaN
    m.kw["router_bias"].fill_(float("-inf"))
    got = m(x)
    assert (got[[0, 2, 4]] == 0).all() and torch.isnan(got[1]).all()
    assert gbw.device_status() == 0


@pytest.mark.gpu
def test_large_layer_of_a_token_with_nan_is_nan():
    m = Large(12, 3, 2112, 3456, 5)
    x = _x(9, 2112, 6)
    _check_bad_tokens(m, x, 2, 7)
    m.rb.fill_(float("-inf"))
    got = m(x)
    rest = [t for t in range(9) if t not in (2, 7)]
    assert (got[rest] == 0).all() and torch.isnan(got[2]).all()
    assert gbw.device_status() == 0


# ---------------------------------------------------------------- rows and batches


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
def test_layer_values_of_tiny_and_huge_rows(fmt):
    """Rows of very different magnitude, each against its own 64-bit value at its
    own scale; the bias chooses their experts, different ones for equal logits.
    (Of 1e-20 and 1e-30, h is below what fp32 holds: zeros.)"""
    m = Layer(fmt, 8, 2, 256, 128, seed=3)
    m.rb = torch.tensor([0.5, -1.0, 3.0, 0.25, -2.0, 2.5, 0.0, 1.0])
    m.kw["router_bias"] = m.rb.to(DEV)
    scale = torch.tensor([1e-12, 1e-4, 0.0, 30.0, 1.0, 1e-30, 1e-8, 1e-15, 1e-20, 3e4, 1e-17])[:, None].to(DEV)
    x = (_x(len(scale), 256, 4).float() * scale).to(torch.bfloat16)
    got = m(x)
    for t in range(len(x)):
        m.check(x[t:t + 1], got[t:t + 1])
    assert (got[2] == 0).all() and (got[0].abs() > 1e-30).any() and (got[9].abs() > 1e6).any()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
def test_layer_of_single_tokens_and_parts_of_a_batch(fmt):
    """A token alone, in a part of the batch and in the whole: the sums may be
    split otherwise, so each is held to the 64-bit value, and two of them to one
    another by twice the allowed error and a rounding each."""
    m = Layer(fmt, 16, 4, 256, 192, seed=6)
    x = _x(24, 256, 8)
    whole = m(x)
    _, tol, _ = m.plain(x)
    for a, b in ((0, 1), (5, 6), (23, 24), (0, 7), (3, 20), (12, 24), (0, 24)):
        part = m(x[a:b].contiguous())
        m.check(x[a:b], part)
        assert torch.equal(m(x[a:b].contiguous()), part)
        p, w = part.cpu().double().numpy(), whole[a:b].cpu().double().numpy()
        assert (np.abs(p - w) <= 2.0 ** -7 * np.maximum(np.abs(p), np.abs(w)) + 2 * tol[a:b]).all()


@pytest.mark.gpu
def test_large_layer_of_single_tokens_and_parts_of_a_batch():
    """The same with a batch that takes rows in pieces and tokens that do not."""
    m = Large(32, 4, 2880, 2880, 8)
    x = _x(32, 2880, 9) * torch.logspace(-6, 1, 32, base=10.0).to(DEV)[:, None].to(torch.bfloat16)
    whole = m(x)
    m.check(x, whole)
    for a, b in ((0, 1), (9, 10), (31, 32), (4, 6), (10, 13), (7, 27)):
        m.check(x[a:b], m(x[a:b].contiguous()))
        m.check(x[a:b], whole[a:b])


class Wide:
    """An NF4 layer of many experts; its 64-bit values are computed on the GPU."""

    def __init__(self, E, k, H, I, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.E, self.k, self.H, self.I = E, k, H, I
        codes = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8, device=DEV)
        absmax = lambda std, *s: std * (2 + torch.rand(s, generator=g, device=DEV))
        self.gu, self.gs = codes(E, 2 * I, H // 2), absmax(H ** -0.5, E, 2 * I, H // 64)
        self.dn, self.ds = codes(E, H, I // 2), absmax(I ** -0.5, E, H, I // 64)
        self.rw = (torch.randn((E, H), generator=g, device=DEV) * 1.5 / H ** 0.5).to(torch.bfloat16)

    def __call__(self, x):
        return gbw.gnf4_moe_layer(x, self.rw, self.gu, self.gs, self.dn, self.ds, k=self.k)

    def weight(self, codes, absmax, e):
        q = torch.stack([codes[e] >> 4, codes[e] & 15], -1).flatten(1).long()
        return torch.from_numpy(mp.NF4).to(DEV)[q] * absmax[e].double().repeat_interleave(64, 1)

    def check(self, x, got):
        xd = x.double()
        l, mag = xd @ self.rw.double().T, xd.abs() @ self.rw.double().abs().T
        ids, w = mp.route(l.cpu().numpy(), self.k, True)
        dl = 2.0 ** -24 * (self.H / 256 * 8 + 16) * mag.max(1).values.cpu().numpy()
        s = -np.sort(-l.cpu().numpy(), 1)
        assert (s[:, self.k - 1] - s[:, self.k] > 2 * dl).all(), "a choice next to a tie"
        ref, tol, var = torch.zeros_like(xd), torch.zeros_like(xd), torch.zeros_like(xd)
        # variance of a weight's error over absmax^2: the levels are off by 7.5e-4 of
        # their root mean square, by 9e-6 of it in the mean
        v0 = (7.5e-4 ** 2) * float((mp.NF4 ** 2).mean())
        sq = lambda v: (v ** 2).reshape(len(v), -1, 64).sum(-1)  # over a block's columns
        # as in Layer.plain: the levels' error, sums of H and I products, h kept to 2^-16
        e1, e2 = (_levels_error() + 2.0 ** -22 + (n + 8) * 2.0 ** -24 for n in (self.H, self.I))
        for e in np.unique(ids):
            t, j = np.nonzero(ids == e)
            we = torch.from_numpy(w[t, j]).to(DEV)[:, None]
            t = torch.from_numpy(t).to(DEV)
            gw, dw = self.weight(self.gu, self.gs, e), self.weight(self.dn, self.ds, e)
            (g, u), (dg, du) = (v.split(self.I, 1) for v in (xd[t] @ gw.T, e1 * (xd[t].abs() @ gw.abs().T)))
            silu = torch.nn.functional.silu(g)
            h = silu * u
            dh = 1.1 * dg * (u.abs() + du) + silu.abs() * du + 2.0 ** -16 * h.abs()
            y, dy = h @ dw.T, (dh + e2 * h.abs()) @ dw.abs().T
            # the codes are random, so the errors of gate, up and down are independent
            vg, vu = (v0 * (sq(xd[t]) @ (self.gs[e].double() ** 2).T)).split(self.I, 1)
            s = torch.sigmoid(g)
            vh = (s * (1 + g * (1 - s))) ** 2 * vg * u ** 2 + silu ** 2 * vu
            vy = v0 * (sq(h) @ (self.ds[e].double() ** 2).T) + vh @ (dw ** 2).T
            var.index_add_(0, t, we ** 2 * vy)
            rel = torch.from_numpy(4 * dl + (17 + self.k) * 2.0 ** -24).to(DEV)[t][:, None]
            ref.index_add_(0, t, we * y)
            tol.index_add_(0, t, we * (dy + rel * y.abs()))
        got, ref, tol = (v.cpu().double().numpy() for v in (got, ref, tol))
        mp.bf16_close(got, ref, tol)
        # and one rounding of the output, 2^-8 / sqrt(3) at most; a tenth for the spread
        err = np.linalg.norm(got - ref) / np.linalg.norm(ref)
        levels = float(var.sum()) / np.linalg.norm(ref) ** 2
        assert err < 1.1 * (levels + 2.0 ** -16 / 3) ** 0.5, (err, levels)
        assert gbw.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 2, 8, 32])
def test_nf4_layer_at_a_decode_shape(T):
    """128 experts of which 8 are chosen, 2048 x 768, from one token to the most."""
    m = Wide(128, 8, 2048, 768, T)
    x = _x(T, 2048, T + 1)
    got = m(x)
    m.check(x, got)
    assert torch.equal(m(x), got)


@pytest.mark.gpu
@pytest.mark.parametrize("mean", [0.25, 1.0, -3.0])
def test_nf4_layer_of_tokens_with_a_mean(mean):
    """The levels' errors have hardly a mean that a mean of x could gather: the
    error stays that of their spread."""
    m = Wide(16, 4, 2048, 768, 5)
    m.rw -= m.rw.float().mean(1, keepdim=True).to(torch.bfloat16)
    x = (_x(8, 2048, 3).float() + mean).to(torch.bfloat16)
    m.check(x, m(x))


# ---------------------------------------------------------------- refusals


def test_layer_refusals():
    z = lambda *s, d=torch.uint8: torch.zeros(s, dtype=d)
    bf = torch.bfloat16
    good = dict(x=z(2, 128, d=bf), router_w=z(4, 128, d=bf), gu_packed=z(4, 128, 64),
                gu_absmax=z(4, 128, 2, d=torch.float32), dn_packed=z(4, 128, 32),
                dn_absmax=z(4, 128, 1, d=torch.float32), k=2)
    for change, text in (
            (dict(x=z(33, 128, d=bf)), "at most 32 tokens"), (dict(k=0), "k=0"), (dict(k=5), "k=5"),
            (dict(router_w=z(4, 64, d=bf)), "router_w"), (dict(gu_packed=z(4, 127, 64)), "gate_up"),
            (dict(gu_absmax=z(4, 128, 1, d=torch.float32)), "gate_up scales"),
            (dict(dn_packed=z(4, 64, 32)), "down"), (dict(dn_packed=z(4, 128, 16)), "down weights"),
            (dict(dn_absmax=z(4, 128, 2, d=torch.float32)), "down scales"),
            (dict(router_bias=z(3, d=torch.float32)), "router_bias"),
            (dict(out=z(2, 64, d=bf)), "out must"), (dict(workspace=z(100)), "workspace"),
            (dict(gu_packed=z(4, 64, 64)), "multiples of 64"), (dict(), "CUDA tensor")):
        with pytest.raises(ValueError, match=text):
            gbw.gnf4_moe_layer(**{**good, **change})
    with pytest.raises(TypeError, match="x must"):
        gbw.gnf4_moe_layer(**{**good, "x": z(2, 128, d=torch.float16)})
    with pytest.raises(ValueError, match="contiguous"):
        gbw.gnf4_moe_layer(**{**good, "x": z(128, 2, d=bf).t()})


def test_layer_host_validation():
    L, p, NULL, SHAPE, ALIGN = gbw.lib, C.c_void_p(256), 1, 2, 3
    assert gbw.lib.gmoe_layer_workspace(33, 8, 2, 64, 64) == 0
    need = L.gmoe_layer_workspace(4, 8, 2, 128, 64)
    assert need > 4 * 8 * 4 + 2 * 8 * 64 * 2 + 8 * 128 * 4

    for fn in (L.gnf4_moe_layer, L.gmxfp4_moe_layer):
        def call(x=p, T=4, H=128, rw=p, rb=None, gu=p, gs=p, dn=p, ds=p, E=8, I=64, k=2, out=p,
                 ws=p, n=need):
            return fn(x, T, H, rw, rb, gu, gs, dn, ds, E, I, k, 1, out, ws, n, None)
        assert call(T=33) == SHAPE and call(T=-1) == SHAPE and call(H=96) == SHAPE
        assert call(I=32) == SHAPE and call(E=1025) == SHAPE and call(k=9) == SHAPE
        assert call(E=64, k=17) == SHAPE and call(n=need - 1) == SHAPE and call(k=0) == SHAPE
        assert call(x=None) == NULL and call(rw=None) == NULL and call(ws=None) == NULL
        assert call(ds=None) == NULL and call(out=None) == NULL
        assert call(x=C.c_void_p(8)) == ALIGN and call(ws=C.c_void_p(16)) == ALIGN
        assert call(rb=C.c_void_p(2)) == ALIGN and call(gs=C.c_void_p(257)) == ALIGN
        assert call(out=C.c_void_p(24)) == ALIGN

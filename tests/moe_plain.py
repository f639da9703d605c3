"""Plain 64-bit implementations (numpy) of the mixture-of-experts operators
around the grouped matmuls, for their tests: routing and its gradient, the
combine and its gradient, MXFP4 rounding, the whole layer."""
import numpy as np

NF4 = np.array([-1.0, -0.6961928009986877, -0.5250730514526367, -0.39491748809814453,
                -0.28444138169288635, -0.18477343022823334, -0.09105003625154495, 0.0,
                0.07958029955625534, 0.16093020141124725, 0.24611230194568634,
                0.33791524171829224, 0.44070982933044434, 0.5626170039176941,
                0.7229568362236023, 1.0])
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)


def route(logits, k, renorm):
    """(ids, weights) of logits [T, E]; NaN counts as -inf, ties go to the
    lowest index, infinite maxima share, a row without any logit has w = 0."""
    v = np.where(np.isnan(logits), -np.inf, np.asarray(logits, np.float64))
    ids = np.argsort(-v, axis=1, kind="stable")[:, :k]
    m = v.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        p = np.where(v == m, 1.0, np.exp(v - m))
    p[np.isneginf(m[:, 0])] = 0.0
    top = np.take_along_axis(p, ids, 1)
    total = (top if renorm else p).sum(1, keepdims=True)
    return ids, np.divide(top, total, out=np.zeros_like(top), where=total > 0)


def route_bwd(logits, ids, w, dw, renorm):
    v = np.where(np.isnan(logits), -np.inf, np.asarray(logits, np.float64))
    t = np.where(w == 0, 0.0, w * np.where(w == 0, 0.0, dw)).sum(1, keepdims=True)
    d = np.zeros_like(v)
    if not renorm:
        _, q = route(logits, v.shape[1], False)
        order, _ = route(logits, v.shape[1], False)
        full = np.zeros_like(v)
        np.put_along_axis(full, order, q, 1)
        d -= full * t
        add = np.where(w == 0, 0.0, w * dw)
    else:
        add = np.where(w == 0, 0.0, w * (dw - t))
    for s in range(ids.shape[1]):
        d[np.arange(len(v)), ids[:, s]] += add[:, s]
    return d


def plan(ids, E):
    """(expert_offsets, row_to_token, row_of_slot, slot_of_row)."""
    flat = ids.reshape(-1)
    slot = np.argsort(flat, kind="stable")
    off = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))])
    row = np.empty_like(slot)
    row[slot] = np.arange(len(slot))
    return off, slot // max(ids.shape[1], 1), row.reshape(ids.shape), slot


def combine(y, row_of_slot, w):
    return np.einsum("tk,tkh->th", w, y[row_of_slot])


def mxfp4(v):
    """(codes 0..15, scale bytes, values) of v [..., K] in MXFP4: scale
    2^(floor(log2 max) - 2), elements to the nearest, halfway to the even code,
    saturating; an all-zero block has scale byte 0; a block that holds a value
    that is not finite has scale byte 255 (NaN) and codes 0."""
    b = np.asarray(v, np.float64)
    b = b.reshape(*b.shape[:-1], -1, 32)
    bad = ~np.isfinite(b).all(-1, keepdims=True)
    b = np.where(bad, 0.0, b)
    m = np.abs(b).max(-1, keepdims=True)
    x = np.where(m > 0, np.frexp(m)[1] - 3, -127).clip(-127, 127)
    t = np.abs(b) * 2.0 ** -x.astype(np.float64)
    hi = np.searchsorted(E2M1, t).clip(1, 7)
    lo_d, hi_d = t - E2M1[hi - 1], E2M1[hi] - t
    q = np.where((lo_d > hi_d) | ((lo_d == hi_d) & (hi % 2 == 0)), hi, hi - 1)
    val = E2M1[q] * 2.0 ** x.astype(np.float64) * np.where(b < 0, -1.0, 1.0)
    codes = np.where(m > 0, q + 8 * np.signbit(b), 0)
    scale = np.where(bad, 255, x + 127)[..., 0]
    val = np.where(bad, np.nan, val)
    flat = lambda a: a.reshape(*a.shape[:-2], -1)
    return flat(codes), scale, flat(val)


def silu(v):
    with np.errstate(over="ignore"):
        return v / (1.0 + np.exp(-v))


def bf16_close(got, ref, extra=0.0):
    """|got - ref| within half a step of bf16 (2^-8 of the value's power of
    two covers it: 2^-8 relative) plus `extra` absolute."""
    d = np.abs(got.astype(np.float64) - ref)
    ok = d <= 2.0 ** -8 * np.abs(ref) + extra + 1e-38
    assert ok.all(), f"worst excess at {np.argmax(~ok)}: {d[~ok][:4]} of {ref[~ok][:4]}"

"""Plain float64 forms of the 8-bit cache, the rotary cache write and attention over the 8-bit cache,
for the tests: NumPy, from the definitions in include/pagedkv.h, sharing no code with the kernels."""
import numpy as np

F32, F64 = np.float32, np.float64
MIN_AMAX = F32(2.0 ** -24)
HALF = 2.0 ** -11             # half a step of binary16, relative


def quantise(x):
    """Codes (uint8) and scales (float32) of rows x [..., 128], in float32 as the definition says."""
    x = np.asarray(x, F32)
    finite = np.isfinite(x)
    amax = np.where(finite, np.abs(x), F32(0)).max(-1)
    scale = (np.maximum(amax, MIN_AMAX) / F32(127)).astype(F32)
    with np.errstate(invalid="ignore"):
        c = np.rint(x / scale[..., None])
    c = np.where(np.isnan(c), 0, np.clip(c, -127, 127))
    return (c + 128).astype(np.uint8), scale


def scatter_int8(k, v, slots, NB, codes_k, codes_v, scales):
    """Writes rows into host copies of an 8-bit cache (in place)."""
    for which, (x, cache) in enumerate(((k, codes_k), (v, codes_v))):
        c, s = quantise(x)
        for i, slot in enumerate(slots):
            if 0 <= slot < NB * 16:
                cache[slot // 16, slot % 16] = c[i]
                scales[slot // 16, :, which, slot % 16] = s[i]


def axis_of(half, sections, cyclic):
    if cyclic:
        A = len(sections)
        return [j % A if j % A > 0 and j < A * sections[j % A] else 0 for j in range(half)]
    return [a for a, n in enumerate(sections) for _ in range(n)]


def rotate(x, positions, inv_freq, sections, pairs, cyclic):
    """Rotary positions of x [T, H, 128] in float64 (angles in long double)."""
    x = np.asarray(x, F64).copy()
    half = len(inv_freq)
    pos = np.atleast_2d(positions)[axis_of(half, sections, cyclic)]            # [half, T]
    a = (pos.astype(np.longdouble) * np.asarray(inv_freq, F32).astype(np.longdouble)[:, None]).T
    a = np.fmod(a, 2 * np.longdouble("3.14159265358979323846264338327950288"))
    cos, sin = np.cos(a).astype(F64)[:, None, :], np.sin(a).astype(F64)[:, None, :]
    i0, i1 = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if pairs else (slice(0, half), slice(half, 2 * half))
    u, w = x[..., i0].copy(), x[..., i1].copy()
    x[..., i0], x[..., i1] = u * cos - w * sin, w * cos + u * sin
    return x


def partner_magnitude(x, half, pairs):
    """|x| + |its pair's other channel| per channel: the scale of a rotation's fp32 errors."""
    m = np.abs(np.asarray(x, F64))
    out = m.copy()
    i0, i1 = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if pairs else (slice(0, half), slice(half, 2 * half))
    s = m[..., i0] + m[..., i1]
    out[..., i0], out[..., i1] = s, s
    return out


def attention(q, codes_k, codes_v, scales, tables, lens, query_start, softmax_scale):
    """(out, bound) in float64 of every query row: the causal attention of the definition, and a bound
    on what a kernel may be off, from its roundings:
      * weights rounded to f16 (half a step), the f16 output (half a step), and, in the matrix-product
        form, values rounded to f16 (half a step): 3 half steps of sum p |v|, one of |out|;
      * logits: fp32 sums of 128 exact terms, fp32 exp2/log2 (2^-21) and the fp32 roundings of the
        logit itself (its scale, the product, the difference to the maximum): a weight is off by
        exp(d), its normalised value by at most exp(2 d);
      * weights below the normal f16 range are off by 2^-25 of the largest;
      * values below it are staged off by half a subnormal step, 2^-25: that much of sum p = 1. (A small
        row's value is rounded at a normal magnitude first, half a step, which is the 2^-11 counted
        above, and then to the subnormal one: the two add.)"""
    B = len(lens)
    Hq, G = q.shape[1], q.shape[1] // codes_k.shape[2]
    out, bound = np.zeros(q.shape, F64), np.zeros(q.shape, F64)
    for b in range(B):
        r0, r1 = int(query_start[b]), int(query_start[b + 1])
        L, n = int(lens[b]), r1 - r0
        if L == 0 or n == 0:
            continue
        blocks = tables[b, :-(-L // 16)]
        kv = []
        for which, codes in enumerate((codes_k, codes_v)):
            c = codes[blocks].astype(F64) - 128                                 # [pages, 16, Hkv, 128]
            s = scales[blocks][:, :, which].astype(F64).transpose(0, 2, 1)[..., None]
            kv.append(((c * s).reshape(-1, *c.shape[2:])[:L], np.abs(c).reshape(-1, *c.shape[2:])[:L],
                       s.reshape(-1, c.shape[2])[:L]))
        (K, _, _), (V, cv, vs) = kv
        for h in range(Hq):
            g = h // G
            qq = q[r0:r1, h].astype(F64)
            x = qq @ K[:, g].T * softmax_scale
            mag = np.abs(qq) @ np.abs(K[:, g]).T * abs(softmax_scale)
            hidden = np.arange(L)[None, :] > (L - n + np.arange(n))[:, None]
            x = np.where(hidden, -np.inf, x)
            mx = x.max(-1, keepdims=True)
            p = np.exp(x - mx)
            p /= p.sum(-1, keepdims=True)
            out[r0:r1, h] = p @ V[:, g]
            absum = p @ np.abs(V[:, g])
            d = np.where(hidden, 0, mag * (130 * 2.0 ** -24)).max(-1) + 2.0 ** -20 \
                + np.where(hidden, 0, np.abs(x) + 64).max(-1) * 2.0 ** -22
            small = 2.0 ** -25 * (np.where(hidden, 0, 1.0) @ cv[:, g]) * vs[:, g].max()
            bound[r0:r1, h] = (3.1 * HALF + np.expm1(2 * d))[:, None] * absum + HALF * np.abs(out[r0:r1, h]) \
                + small + 2 * 2.0 ** -25
    return out, bound


def assert_within(got, ref, bound, what=""):
    got = np.asarray(got, F64)
    assert got.shape == ref.shape
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    over = np.abs(got - ref) / np.maximum(bound, 2.0 ** -40)         # (an empty row must be zero)
    assert (over <= 1).all(), f"{what}: {over.max():.3f} of the bound at {np.unravel_index(over.argmax(), over.shape)}"

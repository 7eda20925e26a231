"""Scales of the 8-bit cache over the whole range that its attention accepts: what the cache holds decides,
not which kernel the chunk's length leads to."""
import numpy as np
import pytest
import torch

import paged_kv_decode_gqa_b200 as pkv
from _gpu_helpers import dev, host
from _int8_reference import HALF
from test_gpu_int8_attention import SCALE, Case, workspace

F16, F32, F64 = np.float16, np.float32, np.float64
D = 128
NEWS = {"decode": [1, 1, 1], "streaming": [1, 1, 1], "narrow": [3, 5, 2], "wide": [90, 17, 300]}


def bound_of(c, scale=SCALE):
    """(out, bound) in float64. What a kernel may be off by, from its roundings:
      * weights rounded to f16 (half a step, HALF) and, in the matrix-product form, values (half a step):
        2 HALF of sum p |v|; the output's own: HALF of it, or half the smallest subnormal, 2^-25;
      * the logit's and the exponential's errors (d, as tests/_int8_reference.py derives it): a normalised
        weight is off by at most exp(2 d);
      * below the normal f16 range, 2^-25 of the row's largest weight. A weight holds its token's V scale (the
        streaming form), or a power of two above 2^-8 and at most 2^-7 of the largest V scale of 64 tokens (the
        matrix-product form, whose staged values are then below 2^8 |code|): a code is off by that much of the
        row's largest p times such a scale, and by a factor of two at most for the power of two;
      * a staged value below it: 2^-25 of that power of two, 2^-32 of the largest V scale of its 64 tokens."""
    out, bound = np.zeros(c.q.shape, F64), np.zeros(c.q.shape, F64)
    G = c.Hq // c.Hkv
    for b in range(c.B):
        r0, r1, L = int(c.qs[b]), int(c.qs[b + 1]), int(c.lens[b])
        n = r1 - r0
        if L == 0 or n == 0:
            continue
        blk, row = c.rows_of(b)
        hidden = np.arange(L)[None, :] > (L - n + np.arange(n))[:, None]
        for h in range(c.Hq):
            g = h // G
            K, V = ((c.codes[w, blk, row, g].astype(F64) - 128) for w in (0, 1))
            ks, vs = (c.scales[blk, g, w, row].astype(F64) for w in (0, 1))
            qq = c.q[r0:r1, h].astype(F64)
            x = np.where(hidden, -np.inf, qq @ (K * ks[:, None]).T * scale)
            mag = np.abs(qq) @ np.abs(K * ks[:, None]).T * abs(scale)
            p = np.exp(x - x.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            w = p * vs
            out[r0:r1, h] = w @ V
            absum = w @ np.abs(V)
            top = np.repeat(np.pad(vs, (0, -L % 64)).reshape(-1, 64).max(-1), 64)[:L]
            d = np.where(hidden, 0, mag * (130 * 2.0 ** -24)).max(-1) + 2.0 ** -20 \
                + np.where(hidden, 0, np.abs(x) + 64).max(-1) * 2.0 ** -22
            small = 2.0 ** -24 * (p * top).max(-1)[:, None] * (np.where(hidden, 0, 1.0) @ np.abs(V))
            small += 2.0 ** -32 * (p * top).sum(-1)[:, None]
            bound[r0:r1, h] = (2.1 * HALF + np.expm1(2 * d))[:, None] * absum + 1.05 * HALF * np.abs(out[r0:r1, h]) \
                + 1.05 * small + 2.0 ** -25
    return out, bound


def large_scales(form, kind):
    """V scales past 511.75, where a code of 127 times its scale is near or past the largest f16."""
    c = Case(500 + len(kind), 14, 2, [100, 17, 640], NEWS[form])
    live = np.isfinite(c.scales[:, :, 1])
    if kind == "largest rows":                                     # as the write stores rows that reach 65504
        c.scales[:, :, 1][live] = F32(65504) / F32(127)
    elif kind in ("scale 1000", "scale 5000"):                     # every value inside the f16 range
        s = int(kind.split()[1])
        c.scales[:, :, 1][live] = s
        most = 65504 // s
        c.codes[1] = np.clip(c.codes[1].astype(np.int32) - 128, -most, most) + 128
    else:                                                          # values past it, at logits far below the rest
        rng = np.random.default_rng(9)
        c.q[..., 0] = 8
        for b in range(c.B):
            blk, row = c.rows_of(b)
            far = np.arange(len(blk)) // 64 % 3 == 1
            c.codes[0, blk[far], row[far]] = 128
            c.codes[0, blk[far], row[far], :, 0] = 1
            c.scales[blk[far], :, 0, row[far]] = F32(0.15)
            c.scales[blk[far], :, 1, row[far]] = np.exp2(rng.uniform(10, 20, (int(far.sum()), c.Hkv))).astype(F32)
    return c


def spread_scales(form, seed):
    """V scales over 2^20 in one row of tokens, zeros among them."""
    c = Case(520 + seed, 14, 2, [100, 17, 640], NEWS[form])
    rng = np.random.default_rng(seed)
    live = np.isfinite(c.scales[:, :, 1])
    s = np.exp2(rng.uniform(-20, 0, live.shape)).astype(F32)
    s[rng.random(live.shape) < 0.1] = 0
    c.scales[:, :, 1][live] = s[live]
    return c


def run(c, form):
    return c.decode() if form == "decode" else c.chunk()


def check(c, got):
    ref, bound = bound_of(c)
    assert (np.abs(ref) < 65520).all()                             # (rounds to at most 65504) the case has an answer in f16
    assert np.isfinite(got).all()
    over = np.abs(got.astype(F64) - ref) / bound
    assert (over <= 1).all(), f"{over.max():.3f} of the bound"
    assert pkv.pkv_device_error() == 0


KINDS = ["largest rows", "scale 1000", "scale 5000", "far above the range"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("form", ["narrow", "wide"])
def test_the_cases_tell_a_clamped_scale_from_a_right_one(form, kind):
    """On the CPU: with every scale cut at 511.75 the answer leaves the bound in many places."""
    c = large_scales(form, kind)
    ref, bound = bound_of(c)
    c.scales[:, :, 1] = np.minimum(c.scales[:, :, 1], F32(511.75))
    assert (np.abs(ref) < 65520).all()
    assert (np.abs(bound_of(c)[0] - ref) > bound).mean() > 0.2


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("form", list(NEWS))
def test_large_value_scales(form, kind):
    pkv.pkv_device_error()
    c = large_scales(form, kind)
    check(c, run(c, form))


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("form", list(NEWS))
def test_value_scales_over_2_to_the_20(form, seed):
    pkv.pkv_device_error()
    c = spread_scales(form, seed)
    check(c, run(c, form))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 4, 40])
def test_written_rows_of_the_largest_f16(n):
    """Through the write: a sequence whose only value row has one channel at 65504. Its output is that row of
    the cache, to half a step."""
    pkv.pkv_device_error()
    rng = np.random.default_rng(n)
    L, Hq, Hkv = n, 12, 2
    k = rng.standard_normal((L, Hkv, D)).astype(F16)
    v = np.tile((rng.standard_normal((1, Hkv, D)) * 9000).clip(-60000, 60000).astype(F16), (L, 1, 1))
    v[..., 3] = 65504
    NB = L // 16 + 2
    slots = np.arange(L, dtype=np.int64) + 16
    kc, vc = (torch.full((NB, 16, Hkv, D), 128, dtype=torch.uint8, device="cuda") for _ in range(2))
    sc = torch.full((NB, Hkv, 2, 16), float("nan"), device="cuda")
    pkv.paged_kv_cache_write_int8(dev(k), dev(v), kc, vc, sc, dev(slots))
    q = dev(rng.standard_normal((n, Hq, D)).astype(F16))
    out = torch.zeros_like(q)
    pkv.paged_gqa_prefill_attention_int8(out, q, kc, vc, sc, dev(np.arange(1, NB, dtype=np.int32)[None]),
                                         dev(np.array([L], np.int32)), dev(np.array([0, n], np.int32)), max_query_len=n,
                                         max_context_len=L, softmax_scale=SCALE, workspace=workspace())
    s = F64(F32(65504) / F32(127))
    row = (host(vc)[1, 0].astype(F64) - 128) * s                   # [Hkv, D], the same for every token
    want = np.repeat(row, Hq // Hkv, 0)[None]
    # half a step each for the weights, the staged value and the output
    assert (np.abs(host(out).astype(F64) - want) <= 3.1 * HALF * np.abs(want)).all()
    assert pkv.pkv_device_error() == 0

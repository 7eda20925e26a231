"""The 8-bit cache write, the cache read of every type, and rotary positions with the cache write,
against the plain float64 forms. The 8-bit write without rotation is bit-exact."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_decode_gqa_b200 as pkv
from _gpu_helpers import dev, host
from _int8_reference import HALF, partner_magnitude, quantise, rotate, scatter_int8

pytestmark = pytest.mark.gpu
F16, F32, F64 = np.float16, np.float32, np.float64
D = 128


@pytest.fixture(autouse=True)
def _clear_device_error():
    pkv.pkv_device_error()
    yield
    torch.cuda.synchronize()


def _rows(rng, T, H, spread=3.0):
    x = rng.standard_normal((T, H, D)) * np.exp2(rng.uniform(-spread, spread, (T, H, 1)))
    return x.astype(F16)


def _pool(NB, H, kv="int8"):
    if kv == "f16":
        return (np.full((NB, 16, H, D), 3.0, F16), np.full((NB, 16, H, D), -3.0, F16), None)
    return (np.full((NB, 16, H, D), 7, np.uint8), np.full((NB, 16, H, D), 9, np.uint8),
            np.full((NB, H, 2, 16), 0.25, F32) if kv == "int8" else None)


def _write_int8(k, v, pool, slots):
    kc, vc, sc = (dev(a) for a in pool)
    pkv.paged_kv_cache_write_int8(dev(k), dev(v), kc, vc, sc, dev(slots))
    return kc, vc, sc


# ------------------------------------------------------------------ the write
@pytest.mark.parametrize("T,Hkv", [(1, 1), (1, 8), (2, 3), (17, 2), (33, 5), (130, 4), (515, 1), (9, 40)])
def test_write_int8_bit_exact(T, Hkv):
    rng = np.random.default_rng(T * 100 + Hkv)
    k, v = _rows(rng, T, Hkv), _rows(rng, T, Hkv)
    NB = T // 16 + 5
    slots = rng.permutation(NB * 16)[:T].astype(np.int64)
    slots[T // 2] = -1 if T > 1 else slots[0]                  # a padding token
    pool = _pool(NB, Hkv)
    got = _write_int8(k, v, pool, slots)
    ref = [a.copy() for a in pool]
    scatter_int8(k, v, slots, NB, *ref)
    for g, r, name in zip(got, ref, ("k codes", "v codes", "scales")):
        assert np.array_equal(host(g).view(np.uint8), r.view(np.uint8)), name
    assert pkv.pkv_device_error() == 0


def test_write_int8_special_rows():
    """Zeros, the smallest and largest f16, infinities, NaN, and ties."""
    x = np.zeros((8, 1, D), F16)
    x[1] = F16(2.0 ** -24)
    x[2] = 65504
    x[2, 0, ::2] = -65504
    x[3, 0] = np.linspace(-1, 1, D)
    x[3, 0, 5], x[3, 0, 6] = np.inf, -np.inf
    x[4, 0] = np.linspace(-2, 2, D)
    x[4, 0, 7] = np.nan
    x[5] = np.nan
    x[6, 0] = np.arange(D) + 0.5                              # amax 127.5: quotients near ties
    x[7, 0] = np.concatenate([np.arange(64) - 0.5, [127], np.arange(63) - 0.5])   # scale 1: exact ties
    slots = np.arange(8, dtype=np.int64)
    pool = _pool(1, 1)
    got = [host(a) for a in _write_int8(x, x[::-1].copy(), pool, slots)]
    ref = [a.copy() for a in pool]
    scatter_int8(x, x[::-1], slots, 1, *ref)
    for g, r in zip(got, ref):
        assert np.array_equal(g, r)
    assert (got[0][0, 0] == 128).all() and (got[0][0, 5] == 128).all()      # zeros and NaN: code of 0
    assert got[0][0, 3, 0, 5] == 255 and got[0][0, 3, 0, 6] == 1            # infinities clamp
    assert np.isfinite(got[2]).all() and (got[2] > 0).all()


def test_write_int8_skips_and_flags_slots():
    rng = np.random.default_rng(1)
    k, v = _rows(rng, 4, 2), _rows(rng, 4, 2)
    slots = np.array([-1, 3 * 16, 5, 1 << 40], np.int64)       # padding, one past the pool, fine, far outside
    pool = _pool(3, 2)
    got = _write_int8(k, v, pool, slots)
    assert pkv.pkv_device_error() == pkv.DEVERR_SLOT
    ref = [a.copy() for a in pool]
    scatter_int8(k, v, slots, 3, *ref)
    for g, r in zip(got, ref):
        assert np.array_equal(host(g), r)


def test_empty_calls_are_no_ops():
    e = torch.empty((0, 2, D), dtype=torch.float16, device="cuda")
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    kc, vc, sc = (dev(a) for a in _pool(2, 2))
    before = [t.clone() for t in (kc, vc, sc)]
    pkv.paged_kv_cache_write_int8(e, e, kc, vc, sc, slots)
    pkv.paged_kv_cache_read(e, e, kc, vc, slots, kv_dtype="int8", kv_scales=sc)
    pkv.paged_kv_rope_cache_write(e, e, e, e, kc, vc, slots, slots, torch.ones(64, device="cuda"), kv_dtype="int8",
                                  kv_scales=sc)
    assert all(torch.equal(a, b) for a, b in zip((kc, vc, sc), before))


# ------------------------------------------------------------------ reading back
@pytest.mark.parametrize("kv", ["f16", "fp8", "int8"])
@pytest.mark.parametrize("T,Hkv", [(1, 1), (5, 3), (67, 4), (300, 2)])
def test_read_is_the_inverse_of_the_write(kv, T, Hkv):
    rng = np.random.default_rng(T + Hkv)
    NB = 24
    codes = rng.integers(0, 256, (2, NB, 16, Hkv, D)).astype(np.uint8)
    scales = np.exp2(rng.uniform(-31, 9, (NB, Hkv, 2, 16))).astype(F32)
    ks, vs = 0.37, 2.5
    slots = rng.integers(0, NB * 16, T).astype(np.int64)       # with repeats
    slots[0] = -1
    if kv == "f16":
        kc, vc = (rng.standard_normal((NB, 16, Hkv, D)).astype(F16) for _ in range(2))
        vals = [kc.astype(F64), vc.astype(F64)]
    elif kv == "fp8":
        kc, vc = codes
        vals = [oracle.e4m3_to_f64(c).astype(F32) * F32(s) for c, s in ((kc, ks), (vc, vs))]
    else:
        kc, vc = codes
        vals = [(c.astype(F32) - 128) * scales[:, :, w].transpose(0, 2, 1)[..., None] for w, c in enumerate(codes)]
    out = [torch.full((T, Hkv, D), 5.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    more = {"kv_scales": dev(scales)} if kv == "int8" else {"k_scale": ks, "v_scale": vs}
    pkv.paged_kv_cache_read(*out, dev(kc), dev(vc), dev(slots), kv_dtype=kv, **more)
    for o, x in zip(out, vals):
        with np.errstate(over="ignore"):
            ref = x.reshape(-1, Hkv, D)[slots].astype(F16)
        ref[0] = 5.0                                            # the skipped row is left as it was
        assert np.array_equal(host(o).view(np.uint16), ref.view(np.uint16)) or \
            np.array_equal(host(o)[~np.isnan(ref)], ref[~np.isnan(ref)])
        assert np.array_equal(np.isnan(host(o)), np.isnan(ref))
    assert pkv.pkv_device_error() == 0


def test_read_flags_slots_outside_the_pool():
    kc, vc, sc = (dev(a) for a in _pool(2, 2))
    out = [torch.full((3, 2, D), 5.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    pkv.paged_kv_cache_read(*out, kc, vc, dev(np.array([32, 0, -7], np.int64)), kv_dtype="int8", kv_scales=sc)
    assert pkv.pkv_device_error() == pkv.DEVERR_SLOT
    assert (out[0][[0, 2]] == 5).all() and (out[0][1] == (7 - 128) * 0.25).all()


def test_blocks_past_32_bit_offsets():
    """A pool whose last blocks lie more than 2^31 bytes in: written, read back and attended to."""
    NB, Hkv, T = 300_000, 4, 40
    rng = np.random.default_rng(3)
    k, v = _rows(rng, T, Hkv), _rows(rng, T, Hkv)
    kc, vc = (torch.empty((NB, 16, Hkv, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    sc = torch.empty((NB, Hkv, 2, 16), dtype=torch.float32, device="cuda")
    blocks = np.array([NB - 1, 3, NB - 2], np.int32)
    slots = np.array([int(blocks[t // 16]) * 16 + t % 16 for t in range(T)], np.int64)
    pkv.paged_kv_cache_write_int8(dev(k), dev(v), kc, vc, sc, dev(slots))
    out = [torch.empty((T, Hkv, D), dtype=torch.float16, device="cuda") for _ in range(2)]
    pkv.paged_kv_cache_read(*out, kc, vc, dev(slots), kv_dtype="int8", kv_scales=sc)
    for o, x in zip(out, (k, v)):
        c, s = quantise(x)
        assert np.array_equal(host(o), ((c.astype(F32) - 128) * s[..., None]).astype(F16))
    assert pkv.pkv_device_error() == 0


# ------------------------------------------------------------------ rotary positions and the write
def _freq(R, base=1e4):
    return (base ** (-np.arange(R // 2, dtype=F64) * 2 / R)).astype(F32)


ROPE = [  # T, Hq, Hkv, rotary, sections, pairs, cyclic
    (1, 4, 1, 128, [64], False, False),
    (3, 28, 4, 128, [64], True, False),
    (65, 12, 2, 128, [16, 24, 24], False, False),
    (65, 12, 2, 128, [22, 21, 21], False, True),
    (17, 5, 1, 96, [12, 18, 18], True, False),
    (9, 8, 8, 64, [17, 15], False, True),
    (130, 7, 7, 16, [8], False, False),
    (6, 32, 8, 32, [4, 4, 4, 4], True, True),
    (5, 0, 3, 112, [56], False, False),
    (4, 80, 10, 128, [64, 0], False, False),
]


def _rope_case(case, seed):
    T, Hq, Hkv, R, sections, pairs, cyclic = case
    rng = np.random.default_rng(seed)
    q, k, v = _rows(rng, T, Hq), _rows(rng, T, Hkv), _rows(rng, T, Hkv)
    pos = rng.integers(0, 1 << 20, (len(sections), T)).astype(np.int64)
    pos[:, 0] = [0, 1, 2, 3][:len(sections)]
    if T > 2:
        pos[:, 1], pos[:, 2] = (1 << 31) - 7, -12345
    NB = T // 16 + 3
    slots = rng.permutation(NB * 16)[:T].astype(np.int64)
    return q, k, v, pos, slots, NB


def _run_rope(case, q, k, v, pos, slots, pool, kv, q_out=None, **more):
    T, Hq, Hkv, R, sections, pairs, cyclic = case
    kc, vc, sc = (None if a is None else dev(a) for a in pool)
    qd = dev(q)
    q_out = torch.full_like(qd, float("nan")) if q_out is None else qd
    p = dev(pos[0]) if len(sections) == 1 else dev(pos)
    pkv.paged_kv_rope_cache_write(q_out, qd, dev(k), dev(v), kc, vc, dev(slots), p, dev(_freq(R)),
                                  sections=sections, interleaved=pairs, cyclic_axes=cyclic, kv_dtype=kv,
                                  kv_scales=sc, **more)
    return host(q_out), host(kc), host(vc), None if sc is None else host(sc)


def _rotated(x, case, pos):
    T, Hq, Hkv, R, sections, pairs, cyclic = case
    exact = rotate(x, pos, _freq(R), sections, pairs, cyclic)
    # fp32: the sine and cosine (2 ulp and the reduced angle's rounding, 2^-25 of a turn each: 2^-21 in
    # all) and three roundings of the products and their sum
    return exact, 2.0 ** -20 * partner_magnitude(x, R // 2, pairs)


@pytest.mark.parametrize("kv", ["f16", "fp8", "int8"])
@pytest.mark.parametrize("i", range(len(ROPE)))
def test_rope_cache_write(i, kv):
    case = ROPE[i]
    T, Hq, Hkv, R, *_ = case
    q, k, v, pos, slots, NB = _rope_case(case, i)
    if T > 3:
        slots[3] = -1
    scales = {"k_scale": float(np.abs(k).max()) / 300, "v_scale": float(np.abs(v).max()) / 448} if kv == "fp8" else {}
    pool = _pool(NB, Hkv, kv)
    got_q, kc, vc, sc = _run_rope(case, q, k, v, pos, slots, pool, kv, **scales)
    exact, err = _rotated(q, case, pos)
    assert (np.abs(got_q.astype(F64) - exact) <= HALF * np.abs(exact) + err + 2.0 ** -25).all()
    assert np.array_equal(got_q[..., R:], q[..., R:])
    exact, err = _rotated(k, case, pos)
    kept = slots >= 0
    rows, ref_rows = slots[kept], slots
    got_k, got_v = (c.reshape(-1, Hkv, D)[rows] for c in (kc, vc))
    exact, err, k, v = exact[kept], err[kept], k[kept], v[kept]
    if kv == "f16":
        assert (np.abs(got_k.astype(F64) - exact) <= HALF * np.abs(exact) + err + 2.0 ** -25).all()
        assert np.array_equal(got_v, v) and np.array_equal(got_k[..., R:], k[..., R:])
    elif kv == "fp8":
        ks, vs = F32(scales["k_scale"]), F32(scales["v_scale"])
        val = oracle.e4m3_to_f64(got_k).reshape(got_k.shape) * F64(ks)
        room = 2.0 ** -4 * np.abs(exact) + (2.0 ** -10 + 448 * 2.0 ** -23) * F64(ks) + 2 * err
        inside = np.abs(exact) <= 448 * F64(ks)
        assert (np.abs(val - exact) <= room)[inside].all()
        assert (np.abs(val[~inside]) == 448 * F64(ks)).all()
        assert np.array_equal(got_v, oracle.quantize_e4m3(v, float(vs)))
        assert np.array_equal(got_k[..., R:], oracle.quantize_e4m3(k, float(ks))[..., R:])
    else:
        blk, row = rows // 16, rows % 16
        ks = sc[blk, :, 0, row].astype(F64)
        amax = np.maximum(np.abs(exact).max(-1), 2.0 ** -24)
        worst = err.max(-1)
        assert (np.abs(ks * 127 - amax) <= worst + 2.0 ** -22 * amax).all()
        val = (got_k.astype(F64) - 128) * ks[..., None]
        assert (np.abs(val - exact) <= (0.5 + 127 * 2.0 ** -22) * ks[..., None] + err + worst[..., None]).all()
        c, s = quantise(v)
        assert np.array_equal(got_v, c) and np.array_equal(sc[blk, :, 1, row], s)
    # nothing else changed
    rest = np.setdiff1d(np.arange(NB * 16), rows)
    for a, b in ((kc, pool[0]), (vc, pool[1])):
        assert np.array_equal(a.reshape(-1, Hkv, D)[rest], b.reshape(-1, Hkv, D)[rest])
    if sc is not None:
        assert (sc.transpose(0, 3, 1, 2).reshape(-1, Hkv, 2)[rest] == 0.25).all()
    assert pkv.pkv_device_error() == 0


@pytest.mark.parametrize("kv", ["f16", "int8"])
def test_rope_in_place_is_the_same(kv):
    case = ROPE[2]
    q, k, v, pos, slots, NB = _rope_case(case, 50)
    a = _run_rope(case, q, k, v, pos, slots, _pool(NB, 2, kv), kv)
    b = _run_rope(case, q, k, v, pos, slots, _pool(NB, 2, kv), kv, q_out="q")
    assert all(x is None or np.array_equal(x, y) for x, y in zip(a, b))


def test_rope_at_position_zero_is_the_write():
    """Position 0 on every axis: the 8-bit cache gets what paged_kv_cache_write_int8 writes, bit for bit."""
    case = ROPE[3]
    q, k, v, pos, slots, NB = _rope_case(case, 51)
    got_q, *got = _run_rope(case, q, k, v, np.zeros_like(pos), slots, _pool(NB, 2), "int8")
    ref = [host(t) for t in _write_int8(k, v, _pool(NB, 2), slots)]
    assert np.array_equal(got_q, q)
    assert all(np.array_equal(a, b) for a, b in zip(got, ref))


def test_equal_axes_are_one_axis():
    """A token with the same position on every axis is a token with one position, bit for bit."""
    one, three, round3 = ROPE[1], ROPE[1][:4] + ([20, 22, 22], True, False), ROPE[1][:4] + ([22, 21, 21], True, True)
    q, k, v, pos, slots, NB = _rope_case(one, 52)
    ref = _run_rope(one, q, k, v, pos, slots, _pool(NB, 4), "int8")
    for case in (three, round3):
        got = _run_rope(case, q, k, v, np.repeat(pos, 3, 0), slots, _pool(NB, 4), "int8")
        assert all(np.array_equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("per_head", [False, True])
def test_rope_fp8_with_device_scales(per_head):
    case = ROPE[1]
    T, Hq, Hkv, R, *_ = case
    q, k, v, pos, slots, NB = _rope_case(case, 53)
    ks = np.linspace(0.5, 2.0, Hkv).astype(F32) if per_head else np.array([0.75], F32)
    vs = (ks * F32(1.5)).astype(F32)
    got = _run_rope(case, q, k, v, pos, slots, _pool(NB, Hkv, "fp8"), "fp8", k_scale=dev(ks), v_scale=dev(vs))
    rows = got[2].reshape(-1, Hkv, D)[slots]
    for h in range(Hkv):
        i = h if per_head else 0
        assert np.array_equal(rows[:, h], oracle.quantize_e4m3(np.ascontiguousarray(v[:, h]), float(vs[i])))
        one = _run_rope(case, q, k, v, pos, slots, _pool(NB, Hkv, "fp8"), "fp8", k_scale=float(ks[i]),
                        v_scale=float(vs[i]))
        assert np.array_equal(got[1][:, :, h], one[1][:, :, h])
    assert pkv.pkv_device_error() == 0
    _run_rope(case, q, k, v, pos, slots, _pool(NB, Hkv, "fp8"), "fp8", k_scale=dev(ks * 0), v_scale=dev(vs))
    assert pkv.pkv_device_error() & pkv.DEVERR_SCALE


def test_rope_flags_slots_and_still_rotates_q():
    case = ROPE[0][:1] + (4, 1, 128, [64], False, False)
    q, k, v, pos, slots, NB = _rope_case(case, 54)
    slots[:] = NB * 16
    pool = _pool(NB, 1)
    got_q, kc, vc, sc = _run_rope(case, q, k, v, pos, slots, pool, "int8")
    assert pkv.pkv_device_error() == pkv.DEVERR_SLOT
    assert np.array_equal(kc, pool[0]) and np.array_equal(vc, pool[1]) and np.array_equal(sc, pool[2])
    exact, err = _rotated(q, case, pos)
    assert (np.abs(got_q.astype(F64) - exact) <= HALF * np.abs(exact) + err + 2.0 ** -25).all()


def test_calls_the_bindings_refuse():
    k = torch.zeros((4, 2, D), dtype=torch.float16, device="cuda")
    kc, vc, sc = (dev(a) for a in _pool(2, 2))
    slots = torch.zeros(4, dtype=torch.int64, device="cuda")
    pos, freq = torch.zeros((2, 4), dtype=torch.int64, device="cuda"), torch.ones(64, device="cuda")
    bad = [
        lambda: pkv.paged_kv_cache_write_int8(k[:3], k, kc, vc, sc, slots),
        lambda: pkv.paged_kv_cache_write_int8(k.float(), k, kc, vc, sc, slots),
        lambda: pkv.paged_kv_cache_write_int8(k, k, kc, vc, sc[:, :1], slots),
        lambda: pkv.paged_kv_cache_write_int8(k, k, kc.cpu(), vc, sc, slots),
        lambda: pkv.paged_kv_cache_write_int8(k.transpose(0, 1), k, kc, vc, sc, slots),
        lambda: pkv.paged_kv_cache_read(k, k, kc, vc, slots, kv_dtype="int8"),
        lambda: pkv.paged_kv_cache_read(k, k, kc, vc, slots, kv_dtype="fp8", kv_scales=sc),
        lambda: pkv.paged_kv_cache_read(k, k, kc, vc, slots, kv_dtype="int4"),
        lambda: pkv.paged_kv_rope_cache_write(k, k, k, k, kc, vc, slots, pos, freq, sections=[64], kv_dtype="int8",
                                              kv_scales=sc),
        lambda: pkv.paged_kv_rope_cache_write(k, k, k, k, kc, vc, slots, pos[:, :3], freq, sections=[32, 32],
                                              kv_dtype="int8", kv_scales=sc),
        lambda: pkv.paged_kv_rope_cache_write(k, k, k, k, kc, vc, slots, pos, freq, sections=[32, 31],
                                              kv_dtype="int8", kv_scales=sc),
        lambda: pkv.paged_kv_rope_cache_write(k, k, k, k, kc, vc, slots, pos, freq[:60].contiguous(),
                                              sections=[30, 30], kv_dtype="int8", kv_scales=sc),
    ]
    for call in bad:
        with pytest.raises((ValueError, TypeError, pkv.PagedKVError)):
            call()

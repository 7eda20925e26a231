"""Refusals of the 8-bit cache, rotary cache write and cache read entry points: every call below is
rejected by the host-side checks, before any launch (fake aligned pointers, no GPU needed)."""
import ctypes

import pytest

import paged_kv_decode_gqa_b200 as pkv

A = 1 << 20
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


def _write(**kw):
    a = dict(k=A, v=A, kc=A, vc=A, sc=A, sm=A, T=4, Hkv=2, D=128, NB=8, bs=16) | kw
    return pkv.load_library().paged_kv_cache_write_int8(*a.values(), None)


def _read(**kw):
    a = dict(k=A, v=A, kc=A, vc=A, sc=A, sm=A, T=4, Hkv=2, D=128, NB=8, bs=16, kv=2, ks=1.0, vs=1.0) | kw
    return pkv.load_library().paged_kv_cache_read(*a.values(), None)


def _rope(sections=(64,), **kw):
    B = 1 << 22
    a = dict(qo=2 * B, q=A, k=3 * B, v=4 * B, kc=A, vc=A, sc=A, sm=A, pos=A, freq=A, T=4, Hq=4, Hkv=2, D=128, R=128,
             axes=len(sections), sections=(ctypes.c_int32 * max(1, len(sections)))(*sections), NB=8, bs=16, kv=2,
             ks=1.0, vs=1.0, flags=0) | kw
    return pkv.load_library().paged_kv_rope_cache_write(*a.values(), None)


def _decode(**kw):
    a = dict(out=A, q=A, k=A, v=A, sc=A, bt=A, cl=A, B=2, Hq=12, Hkv=2, D=128, bs=16, mb=4, NB=64, L=64, scale=0.1,
             ws=A, wsb=1 << 30) | kw
    return pkv.load_library().paged_gqa_decode_attention_int8(*a.values(), None)


def _chunk(**kw):
    a = dict(out=A, q=A, k=A, v=A, sc=A, bt=A, cl=A, qs=A, B=2, total=8, maxq=4, Hq=12, Hkv=2, D=128, bs=16, mb=4,
             NB=64, L=64, scale=0.1, ws=A, wsb=1 << 30) | kw
    return pkv.load_library().paged_gqa_prefill_attention_int8(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(kc=None), INVALID), (dict(sc=None), INVALID),
    (dict(sm=None), INVALID), (dict(k=A + 8), INVALID), (dict(vc=A + 4), INVALID), (dict(sc=A + 4), INVALID),
    (dict(sm=A + 4), INVALID), (dict(T=-1), INVALID), (dict(Hkv=0), INVALID), (dict(NB=0), INVALID),
    (dict(bs=0), INVALID), (dict(D=64), UNSUPPORTED), (dict(bs=32), UNSUPPORTED), (dict(Hkv=70000), UNSUPPORTED),
    (dict(T=1 << 30), UNSUPPORTED),
    (dict(T=0), OK), (dict(T=0, k=None, kc=None), OK),
])
def test_write_int8_arguments(kw, status):
    assert _write(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(v=A + 2), INVALID), (dict(sc=None), INVALID), (dict(kv=3), INVALID),
    (dict(kv=-1), INVALID), (dict(kv=1, ks=0.0), INVALID), (dict(kv=1, vs=float("nan")), INVALID),
    (dict(D=256), UNSUPPORTED), (dict(bs=8), UNSUPPORTED), (dict(T=-3), INVALID), (dict(T=0), OK),
    (dict(T=0, kv=0, bs=8), OK),
])
def test_read_arguments(kw, status):
    assert _read(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(pos=None), INVALID), (dict(freq=None), INVALID),
    (dict(pos=A + 4), INVALID), (dict(freq=A + 2), INVALID), (dict(q=A + 8), INVALID),
    (dict(R=0), INVALID), (dict(R=-16), INVALID), (dict(R=144), INVALID), (dict(R=63), INVALID),
    (dict(R=24, sections=(12,)), UNSUPPORTED), (dict(axes=0), INVALID), (dict(sections=(32, 31)), INVALID),
    (dict(sections=(65, -1)), INVALID), (dict(sections=(16, 16, 16, 8, 8)), UNSUPPORTED),
    (dict(sections=(0, 64), flags=2), INVALID),                # the cyclic order has no room for 64 of axis 1
    (dict(sections=(31, 33), flags=2), INVALID), (dict(flags=4), INVALID), (dict(kv=1, ks=-1.0), INVALID),
    (dict(Hq=-1), INVALID), (dict(D=64, R=64, sections=(32,)), UNSUPPORTED),
    (dict(qo=A + 256), INVALID),                               # q_out overlaps q without being q
    (dict(qo=3 << 22), INVALID),                               # q_out over k_new
    (dict(T=0), OK), (dict(T=0, sections=(32, 32), flags=2), OK), (dict(T=0, sections=(22, 21, 21), flags=3), OK),
])
def test_rope_arguments(kw, status):
    assert _rope(**kw) == status


def test_rope_device_scales_arguments():
    lib, one = pkv.load_library(), (ctypes.c_int32 * 1)(64)
    assert lib.paged_kv_rope_cache_write(A, A, A, A, A, A, A, A, A, A, 4, 4, 2, 128, 128, 1, None, 8, 16, 2, 1.0, 1.0,
                                         0, None) == INVALID          # no sections
    args = [A, A, A, A, A, A, A, A, A, 4, 4, 2, 128, 128, 1, one, 8, 16, A, A, 0, 0]
    for i, bad in ((18, None), (19, None), (18, A + 2), (20, 2)):
        a = list(args)
        a[i] = bad
        assert lib.paged_kv_rope_cache_write_fp8_scaled(*a, None) == INVALID


COMMON = [
    (dict(out=None), INVALID), (dict(q=None), INVALID), (dict(k=A + 8), INVALID), (dict(sc=None), INVALID),
    (dict(sc=A + 8), INVALID), (dict(bt=None), INVALID), (dict(cl=A + 2), INVALID), (dict(B=-1), INVALID),
    (dict(Hq=13), INVALID), (dict(D=64), UNSUPPORTED), (dict(bs=8, L=32), UNSUPPORTED), (dict(Hq=18), UNSUPPORTED),
    (dict(L=65), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(B=0), OK), (dict(B=70000), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(B=8193), UNSUPPORTED), (dict(B=8192, Hq=60000, Hkv=60000, mb=1 << 12, L=1 << 16), UNSUPPORTED),
])
def test_decode_int8_arguments(kw, status):
    assert _decode(**kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(qs=None), INVALID), (dict(qs=A + 1), INVALID), (dict(maxq=65), INVALID), (dict(total=-1), INVALID),
    (dict(maxq=-1), INVALID), (dict(total=0), OK), (dict(maxq=0), OK),
])
def test_chunk_int8_arguments(kw, status):
    assert _chunk(**kw) == status


def test_the_8_bit_type_is_refused_where_it_is_not_named():
    lib = pkv.load_library()
    assert lib.paged_kv_cache_write(A, A, A, A, A, 4, 2, 128, 8, 16, 2, 1.0, 1.0, None) == INVALID
    assert lib.paged_gqa_decode_attention(A, A, A, A, A, A, 2, 12, 2, 128, 16, 4, 64, 64, 0.1, 2, 1.0, 1.0, 0, None, 0,
                                          None) == INVALID
    with pytest.raises(ValueError):
        pkv.kv_dtype_code("int8")


def test_the_binding_refuses_what_is_not_a_dense_cuda_tensor():
    import torch
    x, caches = torch.zeros(1, 2, 128, dtype=torch.float16), torch.zeros(2, 16, 2, 128, dtype=torch.uint8)
    scales, slots = torch.zeros(2, 2, 2, 16), torch.zeros(1, dtype=torch.int64)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        pkv.paged_kv_cache_write_int8(x, x, caches, caches, scales, slots)
    with pytest.raises(TypeError, match="must be a tensor"):
        pkv.paged_kv_cache_write_int8(x, x, None, caches, scales, slots)
    with pytest.raises(ValueError, match="kv_dtype"):
        pkv.paged_kv_cache_read(x, x, caches, caches, slots, kv_dtype="int4")

"""Arguments of the 8-bit cache, rotary cache write and cache read calls that are not tensors of the right shape."""
import numpy as np
import pytest
import torch

import paged_kv_decode_gqa_b200 as pkv

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture
def call():
    """Tensors of a small call."""
    pkv.pkv_device_error()
    z = dict(dtype=torch.float16, device="cuda")
    yield {"k": torch.zeros((4, 2, D), **z), "q": torch.zeros((4, 6, D), **z), "f16": torch.zeros((2, 16, 2, D), **z),
           "u8": torch.full((2, 16, 2, D), 0x38, dtype=torch.uint8, device="cuda"),
           "scales": torch.zeros((2, 2, 2, 16), device="cuda"),
           "slots": torch.arange(4, device="cuda"), "pos": torch.zeros(4, dtype=torch.int64, device="cuda"),
           "freq": torch.ones(64, device="cuda")}
    torch.cuda.synchronize()
    assert pkv.pkv_device_error() == 0


def read(c, kv, **kw):
    pool, more = c["f16"] if kv == "f16" else c["u8"], {"kv_scales": c["scales"]} if kv == "int8" else {}
    pkv.paged_kv_cache_read(c["k"], c["k"].clone(), pool, pool, c["slots"], kv_dtype=kv, **more, **kw)


def rope(c, kv, **kw):
    pool, more = c["f16"] if kv == "f16" else c["u8"], {"kv_scales": c["scales"]} if kv == "int8" else {}
    pkv.paged_kv_rope_cache_write(torch.empty_like(c["q"]), c["q"], c["k"], c["k"], pool, pool.clone(), c["slots"],
                                  c["pos"], c["freq"], kv_dtype=kv, **more, **kw)


@pytest.mark.parametrize("kv", ["f16", "fp8", "int8"])
def test_a_cuda_tensor_is_no_scale_for_the_read(call, kv):
    one = torch.ones((), device="cuda")
    for kw in ({"k_scale": one}, {"v_scale": one}):
        with pytest.raises(TypeError, match="must be a number"):
            read(call, kv, **kw)
    for kw in ({"k_scale": np.float32(2)}, {"k_scale": torch.tensor(2.0), "v_scale": 3}):
        read(call, kv, **kw)
    if kv == "fp8":
        assert (call["k"] == 2).all()                              # the code 0x38 is 1


def test_the_rotary_write_takes_numbers_or_tensors(call):
    one = torch.ones(1, device="cuda")
    rope(call, "fp8", k_scale=one, v_scale=one)
    rope(call, "fp8", k_scale=1, v_scale=np.float64(1))
    for kv, kw in (("fp8", {"k_scale": one}), ("fp8", {"v_scale": one}), ("f16", {"k_scale": one, "v_scale": one}),
                   ("int8", {"v_scale": one})):
        with pytest.raises(TypeError):
            rope(call, kv, **kw)


def test_the_read_is_captured_without_a_copy_of_its_scales(call):
    read(call, "fp8", k_scale=0.5)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        read(call, "fp8", k_scale=0.5)
    call["k"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert (call["k"] == 0.5).all()


def test_an_integer_that_is_no_stream_is_refused(call):
    call["k"].fill_(3)
    with pytest.raises(OverflowError):
        read(call, "f16", stream=1 << 70)
    torch.cuda.synchronize()
    assert (call["k"] == 3).all()                                  # nothing ran on another stream
    read(call, "f16", stream=torch.cuda.current_stream().cuda_stream)
    assert (call["k"] == 0).all()


@pytest.mark.parametrize("of", [list, tuple, np.array, lambda x: [np.int32(v) for v in x], torch.tensor])
def test_sections_are_any_integers(call, of):
    call["pos"] = torch.zeros((2, 4), dtype=torch.int64, device="cuda")
    rope(call, "f16", sections=of([40, 24]))
    for bad in ([40, 25], [40.0, 24.0], [64], [65, -1], ["40", "24"]):
        with pytest.raises((ValueError, pkv.PagedKVError)):
            rope(call, "f16", sections=bad)

"""The 8-bit calls at the far ends of their sizes: as many sequences as the decode takes, more than the streaming
kernel takes, a whole prompt as one chunk, a batch without queries, many tokens in one write; and queries that
are not finite."""
import numpy as np
import pytest
import torch

import paged_kv_decode_gqa_b200 as pkv
from _gpu_helpers import dev, host
from _int8_reference import quantise
from test_gpu_int8_attention import SCALE, Case, workspace

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(autouse=True)
def _clear_device_error():
    pkv.pkv_device_error()
    yield
    torch.cuda.synchronize()


def test_decode_of_8192_sequences():
    rng = np.random.default_rng(1)
    c = Case(600, 2, 1, list(rng.integers(0, 24, 8192)))
    ws = workspace()
    got = c.decode(ws)
    c.check(got, "8192 sequences")
    assert np.array_equal(got, c.decode(ws))


@pytest.mark.parametrize("most", [1, 3])
def test_chunks_of_more_sequences_than_the_streaming_kernel_takes(most):
    rng = np.random.default_rng(most)
    lens = rng.integers(most, 24, 9000)
    c = Case(601 + most, 2, 1, list(lens), list(rng.integers(0, most + 1, 9000)))
    ws = workspace()
    got = c.chunk(ws)
    c.check(got, "9000 sequences")
    assert np.array_equal(got, c.chunk(ws))


@pytest.mark.parametrize("Hq,Hkv,n", [(7, 1, 2900), (2, 2, 1801)])
def test_a_whole_prompt_as_one_chunk(Hq, Hkv, n):
    c = Case(610 + n, Hq, Hkv, [n], [n])
    ws = workspace()
    got = c.chunk(ws)
    c.check(got, f"prompt of {n}")
    assert np.array_equal(got, c.chunk(ws))


@pytest.mark.parametrize("most", [1, 40])
def test_a_batch_without_queries_changes_nothing(most):
    c = Case(620, 14, 2, [50, 300], [1, 1])
    out = torch.full(c.q.shape, 7.0, dtype=torch.float16, device="cuda")
    pkv.paged_gqa_prefill_attention_int8(out, *c.device(), dev(np.zeros(3, np.int32)), max_query_len=most,
                                         max_context_len=300, softmax_scale=SCALE, workspace=workspace())
    assert (host(out) == 7).all() and pkv.pkv_device_error() == 0


def test_write_and_read_of_150001_tokens():
    T, Hkv = 150_001, 1
    rng = np.random.default_rng(3)
    NB = T // 16 + 2
    x = (rng.standard_normal((T, Hkv, D)) * np.exp2(rng.uniform(-3, 3, (T, Hkv, 1)))).astype(np.float16)
    slots = rng.permutation(NB * 16)[:T].astype(np.int64)
    kc, vc = (torch.full((NB, 16, Hkv, D), 128, dtype=torch.uint8, device="cuda") for _ in range(2))
    sc = torch.zeros((NB, Hkv, 2, 16), device="cuda")
    pkv.paged_kv_cache_write_int8(dev(x), dev(x[::-1].copy()), kc, vc, sc, dev(slots))
    out = [torch.empty((T, Hkv, D), dtype=torch.float16, device="cuda") for _ in range(2)]
    pkv.paged_kv_cache_read(*out, kc, vc, dev(slots), kv_dtype="int8", kv_scales=sc)
    codes, scale = quantise(x)
    want = ((codes.astype(np.float32) - 128) * scale[..., None]).astype(np.float16)
    assert np.array_equal(host(out[0]), want) and np.array_equal(host(out[1]), want[::-1])
    assert np.array_equal(host(kc).reshape(-1, Hkv, D)[slots], codes)
    assert pkv.pkv_device_error() == 0


@pytest.mark.parametrize("news", [None, [1, 1, 1], [3, 5, 2], [90, 17, 300]])
@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_a_query_that_is_not_finite_spoils_its_own_row_only(news, value):
    c = Case(630, 14, 2, [100, 17, 640], news)
    ref, bound = c.reference()
    rows, heads = [0, c.q.shape[0] - 1], [3, 8]
    c.q[rows, heads, 5] = value
    got = c.decode() if news is None else c.chunk()
    for r, h in zip(rows, heads):
        assert np.isnan(got[r, h]).any()
        got[r, h], ref[r, h] = 0, 0
    assert (np.abs(got.astype(np.float64) - ref) <= bound).all()
    assert pkv.pkv_device_error() == 0

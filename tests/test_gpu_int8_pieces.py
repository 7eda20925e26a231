"""Pieces of attention items in a workspace that many calls share: each call merges its own."""
import numpy as np
import pytest
import torch

import paged_kv_decode_gqa_b200 as pkv
from _gpu_helpers import dev, host
from test_gpu_int8_attention import SCALE, Case, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_device_error():
    pkv.pkv_device_error()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("Hq,Hkv,lens,n", [(28, 4, [2000, 700, 90], 5), (8, 8, [6000], 20), (7, 1, [9000, 40], 3),
                                           (14, 2, [1500, 800], 90)])
def test_calls_in_a_row_merge_their_own_pieces(Hq, Hkv, lens, n):
    """Two inputs in turn through one workspace, with nothing between the calls: the same places hold one
    input's pieces, then the other's, and every output is bit for bit that of a workspace of its own."""
    cases = [Case(400 + i, Hq, Hkv, lens, [min(n, m) for m in lens]) for i in range(2)]
    want = [c.chunk() for c in cases]
    for c, w in zip(cases, want):
        c.check(w, "alone")
    args, qs, ws = [c.device() for c in cases], [dev(c.qs) for c in cases], workspace()
    outs = []
    for rep in range(30):
        i = rep % 2
        out = torch.full(cases[i].q.shape, float("nan"), dtype=torch.float16, device="cuda")
        pkv.paged_gqa_prefill_attention_int8(out, *args[i], qs[i], max_query_len=n, max_context_len=max(lens),
                                             softmax_scale=SCALE, workspace=ws)
        outs.append((i, out))
    for i, out in outs:
        assert np.array_equal(host(out), want[i])
    assert pkv.pkv_device_error() == 0

"""Memory order that no run can show to be missing: read from the kernels' sources.

A piece of an attention item is stored by one thread block and merged by another in the same launch. What
orders the two is a release-acquire ticket, and around it the steps that carry the order to every thread and
to every kind of access that takes part.
"""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).resolve().parents[1] / "paged_kv_decode_gqa_b200" / "csrc"


def _code(name):
    """A source file without its comments."""
    return re.sub(r"//[^\n]*", "", (CSRC / name).read_text())


def test_pieces_read_by_bulk_copies_are_fenced_between_the_proxies():
    """The narrow chunk merge reads pieces that generic stores wrote through the asynchronous proxy: a fence
    between the proxies for global memory follows the stores, before the barrier and the ticket, and another
    one stands between the ticket and the copies."""
    text = _code("chunk_int8_tc.cuh")
    stores = text.index("__stcg(reinterpret_cast<float2*>(part")
    ticket = text.index("atomic_add_acq_rel_gpu(p.tickets + c_last", stores)
    copy = text.index("bulk_load(base", ticket)
    barrier = text.index("__syncthreads()", stores)
    assert barrier < ticket
    assert "fence_proxy_async_global()" in text[stores:barrier]
    assert "fence_proxy_async_global()" in text[ticket:copy]


@pytest.mark.parametrize("name", ["stream_int8.cuh", "chunk_int8_tc.cuh", "decode_balanced.cuh", "prefill_tc.cuh"])
def test_a_warps_ticket_is_followed_by_a_warp_barrier(name):
    """Lane 0 takes a warp's ticket and tells the others by a shuffle, which orders no memory: a warp barrier
    follows, before any lane reads what the ticket's acquire makes visible."""
    text = _code(name)
    tickets = [m.end() for m in re.finditer(r"prev = __shfl_sync\(0xffffffffu, prev, 0\);", text)]
    assert tickets
    for end in tickets:
        assert re.match(r"\s*__syncwarp\(\);", text[end:]), text[end:end + 120]

"""Decode and chunk attention over the 8-bit cache, against the plain float64 form with the bound that
tests/_int8_reference.py derives; and the step they make with the projection and the rotary write."""
import numpy as np
import pytest
import torch

import paged_kv_decode_gqa_b200 as pkv
from _gpu_helpers import dev, host
from _int8_reference import assert_within, attention

pytestmark = pytest.mark.gpu
F16, F32 = np.float16, np.float32
D = 128
SCALE = float(F32(D ** -0.5))


@pytest.fixture(autouse=True)
def _clear_device_error():
    pkv.pkv_device_error()
    yield
    torch.cuda.synchronize()


class Case:
    """A seeded 8-bit cache in shuffled pages. Rows past a context and free pages hold NaN scales and
    random codes; unused table entries are out of range."""

    def __init__(self, seed, Hq, Hkv, lens, news=None, q_scale=1.0, spread=1.0, values=None):
        rng = np.random.default_rng(seed)
        self.Hq, self.Hkv, self.B = Hq, Hkv, len(lens)
        self.lens = np.array(lens, np.int32)
        self.news = np.array(news if news is not None else [1] * self.B, np.int32)
        self.qs = np.concatenate([[0], np.cumsum(self.news)]).astype(np.int32)
        pages = -(-self.lens // 16)
        self.NB = int(pages.sum()) + 3
        perm = rng.permutation(self.NB).astype(np.int32)
        self.tables = np.full((self.B, max(1, int(pages.max(initial=0))) + 1), -1, np.int32)
        self.codes = rng.integers(0, 256, (2, self.NB, 16, Hkv, D)).astype(np.uint8)
        self.scales = np.full((self.NB, Hkv, 2, 16), np.nan, F32)
        at = 0
        for b, n in enumerate(pages):
            self.tables[b, :n] = perm[at:at + n]
            at += n
            for t in range(int(self.lens[b])):
                blk = self.tables[b, t // 16]
                c = rng.standard_normal((2, Hkv, D)) * 42
                self.codes[:, blk, t % 16] = np.clip(np.rint(c), -127, 127) + 128
                self.scales[blk, :, :, t % 16] = 3.0 / 127 * np.exp2(rng.uniform(-spread, spread, (Hkv, 2)))
        self.q = (rng.standard_normal((int(self.qs[-1]), Hq, D)) * q_scale).astype(F16)
        self.max_len = max(1, int(self.lens.max(initial=0)))

    def rows_of(self, b):
        t = np.arange(int(self.lens[b]))
        return self.tables[b, t // 16], t % 16

    def device(self):
        return (dev(self.q), dev(self.codes[0]), dev(self.codes[1]), dev(self.scales), dev(self.tables),
                dev(self.lens))

    def decode(self, ws=None, scale=SCALE, max_len=None, args=None, out=None):
        out = torch.full(self.q.shape, float("nan"), dtype=torch.float16, device="cuda") if out is None else out
        pkv.paged_gqa_decode_attention_int8(out, *(args or self.device()), max_context_len=max_len or self.max_len,
                                            softmax_scale=scale, workspace=workspace() if ws is None else ws)
        return host(out)

    def chunk(self, ws=None, scale=SCALE, args=None, qs=None, max_new=None):
        out = torch.full(self.q.shape, float("nan"), dtype=torch.float16, device="cuda")
        qs = self.qs if qs is None else qs
        pkv.paged_gqa_prefill_attention_int8(
            out, *(args or self.device()), dev(qs), max_query_len=max_new or max(1, int(self.news.max(initial=0))),
            max_context_len=self.max_len, softmax_scale=scale, workspace=workspace() if ws is None else ws)
        return host(out)

    def reference(self, scale=SCALE):
        return attention(self.q, *self.codes, self.scales, self.tables, self.lens, self.qs, scale)

    def check_rows(self, got, rows, what=""):
        ref, bound = self.reference()
        assert_within(got[rows], ref[rows], bound[rows], what)

    def check(self, got, what="", scale=SCALE):
        assert_within(got, *self.reference(scale), what)
        assert pkv.pkv_device_error() == 0


def workspace():
    return torch.zeros(pkv.paged_gqa_prefill_workspace_size(8, 8, D, "int8"), dtype=torch.uint8, device="cuda")


HEADS = [(12, 2), (28, 4), (8, 8), (10, 2), (8, 1), (6, 6), (5, 1), (3, 1), (16, 4)]


# ------------------------------------------------------------------ decode
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_decode_lengths_and_groups(Hq, Hkv):
    c = Case(Hq * 10 + Hkv, Hq, Hkv, [1, 15, 16, 17, 40, 2, 33, 300, 64, 1000])
    c.check(c.decode(), f"{Hq}/{Hkv}")


def test_decode_empty_contexts_give_zero_rows():
    c = Case(1, 12, 2, [0, 5, 0, 17, 0])
    got = c.decode()
    assert (got[[0, 2, 4]] == 0).all()
    c.check(got, "empty contexts")
    c = Case(2, 12, 2, [0, 0])
    assert (c.decode() == 0).all()


def test_decode_one_token_returns_its_value():
    c = Case(3, 8, 8, [1] * 4)
    blk, _ = zip(*(c.rows_of(b) for b in range(4)))
    want = np.stack([(c.codes[1][k[0], 0].astype(F32) - 128) * c.scales[k[0], :, 1, 0][:, None] for k in blk])
    assert np.abs(c.decode().astype(F32) - want).max() <= 2 * 2.0 ** -11 * np.abs(want).max()


def test_decode_long_sequence_is_merged_over_many_workers():
    c = Case(4, 7, 1, [9000, 3, 200])
    ws = workspace()
    got = c.decode(ws)
    c.check(got, "long")
    assert np.array_equal(got, c.decode(ws))                        # the same workspace, the same bytes
    assert (ws[:1 << 12] == 0).all()                                # tickets are back at zero


def test_decode_many_short_sequences():
    rng = np.random.default_rng(5)
    c = Case(5, 4, 2, list(rng.integers(0, 60, 1700)))
    c.check(c.decode(), "many")


def test_decode_cuts_at_every_warp():
    """Segments about as long as a warp's run: every run begins and ends inside one, so a CTA merges one
    chain more than it has warps, and both its first and its last reach into other CTAs."""
    rng = np.random.default_rng(55)
    c = Case(55, 2, 1, list(rng.integers(150, 230, 1100)))
    ws = workspace()
    got = c.decode(ws)
    c.check(got, "cuts")
    assert np.array_equal(got, c.decode(ws))


def test_decode_one_sequence_over_the_whole_grid():
    """One long sequence and one head: its pieces meet in a ticket tree of two levels."""
    c = Case(56, 1, 1, [40000])
    ws = workspace()
    got = c.decode(ws)
    c.check(got, "whole grid")
    assert np.array_equal(got, c.decode(ws)) and (ws[:1 << 12] == 0).all()


@pytest.mark.parametrize("kind", ["large logits", "zero scale", "negative scale", "tiny values", "huge values",
                                  "zero rows", "mixed", "growing"])
def test_decode_value_ranges(kind):
    c = Case(6, 14, 2, [100, 17, 640], q_scale=6.0 if kind == "large logits" else 1.0)
    scale = {"zero scale": 0.0, "negative scale": -SCALE}.get(kind, SCALE)
    live = np.isfinite(c.scales)
    if kind == "tiny values":
        c.scales[:, :, 1][live[:, :, 1]] = 2.0 ** -24 / 127
    elif kind == "huge values":
        c.scales[:, :, 1][live[:, :, 1]] = 65504 / 127 / 4
    elif kind == "zero rows":                                       # as the write stores rows of zeros; and scale 0
        for b in range(3):
            blk, row = c.rows_of(b)
            c.codes[:, blk[::3], row[::3]] = 128
            c.scales[blk[::3], :, :, row[::3]] = 2.0 ** -24 / 127
            c.scales[blk[1::3], :, :, row[1::3]] = 0.0
    elif kind == "mixed":                                           # value scales over 2^30, logits untouched
        rng = np.random.default_rng(7)
        c.scales[:, :, 1] *= np.exp2(rng.uniform(-25, 5, c.scales[:, :, 1].shape)).astype(F32)
    elif kind == "growing":                                         # the running maximum is raised again and again
        for b in range(3):
            blk, row = c.rows_of(b)
            c.scales[blk, :, 0, row] *= np.linspace(0.1, 8, len(blk)).astype(F32)[:, None]
    c.check(c.decode(scale=scale), kind, scale)


def test_free_rows_and_pages_are_never_read():
    c = Case(8, 12, 2, [1, 30, 95])
    a = c.decode()
    free = ~np.isfinite(c.scales)
    c.scales[free] = 1e30
    c.codes ^= np.where(free.any(2).transpose(0, 2, 1)[..., None], 0xA5, 0).astype(np.uint8)[None]
    assert np.array_equal(a, c.decode())
    assert pkv.pkv_device_error() == 0


def test_block_permutation_is_invisible():
    c = Case(9, 12, 2, [500, 31])
    a = c.decode()
    perm = np.random.default_rng(0).permutation(c.NB)
    inv = np.argsort(perm)
    c.codes, c.scales = c.codes[:, perm], c.scales[perm]
    c.tables = np.where(c.tables >= 0, inv[c.tables], -1).astype(np.int32)
    assert np.array_equal(a, c.decode())


def test_decode_flags_bad_lengths_blocks_and_scales():
    c = Case(10, 12, 2, [40, 100, 20, 64])
    c.check(c.decode(), "good")
    c.lens[0] = 1 << 20                                             # past the table: clamped
    c.lens[2] = -4
    got = c.decode(max_len=112)
    assert pkv.pkv_device_error() & pkv.DEVERR_CONTEXT_LEN
    c.lens[[0, 2]] = 40, 20
    c.check_rows(got, [1, 3], "the other sequences")               # (their split may differ)
    assert (got[2] == 0).all()
    good = c.decode()
    c.tables[1, 3] = c.NB
    c.tables[3, 0] = -2
    got = c.decode()
    assert pkv.pkv_device_error() == pkv.DEVERR_BLOCK_ID
    assert np.isfinite(got).all() and np.array_equal(got[[0, 2]], good[[0, 2]])
    for bad in (np.nan, np.inf, -1.0):
        d = Case(10, 12, 2, [40, 100, 20, 64])
        blk, row = d.rows_of(0)
        d.scales[blk[5], :, :, row[5]] = bad
        got = d.decode()
        assert pkv.pkv_device_error() == pkv.DEVERR_SCALE
        assert np.isfinite(got).all() and np.array_equal(got[1:], good[1:])


# ------------------------------------------------------------------ chunks
CHUNKS = [  # Hq, Hkv, lens, news
    (12, 2, [40, 17, 100, 16, 33], [1, 1, 1, 1, 1]),
    (28, 4, [40, 17, 100, 300, 5], [5, 5, 5, 5, 5]),
    (28, 4, [40, 17, 100, 300, 5], [2, 0, 3, 1, 5]),
    (12, 2, [7, 129, 64, 500], [7, 3, 64, 17]),
    (8, 8, [200, 31, 16], [33, 31, 16]),
    (8, 1, [2000, 15, 90], [4, 15, 9]),
    (10, 2, [700, 65], [130, 65]),
    (6, 6, [1, 2, 260], [1, 2, 260]),
    (3, 1, [50, 1025], [11, 300]),
    (28, 4, [640, 1300], [400, 150]),
    (7, 1, [4000, 12], [3, 1]),
]


@pytest.mark.parametrize("i", range(len(CHUNKS)))
def test_chunk_lengths_and_groups(i):
    Hq, Hkv, lens, news = CHUNKS[i]
    c = Case(100 + i, Hq, Hkv, lens, news)
    ws = workspace()
    got = c.chunk(ws)
    c.check(got, str(CHUNKS[i]))
    assert np.array_equal(got, c.chunk(ws))


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 6, 8, 12, 16, 20, 31, 40, 64])
def test_chunk_lengths_one_by_one(n):
    """Every size of a short chunk, and the lengths around the change between kernels and tiles."""
    c = Case(200 + n, 14, 2, [n, n + 1, n + 15, n + 16, n + 700], [n] * 5)
    c.check(c.chunk(), f"{n} new tokens")


@pytest.mark.parametrize("kind", ["large logits", "zero scale", "negative scale", "growing", "mixed", "small rows"])
@pytest.mark.parametrize("news", [[3, 5, 2], [90, 17, 300]])
def test_chunk_value_ranges(kind, news):
    c = Case(11, 14, 2, [100, 17, 640], news, q_scale=6.0 if kind == "large logits" else 1.0)
    scale = {"zero scale": 0.0, "negative scale": -SCALE}.get(kind, SCALE)
    if kind == "growing":
        for b in range(3):
            blk, row = c.rows_of(b)
            c.scales[blk, :, 0, row] *= np.linspace(0.1, 8, len(blk)).astype(F32)[:, None]
    elif kind == "mixed":
        rng = np.random.default_rng(7)
        c.scales[:, :, 1] *= np.exp2(rng.uniform(-8, 8, c.scales[:, :, 1].shape)).astype(F32)
    elif kind == "small rows":                                        # scales around 2^-12 and down to f16's smallest
        rng = np.random.default_rng(8)
        c.scales *= np.exp2(rng.integers(-24, 1, c.scales.shape)).astype(F32)
        c.scales = np.maximum(c.scales, F32(2.0 ** -24 / 127))
    c.check(c.chunk(scale=scale), kind, scale)


def test_chunk_of_one_is_decode():
    c = Case(12, 28, 4, [100, 1, 700, 16])
    c.check(c.chunk(), "chunk")
    c.check(c.decode(), "decode")


def test_chunk_free_rows_are_never_read():
    for news in ([1, 5, 4], [1, 30, 90]):
        c = Case(13, 12, 2, [1, 30, 95], news)
        a = c.chunk()
        free = ~np.isfinite(c.scales)
        c.scales[free] = 1e30
        c.codes ^= np.where(free.any(2).transpose(0, 2, 1)[..., None], 0xA5, 0).astype(np.uint8)[None]
        assert np.array_equal(a, c.chunk())
        assert pkv.pkv_device_error() == 0


@pytest.mark.parametrize("n", [4, 40])
def test_chunk_flags_inconsistent_lengths_and_leaves_their_rows(n):
    c = Case(14, 12, 2, [200, 200, 200], [n, n, n])
    c.lens[1] = n - 1                                                 # fewer tokens than queries
    out = torch.full(c.q.shape, 7.0, dtype=torch.float16, device="cuda")
    args = c.device()
    pkv.paged_gqa_prefill_attention_int8(out, *args, dev(c.qs), max_query_len=n, max_context_len=200,
                                         softmax_scale=SCALE, workspace=workspace())
    got = host(out)
    assert pkv.pkv_device_error() == pkv.DEVERR_CONTEXT_LEN
    assert (got[n:2 * n] == 7).all()
    c.lens[1] = 200
    c.check_rows(got, np.r_[0:n, 2 * n:3 * n], "the other sequences")
    bad = c.qs.copy()
    bad[3] = 3 * n + 5                                                # past the rows of q
    c.chunk(qs=bad, max_new=n + 5)
    assert pkv.pkv_device_error() == pkv.DEVERR_CONTEXT_LEN


@pytest.mark.parametrize("n", [4, 40])
def test_chunk_flags_blocks_and_scales(n):
    c = Case(15, 12, 2, [200, 100, 60], [n, n, n])
    good = c.chunk()
    c.tables[0, 2] = c.NB + 3
    got = c.chunk()
    assert pkv.pkv_device_error() == pkv.DEVERR_BLOCK_ID
    assert np.isfinite(got).all() and np.array_equal(got[n:], good[n:])
    c = Case(15, 12, 2, [200, 100, 60], [n, n, n])
    blk, row = c.rows_of(0)
    c.scales[blk[5], :, :, row[5]] = np.nan
    got = c.chunk()
    assert pkv.pkv_device_error() == pkv.DEVERR_SCALE
    assert np.isfinite(got).all() and np.array_equal(got[n:], good[n:])


@pytest.mark.parametrize("n", [1, 4, 40])
def test_chunk_leaves_rows_behind_the_last_sequence(n):
    """A batch padded to more rows than its sequences have: the rest of out stays as it was."""
    c = Case(16, 28, 4, [200, 61], [n, n])
    q, kc, vc, sc, bt, cl = c.device()
    q = torch.cat([q, torch.full((5, 28, D), float("nan"), dtype=torch.float16, device="cuda")])
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    pkv.paged_gqa_prefill_attention_int8(out, q, kc, vc, sc, bt, cl, dev(c.qs), max_query_len=n + 3, max_context_len=208,
                                         softmax_scale=SCALE, workspace=workspace())
    got = host(out)
    assert (got[2 * n:] == 7).all()
    c.check(got[:2 * n], f"padded {n}")


def test_chunk_many_sequences_and_ragged_items():
    """More sequences than a block has threads, most without queries; and pieces of one KV tile."""
    rng = np.random.default_rng(17)
    lens = rng.integers(1, 40, 700)
    news = np.where(rng.random(700) < 0.2, np.minimum(lens, rng.integers(1, 12, 700)), 0)
    news[[0, 699]] = 1
    c = Case(17, 14, 2, list(lens), list(news))
    c.check(c.chunk(), "many sequences, narrow")
    lens[5], news[5] = 330, 70
    c = Case(18, 14, 2, list(lens), list(news))
    c.check(c.chunk(), "many sequences, wide")


@pytest.mark.parametrize("B,n,hi", [(64, 5, 2048), (96, 3, 700), (148, 9, 260), (24, 40, 1500)])
def test_chunk_runs_of_many_pieces(B, n, hi):
    """Several items per CTA, of one KV tile to many, so that stages and barriers run on across pieces."""
    rng = np.random.default_rng(B)
    c = Case(300 + B, 14, 2, list(rng.integers(n, hi, B)), [n] * B)
    ws = workspace()
    got = c.chunk(ws)
    c.check(got, f"{B} sequences")
    assert np.array_equal(got, c.chunk(ws))
    assert pkv.pkv_device_error() == 0


@pytest.mark.parametrize("news", [None, [5, 4, 3], [40, 33, 130]])
def test_sequences_that_share_pages(news):
    """A common prefix: three tables name the same pages for the first 160 tokens."""
    c = Case(77, 14, 2, [300, 190, 420], news)
    for b in (1, 2):
        c.tables[b, :10] = c.tables[0, :10]
    c.check(c.decode() if news is None else c.chunk(), "shared prefix")


# ------------------------------------------------------------------ how calls meet
def test_one_workspace_serves_every_plan_in_turn():
    ws = workspace()
    cases = [Case(20, 28, 4, [900, 40]), Case(21, 28, 4, [900, 40], [3, 2]), Case(22, 7, 1, [3000], [40]),
             Case(23, 8, 8, [2500, 9]), Case(24, 28, 4, [900, 40], [5, 5]), Case(25, 8, 8, [700], [300])]
    for rep in range(2):
        for i, c in enumerate(cases):
            c.check(c.chunk(ws) if (c.news > 1).any() else c.decode(ws), f"{rep} {i}")


def test_workspaces_too_small_or_misaligned_are_refused():
    c, d = Case(26, 12, 2, [40], [2]), Case(26, 12, 2, [40])
    n = pkv.paged_gqa_decode_workspace_size_int8()
    full = workspace()
    for ws in (full[:n - 1], full[128:]):
        with pytest.raises(pkv.PagedKVError):
            d.decode(ws)
    with pytest.raises(pkv.PagedKVError):
        c.chunk(full[:n // 2])
    with pytest.raises(ValueError):
        d.decode(full.cpu())


def test_captured_calls_replay_on_new_inputs():
    """Decode and a chunk captured into one graph, replayed after their inputs change in place."""
    a, b = Case(27, 28, 4, [300, 2, 77]), Case(28, 28, 4, [300, 20, 77], [4, 20, 1])
    aa, bb = a.device(), b.device()
    ws = workspace()
    out_a, out_b = (torch.zeros(c.q.shape, dtype=torch.float16, device="cuda") for c in (a, b))
    qs = dev(b.qs)

    def step():
        pkv.paged_gqa_decode_attention_int8(out_a, *aa, max_context_len=300, softmax_scale=SCALE, workspace=ws)
        pkv.paged_gqa_prefill_attention_int8(out_b, *bb, qs, max_query_len=20, max_context_len=300,
                                             softmax_scale=SCALE, workspace=ws)
    step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for c, args in ((a, aa), (b, bb)):
        c.q = (c.q * F16(-0.5)).astype(F16)
        args[0].copy_(dev(c.q))
        c.lens[0] -= 3
        args[5].copy_(dev(c.lens))
    for _ in range(3):
        out_a.zero_(), out_b.zero_()
        graph.replay()
        torch.cuda.synchronize()
        a.check(host(out_a), "captured decode")
        b.check(host(out_b), "captured chunk")


def test_two_streams_with_their_own_workspaces():
    a, b = Case(29, 28, 4, [1500, 40]), Case(30, 28, 4, [1200, 80], [64, 3])
    aa, bb, wa, wb, qs = a.device(), b.device(), workspace(), workspace(), dev(b.qs)
    outs = [torch.zeros(c.q.shape, dtype=torch.float16, device="cuda") for c in (a, b)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        pkv.paged_gqa_decode_attention_int8(outs[0], *aa, max_context_len=1500, softmax_scale=SCALE, workspace=wa,
                                            stream=s1)
        pkv.paged_gqa_prefill_attention_int8(outs[1], *bb, qs, max_query_len=64, max_context_len=1200,
                                             softmax_scale=SCALE, workspace=wb, stream=s2)
    torch.cuda.synchronize()
    a.check(host(outs[0]), "stream 1")
    b.check(host(outs[1]), "stream 2")


def test_a_layer_of_decode_steps():
    """Projection -> rotary write -> decode, three steps in a row, and the same tokens as one chunk: the
    cache grows in place, and every step's attention is the reference's on the bytes in the cache."""
    T, H, Hq, Hkv, NB = 3, 512, 14, 2, 40
    rng = np.random.default_rng(31)
    x = [dev(rng.standard_normal((T, H)).astype(F16)) for _ in range(3)]
    w = dev((rng.standard_normal(((Hq + 2 * Hkv) * D, H)) / np.sqrt(H)).astype(F16))
    gamma = dev(np.ones(H, F16))
    start = np.array([30, 0, 95], np.int32)
    c = Case(32, Hq, Hkv, start)                                       # what earlier steps left
    tables = np.stack([rng.permutation(NB)[:8] + 40 * b for b in range(T)]).astype(np.int32)
    codes = np.full((2, 120, 16, Hkv, D), 128, np.uint8)
    scales = np.full((120, Hkv, 2, 16), np.nan, F32)
    for b in range(T):
        blk, row = c.rows_of(b)
        t = np.arange(start[b])
        codes[:, tables[b, t // 16], t % 16] = c.codes[:, blk, row]
        scales[tables[b, t // 16], :, :, t % 16] = c.scales[blk, :, :, row]
    kc, vc, sc, bt = dev(codes[0]), dev(codes[1]), dev(scales), dev(tables)
    freq = dev((1e6 ** (-np.arange(64) / 64)).astype(F32))
    ws = workspace()
    residual, q, k, v = (torch.zeros(s, dtype=torch.float16, device="cuda") for s in
                         ((T, H), (T, Hq, D), (T, Hkv, D), (T, Hkv, D)))
    queries = []
    for step in range(3):
        lens = start + step + 1
        pos = np.repeat((lens - 1)[None].astype(np.int64), 3, 0)
        slots = np.array([tables[b, p // 16] * 16 + p % 16 for b, p in enumerate(lens - 1)], np.int64)
        pkv.fused_add_rmsnorm_qkv(x[step], torch.zeros_like(residual), gamma, w, None, residual, q, k, v)
        pkv.paged_kv_rope_cache_write(q, q, k, v, kc, vc, dev(slots), dev(pos), freq, sections=[16, 24, 24],
                                      kv_dtype="int8", kv_scales=sc)
        out = torch.full_like(q, float("nan"))
        pkv.paged_gqa_decode_attention_int8(out, q, kc, vc, sc, bt, dev(lens.astype(np.int32)), max_context_len=128,
                                            softmax_scale=SCALE, workspace=ws)
        ref = attention(host(q), host(kc), host(vc), host(sc), tables, lens, np.arange(T + 1), SCALE)
        assert_within(host(out), *ref, f"step {step}")
        queries.append(host(q))
    # the three tokens of every sequence as one chunk see what the steps saw
    chunk_q = np.stack(queries, 1).reshape(3 * T, Hq, D)
    out = torch.full((3 * T, Hq, D), float("nan"), dtype=torch.float16, device="cuda")
    qs = np.arange(T + 1, dtype=np.int32) * 3
    lens = (start + 3).astype(np.int32)
    pkv.paged_gqa_prefill_attention_int8(out, dev(chunk_q), kc, vc, sc, bt, dev(lens), dev(qs), max_query_len=3,
                                         max_context_len=128, softmax_scale=SCALE, workspace=ws)
    assert_within(host(out), *attention(chunk_q, host(kc), host(vc), host(sc), tables, lens, qs, SCALE), "chunk")
    assert pkv.pkv_device_error() == 0

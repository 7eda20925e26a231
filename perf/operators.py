"""Workloads of the 8-bit paged cache and the operators around it, with their plain forms.

Four operators, each on its own sizes:
  write   K/V quantised into the cache as they are written (8-bit codes, one scale per token and KV
          head), and the same tokens read back
  rope    rotary positions (one or several axes) applied to q and k, K/V written to the cache
  decode  one query token per sequence over the 8-bit cache
  chunk   several new query tokens per sequence over the 8-bit cache, causal

The cache is paged: [blocks, 16, KV heads, 128] codes, scales [blocks, KV heads, 2 (K, V), 16].
A code c (0..255) with scale s stands for (c - 128) * s.
"""
import math

import torch

own = False

D = 128          # channels of a head
BS = 16          # tokens of a page
SMALLEST = 2.0 ** -24


def listed():
    return [
        # one token of one sequence: a single-user decode step's cache write, latency only
        {"name": "write 1 token", "op": "write", "T": 1, "Hkv": 2, "scattered": True},
        # a prefill chunk's worth of tokens (odd, so the last page is partly filled), 7B heads
        {"name": "write 16411 tokens", "op": "write", "T": 16411, "Hkv": 4, "scattered": False},
        # the decode step of the 7B-shaped workload: one token of 128 sequences, f16 cache
        {"name": "rope f16 128 tokens", "op": "rope", "T": 128, "Hq": 28, "Hkv": 4, "kv": "f16", "rotary": 128,
         "axes": 1, "pairs": False, "cyclic": False, "scattered": True},
        # the decode step of the 1.5B-shaped workload with image positions, 8-bit cache, read back
        {"name": "rope int8 64 tokens", "op": "rope", "T": 64, "Hq": 12, "Hkv": 2, "kv": "int8", "rotary": 128,
         "axes": 3, "pairs": False, "cyclic": False, "scattered": True},
        # prefill of an image-and-text batch: three position axes, 7B heads
        {"name": "rope f16 16384 tokens", "op": "rope", "T": 16384, "Hq": 28, "Hkv": 4, "kv": "f16", "rotary": 128,
         "axes": 3, "pairs": False, "cyclic": True, "scattered": False},
        # a ragged chunk into an FP8 cache, adjacent channels paired, half of each head rotated
        {"name": "rope fp8 2049 tokens", "op": "rope", "T": 2049, "Hq": 12, "Hkv": 2, "kv": "fp8", "rotary": 64,
         "axes": 1, "pairs": True, "cyclic": False, "scattered": False},
        # the tiny workload: two short sequences, latency only
        {"name": "decode tiny", "op": "decode", "B": 2, "Hq": 12, "Hkv": 2, "lo": 17, "hi": 40, "long": 0},
        # the 1.5B-shaped decode step
        {"name": "decode 64 sequences", "op": "decode", "B": 64, "Hq": 12, "Hkv": 2, "lo": 32, "hi": 2048, "long": 0},
        # the 7B-shaped decode step, the ordinary large one
        {"name": "decode 128 sequences", "op": "decode", "B": 128, "Hq": 28, "Hkv": 4, "lo": 512, "hi": 4096,
         "long": 0},
        # one long document among short chats
        {"name": "decode skewed", "op": "decode", "B": 8, "Hq": 28, "Hkv": 4, "lo": 128, "hi": 1024, "long": 32768},
        # drafted tokens checked against the target: 5 new tokens per sequence, bound by the cache read
        {"name": "chunk 5 of 64 sequences", "op": "chunk", "B": 64, "Hq": 28, "Hkv": 4, "n_lo": 5, "n_hi": 5,
         "lo": 32, "hi": 2048},
        # chunked prefill: 512 new tokens at the end of 2048-token contexts, bound by the products
        {"name": "chunk 512 of 8 sequences", "op": "chunk", "B": 8, "Hq": 28, "Hkv": 4, "n_lo": 512, "n_hi": 512,
         "lo": 2048, "hi": 2048},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(12, 2), (28, 4), (8, 8), (16, 4), (10, 2), (8, 1), (6, 6), (32, 8), (5, 1)]


def draw(rng):
    op = rng.choice(["write", "rope", "decode", "chunk"])
    Hq, Hkv = rng.choice(HEADS)
    if op == "write":
        return {"op": op, "T": _log_int(rng, 1, 65644 // Hkv), "Hkv": Hkv, "scattered": rng.random() < 0.5}
    if op == "rope":
        rotary = rng.choice([32, 64, 96, 128, 128])
        axes = rng.choice([1, 1, 2, 3])
        return {"op": op, "T": _log_int(rng, 1, 16384 * 36 // (Hq + 2 * Hkv)), "Hq": Hq, "Hkv": Hkv,
                "kv": rng.choice(["f16", "fp8", "int8"]), "rotary": rotary, "axes": axes,
                "pairs": rng.random() < 0.4, "cyclic": axes > 1 and rng.random() < 0.5,
                "scattered": rng.random() < 0.5}
    if op == "decode":
        hi = _log_int(rng, 1, 8192)
        lo = rng.randint(1, hi)
        most = 128 * 4096 * 4 // (hi * Hkv)
        return {"op": op, "B": _log_int(rng, 1, max(1, min(256, most))), "Hq": Hq, "Hkv": Hkv, "lo": lo, "hi": hi,
                "long": 0}
    n_hi = _log_int(rng, 1, 512)
    n_lo = rng.randint(1, n_hi)
    hi = n_hi + _log_int(rng, 1, 2048)
    lo = rng.randint(n_hi, hi)
    most = 8 * 512 * 2048 * 28 // (n_hi * hi * Hq)
    return {"op": op, "B": _log_int(rng, 1, max(1, min(64, most))), "Hq": Hq, "Hkv": Hkv, "n_lo": n_lo, "n_hi": n_hi,
            "lo": lo, "hi": hi}


# ------------------------------------------------------------------ sizes that follow from a case
def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi]: the same sum whatever the seed."""
    return [lo + (hi - lo) * (2 * i + 1) // (2 * n) for i in range(n)]


def _lengths(case):
    """Context lengths of a decode or chunk case, before shuffling."""
    if case.get("long"):
        return [case["long"]] + _spread(case["lo"], case["hi"], case["B"] - 1)
    return _spread(case["lo"], case["hi"], case["B"])


def _sections(case):
    """Frequencies of each position axis: about a quarter for the first, the rest shared."""
    half, axes = case["rotary"] // 2, case["axes"]
    if axes == 1:
        return [half]
    if case["cyclic"]:
        rest = half // axes - 1
        return [half - rest * (axes - 1)] + [rest] * (axes - 1)
    first = half // 4 if axes == 3 else half // 2
    rest = (half - first) // (axes - 1)
    return [half - rest * (axes - 1)] + [rest] * (axes - 1)


def _axis_of(case):
    """The position axis of every frequency."""
    half, sections = case["rotary"] // 2, _sections(case)
    if case["cyclic"]:
        axes = case["axes"]
        return [j % axes if j % axes and j < axes * sections[j % axes] else 0 for j in range(half)]
    return [a for a, n in enumerate(sections) for _ in range(n)]


def work(case):
    op = case["op"]
    if op == "write":
        rows = 2 * case["T"] * case["Hkv"]
        return {"bytes": rows * (2 * D + (D + 4)) + rows * ((D + 4) + 2 * D) + 16 * case["T"], "flops": 3 * rows * D}
    if op == "rope":
        T, e = case["T"], {"f16": 2 * D, "fp8": D, "int8": D + 4}[case["kv"]]
        q, kv = T * case["Hq"], 2 * T * case["Hkv"]
        back = kv * (e + 2 * D) + 8 * T if case["kv"] == "int8" else 0
        return {"bytes": q * 4 * D + kv * (2 * D + e) + T * (8 + 8 * case["axes"]) + 2 * case["rotary"] + back,
                "flops": 3 * (q + kv // 2) * case["rotary"]}
    lens = _lengths(case)
    cache = 2 * sum(lens) * case["Hkv"] * (D + 4) + 4 * sum(-(-n // BS) for n in lens) + 4 * len(lens)
    if op == "decode":
        return {"bytes": cache + 4 * case["B"] * case["Hq"] * D, "flops": 4 * D * case["Hq"] * sum(lens)}
    news = _spread(case["n_lo"], case["n_hi"], case["B"])
    seen = sum(n * (L - n) + n * (n + 1) // 2 for n, L in zip(news, lens))
    return {"bytes": cache + 4 * sum(news) * case["Hq"] * D + 4 * len(news), "flops": 4 * D * case["Hq"] * seen}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _activations(g, *shape):
    """f16 rows as a projection gives them: a magnitude per row, and one channel in 32 larger than the rest."""
    x = _normal(g, *shape) * torch.exp2(_normal(g, *shape[:-1], 1))
    big = torch.rand(shape[-1], generator=g, device="cuda") < 1 / 32
    return (x * (1 + 7 * big)).half()


def _slots(g, case, blocks):
    """Slots of the new tokens: scattered over sequences (a decode step), or filling pages in order (a chunk)."""
    T = case["T"]
    perm = torch.randperm(blocks, generator=g, device="cuda")
    t = torch.arange(T, device="cuda")
    if case["scattered"]:
        return perm[t] * BS + torch.randint(0, BS, (T,), generator=g, device="cuda")
    return perm[t // BS] * BS + t % BS


def _pool(g, kv, blocks, Hkv):
    """An empty cache of one type: K, V, scales."""
    dtype = torch.float16 if kv == "f16" else torch.uint8
    fill = 128 if kv == "int8" else 0
    k, v = (torch.full((blocks, BS, Hkv, D), fill, dtype=dtype, device="cuda") for _ in range(2))
    return k, v, torch.zeros((blocks, Hkv, 2, BS), device="cuda") if kv == "int8" else None


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("write", "rope"):
        T, Hkv, kv = case["T"], case["Hkv"], case.get("kv", "int8")
        blocks = (T if case["scattered"] else -(-T // BS)) + 7
        s["k"], s["v"] = _activations(g, T, Hkv, D), _activations(g, T, Hkv, D)
        s["slots"] = _slots(g, case, blocks)
        s["k_cache"], s["v_cache"], s["scales"] = _pool(g, kv, blocks, Hkv)
        s["k_out"], s["v_out"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        if op == "rope":
            R, axes = case["rotary"], case["axes"]
            s["q"] = _activations(g, T, case["Hq"], D)
            s["q_out"] = torch.empty_like(s["q"])
            s["inv_freq"] = (1e6 ** (-torch.arange(R // 2, dtype=torch.float64, device="cuda") * 2 / R)).float()
            # contexts reach far: positions up to 2^20; the further axes are rows and columns of an image
            base = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda")
            grid = torch.randint(0, 64, (axes, T), generator=g, device="cuda")
            grid[0] = 0
            s["positions"] = base + grid
            s["axis"] = torch.tensor(_axis_of(case), device="cuda")
            s["k_divisor"], s["v_divisor"] = (s[n].abs().max().float() * f / 448 for n, f in (("k", 1.42), ("v", 1.0)))
            s["k_scale"], s["v_scale"] = float(s["k_divisor"]), float(s["v_divisor"])
        return s
    lens = torch.tensor(_lengths(case), device="cuda")
    order = torch.randperm(case["B"], generator=g, device="cuda")
    lens = lens[order]
    B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
    pages = (lens + BS - 1) // BS
    blocks = sum(-(-n // BS) for n in _lengths(case)) + 9
    wide = -(-max(_lengths(case)) // BS)
    first = torch.cumsum(pages, 0) - pages
    page = torch.arange(wide, device="cuda")
    perm = torch.randperm(blocks, generator=g, device="cuda")
    used = page[None, :] < pages[:, None]
    table = torch.where(used, perm[(first[:, None] + page[None, :]).clamp(max=blocks - 1)], -1)
    s["block_tables"], s["context_lens"] = table.int().contiguous(), lens.int()
    s["max_len"] = max(_lengths(case))
    # what a quantising write leaves behind: codes that reach +-127 in every row, scales of the rows' magnitudes
    shape = (blocks, BS, Hkv, D)
    s["scales"] = torch.exp2(0.5 * _normal(g, blocks, Hkv, 2, BS)) * (3.0 / 127)
    for name in ("k_cache", "v_cache"):
        c = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16) * 42
        s[name] = (c.round().clamp(-127, 127) + 128).to(torch.uint8)
        s[name][..., 5] = 255
    if op == "decode":
        s["q"] = _normal(g, B, Hq, D).half()
    else:
        n = torch.tensor(_spread(case["n_lo"], case["n_hi"], B), device="cuda")[order]
        start = torch.cumsum(n, 0)
        s["query_start"] = torch.cat([start.new_zeros(1), start]).int()
        s["total"] = sum(_spread(case["n_lo"], case["n_hi"], B))
        s["max_new"] = max(_spread(case["n_lo"], case["n_hi"], B))
        s["q"] = _normal(g, s["total"], Hq, D).half()
    s["out"] = torch.empty_like(s["q"])
    s["softmax_scale"] = D ** -0.5
    s["workspace"] = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms
def _quantise(x):
    """Codes and scales of fp32 rows [..., D]."""
    scale = x.abs().amax(-1).clamp(min=SMALLEST) / 127
    return (torch.round(x / scale[..., None]).clamp(-127, 127) + 128).to(torch.uint8), scale


def _place(slots):
    return slots // BS, slots % BS


def _write_int8(s, k, v):
    block, row = _place(s["slots"])
    for which, (cache, x) in enumerate((("k_cache", k), ("v_cache", v))):
        codes, scale = _quantise(x)
        s[cache].flatten(0, 1)[s["slots"]] = codes
        s["scales"][block, :, which, row] = scale


def _read_int8(s):
    block, row = _place(s["slots"])
    back = []
    for which, cache in enumerate(("k_cache", "v_cache")):
        codes = s[cache].flatten(0, 1)[s["slots"]].float() - 128
        back.append((codes * s["scales"][block, :, which, row][..., None]).half())
    return back


def _rotate(x, cos, sin, pairs, rotary):
    x = x.float()
    r, rest = x[..., :rotary], x[..., rotary:]
    if pairs:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., :rotary // 2], r[..., rotary // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, rest), -1)


def _plain_rope(s, case):
    angle = s["positions"][s["axis"]].t().double() * s["inv_freq"].double()
    cos, sin = (f(angle).float()[:, None, :] for f in (torch.cos, torch.sin))
    q, k = (_rotate(s[n], cos, sin, case["pairs"], case["rotary"]) for n in ("q", "k"))
    if case["kv"] == "int8":
        _write_int8(s, k, s["v"].float())
        return [q.half(), *_read_int8(s), s["scales"]]
    if case["kv"] == "f16":
        k, v = k.half(), s["v"]
    else:
        k, v = ((x / divisor).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                for x, divisor in ((k, s["k_divisor"]), (s["v"].float(), s["v_divisor"])))
    s["k_cache"].flatten(0, 1)[s["slots"]] = k
    s["v_cache"].flatten(0, 1)[s["slots"]] = v
    return [q.half(), *(_values(s[n], case["kv"]) for n in ("k_cache", "v_cache"))]


def _values(cache, kv):
    return cache.view(torch.float8_e4m3fn) if kv == "fp8" else cache


def _context(s):
    """K and V of every sequence, gathered through its table: [B, KV heads, longest, D] fp32, and the lengths."""
    t = torch.arange(s["max_len"], device="cuda")
    block = s["block_tables"].long().clamp(min=0)[:, t // BS]
    for which, cache in enumerate(("k_cache", "v_cache")):
        x = s[cache][block, t % BS].float()
        x -= 128
        x *= s["scales"][block, :, which, t % BS][..., None]
        yield x.transpose(1, 2)


def _plain_attention(s, case):
    B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
    G = Hq // Hkv
    K, V = _context(s)
    lens = s["context_lens"].long()
    if case["op"] == "decode":
        n, start = 1, torch.arange(B, device="cuda")
        new = torch.ones_like(lens)
    else:
        n, start = s["max_new"], s["query_start"].long()[:-1]
        new = s["query_start"].long().diff()
    i = torch.arange(n, device="cuda")
    rows = (start[:, None] + i[None, :]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().view(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    last = (lens - new)[:, None] + i[None, :]                      # the position of every query
    x = torch.matmul(q, K.transpose(2, 3)).mul_(s["softmax_scale"]).view(B, Hkv, n, G, -1)
    hidden = torch.arange(s["max_len"], device="cuda")[None, None, :] > last[:, :, None]
    x.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    x -= x.amax(-1, keepdim=True)
    x.exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, Hkv, n * G, -1), V).view(B, Hkv, n, G, D) / total
    o = o.permute(0, 2, 1, 3, 4).reshape(B * n, Hq, D).half()
    if case["op"] == "decode":
        return o
    seq = torch.bucketize(torch.arange(s["total"], device="cuda"), s["query_start"].long()[1:], right=True)
    return o[seq * n + torch.arange(s["total"], device="cuda") - start[seq]]


# ------------------------------------------------------------------ the framework's calls
def _own_write(s, case):
    import paged_kv_decode_gqa_b200 as pkv
    if case["op"] == "write":
        pkv.paged_kv_cache_write_int8(s["k"], s["v"], s["k_cache"], s["v_cache"], s["scales"], s["slots"])
    else:
        more = {"kv_scales": s["scales"]} if case["kv"] == "int8" else {}
        if case["kv"] == "fp8":
            more = {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}
        pkv.paged_kv_rope_cache_write(
            s["q_out"], s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["positions"],
            s["inv_freq"], sections=_sections(case), interleaved=case["pairs"], cyclic_axes=case["cyclic"],
            kv_dtype=case["kv"], **more)
        if case["kv"] != "int8":
            return [s["q_out"], *(_values(s[n], case["kv"]) for n in ("k_cache", "v_cache"))]
    pkv.paged_kv_cache_read(s["k_out"], s["v_out"], s["k_cache"], s["v_cache"], s["slots"], kv_dtype="int8",
                            kv_scales=s["scales"])
    return ([] if case["op"] == "write" else [s["q_out"]]) + [s["k_out"], s["v_out"], s["scales"]]


def _own_attention(s, case):
    import paged_kv_decode_gqa_b200 as pkv
    if case["op"] == "decode":
        pkv.paged_gqa_decode_attention_int8(
            s["out"], s["q"], s["k_cache"], s["v_cache"], s["scales"], s["block_tables"], s["context_lens"],
            max_context_len=s["max_len"], softmax_scale=s["softmax_scale"], workspace=s["workspace"])
    else:
        pkv.paged_gqa_prefill_attention_int8(
            s["out"], s["q"], s["k_cache"], s["v_cache"], s["scales"], s["block_tables"], s["context_lens"],
            s["query_start"], max_query_len=s["max_new"], max_context_len=s["max_len"],
            softmax_scale=s["softmax_scale"], workspace=s["workspace"])
    return s["out"]


def run(state):
    case = state["case"]
    if case["op"] in ("decode", "chunk"):
        return _own_attention(state, case) if own else _plain_attention(state, case)
    if own:
        return _own_write(state, case)
    if case["op"] == "rope":
        return _plain_rope(state, case)
    _write_int8(state, state["k"].float(), state["v"].float())
    return [*_read_int8(state), state["scales"]]


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_rows(x):
    """Values and scales that quantised rows stand for."""
    scale = x.abs().max(-1).values.clamp(min=SMALLEST) / 127
    return torch.round(x / scale.unsqueeze(-1)).clamp(-127, 127) * scale.unsqueeze(-1), scale


def _exact_scales(s, k_scale, v_scale):
    pool = torch.zeros(s["scales"].shape, dtype=torch.float64, device="cuda")
    pool[s["slots"] // BS, :, 0, s["slots"] % BS] = k_scale
    pool[s["slots"] // BS, :, 1, s["slots"] % BS] = v_scale
    return pool


def _exact_rope(s, case):
    half = case["rotary"] // 2
    phase = torch.stack([s["positions"][a].double() * s["inv_freq"][j].double()
                         for j, a in enumerate(_axis_of(case))], -1)
    turn = torch.polar(torch.ones_like(phase), phase)[:, None, :]
    rotated = []
    for x in (s["q"].double(), s["k"].double()):
        first = slice(0, 2 * half, 2) if case["pairs"] else slice(0, half)
        second = slice(1, 2 * half, 2) if case["pairs"] else slice(half, 2 * half)
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
        x[..., first], x[..., second] = z.real, z.imag
        rotated.append(x)
    q, k = rotated
    v = s["v"].double()
    if case["kv"] == "int8":
        (k, ks), (v, vs) = _exact_rows(k), _exact_rows(v)
        return [q, k, v, _exact_scales(s, ks, vs)]
    if case["kv"] == "fp8":      # codes depend on the roundings of the quotient: the type's bound holds them
        return [q, None, None]
    pools = []
    for x in (k, v):
        pool = torch.zeros(s["k_cache"].shape, dtype=torch.float64, device="cuda")
        pool.view(-1, *pool.shape[2:])[s["slots"]] = x
        pools.append(pool)
    return [q, *pools]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s, case)
    if case["op"] == "write":
        (k, ks), (v, vs) = _exact_rows(s["k"].double()), _exact_rows(s["v"].double())
        return [k, v, _exact_scales(s, ks, vs)]
    Hq, Hkv = case["Hq"], case["Hkv"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lens = s["context_lens"].tolist()
    ends = s["query_start"].tolist() if case["op"] == "chunk" else list(range(len(lens) + 1))
    for b, L in enumerate(lens):
        blocks = s["block_tables"][b, :-(-L // BS)].long()
        kv = []
        for which, name in enumerate(("k_cache", "v_cache")):
            codes = s[name][blocks].double() - 128                             # [pages, 16, KV heads, D]
            scale = s["scales"][blocks][:, :, which, :].double().permute(0, 2, 1)
            kv.append((codes * scale.unsqueeze(-1)).reshape(-1, Hkv, D)[:L])
        lo, hi = ends[b], ends[b + 1]
        n = hi - lo
        limit = torch.arange(L - n, L, device="cuda")
        seen = torch.arange(L, device="cuda")[None, :] <= limit[:, None]
        for h in range(Hq):
            g = h // (Hq // Hkv)
            logits = s["q"][lo:hi, h].double() @ kv[0][:, g].t() * s["softmax_scale"]
            p = torch.softmax(logits.masked_fill(~seen, -math.inf), -1)
            out[lo:hi, h] = p @ kv[1][:, g]
    return out

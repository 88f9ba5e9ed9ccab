"""Workloads of the decoder-cache operators: rotary positions, the quantised paged key-value cache (write and
read back), and the attention of one new token over it.

Each case runs one operator, either through this package's entry points (``own``) or in its plain form of
elementary torch operations.  Sizes are the range a serving process sees: single steps of one to a few hundred
sequences, prompt chunks of some thousands of tokens, contexts from one token to 131072, head widths 64 to 256,
one to many query heads per key-value head.
"""
import math
import random

import torch

own = False

DEV = "cuda"
NV_GLOBAL = (6.0 / 2688.0, 5.0 / 2688.0)  # second-level scales of K and V, as a calibration run would give


# ---- the cases -----------------------------------------------------------------------------------------------

def listed():
    return [
        # a process's start: the table of a short model, and of a 4096-token model stretched to 131072 positions
        dict(name="table_short", op="table", P=4096, rot=64, base=10000.0, scaling=0, factor=1.0, context=0, low=0.0,
             high=0.0, amplitude=1.0),
        dict(name="table_long", op="table", P=131072, rot=128, base=500000.0, scaling=3, factor=32.0, context=4096,
             low=1.0, high=32.0, amplitude=1.3465735902799727),
        # q of one decoding step of 64 sequences; latency
        dict(name="rope_step", op="rope", T=64, H=64, D=128, rot=128, interleaved=0, P=32768, gap=2048),
        # q of a long prompt chunk, part of each head, pairs side by side, an odd number of tokens
        dict(name="rope_prompt", op="rope", T=8191, H=32, D=192, rot=64, interleaved=1, P=131072, gap=0),
        # one decoding step of 64 sequences: q and k rotated, k and v written to 64 scattered places
        dict(name="cache_step_e4m3", op="cache", dtype="e4m3", T=64, R=64, Hkv=8, Hq=64, D=128, page=16, rot=128,
             interleaved=0, P=32768),
        # a prompt chunk of 2048 tokens behind a 30000-token prefix, all of it read back for the chunk's attention
        dict(name="cache_prefix_e4m3", op="cache", dtype="e4m3", T=2048, R=32048, Hkv=8, Hq=0, D=128, page=64, rot=0,
             interleaved=0, P=0),
        # a whole prompt of odd length written with its positions, wide heads, and read back
        dict(name="cache_prompt_nvfp4", op="cache", dtype="nvfp4", T=8191, R=8191, Hkv=4, Hq=16, D=256, page=32,
             rot=128, interleaved=1, P=16384),
        # one sequence, the latency of a single user
        dict(name="attn_one_bf16", op="attn", dtype="bf16", B=1, longest=4097, spread=1.0, Hq=32, Hkv=8, D=128,
             page=16, window=0),
        # a serving batch of ragged lengths
        dict(name="attn_batch_e4m3", op="attn", dtype="e4m3", B=64, longest=8192, spread=32.0, Hq=64, Hkv=8, D=128,
             page=64, window=0),
        # long documents
        dict(name="attn_long_nvfp4", op="attn", dtype="nvfp4", B=8, longest=131072, spread=1.5, Hq=64, Hkv=8, D=128,
             page=64, window=0),
        # many sequences under a sliding window, one key-value head per query head, some slots of the batch empty
        dict(name="attn_window_bf16", op="attn", dtype="bf16", B=125, longest=5000, spread=64.0, Hq=16, Hkv=16, D=64,
             page=32, window=1024),
        # wide heads, 16 query heads to a key-value head
        dict(name="attn_wide_e4m3", op="attn", dtype="e4m3", B=33, longest=16384, spread=8.0, Hq=32, Hkv=2, D=256,
             page=128, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["table", "rope", "cache", "cache", "attn", "attn", "attn"])
    if op == "table":
        return dict(op=op, P=_log(rng, 1, 131072), rot=2 * rng.randint(8, 64), base=rng.choice([10000.0, 500000.0, 1e6]),
                    scaling=rng.randint(0, 3), factor=rng.uniform(2.0, 32.0), context=rng.choice([2048, 4096, 8192]),
                    low=1.0, high=rng.choice([4.0, 32.0]), amplitude=rng.uniform(1.0, 1.4))
    D = rng.choice([64, 128, 128, 192, 256])
    if op == "rope":
        H = rng.choice([1, 4, 8, 32, 64])
        T = _log(rng, 1, 8191 * 32 * 192 // (H * D))
        return dict(op=op, T=min(T, 65536), H=H, D=D, rot=2 * rng.randint(4, D // 2), interleaved=rng.randint(0, 1),
                    P=131072, gap=rng.choice([0, 64, 2048]))
    dtype, page = rng.choice(["bf16", "e4m3", "nvfp4"]), rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "cache":
        R = _log(rng, 1, 30000 * 8 * 128 // (Hkv * D))
        T = rng.choice([R, max(1, R // 8), _log(rng, 1, R)])
        rot = rng.choice([0, D, 64, 32])
        return dict(op=op, dtype=dtype, T=T, R=R, Hkv=Hkv, Hq=Hkv * rng.choice([0, 1, 4, 8]) if rot else 0, D=D,
                    page=page, rot=rot, interleaved=rng.randint(0, 1), P=max(R + 1000, 4096))
    G = rng.choice([1, 2, 4, 5, 7, 8, 12, 16])
    B = _log(rng, 1, 256)
    longest = _log(rng, 1, min(131072, (64 * 8192 * 8 * 128) // (B * Hkv * D)))
    return dict(op=op, dtype=dtype, B=B, longest=longest, spread=rng.choice([1.0, 4.0, 64.0]), Hq=G * Hkv, Hkv=Hkv, D=D,
                page=page, window=rng.choice([0, 0, 0, 1, 100, 4096]))


def _lengths(c):
    """Tokens of each sequence: the longest, one that is empty in larger batches, the others log-uniform between."""
    r = random.Random(c["B"] * 1000003 + c["longest"])
    n = [max(1, int(c["longest"] / math.exp(r.uniform(0.0, math.log(c["spread"]))))) for _ in range(c["B"])]
    n[r.randrange(c["B"])] = c["longest"]
    if c["B"] > 16:
        n[1 if n[0] == c["longest"] else 0] = 0
    return n


def _held_bytes(dtype, D):
    """Bytes of one token's key or value of one head in the cache."""
    return {"bf16": 2 * D, "e4m3": D + 4, "nvfp4": D // 2 + D // 16}[dtype]


def work(c):
    if c["op"] == "table":
        return dict(bytes=4.0 * c["P"] * c["rot"], flops=2.0 * c["P"] * c["rot"])
    if c["op"] == "rope":
        n = c["T"] * c["H"]
        return dict(bytes=4.0 * n * c["D"] + c["T"] * (4.0 * c["rot"] + 4), flops=3.0 * n * c["rot"])
    if c["op"] == "cache":
        kv = 2 * c["Hkv"] * c["D"]
        held = 2 * c["Hkv"] * _held_bytes(c["dtype"], c["D"])
        b = c["T"] * (2.0 * kv + held + 8) + c["R"] * (held + 2.0 * kv + 8)
        if c["rot"]:
            b += c["T"] * (4.0 * c["rot"] + 4 + 4.0 * c["Hq"] * c["D"])
        return dict(bytes=b, flops=2.0 * (c["T"] + c["R"]) * kv + 3.0 * c["T"] * (c["Hq"] + c["Hkv"]) * c["rot"])
    seen = sum(min(n, c["window"]) if c["window"] else n for n in _lengths(c))
    return dict(bytes=seen * 2.0 * c["Hkv"] * _held_bytes(c["dtype"], c["D"]) + 4.0 * c["B"] * c["Hq"] * c["D"]
                + 4.0 * c["B"] * c["Hq"], flops=4.0 * seen * c["Hq"] * c["D"])


# ---- the inputs ----------------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(1000 + seed)


def _normal(shape, g, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(torch.bfloat16)


def _freqs64(c):
    """The rotation's frequencies (radians per position) in 64 bits."""
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device=DEV)
    f = c["base"] ** (-2.0 * i / c["rot"])
    if c["scaling"] == 1:
        f = f / c["factor"]
    if c["scaling"] == 2:
        y = ((c["context"] * f / (2 * math.pi) - c["low"]) / (c["high"] - c["low"])).clamp(0, 1)
        f = f * (y + (1 - y) / c["factor"])
    if c["scaling"] == 3:
        at = lambda n: c["rot"] * math.log(c["context"] / (2 * math.pi * n)) / (2 * math.log(c["base"]))  # noqa: E731
        first, last = max(0, math.floor(at(c["high"]))), min(c["rot"] - 1, math.ceil(at(c["low"])))
        y = 1 - ((i - first) / max(last - first, 0.001)).clamp(0, 1)
        f = f * (y + (1 - y) / c["factor"])
    return f


def _table(rot, P):
    """The fp32 table a program keeps: a plain rotation of base 10000."""
    f = _freqs64(dict(rot=rot, base=10000.0, scaling=0))
    a = torch.arange(P, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _cache_inputs(c, seed):
    """New and earlier keys and values, their slots and positions."""
    g = _gen(seed)
    T, R, Hq, Hkv, D, page = (c[x] for x in ("T", "R", "Hq", "Hkv", "D", "page"))
    pages = -(-R // page) + 3
    if R == T and T <= 256:  # one token of each of T sequences, at places all over the cache
        pages = T + 3
        slots = torch.randperm(pages, generator=g, device=DEV)[:T] * page
        slots = slots + torch.randint(0, page, (T,), generator=g, device=DEV)
    else:                    # one sequence, its pages in any order
        order = torch.randperm(pages, generator=g, device=DEV)
        at = torch.arange(R, device=DEV)
        slots = order[at // page] * page + at % page
    s = dict(c, pages=pages, slots=slots.to(torch.int64), new_slots=slots[R - T:].to(torch.int64).contiguous())
    s["old"] = (_normal((R - T, Hkv, D), g), _normal((R - T, Hkv, D), g, 0.7))
    s["qkv"] = _normal((T, Hq + 2 * Hkv, D), g)  # one projection's output: q heads, k heads, v heads
    s["glob"] = torch.tensor(NV_GLOBAL, device=DEV)
    if c["rot"]:
        first = int(torch.randint(0, c["P"] - R, (1,), generator=g, device=DEV))
        s["pos"] = (torch.arange(R - T, R, device=DEV) + first).to(torch.int32)
        s["table"] = _table(c["rot"], c["P"])
    return s


def _attn_inputs(c, seed):
    g = _gen(seed)
    n = _lengths(c)
    page, most = c["page"], -(-c["longest"] // c["page"])
    need = [-(-x // page) for x in n]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    first = torch.tensor([sum(need[:b]) for b in range(c["B"])], device=DEV)
    have = torch.tensor(need, device=DEV)
    j = torch.arange(most, device=DEV)
    at = torch.where(j < have[:, None], first[:, None] + j, 0)
    table = torch.where(j < have[:, None], order[at], 0).to(torch.int32).contiguous()
    return dict(c, pages=pages, table=table, lens=torch.tensor(n, dtype=torch.int32, device=DEV), most=most,
                q=_normal((c["B"], c["Hq"], c["D"]), g, 2.0), glob=torch.tensor(NV_GLOBAL, device=DEV),
                k=_normal((pages * page, c["Hkv"], c["D"]), g), v=_normal((pages * page, c["Hkv"], c["D"]), g))


def _pages(s, dtype):
    """The pages of this package's cache for a state's sizes, empty."""
    import quantized_gemm_02_b200 as hq
    code = {"bf16": hq.HQ_BF16, "e4m3": hq.HQ_E4M3, "nvfp4": hq.HQ_NVFP4}[dtype]
    kv = hq.KVDesc(dtype=code, heads=s["Hkv"], head_dim=s["D"], page_size=s["page"])
    return kv, torch.zeros(s["pages"] * hq.hq_kv_page_bytes(kv), dtype=torch.uint8, device=DEV)


def prepare(c, seed):
    if c["op"] == "table":
        s = dict(c)
        # the stretched range starts elsewhere for another seed: another base
        s["base"] = c["base"] * (1.0 + (seed % 97) / 1024.0)
        if own:
            import quantized_gemm_02_b200 as hq
            s["rope"] = hq.RopeDesc(rot_dim=s["rot"], scaling=s["scaling"], context=s["context"], base=s["base"],
                                    factor=s["factor"], low=s["low"], high=s["high"], amplitude=s["amplitude"])
            s["out"] = torch.empty(s["P"], s["rot"], device=DEV)
        return s
    if c["op"] == "rope":
        g = _gen(seed)
        s = dict(c, table=_table(c["rot"], c["P"]))
        row = c["H"] * c["D"] + c["gap"]  # the tensor is the first part of a wider projection's output
        s["x"] = _normal((c["T"], row), g)[:, :c["H"] * c["D"]].unflatten(1, (c["H"], c["D"]))
        if c["T"] <= 256:  # a step: each sequence at a place of its own
            s["pos"] = torch.randint(0, c["P"], (c["T"],), generator=g, device=DEV).to(torch.int32)
        else:
            first = int(torch.randint(0, c["P"] - c["T"], (1,), generator=g, device=DEV))
            s["pos"] = (torch.arange(c["T"], device=DEV) + first).to(torch.int32)
        if own:
            import quantized_gemm_02_b200 as hq
            s["rope"] = hq.RopeDesc(rot_dim=c["rot"], interleaved=c["interleaved"])
            s["out"] = torch.empty(c["T"], c["H"], c["D"], dtype=torch.bfloat16, device=DEV)
        return s
    if c["op"] == "cache":
        s = _cache_inputs(c, seed)
        n = c["R"] - c["T"]
        if own:
            import quantized_gemm_02_b200 as hq
            s["kv"], s["buf"] = _pages(s, c["dtype"])
            s["rope"] = hq.RopeDesc(rot_dim=c["rot"], interleaved=c["interleaved"])
            s["g"] = s["glob"] if c["dtype"] == "nvfp4" else None
            row = c["Hkv"] * c["D"]
            hq.hq_kv_write(s["kv"], n, s["old"][0], row, s["old"][1], row, s["slots"][:n].contiguous(), s["g"],
                           s["pages"], s["buf"])
            s["out"] = [torch.empty(c["R"], c["Hkv"], c["D"], dtype=torch.bfloat16, device=DEV) for _ in range(2)]
            s["qout"] = torch.empty(c["T"], c["Hq"], c["D"], dtype=torch.bfloat16, device=DEV)
        else:
            s["held"] = [_empty(c["dtype"], s["pages"] * c["page"], c["Hkv"], c["D"]) for _ in range(2)]
            for i in range(2):
                _store(s["held"][i], s["slots"][:n], _quantise(s["old"][i].float(), c["dtype"], s["glob"][i]))
        del s["old"]
        return s
    s = _attn_inputs(c, seed)
    k, v = s.pop("k"), s.pop("v")
    s["scale"] = 1.0 / math.sqrt(c["D"])
    if own:
        import quantized_gemm_02_b200 as hq
        s["kv"], s["buf"] = _pages(s, c["dtype"])
        s["g"] = s["glob"] if c["dtype"] == "nvfp4" else None
        row = c["Hkv"] * c["D"]
        hq.hq_kv_write(s["kv"], k.shape[0], k, row, v, row, torch.arange(k.shape[0], device=DEV), s["g"], s["pages"],
                       s["buf"])
        s["out"] = torch.empty(c["B"], c["Hq"], c["D"], dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(c["B"], c["Hq"], dtype=torch.float32, device=DEV)
        s["wsb"] = hq.hq_paged_attn_workspace_bytes(s["kv"], c["B"], c["Hq"])
        s["ws"] = torch.zeros(s["wsb"], dtype=torch.uint8, device=DEV)
    else:
        s["held"] = [_quantise(x, c["dtype"], s["glob"][i]) for i, x in enumerate((k, v))]
    return s


# ---- the plain forms -----------------------------------------------------------------------------------------
# A held tensor is (codes, scales): bf16 values; E4M3 values with an fp32 scale per token and head; or E2M1 values
# (kept in an E4M3 tensor, which holds them exactly) with an E4M3 scale per 16 channels and one fp32 scale.

def _empty(dtype, slots, H, D):
    f8 = lambda *d: torch.zeros(*d, device=DEV).to(torch.float8_e4m3fn)  # noqa: E731
    if dtype == "bf16":
        return [torch.zeros(slots, H, D, dtype=torch.bfloat16, device=DEV)]
    if dtype == "e4m3":
        return [f8(slots, H, D), torch.zeros(slots, H, 1, device=DEV)]
    return [f8(slots, H, D), f8(slots, H, D // 16)]


def _e2m1(x):
    """fp32 rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to even), kept in an E4M3 tensor."""
    a = x.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp(max=6.0), x).to(torch.float8_e4m3fn)


def _quantise(x, dtype, g):
    if dtype == "bf16":
        return [x.to(torch.bfloat16)]
    x = x.float()
    # divisors are tensors: a division by a Python number is a product with its rounded reciprocal
    if dtype == "e4m3":
        amax = x.abs().amax(-1, keepdim=True)
        s = torch.where(amax == 0, 1.0, amax / torch.full_like(amax, 448.0))
        return [(x / s).clamp(-448, 448).to(torch.float8_e4m3fn), s]
    b = x.unflatten(-1, (-1, 16))
    amax = b.abs().amax(-1)
    sb = ((amax / torch.full_like(amax, 6.0)) / g).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = (sb.float() * g).unsqueeze(-1)
    return [_e2m1(torch.where(d == 0, 0.0, b / d).flatten(-2)), sb]


def _bits(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _store(held, slots, new):
    for h, x in zip(held, new):
        _bits(h)[slots] = _bits(x)


def _fetch(held, slots):
    return [_bits(h)[slots].view(h.dtype) for h in held]


def _values(held, dtype, g):
    """What is held, in fp32."""
    x = held[0].float()
    if dtype == "e4m3":
        x = x * held[1]
    if dtype == "nvfp4":
        x = (x.unflatten(-1, (-1, 16)) * held[1].float().unsqueeze(-1)).flatten(-2) * g
    return x


def _rotate(x, cos, sin, rot, interleaved):
    """x [T, H, D] fp32 with its first `rot` channels rotated by cos, sin [T, rot / 2]."""
    c, s = cos[:, None], sin[:, None]
    a, b = (x[..., :rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * c - b * s, b * c + a * s
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _plain_table(s):
    a = torch.arange(s["P"], dtype=torch.float64, device=DEV)[:, None] * _freqs64(s)
    return (torch.cat([a.cos(), a.sin()], 1) * s["amplitude"]).float()


def _plain_rope(s, x):
    t = s["table"][s["pos"].long()]
    h = s["rot"] // 2
    return _rotate(x.float(), t[:, :h], t[:, h:], s["rot"], s["interleaved"])


def _plain_cache(s):
    Hq, Hkv = s["Hq"], s["Hkv"]
    q, k, v = s["qkv"].split([Hq, Hkv, Hkv], 1)
    out = []
    if s["rot"]:
        k = _plain_rope(s, k)
        out = [_plain_rope(s, q).to(torch.bfloat16)] if Hq else []
    for i, x in enumerate((k.float(), v.float())):
        _store(s["held"][i], s["new_slots"], _quantise(x, s["dtype"], s["glob"][i]))
    return out + [_values(_fetch(s["held"][i], s["slots"]), s["dtype"], s["glob"][i]).to(torch.bfloat16)
                  for i in range(2)]


def _plain_attn(s):
    B, Hq, Hkv, D, page = s["B"], s["Hq"], s["Hkv"], s["D"], s["page"]
    at = torch.arange(s["most"] * page, device=DEV)
    slots = s["table"].long()[:, at // page] * page + at % page                       # [B, L]
    n = s["lens"][:, None]
    seen = at < n
    if s["window"]:
        seen = seen & (at >= n - s["window"])
    k, v = (_values(_fetch(h, slots), s["dtype"], s["glob"][i]).transpose(1, 2) for i, h in enumerate(s["held"]))
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    x = torch.where(seen[:, None, None], q @ k.transpose(2, 3) * s["scale"], -math.inf)  # [B, Hkv, G, L]
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = (x - m).exp()
    l = p.sum(-1, keepdim=True)
    o = (p @ v) / l.clamp(min=1e-30)
    return [o.reshape(B, Hq, D).to(torch.bfloat16), (m + l.log()).reshape(B, Hq)]


# ---- one pass ------------------------------------------------------------------------------------------------

def run(s):
    if not own:
        return {"table": _plain_table, "cache": _plain_cache, "attn": _plain_attn,
                "rope": lambda s: _plain_rope(s, s["x"]).to(torch.bfloat16)}[s["op"]](s)
    import quantized_gemm_02_b200 as hq
    if s["op"] == "table":
        hq.hq_rope_table(s["rope"], s["P"], s["out"])
        return s["out"]
    if s["op"] == "rope":
        x, o = s["x"], s["out"]
        hq.hq_rope(s["rope"], s["T"], s["H"], s["D"], x, x.stride(0), x.stride(1), s["pos"], s["table"], s["P"], o,
                   o.stride(0), o.stride(1))
        return o
    if s["op"] == "cache":
        Hq, Hkv, T, kv = s["Hq"], s["Hkv"], s["T"], s["kv"]
        q, k, v = s["qkv"].split([Hq, Hkv, Hkv], 1)
        row, okv = s["qkv"].stride(0), s["out"]
        if s["rot"]:
            hq.hq_rope_kv_write(s["rope"], kv, T, Hq, q if Hq else None, row, s["qout"] if Hq else None, Hq * s["D"],
                                k, row, v, row, s["pos"], s["table"], s["P"], s["new_slots"], s["g"], s["pages"],
                                s["buf"])
        else:
            hq.hq_kv_write(kv, T, k, row, v, row, s["new_slots"], s["g"], s["pages"], s["buf"])
        hq.hq_kv_read(kv, s["R"], s["slots"], s["g"], s["pages"], s["buf"], okv[0], okv[0].stride(0), okv[1],
                      okv[1].stride(0))
        return ([s["qout"]] if s["rot"] and Hq else []) + okv
    hq.hq_paged_attn(s["kv"], s["B"], s["Hq"], s["q"], s["q"].stride(0), s["g"], s["pages"], s["buf"], s["table"],
                     s["most"], s["lens"], s["scale"], s["window"], s["out"], s["out"].stride(0), s["lse"], s["ws"],
                     s["wsb"])
    return [s["out"], s["lse"]]


# ---- the definitions in 64 bits ------------------------------------------------------------------------------

def _grid64(x, mantissa, least, largest):
    """x rounded to the nearest float of `mantissa` bits with smallest exponent `least`, ties to even."""
    a = x.abs().clamp(max=largest)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** least)))
    step = torch.exp2(e - mantissa)
    return torch.copysign((torch.round(a / step) * step).clamp(max=largest), x)


def _held64(x, dtype, g):
    """What the cache holds of x.  The recipes are defined by steps rounded to 32 bits, which decide between two
    neighbouring codes; the grids and the values are in 64."""
    if dtype == "bf16":
        return x
    x, f, c = x.float(), torch.float64, lambda v: torch.tensor(v, device=DEV)  # noqa: E731
    if dtype == "e4m3":
        s = x.abs().amax(-1, keepdim=True) / c(448.0)
        s = torch.where(s == 0, torch.ones_like(s), s)
        return _grid64((x / s).to(f), 3, -6, 448.0) * s.to(f)
    b = x.reshape(x.shape[:-1] + (x.shape[-1] // 16, 16))
    sb = _grid64((b.abs().amax(-1, keepdim=True) / c(6.0) / g).to(f), 3, -6, 448.0)
    d = sb.float() * g
    q = _grid64((b / torch.where(d == 0, torch.ones_like(d), d)).to(f), 1, 0, 6.0)
    return (q * sb * g.to(f)).reshape(x.shape)


def _turn64(x, pos, c):
    """The rotation as a product of complex numbers."""
    h = c["rot"] // 2
    a = pos.double()[:, None] * torch.exp(torch.arange(h, device=DEV, dtype=torch.float64) * (-math.log(10000.0) / h))
    y = x.double().clone()
    if c["interleaved"]:
        z = torch.view_as_complex(y[..., :c["rot"]].reshape(*x.shape[:2], h, 2).contiguous())
    else:
        z = torch.complex(y[..., :h].contiguous(), y[..., h:2 * h].contiguous())
    z = z * torch.polar(torch.ones_like(a), a)[:, None]
    y[..., :c["rot"]] = torch.view_as_real(z).flatten(-2) if c["interleaved"] else torch.cat([z.real, z.imag], -1)
    return y


def exact(c, seed):
    if c["op"] == "table":
        s = prepare(c, seed)
        a = torch.outer(torch.arange(s["P"], dtype=torch.float64, device=DEV), _freqs64(s))
        z = torch.polar(torch.full_like(a, s["amplitude"]), a)
        return torch.cat([z.real, z.imag], 1)
    if c["op"] == "rope":
        s = prepare(c, seed)
        return _turn64(s["x"], s["pos"], c)
    if c["op"] == "cache":
        s = _cache_inputs(c, seed)
        q, k, v = s["qkv"][:, :c["Hq"]], s["qkv"][:, c["Hq"]:c["Hq"] + c["Hkv"]], s["qkv"][:, c["Hq"] + c["Hkv"]:]
        out = []
        if c["rot"]:
            k = _turn64(k, s["pos"], c)
            out = [_turn64(q, s["pos"], c)] if c["Hq"] else []
        k, v = (torch.cat([o.double(), x.double()]) for o, x in zip(s["old"], (k, v)))
        return out + [_held64(x, c["dtype"], s["glob"][i]) for i, x in enumerate((k, v))]
    s = _attn_inputs(c, seed)
    # the cache's content is an input: what is held, by the recipe
    held = [_quantise(s.pop(x), c["dtype"], s["glob"][i]) for i, x in enumerate(("k", "v"))]
    B, Hq, Hkv, D, page = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"]
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(_lengths(c)):
        if not n:
            continue
        j = torch.arange(max(0, n - c["window"]) if c["window"] else 0, n, device=DEV)
        slots = s["table"][b][j // page].long() * page + j % page
        k, v = ([t[0].double(), *[u.double() for u in t[1:]]] for t in (_fetch(h, slots) for h in held))
        if c["dtype"] == "e4m3":
            k, v = [k[0] * k[1]], [v[0] * v[1]]
        if c["dtype"] == "nvfp4":
            k, v = ([t[0] * t[1].repeat_interleave(16, -1) * float(s["glob"][i])] for i, t in enumerate((k, v)))
        x = torch.einsum("hgd,lhd->hgl", s["q"][b].double().view(Hkv, -1, D), k[0]) / math.sqrt(D)
        lse[b] = torch.logsumexp(x, -1).reshape(-1)
        out[b] = torch.einsum("hgl,lhd->hgd", torch.softmax(x, -1), v[0]).reshape(Hq, D)
    return [out, lse]

"""Attention over the paged cache where a warp walks many steps, against 64-bit computations on the device.

The units of all sequences and kv heads form one line that is cut over some 450 to 2100 warps; the cases here are
longer than that, so that warps go from page to page, from item to item and around their rings."""
import math
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import quantized_gemm_02_b200 as hq

pytestmark = pytest.mark.gpu

DT = {"bf16": hq.HQ_BF16, "e4m3": hq.HQ_E4M3, "nvfp4": hq.HQ_NVFP4}
GLOB = (6.0 / 2688.0, 5.0 / 2688.0)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * scale).to(torch.bfloat16)


def held64(x, dtype, g):
    """What a cache holds of bf16 x [.., D], in 64 bits; the recipes' steps are fp32 divisions by tensors."""
    if dtype == "bf16":
        return x.double()
    x, c = x.float(), lambda v: torch.tensor(v, device="cuda")  # noqa: E731
    if dtype == "e4m3":
        s = x.abs().amax(-1, keepdim=True) / c(448.0)
        s = torch.where(s == 0, torch.ones_like(s), s)
        return (x / s).clamp(-448, 448).to(torch.float8_e4m3fn).double() * s.double()
    b = x.unflatten(-1, (-1, 16))
    sb = (b.abs().amax(-1, keepdim=True) / c(6.0) / c(g)).clamp(max=448).to(torch.float8_e4m3fn).float()
    d = sb * c(g)
    y = torch.where(d == 0, torch.zeros_like(b), b / d)
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    e = torch.copysign((torch.round(a / step) * step).clamp(max=6), y)
    return (e.double() * sb.double() * c(g).double()).flatten(-2)


class Paged:
    """A cache whose sequences b hold tokens [first[b], lens[b]) on pages in random order; what else is in the pages
    is NaN codes, and the table's entries of pages that are not held are out of range."""

    def __init__(self, dtype, H, D, page, lens, first, seed, make=None):
        self.dtype, self.H, self.D, self.page, self.lens, self.first = dtype, H, D, page, lens, first
        spans = [(f // page, -(-n // page)) if n > f else (0, 0) for f, n in zip(first, lens)]
        used = sum(e - s for s, e in spans)
        self.pages = used + 1
        self.kv = hq.KVDesc(dtype=DT[dtype], heads=H, head_dim=D, page_size=page)
        self.buf = torch.full((self.pages * hq.hq_kv_page_bytes(self.kv),), 0xFF, dtype=torch.uint8, device="cuda")
        self.glob = torch.tensor(GLOB, device="cuda") if dtype == "nvfp4" else None
        perm = torch.randperm(self.pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        table = torch.empty(len(lens), max(max(e for _, e in spans), 1), dtype=torch.int32)
        table[:, ::2], table[:, 1::2] = -1, 1 << 30
        at, seqs, toks = 0, [], []
        for b, (s, e) in enumerate(spans):
            table[b, s:e] = perm[at:at + e - s]
            at += e - s
            toks.append(torch.arange(first[b], max(lens[b], first[b])))
            seqs.append(torch.full_like(toks[-1], b))
        seqs, toks = torch.cat(seqs), torch.cat(toks)
        slots = (table[seqs, toks // page].long() * page + toks % page).cuda()
        n = slots.numel()
        self.k, self.v = make(seqs.cuda(), toks.cuda()) if make else (normal((n, H, D), seed + 1), normal((n, H, D), seed + 2))
        hq.hq_kv_write(self.kv, n, self.k, H * D, self.v, H * D, slots, self.glob, self.pages, self.buf)
        self.table, self.ld = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.ends = [0]
        for f, m in zip(first, lens):
            self.ends.append(self.ends[-1] + max(m - f, 0))

    def call(self, q, scale, window=0, ws=None):
        B, Hq, D = q.shape
        need = hq.hq_paged_attn_workspace_bytes(self.kv, B, Hq)
        ws = torch.zeros(need, dtype=torch.uint8, device="cuda") if ws is None else ws
        out = torch.full((B, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((B, Hq), 7.0, device="cuda")
        hq.hq_paged_attn(self.kv, B, Hq, q, q.stride(0), self.glob, self.pages, self.buf, self.table, self.table.shape[1],
                         self.ld, scale, window, out, out.stride(0), lse, ws, ws.numel())
        return out, lse

    def check(self, q, scale, window=0):
        """Calls twice (the results are the same bit for bit) and compares with the formula."""
        ws = torch.zeros(hq.hq_paged_attn_workspace_bytes(self.kv, q.shape[0], q.shape[1]), dtype=torch.uint8, device="cuda")
        out, lse = self.call(q, scale, window, ws)
        again = self.call(q, scale, window, ws)
        assert hq.hq_device_error() == 0
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
        G = q.shape[1] // self.H
        worst = []
        for b, n in enumerate(self.lens):
            first = max(n - window, 0) if window else 0
            assert n == 0 or first >= self.first[b]
            if n == 0:
                assert torch.all(out[b] == 0) and torch.all(lse[b] == -math.inf)
                continue
            rows = slice(self.ends[b] + first - self.first[b], self.ends[b + 1])
            k, v = held64(self.k[rows], self.dtype, GLOB[0]), held64(self.v[rows], self.dtype, GLOB[1])
            for h in range(self.H):
                worst.append(self._compare(q[b, h * G:(h + 1) * G].double(), k[:, h], v[:, h], scale,
                                           out[b, h * G:(h + 1) * G].double(), lse[b, h * G:(h + 1) * G].double()))
        w = torch.stack(worst).amax(0).tolist()
        assert w[0] <= 1 and w[1] <= 1, w

    def _compare(self, q, k, v, scale, out, lse):
        """Errors of out and lse, each as a share of its bound."""
        x = scale * (q @ k.T)
        wl = torch.logsumexp(x, -1)
        p = torch.exp(x - wl[:, None])
        want, mag = p @ v, p @ v.abs()
        # A score: at most 32 fp32 accumulations, each off by up to 2^-23 of sum |q k| (a tensor core may truncate), and a
        # handful of fp32 products and sums: 2^-18 of the largest sum |q k|.
        dx = 2.0**-18 * abs(scale) * (q.abs() @ k.abs().T).amax(-1)
        # Output: that much of each weight, twice (numerator and denominator); 2^-11 for weights in fp16 and as much for
        # exp and the sums; its own rounding to bf16, 2^-8.  fp16 weights end at a spacing of 2^-24 where the largest one
        # (E4M3: times its token's scale) is at least 2^10: 2^-35 of that from every token.
        small = torch.zeros_like(wl)
        if self.dtype != "bf16":
            top = v.abs().max() if self.dtype == "nvfp4" else (p * v.abs().amax(-1)).amax(-1)
            small = k.shape[0] * 2.0**-35 * top * torch.ones_like(wl)
        tol = 2.0**-8 * want.abs() + (2.0**-10 + 2 * dx[:, None]) * mag + small[:, None] + 1e-37
        ltol = 2.0**-20 * (1 + wl.abs()) + dx
        return torch.stack([((out - want).abs() / tol).max(), ((lse - wl).abs() / ltol).max()]).nan_to_num(nan=math.inf)


FORMS = [("nvfp4", 64), ("nvfp4", 128), ("nvfp4", 192), ("nvfp4", 256), ("e4m3", 64), ("e4m3", 128), ("bf16", 64)]


@pytest.mark.parametrize("dtype,D", FORMS)
@pytest.mark.parametrize("page", [16, 48, 64, 80, 128, 512])
def test_window_that_begins_anywhere(dtype, D, page):
    """256 sequences whose windows begin at every offset in a step; pages before a window are gone."""
    window = 1000
    lens = [window + b + 64 * (b % 5) for b in range(250)] + [1, 999, 0, 17, 1000, 0]
    first = [max(0, n - window) for n in lens]
    c = Paged(dtype, 8, D, page, lens, first, 1)
    c.check(normal((len(lens), 32, D), 5, 1.0), 1.0 / math.sqrt(D), window)


@pytest.mark.parametrize("window", [1, 15, 31, 33, 128, 3001])
@pytest.mark.parametrize("dtype,D,G", [("nvfp4", 128, 12), ("e4m3", 64, 3), ("bf16", 128, 4)])
def test_windows_of_other_lengths(dtype, D, G, window):
    """Short windows have many items a warp, a long one several steps of an item; lengths of every residue."""
    B = 600 if window < 1000 else 80
    lens = [1 + (b * 37) % 4500 for b in range(B)]
    first = [max(0, n - window) for n in lens]
    c = Paged(dtype, 2, D, 64, lens, first, 11)
    c.check(normal((B, 2 * G, D), 12, 1.0), 1.0 / math.sqrt(D), window)


# What the cases below reach (a step is 16 or 32 tokens of a kv head; there are 3 to 14 warps a CTA):
#   ragged       several steps a warp, items that a warp begins, ends or holds whole, two records of a warp, items over
#                several CTAs, one to four equal steps a warp and more, pages that end inside a step
#   many         whole items by the dozen in a warp, shares of two and more sequences in the scan, empty ones among them
#   one_item     every warp goes around its ring (at least STAGES + 2 steps), one item over all CTAs
#   growing      the references move in nearly every step

SHAPES = [(dtype, D, G) for dtype in DT for D in (64, 128, 192, 256) for G in (5, 12)]


@pytest.mark.parametrize("dtype,D,G", SHAPES)
@pytest.mark.parametrize("page", [16, 48, 128])
def test_ragged_lines(dtype, D, G, page):
    lens = [4001, 0, 1, 15, 16, 17, 31, 32, 33, 700, 3333, 2048] + [97 * i + 40 for i in range(24)]
    c = Paged(dtype, 8, D, page, lens, [0] * len(lens), 21)
    c.check(normal((len(lens), 8 * G, D), 22, 1.0), 1.0 / math.sqrt(D))


@pytest.mark.parametrize("dtype,D,G", [("bf16", 256, 4), ("e4m3", 128, 8), ("nvfp4", 128, 8), ("e4m3", 192, 16), ("nvfp4", 64, 16)])
@pytest.mark.parametrize("n", [1999, 4500, 9001, 17000, 26000, 34567, 52000])
def test_steps_a_warp(dtype, D, G, n):
    """The same number of steps in every warp, up to four, and more beyond: one long sequence beside a short one."""
    c = Paged(dtype, 8, D, 64, [7, n], [0, 0], 31)
    c.check(normal((2, 8 * G, D), 32, 1.0), 1.0 / math.sqrt(D))


@pytest.mark.parametrize("dtype,D,G", [("bf16", 128, 8), ("e4m3", 64, 2), ("nvfp4", 128, 16), ("e4m3", 256, 9), ("nvfp4", 256, 1)])
@pytest.mark.parametrize("B", [513, 1000])
def test_many_items(dtype, D, G, B):
    lens = [(b * 53) % 171 for b in range(B)]
    c = Paged(dtype, 4, D, 32, lens, [0] * B, 41)
    c.check(normal((B, 4 * G, D), 42, 1.0), 1.0 / math.sqrt(D))


@pytest.mark.parametrize("dtype,D,G", SHAPES)
def test_one_item_over_the_whole_machine(dtype, D, G):
    """Head i sees little but the units whose number is i modulo 16, and a value is not 0 in the channel of
    (number / 16) modulo D alone: a unit that is left out, taken twice or exchanged is a large part of a result."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = sms * 14 * 14 * (32 if dtype == "nvfp4" or (dtype, D) == ("e4m3", 64) else 16) + 21

    def make(seqs, toks):
        u = toks // 16
        k = normal((n, 1, D), 51, 0.01)
        k[torch.arange(n, device="cuda"), 0, u % 16] = 4.0
        v = torch.zeros(n, 1, D, dtype=torch.bfloat16, device="cuda")
        v[torch.arange(n, device="cuda"), 0, u // 16 % D] = 1.0 + normal((n,), 52).abs()
        return k, v

    c = Paged(dtype, 1, D, 256, [n], [0], 50, make)
    q = normal((1, G, D), 53, 0.01)
    q[0, torch.arange(G), torch.arange(G)] = 3.0
    c.check(q, 1.0)


@pytest.mark.parametrize("dtype,D,G", [("bf16", 64, 8), ("bf16", 256, 16), ("e4m3", 128, 8), ("e4m3", 64, 16), ("nvfp4", 128, 8),
                                       ("nvfp4", 192, 16)])
def test_scores_that_grow(dtype, D, G):
    """Scores that rise by some hundreds along each sequence, and for half of the heads fall."""
    lens = [3001, 20000, 1, 513, 9999]
    total = sum(lens)

    def make(seqs, toks):
        k, v = normal((total, 4, D), 61), normal((total, 4, D), 62)
        k[:, :, 0] = (5.0 * toks / torch.tensor(lens, device="cuda")[seqs]).to(torch.bfloat16)[:, None]
        return k, v

    c = Paged(dtype, 4, D, 64, lens, [0] * len(lens), 60, make)
    q = normal((len(lens), 4 * G, D), 63, 1.0)
    q[:, ::2, 0], q[:, 1::2, 0] = 600.0, -600.0
    c.check(q, 0.125)


def test_bf16_weights_keep_their_bits():
    """Two tokens of nearly equal weight and opposite values, beside one that the softmax refers to: what is left is
    2^-15 of the weights, so that a weight in fewer bits shows."""
    B = 512

    def make(seqs, toks):
        k = torch.zeros(3 * B, 1, 64, dtype=torch.bfloat16, device="cuda")
        k[:, 0, 0] = torch.tensor([1.0, 1.0078125, 0.0], device="cuda")[toks].to(torch.bfloat16)
        k[2::3, 0, 1] = 1.0
        v = torch.zeros_like(k)
        v[0::3], v[1::3] = 1.0, -1.0
        return k, v

    c = Paged("bf16", 1, 64, 16, [3] * B, [0] * B, 81, make)
    q = torch.zeros(B, 8, 64, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0 + normal((B, 8), 82).abs().clamp(max=2.0)
    q[..., 1] = 40.0 + 30.0 * normal((B, 8), 83).abs().clamp(max=4.0)
    out, _ = c.call(q, 0.01)
    x = 0.01 * torch.einsum("bgd,jd->bgj", q.double(), c.k[:3, 0].double())
    p = torch.softmax(x, -1)
    want, mag = (p[..., 0] - p[..., 1])[..., None], (p[..., 0] + p[..., 1])[..., None]
    # exp2 is off by 2^-22, its argument (up to 4) by 2^-23; both of two weights, and some 2^-24 of sums: under 2^-20
    assert torch.all((out.double() - want).abs() <= 2.0**-8 * want.abs() + 2.0**-20 * mag)


def test_calls_from_several_threads():
    """Each thread with a stream and a workspace of its own; in a fresh process these are first calls of their kernels."""
    c = [Paged("e4m3", 2, 192, 48, [700, 0, 33, 1200], [0] * 4, 71), Paged("bf16", 1, 256, 16, [900, 5], [0] * 2, 72)]
    q = [normal((len(x.lens), x.H * 9, x.D), 73) for x in c]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(8)]

    def one(i):
        x, s = c[i % 2], streams[i]
        with torch.cuda.stream(s):
            got = [x.call(q[i % 2], 0.07) for _ in range(5)]
        s.synchronize()
        return got

    with ThreadPoolExecutor(8) as pool:
        got = list(pool.map(one, range(8)))
    assert hq.hq_device_error() == 0
    for i in range(2):
        c[i].check(q[i], 0.07)
        want = c[i].call(q[i], 0.07)
        for runs in got[i::2]:
            assert all(torch.equal(a, b) for r in runs for a, b in zip(r, want))


def test_the_most_sequences():
    """2^20 sequences of 0 to 3 tokens on shared pages: thousands of lengths a thread of the scan."""
    B, D, pages = 1 << 20, 64, 4096
    kv = hq.KVDesc(dtype=hq.HQ_BF16, heads=1, head_dim=D, page_size=16)
    buf = torch.full((pages * hq.hq_kv_page_bytes(kv),), 0xFF, dtype=torch.uint8, device="cuda")
    k, v = normal((pages * 3, 1, D), 91), normal((pages * 3, 1, D), 92)
    at = torch.arange(pages * 3, device="cuda")
    hq.hq_kv_write(kv, pages * 3, k, D, v, D, at // 3 * 16 + at % 3, None, pages, buf)
    page = torch.randint(0, pages, (B, 1), generator=gen(93), device="cuda", dtype=torch.int32)
    lens = torch.randint(0, 4, (B,), generator=gen(94), device="cuda", dtype=torch.int32)
    lens[-5000:] = 0
    q = normal((B, 1, D), 95)
    out, lse = torch.full_like(q, 7.0), torch.full((B, 1), 7.0, device="cuda")
    ws = torch.zeros(hq.hq_paged_attn_workspace_bytes(kv, B, 1), dtype=torch.uint8, device="cuda")
    hq.hq_paged_attn(kv, B, 1, q, D, None, pages, buf, page, 1, lens, 0.125, 0, out, D, lse, ws, ws.numel())
    assert hq.hq_device_error() == 0
    rows = page.long() * 3 + torch.arange(3, device="cuda")
    kk, vv = k[rows, 0].double(), v[rows, 0].double()
    x = 0.125 * torch.einsum("bd,bjd->bj", q[:, 0].double(), kk)
    x = torch.where(torch.arange(3, device="cuda") < lens[:, None], x, -math.inf)
    wl = torch.logsumexp(x, -1)
    p = torch.exp(x - wl[:, None]).nan_to_num(nan=0.0)
    want, mag = torch.einsum("bj,bjd->bd", p, vv), torch.einsum("bj,bjd->bd", p, vv.abs())
    dx = 2.0**-18 * 0.125 * torch.einsum("bd,bjd->bj", q[:, 0].double().abs(), kk.abs()).amax(-1)
    assert torch.all((out[:, 0].double() - want).abs() <= 2.0**-8 * want.abs() + (2.0**-10 + 2 * dx[:, None]) * mag)
    some = lens > 0
    assert torch.all((lse[:, 0].double() - wl).abs()[some] <= (2.0**-20 * (1 + wl.abs()) + dx)[some])
    assert torch.all(lse[~some] == -math.inf)


@pytest.mark.parametrize("dtype,H,D,page", [("bf16", 1024, 64, 16), ("e4m3", 1024, 64, 32), ("nvfp4", 512, 128, 4096)])
def test_the_most_heads_and_the_largest_pages(dtype, H, D, page):
    lens = [40, 0, 1, 333]
    c = Paged(dtype, H, D, page, lens, [0] * 4, 101)
    c.check(normal((4, H, D), 102), 0.1)


@pytest.mark.parametrize("dtype,D,page", [("bf16", 256, 64), ("e4m3", 128, 256), ("nvfp4", 192, 16)])
def test_a_cache_past_32_bits(dtype, D, page):
    """Tokens in the first and the last pages of a cache of more than 4 GB."""
    H, n = 8, 300
    kv = hq.KVDesc(dtype=DT[dtype], heads=H, head_dim=D, page_size=page)
    size = hq.hq_kv_page_bytes(kv)
    pages = (9 << 29) // size
    buf = torch.empty(pages * size, dtype=torch.uint8, device="cuda")
    glob = torch.tensor(GLOB, device="cuda") if dtype == "nvfp4" else None
    need = -(-n // page)
    table = torch.stack([torch.arange(need), pages - 1 - torch.arange(need)]).to(torch.int32)
    slots = (table.long()[:, torch.arange(n) // page] * page + torch.arange(n) % page).reshape(-1).cuda()
    k, v = normal((2 * n, H, D), 111), normal((2 * n, H, D), 112)
    hq.hq_kv_write(kv, 2 * n, k, H * D, v, H * D, slots, glob, pages, buf)
    back = [torch.empty_like(k) for _ in range(2)]
    hq.hq_kv_read(kv, 2 * n, slots, glob, pages, buf, back[0], H * D, back[1], H * D)
    for got, x, g in zip(back, (k, v), GLOB):
        assert torch.equal(got, held64(x, dtype, g).float().to(torch.bfloat16))
    q = normal((2, 4 * H, D), 113)
    ws = torch.zeros(hq.hq_paged_attn_workspace_bytes(kv, 2, 4 * H), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(2, 4 * H, device="cuda")
    lens = torch.full((2,), n, dtype=torch.int32, device="cuda")
    hq.hq_paged_attn(kv, 2, 4 * H, q, q.stride(0), glob, pages, buf, table.cuda(), need, lens, 0.1, 0, out, out.stride(0), lse, ws,
                     ws.numel())
    assert hq.hq_device_error() == 0
    small = Paged(dtype, H, D, page, [n, n], [0, 0], 114, lambda seqs, toks: (k, v))  # the same tokens on few pages
    want = small.call(q, 0.1)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    small.check(q, 0.1)


# ---- prompts and captured steps: what surrounds the attention --------------------

def turned(x, pos, table, rot, inter):
    """The rotation in the entry points' fp32 steps (separate torch operations: nothing is fused)."""
    t = table[pos.long()][:, None]
    co, si = t[..., :rot // 2], t[..., rot // 2:]
    x = x.float()
    a, b = (x[..., :rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * co - b * si, b * co + a * si
    y = x.clone()
    y[..., :rot] = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return y


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D,rot,inter,Hq", [(64, 64, 0, 5), (128, 128, 0, 8), (128, 40, 1, 3), (192, 64, 1, 16), (192, 136, 0, 0),
                                            (256, 256, 1, 1), (256, 136, 1, 7), (256, 18, 0, 12), (128, 0, 0, 0)])
def test_prompts(dtype, D, rot, inter, Hq):
    """A prompt of 3001 tokens on pages in any order, its tail padded: every held value and every q is the recipe's."""
    T, H, page, P = 3001, 3, 48, 5000
    pages = -(-T // page) + 1
    kv = hq.KVDesc(dtype=DT[dtype], heads=H, head_dim=D, page_size=page)
    glob = torch.tensor(GLOB, device="cuda") if dtype == "nvfp4" else None
    buf = torch.full((pages * hq.hq_kv_page_bytes(kv),), 0xA5, dtype=torch.uint8, device="cuda")
    qkv = normal((T, Hq + 2 * H, D), 121)
    q, k, v = qkv.split([Hq, H, H], 1)
    at = torch.arange(T, device="cuda") + 7
    slots = torch.randperm(pages, generator=gen(122), device="cuda")[at // page] * page + at % page
    slots[-9:] = -1
    row = qkv.stride(0)
    if rot:
        a = torch.outer(torch.arange(P, device="cuda").double(), 10000.0 ** (-2.0 * torch.arange(rot // 2, device="cuda").double() / rot))
        table = torch.cat([a.cos(), a.sin()], 1).float()
        pos = torch.randint(0, P, (T,), generator=gen(123), device="cuda", dtype=torch.int32)
        qo = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda") if Hq else None
        hq.hq_rope_kv_write(hq.RopeDesc(rot_dim=rot, interleaved=inter), kv, T, Hq, q if Hq else None, row, qo, Hq * D, k, row, v,
                            row, pos, table, P, slots, glob, pages, buf)
        kx = turned(k, pos, table, rot, inter)
        if Hq:
            assert torch.equal(qo, turned(q, pos, table, rot, inter).to(torch.bfloat16))
    else:
        hq.hq_kv_write(kv, T, k, row, v, row, slots, glob, pages, buf)
        kx = k.float()
    back = [torch.full((T, H, D), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    hq.hq_kv_read(kv, T, slots, glob, pages, buf, back[0], H * D, back[1], H * D)
    assert hq.hq_device_error() == 0
    for got, x, g in zip(back, (kx, v.float()), GLOB):
        want = (x.to(torch.bfloat16) if dtype == "bf16" else held64(x, dtype, g).float().to(torch.bfloat16))
        want[-9:] = 3.0
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("e4m3", 192), ("nvfp4", 128)])
def test_a_captured_step_follows_its_sequences(dtype, D):
    """Rotation, write and attention in one graph; positions, slots, lengths and the projection's output change between
    replays.  The result is that of the same calls outside a graph, and attends what the steps have written."""
    B, H, G, page, P, window = 5, 2, 6, 64, 512, 40
    kv = hq.KVDesc(dtype=DT[dtype], heads=H, head_dim=D, page_size=page)
    glob = torch.tensor(GLOB, device="cuda") if dtype == "nvfp4" else None
    rope, table = hq.RopeDesc(rot_dim=D, base=10000.0), torch.empty(P, D, device="cuda")
    hq.hq_rope_table(rope, P, table)
    most, pages = 3, 16
    pt = torch.randperm(pages - 1, generator=gen(131), device="cuda")[:B * most].to(torch.int32).reshape(B, most)
    steps = [normal((B, H * (G + 2), D), 140 + s) for s in range(130)]

    def program():
        z = lambda *s, dtype: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
        s = dict(buf=torch.full((pages * hq.hq_kv_page_bytes(kv),), 0xFF, dtype=torch.uint8, device="cuda"),
                 qkv=torch.zeros_like(steps[0]), pos=z(B, dtype=torch.int32), slots=z(B, dtype=torch.int64),
                 lens=z(B, dtype=torch.int32), q=z(B, H * G, D, dtype=torch.bfloat16), out=z(B, H * G, D, dtype=torch.bfloat16),
                 lse=z(B, H * G, dtype=torch.float32),
                 ws=z(hq.hq_paged_attn_workspace_bytes(kv, B, H * G), dtype=torch.uint8))
        row = s["qkv"].stride(0)

        def step():
            x = s["qkv"]
            hq.hq_rope_kv_write(rope, kv, B, H * G, x, row, s["q"], H * G * D, x[:, H * G:], row, x[:, H * G + H:], row, s["pos"],
                                table, P, s["slots"], glob, pages, s["buf"])
            hq.hq_paged_attn(kv, B, H * G, s["q"], H * G * D, glob, pages, s["buf"], pt, most, s["lens"], 0.1, window, s["out"],
                             H * G * D, s["lse"], s["ws"], s["ws"].numel())
        return s, step

    def feed(s, i):
        at = torch.full((B,), i, device="cuda")
        s["qkv"].copy_(steps[i])
        s["pos"].copy_(at)
        s["slots"].copy_(pt.long().gather(1, at[:, None] // page)[:, 0] * page + at % page)
        s["lens"].copy_(at + 1)

    (s, step), (e, eager) = program(), program()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(len(steps)):
        feed(s, i)
        g.replay()
        feed(e, i)
        eager()
        assert torch.equal(s["out"], e["out"]) and torch.equal(s["lse"], e["lse"]), i
    assert hq.hq_device_error() == 0
    # the last step against the formula, on what the cache holds by its recipe
    first = len(steps) - window
    pos = torch.arange(first, len(steps), device="cuda")
    for b in range(B):
        x = torch.stack([t[b] for t in steps[first:]])
        k = turned(x[:, H * G:H * G + H], pos, table, D, 0)
        k = k.to(torch.bfloat16).double() if dtype == "bf16" else held64(k, dtype, GLOB[0])
        v = held64(x[:, H * G + H:], dtype, GLOB[1])
        c = Paged.__new__(Paged)
        c.dtype = dtype
        for h in range(H):
            r = slice(h * G, (h + 1) * G)
            w = c._compare(s["q"][b, r].double(), k[:, h], v[:, h], 0.1, s["out"][b, r].double(), s["lse"][b, r].double())
            assert torch.all(w <= 1), w


@pytest.mark.parametrize("dtype", ["e4m3", "nvfp4"])
@pytest.mark.parametrize("D", [64, 192, 256])
def test_every_bf16_number_is_held_as_the_activation_quantiser_has_it(dtype, D):
    """All 65536 bit patterns, infinities and NaN among them, in rows of like sizes and of any: what is read back is what
    hq_quant_act's codes and scales stand for."""
    bits = torch.arange(65536, dtype=torch.int32, device="cuda")
    rows = -(-65536 // D)
    like = torch.cat([bits, bits[:rows * D - 65536]])
    by_size = like[torch.argsort(like & 0x7FFF)]
    mixed = like[torch.randperm(rows * D, generator=gen(151), device="cuda")]
    x = torch.cat([by_size, mixed]).to(torch.int16).view(torch.bfloat16).reshape(2 * rows, 1, D).contiguous()
    T, page = 2 * rows, 64
    pages = -(-T // page)
    kv = hq.KVDesc(dtype=DT[dtype], heads=1, head_dim=D, page_size=page)
    buf = torch.zeros(pages * hq.hq_kv_page_bytes(kv), dtype=torch.uint8, device="cuda")
    # E4M3 takes its scale from the row; both sides of NVFP4 under one second-level scale
    glob = torch.tensor([2.5e-3, 2.5e-3], device="cuda") if dtype == "nvfp4" else None
    slots = torch.arange(T, device="cuda")
    hq.hq_kv_write(kv, T, x, D, x, D, slots, glob, pages, buf)
    back = [torch.empty_like(x) for _ in range(2)]
    hq.hq_kv_read(kv, T, slots, glob, pages, buf, back[0], D, back[1], D)
    desc = hq.QuantDesc(w_dtype=hq.HQ_INT4, w_group=128, w_scale_dtype=hq.HQ_BF16, a_dtype=DT[dtype])
    scales = torch.empty(T * D // 16, dtype=torch.uint8, device="cuda") if dtype == "nvfp4" else torch.empty(T, device="cuda")
    codes = torch.empty(T, D if dtype == "e4m3" else D // 2, dtype=torch.uint8, device="cuda")
    hq.hq_quant_act(desc, T, D, x, codes, scales, None, glob, None, 0)
    if dtype == "e4m3":
        want = codes.view(torch.float8_e4m3fn).float() * scales[:, None]
    else:
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
        e = grid[torch.stack([codes & 15, codes >> 4], -1).long()].reshape(T, D // 16, 16)
        want = (e * scales.view(torch.float8_e4m3fn).float().reshape(T, D // 16, 1) * glob[0]).reshape(T, D)
    want = want.to(torch.bfloat16)
    for got in back:
        got = got[:, 0]
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.view(torch.int16)[~want.isnan()], want.view(torch.int16)[~want.isnan()])

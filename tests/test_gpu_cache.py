"""The decoder-cache operators on the GPU against plain 64-bit computations:
rotation tables, rotation, the quantising cache write and its read back, and
attention of one new token over the paged cache."""
import math

import numpy as np
import pytest
import torch

import oracle as O
import quantized_gemm_02_b200 as hq
import synth

pytestmark = pytest.mark.gpu

DT = {"bf16": hq.HQ_BF16, "e4m3": hq.HQ_E4M3, "nvfp4": hq.HQ_NVFP4}
GLOB = (6.0 / 2688.0, 5.0 / 2688.0)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=gen(seed)) * scale).to(torch.bfloat16)


# ---- oracles (64-bit, on the host) ------------------------------------------

def freqs64(rot, base, scaling=0, context=0, factor=1.0, low=0.0, high=0.0):
    f = []
    for i in range(rot // 2):
        w = base ** (-2.0 * i / rot)
        y = 1.0
        if scaling == hq.HQ_ROPE_LINEAR:
            y = 0.0
        elif scaling == hq.HQ_ROPE_TURNS:
            y = min(max((context * w / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
        elif scaling == hq.HQ_ROPE_INDEX:
            at = lambda n: rot * math.log(context / (2 * math.pi * n)) / (2 * math.log(base))  # noqa: E731
            a, c = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
            y = 1 - min(max((i - a) / max(c - a, 0.001), 0.0), 1.0)
        f.append(w * (y + (1 - y) / factor))
    return np.array(f)


def rope64(x, pos, f, interleaved):
    """x [T, H, D] float64, rotated by pos * f on its first 2 len(f) channels."""
    y = x.copy()
    h = len(f)
    a = pos.astype(np.float64)[:, None, None] * f
    i0, i1 = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    y[..., i0] = x[..., i0] * np.cos(a) - x[..., i1] * np.sin(a)
    y[..., i1] = x[..., i1] * np.cos(a) + x[..., i0] * np.sin(a)
    return y


def held64(x_bits, dtype, g):
    """Values a cache holds for rows x [n, D] (bf16 bits), by the oracle's activation quantisers."""
    n, D = x_bits.shape
    if dtype == "bf16":
        return O.decode_act("bf16", n, D, x_bits)[0]
    if dtype == "e4m3":
        q, s = O.quant_fp8_per_token(x_bits)
        return O.E4M3[q] * s.astype(np.float64)[:, None]
    q, s, _ = O.quant_nvfp4(x_bits, np.float32(g))
    return O.decode_act("nvfp4", n, D, q, s, np.float32(g))[0]


# ---- a cache ----------------------------------------------------------------

class Cache:
    def __init__(self, dtype, heads, D, page, pages, fill=0):
        self.dtype, self.H, self.D, self.page, self.pages = dtype, heads, D, page, pages
        self.kv = hq.KVDesc(dtype=DT[dtype], heads=heads, head_dim=D, page_size=page)
        self.buf = torch.full((pages * hq.hq_kv_page_bytes(self.kv),), fill, dtype=torch.uint8, device="cuda")
        self.glob = torch.tensor(GLOB, device="cuda") if dtype == "nvfp4" else None

    def write(self, k, v, slots):
        k, v = k.cuda(), v.cuda()
        hq.hq_kv_write(self.kv, k.shape[0], k, k.stride(0), v, v.stride(0), slots.cuda(), self.glob, self.pages, self.buf)

    def read(self, slots, fill=0.0):
        n = slots.numel()
        k = torch.full((n, self.H, self.D), fill, dtype=torch.bfloat16, device="cuda")
        v = torch.full_like(k, fill)
        hq.hq_kv_read(self.kv, n, slots.cuda(), self.glob, self.pages, self.buf, k, k.stride(0), v, v.stride(0))
        return k.cpu(), v.cpu()


def bits(t):
    return synth.to_np_bits(t.contiguous())


def expected_read(x, dtype, g):
    """bf16 rounding of what is held for x [T, H, D]."""
    T, H, D = x.shape
    held = held64(bits(x).reshape(T * H, D), dtype, g).reshape(T, H, D)
    return torch.from_numpy(held).to(torch.float32).to(torch.bfloat16), held


# ---- rotation ---------------------------------------------------------------

@pytest.mark.parametrize("rot,base,kw", [
    (2, 10000.0, {}), (10, 10000.0, {}), (128, 500000.0, {}),
    (64, 10000.0, dict(scaling=1, factor=4.0)),
    (128, 500000.0, dict(scaling=2, factor=8.0, context=8192, low=1.0, high=4.0)),
    (128, 10000.0, dict(scaling=3, factor=32.0, context=4096, low=1.0, high=32.0, amplitude=1.3465735902799727)),
    (96, 1e6, dict(scaling=3, factor=2.5, context=3, low=1.0, high=32.0)),
])
@pytest.mark.parametrize("P", [1, 1000, 131073])
def test_table(rot, base, kw, P):
    d = hq.RopeDesc(rot_dim=rot, base=base, **kw)
    t = torch.empty(P, rot, device="cuda")
    hq.hq_rope_table(d, P, t)
    amp = kw.get("amplitude", 1.0)
    f = freqs64(rot, base, **{k: v for k, v in kw.items() if k != "amplitude"})
    pos = np.unique(np.concatenate([[0, P - 1], np.linspace(0, P - 1, 200).astype(np.int64)]))
    got = t.cpu().numpy()[pos].astype(np.float64)
    a = np.outer(pos, f)
    want = amp * np.concatenate([np.cos(a), np.sin(a)], 1)
    # the reduced angle is off by 2^-25 (pi/4), sinf / cosf by 2 steps of values up to 1 (2^-23), the product by amplitude
    # rounds amplitude and itself (2 * 2^-24): under 4 * 2^-23 in all; 64-bit angles add P * 2^-50
    assert np.max(np.abs(got - want)) <= amp * 4 * 2.0**-23 + P * 2.0**-50


@pytest.mark.parametrize("rot,base,kw", [
    (2, 10000.0, {}), (10, 10000.0, {}), (128, 500000.0, {}), (128, 1e6, dict(scaling=1, factor=32.0)), (256, 1e8, {}),
    (1024, 10000.0, {}), (128, 10000.0, dict(scaling=3, factor=32.0, context=4096, low=1.0, high=32.0, amplitude=1.3465735902799727)),
    (96, 1e6, dict(scaling=2, factor=8.0, context=8192, low=1.0, high=4.0, amplitude=1e-3)),
])
def test_table_relative_to_each_entry(rot, base, kw):
    """Small sines, and cosines near a quarter of a turn, have as many bits as the others."""
    P = 70001
    t = torch.empty(P, rot, device="cuda")
    hq.hq_rope_table(hq.RopeDesc(rot_dim=rot, base=base, **kw), P, t)
    amp = kw.get("amplitude", 1.0)
    f = freqs64(rot, base, **{k: v for k, v in kw.items() if k != "amplitude"})
    pos = np.unique(np.concatenate([np.arange(3000), np.linspace(0, P - 1, 3000).astype(np.int64)]))
    a = np.outer(pos, f)
    want = amp * np.concatenate([np.cos(a), np.sin(a)], 1)
    err = np.abs(t.cpu().numpy()[pos].astype(np.float64) - want)
    # fp32 roundings, each 2^-24 of the entry: of the angle (its low part, the constant, their product), of the sum, of the
    # product with the amplitude.  The angle: frequencies here and there are off by some 2^-52 of themselves each (a power,
    # a quotient), the product here by 2^-53, a position by 2^-64 of a turn
    angle = 2.0**-50 * a + 2.0**-61 * pos[:, None]
    assert np.all(err <= 5 * 2.0**-24 * np.abs(want) + amp * np.concatenate([angle, angle], 1))


def test_table_of_the_most_positions():
    P = 2**31 - 1
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 17 GB")
    t = torch.full((P, 2), 7.0, device="cuda")
    hq.hq_rope_table(hq.RopeDesc(rot_dim=2, base=10000.0), P, t)
    pos = torch.cat([torch.arange(5), torch.linspace(5, P - 1, 1000, dtype=torch.float64).long()]).clamp(max=P - 1)
    a = pos.double()  # the frequency is 1
    got = t[pos.cuda()].cpu().double()
    # as above: 1 / 2 pi is off by 2^-53 of itself and cut to 2^-64, over 2^31 positions
    assert torch.all((got - torch.stack([a.cos(), a.sin()], 1)).abs() <= 5 * 2.0**-24 + P * 2.0**-53)


def tab64(f, P):
    a = np.outer(np.arange(P), f)
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1)).float()


@pytest.mark.parametrize("inter", [0, 1])
@pytest.mark.parametrize("T,H,D,rot,gap", [
    (1, 1, 64, 64, 0), (3, 5, 128, 128, 64), (7, 2, 192, 64, 8), (5, 3, 256, 48, 0), (33, 1, 128, 10, 0), (4, 2, 8, 2, 0),
    (6, 2, 40, 36, 16), (300, 9, 96, 96, 32), (5, 3, 24, 16, 0), (5, 3, 24, 18, 8), (9, 4, 256, 250, 0), (700, 2, 64, 34, 0),
    (40, 5, 192, 130, 8),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_rope(inter, T, H, D, rot, gap, in_place):
    P = 5000
    f = freqs64(rot, 10000.0)
    table = tab64(f, P).cuda()
    x = normal((T, H * D + gap), 1)
    pos = torch.randint(0, P, (T,), generator=gen(2)).to(torch.int32)
    xg = x.cuda()
    out = xg if in_place else torch.full((T, H * D + 2 * gap), 7.0, dtype=torch.bfloat16, device="cuda")
    hq.hq_rope(hq.RopeDesc(rot_dim=rot, interleaved=inter), T, H, D, xg, xg.stride(0), D, pos.cuda(), table, P, out,
               out.stride(0), D)
    assert hq.hq_device_error() == 0
    got = out.cpu()
    v = x[:, :H * D].reshape(T, H, D).double().numpy()
    want = rope64(v, pos.numpy(), f, inter)
    # one bf16 rounding of the result (2^-8), and the table's and three fp32 steps of |a| + |b| (under 8 * 2^-24)
    amax = np.abs(v).max(-1, keepdims=True)
    err = np.abs(got[:, :H * D].reshape(T, H, D).double().numpy() - want)
    assert np.all(err <= 2.0**-8 * np.abs(want) + 2.0**-21 * amax), float(err.max())
    assert np.array_equal(got[:, :H * D].reshape(T, H, D)[..., rot:].float().numpy(), v[..., rot:])
    # what lies between the rows stays
    rest = got[:, H * D:].float()
    assert torch.equal(rest, x[:, H * D:].float() if in_place else torch.full_like(rest, 7.0))


def test_rope_head_strides():
    T, H, D, P = 9, 4, 64, 100
    f = freqs64(64, 10000.0)
    x = normal((H, T, D), 3).cuda()       # heads outermost
    out = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 50
    hq.hq_rope(hq.RopeDesc(rot_dim=64), T, H, D, x, D, T * D, pos, tab64(f, P).cuda(), P, out, H * D, D)
    want = rope64(x.cpu().transpose(0, 1).double().numpy(), pos.cpu().numpy(), f, 0)
    err = np.abs(out.cpu().double().numpy() - want)
    assert np.all(err <= 2.0**-8 * np.abs(want) + 2.0**-21 * 8)


def test_rope_inverse_is_the_gradient():
    """The rotation is linear and orthogonal: with the sines negated it maps the output's gradient to the input's."""
    T, H, D, P = 5, 2, 64, 64
    f = freqs64(64, 10000.0)
    table = tab64(f, P)
    inv = torch.cat([table[:, :32], -table[:, 32:]], 1).cuda()
    pos = torch.arange(T, dtype=torch.int32) * 11
    g = normal((T, H, D), 4)
    out = torch.empty_like(g, device="cuda")
    hq.hq_rope(hq.RopeDesc(rot_dim=64), T, H, D, g.cuda(), H * D, D, pos.cuda(), inv, P, out, H * D, D)
    x = normal((T, H, D), 5).double().numpy()
    gd = g.double().numpy()
    num = np.zeros_like(gd)
    for i in range(D):  # differences of sum(rope(x) * g) in each channel (exact for a linear map, any step)
        e = np.zeros_like(x)
        e[..., i] = 1.0
        num[..., i] = ((rope64(x + e, pos.numpy(), f, 0) - rope64(x, pos.numpy(), f, 0)) * gd).sum(-1)
    err = np.abs(out.cpu().double().numpy() - num)
    assert np.all(err <= 2.0**-8 * np.abs(num) + 2.0**-21 * 8)


# ---- cache write and read back ------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("H,D,page,T", [(1, 64, 16, 1), (2, 128, 16, 37), (3, 192, 48, 50), (8, 256, 64, 70),
                                        (5, 64, 32, 129)])
@pytest.mark.parametrize("order", ["runs", "scattered"])
def test_write_read(dtype, H, D, page, T, order):
    pages = -(-T // page) + 2
    c = Cache(dtype, H, D, page, pages, fill=0xA5)
    k, v = normal((T, H, D), 6), normal((T, H, D), 7, 0.5)
    k[0, 0] = 0  # an all-zero row
    if order == "runs":
        perm = torch.randperm(pages, generator=gen(8))
        at = torch.arange(T)
        slots = perm[at // page] * page + at % page
    else:
        slots = torch.randperm(pages * page, generator=gen(9))[:T]
    c.write(k, v, slots)
    rk, rv = c.read(slots)
    assert hq.hq_device_error() == 0
    for got, x, g in ((rk, k, GLOB[0]), (rv, v, GLOB[1])):
        want, _ = expected_read(x, dtype, g)
        # the quantisers are the oracle's bit for bit, and value * scale is rounded to fp32 and then to bf16 on both sides
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["e4m3", "nvfp4"])
@pytest.mark.parametrize("D", [64, 128, 192, 256])
def test_write_read_rows_of_any_size(dtype, D):
    """Rows from the smallest to the largest bf16 numbers, zeros of both signs, and quotients that are ties: the codes
    are the recipe's (fp32 division) bit for bit."""
    exps = [-133, -126, -100, -84, -61, -59, -40, -9, 0, 13, 59, 61, 84, 100, 127]
    T = len(exps) + 17
    c = Cache(dtype, 1, D, 16, 3)
    k, v = normal((T, 1, D), 25), normal((T, 1, D), 26)
    for i, e in enumerate(exps):
        for x in (k, v):
            x[i] = (x[i].double() / 4 * 2.0**e).to(torch.bfloat16).clamp(-3.3e38, 3.3e38)
    k[-1, 0, ::3] = -0.0
    v[-2] = -0.0
    grid = torch.tensor([448, 17, -17, 19, -19, 0.25, 1.0625, -1.1875, 2.5, -3.5, 5, 0.75]).repeat(D // 12 + 1)[:D]
    k[-3, 0], v[-3, 0] = grid.to(torch.bfloat16), (grid / 64).to(torch.bfloat16)
    slots = torch.arange(T) + 5  # a run through units that starts inside one
    c.write(k, v, slots)
    rk, rv = c.read(slots)
    for got, x, g in ((rk, k, GLOB[0]), (rv, v, GLOB[1])):
        want, _ = expected_read(x, dtype, g)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    # a row with infinities spoils no other
    k[3, 0, 5] = math.inf
    c.write(k, v, slots)
    again, _ = c.read(slots)
    keep = [i for i in range(T) if i != 3]
    assert torch.equal(again[keep], rk[keep])


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("first", [0, 1, 7, 8, 9, 15])
@pytest.mark.parametrize("page", [16, 48])
def test_runs_that_start_anywhere(dtype, first, page):
    """A prompt's slots: any first row, page ends inside a group of 16, a gap, and a tail."""
    T, H, D = 70, 2, 128
    perm = torch.randperm(8, generator=gen(27))
    at = torch.arange(T) + first
    slots = perm[at // page] * page + at % page
    slots[40] = -1
    c = Cache(dtype, H, D, page, 8, fill=0x3C)
    k, v = normal((T, H, D), 28), normal((T, H, D), 29)
    c.write(k, v, slots)
    rk, rv = c.read(slots, fill=2.0)
    for got, x, g in ((rk, k, GLOB[0]), (rv, v, GLOB[1])):
        want, _ = expected_read(x, dtype, g)
        want[40] = 2.0
        assert torch.equal(got, want)
    back = torch.arange(T - 1, -1, -1)  # the same slots one by one, in another order
    bk, bv = c.read(slots[back], fill=2.0)
    assert torch.equal(bk[back], rk) and torch.equal(bv[back], rv)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("D", [64, 128, 192, 256])
def test_only_the_named_slots_change(dtype, D):
    H, page, pages = 3, 32, 4
    c = Cache(dtype, H, D, page, pages)
    n = pages * page
    k, v = normal((n, H, D), 10), normal((n, H, D), 11)
    c.write(k, v, torch.arange(n))
    before = c.buf.clone()
    slots = torch.tensor([5, -1, 37, 38, 127, -7, 64])
    k2, v2 = normal((7, H, D), 12), normal((7, H, D), 13)
    c.write(k2, v2, slots)
    assert hq.hq_device_error() == 0
    keep = torch.tensor([s for s in range(n) if s not in slots.tolist()])
    rk, rv = c.read(keep)
    for got, x, g in ((rk, k, GLOB[0]), (rv, v, GLOB[1])):
        want, _ = expected_read(x[keep], dtype, g)
        assert torch.equal(got, want)
    rk, _ = c.read(slots, fill=9.0)
    assert torch.all(rk[1] == 9) and torch.all(rk[5] == 9)
    want, _ = expected_read(k2, dtype, GLOB[0])
    ok = [0, 2, 3, 4, 6]
    assert torch.equal(rk[ok], want[ok])
    # the same tokens written again give the first bytes back: nothing else was touched
    at = slots[ok]
    c.write(k[at], v[at], at)
    assert torch.equal(c.buf, before)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "nvfp4"])
def test_strided_inputs_and_outputs(dtype):
    H, D, T = 2, 128, 21
    c = Cache(dtype, H, D, 16, 4)
    qkv = normal((T, 4 * D + 2 * H * D), 14)
    k, v = qkv[:, 4 * D:4 * D + H * D], qkv[:, 4 * D + H * D:]
    dev = qkv.cuda()
    row = dev.stride(0)
    slots = torch.arange(T) + 3
    hq.hq_kv_write(c.kv, T, dev[:, 4 * D:], row, dev[:, 4 * D + H * D:], row, slots.cuda(), c.glob, 4, c.buf)
    out = torch.full((T, 2, H * D + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    hq.hq_kv_read(c.kv, T, slots.cuda(), c.glob, 4, c.buf, out, out.stride(0), out[:, 1], out.stride(0))
    got = out.cpu()
    for i, x in enumerate((k, v)):
        want, _ = expected_read(x.reshape(T, H, D), dtype, GLOB[i])
        assert torch.equal(got[:, i, :H * D].reshape(T, H, D), want)
    assert torch.all(got[:, :, H * D:] == 3)
    one = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")  # K alone
    hq.hq_kv_read(c.kv, T, slots.cuda(), c.glob, 4, c.buf, one, one.stride(0), None, 0)
    assert torch.equal(one.cpu().reshape(T, -1), got[:, 0, :H * D])


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("inter", [0, 1])
@pytest.mark.parametrize("D,rot,Hq,in_place", [(128, 128, 8, False), (64, 20, 3, True), (192, 64, 0, False),
                                               (256, 240, 5, True)])
def test_rope_kv_write(dtype, inter, D, rot, Hq, in_place):
    H, T, P, page = 2, 19, 300, 16
    f = freqs64(rot, 10000.0)
    table = tab64(f, P)
    c = Cache(dtype, H, D, page, 3)
    k, v, q = normal((T, H, D), 15), normal((T, H, D), 16), normal((T, max(Hq, 1), D), 17)
    pos = torch.randint(0, P, (T,), generator=gen(18)).to(torch.int32)
    slots = torch.randperm(48, generator=gen(19))[:T]
    slots[4] = -1
    qd = q.cuda()
    qo = (qd if in_place else torch.zeros_like(qd)) if Hq else None
    kd, vd = k.cuda(), v.cuda()
    hq.hq_rope_kv_write(hq.RopeDesc(rot_dim=rot, interleaved=inter), c.kv, T, Hq, qd if Hq else None, qd.stride(0), qo,
                        qd.stride(0), kd, kd.stride(0), vd, vd.stride(0), pos.cuda(), table.cuda(), P, slots.cuda(),
                        c.glob, 3, c.buf)
    assert hq.hq_device_error() == 0
    # the rotation in the entry point's fp32 steps, then the quantiser's on its fp32 result
    t = table[pos.long()][:, None].float()
    co, si = t[..., :rot // 2], t[..., rot // 2:]

    def turn(x):
        x = x.float()
        a, b = (x[..., :rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
        a, b = a * co - b * si, b * co + a * si
        y = x.clone()
        y[..., :rot] = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
        return y

    kr = turn(k)
    if dtype == "bf16":
        held = kr.to(torch.bfloat16).double()
    elif dtype == "e4m3":
        am = kr.abs().amax(-1, keepdim=True)
        s = am / torch.tensor(448.0)
        held = (kr / s).to(torch.float8_e4m3fn).double() * s.double()
    else:
        b = kr.unflatten(-1, (-1, 16))
        g = torch.tensor(GLOB[0])
        sb = (b.abs().amax(-1, keepdim=True) / torch.tensor(6.0) / g).to(torch.float8_e4m3fn)
        y = b / (sb.float() * g)
        a = y.abs()
        st = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        e = torch.copysign((torch.round(a / st) * st).clamp(max=6), y)
        held = (e.double() * sb.double() * g.double()).flatten(-2)
    rk, rv = c.read(slots, fill=5.0)
    ok = [i for i in range(T) if i != 4]
    assert torch.all(rk[4] == 5)
    d = (rk.double() - held).abs()[ok]
    assert torch.all(d <= 2.0**-8 * held.abs()[ok]), float(d.max())
    want, _ = expected_read(v, dtype, GLOB[1])
    assert torch.equal(rv[ok], want[ok])
    if Hq:
        want = rope64(q.double().numpy(), pos.numpy(), f, inter)
        err = np.abs(qo.cpu().double().numpy() - want)  # q of the skipped token is rotated too
        assert np.all(err <= 2.0**-8 * np.abs(want) + 2.0**-21 * 8)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "nvfp4"])
def test_rope_kv_write_of_rows_next_to_nothing(dtype):
    """bf16's smallest numbers under a table of small amplitude: finite values, as small as the rows."""
    H, T, D, P = 2, 20, 128, 8
    c = Cache(dtype, H, D, 16, 2)
    k = (normal((T, H, D), 31).float().sign() * 2.0**-133).to(torch.bfloat16)
    v = normal((T, H, D), 32)
    table = (tab64(freqs64(128, 10000.0), P) * torch.exp2(-torch.arange(P).float())[:, None]).cuda()  # to 2^-7
    table[4:] *= 2.0**-8
    pos, slots = torch.arange(T, dtype=torch.int32) % P, torch.arange(T)
    kd, vd = k.cuda(), v.cuda()
    hq.hq_rope_kv_write(hq.RopeDesc(rot_dim=128), c.kv, T, 0, None, 0, None, 0, kd, kd.stride(0), vd, vd.stride(0), pos.cuda(),
                        table, P, slots.cuda(), c.glob, 2, c.buf)
    rk, rv = c.read(slots)
    assert hq.hq_device_error() == 0
    # |a c - b s| <= sqrt(2) 2^-133; what is held is off by no more than the largest channel
    assert torch.all(rk.double().abs() <= 2.0**-132)
    want, _ = expected_read(v, dtype, GLOB[1])
    assert torch.equal(rv, want)


# ---- attention ----------------------------------------------------------------

def attn64(q, k, v, first, n, scale, group):
    """q [Hq, D], k and v [n, H, D] float64 -> (out, lse, bound of |w| |v|)."""
    Hq, D = q.shape
    out, lse, mag = np.zeros((Hq, D)), np.full(Hq, -np.inf), np.zeros((Hq, D))
    if n == 0:
        return out, lse, mag
    for i in range(Hq):
        x = scale * (k[first:n, i // group] @ q[i])
        m = x.max()
        p = np.exp(x - m)
        out[i] = (p @ v[first:n, i // group]) / p.sum()
        mag[i] = (p @ np.abs(v[first:n, i // group])) / p.sum()
        lse[i] = m + math.log(p.sum())
    return out, lse, mag


def run_attn(c, q, table, lens, scale, window=0, ws=None, out=None, lse=True, stream=None):
    B, Hq, D = q.shape
    need = hq.hq_paged_attn_workspace_bytes(c.kv, B, Hq)
    assert need > 0
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda") if ws is None else ws
    out = torch.full((B, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    l = torch.full((B, Hq), 7.0, device="cuda") if lse else None
    hq.hq_paged_attn(c.kv, B, Hq, q, q.stride(0), c.glob, c.pages, c.buf, table, table.shape[1], lens, scale, window, out,
                     out.stride(0), l, ws, ws.numel(), stream=stream)
    return out, l


def fill_cache(dtype, H, D, page, lens, seed, fill=0xFF, spare=1, kscale=1.0, vscale=1.0):
    """A cache with sequences of these lengths on pages in random order; every other byte is `fill` (NaN codes).
    Returns (cache, page table, [(k, v) float64 per sequence])."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    c = Cache(dtype, H, D, page, pages, fill=fill)
    perm = torch.randperm(pages, generator=gen(seed))
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32)
    held, at = [], 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = perm[at:at + need[b]].to(torch.int32)
        at += need[b]
        k, v = normal((n, H, D), seed + 100 + b, kscale), normal((n, H, D), seed + 500 + b, vscale)
        if n:
            j = torch.arange(n)
            c.write(k, v, table[b][j // page].long() * page + j % page)
        held.append(tuple(expected_read(x, dtype, g)[1] if n else np.zeros((0, H, D)) for x, g in zip((k, v), GLOB)))
    return c, table.cuda(), held


def check_attn(c, q, table, lens, held, scale, window=0, got=None):
    out, lse = run_attn(c, q.cuda(), table, torch.tensor(lens, dtype=torch.int32, device="cuda"), scale, window) if got is None else got
    assert hq.hq_device_error() == 0
    group = q.shape[1] // c.H
    o, l = out.cpu().double().numpy(), lse.cpu().double().numpy()
    for b, n in enumerate(lens):
        first = max(0, n - window) if window else 0
        want, wl, mag = attn64(q[b].double().numpy(), held[b][0], held[b][1], first, n, scale, group)
        # scores: at most 32 fp32 accumulations, each off by 2^-24 of sum |q k| (2^-19 of mx in all).  Output: that much of
        # each weight, twice (numerator and denominator); 2^-11 for weights in fp16 and as much for exp and the sums;
        # the result's own rounding to bf16, 2^-8
        qa = np.abs(q[b].double().numpy()).sum(-1, keepdims=True)
        dx = 2.0**-19 * abs(scale) * qa * (np.abs(held[b][0]).max() if n else 0.0)
        # fp16 weights end at a spacing of 2^-24, where the largest one (E4M3: times its token's scale) is at least 2^10:
        # each is off by up to 2^-35 of that, which shows in channels where the heavy tokens hold zeros.  lse gives the
        # largest normalised weight's bound of 1 for NVFP4; for E4M3 the largest product of weight and value
        small = np.zeros((q.shape[1], 1))
        if n and c.dtype != "bf16":
            v = np.abs(held[b][1][first:n])
            for i in range(q.shape[1]):
                w = np.exp(scale * (held[b][0][first:n, i // group] @ q[b, i].double().numpy()) - wl[i])
                top = v[:, i // group].max() if c.dtype == "nvfp4" else (w * v[:, i // group].max(-1)).max()
                small[i] = (n - first) * 2.0**-35 * top
        tol = 2.0**-8 * np.abs(want) + (2.0**-10 + 2 * dx) * mag + small + 1e-37
        err = np.abs(o[b] - want)
        assert np.all(err <= tol), (b, n, float((err / tol).max()))
        if n == 0:
            assert np.all(o[b] == 0) and np.all(l[b] == -np.inf)
        else:
            assert np.all(np.abs(l[b] - wl) <= 2.0**-20 * (1 + np.abs(wl)) + dx[:, 0]), (b, np.abs(l[b] - wl).max())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("H,G,D,page", [(1, 1, 64, 16), (2, 4, 128, 16), (1, 5, 192, 48), (2, 8, 256, 64),
                                        (1, 12, 128, 32), (3, 16, 64, 16), (1, 40, 128, 16), (1, 17, 256, 16)])
def test_attention(dtype, H, G, D, page):
    lens = [1, 0, 15, 16, 17, 130, 63]
    c, table, held = fill_cache(dtype, H, D, page, lens, 20)
    q = normal((len(lens), H * G, D), 21, 2.0)
    check_attn(c, q, table, lens, held, 1.0 / math.sqrt(D))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("B,n", [(1, 1), (1, 31), (1, 4099), (3, 1500), (40, 77), (300, 5)])
def test_attention_lengths(dtype, B, n):
    lens = [n] + [max(0, (n * (i * 37 % 100)) // 100) for i in range(1, B)]
    c, table, held = fill_cache(dtype, 2, 128, 32, lens, 30)
    q = normal((B, 8, 128), 31, 2.0)
    check_attn(c, q, table, lens, held, 0.09)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 5000])
def test_attention_window(dtype, window):
    lens = [1, 0, 16, 100, 101, 333]
    c, table, held = fill_cache(dtype, 2, 64, 16, lens, 40)
    q = normal((len(lens), 6, 64), 41, 2.0)
    check_attn(c, q, table, lens, held, 0.125, window)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "nvfp4"])
def test_attention_window_over_released_pages(dtype):
    """Pages wholly before the window may be gone: their ids are not read."""
    lens = [333, 200]
    c, table, held = fill_cache(dtype, 2, 64, 16, lens, 45)
    q = normal((2, 4, 64), 46, 2.0)
    table[0, :(333 - 20) // 16] = -1
    table[1, :(200 - 20) // 16] = 1 << 30
    check_attn(c, q, table, lens, held, 0.125, 20)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("qs,ks,vs", [(300.0, 1.0, 1.0), (1e-30, 1.0, 1.0), (1.0, 1.0, 1e-20), (1e4, 1e-3, 1e15)])
def test_attention_extremes(dtype, qs, ks, vs):
    """Peaked weights, tiny queries, tiny and huge values.  (The NVFP4 cache's static scale bounds what it holds.)"""
    if dtype == "nvfp4" and (vs != 1.0 or ks != 1.0):
        vs, ks = 1.0, 1.0
    lens = [5, 70, 300]
    c, table, held = fill_cache(dtype, 1, 128, 16, lens, 50, kscale=ks, vscale=vs)
    q = normal((3, 8, 128), 51, qs)
    check_attn(c, q, table, lens, held, 0.0884 if qs < 100 else 0.0884 / 16)


@pytest.mark.parametrize("scale", [1.0, 0.08, 0.0])
def test_attention_scales_that_differ_between_tokens(scale):
    """E4M3 values whose scales span 2^+-60 between tokens: the largest values have a weight of nothing, of 2^-75 (and
    are the result all the same), or of one."""
    H, D, n = 1, 64, 64
    c = Cache("e4m3", H, D, 16, 4)
    k, v = normal((n, H, D), 60), normal((n, H, D), 61)
    v = (v.float() * torch.exp2(torch.linspace(-60, 60, n).round())[:, None, None]).to(torch.bfloat16)
    k[:8] = k[:8].abs()    # the tokens of the smallest values get nearly all of the weight
    k[8:] = -k[8:].abs()
    c.write(k, v, torch.arange(n))
    held = [tuple(expected_read(x, "e4m3", 0)[1] for x in (k, v))]
    q = normal((1, 2, D), 62).abs() * 8
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    check_attn(c, q, table, [n], held, scale)


def test_attention_strides_and_no_lse():
    lens = [40, 3]
    c, table, held = fill_cache("e4m3", 2, 128, 16, lens, 70)
    wide = normal((2, 8 * 128 + 256), 71, 2.0).cuda()
    q = wide[:, :1024].unflatten(1, (8, 128))
    out = torch.full((2, 1024 + 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, none = run_attn(c, q, table, lens_d, 0.1, out=out[:, :1024].unflatten(1, (8, 128)), lse=False)
    assert none is None and torch.all(out[:, 1024:] == 7)
    ref, lse = run_attn(c, q.contiguous(), table, lens_d, 0.1)
    assert torch.equal(o, ref)
    check_attn(c, q.cpu(), table, lens, held, 0.1, got=(o, lse))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "nvfp4"])
def test_attention_workspace_is_left_ready_and_results_repeat(dtype):
    lens = [3000, 0, 1, 700]
    c, table, held = fill_cache(dtype, 2, 128, 16, lens, 80)
    q = normal((4, 8, 128), 81, 2.0).cuda()
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.zeros(hq.hq_paged_attn_workspace_bytes(c.kv, 4, 8), dtype=torch.uint8, device="cuda")
    first = run_attn(c, q, table, ld, 0.1, ws=ws)
    for _ in range(20):
        again = run_attn(c, q, table, ld, 0.1, ws=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    # other lengths, another batch and another head layout with the same workspace
    c2, table2, held2 = fill_cache(dtype, 1, 64, 16, [9, 2000], 82)
    q2 = normal((2, 3, 64), 83, 2.0)
    need = hq.hq_paged_attn_workspace_bytes(c2.kv, 2, 3)
    big = ws if ws.numel() >= need else torch.zeros(need, dtype=torch.uint8, device="cuda")
    got = run_attn(c2, q2.cuda(), table2, torch.tensor([9, 2000], dtype=torch.int32, device="cuda"), 0.2, ws=big)
    check_attn(c2, q2, table2, [9, 2000], held2, 0.2, got=got)


def test_attention_captured_with_lengths_that_change():
    """One captured call serves growing sequences: lengths, tables and pages are read on the device."""
    H, G, D, page = 2, 4, 128, 16
    full = [70, 33, 900]
    c, table, held = fill_cache("e4m3", H, D, page, full, 90)
    q = normal((3, H * G, D), 91, 2.0)
    qd = q.cuda()
    ld = torch.tensor([1, 0, 5], dtype=torch.int32, device="cuda")
    ws = torch.zeros(hq.hq_paged_attn_workspace_bytes(c.kv, 3, H * G), dtype=torch.uint8, device="cuda")
    out = torch.empty(3, H * G, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(3, H * G, device="cuda")
    call = lambda: hq.hq_paged_attn(c.kv, 3, H * G, qd, qd.stride(0), None, c.pages, c.buf, table, table.shape[1], ld, 0.1,  # noqa: E731
                                    0, out, out.stride(0), lse, ws, ws.numel())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([1, 0, 5], [70, 33, 900], [16, 17, 0], [0, 0, 0], [2, 32, 513]):
        ld.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        check_attn(c, q, table, lens, held, 0.1, got=(out, lse))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "nvfp4"])
def test_attention_first_call_of_a_shape_captured(dtype):
    """The first call of a kernel may be a captured one (D = 192 with 9 heads a kv head is used nowhere else)."""
    lens = [100, 40]
    c, table, held = fill_cache(dtype, 1, 192, 32, lens, 95)
    q = normal((2, 9, 192), 96, 2.0)
    qd, ld = q.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.zeros(hq.hq_paged_attn_workspace_bytes(c.kv, 2, 9), dtype=torch.uint8, device="cuda")
    out = torch.empty(2, 9, 192, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(2, 9, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hq.hq_paged_attn(c.kv, 2, 9, qd, qd.stride(0), c.glob, c.pages, c.buf, table, table.shape[1], ld, 0.1, 0, out,
                         out.stride(0), lse, ws, ws.numel())
    for _ in range(3):
        g.replay()
    check_attn(c, q, table, lens, held, 0.1, got=(out, lse))


def test_attention_two_streams_with_their_own_workspaces():
    lens = [700, 0, 33, 1200]
    c, table, held = fill_cache("e4m3", 2, 128, 16, lens, 97)
    q = [normal((4, 8, 128), 98 + i, 2.0) for i in range(2)]
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
    qd, streams = [x.cuda() for x in q], [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty(4, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    wss = [torch.zeros(hq.hq_paged_attn_workspace_bytes(c.kv, 4, 8), dtype=torch.uint8, device="cuda") for _ in range(2)]
    lses = [torch.empty(4, 8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            hq.hq_paged_attn(c.kv, 4, 8, qd[i], qd[i].stride(0), None, c.pages, c.buf, table, table.shape[1], ld, 0.1, 0,
                             outs[i], outs[i].stride(0), lses[i], wss[i], wss[i].numel(), stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        check_attn(c, q[i], table, lens, held, 0.1, got=(outs[i], lses[i]))


def test_attention_refuses_a_line_past_its_counters():
    """2^36 tokens by page tables that name one page over and over: refused at once, and the next call is sound."""
    c, table, held = fill_cache("e4m3", 1, 64, 4096, [50], 99, spare=0)
    q = normal((64, 1, 64), 100, 2.0).cuda()
    pt = torch.zeros(64, 1 << 18, dtype=torch.int32, device="cuda")
    lens = torch.full((64,), 1 << 30, dtype=torch.int32, device="cuda")
    lens[3] = 0
    ws = torch.zeros(hq.hq_paged_attn_workspace_bytes(c.kv, 64, 1), dtype=torch.uint8, device="cuda")
    out, lse = run_attn(c, q, pt, lens, 0.1, ws=ws)
    assert hq.hq_device_error() == 2
    assert torch.all(out[3] == 0) and torch.all(torch.isinf(lse[3]))
    keep = [i for i in range(64) if i != 3]
    assert torch.all(out[keep] == 7) and torch.all(lse[keep] == 7)
    got = run_attn(c, q[:1], table, torch.tensor([50], dtype=torch.int32, device="cuda"), 0.1, ws=ws)
    check_attn(c, q[:1].cpu(), table, [50], held, 0.1, got=got)


def test_attention_shared_prefix_pages():
    """Sequences may share pages (a common prompt)."""
    c, table, held = fill_cache("nvfp4", 2, 128, 32, [64, 100], 101)
    t = table.cpu()
    shared = torch.stack([torch.cat([t[1, :3], t[1, 3:4]]), torch.cat([t[1, :3], t[0, :1]])]).cuda()
    k, v = held[1]
    other = tuple(np.concatenate([x[:96], y[:10]]) for x, y in zip(held[1], held[0]))
    q = normal((2, 8, 128), 102, 2.0)
    check_attn(c, q, shared, [100, 106], [(k, v), other], 0.1)


# ---- together -------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "nvfp4"])
def test_decoding_steps(dtype):
    """A prompt, then steps of one token per sequence: rotation, write and attention on a stream of their own."""
    H, G, D, page, P, rot = 2, 4, 128, 16, 512, 64
    lens = [30, 1, 47]
    B, steps = len(lens), 4
    f = freqs64(rot, 10000.0)
    rope = hq.RopeDesc(rot_dim=rot, base=10000.0)
    table = torch.empty(P, rot, device="cuda")
    hq.hq_rope_table(rope, P, table)
    most = 4
    c = Cache(dtype, H, D, page, B * most + 1, fill=0xFF)
    pt = torch.randperm(B * most, generator=gen(5)).to(torch.int32).reshape(B, most)
    ptd = pt.cuda()
    ws = torch.zeros(hq.hq_paged_attn_workspace_bytes(c.kv, B, H * G), dtype=torch.uint8, device="cuda")
    ks, vs = [np.zeros((0, H, D))] * B, [np.zeros((0, H, D))] * B
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())

    def put(qkv, pos, slots):
        T = qkv.shape[0]
        d = qkv.cuda()
        row = d.stride(0)
        sl, ps = slots.cuda(), pos.to(torch.int32).cuda()
        stream.wait_stream(torch.cuda.current_stream())
        qo = torch.empty(T, H * G, D, dtype=torch.bfloat16, device="cuda")
        hq.hq_rope_kv_write(rope, c.kv, T, H * G, d, row, qo, H * G * D, d[:, H * G:], row, d[:, H * G + H:], row, ps, table,
                            P, sl, c.glob, c.pages, c.buf, stream=stream)
        stream.synchronize()
        return qo

    for b, n in enumerate(lens):
        j = torch.arange(n)
        put(normal((n, H * (G + 2), D), 200 + b), j, pt[b][j // page].long() * page + j % page)
    for step in range(steps):
        n = [x + step + 1 for x in lens]
        pos = torch.tensor(n) - 1
        q = put(normal((B, H * (G + 2), D), 300 + step), pos,
                torch.stack([pt[b, p // page].long() * page + p % page for b, p in enumerate(pos.tolist())]))
        got = run_attn(c, q, ptd, torch.tensor(n, dtype=torch.int32, device="cuda"), 0.088, ws=ws)
        held = []
        for b in range(B):  # what the cache holds, read back (bf16 of the held values)
            j = torch.arange(n[b])
            k, v = c.read(pt[b][j // page].long() * page + j % page)
            x = torch.cat([normal((lens[b], H * (G + 2), D), 200 + b)] +
                          [normal((B, H * (G + 2), D), 300 + s)[b:b + 1] for s in range(step + 1)])
            kx = rope64(x[:, H * G:H * G + H].double().numpy(), np.arange(n[b]), f, 0)
            step_of = {"bf16": 2.0**-8, "e4m3": 2.0**-4, "nvfp4": 0.25}[dtype]  # half a step of the format, and bf16's
            lim = 1.02 * step_of * np.abs(kx).max(-1, keepdims=True)
            assert np.all(np.abs(k.double().numpy() - kx) <= lim)
            held.append((k.double().numpy(), v.double().numpy()))
        out, lse = got
        assert hq.hq_device_error() == 0
        for b in range(B):
            want, wl, mag = attn64(q[b].cpu().double().numpy(), held[b][0], held[b][1], 0, n[b], 0.088, G)
        # the read back rounds k and v to bf16 (2^-8 each): v enters as is, k through 2^-8 sum |q k| scale
            dx = 0.088 * 2.0**-8 * (np.abs(q[b].cpu().double().numpy()).sum(-1) * np.abs(held[b][0]).max())
            tol = (2.0**-7 + 2 * dx[:, None]) * mag + 2.0**-8 * np.abs(want)
            assert np.all(np.abs(out[b].cpu().double().numpy() - want) <= tol)
            assert np.all(np.abs(lse[b].cpu().double().numpy() - wl) <= dx + 1e-4)


# ---- refusals that only the device can see -----------------------------------------

def test_bad_slots_positions_pages_lengths():
    H, D, page = 1, 64, 16
    c = Cache("e4m3", H, D, page, 2)
    k, v = normal((3, H, D), 1), normal((3, H, D), 2)
    before = c.buf.clone()
    c.write(k, v, torch.tensor([32, -1, 1 << 40]))
    assert hq.hq_device_error() == 6 and torch.equal(c.buf, before)
    c.write(k, v, torch.tensor([0, 1, 2]))
    assert hq.hq_device_error() == 0
    rk, _ = c.read(torch.tensor([0, 32, 1]), fill=4.0)
    assert hq.hq_device_error() == 6
    assert torch.all(rk[1] == 4) and not torch.any(rk[0] == 4)
    table = tab64(freqs64(64, 10000.0), 10).cuda()
    x = normal((3, 1, 64), 3).cuda()
    out = torch.full_like(x, 6.0)
    hq.hq_rope(hq.RopeDesc(rot_dim=64), 3, 1, 64, x, 64, 64, torch.tensor([0, 10, -1], dtype=torch.int32, device="cuda"),
               table, 10, out, 64, 64)
    assert hq.hq_device_error() == 6
    assert torch.equal(out[0], x[0]) and torch.all(out[1:] == 6)
    # a page past the cache is left out, a length past the table counts as the table's
    q = normal((2, 2, 64), 4, 2.0).cuda()
    pt = torch.tensor([[0, 2], [0, -3]], dtype=torch.int32, device="cuda")
    out, lse = run_attn(c, q, pt, torch.tensor([3, 3], dtype=torch.int32, device="cuda"), 0.1)
    assert hq.hq_device_error() == 0  # the second page is not needed
    ref = out.clone()
    c.write(normal((13, H, D), 5), normal((13, H, D), 6), torch.arange(3, 16))
    full, _ = run_attn(c, q, pt[:, :1].contiguous(), torch.tensor([16, 16], dtype=torch.int32, device="cuda"), 0.1)
    assert hq.hq_device_error() == 0
    out, lse = run_attn(c, q, pt, torch.tensor([20, 30], dtype=torch.int32, device="cuda"), 0.1)
    assert hq.hq_device_error() == 6
    assert torch.all((out.float() - full.float()).abs() <= 2.0**-6 * full.float().abs() + 2.0**-6)
    near = lambda a, b: torch.all((a.float() - b.float()).abs() <= 2.0**-6 * b.float().abs() + 2.0**-6)  # noqa: E731
    out, lse = run_attn(c, q, pt[:, :1].contiguous(), torch.tensor([3, 17], dtype=torch.int32, device="cuda"), 0.1)
    assert hq.hq_device_error() == 6 and near(out[0], ref[0]) and near(out[1], full[1])
    out, lse = run_attn(c, q, pt[:, :1].contiguous(), torch.tensor([-5, 3], dtype=torch.int32, device="cuda"), 0.1)
    assert hq.hq_device_error() == 6
    assert torch.all(out[0] == 0) and torch.all(torch.isinf(lse[0])) and near(out[1], ref[1])

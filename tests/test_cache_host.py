"""Host-side checks of the decoder-cache entry points (no GPU needed): page
sizes, argument checks before any device work, and no-ops."""
import ctypes

import pytest

import quantized_gemm_02_b200 as hq

OK = hq.KVDesc(dtype=hq.HQ_E4M3, heads=8, head_dim=128, page_size=16)


def kv(**kw):
    d = dict(dtype=hq.HQ_E4M3, heads=8, head_dim=128, page_size=16)
    d.update(kw)
    return hq.KVDesc(**d)


def refused(status, fn, *args):
    with pytest.raises(hq.HQError) as e:
        fn(*args, stream=0)
    assert e.value.status == status, e.value


@pytest.mark.parametrize("heads,D,page", [(1, 64, 16), (8, 128, 64), (3, 192, 48), (16, 256, 4096)])
def test_page_bytes(heads, D, page):
    rows = 2 * heads * page  # K and V of every head and token
    assert hq.hq_kv_page_bytes(kv(dtype=hq.HQ_BF16, heads=heads, head_dim=D, page_size=page)) == rows * 2 * D
    assert hq.hq_kv_page_bytes(kv(heads=heads, head_dim=D, page_size=page)) == rows * (D + 4)
    assert hq.hq_kv_page_bytes(kv(dtype=hq.HQ_NVFP4, heads=heads, head_dim=D, page_size=page)) == rows * (D // 2 + D // 16)


BAD = [dict(dtype=hq.HQ_MXFP8), dict(dtype=99), dict(heads=0), dict(heads=1025), dict(head_dim=96), dict(head_dim=0),
       dict(page_size=0), dict(page_size=8), dict(page_size=24), dict(page_size=8192), dict(reserved=(ctypes.c_int32 * 4)(0, 1))]


@pytest.mark.parametrize("bad", BAD, ids=lambda d: "-".join(d))
def test_descriptions_that_are_refused(bad):
    d = kv(**bad)
    status = 2 if set(bad) & {"dtype", "head_dim"} else 1
    assert hq.hq_kv_page_bytes(d) == 0
    assert hq.hq_paged_attn_workspace_bytes(d, 1, 1024) == 0
    refused(status, hq.hq_kv_write, d, 1, 16, 1024, 16, 1024, 16, None, 4, 16)
    refused(status, hq.hq_kv_read, d, 1, 16, None, 4, 16, 16, 1024, 16, 1024)
    refused(status, hq.hq_paged_attn, d, 1, 1024, 16, 8192, None, 4, 16, 16, 4, 16, 1.0, 0, 16, 8192, None, 16, 1 << 40)


def test_table_arguments():
    ok = dict(rot_dim=64, base=10000.0)
    call = lambda P=4, t=16, **kw: refused(kw.pop("status", 1), hq.hq_rope_table, hq.RopeDesc(**dict(ok, **kw)), P, t)  # noqa: E731
    for bad in (dict(rot_dim=0), dict(rot_dim=63), dict(rot_dim=1026), dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")),
                dict(amplitude=-1.0), dict(amplitude=float("nan")), dict(interleaved=2), dict(scaling=1), dict(scaling=1, factor=float("nan")),
                dict(scaling=2, factor=2.0, context=4, low=1.0, high=1.0), dict(scaling=2, factor=2.0, low=1.0, high=4.0),
                dict(scaling=3, factor=2.0, context=4, low=0.0, high=1.0), dict(scaling=3, factor=-2.0, context=4, low=1.0, high=2.0)):
        call(**bad)
    call(status=2, scaling=4, factor=2.0)
    call(P=-1)
    call(t=None)
    call(t=20)
    hq.hq_rope_table(hq.RopeDesc(**ok), 0, None, stream=0)


def test_table_amplitudes():
    for a in (float("inf"), 1e30):
        refused(1, hq.hq_rope_table, hq.RopeDesc(rot_dim=64, base=10000.0, amplitude=a), 4, 16)


def test_rope_arguments():
    good = dict(T=2, H=2, D=64, x=16, xt=128, xh=64, pos=16, table=16, P=8, out=32, ot=128, oh=64)

    def call(rope=hq.RopeDesc(rot_dim=64), **kw):
        a = dict(good, **kw)
        hq.hq_rope(rope, a["T"], a["H"], a["D"], a["x"], a["xt"], a["xh"], a["pos"], a["table"], a["P"], a["out"],
                   a["ot"], a["oh"], stream=0)

    for bad in (dict(T=-1), dict(H=0), dict(D=60), dict(D=1032), dict(D=0), dict(x=24), dict(x=None), dict(pos=None), dict(table=None),
                dict(table=20), dict(P=0), dict(out=None), dict(out=40), dict(xt=127), dict(xh=-64), dict(ot=4), dict(oh=12),
                dict(rope=hq.RopeDesc(rot_dim=66)), dict(rope=hq.RopeDesc(rot_dim=7)), dict(rope=hq.RopeDesc(rot_dim=64, interleaved=3)),
                dict(out=16, ot=256), dict(ot=64), dict(oh=0), dict(oh=32), dict(ot=0, oh=128), dict(pos=18), dict(H=65537),
                dict(T=1 << 30, H=4)):
        with pytest.raises(hq.HQError) as e:
            call(**bad)
        assert e.value.status == 1, bad
    call(T=0, x=None, out=None)


def test_rope_output_layouts_that_do_not_overlap():
    import torch
    if torch.cuda.is_available():
        pytest.skip("would run")
    for strides in ((128, 64), (64, 128), (64, 4096)):  # heads within tokens, tokens within heads
        refused(7, hq.hq_rope, hq.RopeDesc(rot_dim=64), 2, 2, 64, 16, 0, 0, 16, 16, 8, 1 << 20, *strides)


def test_write_and_read_arguments():
    w = lambda d=OK, T=1, k=16, ks=1024, v=16, vs=1024, slots=16, g=None, n=4, pages=16: (d, T, k, ks, v, vs, slots, g, n, pages)  # noqa: E731
    for bad in (dict(T=-1), dict(k=None), dict(v=None), dict(k=8), dict(v=24), dict(ks=1020), dict(vs=-8), dict(slots=None), dict(n=0),
                dict(slots=20), dict(T=1 << 29), dict(pages=None), dict(pages=8), dict(g=16), dict(d=kv(dtype=hq.HQ_NVFP4)),
                dict(d=kv(dtype=hq.HQ_NVFP4), g=18)):
        refused(1, hq.hq_kv_write, *w(**bad))
    hq.hq_kv_write(*w(T=0, k=None, v=None, slots=None, pages=None), stream=0)
    r = lambda d=OK, T=1, slots=16, g=None, n=4, pages=16, k=16, ks=1024, v=16, vs=1024: (d, T, slots, g, n, pages, k, ks, v, vs)  # noqa: E731
    for bad in (dict(T=-1), dict(slots=None), dict(k=None, v=None), dict(k=8), dict(v=8), dict(ks=4), dict(vs=-8), dict(n=0),
                dict(slots=12), dict(T=2, ks=1016), dict(T=2, vs=0), dict(pages=None), dict(g=16), dict(d=kv(dtype=hq.HQ_NVFP4))):
        refused(1, hq.hq_kv_read, *r(**bad))
    hq.hq_kv_read(*r(T=0, slots=None, pages=None, k=None, v=None), stream=0)


def test_rope_write_arguments():
    rope = hq.RopeDesc(rot_dim=128)
    names = ["rope", "kv", "T", "Hq", "q", "qs", "qo", "qos", "k", "ks", "v", "vs", "pos", "table", "P", "slots", "g", "n", "pages"]
    good = dict(zip(names, [rope, OK, 1, 8, 16, 1024, 16, 1024, 16, 1024, 16, 1024, 16, 16, 4, 16, None, 4, 16]))
    for bad in (dict(rope=hq.RopeDesc(rot_dim=130)), dict(rope=hq.RopeDesc(rot_dim=0)), dict(Hq=-1), dict(q=None), dict(qo=None),
                dict(q=8), dict(qs=4), dict(qos=-8), dict(qos=2048), dict(qo=32, T=2, qos=512), dict(pos=17), dict(pos=None), dict(table=None), dict(table=20), dict(P=0),
                dict(Hq=0), dict(k=None), dict(slots=None), dict(pages=None)):
        refused(1, hq.hq_rope_kv_write, *dict(good, **bad).values())
    hq.hq_rope_kv_write(*dict(good, T=0).values(), stream=0)


def test_attention_arguments():
    names = ["kv", "B", "Hq", "q", "qs", "g", "n", "pages", "pt", "most", "lens", "scale", "window", "out", "os", "lse", "ws", "wsb"]
    need = hq.hq_paged_attn_workspace_bytes(OK, 4, 32)
    assert need > 0
    good = dict(zip(names, [OK, 4, 32, 16, 4096, None, 9, 16, 16, 7, 16, 0.1, 0, 16, 4096, None, 16, need]))
    for bad in (dict(B=-1), dict(B=1 << 21), dict(Hq=0), dict(Hq=4), dict(Hq=33), dict(q=None), dict(q=8), dict(qs=4), dict(g=16), dict(n=0),
                dict(pages=None), dict(pages=8), dict(pt=None), dict(most=0), dict(most=1 << 27), dict(pt=18), dict(lens=18), dict(lse=18), dict(os=2048), dict(os=0), dict(lens=None), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(window=-1), dict(out=None), dict(out=8), dict(os=-8), dict(os=12),
                dict(kv=kv(dtype=hq.HQ_NVFP4))):
        refused(1, hq.hq_paged_attn, *dict(good, **bad).values())
    for bad in (dict(ws=None), dict(ws=8), dict(wsb=need - 1)):
        refused(3, hq.hq_paged_attn, *dict(good, **bad).values())
    hq.hq_paged_attn(*dict(good, B=0, q=None, pt=None, lens=None, out=None, ws=None).values(), stream=0)
    assert hq.hq_paged_attn_workspace_bytes(OK, 4, 33) == 0


def test_attention_scales_that_overflow_in_base_2():
    need = hq.hq_paged_attn_workspace_bytes(OK, 1, 8)
    for scale in (2.5e38, -3e38):
        refused(1, hq.hq_paged_attn, OK, 1, 8, 16, 1024, None, 4, 16, 16, 4, 16, scale, 0, 16, 1024, None, 16, need)


def test_tensors_that_are_not_on_the_device_are_refused():
    import torch
    t = torch.zeros(4, 64)
    refused(1, hq.hq_rope_table, hq.RopeDesc(rot_dim=64, base=10000.0), 4, t)


def test_index_tensors_of_another_width_are_refused():
    import torch
    i32, i64 = torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)
    refused(1, hq.hq_kv_write, OK, 1, 16, 1024, 16, 1024, i32, None, 4, 16)
    refused(1, hq.hq_kv_read, OK, 1, i32, None, 4, 16, 16, 1024, 16, 1024)
    refused(1, hq.hq_rope, hq.RopeDesc(rot_dim=64), 1, 1, 64, 16, 64, 64, i64, 16, 4, 32, 64, 64)
    need = hq.hq_paged_attn_workspace_bytes(OK, 1, 8)
    refused(1, hq.hq_paged_attn, OK, 1, 8, 16, 1024, None, 4, 16, 16, 4, i64, 1.0, 0, 16, 1024, None, 16, need)
    refused(1, hq.hq_paged_attn, OK, 1, 8, 16, 1024, None, 4, 16, torch.zeros(2, 4, dtype=torch.int32).t(), 4, 16, 1.0, 0, 16,
            1024, None, 16, need)


class OnDevice:
    """A host tensor that says it is on the current device (nothing is launched here: no tokens, no sequences)."""
    def __init__(self, t):
        self.t, self.dtype = t, t.dtype

    def get_device(self):
        return 0

    def data_ptr(self):
        return 4096

    def is_contiguous(self):
        return self.t.is_contiguous()


def test_tensors_of_another_type_are_refused(monkeypatch):
    """An lse or a table of 16 bits would be written past its end, rows of 16 other bits would be misread."""
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    t = lambda dtype, *shape: OnDevice(torch.zeros(shape or (4,), dtype=dtype))  # noqa: E731
    bf, f32, f16, f64, i32, i64, u8 = (t(x) for x in (torch.bfloat16, torch.float32, torch.float16, torch.float64, torch.int32,
                                                      torch.int64, torch.uint8))
    strided = OnDevice(torch.zeros(4, 8)[:, ::2])
    rope = hq.RopeDesc(rot_dim=64, base=10000.0)
    nv = kv(dtype=hq.HQ_NVFP4)

    def both(fn, good, *bad):
        fn(*good, stream=0)
        for at, x in bad:
            args = list(good)
            args[at] = x
            refused(1, fn, *args)

    both(hq.hq_rope_table, (rope, 0, f32), (2, f16), (2, f64), (2, bf), (2, strided))
    both(hq.hq_rope, (rope, 0, 1, 64, bf, 64, 64, i32, f32, 4, bf, 64, 64), (4, f16), (4, f32), (10, f16), (8, f16), (8, f64),
         (7, i64), (8, strided))
    both(hq.hq_kv_write, (nv, 0, bf, 1024, bf, 1024, i64, f32, 4, u8), (2, f16), (4, f32), (6, i32), (7, bf), (7, f64))
    both(hq.hq_rope_kv_write, (rope, nv, 0, 8, bf, 1024, bf, 1024, bf, 1024, bf, 1024, i32, f32, 4, i64, f32, 4, u8), (4, f16),
         (6, f32), (8, f16), (10, f16), (12, i64), (13, f16), (15, i32), (16, f16))
    both(hq.hq_kv_read, (nv, 0, i64, f32, 4, u8, bf, 1024, bf, 1024), (2, i32), (3, f64), (6, f16), (8, f32))
    both(hq.hq_paged_attn, (nv, 0, 32, bf, 4096, f32, 4, u8, i32, 4, i32, 1.0, 0, bf, 4096, f32, u8, 1 << 30), (3, f16), (5, f16),
         (8, i64), (10, i64), (13, f32), (15, f16), (15, f64), (15, strided))
    bits = t(torch.int16)  # the bits of bf16 pass, as elsewhere in the library
    hq.hq_rope(rope, 0, 1, 64, bits, 64, 64, i32, f32, 4, bits, 64, 64, stream=0)

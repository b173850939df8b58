"""The 4-bit KV cache without a GPU: the 64-bit reference's own pins (hand-derived rows and places) and the
refusals of the entry points, which come before any device access."""
import ctypes

import pytest
import torch

import kv4_ref as ref
import mixed_precision_quantized_mixq_b200 as mq
from mixed_precision_quantized_mixq_b200 import build as mqbuild


@pytest.fixture(scope="module")
def lib():
    mqbuild.build()
    return mq.lib()


# ------------------------------------------------------------- reference pins
def test_quantize_by_hand():
    # 0..15 in steps of 1: s = 1, codes are the values; shifted and scaled by powers of two
    x = torch.arange(16.0).repeat(4)
    for a, b in ((1, 0), (0.25, -2), (8, 32)):
        codes, s, lo = ref.quantize((x * a + b).half())
        assert codes.tolist() == x.long().tolist() and s.item() == a and lo.item() == b
    # halves go to the even code: 0, 0.5 -> 0, 1.5 -> 2, 2.5 -> 2, 15
    codes, s, _ = ref.quantize(torch.tensor([0, 0.5, 1.5, 2.5, 14.5, 15] + [0] * 58).half())
    assert s.item() == 1 and codes[:6].tolist() == [0, 0, 2, 2, 14, 15]
    # a constant row: s = 0, codes 0, the row is lo
    codes, s, lo = ref.quantize(torch.full((64,), -3.5).bfloat16())
    assert s.item() == 0 and lo.item() == -3.5 and codes.sum() == 0
    for bad in (float("nan"), float("inf"), -float("inf")):
        y = torch.ones(64).half()
        y[5] = bad
        _, s, lo = ref.quantize(y)
        assert torch.isnan(s).all() and torch.isnan(lo).all()
    # finite ends whose distance is not
    y = torch.zeros(64).bfloat16()
    y[0], y[1] = 3e38, -3e38
    assert torch.isnan(ref.quantize(y)[1]).all()


@pytest.mark.parametrize("D", [64, 128])
def test_places_cover_a_record_once(D):
    seen = set()
    for place, lo, hi in ((ref.k_place, 0, 8 * D), (ref.v_place, 8 * D, 16 * D)):
        for tok in range(16):
            for dim in range(D):
                byte, shift = place(tok, dim, D)
                assert lo <= byte < hi and shift in (0, 4)
                seen.add((byte, shift))
    assert len(seen) == 2 * 16 * D
    # by hand: dim 11 of token 3 is the odd one of pair 1 of word 1 -> nibble 5; V: byte column 5, quad 1, byte 2
    assert ref.k_place(3, 11, D) == (3 * D // 2 + 4 + 2, 4)
    assert ref.v_place(3, 11, D) == (8 * D + 5 * 64 + 16 + 0 + 2, 4)
    assert ref.v_place(8, 16, D) == (8 * D + 4 + 1, 0)


def test_reference_round_trip():
    g = torch.Generator().manual_seed(0)
    for dtype in (torch.float16, torch.bfloat16):
        pages = ref.Pages(torch.zeros((3, 2, ref.page_bytes(32, 64)), dtype=torch.uint8), 32, 64, dtype)
        table = torch.tensor([2, 0])
        k, v = (torch.randn((40, 2, 64), generator=g).to(dtype) for _ in range(2))
        for i in range(40):
            pages.write(table, i, k[i], v[i])
        for h in range(2):
            for x, y in zip((k, v), pages.rows(table, range(40), h)):
                c, s, lo = ref.quantize(x[:, h])
                assert torch.equal(y, c.double() * s.double() + lo.double())
                # no value is further off than half a step, the clamp at 15 (s is rounded) and fp32
                step = s.double() * (0.5 + 15 * torch.finfo(dtype).eps / 2 + 2.0 ** -19)
                assert bool(((y - x[:, h].double()).abs() <= step).all())


def test_reference_attention_by_hand():
    # one key: its V row; two equal keys: the mean; window 1: the last one; sinks: the first too
    pages = ref.Pages(torch.zeros((1, 1, ref.page_bytes(16, 64)), dtype=torch.uint8), 16, 64, torch.float16)
    table = torch.tensor([[0]])
    k = torch.zeros((3, 1, 64)).half()
    v = torch.stack([torch.full((1, 64), float(i)) for i in (1, 2, 6)]).half()
    for i in range(3):
        pages.write(table[0], i, k[i], v[i])
    q = torch.ones((1, 2, 64)).half()
    for n, window, sinks, want in ((1, 0, 0, 1), (2, 0, 0, 1.5), (3, 0, 0, 3), (3, 1, 0, 6), (3, 1, 1, 3.5),
                                   (3, 2, 9, 3), (0, 0, 0, 0)):
        out, _ = ref.attention(pages, q, table, [n], None, 0.125, window, sinks)
        assert torch.allclose(out, torch.full_like(out, want))


# ------------------------------------------------------------------- refusals
def test_page_bytes(lib):
    assert lib.mixq_kv4_page_bytes(64, 128) == 64 * 136
    assert lib.mixq_kv4_page_bytes(16, 64) == 16 * 72
    for p, d in ((0, 128), (-16, 128), (24, 128), (64, 96), (64, 256)):
        assert lib.mixq_kv4_page_bytes(p, d) == 0


def test_workspace_size(lib):
    size = lib.mixq_kv4_attention_workspace_size
    assert size(96, 1, 148) == 0 and size(128, -1, 148) == 0
    for d in (64, 128):
        assert 0 < size(d, 1, 148) == size(d, 32, 148) < size(d, 33, 148) == size(d, 0, 148)
        assert size(d, 1, 148) % 16 == 0
    assert size(64, 1, 148) < size(128, 1, 148)


def _desc(**kw):
    f = dict(pages=0x10000, page_stride=8 * 64 * 136, n_pages=4, page_size=64, n_kv_heads=8, head_dim=128, dtype=0)
    f.update(kw)
    return mq._KV4Desc(*[f[n] for n, _ in mq._KV4Desc._fields_])


BAD_CACHE = [(dict(dtype=2), 1), (dict(head_dim=96), 2), (dict(page_size=24), 2), (dict(page_size=0), 2),
             (dict(n_kv_heads=0), 2), (dict(n_pages=-1), 2), (dict(page_stride=8 * 64 * 136 - 16), 1),
             (dict(page_stride=8 * 64 * 136 + 8), 1), (dict(pages=0), 1), (dict(pages=0x10008), 3)]
# k/v or q/out pointers and strides, batch
BAD_ROWS = [(dict(a=0), 1), (dict(a=0x20004), 3), (dict(a_row=1020), 1), (dict(a_head=-8), 1), (dict(b=0), 1),
            (dict(b=0x30002), 3), (dict(n_seqs=-1), 2), (dict(n_rows=-1), 2), (dict(n_rows=9), 1),
            (dict(width=-1), 1), (dict(stride=3), 1), (dict(table=0), 1), (dict(lens=0), 1), (dict(cache=False), 1)]


def _args(**kw):
    a = dict(cache=True, a=0x20000, a_row=1024, a_head=128, b=0x30000, b_row=1024, b_head=128, n_seqs=8, n_rows=8,
             table=0x40000, width=4, stride=4, lens=0x50000, cu=None)
    a.update(kw)
    return a


def _append(lib, desc, **kw):
    x = _args(**kw)
    return lib.mixq_kv4_append(ctypes.byref(desc) if x["cache"] else None, x["a"], x["a_row"], x["a_head"], x["b"],
                               x["b_row"], x["b_head"], x["n_seqs"], x["n_rows"], x["table"], x["width"], x["stride"],
                               x["lens"], x["cu"], None, None)


def _read(lib, desc, **kw):
    x = _args(**kw)
    return lib.mixq_kv4_read(ctypes.byref(desc) if x["cache"] else None, x["a"], x["a_row"], x["a_head"], x["b"],
                             x["b_row"], x["b_head"], x["n_seqs"], x["n_rows"], x["table"], x["width"], x["stride"],
                             x["lens"], x["cu"], None, None)


def _attend(lib, desc, heads=8, max_new=0, scale=0.1, window=0, sinks=0, work=0x60000, work_bytes=1 << 30, **kw):
    x = _args(**kw)
    return lib.mixq_kv4_attention(ctypes.byref(desc) if x["cache"] else None, x["a"], x["a_row"], x["a_head"], x["b"],
                                  x["b_row"], x["b_head"], heads, x["n_seqs"], x["n_rows"], max_new, x["table"],
                                  x["width"], x["stride"], x["lens"], x["cu"], scale, window, sinks, work, work_bytes,
                                  None, None)


@pytest.mark.parametrize("change,status", BAD_CACHE)
def test_bad_cache(lib, change, status):
    for call in (_append, _read, _attend):
        assert call(lib, _desc(**change)) == status, lib.mixq_last_error()


@pytest.mark.parametrize("change,status", BAD_ROWS)
def test_bad_rows(lib, change, status):
    for call in (_append, _read, _attend):
        if call is _read and "lens" in change:
            continue  # read without first positions starts at 0
        assert call(lib, _desc(), **change) == status, lib.mixq_last_error()


def test_bad_attention(lib):
    for change, status in ((dict(heads=12), 2), (dict(heads=0), 2), (dict(scale=float("nan")), 1),
                           (dict(scale=float("inf")), 1), (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(max_new=-1), 1),
                           (dict(work=0), 1), (dict(work=0x60004), 3), (dict(b=0x20000), 1), (dict(b_row=120), 1),
                           (dict(b_head=64), 1)):
        assert _attend(lib, _desc(), **change) == status, (change, lib.mixq_last_error())
    assert _read(lib, _desc(), b_row=64) == 1 and _read(lib, _desc(), a_head=64) == 1


def test_no_rows_is_no_launch(lib):
    for call in (_append, _read, _attend):
        assert call(lib, _desc(), n_seqs=0, n_rows=0) == 0
        assert call(lib, _desc(), n_rows=0, cu=0x70000) == 0


def test_binding_refusals(lib):
    pages = torch.zeros((4, 2, 16 * 72), dtype=torch.uint8)
    with pytest.raises(mq.MixqError):
        mq.KV4Cache(pages, 16, 128)
    with pytest.raises(mq.MixqError):
        mq.KV4Cache(pages.to(torch.int8), 16, 64)
    with pytest.raises(mq.MixqError):
        mq.KV4Cache(pages, 16, 64, torch.float32)
    with pytest.raises(mq.MixqError):
        mq.KV4Cache(pages.transpose(0, 1)[:, :, ::2], 8, 64)
    cache = mq.KV4Cache(pages, 16, 64)
    k = torch.zeros((3, 2, 64)).half()
    table, lens, cu = torch.zeros((3, 2), dtype=torch.int32), torch.ones(3, dtype=torch.int32), torch.arange(4, dtype=torch.int32)
    for bad in (dict(k=k.float()), dict(k=k[:, :1]), dict(k=k[:2]), dict(table=table[0]), dict(table=table.long()),
                dict(lens=lens[:2]), dict(lens=lens.long()), dict(cu=cu[:3]), dict(k=k[:2], v=k[:2]),
                dict(v=torch.zeros((3, 2, 128)).half()[..., ::2]), dict(cu=torch.arange(8, dtype=torch.int32)[::2])):
        a = dict(k=k, v=k, table=table, lens=lens, cu=None)
        a.update(bad)
        with pytest.raises(mq.MixqError) as e:
            mq.kv4_append(a["k"], a["v"], cache, a["table"], a["lens"], cu_new=a["cu"])
        assert e.value.status == 1
    for call in (lambda: mq.kv4_append(k, k, cache, table, lens), lambda: mq.kv4_read(cache, table, None, 3),
                 lambda: mq.kv4_attention(k, cache, table, lens)):
        with pytest.raises(mq.MixqError) as e:  # a cache on the CPU: no fallback
            call()
        assert e.value.status == 6

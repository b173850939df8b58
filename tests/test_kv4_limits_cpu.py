"""Arguments of the 4-bit KV cache calls that the binding refuses because they could not reach the library as they were
given: tables whose rows overlap, numbers past 32 bits, a cache that was changed under its descriptor."""
import pytest
import torch

import mixed_precision_quantized_mixq_b200 as mq


@pytest.fixture()
def cache():
    return mq.KV4Cache(torch.zeros((4, 2, 16 * 72), dtype=torch.uint8), 16, 64)


def rows(n):
    return torch.zeros((n, 2, 64)).half()


def refused(call):
    with pytest.raises(mq.MixqError) as e:
        call()
    return e.value.status


def test_a_table_whose_rows_overlap_is_refused(cache):
    """One row of a table given to every sequence has stride 0: with the row's width for a stride the call would read
    past the tensor.  (A cache on the CPU is refused with status 6 when all else is right.)"""
    lens = torch.ones(3, dtype=torch.int32)
    flat = torch.zeros(40, dtype=torch.int32)
    for table in (flat[:4].expand(3, 4), flat.as_strided((3, 4), (2, 1)), flat.as_strided((3, 4), (3, 1)), flat[:1].expand(3, 1)):
        assert refused(lambda: mq.kv4_append(rows(3), rows(3), cache, table, lens)) == 1
        assert refused(lambda: mq.kv4_read(cache, table, None, 3)) == 1
        assert refused(lambda: mq.kv4_attention(rows(3), cache, table, lens)) == 1
    for table in (flat.as_strided((3, 4), (4, 1)), flat.as_strided((3, 4), (9, 1)), flat.as_strided((3, 0), (0, 1))):
        assert refused(lambda: mq.kv4_attention(rows(3), cache, table, lens)) == 6
    assert refused(lambda: mq.kv4_attention(rows(1), cache, flat[:4].expand(1, 4), lens[:1])) == 6
    assert refused(lambda: mq.kv4_attention(rows(1), cache, flat.as_strided((1, 4), (0, 1)), lens[:1])) == 6


def test_numbers_past_32_bits_are_refused(cache):
    """The C call takes 32-bit integers: 2**32 + 5 would arrive as 5."""
    table, lens = torch.zeros((3, 2), dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    for name in ("window", "sinks", "max_new"):
        for value in (2 ** 31, 2 ** 32, 2 ** 32 + 5, -1, -2 ** 32 + 5, 1 << 70):
            assert refused(lambda: mq.kv4_attention(rows(3), cache, table, lens, **{name: value})) == 1, (name, value)
        for value in (0, 1, 2 ** 31 - 1):
            assert refused(lambda: mq.kv4_attention(rows(3), cache, table, lens, **{name: value})) == 6, (name, value)
    for size in (2 ** 32 + 16, -16, 2 ** 31):
        assert refused(lambda: mq.KV4Cache(torch.zeros((0, 2, 5), dtype=torch.uint8), size, 64)) == 1


def test_workspace_sizes_of_any_bound(monkeypatch):
    """The size for many rows is asked for without a bound, so that neither a bound past 32 bits nor one that is not
    allowed is remembered as a size of 0 for the calls after it."""
    asked = []

    class Lib:
        @staticmethod
        def mixq_kv4_attention_workspace_size(head_dim, max_rows, num_sms):
            n = _c_int(max_rows)
            asked.append(n)
            return 0 if n < 0 else 1000 if 0 < n <= 32 else 3000

    class Cache:
        _torch, _index, head_dim, device = torch, 77, 64, torch.device("cpu")

    def _c_int(x):  # as ctypes passes it
        return (x + 2 ** 31) % 2 ** 32 - 2 ** 31

    import contextlib
    monkeypatch.setattr(mq, "lib", lambda: Lib)
    monkeypatch.setattr(mq, "_kv4_work_bytes", {})
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch, "empty", lambda n, **kw: n)
    for bad in (-1, -2 ** 32 + 5):
        assert refused(lambda: mq.kv4_workspace(Cache, bad)) == 1
    for bound, size in ((2 ** 31 + 3, 3000), (2 ** 32 + 3, 3000), (33, 3000), (0, 3000), (32, 1000), (1, 1000)):
        assert mq.kv4_workspace(Cache, bound) == size, bound
    assert all(n >= 0 for n in asked)


def test_a_cache_keeps_what_its_descriptor_says(cache):
    """The library reads the descriptor made with the cache; pages put in later would not be used, and the old ones
    might be gone."""
    for name, value in (("pages", torch.zeros((4, 2, 16 * 72), dtype=torch.uint8)), ("page_size", 32), ("head_dim", 128),
                        ("dtype", torch.bfloat16), ("n_kv_heads", 1), ("device", torch.device("cuda"))):
        with pytest.raises(AttributeError):
            setattr(cache, name, value)
    with pytest.raises(AttributeError):
        del cache.pages
    cache.layer = 3  # what a user adds is the user's


def test_stall_call_refusals():
    desc = mq._KV4Desc(0x10000, 2 * 16 * 72, 4, 16, 2, 64, 0)
    import ctypes
    call = lambda d, status: mq.lib().mixq_debug_kv4_stall(  # noqa: E731
        None if d is None else ctypes.addressof(d), 0x20000, 0x30000, 2, 1, 1, 0x40000, 4, 0x50000, None, 0x60000, 1 << 30, status, None)
    assert call(None, 0x70000) == 1 and call(desc, None) == 1
    for change in ({"head_dim": 128}, {"dtype": 1}):
        other = mq._KV4Desc(0x10000, 2 * 16 * 136, 4, 16, 2, change.get("head_dim", 64), change.get("dtype", 0))
        assert call(other, 0x70000) == 2

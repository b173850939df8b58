"""The 4-bit KV cache calls at the ends of what they allow: batches with a bad length or bad offsets among good ones,
bytes that no token has written, values at the ends of the types, the largest positions, batches and prompts of many
blocks, and long contexts.  Plain 64-bit forms are in kv4_ref.py."""
import pytest
import torch

import kv4_ref as ref
import mixed_precision_quantized_mixq_b200 as mq
from test_gpu_kv4 import attend, ints, make, offsets, randn

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def env():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mq.lib()


# ------------------------------------------------- bad sequences among good ones
@pytest.mark.parametrize("lens", [[16, 49], [40, 49], [49, 40], [30, 20, 10, 48, 49], [3] * 299 + [49], [3] * 299 + [-1],
                                  [49] + [3] * 299, [3] * 260 + [49] + [3] * 300])
@pytest.mark.parametrize("group", [1, 40])
def test_a_bad_length_is_reported_wherever_it_is(lens, group):
    """A length that the table (48 tokens) cannot hold, or a negative one, at any place of a batch; rows of a kv head on
    the kernel for few rows (1) and on the one for many (40)."""
    D, page, n_kv = 64, 16, 2
    good = [n if 0 <= n <= 48 else 48 for n in lens]
    pages, table, g = make(51, good, n_kv, D, page, F16, width=3)
    cache = mq.KV4Cache(pages.cuda(), page, D, F16)
    q = randn(g, (len(lens), n_kv * group, D), F16)
    status = mq.status_tensor()
    mq.kv4_attention(q.cuda(), cache, table.cuda(), ints(good), status=status)
    mq.check_status(status)
    out = mq.kv4_attention(q.cuda(), cache, table.cuda(), ints(lens), status=status)
    assert int(status.item()) == 1
    first = [i for i, (a, b) in enumerate(zip(lens, good)) if a == b][:4]
    want, tol = ref.attention(ref.Pages(pages, page, D, F16), q[first], table[first], [good[i] for i in first], None, D ** -0.5)
    ref.assert_close(out[first], want, tol)


@pytest.mark.parametrize("cu", [[0, 2, 4, 3], [0, 2, 4, 7], [0, 2, -1, 4], [0, 4, 2, 4], [-1, 2, 3, 4], [0, 0, 0, 1 << 30],
                                list(range(300)) + [298], [0] * 299 + [300, 299]])
@pytest.mark.parametrize("hint", [1, 0])
def test_bad_offsets_are_reported_by_attention(cu, hint):
    """Offsets that fall or leave the rows, at any place of a batch, by the kernel for few rows alone (hint 1) and by
    both.  Sequences that are in order and share no row with others keep their results."""
    D, page, n_kv, heads = 64, 16, 2, 24
    n, rows = len(cu) - 1, max(4, min(len(cu) - 1, 300))
    lens = [20] * n
    pages, table, g = make(52, lens, n_kv, D, page, F16)
    cache = mq.KV4Cache(pages.cuda(), page, D, F16)
    q = randn(g, (rows, heads, D), F16)
    status = mq.status_tensor()
    out = torch.full(q.shape, 5.0, dtype=F16, device="cuda")
    mq.kv4_attention(q.cuda(), cache, table.cuda(), ints(lens), ints(cu), max_new=hint, out=out, status=status)
    assert int(status.item()) == 1
    good = [s for s in range(n) if 0 <= cu[s] <= cu[s + 1] <= rows]
    owners = [sum(cu[s] <= r < cu[s + 1] for s in good) for r in range(rows)]
    assert all(bool((out[r] == 5).all()) for r in range(rows) if owners[r] == 0)
    host = ref.Pages(pages, page, D, F16)
    for s in [s for s in good if cu[s + 1] > cu[s]][:3]:
        r = range(cu[s], cu[s + 1])
        if all(owners[i] == 1 for i in r):
            want, tol = ref.attention(host, q[r.start:r.stop], table[s:s + 1], lens[s:s + 1], [0, len(r)], D ** -0.5)
            ref.assert_close(out[r.start:r.stop], want, tol, f"sequence {s}")


FALLS = [([0, 64, 10, 20], 64), ([0, 1000, 0, 16], 1000), ([0, 40, 80, 40], 80), ([0, 64, 20, 64], 64),
         ([0, 100, 60, 99, 100], 100), ([0] + [500] * 40 + [0, 3], 500), ([0, -40, 5, 6], 64), ([0, 3, 1 << 20, 2], 8),
         ([0] * 200 + [90, 50, 90], 90)]


@pytest.mark.parametrize("cu,rows", FALLS)
def test_falling_offsets_are_reported_by_append_and_read(cu, rows):
    """Offsets that fall by more than two records' rows, so that the record numbers of the sequences fall too."""
    D, page, n_kv = 64, 64, 2
    n = len(cu) - 1
    width = -(-(rows + 8) // page)
    pages = torch.zeros((n * width, n_kv, page * (D + 8)), dtype=torch.uint8, device="cuda")
    cache = mq.KV4Cache(pages, page, D, F16)
    table = torch.arange(n * width, dtype=torch.int32, device="cuda").view(n, width)
    k = torch.randn((rows, n_kv, D), device="cuda").half()
    lens = ints([8 + max(0, min(b, rows) - max(a, 0)) for a, b in zip(cu, cu[1:])])
    status = mq.status_tensor()
    mq.kv4_append(k, k, cache, table, lens, ints(cu), status=status)
    assert int(status.item()) == 1
    status.zero_()
    mq.kv4_read(cache, table, ints(cu), rows, status=status)
    assert int(status.item()) == 1


# ------------------------------------------------------- bytes that no token wrote
@pytest.mark.parametrize("dtype,s,lo", [(F16, -60000.0, -60000.0), (F16, -5000.0, 0.0), (F16, 60000.0, 60000.0),
                                        (BF16, -1e38, -1e38), (BF16, -3e37, 0.0), (BF16, 1e38, 1e38)])
@pytest.mark.parametrize("new", [None, [1, 150], [37, 90]])
@pytest.mark.parametrize("D", [64, 128])
def test_pairs_behind_the_last_token_may_be_any_bytes(dtype, s, lo, new, D):
    """Finite pairs whose values leave the type, in the unwritten rest of the last record."""
    page, lens = 32, [37, 150]

    def rest(host, table, q):
        pair = torch.tensor([s, lo]).to(dtype).view(torch.uint8)
        for b, n in enumerate(lens):
            for pos in range(n, -(-n // page) * page):
                at = pos % page // 16 * 16 * (D + 8) + 16 * D + 4 * (pos % 16)
                for o in (0, 64):
                    host.p[int(table[b, pos // page]), :, at + o:at + o + 4] = pair

    out, _ = attend(53, lens, new, 8, 2, D, page, dtype, prepare=rest)
    assert bool(torch.isfinite(out).all())


# ------------------------------------------------------------ the type's largest values
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [None, [20, 150]])
def test_rows_that_reach_the_largest_value(new, D):
    """fp16 V rows up to +-65504: s is rounded, so 15 s + lo can be above it, and is held there as in reading back.  Each
    query sees one key (window 1), then all.  With one key the weights cancel but for their own rounding on the kernel
    for many rows (2^-12 of the weight and 2^-12 of the result); 2^-10 of 65504 is twice their sum."""
    page, n_kv, lens, top = 16, 2, [40, 150], 65504.0
    g = torch.Generator().manual_seed(54)
    pages, table, _ = make(54, lens, n_kv, D, page, F16)
    n = sum(lens)
    v = torch.rand((n, n_kv, D), generator=g) * 1000
    v[:, 0, 3], v[:, 1, D - 1] = top, top
    v[:, :, 7] = -torch.arange(n)[:, None] * 97.0  # lo, of every residue
    v[::3, :, 9] = -top
    k, v = randn(g, v.shape, F16), v.half()
    over = ref.quantize(v)
    assert bool((15 * over[1].double() + over[2].double() >= 65520).any())  # rounds to infinity
    cache, t, cu_all = mq.KV4Cache(pages.cuda(), page, D, F16), table.cuda(), ints(offsets(lens))
    mq.kv4_append(k.cuda(), v.cuda(), cache, t, ints(lens), cu_all)
    _, back = mq.kv4_read(cache, t, cu_all, n)
    assert bool(torch.isfinite(back).all())
    rows = [1, 1] if new is None else new
    q = randn(g, (sum(rows), 2 * n_kv, D), F16)
    cu = None if new is None else ints(offsets(rows))
    one = mq.kv4_attention(q.cuda(), cache, t, ints(lens), cu, window=1)
    every = mq.kv4_attention(q.cuda(), cache, t, ints(lens), cu)
    assert bool(torch.isfinite(one).all()) and bool(torch.isfinite(every).all())
    at = [offsets(lens)[s] + lens[s] - rows[s] + i for s in range(2) for i in range(rows[s])]
    want = back[at].repeat_interleave(2, 1).float()
    assert (one.float() - want).abs().max().item() <= 2.0 ** -10 * top


# ------------------------------------------------------------------ the last positions
@pytest.mark.parametrize("dtype,new,group,window,sinks", [
    (F16, [1, 1], 1, 300, 4), (F16, [1, 1], 1, 5, 0), (BF16, [1, 1], 8, 31, 40), (F16, [40, 3], 2, 300, 4), (BF16, [70, 1], 1, 7, 0),
    (F16, [3, 200], 1, 130, 200), (BF16, [90, 40], 4, 1, 1)])
def test_positions_up_to_the_last_that_a_sequence_can_have(dtype, new, group, window, sinks):
    """Lengths of 2^31 - 256 and a little less under a window, over a table that names few pages again and again; a
    longer one is reported and cut."""
    D, page = 64, 1 << 20
    lens = [2 ** 31 - 256, 2 ** 31 - 256 - 77]
    g = torch.Generator().manual_seed(55)
    pages, _, _ = make(55, [page], 1, D, page, dtype, spare=1)
    table = (torch.arange(2 * 2048).view(2, 2048) * 7 // 5 % 2).int()
    q = randn(g, (sum(new), group, D), dtype)
    cu = None if new == [1, 1] else offsets(new)
    cache, t = mq.KV4Cache(pages.cuda(), page, D, dtype), table.cuda()
    status = mq.status_tensor()
    out = mq.kv4_attention(q.cuda(), cache, t, ints(lens), None if cu is None else ints(cu), window=window, sinks=sinks,
                           status=status)
    mq.check_status(status)
    host, at = ref.Pages(pages, page, D, dtype), offsets(new)
    for s in range(2):
        # the same keys as a short sequence: its first `sinks` positions, then the last ones
        from_ = lens[s] - new[s] - window
        pos = list(range(sinks)) + list(range(from_, lens[s]))
        k, v = host.rows(table[s], pos, 0)
        pos = torch.tensor(pos)
        for i in range(new[s]):
            p = lens[s] - new[s] + i
            seen = (pos <= p) & ((pos > p - window) | (pos < sinks))
            x = q[at[s] + i].double()
            o = torch.softmax(x @ k[seen].T * D ** -0.5, -1) @ v[seen]
            # weights and V rows rounded once each to at least the type, and the result: 3 half steps of the largest
            # |v|, 4 with what the scores and sums lose
            tol = 4 * torch.finfo(dtype).eps / 2 * v[seen].abs().max().item()
            assert (out[at[s] + i].double().cpu() - o).abs().max().item() <= tol, (s, i)
    for bad in (2 ** 31 - 255, 2 ** 31 - 1):
        status.zero_()
        mq.kv4_attention(q.cuda(), cache, t, ints([bad, 100]), None if cu is None else ints(cu), window=window, sinks=sinks,
                         status=status)
        assert int(status.item()) == 1


# ------------------------------------------------------------ many blocks, long contexts
@pytest.mark.parametrize("dtype,D", [(F16, 64), (BF16, 128)])
def test_more_sequences_than_one_look_takes(dtype, D):
    """150 and 70 sequences on both kernels, some without rows or keys: the search for a CTA's part goes over several
    groups of 64."""
    g = torch.Generator().manual_seed(57)
    for n, most in ((150, 40), (70, 70)):
        new = torch.randint(0, most, (n,), generator=g).tolist()
        new[::7] = [0] * len(new[::7])
        new[3::11] = [1] * len(new[3::11])
        lens = [m + int(x) for m, x in zip(new, torch.randint(0, 30, (n,), generator=g))]
        lens[5] = 0
        attend(57, lens, new, 3, 1, D, 16, dtype, window=20 if n == 70 else 0, sinks=2)


def test_more_blocks_of_rows_than_one_look_takes():
    """A sequence with 9600 and one with 17000 rows of a kv head, 38 and 67 blocks of 256, between short ones."""
    attend(58, [20, 140, 3], [5, 150, 1], 64, 1, 64, 16, F16)
    attend(59, [170, 9], [170, 2], 100, 1, 64, 16, BF16, window=50)


@pytest.mark.parametrize("rows,heads", [(1, 1), (1, 8), (1, 16), (40, 2)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("length", [2000, 131071])
def test_error_over_long_contexts(rows, heads, dtype, length):
    """The error's RMS against what rounding the exact result gives, which is one unit: u = 0.72 2^-11 / sqrt(3) of the
    result's RMS for fp16 (half a step, evenly spread, over a binade), 8 u for bf16.  V is N(0, 1), its rows' lo about
    -2.6, so the codes' part of a row has a mean square of 1 + 2.6^2 = 7.8 against the row's 1.
    Few rows: the weights go in as two fp16 parts for fp16 (2^-22: nothing), and sums lose less than a unit: 1.5 units in
    all; one part would be sqrt(1 + 7.8) = 3.  For bf16 one part is sqrt(7.8) / 8 of a unit and cut-off sums half of one:
    sqrt(1 + 0.12 + 0.25) = 1.17, held to 1.25.
    Many rows: weights and V rows rounded once each to fp16 add a unit each for fp16, sqrt(3) = 1.73, held to 1.9; for
    bf16 1/8 of a unit each, 1.02, held to 1.1."""
    D, page = 128, 128
    g = torch.Generator().manual_seed(60)
    n = -(-length // page)
    cache = mq.KV4Cache.empty(n, 1, D, page, dtype)
    table = torch.randperm(n, generator=g).int()[None]
    k, v, q = randn(g, (length, 1, D), dtype), randn(g, (length, 1, D), dtype), randn(g, (rows, heads, D), dtype)
    k[..., ::16] *= 6
    t, lens = table.cuda(), ints([length])
    mq.kv4_append(k.cuda(), v.cuda(), cache, t, lens, ints([0, length]))
    out = mq.kv4_attention(q.cuda(), cache, t, lens, ints([0, rows])).double().cpu()
    kk, vv = ref.Pages(cache.pages.cpu(), page, D, dtype).rows(table[0], range(length), 0)
    z = q.double().flatten(0, 1) @ kk.T * D ** -0.5
    first = length - rows + torch.arange(rows).repeat_interleave(heads)
    z.masked_fill_(torch.arange(length) > first[:, None], float("-inf"))
    want = (torch.softmax(z, -1) @ vv).view(rows, heads, D)
    unit = (want.to(dtype).double() - want).square().mean().sqrt()
    most = (1.5 if dtype == F16 else 1.25) if rows * heads <= 32 else (1.9 if dtype == F16 else 1.1)
    assert ((out - want).square().mean().sqrt() / unit).item() <= most


# ------------------------------------------------------------------- waits that run out
@pytest.mark.parametrize("new", [[1, 1, 1], [1, 40, 1], [300, 129, 64]])
def test_stalled_attention_times_out_with_status(new):
    """The test variants, whose work never comes, end by themselves with the status, on the kernel for few rows, on both
    and on the one for many; calls after them are right."""
    D, page, n_kv, heads = 64, 16, 2, 4
    lens = [5000, 2100, 900]
    pages, table, g = make(56, lens, n_kv, D, page, F16)
    cache, t, cu, n = mq.KV4Cache(pages.cuda(), page, D, F16), table.cuda(), ints(offsets(new)), ints(lens)
    q = randn(g, (sum(new), heads, D), F16).cuda()
    before = mq.kv4_attention(q, cache, t, n, cu)
    work, out, status = mq.kv4_workspace(cache), torch.empty_like(q), mq.status_tensor()
    for _ in range(2):
        status.zero_()
        mq._check(mq.lib().mixq_debug_kv4_stall(cache._ref, q.data_ptr(), out.data_ptr(), heads, 3, sum(new), t.data_ptr(),
                                                t.shape[1], n.data_ptr(), cu.data_ptr(), work.data_ptr(), work.nbytes,
                                                status.data_ptr(), torch.cuda.current_stream().cuda_stream))
        torch.cuda.synchronize()
        assert int(status.item()) == 5
    assert torch.equal(mq.kv4_attention(q, cache, t, n, cu, work=work), before)

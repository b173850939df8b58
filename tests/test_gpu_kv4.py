"""The 4-bit KV cache on the GPU against the plain 64-bit form in kv4_ref.py.

Codes, pairs and read-back rows are exact outputs (every step is decided in fp32 and rounded once), so their
tolerance is zero; attention is held to the elementwise bound that kv4_ref.attention derives."""
import pytest
import torch

import kv4_ref as ref
import mixed_precision_quantized_mixq_b200 as mq

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def env():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mq.lib()


def randn(g, shape, dtype, spread=1.0):
    return (torch.randn(shape, generator=g) * spread).to(dtype)


def make(seed, lens, n_kv, D, page, dtype, spare=2, width=None):
    """Random page bytes with finite pairs of ordinary size, and a shuffled table."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    width = max(need + [1]) if width is None else width
    total = sum(need) + spare
    pages = torch.randint(0, 256, (total, n_kv, page // 16, 16 * (D + 8)), generator=g, dtype=torch.uint8)
    s = torch.rand((total, n_kv, page // 16, 32), generator=g) * 0.3 + 0.01
    lo = -7.5 * s + torch.randn(s.shape, generator=g) * 0.2
    pairs = torch.stack([s, lo], -1).to(dtype).flatten(-2).view(torch.uint8)
    pages[..., 16 * D:] = pairs
    order = torch.randperm(total, generator=g).int()
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return pages.flatten(2), table, g


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def offsets(new):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return cu


# -------------------------------------------------------------------- append
APPEND = [
    # dtype, D, page, kv heads, stored before, new rows (None: a row each)
    (F16, 128, 16, 1, [0], [1]),
    (F16, 128, 64, 9, [0, 15, 16, 17, 63, 64, 200], None),
    (BF16, 64, 48, 3, [5, 0, 31], None),
    (F16, 128, 32, 2, [0, 3, 40], [70, 0, 29]),
    (BF16, 128, 16, 8, [1, 15, 16, 0, 0, 7], [1, 1, 16, 0, 33, 18]),
    (F16, 64, 128, 5, [120, 9], [150, 7]),
    (BF16, 64, 16, 17, [2] * 40, [(i * 7) % 5 for i in range(40)]),
]


@pytest.mark.parametrize("dtype,D,page,n_kv,ctx,new", APPEND)
@pytest.mark.parametrize("fused", [False, True])
def test_append(dtype, D, page, n_kv, ctx, new, fused):
    rows = [1] * len(ctx) if new is None else new
    lens = [c + n for c, n in zip(ctx, rows)]
    pages, table, g = make(1, lens, n_kv, D, page, dtype)
    T = sum(rows)
    pad = 3 if new is not None else 0  # rows behind the last sequence
    if fused:
        qkv = randn(g, (T + pad, 2 + 2 * n_kv, D), dtype)
        qkv[:, 2:2 + n_kv, :4] *= 9
        dev = qkv.cuda()
        k, v = qkv[:, 2:2 + n_kv], qkv[:, 2 + n_kv:]
        kd, vd = dev[:, 2:2 + n_kv], dev[:, 2 + n_kv:]
    else:
        k, v = randn(g, (T + pad, n_kv, D), dtype, 4.0), randn(g, (T + pad, n_kv, D), dtype, 0.01)
        kd, vd = k.cuda(), v.cuda()
    want = ref.Pages(pages.clone(), page, D, dtype)
    cu = offsets(rows)
    for s in range(len(ctx)):
        for i in range(rows[s]):
            want.write(table[s], ctx[s] + i, k[cu[s] + i], v[cu[s] + i])
    cache = mq.KV4Cache(pages.cuda(), page, D, dtype)
    status = mq.status_tensor()
    mq.kv4_append(kd, vd, cache, table.cuda(), ints(lens), None if new is None else ints(cu), status=status)
    mq.check_status(status)
    got = cache.pages.cpu()
    assert torch.equal(got, want.p), f"{int((got != want.p).sum())} bytes differ"


def special_rows(D, dtype):
    f = torch.finfo(dtype)
    g = torch.Generator().manual_seed(3)
    base = torch.randn((1, D), generator=g)
    rows = [torch.zeros(D), torch.full((D,), -2.5), torch.full((D,), -0.0), base[0] * f.tiny, base[0] * 1e-3,
            torch.linspace(-1, 1, D), torch.arange(D) % 16 - 8.0, torch.arange(D) % 31 / 2.0]
    for big in (f.max, -f.max):
        r = base[0].clone()
        r[7] = big
        rows.append(r)
    r = base[0].clone()
    r[0], r[D - 1] = f.max / 4, -f.max / 4
    rows.append(r)
    for bad in (float("nan"), float("inf"), -float("inf")):
        for at in (0, D // 2 + 1, D - 1):
            r = base[0].clone()
            r[at] = bad
            rows.append(r)
    r = base[0].clone()
    r[1], r[2] = f.max, -f.max  # the distance of the ends is finite in fp32 for fp16, not for bf16
    rows.append(r)
    r = torch.zeros(D)
    r[3] = f.smallest_normal * f.eps  # the smallest subnormal
    rows.append(r)
    return torch.stack(rows).to(dtype)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
def test_append_and_read_special_rows(dtype, D):
    x = special_rows(D, dtype)
    n = len(x)
    k, v = torch.stack([x, x.flip(0)], 1), torch.stack([x.roll(1, 0), x], 1)
    pages, table, _ = make(2, [n], 2, D, 16, dtype)
    want = ref.Pages(pages.clone(), 16, D, dtype)
    for i in range(n):
        want.write(table[0], i, k[i], v[i])
    cache = mq.KV4Cache(pages.cuda(), 16, D, dtype)
    mq.kv4_append(k.cuda(), v.cuda(), cache, table.cuda(), ints([n]), ints([0, n]))
    kr, vr = mq.kv4_read(cache, table.cuda(), ints([0, n]), n)
    for h in range(2):
        for rows, got in zip(want.rows(table[0], range(n), h), (kr, vr)):
            exp = rows.float().clamp(max=torch.finfo(dtype).max).to(dtype)
            g = got[:, h].cpu()
            assert torch.equal(torch.isnan(g), torch.isnan(exp))
            assert torch.equal(torch.nan_to_num(g), torch.nan_to_num(exp))
    # bytes too, except the codes of rows that stand for NaN (they mean nothing)
    got = ref.Pages(cache.pages.cpu(), 16, D, dtype)
    for h in range(2):
        for a, b in zip(got.scales(table[0], range(n), h), want.scales(table[0], range(n), h)):
            assert torch.equal(torch.nan_to_num(a, nan=7.0), torch.nan_to_num(b, nan=7.0))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_append_at_every_range(dtype):
    """Rows from 0 to each positive value of the type: every quotient by 15 and every reciprocal of a scale that
    rows can have, bit for bit."""
    D = 64
    top = torch.arange(1, 0x7C00 if dtype == F16 else 0x7F80, dtype=torch.int16).view(dtype)
    g = torch.Generator().manual_seed(9)
    part = torch.rand((len(top), D), generator=g)
    part[:, 0], part[:, 1] = 0.0, 1.0
    part[:, 2:18] = torch.arange(16) / 15.0 + 1 / 30  # near the borders between codes
    x = (part.clamp(max=1.0) * top.float()[:, None]).to(dtype)
    n = len(top)
    cache = mq.KV4Cache.empty(-(-n // 128), 1, D, 128, dtype)
    table = torch.arange(cache.pages.shape[0], dtype=torch.int32, device="cuda")[None]
    mq.kv4_append(x[:, None].cuda(), x[:, None].flip(0).contiguous().cuda(), cache, table, ints([n]), ints([0, n]))
    codes, s, lo = ref.quantize(x)
    host = ref.Pages(cache.pages.cpu(), 128, D, dtype)
    raw = host.p[:, 0].reshape(-1, 16 * (D + 8))[:-(-n // 16)]
    tok, dim = torch.arange(16)[:, None], torch.arange(D)[None]
    for place, at, flip in ((ref.k_place, 16 * D, False), (ref.v_place, 16 * D + 64, True)):
        byte, shift = place(tok, dim, D)
        got = (raw[:, byte].long() >> shift & 15).reshape(-1, D)[:n]
        pair = raw[:, at:at + 64].contiguous().view(dtype).reshape(-1, 2)[:n]
        want = (codes.flip(0), s.flip(0), lo.flip(0)) if flip else (codes, s, lo)
        assert torch.equal(pair[:, :1], want[1]) and torch.equal(pair[:, 1:], want[2])
        assert torch.equal(got, want[0]), f"{int((got != want[0]).sum())} codes differ"


def test_append_leaves_out_negative_positions_and_bad_offsets():
    D, page, n_kv = 128, 16, 2
    pages, table, g = make(4, [20, 20, 20], n_kv, D, page, F16)
    k, v = randn(g, (3, n_kv, D), F16), randn(g, (3, n_kv, D), F16)
    want = ref.Pages(pages.clone(), page, D, F16)
    want.write(table[1], 4, k[1], v[1])
    cache = mq.KV4Cache(pages.cuda(), page, D, F16)
    status = mq.status_tensor()
    mq.kv4_append(k.cuda(), v.cuda(), cache, table.cuda(), ints([0, 5, -3]), status=status)  # padded entries: length 0
    mq.check_status(status)
    assert torch.equal(cache.pages.cpu(), want.p)
    # three new rows at length 2: only the last two have a position
    want.write(table[0], 0, k[1], v[1])
    want.write(table[0], 1, k[2], v[2])
    mq.kv4_append(k.cuda(), v.cuda(), cache, table.cuda(), ints([2, 0, 0]), ints([0, 3, 3, 3]), status=status)
    mq.check_status(status)
    assert torch.equal(cache.pages.cpu(), want.p)
    for cu in ([0, 2, 1, 1], [0, 1, 2, 4], [-1, 0, 0, 0]):
        status.zero_()
        mq.kv4_append(k[:0].new_zeros((3, n_kv, D)).cuda(), v.cuda(), cache, table.cuda(), ints([0, 0, 0]), ints(cu),
                      status=status)
        assert int(status.item()) == 1, cu
    assert torch.equal(cache.pages.cpu(), want.p)


@pytest.mark.parametrize("bad", [-1, 7, 1 << 30])
def test_bad_pages_are_reported_and_left_alone(bad):
    D, page, n_kv, n = 64, 16, 2, 40
    pages, table, g = make(5, [n], n_kv, D, page, F16, spare=4)  # 7 pages
    assert pages.shape[0] == 7
    table[0, 1] = bad
    k, v = randn(g, (n, n_kv, D), F16), randn(g, (n, n_kv, D), F16)
    want = ref.Pages(pages.clone(), page, D, F16)
    for i in list(range(16)) + list(range(32, n)):
        want.write(table[0], i, k[i], v[i])
    cache = mq.KV4Cache(pages.cuda(), page, D, F16)
    status = mq.status_tensor()
    mq.kv4_append(k.cuda(), v.cuda(), cache, table.cuda(), ints([n]), ints([0, n]), status=status)
    assert int(status.item()) == 1
    assert torch.equal(cache.pages.cpu(), want.p)
    status.zero_()
    out = [torch.full((n, n_kv, D), 7.0, dtype=F16, device="cuda") for _ in range(2)]
    mq.kv4_read(cache, table.cuda(), ints([0, n]), n, k_out=out[0], v_out=out[1], status=status)
    assert int(status.item()) == 1
    assert bool((out[0][16:32] == 7).all()) and not bool((out[0][:16] == 7).all())
    # attention hides the tokens of the bad page
    status.zero_()
    q = randn(g, (1, 4, D), F16)
    got = mq.kv4_attention(q.cuda(), cache, table.cuda(), ints([n]), status=status)
    assert int(status.item()) == 1
    keep = list(range(16)) + list(range(32, n))
    for h in range(n_kv):
        kk, vv = want.rows(table[0].clamp(0, 6), keep, h)
        w = torch.softmax(q[0, 2 * h:2 * h + 2].double() @ kk.T * D ** -0.5, -1)
        assert torch.allclose(got[0, 2 * h:2 * h + 2].cpu().double(), w @ vv, atol=2e-3, rtol=2e-3)
    # a length that the table cannot hold
    status.zero_()
    mq.kv4_attention(q.cuda(), cache, table.clamp(0, 6).cuda(), ints([49]), status=status)
    assert int(status.item()) == 1


# ---------------------------------------------------------------------- read
@pytest.mark.parametrize("dtype,D,page,n_kv,first,rows", [
    (F16, 128, 16, 1, None, [1]), (BF16, 128, 64, 9, None, [100, 0, 17, 64]), (F16, 64, 48, 3, [0, 5, 40, 47], [40, 3, 30, 1]),
    (BF16, 64, 32, 17, [16, 1], [16, 90])])
def test_read(dtype, D, page, n_kv, first, rows):
    lens = [(0 if first is None else first[i]) + n for i, n in enumerate(rows)]
    pages, table, g = make(6, lens, n_kv, D, page, dtype)
    cu, T = offsets(rows), sum(rows)
    cache = mq.KV4Cache(pages.cuda(), page, D, dtype)
    host = ref.Pages(pages, page, D, dtype)
    both = torch.full((T + 2, 2 * n_kv + 1, D), 3.0, dtype=dtype, device="cuda")  # rows behind and a head between
    k, v = both[:, :n_kv], both[:, n_kv + 1:]
    status = mq.status_tensor()
    mq.kv4_read(cache, table.cuda(), ints(cu), T + 2, None if first is None else ints(first), k, v, status=status)
    mq.check_status(status)
    assert bool((both[T:] == 3).all()) and bool((both[:, n_kv] == 3).all())
    for s in range(len(rows)):
        at = range(lens[s] - rows[s], lens[s])
        for h in range(n_kv):
            for want, got in zip(host.rows(table[s], at, h), (k, v)):
                assert torch.equal(got[cu[s]:cu[s + 1], h].cpu(), want.float().to(dtype))


def test_read_single_rows():
    pages, table, _ = make(7, [40, 9, 33], 2, 128, 16, F16)
    cache = mq.KV4Cache(pages.cuda(), 16, 128, F16)
    k, v = mq.kv4_read(cache, table.cuda(), None, 3, first=ints([39, 0, 32]))
    host = ref.Pages(pages, 16, 128, F16)
    for s, p in enumerate((39, 0, 32)):
        for h in range(2):
            a, b = host.rows(table[s], [p], h)
            assert torch.equal(k[s, h].cpu(), a[0].float().half()) and torch.equal(v[s, h].cpu(), b[0].float().half())


# ----------------------------------------------------------------- attention
def attend(seed, lens, new, heads, n_kv, D, page, dtype, window=0, sinks=0, scale=None, max_new=0, spread=1.0,
           prepare=None, pad=0):
    rows = [1] * len(lens) if new is None else new
    pages, table, g = make(seed, lens, n_kv, D, page, dtype)
    cu = offsets(rows)
    q = randn(g, (sum(rows) + pad, heads, D), dtype, spread)
    host = ref.Pages(pages, page, D, dtype)
    if prepare:
        prepare(host, table, q)
    cache = mq.KV4Cache(pages.cuda(), page, D, dtype)
    out = torch.full(q.shape, 5.0, dtype=dtype, device="cuda")
    status = mq.status_tensor()
    mq.kv4_attention(q.cuda(), cache, table.cuda(), ints(lens), None if new is None else ints(cu), max_new, scale, window,
                     sinks, out=out, status=status)
    mq.check_status(status)
    scale = D ** -0.5 if scale is None else scale
    want, tol = ref.attention(host, q[:sum(rows)], table, lens, None if new is None else cu, scale, window, sinks)
    if pad:
        assert bool((out[sum(rows):] == 5).all()), "rows behind the last sequence were written"
    ref.assert_close(out[:sum(rows)], want, tol, f"lens {lens} new {new} heads {heads}/{n_kv} D {D} {dtype}")
    return out, want


STEP = [
    # lens, heads, kv heads, D, page, dtype
    ([1], 1, 1, 128, 16, F16),
    ([1, 2, 15, 16, 17, 31, 32, 33], 8, 1, 128, 16, BF16),
    ([0, 5, 0, 127, 128, 129, 0], 8, 2, 64, 32, F16),
    ([600, 77, 300], 32, 32, 128, 64, F16),
    ([600, 77, 1], 20, 4, 128, 48, BF16),
    ([513], 64, 8, 128, 128, F16),
    ([1025, 3], 24, 2, 64, 16, BF16),  # 12 rows a head: 16-row tiles
    ([70, 40], 71, 1, 64, 16, F16),    # 71 rows a head: several tiles
    ([2500], 3, 1, 128, 64, F16),
    ([3] * 300, 2, 1, 64, 16, F16),    # more sequences than one block looks at together
]


@pytest.mark.parametrize("lens,heads,n_kv,D,page,dtype", STEP)
def test_steps(lens, heads, n_kv, D, page, dtype):
    attend(11, lens, None, heads, n_kv, D, page, dtype)


CHUNK = [
    # lens, new, heads, kv heads, D, page, dtype
    ([5], [5], 4, 4, 128, 16, F16),
    ([40, 0, 133, 64], [1, 0, 133, 17], 8, 2, 128, 32, BF16),
    ([260, 129], [130, 128], 8, 1, 64, 64, F16),
    ([300, 33, 200], [300, 3, 90], 6, 2, 128, 16, F16),
    ([257], [257], 2, 2, 64, 48, BF16),
    ([700, 20], [140, 20], 5, 5, 128, 64, F16),
    ([500, 1], [4, 1], 16, 2, 128, 64, BF16),
    ([3100], [40], 2, 1, 64, 32, F16),    # one item over more CTAs than a join takes at once
    ([2600], [90], 3, 1, 128, 64, BF16),
]


@pytest.mark.parametrize("lens,new,heads,n_kv,D,page,dtype", CHUNK)
@pytest.mark.parametrize("hint", [False, True])
def test_chunks(lens, new, heads, n_kv, D, page, dtype, hint):
    attend(12, lens, new, heads, n_kv, D, page, dtype, max_new=max(new) if hint else 0, pad=3)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
def test_ragged_batches_of_prompts_on_both_kernels(dtype, D):
    """Batches whose blocks fill one row tile here and two there, so that a CTA takes both kinds in a row, against the
    kernel for few rows (which takes all of them under a wrong hint).  Either result is within half a step of the type
    of its own value, and weights and V rows are rounded once each to at least the type: for outputs and V rows of at
    most vmax that is 4 half steps of vmax.  Scratch and shared memory hold other calls' bytes between the runs."""
    n_kv, heads, page = 4, 12, 64
    g = torch.Generator().manual_seed(31)
    junk = mq.KV4Cache(torch.full((40, n_kv, page * (D + 8)), 255, dtype=torch.uint8, device="cuda"), page, D, dtype)
    step = torch.finfo(dtype).eps / 2
    for trial in range(12):
        new = torch.randint(1, 420, (9,), generator=g).tolist()
        new[trial % 9], new[(trial + 4) % 9] = 12, 900
        lens = [n + int(x) for n, x in zip(new, torch.randint(0, 40, (9,), generator=g))]
        pages, table, _ = make(40 + trial, lens, n_kv, D, page, dtype)
        cache, t, cu = mq.KV4Cache(pages.cuda(), page, D, dtype), table.cuda(), ints(offsets(new))
        q = randn(g, (sum(new), heads, D), dtype).cuda()
        want = mq.kv4_attention(q, cache, t, ints(lens), cu, max_new=1).float()
        _, v = mq.kv4_read(cache, t, ints(offsets(lens)), sum(lens))
        for _ in range(4):
            few = torch.arange(40, dtype=torch.int32, device="cuda").view(4, 10)
            mq.kv4_attention(q[:240], junk, few, ints([640] * 4), ints([0, 60, 120, 180, 240]))  # NaN pairs everywhere
            got = mq.kv4_attention(q, cache, t, ints(lens), cu).float()
            off = (got - want).abs().max().item() / v.float().abs().max().item()
            assert off <= 4 * step + 1e-5, (trial, off)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 0), (16, 4), (17, 3), (100, 20), (64, 64), (90, 500), (1000, 4)])
@pytest.mark.parametrize("new", [None, [1, 40, 129], [3, 2, 5]])
def test_windows(window, sinks, new):
    attend(13, [150, 64, 400], new, 8, 2, 64, 16, F16, window, sinks)
    attend(14, [20, 40, 333], new, 4, 2, 128, 32, BF16, window, sinks)


@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 2, 3), (5, 2 ** 31 - 1)])
def test_largest_windows_and_rows_before_the_start(window, sinks):
    attend(14, [150, 6, 40], None, 8, 2, 64, 16, F16, window, sinks)
    attend(14, [150, 6, 40], [3, 11, 2], 4, 2, 128, 16, BF16, window, sinks)
    attend(14, [150, 6], [70, 40], 4, 2, 128, 16, F16, window, sinks)


def test_sinks_without_a_window_change_nothing():
    a, _ = attend(15, [150, 64], None, 8, 2, 64, 16, F16)
    b, _ = attend(15, [150, 64], None, 8, 2, 64, 16, F16, sinks=9)
    assert torch.equal(a, b)


def test_a_wrong_hint_changes_no_result():
    for hint in (1, 2, 50, 100000):
        attend(16, [200, 90], [70, 9], 4, 2, 128, 16, F16, max_new=hint)


@pytest.mark.parametrize("lens,new", [([3, 2, 9], [5, 2, 1]), ([0, 1], [3, 4]), ([100], [140])])
def test_rows_without_a_visible_key_are_zeros(lens, new):
    out, want = attend(17, lens, new, 4, 2, 64, 16, F16)
    short = new[0] - lens[0]
    assert short > 0 and bool((out[:short] == 0).all())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("new", [None, [1, 150]])
def test_hidden_tokens_may_hold_anything(dtype, new):
    """NaN and infinite pairs behind the last key, before the window and in the future of earlier rows."""
    D, page = 128, 32
    lens = [37, 150]

    def poison(host, table, q):
        rec = 16 * (D + 8)
        inf = torch.tensor([float("inf")], dtype=dtype).view(torch.uint8)
        def put(s, pos):
            at = pos % page // 16 * rec + 16 * D + 4 * (pos % 16)
            for h in range(2):
                for o in (0, 64):
                    host.p[int(table[s, pos // page]), h, at + o:at + o + 4] = torch.cat([inf, inf]) if pos % 2 else 0xFF
        for pos in range(37, 64):
            put(0, pos)
        for pos in range(150, 160):
            put(1, pos)
        for pos in (4, 5, 6, 7):  # behind the sinks, before the window of the last rows
            put(0, pos)
        if new is None:
            for pos in (4, 20, 99):
                put(1, pos)
        else:
            put(1, 149)  # the last row alone sees it: NaN there and nowhere else

    out, want = attend(18, lens, new, 8, 2, D, page, dtype, window=20, sinks=4, prepare=poison)
    if new is None:
        assert not bool(torch.isnan(want).any())
    else:
        assert bool(torch.isnan(want[-1]).all()) and not bool(torch.isnan(want[:-1]).any())


def test_a_nan_query_stays_in_its_row():
    def prepare(host, table, q):
        q[1, 3, 17] = float("nan")
    out, want = attend(19, [90, 50], None, 8, 2, 128, 16, F16, prepare=prepare)
    assert int(torch.isnan(want).any(-1).sum()) == 1


@pytest.mark.parametrize("dtype,spread", [(F16, 30.0), (F16, 1e-6), (BF16, 1e-20), (BF16, 1e6), (F16, 1e-3)])
@pytest.mark.parametrize("new", [None, [3, 140]])
def test_query_magnitudes(dtype, spread, new):
    """Peaked and flat distributions; scale undoes half of the magnitude so that scores stay finite."""
    scale = min(0.088, 30.0 / spread) if spread > 1 else 0.088
    attend(20, [200, 140], new, 4, 2, 128, 16, dtype, scale=scale, spread=spread)


@pytest.mark.parametrize("factor", [2.0 ** -14, 1e-3, 500.0])
@pytest.mark.parametrize("new", [None, [3, 140]])
def test_value_scales_far_apart(factor, new):
    """V rows whose scales differ by up to 2^24 within a record and from record to record."""
    D, page = 128, 16

    def prepare(host, table, q):
        p = host.p.view(host.p.shape[0], 2, -1, 16 * (D + 8))
        pairs = p[..., 16 * D + 64:].contiguous().view(F16).view(*p.shape[:3], 16, 2)
        pairs[..., ::3, :] *= factor
        pairs[::2] *= 2.0 ** -6
        pairs[..., 5, 0] = 0.0
        p[..., 16 * D + 64:] = pairs.flatten(-2).view(torch.uint8)

    attend(21, [300, 140], new, 8, 2, D, page, F16, prepare=prepare)


@pytest.mark.parametrize("power", [-7, -10, -12, -14, -17, -20, 10, 13, 16])
def test_bf16_values_at_the_ends_of_fp16_range(power):
    """Single keys (outputs are V rows) whose scales and smallest values lie about the ends of fp16's range."""
    D, page = 64, 16

    def prepare(host, table, q):
        p = host.p.view(host.p.shape[0], 1, -1, 16 * (D + 8))
        pairs = p[..., 16 * D:].contiguous().view(BF16).view(*p.shape[:3], 2, 16, 2)
        pairs[..., 1, :, :] *= 2.0 ** power
        pairs[..., 1, ::2, 1] *= 2.0 ** -6
        pairs[..., 1, ::5, 0] = 0.0
        pairs[..., 1, ::3, 1] = 0.0
        p[..., 16 * D:] = pairs.flatten(-3).view(torch.uint8)

    attend(28, [90, 45], [90, 45], 2, 1, D, page, BF16, prepare=prepare, window=1)
    attend(29, [90, 45], [90, 45], 2, 1, D, page, BF16, prepare=prepare)


@pytest.mark.parametrize("new", [None, [3, 140, 260]])
@pytest.mark.parametrize("D", [64, 128])
def test_bf16_values_out_of_fp16_range(new, D):
    """V rows far above fp16's largest value and far below its smallest, whole records of them and single tokens,
    under scores that rise so that weights of both kinds are scaled again."""
    page = 32

    def prepare(host, table, q):
        p = host.p.view(host.p.shape[0], 2, -1, 16 * (D + 8))
        pairs = p[..., 16 * D:].contiguous().view(BF16).view(*p.shape[:3], 2, 16, 2)
        for b in range(table.shape[0]):
            for slot in range(int((table[b] >= 0).sum())):
                v = pairs[int(table[b, slot]), :, :, 1]
                kind = slot % 5
                if kind == 1:
                    v *= 2.0 ** 20
                elif kind == 2:
                    v *= 2.0 ** -30
                elif kind == 3:
                    v[:, 0, 7] *= 2.0 ** 18  # one token of the page's first record
                elif kind == 4:
                    v[:, 1, ::2] = 0.0
                if b == 1:
                    pairs[int(table[b, slot]), :, :, 0, :, 1] += 0.6 * slot  # K's lo
        p[..., 16 * D:] = pairs.flatten(-3).view(torch.uint8)
        q.abs_()

    attend(27, [300, 400, 260], new, 8, 2, D, page, BF16, prepare=prepare)


@pytest.mark.parametrize("new", [None, [2, 200]])
def test_rising_scores(new):
    """Scores that grow along the sequence move the running maximum in almost every record."""
    def prepare(host, table, q):
        q.fill_(1.0)
        D = host.D
        for s in range(table.shape[0]):
            for pos in range(host.page_size * int((table[s] >= 0).sum())):
                rec, tok = host._record(table[s], pos, 0)
                pair = torch.tensor([0.01, (0.09 * pos if s == 0 else -0.09 * pos)], dtype=F16)
                rec[16 * D + 4 * tok:16 * D + 4 * tok + 4] = pair.view(torch.uint8)
    attend(22, [600, 200], new, 8, 1, 64, 16, F16, prepare=prepare)


def test_strided_and_shared_pages():
    """Pages of a pool shared by layers, queries as part of a projection, an output with gaps, and two
    sequences that share their prefix's pages."""
    D, page, n_kv, heads = 128, 32, 2, 8
    lens = [100, 120]
    pages, table, g = make(23, lens, n_kv, D, page, F16)
    table[1, :3] = table[0, :3]
    pool = torch.randint(0, 256, (pages.shape[0], 3, *pages.shape[1:]), dtype=torch.uint8)
    pool[:, 1] = pages
    pool = pool.cuda()
    cache = mq.KV4Cache(pool[:, 1], page, D, F16)
    qkv = randn(g, (2, heads + 2 * n_kv, D), F16)
    qd = qkv.cuda()
    wide = torch.full((2, 2 * heads, D), 9.0, dtype=F16, device="cuda")
    wt = torch.full((2, table.shape[1] + 5), -7, dtype=torch.int32)
    wt[:, :table.shape[1]] = table
    wt = wt.cuda()
    mq.kv4_attention(qd[:, :heads], cache, wt[:, :table.shape[1]], ints(lens), out=wide[:, ::2])
    want, tol = ref.attention(ref.Pages(pages, page, D, F16), qkv[:, :heads], table, lens, None, D ** -0.5)
    ref.assert_close(wide[:, ::2], want, tol)
    assert bool((wide[:, 1::2] == 9).all())
    # and append through the same view leaves the other layers' bytes
    before = pool.clone()
    mq.kv4_append(qd[:, heads:heads + n_kv], qd[:, heads + n_kv:], cache, wt[:, :table.shape[1]], ints([101, 121]))
    assert torch.equal(pool[:, 0], before[:, 0]) and torch.equal(pool[:, 2], before[:, 2])
    assert not torch.equal(pool[:, 1], before[:, 1])


def test_equal_calls_give_equal_bits():
    pages, table, g = make(24, [3000, 17, 900], 4, 128, 64, F16)
    cache = mq.KV4Cache(pages.cuda(), 64, 128, F16)
    q, t, lens = randn(g, (3, 16, 128), F16).cuda(), table.cuda(), ints([3000, 17, 900])
    work = mq.kv4_workspace(cache)
    first = mq.kv4_attention(q, cache, t, lens, work=work)
    for i in range(20):
        work.random_(0, 256)  # what scratch held before means nothing
        assert torch.equal(mq.kv4_attention(q, cache, t, lens, work=work), first)


def test_streams_and_capture():
    """Two calls at once on two streams with their own scratch; a captured step replayed as the lengths grow."""
    D, page, n_kv, heads = 128, 16, 2, 8
    pages, table, g = make(25, [200, 200], n_kv, D, page, F16)
    t = table.cuda()
    cache = mq.KV4Cache(pages.cuda(), page, D, F16)
    q = randn(g, (2, heads, D), F16).cuda()
    lens = ints([150, 199])
    alone = mq.kv4_attention(q, cache, t, lens)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(10):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            outs.append(mq.kv4_attention(q, cache, t, lens, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, alone) for o in outs)

    k, v = randn(g, (2, n_kv, D), F16).cuda(), randn(g, (2, n_kv, D), F16).cuda()
    n = ints([10, 60])
    graph = torch.cuda.CUDAGraph()
    mq.kv4_append(k, v, cache, t, n)
    mq.kv4_attention(q, cache, t, n)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        n.add_(1)
        mq.kv4_append(k, v, cache, t, n)
        out = mq.kv4_attention(q, cache, t, n)
    for step in range(40):
        k.normal_()
        v.normal_()
        graph.replay()
        if step % 13 == 0:
            now = n.cpu().tolist()
            want, tol = ref.attention(ref.Pages(cache.pages.cpu(), page, D, F16), q.cpu(), table, now, None, D ** -0.5)
            ref.assert_close(out, want, tol, f"step {step}")
    assert n.cpu().tolist() == [50, 100]


def test_chunks_captured_and_on_two_streams():
    """A captured chunk replayed with other lengths and offsets, some sequences with one row and some with many, and
    the same call on two streams at once; against the kernel for few rows under a wrong hint, within the same 4 half
    steps of vmax as above."""
    D, page, n_kv, heads = 128, 32, 2, 8
    pages, table, g = make(33, [700] * 5, n_kv, D, page, F16)
    cache, t = mq.KV4Cache(pages.cuda(), page, D, F16), table.cuda()
    vmax = mq.kv4_read(cache, t, ints(offsets([700] * 5)), 3500)[1].float().abs().max().item()
    rows = 640
    q = randn(g, (rows, heads, D), F16).cuda()
    out = torch.zeros_like(q)
    lens, cu = ints([0] * 5), ints([0] * 6)
    work = mq.kv4_workspace(cache)
    mq.kv4_attention(q, cache, t, lens, cu, out=out, work=work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mq.kv4_attention(q, cache, t, lens, cu, out=out, work=work)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for new, full in (([300, 1, 200, 0, 139], [600, 700, 200, 5, 333]), ([1, 1, 1, 1, 1], [700, 20, 333, 1, 64]),
                      ([128, 129, 127, 256, 0], [128, 640, 700, 300, 0])):
        cu.copy_(ints(offsets(new)))
        lens.copy_(ints(full))
        n = sum(new)
        out.fill_(7.0)
        graph.replay()
        want = mq.kv4_attention(q, cache, t, lens, cu, max_new=1)
        assert (out[:n].float() - want[:n].float()).abs().max().item() <= (4 * 2.0 ** -11 + 1e-5) * vmax
        assert bool((out[n:] == 7).all())
        torch.cuda.synchronize()
        both = [mq.kv4_attention(q, cache, t, lens, cu, stream=s) for s in streams for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(o[:n], out[:n]) for o in both)


def test_offsets_past_32_bits():
    """Pages beyond 4 GiB from the start of the pool."""
    D, page, n_kv = 128, 128, 8
    pages, table, g = make(26, [300], n_kv, D, page, F16, spare=0)
    per = pages[0].numel()
    n = (5 << 30) // per
    pool = torch.zeros((n, *pages.shape[1:]), dtype=torch.uint8, device="cuda")
    far = torch.tensor([[n - 1, 0, n - 2]], dtype=torch.int32)
    for i in range(3):
        pool[far[0, i]] = pages[table[0, i]].cuda()
    cache = mq.KV4Cache(pool, page, D, F16)
    q = randn(g, (1, 16, D), F16)
    got = mq.kv4_attention(q.cuda(), cache, far.cuda(), ints([300]))
    host = ref.Pages(pages, page, D, F16)
    want, tol = ref.attention(host, q, table, [300], None, D ** -0.5)
    ref.assert_close(got, want, tol)
    k, v = randn(g, (40, n_kv, D), F16), randn(g, (40, n_kv, D), F16)
    mq.kv4_append(k.cuda(), v.cuda(), cache, far.cuda(), ints([320]), ints([0, 40]))
    kr, vr = mq.kv4_read(cache, far.cuda(), ints([0, 40]), 40, first=ints([280]))
    for i in range(40):
        host.write(table[0], 280 + i, k[i], v[i])
    for h in range(n_kv):
        a, b = host.rows(table[0], range(280, 320), h)
        assert torch.equal(kr[:, h].cpu(), a.float().half()) and torch.equal(vr[:, h].cpu(), b.float().half())
    del pool, cache
    torch.cuda.empty_cache()


def test_a_decoder_attention_block():
    """The calls as a model makes them: a quantized projection to q, k and v, append, attention over the cache and the
    quantized output projection, a ragged prompt first and then single steps.  The projections are the layer's own (their
    outputs are taken as they come); cache and attention are held to the 64-bit form on the same q, k, v."""
    D, heads, n_kv, hidden, page = 128, 4, 2, 256, 16
    g = torch.Generator().manual_seed(27)
    qkv_w = randn(g, ((heads + 2 * n_kv) * D, hidden), F16, 0.05).cuda()
    out_w = randn(g, (hidden, heads * D), F16, 0.05).cuda()
    idx = torch.tensor([3, 77], dtype=torch.int32, device="cuda")
    wq, wo = mq.prepack(qkv_w, idx, mq.MIXQ_W4G128), mq.prepack(out_w, idx, mq.MIXQ_W8)
    cache = mq.KV4Cache.empty(12, n_kv, D, page)
    table = torch.randperm(12, generator=g).int().view(2, 6)
    t, host = table.cuda(), ref.Pages(torch.zeros((12, n_kv, ref.page_bytes(page, D)), dtype=torch.uint8), page, D, F16)
    lens = [0, 0]
    status = mq.status_tensor()
    for new in ([37, 20], [1, 1], [1, 1], [1, 1]):
        cu = offsets(new)
        x = randn(g, (sum(new), hidden), F16).cuda()
        qkv, _ = mq.linear(x, wq, status=status)
        qkv = qkv.view(-1, heads + 2 * n_kv, D)
        q, k, v = qkv[:, :heads], qkv[:, heads:heads + n_kv], qkv[:, heads + n_kv:]
        lens = [a + b for a, b in zip(lens, new)]
        c = None if max(new) == 1 else ints(cu)
        mq.kv4_append(k, v, cache, t, ints(lens), c, status=status)
        o = mq.kv4_attention(q, cache, t, ints(lens), c, status=status)
        y, _ = mq.linear(o.view(-1, heads * D), wo, status=status)
        mq.check_status(status)
        for s in range(2):
            for i in range(new[s]):
                host.write(table[s], lens[s] - new[s] + i, k[cu[s] + i].cpu(), v[cu[s] + i].cpu())
        assert torch.equal(cache.pages.cpu(), host.p)
        want, tol = ref.attention(host, q.cpu(), table, lens, None if c is None else cu, D ** -0.5)
        ref.assert_close(o, want, tol)
        assert y.shape == (sum(new), hidden) and bool(torch.isfinite(y).all())

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

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

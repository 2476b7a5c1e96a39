"""Attention over the paged cache: what the kernels' arithmetic allows, not a share of the greatest value."""
import pytest
import torch

from test_paged_gpu import attend, make_cache, make_table, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_device):
    from exact_attention_72_gb300 import build
    build.build()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H", [1, 4, 5, 8, 12, 16])      # rows of a kv head: residuals in spare columns, in products of their own
def test_rounded_weights_do_not_show_where_terms_cancel(d, H):
    """Every value is zero + 15 scale = 0: what is left of the sum is the weights' rounding. Each weight is two fp16 numbers,
    2^-22 of itself, and passes some 64 fp32 roundings (products, sums of at most 60 keys, joins), of terms of 15 each. A matrix
    product may cut each of the 16 terms it adds, and the sum so far, at 24 bits of the greatest: 17 units of 2^-23. There are
    fewer tiles than warps, so that a part is one tile, 2 x 16 keys times two numbers: 4 products. Odd dims come out of
    (w (15 + 16 * 15) - w 15) / 16, sums of 17 instead of 15."""
    lens = [1, 2, 3, 7, 40, 60]
    table, pages = make_table(lens, 16, 1)
    cache = make_cache("int4", pages, 16, 1, d)
    cache.k.copy_(torch.randint(0, 256, cache.k.shape, generator=torch.Generator().manual_seed(2), dtype=torch.uint8).cuda())
    cache.k_sz[..., 0], cache.k_sz[..., 1] = 0.3, -2.25
    cache.v.fill_(255)
    cache.v_sz[..., 0], cache.v_sz[..., 1] = 1.0, -15.0
    o, _ = attend(randn((len(lens), 1, H, d), 3), cache, table, lens)
    assert float(o.float().abs().max()) <= 15 * (2.0 ** -22 + (64 + 4 * 17 * 17 / 15) * 2.0 ** -23)

"""Attention over the paged cache, value by value: what the kernels' arithmetic allows, not a share of the greatest value.

check_each, with t the terms a value is summed from (bf16: v; 4 bits: scale * code and zero apart) and A = sum_j P_j |t_j|:
  scores: fp32 sums of d exact products and a few operations: dS = 32 * 2^-23 of scale * sum|q||k| (4 bits: of |q| times
      |zero| + scale * code), the greatest over the keys; a weight moves by dS of itself, and so does their sum: 2 dS A.
  weights: two bf16 numbers, 2^-8 * 2^-8, or (times scale) two fp16 numbers, 2^-11 * 2^-11, of themselves. The second fp16
      number is 2^-25 off at least, where the group's greatest weight times scale is 2^3 or more (2^4 when it is set, at most
      one bit less after a move): 2^-28 of the group's greatest, 15 codes, for each key.
  sums: 64 fp32 roundings; a matrix product may cut each of the 16 terms it adds, and the sum so far, at 24 bits of the greatest,
      17 * 2^-23. The calls here have so few keys that a warp's share holds at most two tiles of 32 (16) keys: 8 products.
  output: bf16, 2^-8 of the value. LSE: dS and 2^-19 (1 + |LSE|).
"""
import numpy as np
import pytest
import torch

from oracle import paged
from test_paged_gpu import attend, make_cache, make_table, np32, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_device):
    from exact_attention_72_gb300 import build
    build.build()


def write(cache, table, rows):
    """rows: per sequence (k, v) float32 [n, Hkv, d], written as they are (quantised by the oracle). Per sequence
    (keys, values, sizes of the keys' and of the values' terms, codes' part of the latter), in fp64."""
    out = []
    for b, kv in enumerate(rows):
        n = len(kv[0])
        if not n:
            out.append(None)
            continue
        pg, at = (torch.tensor(x).cuda() for x in np.array([paged.place(table[b], p, cache.page_size) for p in range(n)]).T)
        got = []
        for t, sz, x in ((cache.k, cache.k_sz, kv[0]), (cache.v, cache.v_sz, kv[1])):
            if sz is None:
                x = paged.bf16_nearest(x)
                t[pg, at] = torch.tensor(x).cuda().bfloat16()
                got.append((np.float64(x), np.abs(np.float64(x)), np.zeros(x.shape)))
                continue
            codes, scale, zero = paged.quantise(x)
            t[pg, at] = torch.tensor(paged.pack(codes)).cuda()
            sz[pg, at] = torch.tensor(np.stack((scale, zero), -1)).cuda().bfloat16()
            got.append((paged.values(codes, scale, zero), paged.values(codes, np.abs(scale), np.abs(zero)),
                        np.repeat(15 * np.float64(scale), 64, -1)))
        out.append((got[0][0], got[1][0], got[0][1], got[1][1], got[1][2]))
    return out


def check_each(q, o, lse, held, scale, causal=True):
    qn, on, ln = (np.float64(np32(x)) for x in (q, o, lse))
    B, Nq, H, d = qn.shape
    for b in range(B):
        if held[b] is None:
            assert np.all(on[b] == 0) and np.all(np.isneginf(ln[b]))
            continue
        keys, vals, ksize, vsize, code = held[b]
        four = bool(code.any())
        n, Hkv = keys.shape[:2]
        for h in range(H):
            j = h // (H // Hkv)
            for i in range(Nq):
                m = n - Nq + i + 1 if causal else n
                if m <= 0:
                    assert np.all(on[b, i, h] == 0) and np.isneginf(ln[b, h, i])
                    continue
                S = scale * (keys[:m, j] @ qn[b, i, h])
                top = S.max()
                L = top + np.log(np.exp(S - top).sum())
                P = np.exp(S - L)
                dS = 32 * 2.0 ** -23 * abs(scale) * (ksize[:m, j] @ np.abs(qn[b, i, h])).max()
                want, A = P @ vals[:m, j], P @ vsize[:m, j]
                rel = 2.0 ** -22 if four else 2.0 ** -16
                room = 2.0 ** -8 * np.abs(want) + (rel + 2 * dS + (64 + 8 * 17) * 2.0 ** -23) * A
                if four:
                    room += m * 2.0 ** -28 * (P[:, None] * code[:m, j]).max(0)
                err = np.abs(on[b, i, h] - want)
                assert np.all(err <= room), (b, h, i, int((err / room).argmax()), float((err / room).max()))
                assert abs(ln[b, h, i] - L) <= dS + 2.0 ** -19 * (1 + abs(L))


def normal(r, *shape):
    return paged.bf16_nearest(r.standard_normal(shape).astype(np.float32))


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


@pytest.mark.parametrize("early", [False, True])
@pytest.mark.parametrize("bits", [10, 14, 17, 20, 60])
@pytest.mark.parametrize("d,H", [(128, 4), (128, 8), (128, 12), (256, 3), (256, 8)])
def test_a_small_group_keeps_its_bits_beside_a_large_one(d, H, bits, early):
    """The groups of every value row span a factor 2^bits, least first or last; with early, the first key has a score 8 above."""
    n = 3000
    r = np.random.default_rng(7)
    for order in (1, -1):
        table, pages = make_table([n], 16, 1)
        cache = make_cache("int4", pages, 16, 1, d)
        k, v = normal(r, n, 1, d), normal(r, n, 1, d)
        q = normal(r, 1, 1, 1, d) + 0.1 * normal(r, 1, 1, H, d)
        if early:
            k[0, 0] = paged.bf16_nearest(np.float32(8 * d ** 0.5 * q[0, 0, 0] / (q[0, 0, 0] @ q[0, 0, 0])))
        groups = d // 64
        v *= np.repeat(2.0 ** -np.round(bits * np.arange(groups) / (groups - 1)), 64)[::order].astype(np.float32)
        held = write(cache, table, [(k, v)])
        q = torch.tensor(q).bfloat16().cuda()
        o, lse = attend(q, cache, table, [n])
        check_each(q, o, lse, held, d ** -0.5)

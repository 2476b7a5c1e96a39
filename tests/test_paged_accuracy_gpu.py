"""Attention over the paged cache, value by value: what the kernels' arithmetic allows, not a share of the greatest value.

check_each, with t the terms a value is summed from (bf16: v; 4 bits: scale * code and zero apart) and A = sum_j P_j |t_j|:
  scores: fp32 sums of d exact products. A matrix product may cut each of the 16 terms it adds, and the sum so far, at 24 bits of
      the greatest: with 8 further roundings dS = (17 d / 16 + 8) * 2^-23 of scale * sum|q||k| (4 bits: of |q| times
      |zero| + scale * code), the greatest over the keys; a weight moves by dS of itself, and so does their sum: 2 dS A.
  weights: two bf16 numbers, 2^-8 * 2^-8, or (times scale) two fp16 numbers, 2^-11 * 2^-11, of themselves. The second fp16
      number is 2^-25 off at least, where the group's greatest weight times scale is 2^3 or more (2^4 when it is set, at most
      one bit less after a move): 2^-28 of the group's greatest, 15 codes, for each key.
  sums: 64 fp32 roundings, and 17 * 2^-23 a product. The calls here have so few keys that a warp's share holds at most two
      tiles of 32 (16) keys: 8 products.
  output: bf16, 2^-8 of the value. LSE: dS and 2^-19 (1 + |LSE|).
"""
import numpy as np
import pytest
import torch

from oracle import paged
from exact_attention_72_gb300 import binding
from test_paged_gpu import attend, i32, make_cache, make_table, np32, randn

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
                dS = (17 * d / 16 + 8) * 2.0 ** -23 * abs(scale) * (ksize[:m, j] @ np.abs(qn[b, i, h])).max()
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


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("d,H,Hkv,Nq", [(64, 4, 2, 1), (128, 8, 1, 1), (128, 4, 2, 3), (128, 16, 1, 1), (64, 12, 1, 1),
                                        (256, 4, 2, 1), (256, 12, 1, 1)])
def test_every_value(kind, d, H, Hkv, Nq):
    """Lengths from one token to units that are cut, each row by its own bound: a long sequence's small values, and what the
    second number of each weight leaves, show beside a short one's."""
    lens = [1, 33, 0, 6000, 200, 2, 900]
    table, pages = make_table(lens, 16, 4)
    cache = make_cache(kind, pages, 16, Hkv, d)
    r = np.random.default_rng(5)
    held = write(cache, table, [(normal(r, n, Hkv, d), normal(r, n, Hkv, d)) for n in lens])
    q = randn((len(lens), Nq, H, d), 6, 2.0)
    o, lse = attend(q, cache, table, lens)
    check_each(q, o, lse, held, d ** -0.5)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_every_row_of_prefill_and_decode_lies_where_it_belongs(kind):
    """Prompts, then tokens one at a time out of a captured graph: each row of the cache is the one that norm, rotation and (4
    bits) the oracle's quantisation give for its token, bit for bit, and what the last step attends to is those rows."""
    B, H, Hkv, d, ps, steps = 3, 6, 2, 128, 16, 19
    prompts = [37, 90, 0]
    table, pages = make_table([n + steps + 1 for n in prompts], ps, 4)
    cache = make_cache(kind, pages, ps, Hkv, d)
    a = np.arange(200)[:, None] * 10000.0 ** (-np.arange(d // 2) / (d // 2))
    cos, sin = (torch.tensor(f(a), dtype=torch.float32).cuda() for f in (np.cos, np.sin))
    w = [torch.ones(d, device="cuda") * 1.5, torch.ones(d, device="cuda") * 0.75]
    total = sum(prompts)
    x = randn((total, H + 2 * Hkv, d), 5)
    pos = i32(np.concatenate([np.arange(n) for n in prompts]))
    _, k = binding.attn_qk_norm_rope(x[:, :H], x[:, H:H + Hkv], cos, sin, pos, *w)
    tab, lens, cu1 = i32(table), i32(prompts), i32([0, 1, 2, 3])
    binding.attn_paged_append(cache, k, x[:, H + Hkv:], i32(np.concatenate(([0], np.cumsum(prompts)))), i32([0, 0, 0]), tab)
    x1 = torch.empty((B, H + 2 * Hkv, d), dtype=torch.bfloat16, device="cuda")

    def step():
        q1, k1 = binding.attn_qk_norm_rope(x1[:, :H], x1[:, H:H + Hkv], cos, sin, lens, *w)
        binding.attn_paged_append(cache, k1, x1[:, H + Hkv:], cu1, lens, tab)
        lens.add_(1)
        return q1, *binding.attn_fwd_paged(q1.unsqueeze(1), cache, tab, lens)
    news = [randn((B, H + 2 * Hkv, d), 100 + i) for i in range(steps)]
    x1.copy_(news[0])
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q1, o, lse = step()
    for new in news[1:]:
        x1.copy_(new)
        graph.replay()
    ends = [n + steps for n in prompts]
    assert lens.tolist() == ends
    got = binding.attn_paged_gather(cache, i32(np.concatenate(([0], np.cumsum(ends)))), tab, sum(ends))
    assert binding.attn_get_status()[0] == binding.ATTN_OK
    rows = [[np32(y[sum(prompts[:b]):sum(prompts[:b + 1])]) for b in range(B)] for y in (k, x[:, H + Hkv:])]
    for i, new in enumerate(news):
        _, k1 = binding.attn_qk_norm_rope(new[:, :H], new[:, H:H + Hkv], cos, sin, i32([n + i for n in prompts]), *w)
        for j, y in enumerate((k1, new[:, H + Hkv:])):
            rows[j] = [np.concatenate((old, np32(y[b:b + 1]))) for b, old in enumerate(rows[j])]
    held = []
    for b in range(B):
        one = []
        for j in range(2):
            here = np32(got[j][sum(ends[:b]):sum(ends[:b + 1])])
            if kind == "bf16":
                assert np.array_equal(here, rows[j][b]), (b, j)
                one.append((np.float64(rows[j][b]), np.abs(np.float64(rows[j][b])), np.zeros(rows[j][b].shape)))
            else:
                codes, scale, zero = paged.quantise(rows[j][b])
                value = paged.values(codes, scale, zero)
                assert np.array_equal(here, paged.bf16_nearest(np.float32(value))), (b, j)
                one.append((value, paged.values(codes, np.abs(scale), np.abs(zero)), np.repeat(15 * np.float64(scale), 64, -1)))
        held.append((one[0][0], one[1][0], one[0][1], one[1][1], one[1][2]))
    check_each(q1.unsqueeze(1), o, lse, held, d ** -0.5)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [40, 20000])     # finished by one warp, and cut over many
def test_a_bad_query_row_among_few_stays_one_row(d, n):
    """With at most 4 rows each holds two columns of the products."""
    table, pages = make_table([n], 16, 1)
    cache = make_cache("int4", pages, 16, 1, d)
    r = np.random.default_rng(8)
    held = write(cache, table, [(normal(r, n, 1, d), normal(r, n, 1, d))])
    q = randn((1, 1, 4, d), 5)
    bad = q.clone()
    bad[0, 0, 2, 7] = float("nan")
    o, lse = attend(bad, cache, table, [n])
    assert bool(torch.isnan(o[0, 0, 2]).all()) and bool(torch.isnan(lse[0, 2]).all())
    good, all_lse = attend(q, cache, table, [n])
    o[0, 0, 2], lse[0, 2] = good[0, 0, 2], all_lse[0, 2]
    check_each(q, o, lse, held, d ** -0.5)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("d,H,Hkv", [(128, 32, 8), (64, 32, 8), (128, 16, 2), (64, 24, 2), (256, 8, 4)])
def test_long_sums_do_not_drift(kind, d, H, Hkv):
    """Hundreds of tiles in every warp's share: 64 sequences of 65536 keys, 4096 of them over and over. Two
    neighbours have the same key, so the same weight, and the same values with the sign turned (4 bits: zero is -7.5 scale, codes c
    and 15 - c): O is 0, what is there is the sums' error. Round to nearest errs up as often as down: over N sums of size A it is
    sqrt(N) 2^-24 A in the mean square, and 4 times that is allowed. A cut towards 0 at each sum would be N 2^-25 A."""
    n, times, B = 4096, 16, 64
    table, pages = make_table([n], 64, 4, spare=0)
    cache = make_cache(kind, pages, 64, Hkv, d)
    r = np.random.default_rng(9)
    v = normal(r, n, Hkv, d)
    v[1::2] = -v[::2]
    k = normal(r, n, Hkv, d)
    k[1::2] = k[::2]
    held = write(cache, table, [(k, v)])[0]
    size = np.abs(v).mean(0)
    if kind == "int4":
        codes = torch.randint(0, 256, (n // 2, Hkv, d // 2), generator=torch.Generator().manual_seed(1), dtype=torch.uint8)
        scale = torch.randint(9, 16, (n // 2, Hkv, d // 64), generator=torch.Generator().manual_seed(2)) / 32
        pg, at = (torch.tensor(x).cuda() for x in np.array([paged.place(table[0], p, 64) for p in range(n)]).T)
        cache.v[pg, at] = torch.stack((codes, 255 - codes), 1).flatten(0, 1).cuda()
        cache.v_sz[pg, at] = torch.stack((scale, -7.5 * scale), -1).bfloat16().repeat_interleave(2, 0).cuda()
        size = np.full((Hkv, d), 15 * float(scale.mean()))      # zero and codes, 7.5 scale each; 4 bits of scale: both exact
    q = randn((B, 1, H, d), 6, 0.5)
    o, lse = attend(q, cache, np.tile(table, (B, times)), [n * times] * B)
    sums = B * Hkv * n * times / 16 / 1000      # at least 1000 warps; a sum for every 16 keys
    rows = np.float64(np32(o)).reshape(B, Hkv, H // Hkv, d)
    room = 4 * sums ** 0.5 * 2.0 ** -24 * np.sqrt((size ** 2).mean(-1))
    assert np.all(np.sqrt((rows ** 2).mean(-1)) <= room[None, :, None]), float((np.sqrt((rows ** 2).mean(-1)) / room[None, :, None]).max())
    for b, h in ((0, 0), (B - 1, H - 1)):
        S = d ** -0.5 * (held[0][:, h // (H // Hkv)] @ np.float64(np32(q[b, 0, h])))
        L = S.max() + np.log(np.exp(S - S.max()).sum()) + np.log(times)
        dS = (17 * d / 16 + 8) * 2.0 ** -23 * d ** -0.5 * (held[2][:, h // (H // Hkv)] @ np.abs(np.float64(np32(q[b, 0, h])))).max()
        assert abs(float(lse[b, h, 0]) - L) <= dS + 2.0 ** -19 * (1 + abs(L))

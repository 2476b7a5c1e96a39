"""Attention of chunks of new tokens over the paged cache, against the formula in 64 bits, value by value.

With P_j the weights, A = sum_j P_j |v_j|, a value may be off by (units of the value, derived from the kernels' roundings):
  scores: fp32 sums of d exact products (4 bits: d + 16 of them, of |scale| |c - 8| and |zero + 8 scale|). A matrix product may
      cut each of the 16 terms it adds, and the sum so far, at 24 bits of the greatest; 8 further roundings:
      dS = (17 (d + 16) / 16 + 8) 2^-23 scale sum |q| |k|, 4 bits 2^-21 more for a zero's and a query sum's two fp16 numbers and
      2^-31 for what fp16 loses of small values; a weight moves by dS of itself, and so does their sum: 2 dS A;
  weights: bf16, 2^-8 of themselves; over 4 bits fp16, 2^-11, and 2^-31 of the greatest weight times value of 32 keys for each key;
  values over 4 bits: fp16, 2^-11 of the value, 2^-11 of the zero - 16 scale that it is made from, and 2^-38 of the greatest of
      32 keys;
  sums: 64 fp32 roundings and 17 * 2^-23 for each product of 16 keys, of A;
  output: bf16, 2^-8 of the value. LSE: dS and 2^-19 (1 + |LSE|).
"""
import math

import numpy as np
import pytest
import torch

from oracle import paged
from exact_attention_72_gb300 import binding
from test_paged_gpu import i32, make_cache, make_table, ok, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_device):
    from exact_attention_72_gb300 import build
    build.build()
    binding.attn_debug_set(timeout_ns=500_000_000)
    yield
    binding.attn_debug_set()


def write(cache, table, lens, seed, k=None, v=None):
    """Random rows (or k, v: float32 per sequence [n, Hkv, d]) at every sequence's positions; the rest of the cache stays NaN.
    Per sequence (keys, values, sizes of the keys' terms and of the values', |zero - 16 scale| of the values) in fp64 on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for b, n in enumerate(lens):
        pos = np.arange(n)
        pg = torch.tensor(table[b][pos // cache.page_size].astype(np.int64)).cuda()
        at = torch.tensor(pos % cache.page_size).cuda()
        got = []
        for t, sz, given in ((cache.k, cache.k_sz, k), (cache.v, cache.v_sz, v)):
            shape = (n, cache.Hkv, cache.d)
            if sz is None:
                x = torch.randn(shape, generator=g, device="cuda") if given is None else given[b].cuda()
                t[pg, at] = x.bfloat16()
                x = t[pg, at].double()
                got.append((x, x.abs(), torch.zeros_like(x)))
                continue
            if given is None:
                codes = torch.randint(0, 16, shape, generator=g, device="cuda", dtype=torch.uint8)
                scale = (0.2 + 0.2 * torch.rand((*shape[:2], cache.d // 64), generator=g, device="cuda")).bfloat16()
                zero = (-7.5 * scale.float() + 0.3 * torch.randn(scale.shape, generator=g, device="cuda")).bfloat16()
            else:
                codes, scale, zero = (torch.tensor(y).cuda() for y in paged.quantise(given[b].cpu().numpy()))
                scale, zero = scale.bfloat16(), zero.bfloat16()
            t[pg, at] = codes[..., 0::2] | (codes[..., 1::2] << 4)
            sz[pg, at] = torch.stack((scale, zero), -1)
            s, z = (y.double().repeat_interleave(64, -1) for y in (scale, zero))
            got.append((z + s * codes.double(), (s * (codes.double() - 8)).abs() + (z + 8 * s).abs(), (z - 16 * s).abs()))
        out.append((got[0][0], got[1][0], got[0][1], got[1][1], got[1][2]))
    return out


def read(cache, table, lens):
    """What the cache holds of every sequence, as `write` returns it."""
    out = []
    for b, n in enumerate(lens):
        pos = np.arange(n)
        pg = torch.tensor(table[b][pos // cache.page_size].astype(np.int64)).cuda()
        at = torch.tensor(pos % cache.page_size).cuda()
        got = []
        for t, sz in ((cache.k, cache.k_sz), (cache.v, cache.v_sz)):
            x = t[pg, at]
            if sz is None:
                got.append((x.double(), x.double().abs(), torch.zeros(x.shape, dtype=torch.float64, device="cuda")))
                continue
            codes = torch.stack((x & 15, x >> 4), -1).flatten(-2).double()
            s, z = (y.double().repeat_interleave(64, -1) for y in sz[pg, at].unbind(-1))
            got.append((z + s * codes, (s * (codes - 8)).abs() + (z + 8 * s).abs(), (z - 16 * s).abs()))
        out.append((got[0][0], got[1][0], got[0][1], got[1][1], got[1][2]))
    return out


def check(q, cu, o, lse, held, scale, causal, four):
    """q, o [total, H, d], lse [H, total] against what `held` (write) says, sequence by sequence."""
    H, d = q.shape[1:]
    for b, (keys, vals, ksize, vsize, vbase) in enumerate(held):
        lo, hi = cu[b], cu[b + 1]
        nq, (nk, Hkv) = hi - lo, keys.shape[:2]
        if nq == 0:
            continue
        for j in range(Hkv):
            heads = slice(j * (H // Hkv), (j + 1) * (H // Hkv))
            qb = q[lo:hi, heads].double().transpose(0, 1)                       # [G, nq, d]
            got, gotl = o[lo:hi, heads].double().transpose(0, 1), lse[heads, lo:hi].double()
            assert not torch.isnan(got).any() and not torch.isnan(gotl).any()
            S = scale * (qb @ keys[:, j].T)
            dS = ((17 * (d + 16) / 16 + 8) * 2.0 ** -23 + (2.0 ** -21 + 2.0 ** -31 if four else 0)) * abs(scale)
            dS = dS * (qb.abs() @ ksize[:, j].T)
            if causal:
                hidden = torch.arange(nk, device="cuda") > torch.arange(nq, device="cuda")[:, None] + nk - nq
                S, dS = S.masked_fill(hidden, -math.inf), dS.masked_fill(hidden, 0.0)
            none = ~torch.isfinite(S).any(-1) if nk else torch.ones(S.shape[:2], dtype=torch.bool, device="cuda")
            assert (got[none] == 0).all() and (gotl[none] == -math.inf).all()
            if none.all():
                continue
            L = torch.logsumexp(S, -1)
            P = torch.exp(S - torch.where(none, 0.0, L)[..., None])
            dS = dS.amax(-1)
            want, A = P @ vals[:, j], P @ vals[:, j].abs()
            rel = 2.0 ** -10 if four else 2.0 ** -8
            room = 2.0 ** -8 * want.abs() + (rel + 2 * dS[..., None] + (64 + 17 * (nk / 16 + 1)) * 2.0 ** -23) * A
            if four:
                pad = torch.nn.functional.pad(vsize[:, j], (0, 0, 0, -nk % 32)).view(-1, 32, d).amax((1, 2)).repeat_interleave(32)[:nk]
                room = room + (nk * 2.0 ** -31 * (P * pad).amax(-1) + 2.0 ** -38 * (P @ pad))[..., None] + 2.0 ** -11 * (P @ vbase[:, j])
            err = (got - want).abs()
            bad = (err > room) & ~none[..., None]
            assert not bad.any(), (b, j, bad.nonzero()[0].tolist(), float((err / room)[~none].max()))
            errl = (gotl - L).abs()[~none]
            assert (errl <= (dS + 2.0 ** -19 * (1 + L.abs()))[~none]).all(), (b, j, float(errl.max()))


def case_of(kind, d, H, Hkv, ps, new, past, causal=True, scale=None, order="head", seed=3, extra=0, std=2.0):
    """The call on random contents, checked; (o, lse)."""
    ends = [n + p for n, p in zip(new, past)]
    table, pages = make_table([max(n, 0) for n in ends], ps, seed)
    cache = make_cache(kind, pages, ps, Hkv, d, order)
    held = write(cache, table, [max(n, 0) for n in ends], seed + 1)
    cu = np.concatenate(([0], np.cumsum(new)))
    q = randn((int(cu[-1]) + extra, H, d), seed + 2, std)
    scale = d ** -0.5 if scale is None else scale
    out, lse = torch.full_like(q, 7.0), torch.full((H, q.shape[0]), 7.0, device="cuda")
    got = binding.attn_fwd_paged_varlen(q, cache, i32(table), i32(cu), i32(ends), causal=causal, scale=scale, out=out, lse=lse)
    ok()
    assert got[0] is out and got[1] is lse
    total = int(cu[-1])
    assert (out[total:] == 7).all() and (lse[:, total:] == 7).all()      # rows behind the last sequence
    check(q, cu, out, lse, held, scale, causal, kind == "int4")
    return out, lse


CASES = [
    # d, H, Hkv, page size, new, past
    (128, 4, 1, 16, [1], [0]),                                   # one token, one key
    (128, 4, 1, 16, [32], [96]),                                 # one full tile of each
    (128, 4, 2, 16, [33, 64, 1, 0, 65], [0, 1, 127, 40, 300]),   # ends around tiles and units, an entry of padding
    (64, 16, 4, 16, [61], [1000]),
    (64, 3, 3, 48, [200, 7], [5, 900]),                          # no grouping; pages that no tile is a multiple of
    (64, 8, 1, 256, [17, 300], [128, 700]),                      # pages of two tiles
    (256, 8, 2, 64, [77, 1, 40], [200, 513, 0]),
    (256, 7, 1, 16, [19, 18, 37], [0, 111, 64]),                 # seven heads: 18 positions a tile, rows left over
    (128, 12, 1, 32, [10, 11, 21], [250, 0, 3]),
    (128, 5, 5, 128, [129, 257, 128], [0, 130, 128]),
    (128, 96, 1, 16, [3, 1], [200, 50]),                         # one position a tile
    (128, 8, 2, 16, [1] * 40, list(range(0, 1200, 30))),         # decoding
    (64, 128, 1, 16, [2], [300]),
    (128, 8, 2, 16, [1, 0, 33, 1, 1, 70, 0, 1, 1], [500, 3, 40, -1, 0, 300, 0, 3000, 31]),     # single tokens among chunks, one without keys
    (64, 24, 2, 32, [1, 1, 5, 1, 1, 1, 1, 2], [9, 2000, 40, 64, 0, 31, 32, 7]),
    (256, 32, 2, 16, [1, 1, 1, 1, 9, 1, 1, 1], [9, 700, 40, 64, 0, 31, 32, 7]),                # sixteen heads: two blocks of rows
    (128, 34, 2, 16, [1] * 8 + [3], [100] * 9),                                                # seventeen: not theirs
]


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_cases(kind, case):
    case_of(kind, *case)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [False, True])
def test_masks_and_scales(kind, d, causal):
    for scale in (None, -0.05, 1.5):
        case_of(kind, d, 4, 2, 16, [70, 3, 130], [60, 0, 500], causal=causal, scale=scale)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_without_keys(kind, d):
    """Fewer keys than queries: the first queries see nothing, in whole units and in parts of one; sequences without keys."""
    case_of(kind, d, 4, 2, 16, [300, 40, 5, 150], [-280, -40, -2, -1], extra=9)
    case_of(kind, d, 4, 2, 16, [300, 40], [-300, -40], causal=False)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("d,H,Hkv", [(64, 4, 1), (128, 4, 1), (128, 8, 8), (256, 4, 1)])
def test_cut_units(kind, d, H, Hkv):
    """One sequence over all CTAs: every unit is cut into many parts."""
    case_of(kind, d, H, Hkv, 16, [5], [20000])
    case_of(kind, d, H, Hkv, 64, [97], [9000])


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("order", ["token", "page_last"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_cache_strides(kind, order, d):
    case_of(kind, d, 6, 2, 32, [20, 50], [100, 7], order=order)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_sequences(kind, d):
    """More sequences than a warp has lanes, most of them empty; units of several CTAs' shares."""
    r = np.random.default_rng(8)
    new = [int(x) if r.random() < 0.4 else 0 for x in r.integers(1, 90, 150)]
    past = [int(x) for x in r.integers(0, 400, 150)]
    case_of(kind, d, 4, 2, 16, new, past)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_sharp_and_growing_scores(kind, d):
    """Scores that grow along the keys move the running maximum on every tile; far larger ones than the others' leave one weight."""
    n = 1500
    table, pages = make_table([n], 16, 1)
    cache = make_cache(kind, pages, 16, 1, d)
    g = torch.Generator().manual_seed(5)
    k, v = torch.randn((n, 1, d), generator=g), torch.randn((n, 1, d), generator=g)
    base = torch.randn(d, generator=g)
    k += base * (torch.arange(n) / 100.0)[:, None, None]
    held = write(cache, table, [n], 2, [k], [v])
    q = (base + 0.3 * torch.randn((90, 4, d), generator=g)).bfloat16().cuda()
    o, lse = binding.attn_fwd_paged_varlen(q, cache, i32(table), i32([0, 90]), i32([n]))
    ok()
    check(q, [0, 90], o, lse, held, d ** -0.5, True, kind == "int4")


@pytest.mark.parametrize("d", [64, 128, 256])
def test_sizes_of_values_and_queries(d):
    """4 bits: keys of far different sizes, query rows too, values of far different sizes beside each other and along the
    sequence, zero values: powers of two of 32 keys and of a row follow them."""
    n = 700
    table, pages = make_table([n], 16, 1)
    cache = make_cache("int4", pages, 16, 1, d)
    g = torch.Generator().manual_seed(6)
    k, v = torch.randn((n, 1, d), generator=g), torch.randn((n, 1, d), generator=g)
    k *= 2.0 ** torch.randint(-12, 1, (n, 1, 1), generator=g)
    v *= 2.0 ** torch.randint(-12, 13, (n, 1, 1), generator=g)
    v[:64] *= 2.0 ** 20
    v[64:128] *= 2.0 ** -30
    v[128:160] = 0
    v += 40.0 * 2.0 ** torch.randint(-3, 4, (n, 1, 1), generator=g)     # far from zero
    held = write(cache, table, [n], 2, [k], [v])
    q = (torch.randn((40, 5, d), generator=g) * 2.0 ** torch.randint(-20, 2, (40, 5, 1), generator=g)).bfloat16().cuda()
    o, lse = binding.attn_fwd_paged_varlen(q, cache, i32(table), i32([0, 40]), i32([n]))
    ok()
    check(q, [0, 40], o, lse, held, d ** -0.5, True, True)


def test_empty_cache_of_zeros():
    """A cache as allocated: all scores 0, all values 0."""
    for kind in ("bf16", "int4"):
        cache = binding.PagedKVCache.allocate(8, 16, 2, 128, kind)
        q = randn((10, 4, 128), 1)
        o, lse = binding.attn_fwd_paged_varlen(q, cache, i32([[1, 2, 3, 4]]), i32([0, 10]), i32([60]), causal=False)
        ok()
        assert (o == 0).all() and torch.allclose(lse, torch.full_like(lse, math.log(60)), rtol=2.0 ** -19, atol=0)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("past", [0, 300, 9000])
def test_nan_query_row_stays_one_row(kind, past):
    """NaN among whole units and cut ones: that row's results are NaN, the others' as without it."""
    new = 40
    table, pages = make_table([new + past], 16, 1)
    cache = make_cache(kind, pages, 16, 2, 128)
    write(cache, table, [new + past], 4)
    q = randn((new, 8, 128), 5)
    args = (cache, i32(table), i32([0, new]), i32([new + past]))
    o, lse = binding.attn_fwd_paged_varlen(q, *args)
    q[17, 3, 5] = float("nan")
    on, ln = binding.attn_fwd_paged_varlen(q, *args)
    ok()
    assert on[17, 3].isnan().all() and ln[3, 17].isnan()
    on[17, 3], ln[3, 17] = o[17, 3], lse[3, 17]
    assert torch.equal(on, o) and torch.equal(ln, lse)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_same_bits_every_time_and_as_alone(kind, d):
    """Two runs give the same bits; a workspace full of NaN, and another stream, change nothing."""
    table, pages = make_table([5000, 300], 16, 1)
    cache = make_cache(kind, pages, 16, 2, d)
    write(cache, table, [5000, 300], 4)
    q = randn((130, 8, d), 5)
    args = (q, cache, i32(table), i32([0, 50, 130]), i32([5000, 300]))
    first = binding.attn_fwd_paged_varlen(*args)
    n = binding.attn_fwd_paged_varlen_workspace_bytes(cache, 2, 8, 130)
    ws = torch.full((n // 4,), float("nan"), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = binding.attn_fwd_paged_varlen(*args, workspace=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    ok()
    for a, b in zip(first, second):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_bad_pages_lengths_and_offsets(kind):
    """Pages outside the pool count as zeros, lengths are cut to the table, sequences with unsound offsets have no rows; each
    is reported, and other sequences are right: with the same bits where all lengths are the same (they say where units are
    cut)."""
    d, ps = 128, 16
    table, pages = make_table([200, 150, 90], ps, 1)
    cache = make_cache(kind, pages, ps, 2, d)
    held = write(cache, table, [200, 150, 90], 4)
    q = randn((60, 4, d), 5)
    cu = [0, 20, 40, 60]

    def run(table, cu, lens):
        out, lse = torch.full_like(q, 7.0), torch.full((4, 60), 7.0, device="cuda")
        binding.attn_fwd_paged_varlen(q, cache, i32(table), i32(cu), i32(lens), out=out, lse=lse)
        st, detail = binding.attn_get_status()
        binding.attn_clear_status()
        return out, lse, st, detail

    good, good_lse, st, _ = run(table, cu, [200, 150, 90])
    assert st == binding.ATTN_OK
    bad = table.copy()
    bad[1, 2], bad[1, 5] = pages, -1
    out, lse, st, detail = run(bad, cu, [200, 150, 90])
    assert st == binding.ATTN_ERR_INVALID_ARG and detail == 0x2000000D
    assert torch.equal(out[:20], good[:20]) and torch.equal(out[40:], good[40:])
    zeroed = [tuple(x.clone() for x in h) for h in held]
    for x in zeroed[1]:
        x[32:48], x[80:96] = 0, 0
    check(q, cu, out, lse, zeroed, d ** -0.5, True, kind == "int4")
    full = table.shape[1] * ps                                  # the table is as wide as sequence 0 needs: 208 keys
    out, lse, st, detail = run(table, cu, [200, 150, 91 + 10 ** 6])   # cut to 208 keys, the last of them on pages of -7
    assert st == binding.ATTN_ERR_INVALID_ARG and detail == 0x2000000D and full == 208
    check(q, cu, out, lse, held[:2], d ** -0.5, True, kind == "int4")
    out, lse, st, detail = run(table, [0, 20, 61, 60], [200, 150, 90])
    assert st == binding.ATTN_ERR_INVALID_ARG and detail == 0x2000000D
    check(q, cu, out, lse, held[:1], d ** -0.5, True, kind == "int4")
    assert (out[20:] == 7).all() and (lse[:, 20:] == 7).all()
    out, lse, st, detail = run(table, cu, [200, -3, 90])
    assert st == binding.ATTN_ERR_INVALID_ARG
    check(q, cu, out, lse, [held[0], tuple(x[:0] for x in held[1]), held[2]], d ** -0.5, True, kind == "int4")


def test_bad_singles():
    """Single tokens of a larger batch over 4 bits: bad pages count as zeros, unsound offsets leave rows, others are as before."""
    d, lens = 128, [200, 150, 90, 40, 64, 1, 17, 300, 0]
    table, pages = make_table(lens, 16, 1)
    cache = make_cache("int4", pages, 16, 2, d)
    held = write(cache, table, lens, 4)
    q = randn((9, 4, d), 5)

    def run(table, cu):
        out, lse = torch.full_like(q, 7.0), torch.full((4, 9), 7.0, device="cuda")
        binding.attn_fwd_paged_varlen(q, cache, i32(table), i32(cu), i32(lens), out=out, lse=lse)
        st, detail = binding.attn_get_status()
        binding.attn_clear_status()
        return out, lse, st, detail

    cu = list(range(10))
    out, lse, st, _ = run(table, cu)
    assert st == binding.ATTN_OK
    check(q, cu, out, lse, held, d ** -0.5, True, True)
    bad = table.copy()
    bad[1, 2], bad[1, 5] = pages, -1
    got, gotl, st, detail = run(bad, cu)
    assert st == binding.ATTN_ERR_INVALID_ARG and detail == 0x2000000D
    keep = [0, 2, 3, 4, 5, 6, 7, 8]
    assert torch.equal(got[keep], out[keep]) and torch.equal(gotl[:, keep], lse[:, keep])
    for x in held[1]:
        x[32:48], x[80:96] = 0, 0
    check(q, cu, got, gotl, held, d ** -0.5, True, True)
    got, gotl, st, detail = run(table, [0, 1, 2, 3, 4, 5, 6, 7, 10, 11])     # the last two sequences pass the rows
    assert st == binding.ATTN_ERR_INVALID_ARG and detail == 0x2000000D
    check(q, cu, got, gotl, write(cache, table, lens, 4)[:7], d ** -0.5, True, True)
    assert (got[7:] == 7).all() and (gotl[:, 7:] == 7).all()


def test_a_missing_copy_is_reported():
    """A tile that never comes: the waits run out, the call ends, and the status says so."""
    table, pages = make_table([400], 16, 1)
    cache = make_cache("bf16", pages, 16, 1, 128)
    write(cache, table, [400], 4)
    q = randn((20, 4, 128), 5)
    args = (q, cache, i32(table), i32([0, 20]), i32([400]))
    good = binding.attn_fwd_paged_varlen(*args)
    ok()
    try:
        binding.attn_debug_set(timeout_ns=20_000_000, skip_load=True)
        binding.attn_fwd_paged_varlen(*args)
        st, detail = binding.attn_get_status()
        assert st == binding.ATTN_ERR_TIMEOUT and detail & 0x40000000
    finally:
        binding.attn_debug_set(timeout_ns=500_000_000)
        binding.attn_clear_status()
    again = binding.attn_fwd_paged_varlen(*args)
    ok()
    assert all(torch.equal(a, b) for a, b in zip(good, again))


def test_captured_and_replayed_with_other_lengths():
    table, pages = make_table([640, 640], 16, 1)
    cache = make_cache("bf16", pages, 16, 2, 128)
    held = write(cache, table, [640, 640], 4)
    q = randn((96, 8, 128), 5)
    cu, lens, t = i32([0, 48, 96]), i32([640, 640]), i32(table)
    ws = torch.empty(binding.attn_fwd_paged_varlen_workspace_bytes(cache, 2, 8, 96), dtype=torch.uint8, device="cuda")
    binding.attn_fwd_paged_varlen(q, cache, t, cu, lens, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = binding.attn_fwd_paged_varlen(q, cache, t, cu, lens, workspace=ws)
    for new, n in (([48, 48], [640, 640]), ([1, 95], [200, 96]), ([96, 0], [600, 3]), ([3, 2], [5, 640])):
        cu.copy_(i32([0, new[0], new[0] + new[1]]))
        lens.copy_(i32(n))
        graph.replay()
        ok()
        check(q, [0, new[0], new[0] + new[1]], o, lse, [tuple(x[:m] for x in h) for h, m in zip(held, n)], 128 ** -0.5, True, False)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_pages_beyond_32_bits(kind):
    """Pages whose bytes lie more than 2^32 from the first one's, for chunks and (4 bits, a batch of 8) single tokens."""
    d, Hkv, ps, lens, new = 256, 8, 64, [300, 77, 128, 1, 40, 500, 16, 333], [30, 1, 100, 1, 1, 1, 1, 50]
    row = 2 * d if kind == "bf16" else d // 2
    first = 2 ** 32 // (ps * Hkv * row) + 3
    table, pages = make_table(lens, ps, 1)
    table = np.where(table >= 0, table + first, table)
    cache = binding.PagedKVCache.allocate(first + pages, ps, Hkv, d, kind)
    held = write(cache, table, lens, 4)
    q = randn((sum(new), 2 * Hkv, d), 5)
    cu = np.concatenate(([0], np.cumsum(new)))
    o, lse = binding.attn_fwd_paged_varlen(q, cache, i32(table), i32(cu), i32(lens))
    ok()
    check(q, cu, o, lse, held, d ** -0.5, True, kind == "int4")


def test_captured_with_single_tokens_that_come_and_go():
    """4 bits, a batch of which some sequences have one token: which ones is known on the GPU only."""
    lens, d = [300, 77, 128, 1, 40, 500, 16, 33], 64
    table, pages = make_table(lens, 16, 1)
    cache = make_cache("int4", pages, 16, 2, d)
    held = write(cache, table, lens, 4)
    q = randn((60, 8, d), 5)
    cu, n, t = i32([0] * 9), i32(lens), i32(table)
    ws = torch.empty(binding.attn_fwd_paged_varlen_workspace_bytes(cache, 8, 8, 60), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((8, 60), device="cuda")
    binding.attn_fwd_paged_varlen(q, cache, t, cu, n, workspace=ws, out=out, lse=lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.attn_fwd_paged_varlen(q, cache, t, cu, n, workspace=ws, out=out, lse=lse)
    for new in ([1] * 8, [1, 0, 30, 1, 2, 1, 16, 1], [40, 1, 1, 1, 1, 1, 1, 1], [0, 0, 0, 1, 0, 0, 0, 0], [7] * 8):
        ends = np.concatenate(([0], np.cumsum(new)))
        cu.copy_(i32(ends))
        out.fill_(7.0), lse.fill_(7.0)
        graph.replay()
        ok()
        check(q, ends, out, lse, held, d ** -0.5, True, True)
        assert (out[ends[-1]:] == 7).all() and (lse[:, ends[-1]:] == 7).all()


@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_two_calls_at_once(kind):
    """On two streams, each with its own workspace: the bits of each alone."""
    d, lens, new = 128, [3000, 5, 700, 64, 1, 900, 257, 33, 2000], [200, 1, 70, 1, 1, 130, 1, 9, 1]
    table, pages = make_table(lens, 16, 1)
    cache = make_cache(kind, pages, 16, 2, d)
    write(cache, table, lens, 4)
    cu, n, t = i32(np.concatenate(([0], np.cumsum(new)))), i32(lens), i32(table)
    qs = [randn((sum(new), 8, d), 5 + i) for i in range(2)]
    alone = [binding.attn_fwd_paged_varlen(q, cache, t, cu, n) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    size = binding.attn_fwd_paged_varlen_workspace_bytes(cache, len(new), 8, sum(new))
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in qs]
    out = [(torch.empty_like(q), torch.empty((8, sum(new)), device="cuda")) for q in qs]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, q in enumerate(qs):
            binding.attn_fwd_paged_varlen(q, cache, t, cu, n, workspace=ws[i], out=out[i][0], lse=out[i][1], stream=streams[i])
    torch.cuda.synchronize()
    ok()
    for got, want in zip(out, alone):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_offsets_of_more_work_than_a_call_may_have():
    """4096 sequences of the same 65536 rows (and as many whose offsets descend) over 2^31 keys each: nothing is computed, and
    the status says so."""
    total, pages = 1 << 16, ((1 << 31) - 1024) // 16
    cache = make_cache("bf16", 1, 16, 1, 64)
    q = torch.zeros((total, 1, 64), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((1, pages), dtype=torch.int32, device="cuda").expand(8191, -1)
    cu = torch.tensor([0, total] * 4096, dtype=torch.int32, device="cuda")
    lens = torch.full((8191,), pages * 16, dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((1, total), 7.0, device="cuda")
    binding.attn_fwd_paged_varlen(q, cache, table, cu, lens, out=out, lse=lse)
    st, detail = binding.attn_get_status()
    binding.attn_clear_status()
    assert st == binding.ATTN_ERR_INVALID_ARG and detail == 0x2000000D
    assert (out == 7).all() and (lse == 7).all()


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_as_decode(kind, d):
    """One token of each sequence: what attn_fwd_paged gives, within both calls' bounds."""
    lens = [1, 17, 300, 0, 2500]
    table, pages = make_table(lens, 16, 1)
    cache = make_cache(kind, pages, 16, 2, d)
    held = write(cache, table, lens, 4)
    q = randn((5, 1, 8, d), 5)
    o, lse = binding.attn_fwd_paged(q, cache, i32(table), i32(lens))
    check(q[:, 0], list(range(6)), o[:, 0], lse[:, :, 0].T, held, d ** -0.5, True, kind == "int4")
    o, lse = binding.attn_fwd_paged_varlen(q[:, 0].contiguous(), cache, i32(table), i32(list(range(6))), i32(lens))
    ok()
    check(q[:, 0], list(range(6)), o, lse, held, d ** -0.5, True, kind == "int4")


def test_refusals():
    cache = binding.PagedKVCache.allocate(8, 16, 2, 128)
    q, t, cu, lens = randn((10, 4, 128), 1), i32([[1, 2]]), i32([0, 10]), i32([20])
    call = binding.attn_fwd_paged_varlen
    for bad in (dict(q=q.float()), dict(q=q[:, :, :64]), dict(q=q[:, :3].contiguous()), dict(q=q.transpose(0, 1)), dict(q=q[None]),
                dict(q=q.cpu()), dict(cu=cu.long()), dict(cu=i32([0, 5, 10])), dict(lens=i32([20, 20])), dict(lens=lens.cpu()),
                dict(t=t.long()), dict(out=q.float()), dict(lse=torch.empty((10, 4), device="cuda")),
                dict(workspace=torch.empty((100, 100), device="cuda")[:, ::2])):
        a = dict(q=q, t=t, cu=cu, lens=lens)
        a.update({x: y for x, y in bad.items() if x in a})
        with pytest.raises(ValueError):
            call(a["q"], cache, a["t"], a["cu"], a["lens"], **{x: y for x, y in bad.items() if x not in a})
    with pytest.raises(TypeError):
        call(None, cache, t, cu, lens)
    for bad in (dict(scale=0.0), dict(scale=float("nan")), dict(out=q), dict(workspace=torch.empty(1000, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(binding.AttnError):
            call(q, cache, t, cu, lens, **bad)
    o, lse = call(q[:0], cache, t, i32([0, 0]), lens)                 # nothing to do
    assert o.shape == (0, 4, 128) and lse.shape == (4, 0)
    ok()


@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_a_step_of_a_multimodal_server(kind):
    """Norm and rotation with three axes, append, attention of the chunk, as they are used together: two steps of prompts (text,
    an image of 5 x 8 patches, text) and decoding, against what the cache holds after each; and q and k as all tokens at once give
    them."""
    H, Hkv, d, ps = 8, 2, 128, 16
    steps = [[70, 33, 1], [1, 64, 200]]
    total = [sum(x) for x in zip(*steps)]
    table, pages = make_table(total, ps, 1)
    cache = binding.PagedKVCache.allocate(pages, ps, Hkv, d, kind)
    half, text, rows, cols = d // 2, 20, 5, 8
    a = torch.arange(400, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    cos, sin = a.cos().float().cuda(), a.sin().float().cuda()
    wq, wk = 1 + 0.1 * torch.rand(d, device="cuda"), 1 + 0.1 * torch.rand(d, device="cuda")
    sections = binding.rope_pair_axes((16, 24, 24), turns=kind == "int4")

    def place(p):   # of a sequence's token p: time, row and column
        if p < text:
            return p, p, p
        if p < text + rows * cols:
            return text, text + (p - text) // cols, text + (p - text) % cols
        return (p - text - rows * cols + text + cols,) * 3

    def turned(qkv, pos):
        where = i32(np.array([place(p) for p in pos]).T.copy())
        return binding.attn_qk_norm_rope_axes(qkv[:, :H], qkv[:, H:H + Hkv], cos, sin, where, sections, wq=wq, wk=wk)

    past, seen = [0, 0, 0], []
    for i, new in enumerate(steps):
        qkv = randn((sum(new), H + 2 * Hkv, d), 9 + i)
        pos = [p + j for p, n in zip(past, new) for j in range(n)]
        q, k = turned(qkv, pos)
        seen.append((qkv, pos, q, k))
        cu = np.concatenate(([0], np.cumsum(new)))
        binding.attn_paged_append(cache, k, qkv[:, H + Hkv:], i32(cu), i32(past), i32(table))
        past = [p + n for p, n in zip(past, new)]
        o, lse = binding.attn_fwd_paged_varlen(q, cache, i32(table), i32(cu), i32(past))
        ok()
        check(q, cu, o, lse, read(cache, table, past), d ** -0.5, True, kind == "int4")
    q, k = turned(torch.cat([x[0] for x in seen]), [p for x in seen for p in x[1]])
    assert torch.equal(q, torch.cat([x[2] for x in seen])) and torch.equal(k, torch.cat([x[3] for x in seen]))
    if kind == "bf16":
        lo = 0
        for b, n in enumerate(steps[0]):   # what was appended is what was turned
            assert torch.equal(read(cache, table, past)[b][0][:n], seen[0][3][lo:lo + n].double())
            lo += n


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,H,Hkv,new", [(64, 32, 2, 1225), (128, 32, 2, 1225), (256, 32, 2, 1225), (256, 128, 1, 1030)])
def test_many_units_of_a_head(kind, causal, d, H, Hkv, new):
    """More units of a (sequence, kv head) than a warp has lanes, and than the square of that: 77 units of 16 positions (step 3 of
    the search, which 77 is no multiple of), 154 of 8 (step 5), 1030 of one (33, then 2). Shares begin in all of them."""
    case_of(kind, d, H, Hkv, 16, [new], [10], causal=causal)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_kv_heads(kind, d):
    """Shares that begin in kv heads behind the 32nd and the 64th; single tokens of such a batch."""
    case_of(kind, d, 134, 67, 16, [5, 40], [300, 20])
    case_of(kind, d, 40, 40, 16, [1, 1, 30, 1, 0, 2, 1, 1, 1], [700, 5, 90, 33, 8, 0, 1200, 31, 0])


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,G", [(64, 3), (128, 3), (256, 3), (64, 6), (128, 6), (256, 6), (64, 12), (128, 12), (256, 12)])
def test_masks_and_scales_of_single_tokens_among_chunks(kind, causal, d, G):
    """Over 4 bits the two kernels of one call agree on the sign of the scale and on the mask. Single tokens' scores there are
    sums of |zero| and scale times code apart: their dS is of |q| times the two."""
    new, past = [1, 70, 1, 3, 1, 1, 0, 1, 130, 1], [60, 0, 500, 9, -1, 0, 40, 1100, 333, 31]
    ends = [n + p for n, p in zip(new, past)]
    table, pages = make_table(ends, 16, 3)
    cache = make_cache(kind, pages, 16, 2, d)
    held = write(cache, table, ends, 4)
    if kind == "int4":
        for b, (keys, vals, ksize, vsize, vbase) in enumerate(held):
            if new[b] == 1 and ends[b]:
                pos = np.arange(ends[b])
                pg, at = torch.tensor(table[b][pos // 16].astype(np.int64)).cuda(), torch.tensor(pos % 16).cuda()
                zero = cache.k_sz[pg, at][..., 1].double().repeat_interleave(64, -1)
                held[b] = keys, vals, torch.maximum(ksize, zero.abs() + (keys - zero).abs()), vsize, vbase
    cu = np.concatenate(([0], np.cumsum(new)))
    q = randn((int(cu[-1]), 2 * G, d), 5, 2.0)
    for scale in (d ** -0.5, -0.05, 1.5):
        o, lse = binding.attn_fwd_paged_varlen(q, cache, i32(table), i32(cu), i32(ends), causal=causal, scale=scale)
        ok()
        check(q, cu, o, lse, held, scale, causal, kind == "int4")

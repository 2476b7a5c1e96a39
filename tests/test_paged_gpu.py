"""The paged cache (append, gather) and the attention over it, against the oracle.

Append and gather are compared bit for bit: the oracle's float32 steps are the library's. Attention's bounds follow from
its arithmetic, per output value and in natural units:
  dS: scores come out of fp32 sums of at most d terms (the tensor core's own included) and a few products:
      64 * 2^-23 of scale * sum|q| * max|k|, with max|k| for 4 bits the greatest |zero| + 15 scale;
  weights: p (times scale) rounded to bf16, 2^-8, or fp16, 2^-11: that part of sum_j P_j |term_j|; and 2 dS of it;
  output: bf16, 2^-8 of the value. LSE: dS and 2^-19 (1 + |LSE|) for exponentials, logarithm and sums.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import paged
from exact_attention_72_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_device):
    from exact_attention_72_gb300 import build
    build.build()


def np32(t):
    return t.detach().float().cpu().numpy()


def ok():
    st, detail = binding.attn_get_status()
    assert st == binding.ATTN_OK, hex(detail)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def tables(n, half):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(half) / half)
    return torch.tensor(np.cos(a), dtype=torch.float32).cuda(), torch.tensor(np.sin(a), dtype=torch.float32).cuda()


def make_cache(kind, pages, ps, Hkv, d, order="head"):
    """A cache full of NaN (bf16; also the scales of 4 bits): what is not written must not be read."""
    def full(*row, dtype, value):
        shape = {"head": (pages, Hkv, ps), "token": (pages, ps, Hkv), "page_last": (ps, Hkv, pages)}[order]
        t = torch.full((*shape, *row), value, dtype=dtype, device="cuda")
        return {"head": lambda: t.transpose(1, 2), "token": lambda: t, "page_last": lambda: t.movedim(2, 0)}[order]()
    nan = float("nan")
    if kind == "bf16":
        return binding.PagedKVCache(full(d, dtype=torch.bfloat16, value=nan), full(d, dtype=torch.bfloat16, value=nan))
    return binding.PagedKVCache(full(d // 2, dtype=torch.uint8, value=255), full(d // 2, dtype=torch.uint8, value=255),
                                full(d // 64, 2, dtype=torch.bfloat16, value=nan), full(d // 64, 2, dtype=torch.bfloat16, value=nan))


def make_table(lens, ps, seed, spare=2, width=None):
    """Scattered pages; entries behind a sequence's last page lead nowhere."""
    need = [-(-n // ps) for n in lens]
    perm = np.random.default_rng(seed).permutation(sum(need) + spare)
    t = np.full((len(lens), width or max(1, max(need))), -7, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = perm[at:at + n]
        at += n
    return t, sum(need) + spare


def randn(shape, seed, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).bfloat16().cuda()


def fill(cache, table, lens, seed, std=1.0):
    """Appends lens[b] random tokens to every empty sequence; what the cache then holds, per sequence in fp64 (k, v)."""
    total = sum(lens)
    k, v = randn((total, cache.Hkv, cache.d), seed, std), randn((total, cache.Hkv, cache.d), seed + 1)
    k[::97, :, 3] = 8.0     # outliers
    cu = np.concatenate(([0], np.cumsum(lens)))
    binding.attn_paged_append(cache, k, v, i32(cu), i32([0] * len(lens)), i32(table))
    ok()
    out = []
    for x in (np32(k), np32(v)):
        if cache.k_sz is not None:
            x = paged.values(*paged.quantise(x))
        out.append([np.float64(x[cu[b]:cu[b + 1]]) for b in range(len(lens))])
    return out


# ------------------------------------------------------------------------------------------------- append and gather

APPENDS = [
    # kind, d, Hkv, page size, rope_dim, interleaved, order, new, past
    ("bf16", 128, 2, 16, 128, False, "head", [5, 1, 40], [0, 15, 3]),
    ("bf16", 64, 3, 32, 32, True, "token", [1, 1, 1, 1], [31, 32, 33, 0]),
    ("bf16", 256, 1, 16, 0, False, "page_last", [17], [16]),
    ("bf16", 64, 5, 16, 16, False, "head", [0, 9, 0], [4, 100, 0]),
    ("int4", 128, 2, 16, 128, False, "head", [5, 1, 40], [0, 15, 3]),
    ("int4", 64, 3, 48, 32, True, "token", [1, 1, 1, 1], [31, 32, 47, 48]),
    ("int4", 256, 1, 16, 256, False, "page_last", [17], [16]),
    ("int4", 256, 4, 64, 80, True, "head", [70, 3], [0, 61]),
    ("int4", 128, 8, 16, 0, False, "token", [2] * 50, list(range(50))),      # more sequences than lanes of a row
]


@pytest.mark.parametrize("case", APPENDS, ids=str)
def test_append_and_gather(case):
    kind, d, Hkv, ps, rd, il, order, new, past = case
    ends = [n + p for n, p in zip(new, past)]
    table, pages = make_table(ends, ps, 5)
    cache = make_cache(kind, pages, ps, Hkv, d, order)
    before = [t.clone() for t in (cache.k, cache.v, cache.k_sz, cache.v_sz) if t is not None]
    total = sum(new)
    kv = randn((total + 3, 2 * Hkv, d), 6)      # keys and values of one projection; three tokens behind the last sequence
    k, v = kv[:, :Hkv], kv[:, Hkv:]
    cos, sin = tables(max(ends) + 1, rd // 2) if rd else (None, None)
    cu = np.concatenate(([0], np.cumsum(new)))
    binding.attn_paged_append(cache, k, v, i32(cu), i32(past), i32(table), cos, sin, il)
    ok()

    kx, vx = np32(k)[:total], np32(v)[:total]
    pos = np.concatenate([np.arange(p, p + n) for n, p in zip(new, past)]).astype(int)
    seq = np.repeat(np.arange(len(new)), new)
    if rd:
        kx = paged.turn_f32(kx, np32(cos)[pos], np32(sin)[pos], il)
    want = [t.clone() for t in before]
    pg, at = np.array([paged.place(table[b], p, ps) for b, p in zip(seq, pos)]).T
    pg, at = torch.tensor(pg).cuda(), torch.tensor(at).cuda()
    shown = []
    for i, x in enumerate((kx, vx)):
        if kind == "bf16":
            want[i][pg, at] = torch.tensor(paged.bf16_nearest(x)).cuda().bfloat16()
            shown.append(paged.bf16_nearest(x))
        else:
            codes, scale, zero = paged.quantise(x)
            want[i][pg, at] = torch.tensor(paged.pack(codes)).cuda()
            want[2 + i][pg, at] = torch.tensor(np.stack((scale, zero), -1)).cuda().bfloat16()
            shown.append(paged.bf16_nearest(np.float32(paged.values(codes, scale, zero))))
    for name, t, w in zip(("k", "v", "k_sz", "v_sz"), (cache.k, cache.v, cache.k_sz, cache.v_sz), want):
        bits = torch.int16 if t.dtype == torch.bfloat16 else torch.uint8
        assert torch.equal(t.contiguous().view(bits), w.contiguous().view(bits)), name     # the other rows included

    # Read back with the whole of every sequence; only the new rows are known.
    cu_all = np.concatenate(([0], np.cumsum(ends)))
    n = int(cu_all[-1])
    out = [torch.full((n + 2, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    binding.attn_paged_gather(cache, i32(cu_all), i32(table), n + 2, k=out[0], v=out[1])
    ok()
    rows = cu_all[seq] + pos
    for y, x in zip(out, shown):
        assert np.array_equal(np32(y)[rows], x)
        assert bool((y[n:] == 7).all())        # rows behind the last sequence


def test_append_refuses_bad_pages_positions_and_offsets_on_the_device():
    """Each is reported and leaves its rows out; nothing else changes."""
    ps, Hkv, d = 16, 2, 128
    k, v = randn((6, Hkv, d), 1), randn((6, Hkv, d), 2)
    good = dict(cu=[0, 3, 6], past=[0, 14], table=[[0, 1], [2, 3]])
    # (positions 14, 15 and 16 of the second sequence: the last alone lies on its second page)
    cases = [(dict(table=[[0, 1], [2, 9]]), [5]), (dict(table=[[-1, 1], [2, 3]]), [0, 1, 2]),
             (dict(past=[0, 31]), [4, 5]), (dict(past=[-1, 14]), [0, 1, 2]), (dict(past=[2 ** 31 - 2, 14]), [0, 1, 2]),
             (dict(past=[0, 21]), [5])]      # past the tables of angles
    for bad, lost in cases:
        a = dict(good, **bad)
        for kind in ("bf16", "int4"):
            cache, ref = make_cache(kind, 4, ps, Hkv, d), make_cache(kind, 4, ps, Hkv, d)
            cos, sin = tables(23 if bad.get("past") == [0, 21] else 64, 64)
            try:
                binding.attn_paged_append(cache, k, v, i32(a["cu"]), i32(a["past"]), i32(a["table"]), cos, sin)
                assert binding.attn_get_status() == (binding.ATTN_ERR_INVALID_ARG, 0x2000000D), bad
            finally:
                binding.attn_clear_status()
            # the rest as one call for each sequence without the lost tokens
            for b in range(2):
                keep = [t for t in range(a["cu"][b], a["cu"][b + 1]) if t not in lost]
                if keep:
                    binding.attn_paged_append(ref, k[keep], v[keep], i32([0, len(keep)]), i32(a["past"][b:b + 1]),
                                              i32([a["table"][b]]), cos, sin)
            ok()
            for t, w in ((cache.k, ref.k), (cache.v, ref.v)):
                bits = torch.int16 if t.dtype == torch.bfloat16 else torch.uint8
                assert torch.equal(t.contiguous().view(bits), w.contiguous().view(bits)), bad


def test_gather_reports_bad_pages():
    cache = make_cache("int4", 4, 16, 2, 64)
    fill(cache, np.array([[0, 1]]), [20], 3)
    out = [torch.full((20, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    try:
        binding.attn_paged_gather(cache, i32([0, 20]), i32([[0, 4]]), 20, *out)
        assert binding.attn_get_status()[1] == 0x2000000D
    finally:
        binding.attn_clear_status()
    assert bool((out[0][16:] == 7).all()) and not bool((out[0][:16] == 7).all())


# ------------------------------------------------------------------------------------------------- attention

def check(q, o, lse, keys, vals, scale, causal, kind):
    qn = np.float64(np32(q))
    B, Nq, H, d = qn.shape
    o_ref, lse_ref = paged.attention_paged(qn, keys, vals, scale, causal)
    on, ln = np.float64(np32(o)), np.float64(np32(lse))
    empty = np.isneginf(lse_ref)
    assert np.array_equal(np.isneginf(ln), empty)
    assert np.all(on.transpose(0, 2, 1, 3)[empty] == 0)
    half = 2.0 ** -8 if kind == "bf16" else 2.0 ** -11
    for b in range(B):
        if not len(keys[b]):
            continue
        top_k, top_v = np.abs(keys[b]).max(), np.abs(vals[b]).max()
        if kind == "int4":      # |zero| + 15 scale <= 3 max|x| for a group that has its zero among its values
            top_k, top_v = 3 * top_k, 3 * top_v
        for h in range(H):
            for i in range(Nq):
                if empty[b, h, i]:
                    continue
                dS = 64 * 2.0 ** -23 * abs(scale) * np.abs(qn[b, i, h]).sum() * top_k
                err, size = np.abs(on[b, i, h] - o_ref[b, i, h]), np.abs(o_ref[b, i, h])
                assert np.all(err <= 2.0 ** -8 * size + (half + 2 * dS) * top_v), (b, h, i, err.max())
                assert abs(ln[b, h, i] - lse_ref[b, h, i]) <= dS + 2.0 ** -19 * (1 + abs(lse_ref[b, h, i]))
    fin = ~empty.transpose(0, 2, 1)
    if fin.any():   # and over all values the rounding of weights and output averages out
        assert np.linalg.norm(on - o_ref) <= 2.0 ** -8 * np.linalg.norm(o_ref) + 1e-30


def attend(q, cache, table, lens, causal=True, **kw):
    o, lse = binding.attn_fwd_paged(q, cache, i32(table), i32(lens), causal=causal, **kw)
    ok()
    return o, lse


ATTENDS = [
    # d, H, Hkv, Nq, page size, order, lengths, causal
    (128, 1, 1, 1, 16, "head", [1], True),
    (128, 8, 2, 1, 16, "head", [1, 15, 16, 17, 31, 32, 33, 0], True),
    (128, 8, 1, 1, 16, "token", [127, 128, 129, 1000], True),
    (64, 4, 4, 1, 32, "page_last", [63, 64, 65, 300], True),
    (256, 6, 2, 1, 16, "head", [1, 47, 200], True),
    (128, 16, 1, 1, 64, "head", [500], True),                       # 16 rows of a kv head
    (64, 20, 1, 1, 16, "head", [77, 1], True),                      # 20 rows: two blocks
    (256, 24, 2, 1, 16, "token", [130], True),                      # 12 rows at d = 256: two blocks
    (128, 4, 2, 3, 16, "head", [0, 1, 2, 3, 4, 200], True),         # rows that see no key
    (64, 12, 4, 4, 48, "head", [3, 96, 97, 1], True),
    (256, 4, 1, 5, 64, "head", [64, 4, 333], True),
    (128, 8, 2, 5, 16, "head", [1, 100, 0, 33], False),
    (128, 10, 2, 1, 16, "head", [40 + 3 * i for i in range(200)], True),     # more sequences than a block has threads
]


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("case", ATTENDS, ids=lambda c: "-".join(map(str, c))[:60])
def test_attention(case, kind):
    d, H, Hkv, Nq, ps, order, lens, causal = case
    table, pages = make_table(lens, ps, 9)
    cache = make_cache(kind, pages, ps, Hkv, d, order)
    keys, vals = fill(cache, table, lens, 10)
    q = randn((len(lens), Nq, H, d), 12, 2.0)
    o, lse = attend(q, cache, table, lens, causal)
    check(q, o, lse, keys, vals, d ** -0.5, causal, kind)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("d,H,Hkv,n", [(128, 8, 1, 40000), (64, 2, 2, 30001), (256, 3, 1, 20011)])
def test_one_long_sequence_cut_over_many_ctas(kind, d, H, Hkv, n):
    table, pages = make_table([n], 16, 1)
    cache = make_cache(kind, pages, 16, Hkv, d)
    keys, vals = fill(cache, table, [n], 2)
    q = randn((1, 1, H, d), 3, 4.0)
    ws = torch.full((binding.attn_fwd_paged_workspace_bytes(cache, 1, H, 1),), 255, dtype=torch.uint8, device="cuda")
    o, lse = attend(q, cache, table, [n], workspace=ws)
    check(q, o, lse, keys, vals, d ** -0.5, True, kind)
    o2, lse2 = attend(q, cache, table, [n])          # another workspace, other contents: the same bits
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("scale", [-0.125, 3.0, 1e-3])
def test_scales(kind, scale):
    table, pages = make_table([200, 37], 16, 1)
    cache = make_cache(kind, pages, 16, 2, 64)
    keys, vals = fill(cache, table, [200, 37], 2)
    q = randn((2, 2, 4, 64), 3)
    o, lse = attend(q, cache, table, [200, 37], scale=scale)
    check(q, o, lse, keys, vals, scale, True, kind)


def write_rows(cache, table, k, v):
    """k, v float32 [n, Hkv, d] into one sequence's rows, quantised by the oracle."""
    n = len(k)
    pg, at = np.array([paged.place(table[0], p, cache.page_size) for p in range(n)]).T
    pg, at = torch.tensor(pg).cuda(), torch.tensor(at).cuda()
    vals = []
    for t, sz, x in ((cache.k, cache.k_sz, k), (cache.v, cache.v_sz, v)):
        codes, scale, zero = paged.quantise(x)
        t[pg, at] = torch.tensor(paged.pack(codes)).cuda()
        sz[pg, at] = torch.tensor(np.stack((scale, zero), -1)).cuda().bfloat16()
        vals.append([paged.values(codes, scale, zero)])
    return vals


@pytest.mark.parametrize("what", ["constant", "tiny", "large", "one_large_value", "one_large_key", "zero_values", "mixed"])
def test_four_bit_values_of_any_size(what):
    """Scales over many orders of magnitude: the weights times scale must neither overflow nor vanish."""
    r = np.random.default_rng(3)
    n, d = 150, 128
    k, v = (paged.bf16_nearest(r.standard_normal((n, 1, d)).astype(np.float32)) for _ in range(2))
    if what == "constant":
        v[:] = 2.5
    if what == "tiny":
        v *= np.float32(2.0 ** -60)
    if what == "large":
        v *= np.float32(2.0 ** 60)
    if what == "one_large_value":
        v[77] *= np.float32(2.0 ** 16)
    if what == "one_large_key":
        k[33] *= 64
    if what == "zero_values":
        v[:100] = 0
    if what == "mixed":
        v *= np.exp2(r.integers(-40, 40, (n, 1, 1))).astype(np.float32)
    table, pages = make_table([n], 16, 1)
    cache = make_cache("int4", pages, 16, 1, d)
    keys, vals = write_rows(cache, table, k, v)
    q = randn((1, 1, 4, d), 5)
    o, lse = attend(q, cache, table, [n])
    check(q, o, lse, keys, vals, d ** -0.5, True, "int4")
    if what == "constant":
        assert bool((o == 2.5).all())


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -20, 2.0 ** 30])
def test_queries_of_any_size(size):
    table, pages = make_table([90], 16, 1)
    cache = make_cache("int4", pages, 16, 1, 64)
    keys, vals = fill(cache, table, [90], 4)
    q = randn((1, 1, 3, 64), 5) * size
    o, lse = attend(q, cache, table, [90], scale=0.125 / size)
    check(q, o, lse, keys, vals, 0.125 / size, True, "int4")
    z = torch.zeros_like(q)      # all scores 0: the mean of the values
    o, lse = attend(z, cache, table, [90])
    check(z, o, lse, keys, vals, 0.125, True, "int4")


@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_offsets_beyond_32_bits(kind):
    """A pool of over 2^32 bytes for keys alone, the sequence's pages at its two ends."""
    d, ps, Hkv = 128, 64, 8
    row = 256 if kind == "bf16" else 64
    pages = (1 << 32) // (ps * Hkv * row) + 40
    cache = binding.PagedKVCache.allocate(pages, ps, Hkv, d, kind)
    table = np.array([[pages - 1, 0, pages - 2, 7]], dtype=np.int32)
    keys, vals = fill(cache, table, [250], 6)
    q = randn((1, 1, 16, d), 7)
    o, lse = attend(q, cache, table, [250])
    check(q, o, lse, keys, vals, d ** -0.5, True, kind)
    k, v = binding.attn_paged_gather(cache, i32([0, 250]), i32(table), 250)
    assert np.array_equal(np32(k), paged.bf16_nearest(np.float32(keys[0])))
    assert np.array_equal(np32(v), paged.bf16_nearest(np.float32(vals[0])))


@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_bad_pages_and_lengths_are_reported_and_stay_in_their_sequence(kind):
    lens = [100, 64, 30]
    table, pages = make_table(lens, 16, 1)
    cache = make_cache(kind, pages, 16, 2, 128)
    fill(cache, table, lens, 2)
    q = randn((3, 1, 8, 128), 3)
    want, lse = attend(q, cache, table, lens)
    for change in ("high", "negative", "long", "below"):
        t, n = table.copy(), list(lens)
        if change == "high":
            t[0, 3] = pages
        if change == "negative":
            t[0, 0] = -1
        if change == "long":
            n[0] = table.shape[1] * 16 + 1
        if change == "below":
            n[0] = -5
        try:
            o, _ = binding.attn_fwd_paged(q, cache, i32(t), i32(n))
            assert binding.attn_get_status() == (binding.ATTN_ERR_INVALID_ARG, 0x2000000D), change
        finally:
            binding.attn_clear_status()
        # shares are dealt by length: a changed length moves the cuts of the others and with them the last bits
        assert torch.allclose(o[1:].float(), want[1:].float(), atol=0, rtol=2.0 ** -6 if change in ("long", "below") else 0), change


def test_pages_shared_by_sequences():
    """A common prefix: two tables lead to the same pages."""
    cache = make_cache("int4", 8, 16, 2, 64)
    keys, vals = fill(cache, np.array([[0, 1, 2, 3]]), [60], 2)
    q = randn((2, 1, 4, 64), 3)
    o, lse = attend(q, cache, np.array([[0, 1, 2, 3], [0, 1, -1, -1]], dtype=np.int32), [60, 32])
    check(q, o, lse, [keys[0], keys[0][:32]], [vals[0], vals[0][:32]], 64 ** -0.5, True, "int4")


@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_prefill_then_decode(kind):
    """As a server runs it: prompts through norm and rotation and the ragged forward, their rows into the cache, then one
    token at a time, captured once and replayed while the lengths grow; a padded entry of the batch stays empty."""
    H, Hkv, d, ps = 8, 2, 128, 16
    prompts, steps = [37, 90, 0], 20
    ends = [n + steps if n else 0 for n in prompts]
    table, pages = make_table(ends, ps, 4)
    cache = make_cache(kind, pages, ps, Hkv, d)
    cos, sin = tables(200, d // 2)
    w = [torch.ones(d, device="cuda") * 1.5, torch.ones(d, device="cuda")]
    total = sum(prompts)
    cu = i32(np.concatenate(([0], np.cumsum(prompts))))
    pos = i32(np.concatenate([np.arange(n) for n in prompts]))
    x = randn((total, H + 2 * Hkv, d), 5)
    q, k = binding.attn_qk_norm_rope(x[:, :H], x[:, H:H + Hkv], cos, sin, pos, *w)
    v = x[:, H + Hkv:]
    tab = i32(table)
    binding.attn_paged_append(cache, k, v, cu, i32([0, 0, 0]), tab)
    ok()

    B = 3
    lens = i32(prompts)
    live = i32([1, 1, 0])
    x1 = torch.empty((B, H + 2 * Hkv, d), dtype=torch.bfloat16, device="cuda")
    cu1 = i32([0, 1, 2, 2])       # the third entry brings no token
    ws = torch.empty(binding.attn_fwd_paged_workspace_bytes(cache, B, H, 1), dtype=torch.uint8, device="cuda")

    def step():
        q1, k1 = binding.attn_qk_norm_rope(x1[:, :H], x1[:, H:H + Hkv], cos, sin, lens, *w)
        binding.attn_paged_append(cache, k1, x1[:, H + Hkv:], cu1, lens, tab)
        lens.add_(live)
        return q1, binding.attn_fwd_paged(q1.unsqueeze(1), cache, tab, lens, workspace=ws)

    news = [randn((B, H + 2 * Hkv, d), 100 + i) for i in range(steps)]
    x1.copy_(news[0])
    step()                        # once as it is, then captured
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        q1, (o, lse) = step()
    for i in range(1, steps):
        x1.copy_(news[i])
        graph.replay()
    ok()
    assert lens.tolist() == [57, 110, 0]

    # What the cache holds now, read back, and the last step's attention over it.
    n = [57, 110, 0]
    kk, vv = binding.attn_paged_gather(cache, i32([0, 57, 167, 167]), tab, 167)
    ok()
    _, knew = binding.attn_qk_norm_rope(news[-1][:, :H], news[-1][:, H:H + Hkv], cos, sin, i32([56, 109, 0]), *w)
    assert torch.equal(kk[:37], k[:37]) or kind == "int4"
    last = np32(knew[1])
    if kind == "int4":
        last = paged.bf16_nearest(np.float32(paged.values(*paged.quantise(last))))
    assert np.array_equal(np32(kk[166]), last)
    if kind == "bf16":            # the same attention through the ragged forward
        plan = binding.attn_varlen_plan(i32([0, 1, 2, 2]), i32([0, 57, 167, 167]), H, 2, 167, d, True)
        o2, lse2 = binding.attn_fwd_varlen(q1[:2].contiguous(), kk, vv, i32([0, 1, 2, 2]), i32([0, 57, 167, 167]), plan, True)
        ok()
        assert float((o[:2, 0].float() - o2.float()).norm() / o2.float().norm()) <= 2.0 ** -7     # two sides, 2^-8 each
        assert float((lse[:2, :, 0] - lse2.T).abs().max()) <= 1e-3
    keys, vals = ([np.float64(np32(t[a:b])) for a, b in ((0, 57), (57, 167), (167, 167))] for t in (kk, vv))
    o_ref, lse_ref = paged.attention_paged(np32(q1)[:, None], keys, vals, d ** -0.5, True)
    # 4-bit values read back are rounded to bf16 once more, 2^-8 of each
    diff = np32(o) - o_ref
    assert np.linalg.norm(diff) <= (2.0 ** -8 + (2.0 ** -8 if kind == "bf16" else 2.0 ** -7)) * np.linalg.norm(o_ref)
    assert bool((o[2] == 0).all()) and bool(torch.isneginf(lse[2]).all())


def test_two_graphs_with_workspaces_of_their_own_run_at_once():
    table, pages = make_table([5000], 16, 1)
    cache = make_cache("int4", pages, 16, 1, 128)
    fill(cache, table, [5000], 2)
    tab, n = i32(table), i32([5000])
    qs = [randn((1, 1, 8, 128), s) for s in (3, 4)]
    want = [binding.attn_fwd_paged(q, cache, tab, n) for q in qs]
    graphs, outs = [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(binding.attn_fwd_paged(q, cache, tab, n))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    ok()
    for (o, lse), (ow, lw) in zip(outs, want):
        assert torch.equal(o, ow) and torch.equal(lse, lw)


def test_binding_checks():
    cache = binding.PagedKVCache.allocate(4, 16, 2, 128, "int4")
    table, n = i32([[0, 1]]), i32([5])
    q = randn((1, 1, 8, 128), 1)
    k = randn((3, 2, 128), 1)
    bad = [
        lambda: binding.attn_fwd_paged(q[..., :64], cache, table, n), lambda: binding.attn_fwd_paged(q.float(), cache, table, n),
        lambda: binding.attn_fwd_paged(q[:, :, :7].contiguous(), cache, table, n),
        lambda: binding.attn_fwd_paged(q, cache, table.long(), n), lambda: binding.attn_fwd_paged(q, cache, table, i32([5, 5])),
        lambda: binding.attn_fwd_paged(q.expand(2, 1, 8, 128).contiguous(), cache, table, n),
        lambda: binding.attn_fwd_paged(q, cache, table.cpu(), n), lambda: binding.attn_fwd_paged(q, cache, table, n, lse=n),
        lambda: binding.attn_paged_append(cache, k, k[:2], i32([0, 3]), n, table),
        lambda: binding.attn_paged_append(cache, k[:, :1], k[:, :1], i32([0, 3]), n, table),
        lambda: binding.attn_paged_append(cache, k, k, i32([3]), n, table),
        lambda: binding.attn_paged_append(cache, k, k, i32([0, 3]), n, table, cos=torch.ones(9, 64).cuda()),
        lambda: binding.attn_paged_gather(cache, i32([0, 3]), table, 3, k=k.float()),
        lambda: binding.PagedKVCache(cache.k, cache.v), lambda: binding.PagedKVCache(cache.k, cache.v, cache.k_sz),
        lambda: binding.PagedKVCache(cache.k, cache.v[:3], cache.k_sz, cache.v_sz),
        lambda: binding.PagedKVCache(cache.k.transpose(2, 3), cache.v.transpose(2, 3), cache.k_sz, cache.v_sz),
        lambda: binding.PagedKVCache.allocate(4, 16, 2, 128, "int8"),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(binding.AttnError):      # too small a workspace
        binding.attn_fwd_paged(q, cache, table, n, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(binding.AttnError):
        binding.attn_paged_append(binding.PagedKVCache.allocate(4, 24, 2, 128), k, k, i32([0, 3]), n, table)
    ok()


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("n", [40, 20000])     # finished by one warp, and cut over many
def test_a_bad_query_row_stays_one_row(kind, n):
    table, pages = make_table([n], 16, 1)
    cache = make_cache(kind, pages, 16, 1, 64)
    keys, vals = fill(cache, table, [n], 4)
    q = randn((1, 1, 8, 64), 5)
    bad = q.clone()
    bad[0, 0, 3, 7], bad[0, 0, 5, 0] = float("nan"), float("inf")
    want, want_lse = attend(q, cache, table, [n])
    o, lse = attend(bad, cache, table, [n])
    good = [0, 1, 2, 4, 6, 7]
    assert bool(torch.isnan(o[0, 0, 3]).all()) and bool(torch.isnan(lse[0, 3]).all())
    assert bool(torch.isnan(o[0, 0, 5]).all())
    # the running maximum of other rows may move at other tiles: the last bit of a weight
    assert torch.allclose(o[0, 0, good].float(), want[0, 0, good].float(), rtol=2.0 ** -7, atol=2.0 ** -10)
    assert torch.allclose(lse[0, good], want_lse[0, good], rtol=2.0 ** -19)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_many_parts_few_parts_and_whole_units_in_one_call(kind):
    """One sequence over most warps (joined by four warps), some over a few (by one), some inside a share, empty ones
    between them; every call the same bits."""
    lens = [60000, 1, 0, 3000, 17, 0, 0, 900, 5000] + [5] * 40 + [2500]
    table, pages = make_table(lens, 32, 3)
    cache = make_cache(kind, pages, 32, 2, 128)
    keys, vals = fill(cache, table, lens, 4)
    q = randn((len(lens), 1, 6, 128), 5, 2.0)
    o, lse = attend(q, cache, table, lens)
    check(q, o, lse, keys, vals, 128 ** -0.5, True, kind)
    for _ in range(5):
        o2, lse2 = attend(q, cache, table, lens)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_every_number_of_keys_around_the_tiles():
    """Lengths 1 .. 140, each as its own call and all in one batch, d = 64 with 2 kv heads."""
    lens = list(range(1, 141))
    table, pages = make_table(lens, 16, 3)
    for kind in ("bf16", "int4"):
        cache = make_cache(kind, pages, 16, 2, 64)
        keys, vals = fill(cache, table, lens, 4)
        q = randn((len(lens), 2, 4, 64), 5, 2.0)
        o, lse = attend(q, cache, table, lens)
        check(q, o, lse, keys, vals, 0.125, True, kind)
        for b in range(0, 140, 13):
            o1, lse1 = attend(q[b:b + 1], cache, table[b:b + 1], lens[b:b + 1])
            check(q[b:b + 1], o1, lse1, keys[b:b + 1], vals[b:b + 1], 0.125, True, kind)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("d,H,Nq,lens", [
    (128, 8, 1, [30000, 33, 500, 70, 900, 0, 40, 1200]),    # one over nearly all warps, several cut in the rest
    (64, 4, 3, [9000, 700, 2, 650]),                        # 12 rows
    (256, 3, 1, [5000, 4000, 17, 3000]),
    (64, 20, 1, [4000]),                                    # two units
])
def test_few_units_of_any_length(kind, d, H, Nq, lens):
    """One kv head: few units for all warps, so a CTA of the joining kernel looks through many of them, and may find several."""
    table, pages = make_table(lens, 16, 13)
    cache = make_cache(kind, pages, 16, 1, d)
    keys, vals = fill(cache, table, lens, 14)
    q = randn((len(lens), Nq, H, d), 15, 2.0)
    o, lse = attend(q, cache, table, lens)
    check(q, o, lse, keys, vals, d ** -0.5, True, kind)


def test_calls_of_two_threads_at_once():
    """Each on a stream of its own, with its own cache; the results are those of calls one after the other."""
    import threading
    lens = [700, 45, 3000]
    table, pages = make_table(lens, 16, 3)
    jobs = []
    for seed in (1, 2):
        cache = make_cache("int4", pages, 16, 2, 128)
        fill(cache, table, lens, seed)
        q = randn((3, 1, 8, 128), seed + 5)
        jobs.append((cache, q, attend(q, cache, table, lens)))
    tab, n = i32(table), i32(lens)
    torch.cuda.synchronize()
    wrong, errors = [], []

    def run(cache, q, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(50):
                    got = binding.attn_fwd_paged(q, cache, tab, n)
                    if not all(torch.equal(x, y) for x, y in zip(got, want)):
                        wrong.append(1)
        except Exception as e:   # shown in the main thread
            errors.append(e)
    threads = [threading.Thread(target=run, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and not wrong
    ok()


def test_strides_of_single_tokens_and_heads_do_not_count():
    """A dimension of one entry may have any stride (exchange formats set it to 1)."""
    lens = [5]
    table, pages = make_table(lens, 16, 3)
    cache = make_cache("bf16", pages, 16, 1, 64)
    k, v = randn((1, 1, 64), 1), randn((1, 1, 64), 2)
    odd = [torch.as_strided(x, x.shape, (1, 1, 1)) for x in (k, v)]
    binding.attn_paged_append(cache, *odd, i32([0, 1]), i32([0]), i32(table))
    got = binding.attn_paged_gather(cache, i32([0, 1]), i32(table), 1)
    assert torch.equal(got[0], k) and torch.equal(got[1], v)
    y, _ = binding.attn_qk_norm_rope(odd[0])
    assert torch.equal(y, binding.attn_qk_norm_rope(k)[0])
    ok()


def test_captured_without_a_workspace_of_the_callers():
    """What a captured call allocates for itself stays with the graph: replays between other calls and allocations."""
    lens = [4000, 9, 700]
    table, pages = make_table(lens, 16, 3)
    cache = make_cache("int4", pages, 16, 2, 64)
    fill(cache, table, lens, 4)
    q, tab, n = randn((3, 1, 8, 64), 5), i32(table), i32(lens)
    want = attend(q, cache, table, lens)
    w = torch.ones(64, device="cuda")
    grads = binding.attn_qk_norm_rope_bwd(q, None, q, wq=w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = binding.attn_fwd_paged(q, cache, tab, n)
        again = binding.attn_qk_norm_rope_bwd(q, None, q, wq=w)
    for i in range(4):
        graph.replay()
        other = torch.full((1 << 22,), float(i), device="cuda")
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert torch.equal(again[0], grads[0]) and torch.equal(again[2], grads[2])
        assert all(torch.equal(x, y) for x, y in zip(attend(q, cache, table, lens), want))
        del other
    ok()


@pytest.mark.parametrize("d,rd,il", [(128, 128, False), (64, 64, False), (256, 256, False), (128, 64, False), (128, 128, True),
                                     (64, 32, True)])
def test_rotation_rounds_both_products(d, rd, il):
    """Pairs (a, a) and (a, -a) turned by cos = sin: one of the two sums is of equal products and has to be 0 exactly. A fused
    multiply-add would leave the product's rounding error there."""
    n, half = 64, rd // 2
    a = randn((n, 2, half), 3)
    sign = torch.where(torch.arange(half, device="cuda") % 2 == 0, 1.0, -1.0).bfloat16()
    k = randn((n, 2, d), 4)
    first, second = (slice(0, rd, 2), slice(1, rd, 2)) if il else (slice(0, half), slice(half, rd))
    k[..., first], k[..., second] = a, a * sign
    t = torch.rand((n, half), generator=torch.Generator().manual_seed(5)).cuda() + 0.3
    table, pages = make_table([n], 16, 3)
    cache = make_cache("bf16", pages, 16, 2, d)
    binding.attn_paged_append(cache, k, k, i32([0, n]), i32([0]), i32(table), cos=t, sin=t, interleaved=il)
    got, _ = binding.attn_paged_gather(cache, i32([0, n]), i32(table), n)
    ok()
    assert bool((got[..., first][..., sign > 0] == 0).all()) and bool((got[..., second][..., sign < 0] == 0).all())
    want = a.float() * t[:, None] * 2
    assert torch.allclose(got[..., second][..., sign > 0].float(), want[..., sign > 0], rtol=2 ** -8 + 2 ** -22, atol=0)


def test_no_room_for_an_output_is_torchs_error():
    """What torch.empty raises there, as in the rest of the binding: what a caller's retry catches. Nothing is launched."""
    cache, cu, table = binding.PagedKVCache.allocate(1, 16, 64, 256), i32([0, 1 << 28]), i32([[0]])
    with pytest.raises(torch.OutOfMemoryError):     # 2^28 rows of 64 * 256 bf16 values: 8 TB
        binding.attn_paged_gather(cache, cu, table, 1 << 28)
    ok()


@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_batches_without_sequences_or_tokens(kind):
    """Every call of a decoding step takes them, as the norm does, and leaves the cache as it was."""
    cache = binding.PagedKVCache.allocate(4, 16, 2, 128, kind)
    for B, Nq in ((0, 1), (0, 3), (2, 0), (0, 0)):
        q = torch.empty((B, Nq, 8, 128), dtype=torch.bfloat16, device="cuda")
        table, lens = torch.zeros((B, 2), dtype=torch.int32, device="cuda"), torch.full((B,), 5, dtype=torch.int32, device="cuda")
        for ws in (None, torch.empty(256, dtype=torch.uint8, device="cuda")):
            o, lse = binding.attn_fwd_paged(q, cache, table, lens, workspace=ws)
            assert o.shape == (B, Nq, 8, 128) and o.dtype == torch.bfloat16 and lse.shape == (B, 8, Nq) and lse.dtype == torch.float32
        out = torch.empty_like(q)
        assert binding.attn_fwd_paged(q, cache, table, lens, out=out)[0] is out
        k, cu = torch.empty((0, 2, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros(B + 1, dtype=torch.int32, device="cuda")
        binding.attn_paged_append(cache, k, k, cu, lens, table)
        assert binding.attn_paged_gather(cache, cu, table, 0)[0].shape == (0, 2, 128)
    ok()
    assert not bool(cache.k.any()) and not bool(cache.v.any())


@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_strides_of_single_pages_and_heads_of_a_cache_do_not_count(kind):
    """As those of single tokens: k's and v's may differ there, and need not be multiples of a row's pieces."""
    plain = binding.PagedKVCache.allocate(1, 16, 1, 64, kind)
    other = binding.PagedKVCache.allocate(1, 16, 1, 64, kind)

    def odd(t, page, head):
        return None if t is None else torch.as_strided(t, t.shape, (page, t.stride(1), head, *t.stride()[3:]))
    cache = binding.PagedKVCache(odd(other.k, 1, 1), odd(other.v, 3, 5), odd(other.k_sz, 1, 1), odd(other.v_sz, 7, 3))
    k, v, q = randn((9, 1, 64), 1), randn((9, 1, 64), 2), randn((1, 1, 4, 64), 3)
    got = []
    for c in (plain, cache):
        binding.attn_paged_append(c, k, v, i32([0, 9]), i32([0]), i32([[0]]))
        got.append((*binding.attn_fwd_paged(q, c, i32([[0]]), i32([9])), *binding.attn_paged_gather(c, i32([0, 9]), i32([[0]]), 9)))
    ok()
    assert all(torch.equal(x, y) for x, y in zip(*got))

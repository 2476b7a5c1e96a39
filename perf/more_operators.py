"""Cases of attention of new tokens' chunks over the paged key/value cache (bf16 or 4 bits), and of per-head norm with
rotary positions on several axes.

``run`` computes a case in plain torch operations, or, where ``own`` is true, through the library's entry points;
``exact`` gives the same results in 64 bits. Shapes follow the library's own workloads (32 query heads on 8 kv heads,
d = 128, 8192- and 16384-key sequences; d = 64 and 256 beside them).
"""
import math
import random

import torch

own = False

GROUP = 64                 # dims per (scale, zero) pair of the 4-bit cache
LOG = math.log
EPS = 1e-6
MOST_FLOPS = 1.9e12        # of a drawn attention case: the largest listed ones
MOST_BYTES = 1.6e9
MOST_ROWS = 2 * 8192 * 40 * 128   # values of a drawn norm case


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a batch: 32 new text tokens behind images, positions on three axes (latency counts)
        axes("axes_decode", False, B=32, N=1, H=32, Hkv=8, d=128, sections=(16, 24, 24), max_pos=16384),
        # prefill or training forward in the headline attention shape: text, images and video, q and k out of a fused projection
        axes("axes_prefill", False, B=2, N=8192, H=32, Hkv=8, d=128, sections=(16, 24, 24), max_pos=8192),
        # its backward, axes taking turns over the frequencies
        axes("axes_bwd_train", True, B=2, N=8192, H=32, Hkv=8, d=128, sections=(24, 20, 20), max_pos=8192, turns=True),
        # backward of a smaller image model: height and width alone, odd length, neighbouring pairs, half of each head rotated
        axes("axes_bwd_image", True, B=3, N=1777, H=12, Hkv=4, d=64, sections=(8, 8), max_pos=2048, interleaved=True),
        # the rest of a short prompt after a cached prefix, d = 64 model (latency counts)
        chunk("chunk_bf16_small", "bf16", B=1, decoding=0, new=61, past=1000, H=16, Hkv=4, d=64, ps=16),
        # a step of a server: 28 sequences decode, 4 have 500-odd tokens of their prompts computed, some entries are padding
        chunk("chunk_bf16_mixed", "bf16", B=34, decoding=28, new=512, past=16384, H=32, Hkv=8, d=128, ps=16),
        # chunks of long prompts over what is cached of them (the largest)
        chunk("chunk_bf16_prompt", "bf16", B=4, decoding=0, new=4096, past=8192, H=32, Hkv=8, d=128, ps=16),
        # d = 256, odd lengths, larger pages, four heads a group
        chunk("chunk_bf16_d256", "bf16", B=5, decoding=2, new=777, past=5000, H=16, Hkv=4, d=256, ps=64),
        # seven query heads on each of four kv heads, drafted tokens of many sequences: a short piece each
        chunk("chunk_bf16_drafts", "bf16", B=24, decoding=0, new=9, past=8192, H=28, Hkv=4, d=128, ps=32),
        # the prompts' chunks over a 4-bit cache
        chunk("chunk_int4_prompt", "int4", B=4, decoding=0, new=4096, past=8192, H=32, Hkv=8, d=128, ps=16),
        # the server's step over a 4-bit cache
        chunk("chunk_int4_mixed", "int4", B=34, decoding=28, new=512, past=16384, H=32, Hkv=8, d=128, ps=16),
        # a question of 300 tokens about one long cached document, 4-bit cache
        chunk("chunk_int4_long", "int4", B=1, decoding=0, new=300, past=65536, H=32, Hkv=8, d=128, ps=64),
    ]


def axes(name, backward, B, N, H, Hkv, d, sections, max_pos, turns=False, interleaved=False):
    """sections: pairs of each axis, in blocks, or the axes taking turns while they have pairs left."""
    return {"name": name, "op": "axes", "backward": backward, "B": B, "N": N, "H": H, "Hkv": Hkv, "d": d,
            "sections": ",".join(map(str, sections)), "max_pos": max_pos, "turns": turns, "interleaved": interleaved}


def chunk(name, cache, B, decoding, new, past, H, Hkv, d, ps):
    return {"name": name, "op": "chunk", "cache": cache, "B": B, "decoding": decoding, "new": new, "past": past, "H": H,
            "Hkv": Hkv, "d": d, "ps": ps, "lens_seed": 21}


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(LOG(lo), LOG(hi)))))


def draw(rng):
    d = rng.choice((64, 128, 128, 256))
    Hkv = rng.choice((1, 2, 4, 8, 16))
    G = rng.choice((1, 2, 3, 4, 4, 5, 7, 8, 12))
    if rng.random() < 0.4:
        B = log_int(rng, 1, 40)
        N = max(1, min(log_int(rng, 1, 9000), MOST_ROWS // (B * Hkv * (G + 1) * d)))
        pairs = rng.choice((8, 16, d // 4, d // 2, d // 2))
        n_axes = rng.choice((2, 3, 3, 4))
        cuts = sorted(rng.randrange(pairs + 1) for _ in range(n_axes - 1))
        sections = [b - a for a, b in zip([0] + cuts, cuts + [pairs])]
        c = axes("", rng.random() < 0.5, B, N, Hkv * G, Hkv, d, sections, N + rng.randrange(1, 5000), rng.random() < 0.5,
                 rng.random() < 0.4)
    else:
        while True:
            B = log_int(rng, 1, 40)
            c = chunk("", rng.choice(("bf16", "int4")), B, rng.randrange(B + 1) if rng.random() < 0.5 else 0,
                      log_int(rng, 1, 4096), log_int(rng, 1, 65536), Hkv * G, Hkv, d, rng.choice((16, 32, 48, 64, 256)))
            c["lens_seed"] = rng.randrange(1 << 20)
            w = work(c)
            if w["flops"] <= MOST_FLOPS and w["bytes"] <= MOST_BYTES:
                break
    del c["name"]
    return c


def lengths(case):
    """(new tokens, keys cached before them) of every sequence, from the case alone."""
    r = random.Random(case["lens_seed"])
    B = case["B"]
    chunks = B - case["decoding"]
    new = [max(1, case["new"] - r.randrange(1 + case["new"] // 4)) for _ in range(chunks)] + [1] * case["decoding"]
    past = [r.randrange(case["past"] // 2, case["past"] + 1) for _ in range(B)]
    if B > 30:             # padding of a captured batch
        new[chunks - 1] = new[chunks // 2] = past[chunks - 1] = 0
    order = list(range(B))
    r.shuffle(order)
    return [new[i] for i in order], [past[i] for i in order]


def pair_axes(case):
    """The axis of each pair."""
    left = [int(x) for x in case["sections"].split(",")]
    if not case["turns"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    order = []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                order.append(a)
    return order


# ---------------------------------------------------------------------------------------------- inputs

def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def tables(max_pos, pairs):
    """cos and sin of pos * 10000^(-i/pairs), angles in 64 bits."""
    inv = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device="cuda") / pairs)
    a = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * inv
    return a.cos().float(), a.sin().float()


def randn(shape, g, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()


def page_tables(lens, ps, g):
    """Pages of every sequence, scattered over the pool; entries past a sequence's pages are -1. (table, pages in the pool)"""
    need = [-(-n // ps) for n in lens]
    pool = sum(need) + 3
    perm = torch.randperm(pool, generator=g, device="cuda").int()
    width = max(1, max(need))
    n = torch.tensor(need, device="cuda")
    col = torch.arange(width, device="cuda")
    first = torch.cumsum(n, 0) - n
    at = (first[:, None] + col).clamp(max=pool - 1)
    return torch.where(col < n[:, None], perm[at], torch.tensor(-1, dtype=torch.int32, device="cuda")).contiguous(), pool


def make_cache(case, pool, g):
    """A pool of pages with contents as after many tokens: [page, row, kv head, ...] views of head-major pages."""
    ps, Hkv, d = case["ps"], case["Hkv"], case["d"]
    c = {}
    for x in "kv":
        if case["cache"] == "bf16":
            c[x] = randn((pool, Hkv, ps, d), g).transpose(1, 2)
        else:
            c[x] = torch.randint(0, 256, (pool, Hkv, ps, d // 2), generator=g, device="cuda", dtype=torch.uint8).transpose(1, 2)
            scale = 0.2 + 0.2 * torch.rand((pool, Hkv, ps, d // GROUP), generator=g, device="cuda")
            zero = -7.5 * scale + 0.3 * torch.randn(scale.shape, generator=g, device="cuda")
            c[x + "_sz"] = torch.stack((scale, zero), -1).bfloat16().transpose(1, 2)
    return c


def grid_positions(case, n_axes, g):
    """int32 [axes, B, N]: a run of text (all axes alike), then frames of a raster whose last two axes are row and column
    and whose first is the frame, then text again behind the greatest position so far."""
    B, N, top = case["B"], case["N"], case["max_pos"]
    t = torch.arange(N, device="cuda")
    text = N // 4
    side = max(1, math.isqrt(max(1, N // 8)))
    i = (t - text).clamp(min=0)
    raster = [i // (side * side), i // side % side, i % side]
    raster = [raster[0]] * (n_axes - 3) + raster[max(0, 3 - n_axes):]
    image_end = text + N // 2
    after = text + max(side, -(-max(1, N // 2) // (side * side))) + (t - image_end)
    pos = torch.stack([torch.where(t < text, t, torch.where(t < image_end, text + a, after)) for a in raster])
    shift = torch.randint(0, max(1, top - N + 1), (1, B, 1), generator=g, device="cuda")
    return (pos[:, None] + shift).clamp(max=top - 1).int().contiguous()


def prepare(case, seed):
    g = generator(seed)
    s = {"case": case}
    d, H, Hkv = case["d"], case["H"], case["Hkv"]
    if case["op"] == "axes":
        B, N = case["B"], case["N"]
        order = pair_axes(case)
        qkv = randn((B, N, H + 2 * Hkv, d), g)
        s["q"], s["k"] = qkv[:, :, :H], qkv[:, :, H:H + Hkv]
        s["wq"], s["wk"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
        s["cos"], s["sin"] = tables(case["max_pos"], len(order))
        s["positions"] = grid_positions(case, len(case["sections"].split(",")), g)
        s["pair_axis"] = bytes(order)
        if case["backward"]:
            s["dq_out"], s["dk_out"] = randn((B, N, H, d), g, 0.1), randn((B, N, Hkv, d), g, 0.1)
        return s
    new, past = lengths(case)
    s["new"], s["keys"] = new, [n + p for n, p in zip(new, past)]
    s["table"], pool = page_tables(s["keys"], case["ps"], g)
    s.update(make_cache(case, pool, g))
    s["cu"] = torch.tensor([0] + new, device="cuda").cumsum(0).int()
    s["lens"] = torch.tensor(s["keys"], dtype=torch.int32, device="cuda")
    s["q"] = randn((sum(new), H, d), g, 2.0)
    if own:
        from exact_attention_72_gb300 import binding
        s["handle"] = binding.PagedKVCache(s["k"], s["v"], s.get("k_sz"), s.get("v_sz"))
        n = binding.attn_fwd_paged_varlen_workspace_bytes(s["handle"], case["B"], H, sum(new))
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if own:
        return run_own(s, case)
    if case["op"] == "axes":
        return plain_axes_bwd(s, case) if case["backward"] else plain_axes(s, case)
    return plain_chunk(s, case)


def run_own(s, case):
    from exact_attention_72_gb300 import binding
    if case["op"] == "axes":
        kw = dict(cos=s["cos"], sin=s["sin"], positions=s["positions"], pair_axis=s["pair_axis"], wq=s["wq"], wk=s["wk"],
                  eps=EPS, interleaved=case["interleaved"])
        if case["backward"]:
            return binding.attn_qk_norm_rope_axes_bwd(s["q"], s["k"], s["dq_out"], s["dk_out"], **kw)
        return binding.attn_qk_norm_rope_axes(s["q"], s["k"], **kw)
    return binding.attn_fwd_paged_varlen(s["q"], s["handle"], s["table"], s["cu"], s["lens"], causal=True,
                                         workspace=s["workspace"])


def angles(s):
    """cos and sin [B, N, 1, pairs] of every token's pairs."""
    pos = s["positions"].long()
    axis = torch.tensor(list(s["pair_axis"]), device="cuda")
    column = torch.arange(axis.numel(), device="cuda")
    row = pos.permute(1, 2, 0)[:, :, axis]                          # [B, N, pairs]
    return s["cos"][row, column][:, :, None], s["sin"][row, column][:, :, None]


def rotate(x, cos, sin, interleaved):
    """x [..., d] with cos and sin [..., pairs] of its positions."""
    h = cos.shape[-1]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        y[..., 0:2 * h:2], y[..., 1:2 * h:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        y[..., :h], y[..., h:2 * h] = a * cos - b * sin, b * cos + a * sin
    return y


def plain_axes(s, case):
    cos, sin = angles(s)

    def one(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        return rotate(x, cos, sin, case["interleaved"]).bfloat16()

    return one(s["q"], s["wq"]), one(s["k"], s["wk"])


def plain_axes_bwd(s, case):
    cos, sin = angles(s)

    def one(x, dy, w):
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        n = x * r
        du = rotate(dy.float(), cos, -sin, case["interleaved"])
        dw = (du * n).sum((0, 1, 2), dtype=torch.float64).float()
        gr = du * w
        return (r * (gr - n * (gr * n).mean(-1, keepdim=True))).bfloat16(), dw

    (dq, dwq), (dk, dwk) = one(s["q"], s["dq_out"], s["wq"]), one(s["k"], s["dk_out"], s["wk"])
    return dq, dk, dwq, dwk


def dequantise(codes, sz):
    """fp32 values of 4-bit rows codes [..., d/2] with sz [..., d/64, 2]."""
    x = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    sz = sz.float()
    return (sz[..., 1:] + sz[..., :1] * x).flatten(-2)


def plain_chunk(s, case):
    H, Hkv, d, ps = (case[x] for x in ("H", "Hkv", "d", "ps"))
    o = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((H, s["q"].shape[0]), device="cuda")
    first = 0
    for b, (nq, nk) in enumerate(zip(s["new"], s["keys"])):
        if nq == 0:
            continue
        at = s["table"][b, :-(-nk // ps)].long()
        kv = []
        for x in "kv":
            pages = s[x][at]
            pages = pages.float() if case["cache"] == "bf16" else dequantise(pages, s[x + "_sz"][at])
            kv.append(pages.flatten(0, 1)[:nk].transpose(0, 1))     # [Hkv, keys, d]
        q = s["q"][first:first + nq].float().unflatten(1, (Hkv, -1)).permute(1, 2, 0, 3).flatten(1, 2)
        S = (q @ kv[0].transpose(-1, -2)).unflatten(1, (-1, nq)) / math.sqrt(d)     # [Hkv, heads, nq, keys]
        last = torch.arange(nq, device="cuda")[:, None] + (nk - nq)
        S = S.masked_fill(torch.arange(nk, device="cuda") > last, -math.inf)
        m = S.amax(-1, keepdim=True)
        P = torch.exp(S - m)
        L = P.sum(-1, keepdim=True)
        x = (P / L).flatten(1, 2) @ kv[1]
        o[first:first + nq] = x.unflatten(1, (-1, nq)).permute(2, 0, 1, 3).flatten(1, 2).bfloat16()
        lse[:, first:first + nq] = (m + torch.log(L))[..., 0].flatten(0, 1)
        first += nq
    return o, lse


# ---------------------------------------------------------------------------------------------- what a pass needs

def work(case):
    d, H, Hkv = case["d"], case["H"], case["Hkv"]
    if case["op"] == "axes":
        tokens = case["B"] * case["N"]
        rows = tokens * (H + Hkv)
        pairs = sum(int(x) for x in case["sections"].split(","))
        small = min(case["max_pos"], tokens) * pairs * 8 + tokens * 4 * len(case["sections"].split(","))
        if case["backward"]:
            return {"bytes": rows * d * 6 + small, "flops": rows * d * 20}
        return {"bytes": rows * d * 4 + small, "flops": rows * d * 10}
    new, past = lengths(case)
    row = 2 * d if case["cache"] == "bf16" else d // 2 + 4 * (d // GROUP)
    keys = sum(n + p for n, p in zip(new, past) if n)
    seen = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, past))
    return {"bytes": 2 * Hkv * keys * row + sum(new) * H * (4 * d + 4), "flops": 4 * H * d * seen}


# ---------------------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return exact_axes(s, case) if case["op"] == "axes" else exact_chunk(s, case)


def exact_axes(s, case):
    d = case["d"]
    order = s["pair_axis"]
    z = torch.empty(case["B"], case["N"], 1, len(order), dtype=torch.complex128, device="cuda")
    for i, a in enumerate(order):
        row = s["positions"][a].long()
        z[:, :, 0, i] = torch.complex(s["cos"][row, i].double(), s["sin"][row, i].double())
    i = torch.arange(len(order), device="cuda")
    first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + len(order))

    def turned(x, by):
        y = x.clone()
        t = torch.complex(x[..., first], x[..., second]) * by
        y[..., first], y[..., second] = t.real, t.imag
        return y

    def forward(x, w):
        x = x.double()
        return turned(x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + EPS) * w.double(), z)

    if not case["backward"]:
        return forward(s["q"], s["wq"]), forward(s["k"], s["wk"])

    def backward(x, dy, w):
        # y = T (w x / a), a = sqrt(mean x^2 + eps): dx = w u / a - x (sum u w x) / (d a^3), with u = T^-1 dy
        x, u = x.double(), turned(dy.double(), z.conj())
        a2 = x.square().sum(-1, keepdim=True) / d + EPS
        uw = u * w.double()
        dx = uw / a2.sqrt() - x * (uw * x).sum(-1, keepdim=True) / (d * a2 ** 1.5)
        return dx, (u * x / a2.sqrt()).sum((0, 1, 2))

    (dq, dwq), (dk, dwk) = backward(s["q"], s["dq_out"], s["wq"]), backward(s["k"], s["dk_out"], s["wk"])
    return dq, dk, dwq, dwk


def exact_chunk(s, case):
    H, Hkv, d = (case[x] for x in ("H", "Hkv", "d"))
    G = H // Hkv
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros((H, s["q"].shape[0]), dtype=torch.float64, device="cuda")
    first = 0
    for b, (nq, nk) in enumerate(zip(s["new"], s["keys"])):
        if nq == 0:
            continue
        rows = slice(first, first + nq)
        first += nq
        pos = torch.arange(nk, device="cuda")
        page = s["table"][b, pos // case["ps"]].long()
        hidden = pos[None] > pos[nk - nq:, None]                    # query i stands at position nk - nq + i
        for j in range(Hkv):
            kv = []
            for x in "kv":
                value = s[x][page, pos % case["ps"], j]
                if case["cache"] == "int4":
                    sz = s[x + "_sz"][page, pos % case["ps"], j].double().repeat_interleave(GROUP, -2)
                    value = torch.stack((value % 16, value // 16), -1).reshape(nk, d).double() * sz[..., 0] + sz[..., 1]
                kv.append(value.double())
            for h in range(j * G, (j + 1) * G):
                S = (s["q"][rows, h].double() @ kv[0].T / d ** 0.5).masked_fill_(hidden, -math.inf)
                lse[h, rows] = torch.logsumexp(S, -1)
                o[rows, h] = torch.softmax(S, -1) @ kv[1]
    return o, lse

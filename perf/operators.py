"""Cases of the operators around the attention kernels: per-head norm and rotation of queries and keys, the paged
key/value cache in bf16 or 4 bits, and the attention that reads it.

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


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a batch: q and k of 32 new tokens at scattered positions (latency counts)
        norm_rope("norm_rope_decode", False, B=32, N=1, H=32, Hkv=8, d=128, rd=128, max_pos=16384),
        # prefill or training forward in the headline attention shape, q and k out of a fused projection
        norm_rope("norm_rope_prefill", False, B=2, N=8192, H=32, Hkv=8, d=128, rd=128, max_pos=8192),
        # its backward
        norm_rope("norm_rope_bwd_train", True, B=2, N=8192, H=32, Hkv=8, d=128, rd=128, max_pos=8192),
        # backward of a smaller model: odd length, interleaved pairs, half of each head rotated
        norm_rope("norm_rope_bwd_odd", True, B=3, N=1777, H=12, Hkv=4, d=64, rd=32, max_pos=2048, interleaved=True),
        # one decode step: a token for each of 64 sequences into a bf16 cache
        append("append_bf16_decode", "bf16", B=64, new=1, past=1500, Hkv=8, d=128, rd=128, ps=16),
        # chunks of prompts into a 4-bit cache, then the whole context read back to prefill on
        append("append_int4_prompt", "int4", B=4, new=4096, past=8192, Hkv=8, d=128, rd=128, ps=16),
        # short ragged prompts of a d = 64 model, interleaved pairs, part of each head rotated
        append("append_int4_d64", "int4", B=9, new=333, past=100, Hkv=4, d=64, rd=32, ps=32, interleaved=True),
        # decode in the library's split-KV workload shape, 4-bit cache
        attend("attend_int4_16k", "int4", B=8, Nq=1, H=32, Hkv=8, d=128, longest=16384, ragged=False, ps=16),
        # serving batch of very different lengths, 4-bit cache (the largest)
        attend("attend_int4_serving", "int4", B=32, Nq=1, H=32, Hkv=8, d=128, longest=32768, ragged=True, ps=16),
        # one short conversation of a d = 64 model (latency counts)
        attend("attend_int4_small", "int4", B=1, Nq=1, H=16, Hkv=4, d=64, longest=1000, ragged=False, ps=16),
        # the split-KV workload shape on a bf16 cache
        attend("attend_bf16_16k", "bf16", B=8, Nq=1, H=32, Hkv=8, d=128, longest=16384, ragged=False, ps=16),
        # three drafted tokens each, d = 256, odd lengths, larger pages, one padded entry of the batch
        attend("attend_bf16_draft_d256", "bf16", B=13, Nq=3, H=16, Hkv=4, d=256, longest=5000, ragged=True, ps=64),
    ]


def norm_rope(name, backward, B, N, H, Hkv, d, rd, max_pos, interleaved=False):
    return {"name": name, "op": "norm_rope", "backward": backward, "B": B, "N": N, "H": H, "Hkv": Hkv, "d": d, "rd": rd,
            "max_pos": max_pos, "interleaved": interleaved}


def append(name, cache, B, new, past, Hkv, d, rd, ps, interleaved=False):
    return {"name": name, "op": "append", "cache": cache, "B": B, "new": new, "past": past, "Hkv": Hkv, "d": d, "rd": rd,
            "ps": ps, "interleaved": interleaved, "lens_seed": 11}


def attend(name, cache, B, Nq, H, Hkv, d, longest, ragged, ps):
    return {"name": name, "op": "attend", "cache": cache, "B": B, "Nq": Nq, "H": H, "Hkv": Hkv, "d": d,
            "longest": longest, "ragged": ragged, "ps": ps, "lens_seed": 12}


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(LOG(lo), LOG(hi)))))


def draw(rng):
    kind = rng.choice(("forward", "backward", "append", "append", "attend", "attend", "attend"))
    d = rng.choice((64, 128, 128, 256))
    Hkv = rng.choice((1, 2, 4, 8, 16))
    if kind in ("forward", "backward"):
        G = rng.choice((1, 2, 3, 4, 7, 8))
        B = log_int(rng, 1, 40)
        N = max(1, min(log_int(rng, 1, 9000), 2 * 8192 * 40 * 128 // (B * Hkv * (G + 1) * d)))
        c = norm_rope("", kind == "backward", B, N, Hkv * G, Hkv, d, rng.choice((16, d // 2, d, d)), N + rng.randrange(5000),
                      rng.random() < 0.4)
    elif kind == "append":
        B = log_int(rng, 1, 70)
        new = log_int(rng, 1, 4096)
        past = log_int(rng, 1, 8192)
        fit = 4 * 12288 * 8 * 128 / (B * (new + past) * Hkv * d)
        if fit < 1:
            new, past = max(1, int(new * fit)), max(1, int(past * fit))
        c = append("", rng.choice(("bf16", "int4")), B, new, past, Hkv, d, rng.choice((16, d // 2, d, d)),
                   rng.choice((16, 32, 64, 256)), rng.random() < 0.4)
    else:
        B = log_int(rng, 1, 40)
        G = rng.choice((1, 2, 3, 4, 5, 8, 12))
        Nq = rng.choice((1, 1, 1, 2, 4))
        kind = rng.choice(("bf16", "int4", "int4"))
        most = 32 * 16000 * 8 * 128 if kind == "int4" else 8 * 16384 * 8 * 128
        longest = max(16, min(log_int(rng, 16, 65536), most // (B * Hkv * d * max(1, Nq * G // 8))))
        c = attend("", kind, B, Nq, Hkv * G, Hkv, d, longest, rng.random() < 0.6, rng.choice((16, 32, 64, 256)))
    del c["name"]
    if "lens_seed" in c:
        c["lens_seed"] = rng.randrange(1 << 20)
    return c


def lengths(case):
    """Key lengths of an attend case, or (new, past) of an append case: from the case alone."""
    r = random.Random(case["lens_seed"])
    if case["op"] == "attend":
        if not case["ragged"]:
            return [case["longest"] - (b % 3) for b in range(case["B"])]
        lens = [max(1, int(case["longest"] * r.random())) for _ in range(case["B"])]
        lens[0] = case["longest"]
        if case["B"] > 8:
            lens[r.randrange(1, case["B"])] = 0
        return lens
    new = [max(1, case["new"] - r.randrange(1 + case["new"] // 3)) for _ in range(case["B"])]
    past = [r.randrange(case["past"] + 1) for _ in range(case["B"])]
    return new, past


# ---------------------------------------------------------------------------------------------- inputs

def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def tables(max_pos, rd):
    """cos and sin of pos * 10000^(-2i/rd), angles in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, rd, 2, dtype=torch.float64, device="cuda") / rd)
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


def prepare(case, seed):
    g = generator(seed)
    s = {"case": case}
    d = case["d"]
    if case["op"] == "norm_rope":
        B, N, H, Hkv, rd = (case[x] for x in ("B", "N", "H", "Hkv", "rd"))
        qkv = randn((B, N, H + 2 * Hkv, d), g)
        s["q"], s["k"] = qkv[:, :, :H], qkv[:, :, H:H + Hkv]
        s["wq"], s["wk"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
        s["cos"], s["sin"] = tables(case["max_pos"], rd)
        start = torch.randint(0, case["max_pos"] - N + 1, (B, 1), generator=g, device="cuda")
        s["positions"] = (start + torch.arange(N, device="cuda")).int()
        if case["backward"]:
            s["dq_out"], s["dk_out"] = randn((B, N, H, d), g, 0.1), randn((B, N, Hkv, d), g, 0.1)
        return s
    if case["op"] == "append":
        new, past = lengths(case)
        s["table"], pool = page_tables([n + p for n, p in zip(new, past)], case["ps"], g)
        s.update(make_cache(case, pool, g))
        s["total"] = sum(new)
        kv = randn((s["total"], 2 * case["Hkv"], d), g)
        s["k_new"], s["v_new"] = kv[:, :case["Hkv"]], kv[:, case["Hkv"]:]
        s["cu"] = torch.tensor([0] + new, device="cuda").cumsum(0).int()
        s["past"] = torch.tensor(past, dtype=torch.int32, device="cuda")
        s["cu_all"] = torch.tensor([0] + [n + p for n, p in zip(new, past)], device="cuda").cumsum(0).int()
        s["total_all"] = sum(new) + sum(past)
        s["cos"], s["sin"] = tables(case["new"] + case["past"], case["rd"])
    else:
        lens = lengths(case)
        s["table"], pool = page_tables(lens, case["ps"], g)
        s.update(make_cache(case, pool, g))
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = randn((case["B"], case["Nq"], case["H"], d), g, 2.0)
    if own:
        from exact_attention_72_gb300 import binding
        s["handle"] = binding.PagedKVCache(s["k"], s["v"], s.get("k_sz"), s.get("v_sz"))
        if case["op"] == "attend":
            n = binding.attn_fwd_paged_workspace_bytes(s["handle"], case["B"], case["H"], case["Nq"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if own:
        return run_own(s, case)
    if case["op"] == "norm_rope":
        return plain_norm_rope_bwd(s, case) if case["backward"] else plain_norm_rope(s, case)
    return plain_append(s, case) if case["op"] == "append" else plain_attend(s, case)


def run_own(s, case):
    from exact_attention_72_gb300 import binding
    if case["op"] == "norm_rope":
        kw = dict(cos=s["cos"], sin=s["sin"], positions=s["positions"], wq=s["wq"], wk=s["wk"], eps=1e-6,
                  interleaved=case["interleaved"])
        if case["backward"]:
            return binding.attn_qk_norm_rope_bwd(s["q"], s["k"], s["dq_out"], s["dk_out"], **kw)
        return binding.attn_qk_norm_rope(s["q"], s["k"], **kw)
    if case["op"] == "append":
        binding.attn_paged_append(s["handle"], s["k_new"], s["v_new"], s["cu"], s["past"], s["table"], cos=s["cos"],
                                  sin=s["sin"], interleaved=case["interleaved"])
        if case["cache"] == "bf16":
            return s["k"], s["v"]
        return binding.attn_paged_gather(s["handle"], s["cu_all"], s["table"], s["total_all"])
    return binding.attn_fwd_paged(s["q"], s["handle"], s["table"], s["lens"], causal=True, workspace=s["workspace"])


def rotate(x, cos, sin, interleaved):
    """x [..., d] with cos and sin [..., rd/2] of its positions."""
    h = cos.shape[-1]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        y[..., 0:2 * h:2], y[..., 1:2 * h:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        y[..., :h], y[..., h:2 * h] = a * cos - b * sin, b * cos + a * sin
    return y


def plain_norm_rope(s, case):
    cos, sin = (s[x][s["positions"].long()][:, :, None] for x in ("cos", "sin"))

    def one(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        return rotate(x, cos, sin, case["interleaved"]).bfloat16()

    return one(s["q"], s["wq"]), one(s["k"], s["wk"])


def plain_norm_rope_bwd(s, case):
    cos, sin = (s[x][s["positions"].long()][:, :, None] for x in ("cos", "sin"))

    def one(x, dy, w):
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        n = x * r
        du = rotate(dy.float(), cos, -sin, case["interleaved"])
        dw = (du * n).sum((0, 1, 2), dtype=torch.float64).float()
        gr = du * w
        return (r * (gr - n * (gr * n).mean(-1, keepdim=True))).bfloat16(), dw

    (dq, dwq), (dk, dwk) = one(s["q"], s["dq_out"], s["wq"]), one(s["k"], s["dk_out"], s["wk"])
    return dq, dk, dwq, dwk


def toward(x, up):
    """fp32 x rounded to bf16 upward or downward."""
    bits = x.view(torch.int32)
    cut = bits & -65536
    away = (cut != bits) & ((bits < 0) != up)      # what was cut off has to count: away from zero
    return (cut + away.int() * 65536).view(torch.float32)


def quantise(x):
    """x fp32 [T, Hkv, d] in 4 bits: bytes [T, Hkv, d/2] (even dims in the low half), (scale, zero) [T, Hkv, d/64, 2]."""
    x = x.unflatten(-1, (-1, GROUP))
    lo, hi = x.amin(-1), x.amax(-1)
    zero = toward(lo, False)
    least = torch.maximum(lo.abs(), hi.abs()) * 2.0 ** -20
    fifteen = torch.full_like(hi, 15.0)             # a tensor: a number would be turned into a product with 1/15
    scale = toward(torch.maximum((hi - zero) / fifteen, least).clamp(min=2.0 ** -100), True)
    code = torch.round((x - zero[..., None]) / scale[..., None]).clamp(0, 15).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.stack((scale, zero), -1).bfloat16()


def dequantise(codes, sz):
    """fp32 values of 4-bit rows codes [..., d/2] with sz [..., d/64, 2]."""
    x = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    sz = sz.float()
    return (sz[..., 1:] + sz[..., :1] * x).flatten(-2)


def plain_append(s, case):
    n, ps = s["total"], case["ps"]
    row = torch.arange(n, device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), row, right=True)
    pos = s["past"][b].long() + row - s["cu"][b].long()
    page, at = s["table"][b, pos // ps].long(), pos % ps
    k = rotate(s["k_new"].float(), s["cos"][pos][:, None], s["sin"][pos][:, None], case["interleaved"])
    if case["cache"] == "bf16":
        s["k"][page, at], s["v"][page, at] = k.bfloat16(), s["v_new"]
        return s["k"], s["v"]
    s["k"][page, at], s["k_sz"][page, at] = quantise(k)
    s["v"][page, at], s["v_sz"][page, at] = quantise(s["v_new"].float())
    row = torch.arange(s["total_all"], device="cuda")
    b = torch.searchsorted(s["cu_all"][1:].long(), row, right=True)
    pos = row - s["cu_all"][b].long()
    page, at = s["table"][b, pos // ps].long(), pos % ps
    return tuple(dequantise(s[x][page, at], s[x + "_sz"][page, at]).bfloat16() for x in "kv")


def plain_attend(s, case):
    B, Nq, H, Hkv, d = (case[x] for x in ("B", "Nq", "H", "Hkv", "d"))
    at = s["table"].long().clamp(min=0)
    kv = []
    for x in "kv":
        pages = s[x][at]
        pages = pages.float() if case["cache"] == "bf16" else dequantise(pages, s[x + "_sz"][at])
        kv.append(pages.flatten(1, 2).transpose(1, 2))              # [B, Hkv, keys, d]
    q = s["q"].float().reshape(B, Nq, Hkv, H // Hkv, d).permute(0, 2, 1, 3, 4).flatten(2, 3)
    S = (q @ kv[0].transpose(-1, -2)).unflatten(2, (Nq, -1)) / math.sqrt(d)
    key = torch.arange(S.shape[-1], device="cuda")
    sees = s["lens"].long()[:, None] - Nq + 1 + torch.arange(Nq, device="cuda")      # keys that query i sees: the first so many
    S = S.masked_fill((key >= sees[..., None])[:, None, :, None], -math.inf)
    m = S.amax(-1, keepdim=True)
    P = torch.exp(S - torch.where(m == -math.inf, torch.zeros_like(m), m))
    L = P.sum(-1, keepdim=True)
    o = (P / torch.where(L == 0, torch.ones_like(L), L)).flatten(2, 3) @ kv[1]
    o = o.unflatten(2, (Nq, -1)).permute(0, 2, 1, 3, 4).flatten(2, 3).bfloat16()
    lse = (m + torch.log(L))[..., 0].permute(0, 1, 3, 2).reshape(B, H, Nq)
    return o, lse


# ---------------------------------------------------------------------------------------------- what a pass needs

def row_bytes(case):
    """A key's or value's row of one head in the cache."""
    return 2 * case["d"] if case["cache"] == "bf16" else case["d"] // 2 + 4 * (case["d"] // GROUP)


def work(case):
    d, Hkv = case["d"], case["Hkv"]
    if case["op"] == "norm_rope":
        rows = case["B"] * case["N"] * (case["H"] + Hkv)
        table = min(case["max_pos"], case["B"] * case["N"]) * case["rd"] * 4
        if case["backward"]:
            return {"bytes": rows * d * 6 + table, "flops": rows * d * 20}
        return {"bytes": rows * d * 4 + table, "flops": rows * d * 10}
    if case["op"] == "append":
        new, past = (sum(x) for x in lengths(case))
        n = 2 * Hkv * (new * (2 * d + row_bytes(case)))
        if case["cache"] == "int4":
            n += 2 * Hkv * (new + past) * (row_bytes(case) + 2 * d)
        return {"bytes": n, "flops": 2 * Hkv * new * d * 8}
    lens = lengths(case)
    rows = case["B"] * case["Nq"] * case["H"]
    return {"bytes": 2 * Hkv * sum(lens) * row_bytes(case) + rows * (4 * d + 4),
            "flops": 4 * case["Nq"] * case["H"] * d * sum(lens)}


# ---------------------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return exact_norm_rope(s, case)
    return exact_append(s, case) if case["op"] == "append" else exact_attend(s, case)


def rotation(pos, s, d, interleaved):
    """Per token: complex rotation factors and the dims of each pair's two members."""
    h = s["cos"].shape[1]
    i = torch.arange(h, device="cuda")
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    return torch.complex(s["cos"][pos].double(), s["sin"][pos].double()), first, second


def turned(x, rot):
    z, first, second = rot
    y = x.clone()
    t = torch.complex(x[..., first], x[..., second]) * z
    y[..., first], y[..., second] = t.real, t.imag
    return y


def exact_norm_rope(s, case):
    z, first, second = rotation(s["positions"].long(), s, case["d"], case["interleaved"])
    z = z[:, :, None]

    def forward(x, w):
        x = x.double()
        return turned(x / torch.sqrt(x.square().sum(-1, keepdim=True) / case["d"] + 1e-6) * w.double(), (z, first, second))

    if not case["backward"]:
        return forward(s["q"], s["wq"]), forward(s["k"], s["wk"])

    def backward(x, dy, w):
        # y = T (w x / a), a = sqrt(mean x^2 + eps): dx = w u / a - x (sum u w x) / (d a^3), with u = T^-1 dy
        x, u = x.double(), turned(dy.double(), (z.conj(), first, second))
        a2 = x.square().sum(-1, keepdim=True) / case["d"] + 1e-6
        uw = u * w.double()
        dx = uw / a2.sqrt() - x * (uw * x).sum(-1, keepdim=True) / (case["d"] * a2 ** 1.5)
        return dx, (u * x / a2.sqrt()).sum((0, 1, 2))

    (dq, dwq), (dk, dwk) = backward(s["q"], s["dq_out"], s["wq"]), backward(s["k"], s["dk_out"], s["wk"])
    return dq, dk, dwq, dwk


def as_bf16(x, up):
    """x (64 bits) to the nearest bf16 that is not below (up) or not above it."""
    m, _ = torch.frexp(x)
    power = torch.where(x == 0, torch.ones_like(x), x / m)         # 2 to the exponent
    m = m * 256
    return (torch.ceil(m) if up else torch.floor(m)) / 256 * power


def exact_append(s, case):
    new, past = lengths(case)
    ps, d = case["ps"], case["d"]
    rows = {"k": s["k"].clone(), "v": s["v"].clone()} if case["cache"] == "bf16" else {}
    out = {"k": [], "v": []}
    at = 0
    for b, (n, p) in enumerate(zip(new, past)):
        pos = torch.arange(p, p + n, device="cuda")
        z, first, second = rotation(pos, s, d, case["interleaved"])
        fresh = {"k": turned(s["k_new"][at:at + n].double(), (z[:, None], first, second)), "v": s["v_new"][at:at + n].double()}
        at += n
        for x in "kv":
            if case["cache"] == "bf16":
                rows[x] = rows[x].double()
                rows[x][s["table"][b, pos // ps].long(), pos % ps] = fresh[x]
                continue
            old = torch.arange(p, device="cuda")
            page = s["table"][b, old // ps].long()
            code, sz = s[x][page, old % ps], s[x + "_sz"][page, old % ps].double()
            value = torch.empty(p, case["Hkv"], d, dtype=torch.float64, device="cuda")
            value[..., 0::2], value[..., 1::2] = (code & 15).double(), (code >> 4).double()
            value = sz[..., 1].repeat_interleave(GROUP, -1) + value * sz[..., 0].repeat_interleave(GROUP, -1)
            f = fresh[x].view(n, case["Hkv"], -1, GROUP)
            lo, hi = f.min(-1, keepdim=True)[0], f.max(-1, keepdim=True)[0]
            zero = as_bf16(lo, False)
            scale = as_bf16(torch.stack(((hi - zero) / torch.full_like(hi, 15), lo.abs() / 2 ** 20, hi.abs() / 2 ** 20)).amax(0).clamp(min=2.0 ** -100), True)
            f = zero + scale * torch.round((f - zero) / scale).clamp(0, 15)
            out[x].append(torch.cat((value, f.flatten(2))))
    if case["cache"] == "bf16":
        return rows["k"], rows["v"]
    return torch.cat(out["k"]), torch.cat(out["v"])


def exact_attend(s, case):
    Nq, H, Hkv, d = (case[x] for x in ("Nq", "H", "Hkv", "d"))
    o = torch.zeros(case["B"], Nq, H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((case["B"], H, Nq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lengths(case)):
        if n == 0:
            continue
        pos = torch.arange(n, device="cuda")
        page = s["table"][b, pos // case["ps"]].long()
        kv = []
        for x in "kv":
            rows = s[x][page, pos % case["ps"]]
            if case["cache"] == "int4":
                sz = s[x + "_sz"][page, pos % case["ps"]].double().repeat_interleave(GROUP, -2)
                rows = torch.stack((rows % 16, rows // 16), -1).reshape(n, Hkv, d).double() * sz[..., 0] + sz[..., 1]
            kv.append(rows.double())
        for i in range(Nq):
            n_i = n - Nq + i + 1
            if n_i <= 0:
                continue
            for j in range(Hkv):
                heads = slice(j * (H // Hkv), (j + 1) * (H // Hkv))
                S = s["q"][b, i, heads].double() @ kv[0][:n_i, j].T / d ** 0.5
                lse[b, heads, i] = torch.logsumexp(S, -1)
                o[b, i, heads] = torch.softmax(S, -1) @ kv[1][:n_i, j]
    return o, lse

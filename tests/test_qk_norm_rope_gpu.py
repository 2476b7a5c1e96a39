"""attn_qk_norm_rope and its gradient against the fp64 oracle.

Tolerances, from the arithmetic: everything is fp32 between bf16 loads and one rounding to bf16.
  forward: the rounding is off by at most 2^-8 |y|. Before it, a value passes some 12 roundings (square sum of d
    values in a tree of depth <= 13, square root, two or three products, a sum): 32 * 2^-24 of the greatest
    |u| of the row (a pair's members add).
  dx: the same rounding, and 64 * 2^-24 of r max|g| + r max|n| mean|g n| (the row sum has two products more).
  dw: a thread adds at most 4 * 4 terms in the cases here, a CTA 32 of those, 32 lanes up to 19 of these and
    32 of the sums: below 128 roundings of 2^-24 of sum |du n|, the terms' own included.
"""
import numpy as np
import pytest
import torch

import oracle
from exact_attention_72_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_device):
    from exact_attention_72_gb300 import build
    build.build()


def f64(t):
    return t.detach().float().cpu().double().numpy()


def tables(n, half):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(half) / half)
    return torch.tensor(np.cos(a), dtype=torch.float32).cuda(), torch.tensor(np.sin(a), dtype=torch.float32).cuda()


def make(T, H, Hkv, d, seed, fused=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H + 2 * Hkv, d), generator=g).bfloat16().cuda()
    q, k = x[:, :H], x[:, H:H + Hkv] if Hkv else None
    if not fused:
        q, k = q.contiguous(), k.contiguous() if Hkv else None
    w = [(1 + 0.3 * torch.randn(d, generator=g)).cuda() for _ in range(2)]
    dy = [0.1 * torch.randn((T, h, d), generator=g) for h in (H, Hkv)]
    return q, k, w, [y.bfloat16().cuda() for y in dy], torch.randint(0, 50, (T,), generator=g, dtype=torch.int32).cuda()


def ok():
    st, detail = binding.attn_get_status()
    assert st == binding.ATTN_OK, hex(detail)


CASES = [
    # T, H, Hkv, d, rope_dim, norm, weights, interleaved, fused
    (1, 1, 1, 128, 128, True, True, False, True),
    (1, 32, 8, 128, 128, True, True, False, True),
    (7, 5, 5, 64, 64, True, True, False, True),         # heads not a multiple of a task's 4
    (33, 6, 2, 64, 32, True, True, True, True),         # part of the head, interleaved
    (19, 3, 1, 64, 16, True, False, False, True),       # no weights
    (50, 7, 0, 128, 128, True, True, True, False),      # queries alone
    (9, 4, 4, 256, 256, True, True, False, True),
    (11, 9, 3, 256, 128, True, True, True, True),
    (21, 8, 2, 256, 48, True, True, False, False),
    (40, 8, 2, 128, 96, False, False, False, True),     # rotation alone
    (40, 8, 2, 128, 0, True, True, False, True),        # norm alone
    (300, 12, 4, 128, 64, True, True, False, True),
]


def kwargs(case, w, pos):
    T, H, Hkv, d, rd, norm, weights, il, _ = case
    cos, sin = tables(50, rd // 2) if rd else (None, None)
    return dict(cos=cos, sin=sin, positions=pos if rd else None, wq=w[0] if weights else None,
                wk=w[1] if weights and Hkv else None, eps=1e-5, norm=norm, interleaved=il)


def oracle_kw(kw, w):
    c = {n: None if kw[n] is None else f64(kw[n]) for n in ("cos", "sin")}
    return dict(w=None if w is None else f64(w), eps=kw["eps"], norm=kw["norm"], interleaved=kw["interleaved"], **c)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case):
    T, H, Hkv, d, rd, norm, *_ = case
    q, k, w, _, pos = make(T, H, Hkv, d, 1, case[-1])
    kw = kwargs(case, w, pos)
    q_out, k_out = binding.attn_qk_norm_rope(q, k, **kw)
    ok()
    for x, y, wx in ((q, q_out, kw["wq"]), (k, k_out, kw["wk"])):
        if x is None:
            assert y is None
            continue
        ref = oracle.norm_rope(f64(x), f64(pos).astype(int), **oracle_kw(kw, wx))
        top = np.abs(ref).max(-1, keepdims=True) * 2 ** 0.5
        assert np.all(np.abs(f64(y) - ref) <= 2.0 ** -8 * np.abs(ref) + 32 * 2.0 ** -24 * top)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    T, H, Hkv, d, rd, norm, *_ = case
    q, k, w, dy, pos = make(T, H, Hkv, d, 2, case[-1])
    kw = kwargs(case, w, pos)
    dq, dk, dwq, dwk = binding.attn_qk_norm_rope_bwd(q, k, dy[0], dy[1] if Hkv else None, **kw)
    ok()
    for x, g, dx, dw, wx in ((q, dy[0], dq, dwq, kw["wq"]), (k, dy[1], dk, dwk, kw["wk"])):
        if x is None:
            assert dx is None and dw is None
            continue
        okw = oracle_kw(kw, wx)
        p = f64(pos).astype(int)
        ref, ref_w = oracle.norm_rope_backward(f64(x), f64(g), p, **okw)
        okw.pop("w"), okw.pop("norm"), okw.pop("eps")
        if okw["sin"] is not None:
            okw["sin"] = -okw["sin"]
        du = oracle.norm_rope(f64(g), p, norm=False, **okw)
        if norm:
            r = 1 / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True) + kw["eps"])
            n, gw = f64(x) * r, du * (1 if wx is None else f64(wx))
            size = r * (np.abs(gw).max(-1, keepdims=True) * 2 + np.abs(n).max(-1, keepdims=True) * np.abs(gw * n).mean(-1, keepdims=True))
        else:
            size = np.abs(du).max(-1, keepdims=True) * 2
        assert np.all(np.abs(f64(dx) - ref) <= 2.0 ** -8 * np.abs(ref) + 64 * 2.0 ** -24 * size)
        assert (dw is None) == (wx is None)
        if wx is not None:
            assert np.all(np.abs(f64(dw) - ref_w) <= 128 * 2.0 ** -24 * np.abs(du * n).sum((0, 1)) + 1e-30)


def test_batched_shape_and_default_positions():
    q, k, w, dy, _ = make(2 * 13, 8, 2, 128, 3)
    cos, sin = tables(13, 64)
    pos = torch.arange(13, dtype=torch.int32).repeat(2).cuda()
    a = binding.attn_qk_norm_rope(q, k, cos, sin, pos, *w)
    q4, k4 = q.unflatten(0, (2, 13)), k.unflatten(0, (2, 13))
    b = binding.attn_qk_norm_rope(q4, k4, cos, sin, None, *w)
    assert b[0].shape == (2, 13, 8, 128) and torch.equal(a[0], b[0].flatten(0, 1)) and torch.equal(a[1], b[1].flatten(0, 1))
    one = binding.attn_qk_norm_rope(q.unflatten(0, (26, 1)), k.unflatten(0, (26, 1)), cos, sin, pos[:, None].contiguous(), *w)
    assert torch.equal(a[0], one[0].flatten(0, 1))
    ga = binding.attn_qk_norm_rope_bwd(q, k, dy[0], dy[1], cos, sin, pos, *w)
    gb = binding.attn_qk_norm_rope_bwd(q4, k4, dy[0].unflatten(0, (2, 13)), dy[1].unflatten(0, (2, 13)), cos, sin, None, *w)
    for x, y in zip(ga, gb):
        assert torch.equal(x.flatten(), y.flatten())


@pytest.mark.parametrize("il", [False, True])
def test_in_place_gives_the_same_bits(il):
    q, k, w, dy, pos = make(37, 6, 2, 128, 4, fused=False)
    cos, sin = tables(50, 32)
    kw = dict(cos=cos, sin=sin, positions=pos, wq=w[0], wk=w[1], interleaved=il)
    want = binding.attn_qk_norm_rope(q, k, **kw)
    grads = binding.attn_qk_norm_rope_bwd(q, k, dy[0], dy[1], **kw)
    got = binding.attn_qk_norm_rope_bwd(q, k, dy[0], dy[1], dq=dy[0], dk=dy[1], **kw)
    for x, y in zip(grads, got):
        assert torch.equal(x, y)
    assert got[0] is dy[0]
    binding.attn_qk_norm_rope(q, k, q_out=q, k_out=k, **kw)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_positions_outside_the_tables_are_left_out():
    q, k, w, dy, pos = make(20, 8, 2, 128, 5)
    cos, sin = tables(50, 64)
    bad = pos.clone()
    bad[3], bad[11] = 50, -1
    out = [torch.full((20, h, 128), 7.0, dtype=torch.bfloat16, device="cuda") for h in (8, 2)]
    want = binding.attn_qk_norm_rope(q, k, cos, sin, pos, *w)
    ok()
    try:
        binding.attn_qk_norm_rope(q, k, cos, sin, bad, *w, q_out=out[0], k_out=out[1])
        assert binding.attn_get_status() == (binding.ATTN_ERR_INVALID_ARG, 0x2000000E)
        binding.attn_clear_status()
        got = binding.attn_qk_norm_rope_bwd(q, k, dy[0], dy[1], cos, sin, bad, *w)
        assert binding.attn_get_status()[0] == binding.ATTN_ERR_INVALID_ARG
    finally:
        binding.attn_clear_status()
    keep = [t for t in range(20) if t not in (3, 11)]
    for y, x in zip(out, want):
        assert torch.equal(y[keep], x[keep]) and bool((y[[3, 11]] == 7).all())
    ref = oracle.norm_rope_backward(f64(q)[keep], f64(dy[0])[keep], f64(pos).astype(int)[keep], w=f64(w[0]), eps=1e-6, cos=f64(cos),
                                    sin=f64(sin))[1]
    assert np.abs(f64(got[2]) - ref).max() <= 2.0 ** -16 * 20 * 8      # |du n| is of the order 0.1 to 1


def test_zero_rows_infinities_and_empty_calls():
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    q[1, 2, 5], q[2, 0, 0] = float("inf"), float("nan")
    y, _ = binding.attn_qk_norm_rope(q)
    assert bool((y[0] == 0).all()) and bool((y[1, :2] == 0).all())     # a bad row stays in its row
    assert bool(torch.isnan(y[2, 0]).all()) and bool((y[2, 1:] == 0).all())
    dx, _, _, _ = binding.attn_qk_norm_rope_bwd(q, None, torch.ones_like(q), eps=1e-6)
    assert torch.allclose(dx[0].float(), torch.full((4, 64), 1000.0).cuda(), rtol=2 ** -8)   # 1 / sqrt(eps)
    e = q[:0]
    assert binding.attn_qk_norm_rope(e)[0].shape == (0, 4, 64)
    w = torch.ones(64, device="cuda")
    assert bool((binding.attn_qk_norm_rope_bwd(e, None, e, wq=w)[2] == 0).all())


def test_same_bits_every_time_with_any_workspace():
    q, k, w, dy, pos = make(3000, 12, 4, 128, 6)
    cos, sin = tables(50, 64)
    n = binding.attn_qk_norm_rope_bwd_workspace_bytes(3000, 12, 4, 128)
    first = binding.attn_qk_norm_rope_bwd(q, k, dy[0], dy[1], cos, sin, pos, *w)
    for fill in (0, 255):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        again = binding.attn_qk_norm_rope_bwd(q, k, dy[0], dy[1], cos, sin, pos, *w, workspace=ws)
        assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_other_stream_and_captured():
    q, k, w, dy, pos = make(64, 8, 2, 128, 7)
    cos, sin = tables(50, 64)
    want = binding.attn_qk_norm_rope(q, k, cos, sin, pos, *w)
    grads = binding.attn_qk_norm_rope_bwd(q, k, dy[0], dy[1], cos, sin, pos, *w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = binding.attn_qk_norm_rope(q, k, cos, sin, pos, *w, stream=s)
    b = binding.attn_qk_norm_rope_bwd(q, k, dy[0], dy[1], cos, sin, pos, *w, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((*want, *grads), (*a, *b)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = binding.attn_qk_norm_rope(q, k, cos, sin, pos, *w)
        e = binding.attn_qk_norm_rope_bwd(q, k, dy[0], dy[1], cos, sin, pos, *w)
    q.mul_(0.5)      # the norm takes a factor out, up to eps: replay reads what the tensors hold now
    dy[0].mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(e[0], binding.attn_qk_norm_rope_bwd(q, k, dy[0], dy[1], cos, sin, pos, *w)[0])
    assert torch.equal(c[0], binding.attn_qk_norm_rope(q, k, cos, sin, pos, *w)[0])


def test_training_step_through_the_attention():
    """q, k, v out of one projection: norm and rotation, attn_fwd, attn_bwd, and back through norm and rotation, against the
    same chain in 64 bits. Each stage rounds to bf16 (2^-8 at most, about 2^-9.8 in the mean square) and passes it on: 2e-2
    of a gradient's norm is five such roundings at their most."""
    B, N, H, Hkv, d = 2, 150, 4, 2, 64
    g = torch.Generator().manual_seed(8)
    qkv = torch.randn((B, N, H + 2 * Hkv, d), generator=g).bfloat16()
    do = torch.randn((B, N, H, d), generator=g).bfloat16()
    w = [1 + 0.3 * torch.randn(d, generator=g) for _ in range(2)]
    cos, sin = tables(N, d // 2)
    dev = qkv.cuda()
    q, k, v = dev[:, :, :H], dev[:, :, H:H + Hkv], dev[:, :, H + Hkv:].contiguous()
    kw = dict(cos=cos, sin=sin, wq=w[0].cuda(), wk=w[1].cuda())
    qr, kr = binding.attn_qk_norm_rope(q, k, **kw)
    o, lse = binding.attn_fwd(qr, kr, v, causal=True)
    dqr, dkr, dv = binding.attn_bwd(qr, kr, v, o, lse, do.cuda(), causal=True)
    dq, dk, dwq, dwk = binding.attn_qk_norm_rope_bwd(q, k, dqr, dkr, **kw)
    ok()

    x = qkv.double().requires_grad_()
    ws = [t.double().requires_grad_() for t in w]
    c, s = (t.cpu().double()[None, :, None] for t in (cos, sin))

    def turn(u):
        a, b = u.chunk(2, -1)
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    def nr(u, wt):
        return turn(u * torch.rsqrt(u.square().mean(-1, keepdim=True) + 1e-6) * wt)
    qq, kk, vv = nr(x[:, :, :H], ws[0]), nr(x[:, :, H:H + Hkv], ws[1]), x[:, :, H + Hkv:]
    kk, vv = kk.repeat_interleave(H // Hkv, 2), vv.repeat_interleave(H // Hkv, 2)
    S = torch.einsum("bihd,bjhd->bhij", qq, kk) / d ** 0.5
    S = S.masked_fill(torch.ones(N, N).triu(1).bool(), float("-inf"))
    out = torch.einsum("bhij,bjhd->bihd", S.softmax(-1), vv)
    out.backward(do.double())
    for got, want in ((o, out), (dq, x.grad[:, :, :H]), (dk, x.grad[:, :, H:H + Hkv]), (dv, x.grad[:, :, H + Hkv:]),
                      (dwq, ws[0].grad), (dwk, ws[1].grad)):
        diff = got.cpu().double() - want.detach()
        assert float(diff.norm() / want.detach().norm()) <= 2e-2


def test_batches_without_tokens():
    w = torch.ones(64, device="cuda")
    for shape in ((2, 0, 4, 64), (0, 5, 4, 64), (0, 4, 64)):
        q = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        y, z = binding.attn_qk_norm_rope(q, q[..., :2, :], wq=w, wk=w)
        assert y.shape == q.shape and z.shape == (*shape[:-2], 2, 64)
        dq, _, dwq, dwk = binding.attn_qk_norm_rope_bwd(q, None, q, wq=w)
        assert dq.shape == q.shape and bool((dwq == 0).all()) and dwk is None
    ok()


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan"), -0.0])
@pytest.mark.parametrize("d,rd,il", [(64, 0, False), (64, 32, False), (128, 64, False), (128, 0, False), (128, 32, True),
                                     (256, 16, False), (256, 240, True)])
def test_values_behind_the_rotated_ones_are_unchanged(d, rd, il, value):
    """Without the norm every value behind rope_dim comes out as it is, whatever stands beside it: each of them once infinite,
    NaN or -0 in a row of its own. The same of the gradient."""
    T = d - rd
    q, _, _, _, _ = make(T, 3, 0, d, 11, fused=False)
    cos, sin = tables(T, rd // 2) if rd else (None, None)
    kw = dict(cos=cos, sin=sin, norm=False, interleaved=il)
    want = binding.attn_qk_norm_rope(q, **kw)[0], binding.attn_qk_norm_rope_bwd(q, None, q, **kw)[0]
    x = q.clone()
    rows = torch.arange(T, device="cuda")
    x[rows, 1, rd + rows] = value
    got = binding.attn_qk_norm_rope(x, **kw)[0], binding.attn_qk_norm_rope_bwd(x, None, x, **kw)[0]
    ok()
    for y, w in zip(got, want):
        w[..., rd:] = x[..., rd:]
        same = y.view(torch.int16) == w.view(torch.int16)
        assert bool((same | (y.isnan() & w.isnan())).all())


def plain64(x, pos, w, cos, sin, norm, il, dy=None, eps=1e-5):
    """The forward, or with dy (dx, dw, sum |du n|), in 64 bits on the GPU."""
    x, d, half = x.double(), x.shape[-1], 0 if cos is None else cos.shape[1]
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if il else (slice(0, half), slice(half, 2 * half))

    def turn(u, sign):
        y = u.clone()
        if half:
            c, s = cos.double()[pos.long()][:, None], sign * sin.double()[pos.long()][:, None]
            y[..., first], y[..., second] = u[..., first] * c - u[..., second] * s, u[..., second] * c + u[..., first] * s
        return y
    n, r = x, 1.0
    if norm:
        r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
        n = x * r
    wd = 1.0 if w is None else w.double()
    if dy is None:
        return turn(n * wd, 1.0)
    du = turn(dy.double(), -1.0)
    if not norm:
        return du, None, None
    g = du * wd
    return r * (g - n * (g * n).mean(-1, keepdim=True)), (du * n).sum((0, 1)), (du * n).abs().sum((0, 1))


LONG = [
    # more tasks than threads take in one round, and no multiple of it
    (6001, 12, 4, 128, 128, True, True, False, True),       # T, H, Hkv, d, rope_dim, norm, weights, interleaved, fused
    (3001, 9, 3, 256, 128, True, True, True, True),
    (9003, 8, 2, 64, 32, True, True, False, False),
    (5003, 13, 0, 128, 64, False, False, False, False),
    (4999, 7, 7, 128, 0, True, True, False, True),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", LONG, ids=str)
def test_threads_with_several_tasks(case, in_place):
    """Rows of the next task are loaded while those of one are turned. Bounds as above; a thread adds the terms of at most 6
    tasks, 24, a CTA at most 32 threads, the last kernel 10 sums and 32 of those: still below 128 roundings. Two tokens have
    positions outside the tables, one in the last round: not written, and not in the weights' gradients."""
    T, H, Hkv, d, rd, norm, weights, il, fused = case
    q, k, w, dy, pos = make(T, H, Hkv, d, 21, fused and not in_place)
    kw = kwargs(case, w, pos)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    if rd:
        pos[5], pos[T - 2] = 50, -1
        keep[5] = keep[T - 2] = False
    outs = [x.clone() if in_place and x is not None else None for x in (q, k)]
    args = outs if in_place else [q, k]
    plain = lambda x, wx, g=None: plain64(x[keep], pos[keep], wx, kw["cos"], kw["sin"], norm, il, None if g is None else g[keep])
    try:
        got = binding.attn_qk_norm_rope(*args, **kw, q_out=outs[0], k_out=outs[1])
        g = [x.clone() for x in dy]
        grads = binding.attn_qk_norm_rope_bwd(q, k, g[0], g[1] if Hkv else None, **kw, dq=g[0] if in_place else None,
                                              dk=g[1] if in_place and Hkv else None)
        st = binding.attn_get_status()
        assert st == ((binding.ATTN_ERR_INVALID_ARG, 0x2000000E) if rd else (binding.ATTN_OK, 0))
    finally:
        binding.attn_clear_status()
    for i, (x, wx) in enumerate(((q, kw["wq"]), (k, kw["wk"]))):
        if x is None:
            continue
        ref = plain(x, wx)
        top = ref.abs().amax(-1, keepdim=True) * 2 ** 0.5
        assert bool(((got[i][keep].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 32 * 2.0 ** -24 * top).all())
        dx, dw, size = plain(x, wx, dy[i])
        du = plain64(x[keep], pos[keep], wx, kw["cos"], kw["sin"], False, il, dy[i][keep])[0]
        room = du.abs().amax(-1, keepdim=True) * 2
        if norm:
            r = 1 / (x[keep].double().square().mean(-1, keepdim=True) + 1e-5).sqrt()
            n, gw = x[keep].double() * r, du * (1 if wx is None else wx.double())
            room = r * (gw.abs().amax(-1, keepdim=True) * 2 + n.abs().amax(-1, keepdim=True) * (gw * n).abs().mean(-1, keepdim=True))
        assert bool(((grads[i][keep].double() - dx).abs() <= 2.0 ** -8 * dx.abs() + 64 * 2.0 ** -24 * room).all())
        if wx is not None:
            assert bool(((grads[2 + i].double() - dw).abs() <= 128 * 2.0 ** -24 * size).all())
        if in_place:      # rows without a position are as they were
            assert torch.equal(got[i][~keep], x[~keep]) and torch.equal(grads[i][~keep], dy[i][~keep])


def test_the_plain_form_is_the_oracles():
    q, _, w, dy, pos = make(9, 3, 1, 64, 22)
    cos, sin = tables(50, 16)
    for norm, il in ((True, False), (True, True), (False, True)):
        wx = w[0] if norm else None
        okw = dict(w=None if wx is None else f64(wx), eps=1e-5, norm=norm, cos=f64(cos), sin=f64(sin), interleaved=il)
        p = f64(pos).astype(int)
        y = plain64(q, pos, wx, cos, sin, norm, il)
        dx, dw, _ = plain64(q, pos, wx, cos, sin, norm, il, dy[0])
        ref_dx, ref_dw = oracle.norm_rope_backward(f64(q), f64(dy[0]), p, **okw)
        for a, b in ((y, oracle.norm_rope(f64(q), p, **okw)), (dx, ref_dx), (dw, ref_dw if norm else None)):
            assert b is None or np.abs(a.cpu().numpy() - b).max() <= 1e-12 * (1 + np.abs(b).max())

"""attn_qk_norm_rope_axes and its gradient: positions on several axes.

Gathered for every token, cos[pos[axis(i)], i] is a table of one row a token, and the calls with one axis at positions 0, 1, ..
are the same arithmetic: the results have to have the same bits. Against the fp64 oracle with those tables the bounds are those of
test_qk_norm_rope_gpu.py (forward 2^-8 of the value and 32 * 2^-24 of the row's greatest pair; dx 2^-8 and 64 * 2^-24 of its
terms; dw 128 * 2^-24 of its terms' sum).
"""
import numpy as np
import pytest
import torch

import oracle
from exact_attention_72_gb300 import binding
from test_qk_norm_rope_gpu import f64, make, ok, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_device):
    from exact_attention_72_gb300 import build
    build.build()


CASES = [
    # T, H, Hkv, d, sections, turns, norm, weights, interleaved pairs
    (1, 1, 1, 128, (16, 24, 24), False, True, True, False),
    (1, 32, 8, 128, (24, 20, 20), True, True, True, False),
    (37, 5, 5, 64, (8, 12, 12), False, True, True, False),
    (33, 6, 2, 64, (8, 8), False, True, True, True),              # half of the head, two axes
    (19, 3, 1, 64, (3, 5), True, True, False, False),             # no weights, blocks that no lane's 4 pairs agree with
    (50, 7, 0, 128, (1, 2, 61), False, True, True, True),         # queries alone
    (9, 4, 4, 256, (32, 48, 48), True, True, True, False),
    (11, 9, 3, 256, (30, 0, 33, 1), False, True, True, True),     # four axes, one of them without pairs
    (21, 8, 2, 256, (24,), False, True, True, False),             # one axis
    (40, 8, 2, 128, (20, 14, 14), True, False, False, False),     # rotation alone
    (300, 12, 4, 128, (16, 16), True, True, True, False),
    (2000, 8, 2, 64, (16, 8, 8), True, True, True, True),         # a thread has several tasks
]


def setup(case, seed):
    T, H, Hkv, d, sections, turns, norm, weights, il = case
    q, k, w, dy, _ = make(T, H, Hkv, d, seed)
    axis = binding.rope_pair_axes(sections, turns)
    cos, sin = tables(50, len(axis))
    g = torch.Generator().manual_seed(seed)
    pos = torch.randint(0, 50, (len(sections), T), generator=g, dtype=torch.int32)
    pos[:, ::3] = pos[0, ::3]                                     # text among them: the same on each axis
    pos = pos.cuda()
    i = torch.arange(len(axis)).cuda()
    row = pos.long()[torch.tensor(list(axis)).cuda()].T           # [T, pairs]
    kw = dict(wq=w[0] if weights else None, wk=w[1] if weights and Hkv else None, eps=1e-5, norm=norm, interleaved=il)
    return q, k, dy, dict(cos=cos, sin=sin, positions=pos, pair_axis=axis, **kw), \
        dict(cos=cos[row, i], sin=sin[row, i], positions=torch.arange(T, dtype=torch.int32).cuda(), **kw)


def same(a, b):
    assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case):
    q, k, _, kw, gathered = setup(case, 1)
    y = binding.attn_qk_norm_rope_axes(q, k, **kw)
    for a, b in zip(y, binding.attn_qk_norm_rope(q, k, **gathered)):
        same(a, b)
    ok()
    for x, got, w in ((q, y[0], kw["wq"]), (k, y[1], kw["wk"])):
        if x is None:
            continue
        ref = oracle.norm_rope(f64(x[:64]), np.arange(len(x[:64])), w=None if w is None else f64(w), eps=kw["eps"], norm=kw["norm"],
                               cos=f64(gathered["cos"]), sin=f64(gathered["sin"]), interleaved=kw["interleaved"])
        top = np.abs(ref).max(-1, keepdims=True) * 2 ** 0.5
        assert np.all(np.abs(f64(got[:64]) - ref) <= 2.0 ** -8 * np.abs(ref) + 32 * 2.0 ** -24 * top)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    q, k, dy, kw, gathered = setup(case, 2)
    dk_out = dy[1] if k is not None else None
    got = binding.attn_qk_norm_rope_axes_bwd(q, k, dy[0], dk_out, **kw)
    for a, b in zip(got, binding.attn_qk_norm_rope_bwd(q, k, dy[0], dk_out, **gathered)):
        same(a, b)
    ok()
    T, heads = min(len(q), 64), q.shape[1]
    if len(q) > 64:       # dw is over all tokens: the comparison above has it
        return
    okw = dict(cos=f64(gathered["cos"]), sin=f64(gathered["sin"]), interleaved=kw["interleaved"])
    for x, g, dx, dw, w in ((q, dy[0], got[0], got[2], kw["wq"]), (k, dy[1], got[1], got[3], kw["wk"])):
        if x is None:
            continue
        ww = None if w is None else f64(w)
        ref, ref_w = oracle.norm_rope_backward(f64(x), f64(g), np.arange(T), w=ww, eps=kw["eps"], norm=kw["norm"], **okw)
        du = oracle.norm_rope(f64(g), np.arange(T), norm=False, cos=okw["cos"], sin=-okw["sin"], interleaved=okw["interleaved"])
        size = np.abs(du).max(-1, keepdims=True) * 2
        if kw["norm"]:
            r = 1 / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True) + kw["eps"])
            n, gw = f64(x) * r, du * (1 if ww is None else ww)
            size = r * (np.abs(gw).max(-1, keepdims=True) * 2 + np.abs(n).max(-1, keepdims=True) * np.abs(gw * n).mean(-1, keepdims=True))
            if w is not None:
                assert np.all(np.abs(f64(dw) - ref_w) <= 128 * 2.0 ** -24 * np.abs(du * n).sum((0, 1)))
        assert np.all(np.abs(f64(dx) - ref) <= 2.0 ** -8 * np.abs(ref) + 64 * 2.0 ** -24 * size)


@pytest.mark.parametrize("case", [c for c in CASES if c[0] <= 50 and c[2]], ids=str)
def test_gradient_against_differences(case):
    """Along a random direction v: sum dx v is the derivative of sum dy y. The difference of the fp64 forward, step 1e-4, is off by
    some 1e-8 of the terms; dx by 2^-8 of each value."""
    q, k, dy, kw, gathered = setup(case, 3)
    dx = f64(binding.attn_qk_norm_rope_axes_bwd(q, k, dy[0], dy[1], **kw)[0])
    ok()
    v = np.random.default_rng(4).standard_normal(dx.shape)
    T = len(q)

    def f(x):
        y = oracle.norm_rope(x, np.arange(T), w=None if kw["wq"] is None else f64(kw["wq"]), eps=kw["eps"], norm=kw["norm"],
                             cos=f64(gathered["cos"]), sin=f64(gathered["sin"]), interleaved=kw["interleaved"])
        return (f64(dy[0]) * y).sum((1, 2))

    x, h = f64(q), 1e-4
    slope = (f(x + h * v) - f(x - h * v)) / (2 * h)
    size = np.abs(dx * v).sum((1, 2))
    assert np.all(np.abs((dx * v).sum((1, 2)) - slope) <= (2.0 ** -8 + 1e-5) * size + 1e-6)


def test_batches_in_place_and_parts_of_a_projection():
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn((3, 7, 12, 128), generator=g).bfloat16().cuda()
    axis = binding.rope_pair_axes((16, 24, 24))
    cos, sin = tables(60, 64)
    pos = torch.randint(0, 60, (3, 3, 7), generator=g, dtype=torch.int32).cuda()
    q, k = qkv[:, :, :8], qkv[:, :, 8:10]
    a, b = binding.attn_qk_norm_rope_axes(q, k, cos, sin, pos, axis)
    qc, kc = q.contiguous(), k.contiguous()
    assert torch.equal(binding.attn_qk_norm_rope_axes(qc.view(21, 8, 128), kc.view(21, 2, 128), cos, sin, pos.view(3, 21), list(axis))[0].view_as(a), a)
    out = binding.attn_qk_norm_rope_axes(qc, kc, cos, sin, pos, axis, q_out=qc, k_out=kc)
    ok()
    assert out[0] is qc and torch.equal(qc, a) and torch.equal(kc, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c, _ = binding.attn_qk_norm_rope_axes(q, k, cos, sin, pos, axis, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(c, a)


@pytest.mark.parametrize("axis", [0, 1, 2])
@pytest.mark.parametrize("bad", [-1, 50])
def test_bad_positions(axis, bad):
    """A token with one bad position is not written and adds nothing to dw; on an axis without pairs it is not looked at."""
    q, k, dy, kw, _ = setup((20, 4, 2, 128, (40, 24, 0), False, True, True, False), 5)
    good = binding.attn_qk_norm_rope_axes(q, k, **kw)
    pos = kw["positions"].clone()
    pos[axis, 7] = bad
    y = [torch.full_like(x, 7.0) for x in good]
    binding.attn_qk_norm_rope_axes(q, k, **{**kw, "positions": pos}, q_out=y[0], k_out=y[1])
    st, detail = binding.attn_get_status()
    binding.attn_clear_status()
    if axis == 2:
        assert st == binding.ATTN_OK and all(torch.equal(a, b) for a, b in zip(y, good))
        return
    assert st == binding.ATTN_ERR_INVALID_ARG and detail == 0x2000000E
    for a, b in zip(y, good):
        assert (a[7] == 7).all()
        a[7] = b[7]
        assert torch.equal(a, b)
    grads = binding.attn_qk_norm_rope_axes_bwd(q, k, dy[0], dy[1], **{**kw, "positions": pos})
    binding.attn_get_status()
    binding.attn_clear_status()
    dy[0][7], dy[1][7] = 0, 0
    want = binding.attn_qk_norm_rope_axes_bwd(q, k, dy[0], dy[1], **kw)
    ok()
    assert torch.equal(grads[2], want[2]) and torch.equal(grads[3], want[3])


def test_captured_and_replayed_with_other_positions():
    q, k, dy, kw, _ = setup((24, 4, 2, 128, (16, 24, 24), True, True, True, False), 6)
    n = binding.attn_qk_norm_rope_bwd_workspace_bytes(24, 4, 2, 128)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    binding.attn_qk_norm_rope_axes_bwd(q, k, dy[0], dy[1], **kw, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = binding.attn_qk_norm_rope_axes(q, k, **kw)
        g = binding.attn_qk_norm_rope_axes_bwd(q, k, dy[0], dy[1], **kw, workspace=ws)
    for seed in range(2):
        kw["positions"].copy_(torch.randint(0, 50, kw["positions"].shape, generator=torch.Generator().manual_seed(seed), dtype=torch.int32))
        graph.replay()
        for a, b in zip((*y, *g), (*binding.attn_qk_norm_rope_axes(q, k, **kw),
                                   *binding.attn_qk_norm_rope_axes_bwd(q, k, dy[0], dy[1], **kw))):
            assert torch.equal(a, b)
    ok()


def test_refusals():
    q, k, dy, kw, _ = setup((6, 4, 2, 128, (16, 24, 24), False, True, True, False), 5)
    pos = kw["positions"]
    for bad in (dict(positions=None), dict(positions=pos[0]), dict(positions=pos[:, :5]), dict(positions=pos.long()),
                dict(positions=pos.T.contiguous().T), dict(positions=torch.cat((pos, pos))), dict(positions=pos[:0]),
                dict(positions=pos.cpu()), dict(pair_axis=kw["pair_axis"][:-1]), dict(pair_axis=b""), dict(cos=None, sin=None),
                dict(pair_axis=[300] * 64)):
        with pytest.raises(ValueError):
            binding.attn_qk_norm_rope_axes(q, k, **{**kw, **bad})
        with pytest.raises(ValueError):
            binding.attn_qk_norm_rope_axes_bwd(q, k, dy[0], dy[1], **{**kw, **bad})
    for bad in (dict(pair_axis=bytes([0] * 63 + [3])), dict(eps=-1.0)):
        with pytest.raises(binding.AttnError):
            binding.attn_qk_norm_rope_axes(q, k, **{**kw, **bad})
        with pytest.raises(binding.AttnError):
            binding.attn_qk_norm_rope_axes_bwd(q, k, dy[0], dy[1], **{**kw, **bad})
    empty = binding.attn_qk_norm_rope_axes(q[:0], k[:0], **{**kw, "positions": pos[:, :0].contiguous()})
    assert empty[0].shape == (0, 4, 128)
    ok()

"""Refusals of the norm-and-rotation and paged-cache entry points that need no GPU: every bad argument is turned
away before any CUDA call. Addresses are made up and never read."""
import ctypes

import pytest
import torch

from exact_attention_72_gb300 import binding, build

INV, UNS, OK = binding.ATTN_ERR_INVALID_ARG, binding.ATTN_ERR_UNSUPPORTED, binding.ATTN_OK
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def norm_rope(lib, q=16 * MB, k=32 * MB, qo=48 * MB, ko=64 * MB, T=10, H=8, Hkv=2, d=128, st=(1024, 128, 256, 128), norm=1,
              wq=MB, wk=2 * MB, eps=1e-6, cos=4 * MB, sin=5 * MB, rd=128, max_pos=100, il=0, pos=None, seq=10):
    return lib.attn_qk_norm_rope(q, k, qo, ko, T, H, Hkv, d, *st, norm, wq, wk, eps, cos, sin, rd, max_pos, il, pos, seq,
                                 None)


@pytest.mark.parametrize("bad", [
    dict(q=0), dict(k=0), dict(qo=0), dict(ko=0), dict(T=0), dict(H=0), dict(Hkv=-1), dict(q=16 * MB + 8),
    dict(Hkv=0),                                  # k given without heads
    dict(k=0, ko=0),                              # heads without k
    dict(st=(1020, 128, 256, 128)), dict(st=(-1024, 128, 256, 128)), dict(st=(1 << 41, 128, 256, 128)),
    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(norm=0),   # weights without a norm
    dict(wq=MB + 2), dict(cos=0), dict(sin=0), dict(cos=4 * MB + 4), dict(max_pos=0), dict(seq=0), dict(pos=7),
    dict(rd=0), dict(rd=8), dict(rd=24), dict(rd=144),
    dict(qo=16 * MB + 2048), dict(qo=32 * MB), dict(ko=48 * MB), dict(ko=16 * MB),
    dict(qo=16 * MB, st=(2048, 128, 256, 128)),   # in place, but not contiguous
])
def test_norm_rope_refuses(lib, bad):
    assert norm_rope(lib, **bad) == INV


@pytest.mark.parametrize("bad", [dict(d=96), dict(d=32, rd=32), dict(T=1 << 30)])
def test_norm_rope_unsupported(lib, bad):
    assert norm_rope(lib, **bad) == UNS


def bwd(lib, q=16 * MB, k=32 * MB, gq=80 * MB, gk=96 * MB, dq=48 * MB, dk=64 * MB, dwq=3 * MB, dwk=3 * MB + 4096, T=10, H=8,
        Hkv=2, d=128, norm=1, wq=MB, wk=2 * MB, ws=128 * MB, nbytes=MB):
    return lib.attn_qk_norm_rope_bwd(q, k, gq, gk, dq, dk, dwq, dwk, T, H, Hkv, d, 1024, 128, 256, 128, norm, wq, wk, 1e-6,
                                     4 * MB, 5 * MB, 128, 100, 0, None, 10, ws, nbytes, None)


@pytest.mark.parametrize("bad", [
    dict(q=0), dict(k=0), dict(gq=0), dict(gk=0), dict(dq=0), dict(dk=0), dict(dwq=0), dict(dwk=0), dict(wq=0), dict(wk=0),
    dict(gq=80 * MB + 8), dict(dwq=3 * MB + 2), dict(ws=0), dict(ws=128 * MB + 8), dict(nbytes=16),
    dict(dq=16 * MB), dict(dq=80 * MB + 2048), dict(dq=96 * MB), dict(dk=80 * MB), dict(dk=48 * MB), dict(ws=48 * MB),
    dict(dwq=48 * MB), dict(dwk=3 * MB), dict(T=0),
])
def test_norm_rope_bwd_refuses(lib, bad):
    assert bwd(lib, **bad) == INV


def test_norm_rope_bwd_workspace(lib):
    n = binding.attn_qk_norm_rope_bwd_workspace_bytes
    assert n(1, 4, 4, 128) == 2 * 128 * 4            # a CTA each for q and k
    assert n(1, 4, 0, 128) == 128 * 4
    assert n(1 << 20, 32, 8, 128) == n(1 << 21, 32, 8, 128) > 0     # one wave, whatever the length
    assert n(0, 4, 4, 128) == n(1, 0, 4, 128) == n(1, 4, 4, 96) == 0
    assert bwd(lib, d=96) == UNS


def cache(type=0, k=256 * MB, v=512 * MB, k_sz=768 * MB, v_sz=800 * MB, strides=(8192, 512, 128), sz=(256, 16, 4), pages=10,
          ps=16, Hkv=4, d=128):
    return binding._PagedCacheStruct(k, v, k_sz, v_sz, *strides, *sz, pages, ps, Hkv, d, type)


def append(lib, c, k=16 * MB, v=32 * MB, st=(512, 128, 512, 128), cu=MB, lens=2 * MB, table=3 * MB, ts=8, mp=8, B=2, total=10,
           cos=4 * MB, sin=5 * MB, rd=128, max_pos=100):
    return lib.attn_paged_append(ctypes.byref(c), k, v, *st, cu, lens, table, ts, mp, B, total, cos, sin, rd, max_pos, 0, None)


def gather(lib, c, k=16 * MB, v=32 * MB, cu=MB, table=3 * MB, ts=8, mp=8, B=2, total=10):
    return lib.attn_paged_gather(ctypes.byref(c), k, v, cu, table, ts, mp, B, total, None)


def attend(lib, c, q=16 * MB, o=32 * MB, lse=48 * MB, table=3 * MB, ts=8, mp=8, lens=2 * MB, B=2, H=8, Nq=1, scale=0.1,
           ws=1024 * MB, nbytes=64 * MB):
    return lib.attn_fwd_paged(q, ctypes.byref(c), o, lse, table, ts, mp, lens, B, H, Nq, scale, 1, ws, nbytes, None)


BAD_CACHES = [
    (dict(k=0), INV), (dict(v=0), INV), (dict(k=256 * MB + 8), INV), (dict(pages=0), INV), (dict(ps=0), INV),
    (dict(Hkv=0), INV), (dict(type=2), INV), (dict(strides=(8192, 516, 128)), INV), (dict(strides=(-8192, 512, 128)), INV),
    (dict(d=96), UNS), (dict(ps=24), UNS), (dict(ps=8), UNS),
    (dict(type=1, k_sz=0), INV), (dict(type=1, v_sz=0), INV), (dict(type=1, k_sz=768 * MB + 4), INV),
    (dict(type=1, sz=(256, 16, 2)), INV), (dict(type=1, sz=(256, -16, 4)), INV), (dict(type=1, strides=(8192, 512, 72)), INV),
]


@pytest.mark.parametrize("bad,want", BAD_CACHES)
def test_every_entry_refuses_a_bad_cache(lib, bad, want):
    c = cache(**bad)
    assert append(lib, c) == want and gather(lib, c) == want and attend(lib, c) == want


@pytest.mark.parametrize("bad", [
    dict(k=0), dict(v=0), dict(cu=0), dict(lens=0), dict(table=0), dict(k=16 * MB + 8), dict(st=(516, 128, 512, 128)),
    dict(st=(512, 128, -512, 128)), dict(B=0), dict(total=-1), dict(mp=0), dict(ts=-1), dict(cos=0), dict(sin=0), dict(rd=8),
    dict(rd=256), dict(max_pos=0), dict(cu=MB + 2),
])
def test_append_refuses(lib, bad):
    assert append(lib, cache(), **bad) == INV


@pytest.mark.parametrize("bad", [dict(k=0), dict(v=0), dict(cu=0), dict(table=0), dict(v=16 * MB + 1024), dict(v=32 * MB + 8),
                                 dict(B=0), dict(total=-1), dict(mp=0)])
def test_gather_refuses(lib, bad):
    assert gather(lib, cache(), **bad) == INV


def test_nothing_to_do(lib):
    assert append(lib, cache(), total=0) == OK and gather(lib, cache(), total=0) == OK
    assert append(lib, cache(Hkv=64), total=1 << 27) == UNS


@pytest.mark.parametrize("bad", [
    dict(q=0), dict(o=0), dict(lse=0), dict(table=0), dict(lens=0), dict(ws=0), dict(q=16 * MB + 8), dict(o=32 * MB + 8),
    dict(lse=48 * MB + 2), dict(ws=1024 * MB + 128), dict(B=0), dict(H=0), dict(H=6), dict(Nq=0), dict(mp=0), dict(ts=-1),
    dict(scale=float("nan")), dict(scale=float("inf")),
])
def test_attend_refuses(lib, bad):
    assert attend(lib, cache(), **bad) == INV


def test_attend_unsupported(lib):
    assert attend(lib, cache(), scale=0.0) == UNS
    assert attend(lib, cache(), B=1 << 28, H=32) == UNS


def test_attend_workspace_size(lib):
    n = lib.attn_fwd_paged_workspace_bytes
    for t in (0, 1):
        for d in (64, 128, 256):
            one = n(1, 8, 8, 1, d, t)
            assert one > 0 and n(1000, 8, 8, 1, d, t) == one     # neither the batch nor the lengths count
            assert n(1, 64, 8, 1, d, t) == one                  # 8 rows
            assert n(1, 72, 8, 1, d, t) > 0
    assert n(0, 8, 8, 1, 128, 0) == n(1, 8, 3, 1, 128, 0) == n(1, 8, 8, 0, 128, 0) == 0
    assert n(1, 8, 8, 1, 96, 0) == n(1, 8, 8, 1, 128, 7) == 0


def test_binding_refuses_before_the_library():
    """Shapes and types that the wrappers turn away: host tensors never reach a launch."""
    q = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.attn_qk_norm_rope(q.float())
    with pytest.raises(ValueError):
        binding.attn_qk_norm_rope(q.transpose(1, 2))
    with pytest.raises(ValueError):
        binding.attn_qk_norm_rope(q, q[:2])
    with pytest.raises(ValueError):
        binding.attn_qk_norm_rope(torch.zeros(2, 4, 8, 128, dtype=torch.bfloat16)[:, ::2][:, :2].expand(2, 2, 8, 128)[::1, 1:])
    with pytest.raises(ValueError):
        binding.attn_qk_norm_rope(q, wq=torch.ones(64))
    with pytest.raises(ValueError):
        binding.attn_qk_norm_rope(q, wk=torch.ones(128))
    with pytest.raises(ValueError):
        binding.attn_qk_norm_rope(q, positions=torch.zeros(4))
    with pytest.raises(ValueError):
        binding.PagedKVCache(q, q)


def test_tables_for_more_keys_than_are_counted(lib):
    """Keys are counted in 32 bits: a table that could hold more is refused, one that just fits is not this check's."""
    assert attend(lib, cache(ps=1 << 20), mp=2048) == UNS
    assert attend(lib, cache(ps=1 << 20), mp=1 << 30) == UNS


def test_compiled_calls_turn_errors_into_exceptions():
    calls = binding._calls()
    with pytest.raises(TypeError):
        calls.qk_norm_rope(torch.zeros(1, 1, 64, dtype=torch.bfloat16))                  # the number of arguments
    with pytest.raises(TypeError, match="q must be a torch tensor"):
        binding.attn_qk_norm_rope([[0.0]])
    with pytest.raises(TypeError, match="cos must be a torch tensor"):
        binding.attn_qk_norm_rope(torch.zeros(1, 1, 64, dtype=torch.bfloat16), cos=1.0)
    with pytest.raises(TypeError):
        binding.attn_qk_norm_rope(torch.zeros(1, 1, 64, dtype=torch.bfloat16), eps="x")
    with pytest.raises((ValueError, RuntimeError)):                                       # a tensor without rows
        binding.attn_qk_norm_rope(torch.zeros(1, 1, 64, dtype=torch.bfloat16).to_sparse())
    with pytest.raises(ValueError, match="CUDA tensor on the current device"):
        binding.attn_qk_norm_rope(torch.zeros(1, 1, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA tensor on the current device"):
        binding.attn_qk_norm_rope(torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="meta"))


def test_a_workspace_has_the_bytes_that_its_size_says():
    """Expanded or cut with gaps: fewer or other bytes than numel() counts. Refused before anything else is looked at."""
    calls = binding._calls()
    c = cache()
    q, table, lens = torch.zeros(1, 1, 8, 128, dtype=torch.bfloat16), torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    x, w = torch.zeros(4, 8, 128, dtype=torch.bfloat16), torch.ones(128)
    for ws in (torch.empty(1, dtype=torch.uint8).expand(1 << 24), torch.empty(1 << 10, 2, dtype=torch.uint8)[:, 0]):
        with pytest.raises(ValueError, match="workspace must be a contiguous"):
            calls.fwd_paged(ctypes.addressof(c), 0, q, table, lens, True, None, ws, None, None)
        with pytest.raises(ValueError, match="workspace must be a contiguous"):
            binding.attn_qk_norm_rope_bwd(x, None, x, wq=w, workspace=ws)


@pytest.mark.parametrize("shape", [(0, 64), (50, 0), (0, 0)])
def test_tables_without_angles_are_no_rotation_left_out(shape):
    """cos[:n] with n = 0 is a mistake of the caller's, not a call without rotation; refused before the tensors' device counts."""
    t = torch.zeros(shape)
    x = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    ints = [torch.zeros(n, dtype=torch.int32) for n in (2, 1)]
    with pytest.raises(ValueError, match="no angles"):
        binding.attn_qk_norm_rope(x, cos=t, sin=t)
    with pytest.raises(ValueError, match="no angles"):
        binding.attn_qk_norm_rope_bwd(x, None, x, cos=t, sin=t)
    c = cache(Hkv=8)
    with pytest.raises(ValueError, match="no angles"):
        binding._calls().paged_append(ctypes.addressof(c), 0, x, x, *ints, torch.zeros(1, 2, dtype=torch.int32), t, t, False)
    with pytest.raises(ValueError, match="on the current device"):     # without tokens there is nothing to turn
        binding.attn_qk_norm_rope(x[:0], cos=t, sin=t)

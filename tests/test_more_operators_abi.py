"""Refusals of norm and rotation with several axes and of attention of chunks over the paged cache that need no GPU: every bad
argument is turned away before any CUDA call. Addresses are made up and never read."""
import ctypes
import types

import numpy as np
import pytest
import torch

from exact_attention_72_gb300 import binding, build

INV, UNS, OK = binding.ATTN_ERR_INVALID_ARG, binding.ATTN_ERR_UNSUPPORTED, binding.ATTN_OK
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def axes(lib, q=16 * MB, pos=6 * MB, stride=10, n=3, of=bytes([0] * 16 + [1] * 24 + [2] * 24), cos=4 * MB, sin=5 * MB, rd=128, d=128,
         max_pos=100, T=10, qo=48 * MB):
    return lib.attn_qk_norm_rope_axes(q, 32 * MB, qo, 64 * MB, T, 8, 2, d, 1024, 128, 256, 128, 1, MB, 2 * MB, 1e-6, cos, sin, rd,
                                      max_pos, 0, pos, stride, n, of, None)


def axes_bwd(lib, q=16 * MB, pos=6 * MB, stride=10, n=3, of=bytes([0] * 16 + [1] * 24 + [2] * 24), cos=4 * MB, sin=5 * MB, rd=128,
             d=128, max_pos=100, T=10, qo=48 * MB):
    return lib.attn_qk_norm_rope_axes_bwd(q, 32 * MB, 80 * MB, 96 * MB, qo, 64 * MB, 3 * MB, 3 * MB + 4096, T, 8, 2, d, 1024, 128,
                                          256, 128, 1, MB, 2 * MB, 1e-6, cos, sin, rd, max_pos, 0, pos, stride, n, of, 128 * MB, MB,
                                          None)


@pytest.mark.parametrize("call", [axes, axes_bwd])
@pytest.mark.parametrize("bad", [
    dict(pos=0), dict(pos=6 * MB + 2), dict(stride=9), dict(stride=1 << 41), dict(n=0), dict(n=5), dict(n=2), dict(of=None),
    dict(of=bytes([0] * 63 + [3])), dict(cos=0), dict(sin=0), dict(cos=0, sin=0), dict(rd=24), dict(rd=0), dict(max_pos=0), dict(T=0),
    dict(q=0), dict(q=16 * MB + 8), dict(qo=32 * MB),
])
def test_axes_refuses(lib, call, bad):
    assert call(lib, **bad) == INV


@pytest.mark.parametrize("call", [axes, axes_bwd])
def test_axes_unsupported(lib, call):
    assert call(lib, d=96) == UNS


@pytest.mark.parametrize("sections,turns,want", [
    ((2, 1, 3), False, [0, 0, 1, 2, 2, 2]), ((2, 1, 3), True, [0, 1, 2, 0, 2, 2]), ((0, 2), True, [1, 1]), ((), False, []), ((), True, []),
])
def test_pair_axes(sections, turns, want):
    assert list(binding.rope_pair_axes(sections, turns)) == want


def cache_struct(kind="bf16", **over):
    d = over.pop("d", 128)
    row = d if kind == "bf16" else d // 2
    f = dict(k=1 << 30, v=2 << 30, k_sz=None if kind == "bf16" else 3 << 30, v_sz=None if kind == "bf16" else 4 << 30,
             page_stride=16 * 2 * row, token_stride=row, head_stride=16 * row, sz_page_stride=16 * 2 * d // 32,
             sz_token_stride=d // 32, sz_head_stride=16 * d // 32, num_pages=64, page_size=16, Hkv=2, d=d,
             type=0 if kind == "bf16" else 1)
    f.update(over)
    return binding._PagedCacheStruct(*[f[n] for n, _ in binding._PagedCacheStruct._fields_])


def chunk(lib, c=None, q=16 * MB, o=32 * MB, lse=48 * MB, table=MB, stride=8, max_pages=8, cu=2 * MB, lens=3 * MB, B=4, H=8, total=20,
          scale=0.1, ws=512 * MB, nbytes=1 << 28):
    c = cache_struct() if c is None else c
    return lib.attn_fwd_paged_varlen(q, ctypes.byref(c), o, lse, table, stride, max_pages, cu, lens, B, H, total, scale, 1, ws, nbytes,
                                     None)


@pytest.mark.parametrize("bad", [
    dict(q=0), dict(o=0), dict(lse=0), dict(table=0), dict(cu=0), dict(lens=0), dict(ws=0), dict(q=16 * MB + 8), dict(o=32 * MB + 8),
    dict(lse=48 * MB + 2), dict(table=MB + 2), dict(cu=2 * MB + 1), dict(lens=3 * MB + 2), dict(ws=512 * MB + 128), dict(B=0),
    dict(H=0), dict(H=7), dict(total=-1), dict(max_pages=0), dict(stride=-1), dict(scale=float("nan")), dict(scale=float("inf")),
])
@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_chunk_refuses(lib, kind, bad):
    assert chunk(lib, cache_struct(kind), **bad) == INV


@pytest.mark.parametrize("bad", [
    dict(k=0), dict(v=0), dict(k=(1 << 30) + 8), dict(page_stride=-16), dict(token_stride=4), dict(num_pages=0), dict(Hkv=0),
    dict(type=2), dict(head_stride=1 << 41),
])
@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_chunk_refuses_caches(lib, kind, bad):
    assert chunk(lib, cache_struct(kind, **bad)) == INV


def test_chunk_refuses_4_bit_caches_without_pairs(lib):
    assert chunk(lib, cache_struct("int4", k_sz=0)) == INV
    assert chunk(lib, cache_struct("int4", sz_token_stride=3)) == INV


@pytest.mark.parametrize("bad,over", [
    (dict(scale=0.0), {}), (dict(H=2 * 129), {}), (dict(total=2 ** 31 - 1), {}), (dict(max_pages=1 << 28), {}), ({}, dict(d=96)),
    ({}, dict(page_size=24)), (dict(max_pages=1 << 26, total=1 << 30, B=1 << 20), {}),
])
def test_chunk_unsupported(lib, bad, over):
    assert chunk(lib, cache_struct(**over), **bad) == UNS


def test_workspace_sizes(lib):
    n = lib.attn_fwd_paged_varlen_workspace_bytes
    assert n(1, 8, 2, 10, 128, 0) == n(50, 64, 8, 9999, 128, 1) >= 2 * 256 * 128 * 4
    for bad in ((0, 8, 2, 10, 128, 0), (1, 7, 2, 10, 128, 0), (1, 8, 0, 10, 128, 0), (1, 8, 2, -1, 128, 0), (1, 8, 2, 10, 96, 0),
                (1, 8, 2, 10, 128, 2)):
        assert n(*bad) == 0


@pytest.mark.parametrize("bad", [64, 3, True, 1.5, None, "0" * 64, [0.0] * 64, np.zeros(64)])
def test_pair_axis_is_a_sequence_of_whole_numbers(bad, monkeypatch):
    """bytes(64) would be 64 pairs of axis 0."""
    monkeypatch.setattr(binding, "_CALLS", types.SimpleNamespace(qk_norm_rope=None, qk_norm_rope_bwd=None))
    with pytest.raises(TypeError, match="iterable|interpreted as an integer"):
        binding.attn_qk_norm_rope_axes(None, None, None, None, None, bad)
    with pytest.raises(TypeError, match="iterable|interpreted as an integer"):
        binding.attn_qk_norm_rope_axes_bwd(None, None, None, None, None, None, None, bad)


@pytest.mark.parametrize("kind", [bytes, bytearray, list, tuple, iter, np.array, lambda x: np.array(x, np.uint8), torch.tensor])
def test_pair_axis_by_elements(kind, monkeypatch):
    """Arrays count by their elements, not by the bytes that hold them: 8 numbers of 64 bits are not 64 axes."""
    axes = [0, 1, 2, 0, 1, 2, 1, 0]
    calls = types.SimpleNamespace(qk_norm_rope=lambda *a: a[10], qk_norm_rope_bwd=lambda *a: a[10])
    monkeypatch.setattr(binding, "_CALLS", calls)
    assert binding.attn_qk_norm_rope_axes(None, None, None, None, None, kind(axes)) == bytes(axes)
    assert binding.attn_qk_norm_rope_axes_bwd(None, None, None, None, None, None, None, kind(axes)) == bytes(axes)

"""Argument validation of the packed-prompt and cache-eviction entry points: every refusal comes
before any CUDA call, so none of this needs a GPU."""
import ctypes

import pytest
import torch

import rope_context_extension_bifocal_b200 as bfl
from tests.test_abi import FAKE, lib, params  # noqa: F401  (fixture)

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5


def test_prefill_packed_validation(lib):
    f = lib.bifocal_prefill_packed

    def call(p=None, q=FAKE, k=FAKE, cu=FAKE, T=100, B=3, max_len=60, dtype=0, out=FAKE, lse=None, kc=None, vc=None,
             kpos=None, rows=0, page=0, table=None, max_pages=0, ws=FAKE, wsb=0):
        return f(q, k, FAKE, dtype, T, B, cu, max_len, ctypes.byref(p or params()), out, lse, kc, vc, kpos, rows, page,
                 table, max_pages, ws, wsb, None)

    assert call() == WORKSPACE  # valid up to the (empty) workspace
    assert call(ws=None) == WORKSPACE
    assert call(ws=FAKE + 16, wsb=1 << 40) == WORKSPACE
    for bad in (dict(q=None), dict(k=FAKE + 4), dict(cu=None), dict(cu=FAKE + 2), dict(out=None), dict(out=FAKE + 2),
                dict(lse=FAKE + 1), dict(T=0), dict(B=0), dict(max_len=0), dict(p=params(w0=-1)),
                dict(p=params(w_pretrained=0)), dict(p=params(hq=30)), dict(p=params(theta=1.0)),
                dict(p=params(flags=bfl.FLAG_WINDOW, w0=0)),
                dict(kc=FAKE), dict(kpos=FAKE), dict(kc=FAKE, vc=FAKE), dict(kc=FAKE, vc=FAKE, rows=99),
                dict(kc=FAKE, vc=FAKE + 2, rows=100), dict(kc=FAKE, vc=FAKE, kpos=FAKE + 1, rows=100),
                dict(kc=FAKE, vc=FAKE, rows=96, table=FAKE, page=0, max_pages=8),
                dict(kc=FAKE, vc=FAKE, rows=100, table=FAKE, page=16, max_pages=8),   # not whole pages
                dict(kc=FAKE, vc=FAKE, rows=96, table=FAKE, page=16, max_pages=3),    # 48 < max_len
                dict(kc=FAKE, vc=FAKE, rows=96, table=FAKE + 2, page=16, max_pages=8),
                dict(kc=FAKE, vc=FAKE, rows=1 << 31, table=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dtype=5), dict(p=params(head_dim=96)), dict(p=params(flags=bfl.FLAG_MMA_SYNC)),
                dict(p=params(flags=bfl.FLAG_WINDOW, w0=8, hq=24))):
        assert call(**bad) == UNSUPPORTED, bad
    for good in (dict(p=params(flags=bfl.FLAG_WINDOW, w0=8, head_dim=64)), dict(kc=FAKE, vc=FAKE, rows=100), dict(kc=FAKE, vc=FAKE, rows=96, table=FAKE, page=48, max_pages=2)):
        assert call(**good) == WORKSPACE, good


def test_prefill_packed_workspace_size(lib):
    T, B = 1000, 4
    s = bfl.prefill_packed_workspace_size(bfl.DTYPE_BF16, B, T, params())
    forms = 2 * (T * 32 * 128 * 2) + 2 * (T * 8 * 128 * 2)
    assert forms < s <= forms + 4096
    assert bfl.prefill_packed_workspace_size(bfl.DTYPE_FP32, B, T, params()) == s + T * 8 * 128 * 2
    assert bfl.prefill_packed_workspace_size(bfl.DTYPE_BF16, 0, T, params()) == 0
    assert bfl.prefill_packed_workspace_size(bfl.DTYPE_BF16, B, 0, params()) == 0
    assert bfl.prefill_packed_workspace_size(9, B, T, params()) == 0


def test_binding_refuses_cpu_and_strided_tensors(lib):
    q = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(bfl.BifocalError) as e:
        bfl.bifocal_prefill_packed(q, q, q, cu, 4, w0=1, w_pretrained=8, theta=1e6)
    assert e.value.status == INVALID


def test_decode_kept_validation(lib):
    f = lib.bifocal_decode_kept

    def call(p=None, q=FAKE, kn=FAKE, kc=FAKE, vc=FAKE, kpos=FAKE, kw=FAKE, rows=160, page=16, table=FAKE, max_pages=5,
             lens=FAKE, pos=FAKE, max_len=80, B=2, out=FAKE, lse=None, ws=FAKE, wsb=0):
        return f(q, kn, FAKE, kc, vc, kpos, kw, rows, page, table, max_pages, lens, pos, max_len, B, ctypes.byref(p or params()),
                 out, lse, ws, wsb, None)

    assert call() == WORKSPACE and call(kw=None) == WORKSPACE and call(ws=None) == WORKSPACE
    for bad in (dict(q=None), dict(kn=FAKE + 8), dict(kc=None), dict(vc=FAKE + 2), dict(kpos=None), dict(kpos=FAKE + 2),
                dict(kw=FAKE + 2), dict(rows=0), dict(rows=161), dict(page=0), dict(table=None), dict(table=FAKE + 1),
                dict(max_pages=4), dict(max_pages=0), dict(lens=None), dict(pos=None), dict(pos=FAKE + 2), dict(max_len=0),
                dict(B=0), dict(out=None), dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(p=params(w0=-1)),
                dict(p=params(theta=0.5)), dict(p=params(flags=bfl.FLAG_WINDOW, w0=0))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(p=params(head_dim=96)), dict(p=params(hq=72, hkv=8)), dict(B=65536)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(p=params(hq=64, hkv=8)) == WORKSPACE and call(p=params(flags=bfl.FLAG_WINDOW, w0=8)) == WORKSPACE
    small = bfl.decode_kept_workspace_size(2, 80, False, params())
    assert 0 < small < bfl.decode_kept_workspace_size(2, 80, True, params())
    assert bfl.decode_kept_workspace_size(0, 80, True, params()) == 0


def test_cache_evict_validation(lib):
    f = lib.bifocal_cache_evict

    def call(kc=FAKE, vc=FAKE, kpos=FAKE, kw=FAKE, rows=160, page=16, table=FAKE, max_pages=5, dst=None, dst_pages=0, lens=FAKE,
             pos=FAKE, new=FAKE, B=2, hkv=8, D=128, max_len=80, budget=32, recent=8, sink=4, ws=FAKE, wsb=0):
        return f(kc, vc, kpos, kw, rows, page, table, max_pages, dst, dst_pages, lens, pos, new, B, hkv, D, max_len, budget,
                 recent, sink, ws, wsb, None)

    assert call() == WORKSPACE and call(ws=None) == WORKSPACE and call(recent=28) == WORKSPACE
    for bad in (dict(kc=None), dict(vc=FAKE + 8), dict(kpos=None), dict(kw=None), dict(kw=FAKE + 2), dict(rows=150),
                dict(rows=1 << 32), dict(page=0), dict(table=None), dict(max_pages=4), dict(lens=None), dict(pos=None),
                dict(new=None), dict(new=FAKE + 2), dict(B=0), dict(hkv=0), dict(max_len=0), dict(budget=0), dict(recent=-1),
                dict(sink=-1), dict(recent=29), dict(recent=1 << 30, sink=1 << 30), dict(dst=FAKE, dst_pages=1),
                dict(dst=FAKE + 2, dst_pages=2)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(D=96), dict(B=65536), dict(hkv=65536)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(dst=FAKE, dst_pages=2) == WORKSPACE
    assert bfl.cache_evict_workspace_size(2, 8, 80, 32) > 0 and bfl.cache_evict_workspace_size(2, 8, 80, 0) == 0


def test_key_weights_validation(lib):
    f = lib.bifocal_key_weights

    def call(p=None, q=FAKE, k=FAKE, dtype=0, lse=FAKE, T=100, B=3, cu=FAKE, max_len=60, obs=16, kw=FAKE, rows=100, page=0,
             table=None, max_pages=0, ws=FAKE, wsb=0):
        return f(q, k, dtype, lse, T, B, cu, max_len, obs, ctypes.byref(p or params()), kw, rows, page, table, max_pages, ws,
                 wsb, None)

    assert call() == WORKSPACE and call(ws=None) == WORKSPACE and call(obs=1 << 30) == WORKSPACE
    assert call(p=params(hq=72, head_dim=64)) == WORKSPACE  # any group
    assert call(rows=96, table=FAKE, page=24, max_pages=3) == WORKSPACE
    for bad in (dict(q=None), dict(k=FAKE + 8), dict(lse=None), dict(lse=FAKE + 2), dict(T=0), dict(B=0), dict(cu=None),
                dict(max_len=0), dict(obs=0), dict(kw=None), dict(kw=FAKE + 1), dict(rows=99), dict(rows=0),
                dict(rows=96, table=FAKE, page=24, max_pages=2), dict(rows=97, table=FAKE, page=24, max_pages=3),
                dict(p=params(w0=-1)), dict(p=params(flags=bfl.FLAG_WINDOW, w0=0))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dtype=3), dict(p=params(head_dim=32)), dict(p=params(flags=bfl.FLAG_MMA_SYNC))):
        assert call(**bad) == UNSUPPORTED, bad
    small = bfl.key_weights_workspace_size(3, 1000, 600, 16, params())
    assert 0 < small < bfl.key_weights_workspace_size(3, 1000, 600, 600, params())
    assert bfl.key_weights_workspace_size(3, 1000, 600, 0, params()) == 0


def test_binding_refuses_a_stream_of_another_device():
    """Its kernels would run on that device, over pointers of another one."""
    class Stream:
        device = torch.device("cuda", 1)
    with pytest.raises(bfl.BifocalError) as e:
        bfl._On(torch.device("cuda", 0), Stream(), "bifocal_decode_kept")
    assert e.value.status == INVALID and "bifocal_decode_kept" in str(e.value)
    assert bfl._On(torch.device("cuda", 1), Stream(), "bifocal_decode_kept").stream is not None
    assert bfl._On(torch.device("cuda", 0), None, "bifocal_decode_kept").stream is None

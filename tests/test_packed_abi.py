"""Packed prompts and page calls: what the C ABI and the Python binding refuse, on the host
and before any launch.  No test here touches device memory."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

from bit_asymmetric_kv_gb300 import build as kbuild
from bit_asymmetric_kv_gb300 import kivi

FAKE = 1 << 20  # an aligned, never dereferenced address


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kivi.lib()


def _rows(data=FAKE, ts=1024, hs=128):
    return kivi.kivi_rows(data, ts, hs)


def _attention(L, Hq=8, Hkv=2, D=128, n_seqs=3, cu=FAKE, T=100, q=None, k=None, v=None, scale=0.1, out=None):
    rows = [r or _rows() for r in (q, k, v, out)]
    return L.kivi_prefill_attention_packed(Hq, Hkv, D, n_seqs, cu, T, rows[0], rows[1], rows[2], scale, rows[3], 0)


@pytest.mark.parametrize("bad,status", [
    (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(Hq=-4), 1), (dict(Hq=7), 3), (dict(D=64), 3), (dict(D=256), 3),
    (dict(n_seqs=0), 1), (dict(n_seqs=513), 3), (dict(cu=0), 1), (dict(cu=FAKE + 2), 2), (dict(T=-1), 1),
    (dict(T=1 << 31), 3), (dict(q=_rows(0)), 1), (dict(k=_rows(0)), 1), (dict(v=_rows(0)), 1), (dict(out=_rows(0)), 1),
    (dict(q=_rows(FAKE + 8)), 2), (dict(v=_rows(ts=1028)), 2), (dict(k=_rows(hs=132)), 2), (dict(k=_rows(hs=0)), 1),
    (dict(q=_rows(ts=-1024)), 1), (dict(v=_rows(ts=(1 << 38) + 8)), 3), (dict(v=_rows(hs=(1 << 38) + 8)), 3),
    (dict(scale=0.0), 1), (dict(scale=-0.1), 1), (dict(scale=math.inf), 1), (dict(scale=math.nan), 1),
    (dict(scale=2.0**127 * 1.01), 1),
    (dict(out=_rows(ts=128, hs=128)), 1),        # every head of a token on the next token's first
    (dict(out=_rows(ts=1016, hs=128)), 1),       # the last head reaches into the next token
    (dict(out=_rows(ts=128, hs=99 * 128)), 1),   # the last token reaches into the next head
    (dict(T=2**31 - 1, Hq=4096, Hkv=4096, out=_rows(ts=4096 * 128)), 3),  # more blocks than a grid holds
])
def test_attention_refuses(L, bad, status):
    assert _attention(L, **bad) == status


def test_attention_of_nothing_launches_nothing(L):
    assert _attention(L, T=0) == 0


def _dims(**kw):
    d = dict(B=2, Hkv=4, D=128, G=32, bits=2, value_residual=0, page_tokens=64, max_pages_per_seq=8, num_pages=20)
    d.update(kw)
    return kivi.kivi_paged_dims(*d.values())


def _cache(table=FAKE, v_res=0):
    return kivi.kivi_paged_cache(FAKE, FAKE, FAKE, FAKE, FAKE, v_res, table, FAKE)


@pytest.mark.parametrize("bad,status", [
    (dict(dims=_dims(B=0)), 1), (dict(dims=_dims(G=48)), 3), (dict(dims=_dims(page_tokens=96)), 3),
    (dict(dims=_dims(value_residual=1)), 1), (dict(cache=_cache(table=0)), 1),
    (dict(cu=0), 1), (dict(cu=FAKE + 1), 2), (dict(T=-1), 1), (dict(T=1 << 31), 3), (dict(k=_rows(0)), 1),
    (dict(v=_rows(FAKE + 2)), 2), (dict(k=_rows(ts=4)), 1), (dict(v=_rows(hs=129)), 2),
])
def test_packed_quantizer_refuses(L, bad, status):
    a = dict(dims=_dims(), cache=_cache(), cu=FAKE, T=10, k=_rows(), v=_rows())
    a.update(bad)
    assert L.kivi_paged_prefill_packed(a["dims"], a["cache"], a["cu"], a["T"], a["k"], a["v"], 0) == status


CALLS = ["kivi_paged_reserve", "kivi_paged_reorder", "kivi_paged_compact"]


@pytest.mark.parametrize("name", CALLS)
def test_page_calls_refuse(L, name):
    dims, ws = _dims(), kivi.kivi_paged_pool_workspace_bytes(_dims())
    assert ws > 0

    def call(dims=dims, cache=_cache(), table=FAKE, refs=FAKE, info=FAKE, array=FAKE, at=FAKE, nbytes=ws):
        pool = kivi.kivi_page_pool(table, refs, info)
        return getattr(L, name)(dims, cache, pool, array, at, nbytes, 0)

    assert call(dims=_dims(Hkv=0)) == 1
    assert call(dims=_dims(bits=3)) == 3
    assert call(dims=_dims(value_residual=1)) == 1           # no v_res
    assert call(dims=_dims(Hkv=1, num_pages=(1 << 30) + 1)) == 3
    assert call(table=FAKE + 4096) == 1                      # not the cache's table
    assert call(refs=0) == 1 and call(info=0) == 1 and call(array=0) == 1
    assert call(refs=FAKE + 4) == 2 and call(info=FAKE + 1) == 2 and call(array=FAKE + 2) == 2
    assert call(at=0) == 5 and call(nbytes=ws - 1) == 5 and call(nbytes=0) == 5
    assert call(at=FAKE + 8) == 2
    assert getattr(L, name)(dims, _cache(), None, FAKE, FAKE, ws, 0) == 1


def test_pool_workspace_bytes(L):
    d = dict(B=3, Hkv=5, G=64, max_pages_per_seq=7, num_pages=21)
    lists, table, plan, res = 2 * 96, 96, 80, 3 * 5 * 64 * 128 * 2
    assert kivi.kivi_paged_pool_workspace_bytes(_dims(**d)) == lists + table + plan + 16 + res
    assert kivi.kivi_paged_pool_workspace_bytes(_dims(value_residual=1, **d)) == lists + table + plan + 16 + 2 * res
    assert kivi.kivi_paged_pool_workspace_bytes(_dims(D=64)) == 0
    assert kivi.kivi_paged_pool_workspace_bytes(_dims(Hkv=1, num_pages=(1 << 30) + 1)) == 0


def test_binding_refuses_host_and_misshapen_tensors():
    half = torch.zeros((4, 2, 128), dtype=torch.float16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(TypeError):
        kivi.kivi_prefill_attention_packed(half, half, half, cu, 0.1)
    with pytest.raises(TypeError):
        kivi.kivi_prefill_attention_packed(half.float(), half, half, cu, 0.1)


def test_structs_match_the_header():
    assert ctypes.sizeof(kivi.kivi_rows) == 24 and ctypes.sizeof(kivi.kivi_page_pool) == 24

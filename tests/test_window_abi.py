"""Sliding-window calls: what the C ABI and the Python binding refuse, on the host and before any
launch.  No test here touches device memory."""
from __future__ import annotations

import math
import os
import re

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


def _attention(L, Hq=8, Hkv=2, D=128, n_seqs=3, cu=FAKE, T=100, cu_kv=FAKE, Tk=200, q=None, k=None, v=None, scale=0.1,
               window=10, sinks=4, out=None):
    rows = [r or _rows() for r in (q, k, v, out)]
    return L.kivi_prefill_attention_window(Hq, Hkv, D, n_seqs, cu, T, cu_kv, Tk, rows[0], rows[1], rows[2], scale,
                                           window, sinks, rows[3], 0)


@pytest.mark.parametrize("bad,status", [
    (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(Hq=7), 3), (dict(D=64), 3), (dict(n_seqs=0), 1), (dict(n_seqs=513), 3),
    (dict(cu=0), 1), (dict(cu=FAKE + 2), 2), (dict(T=-1), 1), (dict(T=1 << 31), 3),
    (dict(cu_kv=0), 1),                          # the same rows, and another number of them
    (dict(cu_kv=FAKE + 1), 2), (dict(Tk=-1), 1), (dict(Tk=1 << 31), 3),
    (dict(window=0), 1), (dict(window=-5), 1), (dict(sinks=-1), 1),
    (dict(q=_rows(0)), 1), (dict(k=_rows(0)), 1), (dict(v=_rows(0)), 1), (dict(out=_rows(0)), 1),
    (dict(q=_rows(FAKE + 8)), 2), (dict(v=_rows(ts=1028)), 2), (dict(k=_rows(hs=132)), 2), (dict(k=_rows(hs=0)), 1),
    (dict(v=_rows(ts=(1 << 38) + 8)), 3), (dict(scale=0.0), 1), (dict(scale=math.inf), 1), (dict(scale=math.nan), 1),
    (dict(out=_rows(ts=128, hs=128)), 1),        # every head of a token on the next token's first
    (dict(T=2**31 - 1, Hq=4096, Hkv=4096, out=_rows(ts=4096 * 128)), 3),  # more blocks than a grid holds
])
def test_attention_refuses(L, bad, status):
    assert _attention(L, **bad) == status


def test_attention_of_nothing_launches_nothing(L):
    assert _attention(L, T=0) == 0
    assert _attention(L, T=0, Tk=0, k=_rows(0), v=_rows(0)) == 0
    assert _attention(L, T=0, Tk=0, cu_kv=0) == 0


def _dims(**kw):
    d = dict(B=2, Hkv=4, D=128, G=32, bits=2, value_residual=0, page_tokens=64, max_pages_per_seq=8, num_pages=20)
    d.update(kw)
    return kivi.kivi_paged_dims(*d.values())


def _cache(table=FAKE, v_res=0):
    return kivi.kivi_paged_cache(FAKE, FAKE, FAKE, FAKE, FAKE, v_res, table, FAKE)


@pytest.mark.parametrize("bad,status", [
    (dict(window=0), 1), (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(dims=_dims(B=0)), 1),
    (dict(dims=_dims(B=513)), 3), (dict(dims=_dims(page_tokens=48)), 3), (dict(dims=_dims(value_residual=1)), 1),
    (dict(cache=_cache(table=0)), 1), (dict(Hq=0), 1), (dict(Hq=12), 3), (dict(q=0), 1), (dict(out=0), 1),
    (dict(q=FAKE + 8), 2), (dict(out=FAKE + 2), 2),
])
@pytest.mark.parametrize("step", [False, True])
def test_decode_refuses(L, bad, status, step):
    a = dict(dims=_dims(), cache=_cache(), q=FAKE, Hq=8, window=5, sinks=1, out=FAKE)
    a.update(bad)
    rest = (a["q"], a["Hq"], 0.1, a["window"], a["sinks"], a["out"], FAKE, 1 << 40, 0)
    if step:
        assert L.kivi_paged_decode_step_window(a["dims"], a["cache"], FAKE, FAKE, *rest) == status
    else:
        assert L.kivi_paged_decode_attention_window(a["dims"], a["cache"], *rest) == status


def test_step_refuses_its_token(L):
    rest = (FAKE, 8, 0.1, 5, 1, FAKE, FAKE, 1 << 40, 0)
    call = L.kivi_paged_decode_step_window
    assert call(_dims(), _cache(), 0, FAKE, *rest) == 1 and call(_dims(), _cache(), FAKE, 0, *rest) == 1
    assert call(_dims(), _cache(), FAKE + 4, FAKE, *rest) == 2 and call(_dims(), _cache(), FAKE, FAKE + 8, *rest) == 2


@pytest.mark.parametrize("bad,status", [
    (dict(dims=_dims(B=0)), 1), (dict(dims=_dims(G=48)), 3), (dict(dims=_dims(value_residual=1)), 1),
    (dict(cache=_cache(table=0)), 1), (dict(cu=0), 1), (dict(cu=FAKE + 1), 2), (dict(T=-1), 1), (dict(T=1 << 31), 3),
    (dict(k=_rows(0)), 1), (dict(v=_rows(FAKE + 2)), 2), (dict(k=_rows(ts=4)), 1), (dict(v=_rows(hs=129)), 2),
])
def test_extend_and_read_refuse(L, bad, status):
    a = dict(dims=_dims(), cache=_cache(), cu=FAKE, T=10, k=_rows(), v=_rows())
    a.update(bad)
    assert L.kivi_paged_extend_packed(a["dims"], a["cache"], a["cu"], a["T"], a["k"], a["v"], 0) == status
    for take in (0, FAKE):
        assert L.kivi_paged_read(a["dims"], a["cache"], a["cu"], a["T"], take, 4, a["k"], a["v"], 0) == status


def test_read_refuses(L):
    def call(take=FAKE, first=0, k=_rows(), v=_rows(), T=10):
        return L.kivi_paged_read(_dims(), _cache(), FAKE, T, take, first, k, v, 0)

    assert call(take=FAKE + 2) == 2 and call(first=-1) == 1
    assert call(k=_rows(ts=128, hs=128)) == 1 and call(v=_rows(ts=128, hs=9 * 128)) == 1  # elements on one another
    assert call(T=0) == 0 and L.kivi_paged_extend_packed(_dims(), _cache(), FAKE, 0, _rows(), _rows(), 0) == 0


def test_reserve_window_refuses(L):
    dims, ws = _dims(), kivi.kivi_paged_pool_workspace_bytes(_dims())

    def call(dims=dims, table=FAKE, refs=FAKE, info=FAKE, extra=FAKE, window=5, sinks=1, at=FAKE, nbytes=ws):
        pool = kivi.kivi_page_pool(table, refs, info)
        return L.kivi_paged_reserve_window(dims, _cache(), pool, extra, window, sinks, at, nbytes, 0)

    assert call(window=0) == 1 and call(window=-1) == 1 and call(sinks=-1) == 1
    assert call(dims=_dims(Hkv=0)) == 1 and call(dims=_dims(bits=3)) == 3 and call(table=FAKE + 4096) == 1
    assert call(refs=0) == 1 and call(info=0) == 1 and call(extra=0) == 1
    assert call(refs=FAKE + 4) == 2 and call(extra=FAKE + 2) == 2
    assert call(at=0) == 5 and call(nbytes=ws - 1) == 5 and call(at=FAKE + 8) == 2


def test_binding_refuses(L):
    half = torch.zeros((4, 2, 128), dtype=torch.float16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(TypeError):  # host tensors
        kivi.kivi_prefill_attention_window(half, half, half, cu, 4, 0, 0.1)
    assert kivi._count(2**40, "window", 1) == 2**31 - 1
    for bad in (0, -3):
        with pytest.raises(ValueError):
            kivi._count(bad, "window", 1)
    with pytest.raises(ValueError):
        kivi._count(-1, "sinks", 0)


@pytest.mark.parametrize("source", ["kivi_window_attention.cu", "kivi_read.cu"])
def test_grids_follow_the_device(source):
    """As test_launch_grids.py for the sources of these calls."""
    with open(os.path.join(kbuild.CSRC, source)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.search(r"\b(132|144|148|152|160)\b", code)  # SMs of a device as a number
    assert "device_sms(" in code

"""Window decode on batches with more units than the grid has warps, where units are counted and heads change within
a warp: every head layout, group size, code width and value residual, calls and steps.  Each test asserts that
its batch is that large.  Tolerance: that of test_gpu_window_decode.py."""
from __future__ import annotations

import math
import random

import pytest
import torch

from bit_asymmetric_kv_gb300 import build as kbuild
from bit_asymmetric_kv_gb300 import kivi
from paged_values import D, filled, seen, tokens
from test_gpu_window_decode import close, forget

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(D)
FORMS = [(G, bits, v_res) for G in (32, 64) for bits in (2, 4) for v_res in (False, True)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    kbuild.build()
    kivi.lib()


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def warps(c, Hq):
    """Warps of the paged decode grid, from its workspace: {int2 a head, n_warps + heads partials of D + 2 floats
    a query head}.  The window's kernel has no more."""
    heads = c.dims.B * c.dims.Hkv
    nbytes = kivi.kivi_paged_decode_workspace_bytes(c.dims, Hq)
    return (nbytes - 8 * heads) // (Hq // c.dims.Hkv * (D + 2) * 4) - heads


def units(n, G, window, sinks):
    nq = n // G * G
    return len({t // 64 for t in seen(n, window, sinks) if t < nq}) + (n > nq)


def assert_several_units_a_warp(c, Hq, window, sinks, lens):
    total = sum(units(n, c.dims.G, window, sinks) for n in lens) * c.dims.Hkv
    assert total > warps(c, Hq) >= sms(), (total, warps(c, Hq))


def aimed(c, Hq, window, sinks, seed, ahead=0):
    """Queries [B, Hq, D]; of the query heads of a KV head in turn, some point at the tokens next to the ends."""
    R = Hq // c.dims.Hkv
    q = torch.randn((c.dims.B, c.dims.Hkv, R, D), generator=torch.Generator().manual_seed(seed)).to(torch.float16).cuda()
    for b, n in enumerate(c.seq_lens.tolist()):
        edges = [t for t in (n + ahead - window - 1, n + ahead - window, sinks - 1, sinks) if 0 <= t < n]
        if edges:
            k = tokens(c, b, edges)[0]
            k = (k * (30 / (k.norm(dim=-1, keepdim=True) ** 2 * SCALE).clamp(min=1e-3))).to(torch.float16)
            for h in range(c.dims.Hkv):
                i = (b + h) % 5
                if i < len(edges):
                    q[b, h, (b + seed) % R] = k[i, h]
    return q.view(c.dims.B, Hq, D)


def reference(c, q, window, sinks):
    d = c.dims
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(c.seq_lens.tolist()):
        if n:
            k, v = tokens(c, b, seen(n, window, sinks))
            x = torch.einsum("hrd,jhd->hrj", q[b].double().view(d.Hkv, -1, D), k) * SCALE
            out[b] = torch.einsum("hrj,jhd->hrd", torch.softmax(x, -1), v).reshape(q.shape[1], D)
    return out


def ragged(B, most, G, seed):
    """Lengths without a residual, with one, of nothing but a residual, of nothing."""
    rng = random.Random(seed)
    lens = [0, 1, G - 1, G, 2 * G, 64, 65, most, 0, 0]
    lens += [rng.choice([G * rng.randrange(1, most // G), rng.randrange(1, most), rng.randrange(1, most)]) for _ in range(B - len(lens))]
    rng.shuffle(lens)
    return lens


WINDOWS = [(400, 4), (330, 0), (1000, 70)]


@pytest.mark.parametrize("G,bits,v_res", FORMS)
@pytest.mark.parametrize("R", [1, 2, 4])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_more_units_than_warps(G, bits, v_res, R, window, sinks):
    Hkv, P = 8, 64 if G == 32 else 128
    lens = ragged(72, 1300, G, R * window)
    c = filled(lens, Hkv, G, P, bits, v_res, seed=R)
    assert_several_units_a_warp(c, Hkv * R, window, sinks, lens)
    q = aimed(c, Hkv * R, window, sinks, window)
    ref = reference(c, q, window, sinks)
    forget(c, window, sinks)
    out = kivi.kivi_paged_decode_attention_window(c, q, window, sinks, SCALE)
    close(out, ref)
    assert all((out[b] == 0).all() for b, n in enumerate(lens) if n == 0)
    assert c.seq_lens.tolist() == lens
    for _ in range(3):
        assert torch.equal(out, kivi.kivi_paged_decode_attention_window(c, q, window, sinks, SCALE))


@pytest.mark.parametrize("G,bits,v_res", FORMS)
@pytest.mark.parametrize("R", [1, 4])
def test_many_heads_of_hardly_a_unit(G, bits, v_res, R):
    """More heads than warps, most of them a residual or a unit and a residual: a warp has several whole heads."""
    Hkv = 8
    lens = [(19 * i) % 140 for i in range(512)]
    c = filled(lens, Hkv, G, 64, bits, v_res, seed=21)
    assert_several_units_a_warp(c, Hkv * R, 30, 2, lens)
    q = aimed(c, Hkv * R, 30, 2, 1)
    close(kivi.kivi_paged_decode_attention_window(c, q, 30, 2, SCALE), reference(c, q, 30, 2))


@pytest.mark.parametrize("G,bits,v_res", FORMS)
@pytest.mark.parametrize("R", [1, 2, 4])
def test_steps_with_more_units_than_warps(G, bits, v_res, R):
    """Steps in a graph, over flushes: the append as kivi_paged_append_token writes it, the new token seen."""
    Hkv, window, sinks = 8, 500, 5
    lens = [n + (G - 2 - n % G if i % 3 == 0 else 0) for i, n in enumerate(ragged(64, 1200, G, 7))]
    a, b = (filled(lens, Hkv, G, 128, bits, v_res, seed=22, room=5) for _ in range(2))
    assert_several_units_a_warp(a, Hkv * R, window, sinks, lens)
    forget(a, window, sinks, ahead=1)
    k, v = (torch.empty((64, Hkv, D), dtype=torch.float16, device="cuda") for _ in "kv")
    q, out = (torch.empty((64, Hkv * R, D), dtype=torch.float16, device="cuda") for _ in "qo")
    ws = kivi.paged_workspace(a, Hkv * R)
    gen = torch.Generator("cuda").manual_seed(23)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kivi.kivi_paged_decode_step_window(a, k, v, q, window, sinks, SCALE, out=out, ws=ws)
    for step in range(4):
        k.normal_(generator=gen), v.normal_(generator=gen)
        kivi.kivi_paged_append_token(b, k, v)
        q.copy_(aimed(b, Hkv * R, window, sinks, step))
        if step % 2:
            g.replay()
        else:
            kivi.kivi_paged_decode_step_window(a, k, v, q, window, sinks, SCALE, out=out, ws=ws)
        close(out, reference(b, q, window, sinks))
        assert a.seq_lens.tolist() == b.seq_lens.tolist() == [n + step + 1 for n in lens]
        assert torch.equal(a.k_res, b.k_res) and (not v_res or torch.equal(a.v_res, b.v_res))
        for s, n in enumerate(a.seq_lens.tolist()):
            page, row = int(a.block_table[s, (n - 1) // 128]), (n - 1) % 128
            if not v_res:
                assert torch.equal(a.v_meta[page, :, row], b.v_meta[page, :, row]), (s, n)
                assert torch.equal(a.v_codes[page, :, row], b.v_codes[page, :, row]), (s, n)
            if n % G == 0:
                rows = slice(row - G + 1, row + 1)
                assert torch.equal(a.k_meta[page, :, row // G], b.k_meta[page, :, row // G]), (s, n)
                assert all(torch.equal(getattr(a, x)[page, :, rows], getattr(b, x)[page, :, rows])
                           for x in (("k_codes", "v_codes") if v_res else ("k_codes",))), (s, n)

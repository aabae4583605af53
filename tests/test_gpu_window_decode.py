"""Decode attention over a paged cache with a sliding window and sinks, against the formula in 64 bits over
the cache's own dequantized tokens, within the tolerance that the framework states for its decode
attention (2e-3).  Queries are aimed at the tokens next to the window's and the sinks' ends, so that one
token too many or too few changes the output by far more."""
from __future__ import annotations

import math

import pytest
import torch

from bit_asymmetric_kv_gb300 import build as kbuild
from bit_asymmetric_kv_gb300 import kivi
from helpers import ATOL
from paged_values import D, filled, seen, tokens

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(D)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    kbuild.build()
    kivi.lib()


def aimed(c, Hq, window, sinks, seed, ahead=0):
    """Queries [B, Hq, D]: of every four heads of the call, three that point at tokens at the edges."""
    d = c.dims
    R = Hq // d.Hkv
    q = torch.randn((d.B, Hq, D), generator=torch.Generator().manual_seed(seed)).to(torch.float16).cuda()
    for b, n in enumerate(c.seq_lens.tolist()):
        n = min(max(n, 0), d.max_pages_per_seq * d.page_tokens)
        lo = n + ahead - window
        for h in range(Hq):
            t = [None, lo - 1, lo, sinks if h % 8 < 4 else sinks - 1][(h + b) % 4]
            if t is not None and 0 <= t < n:
                k = tokens(c, b, [t])[0][0, h // R]
                q[b, h] = (k * (30 / (k.norm() * SCALE * k.norm()).clamp(min=1e-3))).to(torch.float16)
    return q


def reference(c, q, window, sinks, lens=None):
    d = c.dims
    R = q.shape[1] // d.Hkv
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(c.seq_lens.tolist() if lens is None else lens):
        n = min(max(n, 0), d.max_pages_per_seq * d.page_tokens)
        if n == 0:
            continue
        k, v = tokens(c, b, seen(n, window, sinks))
        for h in range(q.shape[1]):
            w = torch.softmax(k[:, h // R] @ q[b, h].double() * SCALE, 0)
            out[b, h] = w @ v[:, h // R]
    return out


def close(out, ref):
    err = (out.double() - ref).abs()
    assert torch.isfinite(out).all() and float(err.max()) <= ATOL, (float(err.max()), torch.nonzero(err > ATOL)[:4].tolist())


def forget(c, window, sinks, ahead=0):
    """Pages that hold no visible token lose their table entries; in the others, what no visible token
    needs becomes garbage (infinite scales among it)."""
    d = c.dims
    P, G = d.page_tokens, d.G
    for b, n in enumerate(c.seq_lens.tolist()):
        vis = set(seen(n + ahead, window, sinks))
        for j in range(-(-n // P)):
            if not vis & set(range(j * P, j * P + P)):
                c.block_table[b, j] = [-1, d.num_pages, 2**31 - 1, -2**31][(b + j) % 4]
                continue
            page = int(c.block_table[b, j])
            for g in range(P // G):
                at = set(range(j * P + g * G, j * P + g * G + G))
                if not vis & at and max(at) < n // G * G:
                    c.k_meta[page, :, g] = -1  # NaN
                    c.k_codes[page, :, g * G:g * G + G] = -1
            for t in range(j * P, min(n, j * P + P)):
                if t not in vis:
                    c.v_meta[page, :, t % P] = -1


SHAPES = [(32, 64, 2, False, 1, 1), (32, 64, 2, False, 2, 4), (64, 128, 2, False, 2, 2), (64, 64, 4, False, 1, 4),
          (32, 128, 4, True, 3, 1), (64, 256, 2, True, 1, 4), (32, 64, 4, True, 2, 2), (64, 64, 4, False, 2, 1)]


@pytest.mark.parametrize("G,P,bits,v_res,Hkv,R", SHAPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 4), (31, 0), (64, 64), (100, 4), (129, 65), (256, 32),
                                          (300, 500), (40, 5000), (2**31 - 1, 0), (33, 33)])
def test_lengths_windows_and_shapes(G, P, bits, v_res, Hkv, R, window, sinks):
    lens = [1, 0, 31, 32, 33, 63, 64, 65, 96, 127, 128, 200, 321, 640, 1000]
    c = filled(lens, Hkv, G, P, bits, v_res, seed=window + sinks)
    q = aimed(c, Hkv * R, window, sinks, 1)
    ref = reference(c, q, window, sinks)
    forget(c, window, sinks)
    out = kivi.kivi_paged_decode_attention_window(c, q, window, sinks, SCALE)
    close(out, ref)
    assert (out[1] == 0).all()
    assert c.seq_lens.tolist() == lens


@pytest.mark.parametrize("G,P,bits,v_res,Hkv,R", SHAPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (70, 4), (128, 0), (500, 30)])
def test_steps_across_flushes(G, P, bits, v_res, Hkv, R, window, sinks):
    """The step appends as kivi_paged_append_token does and sees the new token."""
    lens = [0, 1, G - 2, G, 63, 200, 444]
    B = len(lens)
    a = filled(lens, Hkv, G, P, bits, v_res, seed=3, room=6)
    b = filled(lens, Hkv, G, P, bits, v_res, seed=3, room=6)
    gen = torch.Generator().manual_seed(4)
    out = torch.empty((B, Hkv * R, D), dtype=torch.float16, device="cuda")
    ws = kivi.paged_workspace(a, Hkv * R)
    forget(a, window, sinks, ahead=1)
    for step in range(5):
        k, v = (torch.randn((B, Hkv, D), generator=gen).to(torch.float16).cuda() for _ in "kv")
        kivi.kivi_paged_append_token(b, k, v)
        q = aimed(b, Hkv * R, window, sinks, step)
        got = kivi.kivi_paged_decode_step_window(a, k, v, q, window, sinks, SCALE, out=out, ws=ws)
        assert got is out
        close(out, reference(b, q, window, sinks))
        assert torch.equal(a.seq_lens, b.seq_lens) and a.seq_lens.tolist() == [n + step + 1 for n in lens]
        same = torch.equal(a.k_res, b.k_res) and (not v_res or torch.equal(a.v_res, b.v_res))
        assert same
        for s, n in enumerate(a.seq_lens.tolist()):
            page, row = int(a.block_table[s, (n - 1) // P]), (n - 1) % P
            same = torch.equal(a.v_meta[page, :, row], b.v_meta[page, :, row])
            if n % G == 0:
                same &= torch.equal(a.k_meta[page, :, row // G], b.k_meta[page, :, row // G])
                same &= torch.equal(a.k_codes[page, :, row - G + 1:row + 1], b.k_codes[page, :, row - G + 1:row + 1])
            assert same, (s, n)


def test_a_window_over_everything_is_the_whole_context():
    lens = [5, 300, 0, 1200, 64]
    c = filled(lens, 2, 32, 64, 2, False, seed=5)
    q = torch.randn((5, 8, D), device="cuda").to(torch.float16)
    whole = kivi.kivi_paged_decode_attention(c, q, SCALE)
    for window, sinks in ((1200, 0), (2**40, 2**40), (1, 1200)):
        out = kivi.kivi_paged_decode_attention_window(c, q, window, sinks, SCALE).float()
        # Both sum the same terms in fp32, in other orders, and round once to fp16: half a step, 2^-11 |out|, each.
        # The sums: |out| < 4 here, at most 1200 terms in groups of 16, 2^-24 each: below 2^-13 in all.
        assert ((out - whole.float()).abs() <= 2 * 2.0**-11 * whole.float().abs() + 2.0**-13).all()


def test_long_contexts_and_many_sequences():
    lens = [(37 * i) % 700 for i in range(200)] + [9000, 16385]
    c = filled(lens, 1, 64, 128, 2, False, seed=6)
    for window, sinks in ((4096, 4), (130, 0)):
        q = aimed(c, 4, window, sinks, 7)
        close(kivi.kivi_paged_decode_attention_window(c, q, window, sinks, SCALE), reference(c, q, window, sinks))


def test_the_largest_batch():
    lens = [(13 * i) % 90 for i in range(512)]
    c = filled(lens, 1, 32, 64, 2, False, seed=8)
    q = torch.randn((512, 2, D), device="cuda").to(torch.float16)
    close(kivi.kivi_paged_decode_attention_window(c, q, 20, 2, SCALE), reference(c, q, 20, 2))


def test_lengths_that_make_no_sense_are_clamped():
    lens = [100, 128, 60]
    c = filled(lens, 1, 32, 64, 2, False, seed=9)
    c.seq_lens.copy_(torch.tensor([-5, 1000, 60], dtype=torch.int32))  # the capacity is 128
    q = torch.randn((3, 1, D), device="cuda").to(torch.float16)
    out = kivi.kivi_paged_decode_attention_window(c, q, 50, 2, SCALE)
    assert (out[0] == 0).all()
    close(out, reference(c, q, 50, 2))


@pytest.mark.parametrize("window,sinks", [(70, 4), (2000, 4)])  # one CTA a head, and the whole grid
@pytest.mark.parametrize("v_res", [False, True])
def test_steps_at_the_capacity(window, sinks, v_res):
    """A full sequence drops the token and attends to what it holds."""
    lens = [640, 640 - 1, 200, 0, 31]
    a = filled(lens, 2, 32, 64, 2, v_res, seed=14)
    b = filled(lens, 2, 32, 64, 2, v_res, seed=14)
    for c in (a, b):
        assert c.dims.max_pages_per_seq == 10
        c.block_table[3, 0] = c.dims.num_pages - 1
    for step in range(3):
        k, v = (torch.randn((5, 2, D), device="cuda", generator=torch.Generator("cuda").manual_seed(step)).to(torch.float16) for _ in "kv")
        q = aimed(a, 8, window, sinks, step)
        out = kivi.kivi_paged_decode_step_window(a, k, v, q, window, sinks, SCALE)
        kivi.kivi_paged_append_token(b, k, v)
        assert a.seq_lens.tolist() == b.seq_lens.tolist() == [640, 640, 201 + step, 1 + step, 32 + step]
        close(out, reference(b, q, window, sinks))


def test_offsets_past_32_bits():
    """Pages whose code words lie past element 2^31."""
    Hkv, P, lens = 8, 64, [300, 70]
    num = 2**31 // (Hkv * P * 8) + 20
    small = filled(lens, Hkv, 32, P, 2, False, seed=10)
    c = kivi.PagedCache.allocate(2, Hkv, 32, P, small.dims.max_pages_per_seq, num)
    shift = num - small.dims.num_pages
    for name in ("k_codes", "k_meta", "v_codes", "v_meta"):
        getattr(c, name)[shift:] = getattr(small, name)
    assert c.k_codes.numel() > 2**31
    c.k_res.copy_(small.k_res)
    c.seq_lens.copy_(small.seq_lens)
    c.block_table.copy_(torch.where(small.block_table >= 0, small.block_table + shift, -1))
    q = aimed(small, 16, 90, 3, 11)
    out = kivi.kivi_paged_decode_attention_window(c, q, 90, 3, SCALE)
    assert torch.equal(out, kivi.kivi_paged_decode_attention_window(small, q, 90, 3, SCALE))
    close(out, reference(small, q, 90, 3))


def test_in_a_graph_it_follows_the_lengths_and_on_two_streams():
    lens = [40, 63, 300, 500]
    a = filled(lens, 2, 32, 64, 2, False, seed=12, room=8)
    b = filled(lens, 2, 32, 64, 2, False, seed=12, room=8)
    k, v = (torch.randn((4, 2, D), device="cuda").to(torch.float16) for _ in "kv")
    q, out = torch.randn((4, 8, D), device="cuda").to(torch.float16), torch.empty((4, 8, D), dtype=torch.float16, device="cuda")
    ws = kivi.paged_workspace(a, 8)
    kivi.kivi_paged_decode_attention_window(a, q, 70, 4, SCALE, out=out, ws=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kivi.kivi_paged_decode_step_window(a, k, v, q, 70, 4, SCALE, out=out, ws=ws)
    for i in range(4):
        k.normal_(), v.normal_(), q.normal_()
        g.replay()
        kivi.kivi_paged_append_token(b, k, v)
        close(out, reference(b, q, 70, 4))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [kivi.kivi_paged_decode_attention_window(a, q, 70, 4, SCALE, stream=streams[i % 2]) for i in range(6)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in outs)


def test_binding_refuses():
    c = filled([40, 3], 2, 32, 64, 2, False, seed=13)
    q = torch.zeros((2, 4, D), dtype=torch.float16, device="cuda")
    call = kivi.kivi_paged_decode_attention_window
    for bad in (lambda: call(c, q, 0, 0, 1.0), lambda: call(c, q, 1, -1, 1.0), lambda: call(c, q[:1], 1, 0, 1.0),
                lambda: call(c, q, 1, 0, 1.0, out=q[:, :2].contiguous()),
                lambda: kivi.kivi_paged_decode_step_window(c, q, q, q, 1, 0, 1.0)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        call(c, q.float(), 1, 0, 1.0)
    with pytest.raises(kivi.KiviError) as e:
        call(c, q, 1, 0, 1.0, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == kivi.KIVI_ERR_WORKSPACE
    with pytest.raises(kivi.KiviError) as e:
        call(c, torch.zeros((2, 6, D), dtype=torch.float16, device="cuda"), 1, 0, 1.0,
             ws=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
    assert e.value.status == kivi.KIVI_ERR_UNSUPPORTED

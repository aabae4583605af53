"""Attention of packed prompts and chunks with a sliding window and sinks, against the formula in 64 bits.

Tolerance, element by element, before any run: that of the attention over whole prompts
(test_gpu_packed_prefill.py), with the visible keys of a row in place of all.  With A = sum_j p_j |v_j| / l
over them and c their number: the output's rounding, 2^-11 |out| and 2^-25 for fp16's smallest; the
probabilities' rounding to fp16, 2^-11 A, and 2^-24 max |v| c for those below its normal numbers; the scores,
2 e A with e = (128 * 2^-23 + 4 * 2^-24) max_j sum_c |q_c k_c| scale; the sums in fp32, at most
(c / 16 + 4 + 2 * 128 / 16) 2^-22 A (a tile at each end holds masked keys, which are added as zeros).
"""
from __future__ import annotations

import math
import random

import pytest
import torch

from bit_asymmetric_kv_gb300 import build as kbuild
from bit_asymmetric_kv_gb300 import kivi

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    kbuild.build()
    kivi.lib()


def pack(lens, heads, layout, seed, pad=0, lead=0, fill=math.nan):
    """fp16 tensors [T, count, D] of the given head counts, as views of one buffer, and the bounds; rows of no
    sequence hold `fill`."""
    T, total = lead + sum(lens) + pad, sum(heads)
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((T, total, D), generator=gen).to(torch.float16)
    x[:lead] = fill
    x[lead + sum(lens):] = fill
    if layout == "tokens":
        buf = x.cuda()
    elif layout == "heads":
        buf = x.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    else:  # rows longer than their heads, and a gap behind each head
        big = torch.full((T, total + 1, D + 24), fill, dtype=torch.float16, device="cuda")
        big[:, :total, 8:8 + D] = x.cuda()
        buf = big[:, :total, 8:8 + D]
    out, at = [], 0
    for c in heads:
        out.append(buf[:, at:at + c])
        at += c
    cu = torch.tensor([lead] + [lead + sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32).cuda()
    return out, cu


def visible(n, m, window, sinks, dev="cuda"):
    p = torch.arange(n, device=dev)[:, None] + m - n
    j = torch.arange(m, device=dev)[None]
    return (j <= p) & ((j > p - window) | (j < sinks))


def check(out, q, k, v, cu, window, sinks, scale, cu_kv=None, seqs=None, heads=None):
    """Every element of the given sequences and heads within the tolerance above."""
    bounds, kb = cu.tolist(), (cu if cu_kv is None else cu_kv).tolist()
    R = q.shape[1] // k.shape[1]
    for s in range(len(bounds) - 1) if seqs is None else seqs:
        a, b, ka, kz = bounds[s], bounds[s + 1], kb[s], kb[s + 1]
        n, m = b - a, kz - ka
        if n == 0:
            continue
        seen = visible(n, m, window, sinks)
        used = seen.any(0)  # keys and values that no row sees may be anything
        none = ~seen.any(1)
        for h in range(q.shape[1]) if heads is None else heads:
            Q = q[a:b, h].double()
            K, V = (torch.where(used[:, None], t[ka:kz, h // R].double(), 0.0) for t in (k, v))
            x = (Q @ K.t() * scale).masked_fill(~seen, -math.inf)
            p = torch.softmax(x, -1).masked_fill(none[:, None], 0)
            ref, A = p @ V, p @ V.abs()
            mag = (Q.abs() @ K.abs().t() * scale).masked_fill(~seen, 0)
            mag = mag.amax(-1, keepdim=True) if m else torch.zeros((n, 1), device="cuda")
            e = 128 * 2.0**-23 * mag + 4 * 2.0**-24 * mag
            c = seen.sum(-1, keepdim=True)
            tol = 2.0**-11 * ref.abs() + 2.0**-25 + (2.0**-11 + 2 * e + (c / 16 + 20) * 2.0**-22) * A
            tol = tol * 1.01 + 2.0**-24 * c * (V.abs().max() if m else 0)
            got = out[a:b, h].double()
            assert torch.isfinite(got).all(), (s, h)
            assert (got[none] == 0).all(), (s, h)
            err = (got - ref).abs()
            worst = (err - tol).amax()
            assert worst <= 0, (s, h, float(err.max()), float(worst), torch.where(err > tol)[0][:5].tolist())


LENS = [[1], [2], [17, 0, 64], [0, 5, 0, 128, 129, 0], [127, 128, 129, 255, 256, 257], [300], [640, 1], [1000, 0, 513],
        [0, 0, 7]]
WINDOWS = [(1, 0), (1, 1), (2, 4), (37, 0), (64, 4), (128, 0), (128, 130), (129, 3), (300, 4), (200, 200), (5, 1000),
           (5000, 0), (5000, 9)]


@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 2), (4, 2), (4, 1)])
def test_lengths_and_windows(lens, window, sinks, Hq, Hkv):
    (q, k, v), cu = pack(lens, [Hq, Hkv, Hkv], "tokens", 1, pad=3)
    out = kivi.kivi_prefill_attention_window(q, k, v, cu, window, sinks, 1 / math.sqrt(D))
    check(out, q, k, v, cu, window, sinks, 1 / math.sqrt(D))
    assert (out[sum(lens):] == 0).all()


CHUNKS = [([1], [1]), ([1], [700]), ([5, 0, 130, 1], [300, 40, 131, 0]), ([128, 256, 1], [1000, 129, 128]),
          ([300], [299]), ([300, 40], [17, 0]), ([257, 64, 200], [900, 63, 70]), ([40, 7], [0, 0]), ([513], [1]),
          ([260, 129], [128, 5])]


@pytest.mark.parametrize("lens,keys", CHUNKS, ids=str)
@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 4), (128, 0), (100, 4), (256, 128), (37, 300), (5000, 2)])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (8, 2), (16, 1)])
def test_chunks_behind_earlier_tokens(lens, keys, window, sinks, Hq, Hkv):
    """Queries as the last rows of their keys; more queries than keys; no keys at all."""
    (q,), cu = pack(lens, [Hq], "tokens", 2, pad=5, lead=2)
    (k, v), cu_kv = pack(keys, [Hkv, Hkv], "heads", 3, pad=30, lead=140)
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    got = kivi.kivi_prefill_attention_window(q, k, v, cu, window, sinks, 0.11, cu_seqlens_kv=cu_kv, out=out)
    assert got is out
    check(out, q, k, v, cu, window, sinks, 0.11, cu_kv)
    assert (out[:2] == 7).all() and (out[2 + sum(lens):] == 7).all()  # rows of no sequence


@pytest.mark.parametrize("layout", ["tokens", "heads", "gaps"])
@pytest.mark.parametrize("Hq,Hkv", [(3, 3), (6, 2), (7, 1), (12, 3), (16, 1), (32, 8), (32, 1), (5, 5)])
def test_heads_and_layouts(layout, Hq, Hkv):
    lens = [70, 0, 400, 1]
    (q, k, v), cu = pack(lens, [Hq, Hkv, Hkv], layout, 4, pad=40, lead=9)
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    if layout == "heads":
        out = out.transpose(0, 1).contiguous().transpose(0, 1)
    kivi.kivi_prefill_attention_window(q, k, v, cu, 50, 5, 0.11, out=out)
    check(out, q, k, v, cu, 50, 5, 0.11)
    assert (out[:9] == 7).all() and (out[9 + sum(lens):] == 7).all()


@pytest.mark.parametrize("width,at", [(160, 16), (160, 8), (152, 8), (128, 0)])  # rows on 32 bytes, and on 16 only
def test_writes_only_its_elements(width, at):
    (q, k, v), cu = pack([90, 130], [4, 2, 2], "tokens", 5)
    big = torch.full((222, 6, width), 5.0, dtype=torch.float16, device="cuda")
    out = big[1:221, 1:5, at:at + D]
    kivi.kivi_prefill_attention_window(q, k, v, cu, 40, 3, 0.1, out=out)
    check(out, q, k, v, cu, 40, 3, 0.1)
    out.fill_(5.0)
    assert (big == 5).all()


@pytest.mark.parametrize("poison", [math.inf, -math.inf, math.nan, 65504.0])
@pytest.mark.parametrize("window,sinks", [(20, 0), (20, 3), (200, 130), (90, 10)])
@pytest.mark.parametrize("Hq", [2, 8])
def test_what_no_query_sees_may_hold_anything(poison, window, sinks, Hq):
    """Other sequences, padding, and this one's keys between the sinks and the first query's window."""
    lens, keys = [40, 50, 300, 33], [700, 50, 800, 900]
    (q,), cu = pack(lens, [Hq], "tokens", 6, pad=20, fill=poison)
    (k, v), cu_kv = pack(keys, [2, 2], "tokens", 7, pad=200, lead=150, fill=poison)
    kb = cu_kv.tolist()
    for i, (n, m) in enumerate(zip(lens, keys)):
        unseen = ~visible(n, m, window, sinks).any(0)
        for t in (k, v):
            t[kb[i]:kb[i + 1]][unseen] = poison
    q[40:90] = poison  # a whole sequence of them
    k[kb[1]:kb[2]] = poison
    v[kb[1]:kb[2]] = poison
    out = kivi.kivi_prefill_attention_window(q, k, v, cu, window, sinks, 0.1, cu_seqlens_kv=cu_kv)
    check(out, q, k, v, cu, window, sinks, 0.1, cu_kv, seqs=[0, 2, 3])


@pytest.mark.parametrize("kind", ["rising", "falling", "spike", "equal", "large", "huge", "zero-q"])
def test_score_patterns(kind):
    """Running maxima that grow at every tile, never, or once; one-hot and uniform rows."""
    lens = [700, 130]
    (q, k, v), cu = pack(lens, [2, 1, 1], "tokens", 8)
    i = torch.arange(sum(lens), device="cuda").float()
    if kind in ("rising", "falling"):
        q[:] = 1.0
        ramp = i / 700 * 40 if kind == "rising" else 40 - i / 700 * 40
        k[:] = (ramp / 12.8)[:, None, None].to(torch.float16)
    elif kind == "spike":
        k[2] = q[650, 0] * 4
    elif kind == "equal":
        k[:] = k[:1]
        v[1::2] = -1.0
    elif kind == "large":
        q.mul_(30)
        k.mul_(30)
    elif kind == "huge":  # scores of 2^25 and more, small integers apart
        q.zero_()
        q[:, :, 0], q[:, :, 1] = 32768.0, 16.0
        k.zero_()
        k[:, :, 0] = 16384.0
        k[:, :, 1] = torch.randint(-3, 4, k[:, :, 1].shape, device="cuda").to(torch.float16)
    else:
        q.zero_()
    out = kivi.kivi_prefill_attention_window(q, k, v, cu, 260, 5, 0.1)
    check(out, q, k, v, cu, 260, 5, 0.1)


@pytest.mark.parametrize("scale", [1e-30, 2.0**100, 2.0**127])
def test_extreme_scales(scale):
    """Every weight the same; and the largest score alone."""
    (q, k, v), cu = pack([350], [1, 1, 1], "tokens", 9)
    out = kivi.kivi_prefill_attention_window(q, k, v, cu, 100, 3, scale)
    seen = visible(350, 350, 100, 3)
    x = (q[:, 0].double() @ k[:, 0].double().t()).masked_fill(~seen, -math.inf)
    w = torch.softmax(x * 1e9, -1) if scale > 1 else seen.double() / seen.sum(-1, keepdim=True)
    # the weights are exact or 2^-11 off; the output is rounded once
    assert (out[:, 0].double() - w @ v[:, 0].double()).abs().max() <= 2 * 2.0**-11 * float(v.abs().max())


def test_long_sequences():
    lens, old = [3000, 1, 5001], [4000, 9000, 0]
    (q,), cu = pack(lens, [4], "tokens", 10)
    (k, v), cu_kv = pack([n + o for n, o in zip(lens, old)], [1, 1], "tokens", 11)
    for window, sinks in ((1024, 4), (4096, 0)):
        out = kivi.kivi_prefill_attention_window(q, k, v, cu, window, sinks, 1 / math.sqrt(D), cu_seqlens_kv=cu_kv)
        check(out, q, k, v, cu, window, sinks, 1 / math.sqrt(D), cu_kv, heads=[0, 3])


def test_many_sequences():
    rng = random.Random(3)
    lens = [rng.choice([0, 1, 3, 40, 100, 140]) for _ in range(512)]
    keys = [max(0, n + rng.choice([0, 0, 50, 200, -20])) for n in lens]
    (q,), cu = pack(lens, [2], "tokens", 12)
    (k, v), cu_kv = pack(keys, [1, 1], "tokens", 13)
    out = kivi.kivi_prefill_attention_window(q, k, v, cu, 60, 4, 0.1, cu_seqlens_kv=cu_kv)
    check(out, q, k, v, cu, 60, 4, 0.1, cu_kv)


def test_offsets_past_32_bits():
    """Rows whose element offset passes 2^31 (and byte offset 2^32)."""
    H, far = 40, 430000
    buf = torch.empty((far + 300, H, D), dtype=torch.float16, device="cuda")
    assert far * H * D > 2**31
    buf[far - 10:] = torch.randn((310, H, D), device="cuda").to(torch.float16)
    q, k, v, out = buf[:, :4], buf[:, 36:38], buf[:, 38:], torch.empty_like(buf[:, 4:36])
    cu = torch.tensor([far, far + 1, far + 290], dtype=torch.int32, device="cuda")
    o = out[:, 28:]
    kivi.kivi_prefill_attention_window(q, k, v, cu, 100, 2, 0.1, out=o)
    check(o, q, k, v, cu, 100, 2, 0.1)


def test_a_window_as_long_as_the_prompt_is_the_whole_attention():
    lens = [500, 3, 0, 1111]
    (q, k, v), cu = pack(lens, [8, 2, 2], "tokens", 14)
    whole = kivi.kivi_prefill_attention_packed(q, k, v, cu, 0.1).float()
    for window, sinks in ((1111, 0), (2**31 - 1, 0), (2**40, 2**40), (1, 1111)):
        out = kivi.kivi_prefill_attention_window(q, k, v, cu, window, sinks, 0.1)
        # both round to fp16 (|out| < 4, half a step 2^-10 each); P adds 2^-11 |v| to each (|v| < 6)
        assert (out.float() - whole).abs().max() <= 2 * 2.0**-10 + 2 * 6 * 2.0**-11


def test_sinks_and_newest_rows_side_by_side_are_the_whole_sequence():
    """Keys cut to the sinks and what the chunk's windows reach give the whole sequence's result."""
    n, m, window, sinks = 70, 900, 130, 6
    (q,), cu = pack([n], [4], "tokens", 15)
    (k, v), cu_kv = pack([m], [2, 2], "tokens", 16)
    whole = kivi.kivi_prefill_attention_window(q, k, v, cu, window, sinks, 0.1, cu_seqlens_kv=cu_kv)
    kept = list(range(sinks)) + list(range(m - n - window + 1, m))
    cut = torch.tensor([0, len(kept)], dtype=torch.int32, device="cuda")
    out = kivi.kivi_prefill_attention_window(q, k[kept], v[kept], cu, window, sinks, 0.1, cu_seqlens_kv=cut)
    check(out, q, k, v, cu, window, sinks, 0.1, cu_kv)
    assert (out.float() - whole.float()).abs().max() <= 2 * 2.0**-10 + 2 * 6 * 2.0**-11


def test_the_same_bits_whatever_stands_around():
    lens, keys = [64, 333, 90], [200, 1000, 91]
    (q,), cu = pack(lens, [8], "tokens", 17)
    (k, v), cu_kv = pack(keys, [2, 2], "tokens", 18)
    out = kivi.kivi_prefill_attention_window(q, k, v, cu, 150, 4, 0.1, cu_seqlens_kv=cu_kv)
    one, kone = torch.tensor([0, 333], dtype=torch.int32, device="cuda"), torch.tensor([0, 1000], dtype=torch.int32, device="cuda")
    alone = kivi.kivi_prefill_attention_window(q[64:397], k[200:1200], v[200:1200], one, 150, 4, 0.1, cu_seqlens_kv=kone)
    assert torch.equal(out[64:397], alone)


@pytest.mark.parametrize("Hq,Hkv", [(25, 25), (50, 25), (96, 24)])
def test_head_sets(Hq, Hkv):
    """A key axis so long that the heads are taken in sets (K and V past the L2 cache): the same bits as
    the same sequences on a short axis."""
    T, lens = 20000, [2100, 0, 900, 33]
    x = torch.randn((T, Hq + 2 * Hkv, D), device="cuda", generator=torch.Generator("cuda").manual_seed(19),
                    dtype=torch.float32).to(torch.float16)
    cu = torch.tensor([0, 2100, 2100, 3000, 3033], dtype=torch.int32, device="cuda")
    n = sum(lens)
    out = [kivi.kivi_prefill_attention_window(t[:, :Hq], t[:, Hq:Hq + Hkv], t[:, Hq + Hkv:], cu, 500, 4, 0.1)
           for t in (x, x[:n])]
    assert torch.equal(out[0][:n], out[1]) and (out[0][n:] == 0).all()
    check(out[0], x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cu, 500, 4, 0.1, seqs=[0, 3], heads=[0, Hq - 1])


def test_bounds_that_make_no_sense():
    """Bounds outside the axes are clamped; falling ones are empty sequences.  Sequences that overlap give
    unspecified results, and nothing is touched outside the buffers."""
    (q, k, v), _ = pack([200], [2, 1, 1], "tokens", 20)
    big = torch.full((260, 2, D), 3.0, dtype=torch.float16, device="cuda")
    out = big[30:230]
    cu = torch.tensor([-50, 90, 60, 60, 2**31 - 1], dtype=torch.int32, device="cuda")
    kv = torch.tensor([-2**31, 70, 5, 2**31 - 1, 11], dtype=torch.int32, device="cuda")
    for cu_kv in (None, kv, torch.full_like(cu, 2**31 - 1), torch.zeros_like(cu)):
        kivi.kivi_prefill_attention_window(q, k, v, cu, 40, 2, 0.1, cu_seqlens_kv=cu_kv, out=out)
        assert (big[:30] == 3).all() and (big[230:] == 3).all()
    kivi.kivi_prefill_attention_window(q, k, v, cu, 40, 2, 0.1, out=out)
    # 0 .. 90, nothing, nothing, 60 .. 200: the rows past 90 belong to one sequence only
    ok = torch.tensor([60, 200], dtype=torch.int32, device="cuda")
    ref = kivi.kivi_prefill_attention_window(q, k, v, ok, 40, 2, 0.1)
    check(ref, q, k, v, ok, 40, 2, 0.1)
    assert torch.equal(out[90:], ref[90:])


def test_no_keys_at_all_and_no_queries():
    (q,), cu = pack([40, 0, 3], [4], "tokens", 21, pad=2)
    empty = torch.zeros((0, 2, D), dtype=torch.float16, device="cuda")
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    kivi.kivi_prefill_attention_window(q, empty, empty, cu, 5, 1, 0.1, cu_seqlens_kv=torch.zeros_like(cu), out=out)
    assert (out[:43] == 0).all() and (out[43:] == 7).all()
    none = kivi.kivi_prefill_attention_window(q[:0], empty, empty, torch.zeros_like(cu), 5, 1, 0.1)
    assert none.shape == (0, 4, D)


def test_same_result_every_time_and_on_two_streams():
    lens, keys = [500, 3, 0, 1111], [900, 3, 7, 1300]
    (q,), cu = pack(lens, [8], "tokens", 22)
    (k, v), cu_kv = pack(keys, [2, 2], "tokens", 23)
    first = kivi.kivi_prefill_attention_window(q, k, v, cu, 300, 4, 0.1, cu_seqlens_kv=cu_kv)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [kivi.kivi_prefill_attention_window(q, k, v, cu, 300, 4, 0.1, cu_seqlens_kv=cu_kv, stream=streams[i % 2])
            for i in range(6)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)


def test_in_a_graph_it_follows_the_device_lengths():
    (q,), cu = pack([100, 200, 44], [4], "tokens", 24)
    (k, v), cu_kv = pack([300, 400, 44], [1, 1], "tokens", 25)
    out = torch.zeros_like(q)
    kivi.kivi_prefill_attention_window(q, k, v, cu, 90, 3, 0.1, cu_seqlens_kv=cu_kv, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kivi.kivi_prefill_attention_window(q, k, v, cu, 90, 3, 0.1, cu_seqlens_kv=cu_kv, out=out)
    for bounds, kb in (([0, 100, 300, 344], [0, 300, 700, 744]), ([0, 0, 1, 344], [0, 0, 1, 744]),
                       ([0, 344, 344, 344], [0, 744, 744, 744]), ([0, 10, 20, 30], [700, 710, 711, 744])):
        cu.copy_(torch.tensor(bounds, dtype=torch.int32))
        cu_kv.copy_(torch.tensor(kb, dtype=torch.int32))
        out.zero_()
        g.replay()
        check(out, q, k, v, cu, 90, 3, 0.1, cu_kv)

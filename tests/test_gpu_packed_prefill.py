"""Packed prompts on the GPU: causal attention against the formula in 64 bits, and the packed
quantizer bit for bit against the one-sequence call and the CPU oracle.

Tolerance of the attention, element by element, before any run.  With A = sum_j p_j |v_j| / l:
  - the output is rounded to fp16 once: 2^-11 |out|;
  - the probabilities enter the P.V product in fp16, each off by at most 2^-11 of itself
    (they are scaled so that fp16 subnormals lie below 2^-24 of the largest): 2^-11 A + 2^-24 max |v|
    n / l, which is below 2^-24 max|v| n as l >= 1;
  - scores: products of fp16 are exact in fp32; a sum of 128 of them is off by at most
    128 * 2^-23 sum_c |q_c k_c| (an accumulator that truncates), the scale and the maximum by a few
    2^-24 of the score; e such steps change p by e relative, numerator and denominator: 2 e A;
  - the sums over the keys in fp32: 2^-23 per step of 16 keys, and 2^-22 per exponential:
    (n / 16 + 4) 2^-22 A.
"""
from __future__ import annotations

import math
import random

import numpy as np
import pytest
import torch

import oracle
from bit_asymmetric_kv_gb300 import build as kbuild
from bit_asymmetric_kv_gb300 import kivi
from helpers import u16, u32

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    kbuild.build()
    kivi.lib()


def pack(lens, heads, layout, seed, pad=0, lead=0, fill=math.nan):
    """fp16 tensors [T, count, D] of the given head counts, as views of one buffer; rows of no
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


def check_attention(out, q, k, v, cu, scale, seqs=None, heads=None):
    """Every element of the given sequences and heads within the tolerance above."""
    bounds = cu.tolist()
    R = q.shape[1] // k.shape[1]
    for s in range(len(bounds) - 1) if seqs is None else seqs:
        a, b = bounds[s], bounds[s + 1]
        n = b - a
        if n == 0:
            continue
        mask = torch.ones((n, n), dtype=torch.bool, device=q.device).triu(1)
        for h in range(q.shape[1]) if heads is None else heads:
            Q, K, V = q[a:b, h].double(), k[a:b, h // R].double(), v[a:b, h // R].double()
            x = (Q @ K.t() * scale).masked_fill(mask, -math.inf)
            p = torch.softmax(x, -1)
            ref, A = p @ V, p @ V.abs()
            mag = (Q.abs() @ K.abs().t() * scale).masked_fill(mask, 0).amax(-1, keepdim=True)
            e = 128 * 2.0**-23 * mag + 4 * 2.0**-24 * mag
            tol = 2.0**-11 * ref.abs() + 2.0**-25 + (2.0**-11 + 2 * e + (n / 16 + 4) * 2.0**-22) * A
            tol = tol * 1.01 + 2.0**-24 * n * V.abs().max()
            err = (out[a:b, h].double() - ref).abs()
            assert torch.isfinite(out[a:b, h]).all(), (s, h)
            worst = (err - tol).amax()
            assert worst <= 0, (s, h, float(err.max()), float(worst), [int(i) for i in torch.where(err > tol)[0][:5]])


LENS = [
    [1], [2], [17], [64], [1, 17, 64], [0, 5, 0, 128, 129, 0], [127, 128, 129, 255, 256, 257], [31, 32, 33, 63, 65, 1],
    [300], [640, 1], [1000, 0, 513], [385] * 3, [0, 0, 7],
]


@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 2), (4, 2), (4, 1)])
def test_attention_lengths(lens, Hq, Hkv):
    (q, k, v), cu = pack(lens, [Hq, Hkv, Hkv], "tokens", 1, pad=3)
    out = kivi.kivi_prefill_attention_packed(q, k, v, cu, 1 / math.sqrt(D))
    check_attention(out, q, k, v, cu, 1 / math.sqrt(D))


@pytest.mark.parametrize("layout", ["tokens", "heads", "gaps"])
@pytest.mark.parametrize("Hq,Hkv", [(3, 3), (6, 2), (7, 1), (8, 1), (12, 3), (16, 1), (32, 8), (32, 1), (5, 5)])
def test_attention_heads_and_layouts(layout, Hq, Hkv):
    lens = [70, 0, 200, 1]
    (q, k, v), cu = pack(lens, [Hq, Hkv, Hkv], layout, 2, pad=40, lead=9)
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    if layout == "heads":
        out = out.transpose(0, 1).contiguous().transpose(0, 1)
    got = kivi.kivi_prefill_attention_packed(q, k, v, cu, 0.11, out=out)
    assert got is out
    check_attention(out, q, k, v, cu, 0.11)
    assert (out[:9] == 7).all() and (out[9 + sum(lens):] == 7).all()  # rows of no sequence


@pytest.mark.parametrize("width,at", [(160, 16), (160, 8), (152, 8), (128, 0)])  # rows on 32 bytes, and on 16 only
def test_attention_writes_only_its_elements(width, at):
    (q, k, v), cu = pack([90, 130], [4, 2, 2], "tokens", 3)
    big = torch.full((222, 6, width), 5.0, dtype=torch.float16, device="cuda")
    out = big[1:221, 1:5, at:at + D]
    kivi.kivi_prefill_attention_packed(q, k, v, cu, 0.1, out=out)
    check_attention(out, q, k, v, cu, 0.1)
    out.fill_(5.0)
    assert (big == 5).all()


@pytest.mark.parametrize("scale", [1e-30, 2.0**100, 2.0**127])
def test_attention_extreme_scales(scale):
    """Every weight the same; and the largest score alone."""
    (q, k, v), cu = pack([150], [1, 1, 1], "tokens", 16)
    out = kivi.kivi_prefill_attention_packed(q, k, v, cu, scale)
    x = (q[:, 0].double() @ k[:, 0].double().t()).masked_fill(
        torch.ones((150, 150), dtype=torch.bool, device="cuda").triu(1), -math.inf)
    ref = torch.softmax(x * 1e9, -1) if scale > 1 else None
    if ref is None:
        ref = torch.ones_like(x).tril() / torch.arange(1, 151, device="cuda").double()[:, None]
    # the weights are exact or 2^-11 off; the output is rounded once
    assert (out[:, 0].double() - ref @ v[:, 0].double()).abs().max() <= 2 * 2.0**-11 * float(v.abs().max())


@pytest.mark.parametrize("poison", [math.inf, -math.inf, math.nan])
def test_attention_ignores_the_neighbours_values(poison):
    lens = [40, 50, 100, 33]
    (q, k, v), cu = pack(lens, [4, 2, 2], "tokens", 4, pad=200, fill=poison)
    for t in (q, k, v):
        t[40:90] = poison  # a whole sequence of them
    out = kivi.kivi_prefill_attention_packed(q, k, v, cu, 0.1)
    check_attention(out, q, k, v, cu, 0.1, seqs=[0, 2, 3])


@pytest.mark.parametrize("kind", ["rising", "falling", "spike", "equal", "large", "huge", "zero-q"])
def test_attention_score_patterns(kind):
    """Running maxima that grow at every tile, never, or once; one-hot and uniform rows."""
    lens = [700, 130]
    (q, k, v), cu = pack(lens, [2, 1, 1], "tokens", 5)
    i = torch.arange(sum(lens), device="cuda").float()
    if kind in ("rising", "falling"):
        q[:] = 1.0
        ramp = i / 700 * 40 if kind == "rising" else 40 - i / 700 * 40
        k[:] = (ramp / 12.8)[:, None, None].to(torch.float16)
    elif kind == "spike":
        k[300] = q[650, 0] * 4
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
    scale = 0.1
    out = kivi.kivi_prefill_attention_packed(q, k, v, cu, scale)
    check_attention(out, q, k, v, cu, scale)


def test_attention_many_small_weights():
    """A first key far above the others: their weights lie near the smallest that fp16 holds, and together
    they count."""
    n = 9000
    (q, k, v), cu = pack([n], [1, 1, 1], "tokens", 6)
    q[:] = 1.0
    k[:] = 0.0
    k[0] = 0.9
    v[:] = 1.0
    v[0] = -1.0
    out = kivi.kivi_prefill_attention_packed(q, k, v, cu, 0.1)  # weights e^-11.5 = 1e-5
    check_attention(out, q, k, v, cu, 0.1)


def test_attention_long_sequence():
    lens = [5000, 1, 9001]
    (q, k, v), cu = pack(lens, [4, 1, 1], "tokens", 7)
    out = kivi.kivi_prefill_attention_packed(q, k, v, cu, 1 / math.sqrt(D))
    check_attention(out, q, k, v, cu, 1 / math.sqrt(D), seqs=[1, 2], heads=[0, 3])
    check_attention(out, q, k, v, cu, 1 / math.sqrt(D), seqs=[0], heads=[1, 2])


def test_attention_many_sequences():
    rng = random.Random(3)
    lens = [rng.choice([0, 1, 3, 40, 100, 140]) for _ in range(512)]
    (q, k, v), cu = pack(lens, [2, 1, 1], "tokens", 8)
    out = kivi.kivi_prefill_attention_packed(q, k, v, cu, 0.1)
    check_attention(out, q, k, v, cu, 0.1)


def test_attention_offsets_past_32_bits():
    """Rows whose element offset passes 2^31 (and byte offset 2^32)."""
    H, far = 40, 430000
    buf = torch.empty((far + 300, H, D), dtype=torch.float16, device="cuda")
    assert far * H * D > 2**31
    buf[far - 10:] = torch.randn((310, H, D), device="cuda").to(torch.float16)
    q, k, v, out = buf[:, :4], buf[:, 36:38], buf[:, 38:], torch.empty_like(buf[:, 4:36])
    cu = torch.tensor([far, far + 1, far + 290], dtype=torch.int32, device="cuda")
    o = out[:, 28:]
    kivi.kivi_prefill_attention_packed(q, k, v, cu, 0.1, out=o)
    check_attention(o, q, k, v, cu, 0.1)


@pytest.mark.parametrize("Hq,Hkv", [(25, 25), (50, 25), (24, 24), (96, 24)])
def test_attention_head_sets(Hq, Hkv):
    """A token axis so long that the heads are taken in sets (K and V past the L2 cache), of even and uneven
    sizes: the same bits as the same sequences at the start of a short axis."""
    T, lens = 20000, [2100, 0, 900, 33]
    x = torch.randn((T, Hq + 2 * Hkv, D), device="cuda", generator=torch.Generator("cuda").manual_seed(17),
                    dtype=torch.float32).to(torch.float16)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
    n = sum(lens)
    out = [kivi.kivi_prefill_attention_packed(t[:, :Hq], t[:, Hq:Hq + Hkv], t[:, Hq + Hkv:], cu, 0.1)
           for t in (x, x[:n])]
    assert torch.equal(out[0][:n], out[1]) and (out[0][n:] == 0).all()
    check_attention(out[0], x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cu, 0.1, seqs=[0, 3], heads=[0, Hq // 2, Hq - 1])


def test_attention_bounds_that_make_no_sense():
    """Bounds outside the axis are clamped; falling ones are empty sequences."""
    (q, k, v), _ = pack([200], [2, 1, 1], "tokens", 9)
    out = torch.full(q.shape, 3.0, dtype=torch.float16, device="cuda")
    cu = torch.tensor([-50, 90, 60, 60, 2**31 - 1], dtype=torch.int32, device="cuda")
    kivi.kivi_prefill_attention_packed(q, k, v, cu, 0.1, out=out)
    # 0 .. 90, nothing, nothing, 60 .. 200: the rows past 90 belong to one sequence only
    ok = torch.tensor([60, 200], dtype=torch.int32, device="cuda")
    bounds = ok.tolist()
    Q, K, V = q[60:200, 0].double(), k[60:200, 0].double(), v[60:200, 0].double()
    x = (Q @ K.t() * 0.1).masked_fill(torch.ones((140, 140), dtype=torch.bool, device="cuda").triu(1), -math.inf)
    ref = torch.softmax(x, -1) @ V
    assert (out[90:, 0].double() - ref[30:]).abs().max() < 5e-3 and bounds == [60, 200]


def test_attention_same_result_every_time_and_on_two_streams():
    lens = [500, 3, 0, 1111]
    (q, k, v), cu = pack(lens, [8, 2, 2], "tokens", 10)
    first = kivi.kivi_prefill_attention_packed(q, k, v, cu, 0.1)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for i in range(6):
        outs.append(kivi.kivi_prefill_attention_packed(q, k, v, cu, 0.1, stream=streams[i % 2]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)


def test_attention_in_a_graph_follows_the_device_lengths():
    (q, k, v), cu = pack([100, 200, 44], [4, 1, 1], "tokens", 11)
    out = torch.zeros_like(q)
    kivi.kivi_prefill_attention_packed(q, k, v, cu, 0.1, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kivi.kivi_prefill_attention_packed(q, k, v, cu, 0.1, out=out)
    for bounds in ([0, 100, 300, 344], [0, 0, 1, 344], [0, 344, 344, 344]):
        cu.copy_(torch.tensor(bounds, dtype=torch.int32))
        out.zero_()
        g.replay()
        check_attention(out, q, k, v, cu, 0.1)


def test_attention_agrees_with_the_rectangular_call():
    B, Hq, Hkv, n = 3, 4, 2, 333
    gen = torch.Generator().manual_seed(12)
    q, k, v = (torch.randn((B, h, n, D), generator=gen).to(torch.float16).cuda() for h in (Hq, Hkv, Hkv))
    dims = kivi.make_dims(B, Hkv, 32, 352)
    a = kivi.kivi_prefill_attention(None, q, k, v, 0.1, dims=dims)
    cu = torch.tensor([0, n, 2 * n, 3 * n], dtype=torch.int32, device="cuda")
    pq, pk, pv = (t.transpose(1, 2).reshape(B * n, -1, D) for t in (q, k, v))
    b = kivi.kivi_prefill_attention_packed(pq, pk, pv, cu, 0.1).reshape(B, n, Hq, D).transpose(1, 2)
    # both round the output to fp16 (|out| < 4, half a step 2^-10 each); P adds 2^-11 |v| (|v| < 6)
    assert (a.float() - b.float()).abs().max() <= 2 * 2.0**-10 + 6 * 2.0**-11


# ------------------------------------------------------------------ packed quantizer
POOLS = ("k_codes", "k_meta", "v_codes", "v_meta", "k_res", "seq_lens", "v_res")


def paged(B, Hkv, G, P, maxp, num, bits, v_res, seed):
    c = kivi.PagedCache.allocate(B, Hkv, G, P, maxp, num, bits=bits, value_residual=v_res)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    for name in POOLS[:4]:
        t = getattr(c, name)
        t.copy_(torch.randint(-2**31, 2**31 - 1, t.shape, dtype=torch.int32, device="cuda", generator=gen))
    c.k_res.normal_(generator=gen)
    if v_res:
        c.v_res.normal_(generator=gen)
    c.seq_lens.fill_(5)
    return c


QLENS = [[1], [31, 32, 33], [63, 64, 65, 0], [0, 200, 1, 129], [700, 0, 256, 95, 128]]


@pytest.mark.parametrize("lens", QLENS, ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("G,P,bits,v_res", [(32, 64, 2, False), (64, 128, 2, False), (32, 128, 4, False),
                                            (64, 64, 4, True), (32, 256, 2, True)])
@pytest.mark.parametrize("layout", ["tokens", "heads", "gaps"])
def test_packed_quantizer_is_the_one_sequence_call(lens, G, P, bits, v_res, layout):
    B, Hkv = len(lens), 3
    maxp = max(1, max(-(-n // P) for n in lens))
    num = B * maxp + 2
    (k, v), cu = pack(lens, [Hkv, Hkv], layout, sum(lens) + G + bits, pad=11, lead=3)
    k[:, :, 7] *= 40
    a, b = (paged(B, Hkv, G, P, maxp, num, bits, v_res, 1) for _ in range(2))
    table = torch.randperm(num, generator=torch.Generator().manual_seed(2))[:B * maxp].reshape(B, maxp).int().cuda()
    a.block_table.copy_(table)
    b.block_table.copy_(table)
    kivi.kivi_paged_prefill_packed(a, k, v, cu)
    at = 3
    for s, n in enumerate(lens):
        if n:
            kivi.kivi_paged_prefill(b, s, k[at:at + n].transpose(0, 1).contiguous(),
                                    v[at:at + n].transpose(0, 1).contiguous())
        at += n
    for name in POOLS[:6] + (("v_res",) if v_res else ()):
        assert torch.equal(getattr(a, name), getattr(b, name)), name


def test_packed_quantizer_against_the_oracle():
    lens, Hkv, G, P = [150, 64, 33], 2, 32, 64
    (k, v), cu = pack(lens, [Hkv, Hkv], "tokens", 13)
    c = paged(3, Hkv, G, P, 3, 9, 2, False, 4)
    c.block_table.copy_(torch.tensor([[8, 0, 5], [1, -1, -1], [3, 9, -1]], dtype=torch.int32))
    kivi.kivi_paged_prefill_packed(c, k, v, cu)
    bt, at = c.block_table.tolist(), 0
    for s, n in enumerate(lens):
        kk, vv = (t[at:at + n].transpose(0, 1).contiguous()[None].cpu().numpy() for t in (k, v))
        o = oracle.prefill(kk, vv, G, 192)
        for t0 in range(0, n, P):
            m, page = min(P, n - t0), bt[s][t0 // P]
            g = min(n // G * G - t0, P) // G if n // G * G > t0 else 0
            assert np.array_equal(u32(c.k_codes)[page, :, :g * G], o.k_codes[0, :, t0:t0 + g * G])
            assert np.array_equal(u32(c.k_meta)[page, :, :g], o.k_meta[0, :, t0 // G:t0 // G + g])
            assert np.array_equal(u32(c.v_codes)[page, :, :m], o.v_codes[0, :, t0:t0 + m])
            assert np.array_equal(u32(c.v_meta)[page, :, :m], o.v_meta[0, :, t0:t0 + m])
        assert np.array_equal(u16(c.k_res)[s, :, :n % G], o.k_res[0, :, :n % G])
        assert int(c.seq_lens[s]) == n
        at += n


def test_packed_quantizer_adversarial_values():
    """Rows that take the fp32 forms: ties, thresholds next to zero, constant channels, the largest values."""
    lens, Hkv, G, P = [96, 64], 2, 32, 64
    for bits in (2, 4):
        (k, v), cu = pack(lens, [Hkv, Hkv], "tokens", 14)
        for t in (k, v):
            t[0:32] = torch.randint(0, 4, t[0:32].shape, device="cuda").to(torch.float16) / 2
            t[32:64] = 1.5
            t[64:80] = -65504.0
            t[80:96] = 65504.0
            t[96:128, :, ::3] = -3.0e-5
            t[128:160, :, 1::2] = -60000.0
        a, b = (paged(2, Hkv, G, P, 2, 4, bits, False, 5) for _ in range(2))
        for c in (a, b):
            c.block_table.copy_(torch.tensor([[2, 0], [3, 1]], dtype=torch.int32))
        kivi.kivi_paged_prefill_packed(a, k, v, cu)
        kivi.kivi_paged_prefill(b, 0, k[:96].transpose(0, 1).contiguous(), v[:96].transpose(0, 1).contiguous())
        kivi.kivi_paged_prefill(b, 1, k[96:].transpose(0, 1).contiguous(), v[96:].transpose(0, 1).contiguous())
        for name in POOLS[:6]:
            assert torch.equal(getattr(a, name), getattr(b, name)), (bits, name)


def test_packed_quantizer_cuts_at_the_capacity_and_skips_missing_pages():
    lens, Hkv, G, P = [200, 100, 70], 1, 32, 64
    (k, v), cu = pack(lens, [Hkv, Hkv], "tokens", 15)
    a = paged(3, Hkv, G, P, 2, 6, 2, False, 6)
    b = paged(3, Hkv, G, P, 2, 6, 2, False, 6)
    table = torch.tensor([[4, 0], [-1, 2], [6, 5]], dtype=torch.int32)  # sequence 1: no first page; 2: 6 is no page
    a.block_table.copy_(table)
    b.block_table.copy_(table)
    kivi.kivi_paged_prefill_packed(a, k, v, cu)
    assert a.seq_lens.tolist() == [128, 100, 70]
    at = 0
    for s, n in enumerate(lens):
        m = min(n, 128)
        kivi.kivi_paged_prefill(b, s, k[at:at + m].transpose(0, 1).contiguous(), v[at:at + m].transpose(0, 1).contiguous())
        at += n
    for name in POOLS[:6]:
        assert torch.equal(getattr(a, name), getattr(b, name)), name

"""What the paged cache does for sliding-window attention: chunks appended (bit for bit what the
one-sequence and one-token calls write), tokens read back (the exact value rounded once), pages rolled
(against a plain model), and all of it together with both attentions."""
from __future__ import annotations

import math
import random

import numpy as np
import pytest
import torch

from bit_asymmetric_kv_gb300 import build as kbuild
from bit_asymmetric_kv_gb300 import kivi
from helpers import ATOL
from paged_values import D, filled, seen, tokens
from test_gpu_pages import Both
from test_gpu_window_attention import pack

pytestmark = pytest.mark.gpu
POOLS = ("k_codes", "k_meta", "v_codes", "v_meta")
SHAPES = [(32, 64, 2, False), (64, 128, 2, False), (32, 128, 4, False), (64, 64, 4, True), (32, 256, 2, True)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    kbuild.build()
    kivi.lib()


def same(a, b, dropped=()):
    """Where two caches differ ("" where they do not): pools bit for bit, lengths, residual slots in use (but
    those of sequences whose newest tokens were dropped)."""
    for name in POOLS:
        if not torch.equal(getattr(a, name), getattr(b, name)):
            return name
    if not torch.equal(a.seq_lens, b.seq_lens):
        return "seq_lens"
    for s, n in enumerate(a.seq_lens.tolist()):
        r = 0 if s in dropped else max(n, 0) % a.dims.G
        for name in ("k_res", "v_res"):
            x, y = getattr(a, name), getattr(b, name)
            if x is not None and not torch.equal(x[s, :, :r], y[s, :, :r]):
                return f"{name} of {s}"
    return ""


# ---------------------------------------------------------------------------- extend
def twins(span, B, Hkv, G, P, bits, v_res, seed):
    """Two empty caches of the same pages, `span` tokens for each of B sequences, and that many keys and values."""
    maxp, out = -(-span // P), []
    ids = torch.randperm(B * maxp + 2, generator=torch.Generator().manual_seed(seed))[:B * maxp]
    for _ in range(2):
        c = kivi.PagedCache.allocate(B, Hkv, G, P, maxp, B * maxp + 2, bits=bits, value_residual=v_res)
        for name in POOLS:
            getattr(c, name).fill_(-1)
        c.k_res.fill_(-30000.0)
        if v_res:
            c.v_res.fill_(-30000.0)
        c.block_table.copy_(ids.reshape(B, maxp))
        out.append(c)
    gen = torch.Generator().manual_seed(seed + 1)
    return out[0], out[1], [[torch.randn((Hkv, span, D), generator=gen).to(torch.float16).cuda() for _ in "kv"] for _ in range(B)]


OLD_NEW = [([0], [1]), ([1], [1]), ([31, 32, 33], [1, 1, 1]), ([0, 5, 63, 64], [130, 0, 1, 64]), ([40, 90, 10, 100], [24, 6, 54, 28]),
           ([17, 128, 77], [300, 1, 179]), ([95, 96, 97], [1, 32, 127]), ([60, 0, 33], [3, 0, 30])]


@pytest.mark.parametrize("old,new", OLD_NEW, ids=str)
@pytest.mark.parametrize("G,P,bits,v_res", SHAPES)
@pytest.mark.parametrize("layout", ["tokens", "heads", "gaps"])
def test_extend_is_the_whole_prompt(old, new, G, P, bits, v_res, layout):
    """Prompt and chunk give the cache of the whole prompt; rows of no sequence hold NaN."""
    Hkv = 3
    a, b, kv = twins(max(old) + max(new), len(old), Hkv, G, P, bits, v_res, 3)
    (k, v), cu = pack(new, [Hkv, Hkv], layout, 4, pad=70, lead=9)
    k[:, :, 7] *= 40
    for s, n in enumerate(old):
        ks, vs = (t[:, :n].contiguous() for t in kv[s])
        if n:
            kivi.kivi_paged_prefill(a, s, ks, vs)
        if n + new[s]:
            lo, hi = cu.tolist()[s], cu.tolist()[s + 1]
            kivi.kivi_paged_prefill(b, s, torch.cat([ks, k[lo:hi].transpose(0, 1)], 1).contiguous(),
                                    torch.cat([vs, v[lo:hi].transpose(0, 1)], 1).contiguous())
    kivi.kivi_paged_extend_packed(a, k, v, cu)
    assert same(a, b) == ""
    assert a.seq_lens.tolist() == [o + n for o, n in zip(old, new)]


@pytest.mark.parametrize("G,P,bits,v_res", SHAPES)
def test_extend_is_one_token_after_the_other(G, P, bits, v_res):
    B, Hkv, steps = 4, 2, 5
    old = [0, G - 3, 2 * G - 1, 100]
    a = filled(old, Hkv, G, P, bits, v_res, 5, room=steps)
    b = filled(old, Hkv, G, P, bits, v_res, 5, room=steps)
    (k, v), cu = pack([steps] * B, [Hkv, Hkv], "tokens", 6)
    kivi.kivi_paged_extend_packed(a, k, v, cu)
    for i in range(steps):
        kivi.kivi_paged_append_token(b, k[i::steps].contiguous(), v[i::steps].contiguous())
    assert same(a, b) == ""


@pytest.mark.parametrize("seed", range(6))
def test_extend_in_random_chunks(seed):
    rng = random.Random(seed)
    G, P, bits, v_res = SHAPES[seed % len(SHAPES)]
    B, Hkv, most = 5, 2, 400
    a, b, kv = twins(most, B, Hkv, G, P, bits, v_res, seed)
    at = [0] * B
    for _ in range(6):
        new = [min(most - n, rng.choice([0, 1, 2, G, G - 1, rng.randrange(90)])) for n in at]
        cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
        if sum(new):
            k, v = (torch.cat([kv[s][i][:, at[s]:at[s] + new[s]] for s in range(B)], 1).transpose(0, 1) for i in range(2))
            kivi.kivi_paged_extend_packed(a, k, v, cu)
        at = [x + y for x, y in zip(at, new)]
    for s, n in enumerate(at):
        kivi.kivi_paged_prefill(b, s, kv[s][0][:, :n].contiguous(), kv[s][1][:, :n].contiguous())
    assert same(a, b) == ""


def test_extend_many_sequences():
    rng = random.Random(9)
    old = [rng.choice([0, 0, 1, 31, 60, 64, 90]) for _ in range(512)]
    new = [rng.choice([0, 1, 1, 2, 7, 40, 128]) for _ in range(512)]
    a, b, kv = twins(218, 512, 1, 32, 64, 2, False, 10)
    (k, v), cu = pack(new, [1, 1], "tokens", 11)
    pre = torch.tensor([0] + list(np.cumsum(old)), dtype=torch.int32, device="cuda")
    kivi.kivi_paged_prefill_packed(a, *(torch.cat([kv[s][i][:, :n] for s, n in enumerate(old)], 1).transpose(0, 1) for i in range(2)), pre)
    kivi.kivi_paged_extend_packed(a, k, v, cu)
    bounds = cu.tolist()
    whole = [torch.cat([torch.cat([kv[s][i][:, :old[s]], (k, v)[i][bounds[s]:bounds[s + 1]].transpose(0, 1)], 1)
                        for s in range(512)], 1).transpose(0, 1) for i in range(2)]
    both = torch.tensor([0] + list(np.cumsum([o + n for o, n in zip(old, new)])), dtype=torch.int32, device="cuda")
    kivi.kivi_paged_prefill_packed(b, *whole, both)
    assert same(a, b) == ""


def test_extend_stops_at_the_capacity_and_skips_missing_pages():
    G, P = 32, 64
    old, new = [100, 128, 30, -7, 50], [60, 5, 90, 40, 0]
    a = filled([100, 128, 30, 0, 50], 1, G, P, 2, False, 12, room=0)
    b = filled([100, 128, 30, 0, 50], 1, G, P, 2, False, 12, room=0)
    spare = [p for p in range(a.dims.num_pages) if p not in a.block_table.flatten().tolist()]
    for c in (a, b):
        assert c.dims.max_pages_per_seq == 2
        c.block_table[2, 1] = 2**31 - 1      # no page: its tokens are dropped, and count
        c.block_table[3, 0] = spare[0]
        c.seq_lens[3] = -7                   # clamped to 0
        c.seq_lens[4] = 50
    (k, v), cu = pack(new, [1, 1], "tokens", 13)
    kivi.kivi_paged_extend_packed(a, k, v, cu)
    assert a.seq_lens.tolist() == [128, 128, 120, 40, 50]
    b.seq_lens[3] = 0
    for i in range(max(new)):
        for s, (n, m) in enumerate(zip(old, new)):
            if i >= m:
                continue
            one = torch.zeros((5, 1, D), dtype=torch.float16, device="cuda")
            vv = one.clone()
            one[s], vv[s] = k[cu.tolist()[s] + i], v[cu.tolist()[s] + i]
            keep = b.seq_lens.clone(), b.k_res.clone(), [getattr(b, x).clone() for x in POOLS]
            kivi.kivi_paged_append_token(b, one, vv)
            for o in range(5):  # the other sequences as they were
                if o != s:
                    b.seq_lens[o], b.k_res[o] = keep[0][o], keep[1][o]
                    pages = [p for p in b.block_table[o].tolist() if 0 <= p < b.dims.num_pages]
                    for x, was in zip(POOLS, keep[2]):
                        getattr(b, x)[pages] = was[pages]
    b.seq_lens[2] = 120
    assert same(a, b, dropped=[2]) == ""


def test_extend_leaves_sequences_without_rows_as_they_are():
    a = filled([70, 40], 2, 32, 64, 2, True, 14, room=100)
    a.seq_lens[0] = -3
    was = [getattr(a, x).clone() for x in POOLS + ("k_res", "v_res", "seq_lens")]
    (k, v), cu = pack([0, 0], [2, 2], "tokens", 15, pad=90, lead=3)
    kivi.kivi_paged_extend_packed(a, k, v, cu)
    assert all(torch.equal(x, getattr(a, n)) for x, n in zip(was, POOLS + ("k_res", "v_res", "seq_lens")))


def test_extend_adversarial_values():
    """Ties, thresholds next to zero, constant channels, the largest values, over the residual's border."""
    old, new, Hkv, G, P = [20, 50], [96, 64], 2, 32, 64
    for bits in (2, 4):
        a, b, kv = twins(150, 2, Hkv, G, P, bits, False, 16)
        (k, v), cu = pack(new, [Hkv, Hkv], "tokens", 17)
        for t in (k, v):
            t[0:32] = torch.randint(0, 4, t[0:32].shape, device="cuda").to(torch.float16) / 2
            t[32:64] = 1.5
            t[64:80] = -65504.0
            t[80:96] = 65504.0
            t[96:128, :, ::3] = -3.0e-5
            t[128:160, :, 1::2] = -60000.0
        for s, n in enumerate(old):
            ks, vs = (t[:, :n].contiguous() for t in kv[s])
            lo, hi = cu.tolist()[s], cu.tolist()[s + 1]
            kivi.kivi_paged_prefill(a, s, ks, vs)
            kivi.kivi_paged_prefill(b, s, torch.cat([ks, k[lo:hi].transpose(0, 1)], 1).contiguous(),
                                    torch.cat([vs, v[lo:hi].transpose(0, 1)], 1).contiguous())
        kivi.kivi_paged_extend_packed(a, k, v, cu)
        assert same(a, b) == "", bits


def test_extend_in_a_graph_and_on_streams():
    old, steps = [10, 31, 64], 3
    a = filled(old, 2, 32, 64, 2, False, 18, room=60)
    b = filled(old, 2, 32, 64, 2, False, 18, room=60)
    (k, v), cu = pack([7, 1, 12], [2, 2], "tokens", 19)
    kivi.kivi_paged_extend_packed(a, k, v, cu)
    kivi.kivi_paged_extend_packed(b, k, v, cu)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kivi.kivi_paged_extend_packed(a, k, v, cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(steps):
        g.replay()
        kivi.kivi_paged_extend_packed(b, k, v, cu, stream=side)
    torch.cuda.synchronize()
    assert same(a, b) == "" and a.seq_lens.tolist() == [o + 4 * n for o, n in zip(old, [7, 1, 12])]


# ------------------------------------------------------------------------------ read
def rounded(x):
    """fp16 of values in 64 bits, rounded once, at most the largest."""
    return np.clip(x.cpu().numpy(), -65504, 65504).astype(np.float16)


def check_read(c, cu, take, first, k, v, fill):
    """Rows as they must be, and the others as they were."""
    bounds = cu.tolist()
    lens = [min(max(n, 0), c.dims.max_pages_per_seq * c.dims.page_tokens) for n in c.seq_lens.tolist()]
    want = [np.full(tuple(t.shape), fill, np.float16) for t in (k, v)]
    for b, n in enumerate(lens):
        room = bounds[b + 1] - bounds[b]
        m = min(room, n, room if take is None else max(take[b], 0))
        if m <= 0:
            continue
        f = min(first, m)
        p = list(range(f)) + list(range(n - (m - f), n))
        for w, t in zip(want, tokens(c, b, p)):
            t = rounded(t)
            for i, pos in enumerate(p):  # a position without a page reads as zeros, but for what is in the residual
                page = int(c.block_table[b, pos // c.dims.page_tokens])
                late = pos >= n // c.dims.G * c.dims.G
                if not 0 <= page < c.dims.num_pages and not (late and (w is want[0] or c.v_res is not None)):
                    t[i] = 0
            w[bounds[b]:bounds[b] + m] = t
    for name, w, t in zip("kv", want, (k, v)):
        got = t.cpu().numpy()
        bad = np.argwhere(got != w)
        assert len(bad) == 0, (name, len(bad), bad[:4].tolist(), got[tuple(bad[0])], w[tuple(bad[0])])


def outputs(T, Hkv, layout, fill=7.0):
    out = []
    for _ in "kv":
        if layout == "tokens":
            t = torch.full((T, Hkv, D), fill, dtype=torch.float16, device="cuda")
        elif layout == "heads":
            t = torch.full((Hkv, T, D), fill, dtype=torch.float16, device="cuda").transpose(0, 1)
        else:
            t = torch.full((T, Hkv + 1, D + 24), fill, dtype=torch.float16, device="cuda")[:, :Hkv, 8:8 + D]
        out.append(t)
    return out


@pytest.mark.parametrize("G,P,bits,v_res", SHAPES)
@pytest.mark.parametrize("first", [0, 1, 4, 33, 1000])
@pytest.mark.parametrize("layout", ["tokens", "heads", "gaps"])
def test_read_lengths(G, P, bits, v_res, first, layout):
    lens = [1, 0, 31, 32, 33, 64, 127, 200, 333, 640]
    c = filled(lens, 2, G, P, bits, v_res, 20)
    rooms = [5, 3, 31, 40, 20, 64, 100, 150, 400, 90]
    take = [9, 2, 31, 0, 20, -4, 99, 77, 400, 65]
    cu = torch.tensor([4] + [4 + x for x in np.cumsum(rooms)], dtype=torch.int32, device="cuda")
    for t in (None, take):
        k, v = outputs(4 + sum(rooms) + 6, 2, layout)
        dev = None if t is None else torch.tensor(t, dtype=torch.int32, device="cuda")
        kivi.kivi_paged_read(c, cu, dev, k, v, first=first)
        check_read(c, cu, t, first, k, v, 7.0)


def test_read_missing_pages_and_lengths_that_make_no_sense():
    c = filled([300, 64, 200, 128], 2, 32, 64, 2, False, 21)
    c.block_table[0, 1], c.block_table[0, 4], c.block_table[2, 3] = -1, 2**31 - 1, -2**31
    c.seq_lens[1], c.seq_lens[3] = -9, 2**31 - 1   # clamped: nothing, and the capacity (pages of nothing behind)
    cu = torch.tensor([0, 300, 340, 560, 700], dtype=torch.int32, device="cuda")
    k, v = outputs(700, 2, "tokens")
    kivi.kivi_paged_read(c, cu, None, k, v, first=70)
    check_read(c, cu, None, 70, k, v, 7.0)


def test_read_rounds_once_and_stays_finite():
    """Scales and zeros of any size: ties between fp16 values that a rounding to fp32 first would move, sums
    beyond the largest fp16, subnormals."""
    for bits in (2, 4):
        c = filled([64 * 40], 2, 32, 64, bits, False, 22)
        gen = torch.Generator(device="cuda").manual_seed(23)
        for m in (c.k_meta, c.v_meta):
            s = torch.randint(0, 0x7c00, m.shape, generator=gen, device="cuda")       # finite, positive
            z = torch.randint(0, 0x7c00, m.shape, generator=gen, device="cuda") | (torch.randint(0, 2, m.shape, generator=gen, device="cuda") << 15)
            w = s | z << 16
            m.copy_(torch.where(w >= 2**31, w - 2**32, w))
        for t in (c.k_codes, c.v_codes):
            t.copy_(torch.randint(-2**31, 2**31 - 1, t.shape, dtype=torch.int32, device="cuda", generator=gen))
        cu = torch.tensor([0, 2560], dtype=torch.int32, device="cuda")
        k, v = outputs(2560, 2, "tokens")
        kivi.kivi_paged_read(c, cu, None, k, v)
        assert torch.isfinite(k).all() and torch.isfinite(v).all()
        check_read(c, cu, None, 0, k, v, 7.0)


def test_read_many_sequences_and_overlapping_bounds():
    rng = random.Random(24)
    lens = [rng.randrange(0, 150) for _ in range(512)]
    c = filled(lens, 1, 32, 64, 4, False, 25)
    take = [rng.randrange(0, 150) for _ in range(512)]
    cu = torch.tensor([0] + list(np.cumsum([t + 3 for t in take])), dtype=torch.int32, device="cuda")
    k, v = outputs(int(cu[-1]), 1, "tokens")
    kivi.kivi_paged_read(c, cu, torch.tensor(take, dtype=torch.int32, device="cuda"), k, v, first=5)
    check_read(c, cu, take, 5, k, v, 7.0)
    big = torch.full((400, 1, D), 3.0, dtype=torch.float16, device="cuda")
    k, v = big[100:200], big[250:350]
    nonsense = torch.tensor([rng.choice([-5, 0, 50, 2**31 - 1]) for _ in range(513)], dtype=torch.int32, device="cuda")
    kivi.kivi_paged_read(c, nonsense, None, k, v, first=5)  # unspecified rows, none outside
    torch.cuda.synchronize()
    assert (big[:100] == 3).all() and (big[200:250] == 3).all() and (big[350:] == 3).all()


def test_read_in_a_graph_follows_the_lengths():
    c = filled([100, 40], 2, 32, 64, 2, False, 26, room=64)
    (kn, vn), one = pack([20, 1], [2, 2], "tokens", 27)
    cu = torch.tensor([0, 70, 130], dtype=torch.int32, device="cuda")
    k, v = outputs(130, 2, "tokens")
    kivi.kivi_paged_read(c, cu, None, k, v, first=4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kivi.kivi_paged_read(c, cu, None, k, v, first=4)
    for _ in range(3):
        kivi.kivi_paged_extend_packed(c, kn, vn, one)
        k.fill_(7), v.fill_(7)
        g.replay()
        check_read(c, cu, None, 4, k, v, 7.0)


def test_read_and_extend_offsets_past_32_bits():
    """Pages whose code words lie past element 2^31, and rows whose elements do."""
    Hkv, P = 8, 64
    num = 2**31 // (Hkv * P * 8) + 20
    small = filled([150, 70], Hkv, 32, P, 2, False, 28, room=64)
    c = kivi.PagedCache.allocate(2, Hkv, 32, P, small.dims.max_pages_per_seq, num)
    shift = num - small.dims.num_pages
    for name in POOLS:
        getattr(c, name)[shift:] = getattr(small, name)
    c.k_res.copy_(small.k_res)
    c.seq_lens.copy_(small.seq_lens)
    c.block_table.copy_(torch.where(small.block_table >= 0, small.block_table + shift, -1))
    far = 2**31 // (Hkv * D) + 5
    buf = torch.empty((far + 400, Hkv, D), dtype=torch.float16, device="cuda")
    buf[far:] = torch.randn((400, Hkv, D), device="cuda").to(torch.float16)
    kn, vn = buf, buf
    cu = torch.tensor([far, far + 40, far + 100], dtype=torch.int32, device="cuda")
    kivi.kivi_paged_extend_packed(c, kn, vn, cu)
    near = torch.tensor([0, 40, 100], dtype=torch.int32, device="cuda")
    kivi.kivi_paged_extend_packed(small, buf[far:far + 100], buf[far:far + 100], near)
    for name in POOLS:
        assert torch.equal(getattr(c, name)[shift:], getattr(small, name)), name
    out = torch.tensor([far, far + 190, far + 320], dtype=torch.int32, device="cuda")
    other = torch.empty_like(buf)
    kivi.kivi_paged_read(c, out, None, buf, other)
    k, v = outputs(320, Hkv, "tokens")
    kivi.kivi_paged_read(small, torch.tensor([0, 190, 320], dtype=torch.int32, device="cuda"), None, k, v)
    assert torch.equal(buf[far:far + 190], k[:190]) and torch.equal(other[far + 190:far + 320], v[190:])


# --------------------------------------------------------------------------- reserve
class Windows(Both):
    def reserve_window(self, extra, window, sinks):
        kivi.kivi_paged_reserve_window(self.c, self.pool, torch.tensor(extra, dtype=torch.int32, device="cuda"), window, sinks)
        m, P = self.m, self.m.P
        before = m._in_use()
        wanted = []
        for b, e in enumerate(extra):
            if e <= 0:
                continue
            n = min(max(m.lens[b], 0), m.max_pages * P)
            for j in range(m.max_pages):
                unseen = j * P >= sinks and (j + 1) * P <= n - window + 1
                if unseen:
                    if m._held(m.rows[b][j]):
                        m.refs[m.rows[b][j]] -= 1
                    m.rows[b][j] = -1
                elif j * P < min(max(m.lens[b], 0) + e, m.max_pages * P) and not m._held(m.rows[b][j]):
                    wanted.append((b, j))
        given = before - m._in_use()
        free = m._free()
        for i, (b, j) in enumerate(wanted):
            m.rows[b][j] = free[i] if i < len(free) else -1
            if i < len(free):
                m.refs[free[i]] = 1
        got = min(len(wanted), len(free))
        m.info = [got, len(wanted) - got, m._in_use(), given]
        self.same()


def test_reserve_window_by_hand():
    t = Windows(3, 8, 12, 64)
    t.reserve([500, 0, 64])
    t.m.lens = [450, 0, 64]
    t.put()
    t.reserve_window([1, 5, 1], 100, 4)      # sequence 0: pages 1 .. 4 go (positions 64 .. 319), 0 holds the sinks
    assert t.m.rows[0][1:5] == [-1] * 4 and t.m.rows[0][0] >= 0 and t.m.info[3] == 4
    t.reserve_window([1, 5, 1], 100, 4)      # nothing changes
    t.reserve_window([0, -1, 0], 1, 0)       # nor without tokens to come
    t.reserve_window([1, 1, 1], 1, 0)        # the newest token alone, no sinks
    t.reserve_window([2**31 - 1, 1, 1], 2**31 - 1, 2**31 - 1)  # everything is seen: holes are filled


@pytest.mark.parametrize("B,maxp,num,P", [(1, 1, 1, 64), (1, 2048, 2100, 64), (7, 33, 200, 128), (512, 5, 2000, 64),
                                          (40, 130, 40000, 64), (511, 3, 100, 64), (9, 2, 4096, 1024)])
def test_reserve_window_sizes(B, maxp, num, P):
    rng = random.Random(B + num)
    t = Windows(B, maxp, num, P, Hkv=1, G=64)
    t.m.refs = [rng.choice([0, 0, 1]) if num > 1 else 0 for _ in range(num)]
    t.put()
    for _ in range(4):
        t.reserve_window([rng.choice([0, 1, P, rng.randrange(maxp * P + 1)]) for _ in range(B)],
                         rng.choice([1, P, 2 * P - 1, rng.randrange(1, maxp * P + 5)]), rng.choice([0, 1, 4, P, 3 * P + 1]))
        t.m.lens = [rng.choice([-3, rng.randrange(maxp * P + 1), maxp * P + 7]) for _ in range(B)]
        t.put()


def test_reserve_window_with_shared_pages_forks_and_compaction():
    rng = random.Random(30)
    t = Windows(8, 10, 60, 64, Hkv=2, G=32)
    for step in range(14):
        t.reserve_window([rng.choice([0, 1, 64, 150]) for _ in range(8)], rng.choice([100, 200]), 4)
        for b in range(8):
            n = t.m.lens[b]
            while n < 640 and t.m.rows[b][n // 64] >= 0 and n < t.m.lens[b] + 90:
                n += 1
            t.m.lens[b] = n
        t.c.seq_lens.copy_(torch.tensor(t.m.lens, dtype=torch.int32))
        if step % 3 == 1:
            t.reorder([rng.choice([b, b, rng.randrange(-1, 8)]) for b in range(8)])
        elif step % 3 == 2:
            t.compact()


def test_reserve_window_in_a_graph():
    t = Windows(4, 6, 30, 64)
    extra = torch.tensor([1, 70, 0, 200], dtype=torch.int32, device="cuda")
    kivi.kivi_paged_reserve_window(t.c, t.pool, extra, 80, 4)
    t.m.lens = [0] * 4
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kivi.kivi_paged_reserve_window(t.c, t.pool, extra, 80, 4)
    for lens in ([10, 64, 5, 300], [200, 380, 5, 100]):
        rows, refs = t.c.block_table.tolist(), t.c.block_table.clone()
        t.m.rows, t.m.refs, t.m.lens = rows, t.pool.ref_counts.tolist(), lens
        t.c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        after = t.c.block_table.clone(), t.pool.ref_counts.clone()
        t.c.block_table.copy_(refs)
        t.pool.ref_counts.copy_(torch.tensor(t.m.refs, dtype=torch.int32))
        t.reserve_window(extra.tolist(), 80, 4)
        assert torch.equal(after[0], t.c.block_table) and torch.equal(after[1], t.pool.ref_counts)


# ------------------------------------------------------------------------ all of them
@pytest.mark.parametrize("G,P,bits,v_res", SHAPES)
@pytest.mark.parametrize("window,sinks", [(130, 4), (64, 0), (300, 70)])
def test_chunks_and_steps_of_a_rolling_cache(G, P, bits, v_res, window, sinks):
    """Prompts in chunks (pages rolled, what the chunk sees read back beside its own keys, attention, append), then
    steps, from a pool too small for the whole sequences.  Reference: the formula in 64 bits over what the
    cache holds.  Tolerances: test_gpu_window_attention.py's shape for chunks (a rounding to fp16 of the read
    rows, 2^-11 of a key's and a value's elements, comes on top), 2e-3 for steps."""
    B, Hkv, R, scale = 3, 2, 2, 1 / math.sqrt(D)
    total, chunk, steps = [500, 260, 700], 110, 70
    maxp = -(-(max(total) + steps) // P)
    num = B * (-(-(window + chunk) // P) + 2 + -(-sinks // P))
    c = kivi.PagedCache.allocate(B, Hkv, G, P, maxp, num, bits=bits, value_residual=v_res)
    pool = kivi.PagePool.allocate(c)
    gen = torch.Generator().manual_seed(31)
    q, k, v = ([torch.randn((n, h, D), generator=gen).to(torch.float16).cuda() for n in total] for h in (Hkv * R, Hkv, Hkv))
    done = [0] * B
    while any(d < n for d, n in zip(done, total)):
        new = [min(chunk, n - d) for d, n in zip(done, total)]
        old = [min(d, window - 1 + sinks) if n else 0 for d, n in zip(done, new)]
        extra = torch.tensor(new, dtype=torch.int32, device="cuda")
        kivi.kivi_paged_reserve_window(c, pool, extra, window, sinks)
        assert pool.info.tolist()[1] == 0
        cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
        cu_kv = torch.tensor([0] + list(np.cumsum([n + o for n, o in zip(new, old)])), dtype=torch.int32, device="cuda")
        ks, vs = (torch.full((int(cu_kv[-1]), Hkv, D), math.nan, dtype=torch.float16, device="cuda") for _ in "kv")
        kivi.kivi_paged_read(c, cu_kv, torch.tensor(old, dtype=torch.int32, device="cuda"), ks, vs, first=sinks)
        for b in range(B):
            at = int(cu_kv[b + 1])
            ks[at - new[b]:at], vs[at - new[b]:at] = (t[b][done[b]:done[b] + new[b]] for t in (k, v))
        qs = torch.cat([q[b][done[b]:done[b] + new[b]] for b in range(B)])
        out = kivi.kivi_prefill_attention_window(qs, ks, vs, cu, window, sinks, scale, cu_seqlens_kv=cu_kv)
        for b in range(B):
            if not new[b]:
                continue
            d, n = done[b], new[b]
            p = [t for t in range(d) if t < sinks or t > d - window]
            kk, vv = (torch.cat([x, y[b][d:d + n].double()]) for x, y in zip(tokens(c, b, p), (k, v)))
            pos = torch.tensor(p + list(range(d, d + n)), device="cuda")
            i = torch.arange(d, d + n, device="cuda")[:, None]
            vis = (pos <= i) & ((pos > i - window) | (pos < sinks))
            for h in range(Hkv * R):
                Q = q[b][d:d + n, h].double()
                x = (Q @ kk[:, h // R].t() * scale).masked_fill(~vis, -math.inf)
                w = torch.softmax(x, -1)
                ref, A = w @ vv[:, h // R], w @ vv[:, h // R].abs()
                mag = (Q.abs() @ kk[:, h // R].abs().t() * scale).amax(-1, keepdim=True)
                e = 2.0**-11 * mag + 132 * 2.0**-23 * mag            # the read keys' rounding, the scores'
                tol = 2.0**-11 * ref.abs() + 2.0**-25 + (2 * 2.0**-11 + 2 * e + 60 * 2.0**-22) * A + 2.0**-24 * 500 * 6
                err = (out[int(cu[b]):int(cu[b]) + n, h].double() - ref).abs()
                assert (err <= tol * 1.01).all(), (b, h, float((err - tol).max()))
        kivi.kivi_paged_extend_packed(c, torch.cat([k[b][done[b]:done[b] + new[b]] for b in range(B)]),
                                      torch.cat([v[b][done[b]:done[b] + new[b]] for b in range(B)]), cu)
        done = [d + n for d, n in zip(done, new)]
    assert c.seq_lens.tolist() == total
    one = torch.ones(B, dtype=torch.int32, device="cuda")
    for step in range(steps):
        kivi.kivi_paged_reserve_window(c, pool, one, window, sinks)
        kn, vn, qn = (torch.randn((B, h, D), generator=gen).to(torch.float16).cuda() for h in (Hkv, Hkv, Hkv * R))
        out = kivi.kivi_paged_decode_step_window(c, kn, vn, qn, window, sinks, scale)
        if step % 7:
            continue
        for b, n in enumerate(c.seq_lens.tolist()):
            kk, vv = tokens(c, b, seen(n, window, sinks))
            for h in range(Hkv * R):
                w = torch.softmax(kk[:, h // R] @ qn[b, h].double() * scale, 0)
                assert (out[b, h].double() - w @ vv[:, h // R]).abs().max() <= ATOL
    assert pool.info.tolist()[1] == 0 and c.seq_lens.tolist() == [n + steps for n in total]

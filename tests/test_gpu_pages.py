"""Pages handed out, shared, copied, given back and moved on the GPU: every table entry, count,
length and info value against the plain model, and the tokens of every sequence bit for bit."""
from __future__ import annotations

import math
import random

import numpy as np
import pytest
import torch

import oracle
from bit_asymmetric_kv_gb300 import build as kbuild
from bit_asymmetric_kv_gb300 import kivi
from helpers import assert_close
from page_model import Pages

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    kbuild.build()
    kivi.lib()


class Both:
    """A paged cache on the GPU beside the model, pool contents tracked on the host."""

    def __init__(self, B, maxp, num, P, Hkv=2, G=32, bits=2, v_res=False, seed=0):
        self.c = kivi.PagedCache.allocate(B, Hkv, G, P, maxp, num, bits=bits, value_residual=v_res)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for name in ("k_codes", "k_meta", "v_codes", "v_meta"):
            t = getattr(self.c, name)
            t.copy_(torch.randint(-2**31, 2**31 - 1, t.shape, dtype=torch.int32, device="cuda", generator=gen))
        self.c.k_res.normal_(generator=gen)
        if v_res:
            self.c.v_res.normal_(generator=gen)
        self.pool = kivi.PagePool.allocate(self.c)
        self.m = Pages(B, maxp, num, P)
        self.G = G

    def put(self):
        """The model's state into the cache (after a test changed it by hand)."""
        self.c.block_table.copy_(torch.tensor(self.m.rows, dtype=torch.int32))
        self.pool.ref_counts.copy_(torch.tensor(self.m.refs, dtype=torch.int32))
        self.c.seq_lens.copy_(torch.tensor(self.m.lens, dtype=torch.int32))

    def same(self):
        assert self.c.block_table.tolist() == self.m.rows
        assert self.pool.ref_counts.tolist() == self.m.refs
        assert self.c.seq_lens.tolist() == self.m.lens
        assert self.pool.info.tolist() == self.m.info

    def grab(self):
        c = self.c
        return [t.cpu().numpy().copy() for t in (c.k_codes, c.k_meta, c.v_codes, c.v_meta)] + [
            c.k_res.cpu().numpy().view(np.uint16).copy(),
            None if c.v_res is None else c.v_res.cpu().numpy().view(np.uint16).copy()]

    def reserve(self, extra):
        kivi.kivi_paged_reserve(self.c, self.pool, torch.tensor(extra, dtype=torch.int32, device="cuda"))
        self.m.reserve(extra)
        self.same()

    def reorder(self, parent):
        kc, km, vc, vm, kr, vr = self.grab()
        old_kr, old_vr = kr.copy(), None if vr is None else vr.copy()
        kivi.kivi_paged_reorder(self.c, self.pool, torch.tensor(parent, dtype=torch.int32, device="cuda"))
        P, G = self.m.P, self.G
        for b, s, f, t in self.m.reorder(parent):
            n = self.m.lens[b]
            if t >= 0:
                r = n % P
                rg = r // G * G
                rv = r if vr is None else rg
                kc[t, :, :rg], km[t, :, :rg // G] = kc[f, :, :rg], km[f, :, :rg // G]
                vc[t, :, :rv], vm[t, :, :rv] = vc[f, :, :rv], vm[f, :, :rv]
            kr[b, :, :n % G] = old_kr[s, :, :n % G]
            if vr is not None:
                vr[b, :, :n % G] = old_vr[s, :, :n % G]
        self.same()
        self.contents(kc, km, vc, vm, kr, vr)

    def compact(self):
        kc, km, vc, vm, kr, vr = self.grab()
        got = kivi.kivi_paged_compact(self.c, self.pool)
        new = self.m.compact()
        assert got.tolist() == new
        for old, to in enumerate(new):
            if to >= 0 and to != old:
                kc[to], km[to], vc[to], vm[to] = kc[old], km[old], vc[old], vm[old]
        self.same()
        self.contents(kc, km, vc, vm, kr, vr)

    def contents(self, *want):
        for name, a, b in zip(("k_codes", "k_meta", "v_codes", "v_meta", "k_res", "v_res"), self.grab(), want):
            assert (a is None and b is None) or np.array_equal(a, b), name


def test_reserve_by_hand():
    t = Both(3, 4, 8, 64)
    t.reserve([200, 0, 64])
    t.reserve([200, 0, 64])       # everything is there already
    t.m.lens = [190, 0, 64]
    t.put()
    t.reserve([2, 1, 1])          # 192 tokens fit; a first page; position 64 needs a second one
    t.reserve([-5, 1000, 0])      # more than the capacity, and than the pool
    assert t.m.info == [1, 2, 8, 0]


def test_reserve_fills_holes_and_unusable_entries():
    t = Both(2, 4, 12, 64)
    t.m.rows = [[3, -1, 12, 7], [-2, 2**31 - 1, -2**31, 5]]
    t.m.refs = [0, 0, 0, 1, 0, 1, 0, 1, 0, -3, 0, 0]
    t.m.lens = [1, -7]
    t.put()
    t.reserve([250, 129])


@pytest.mark.parametrize("B,maxp,num,P", [(1, 1, 1, 64), (1, 2048, 2100, 64), (7, 33, 200, 128), (512, 5, 2000, 64),
                                          (40, 130, 40000, 64), (511, 3, 100, 64), (9, 2, 4096, 1024)])
def test_reserve_sizes(B, maxp, num, P):
    rng = random.Random(B + num)
    t = Both(B, maxp, num, P, Hkv=1, G=64)
    t.m.refs = [rng.choice([0, 0, 1]) if num > 1 else 0 for _ in range(num)]
    t.put()
    for _ in range(3):
        t.reserve([rng.choice([0, 1, P, rng.randrange(maxp * P + 1)]) for _ in range(B)])
        t.m.lens = [rng.randrange(maxp * P + 1) for _ in range(B)]
        t.put()


CASES = {
    "fork": [0, 0, 2, 3, 2], "free": [0, -1, 2, 3, -1], "swap": [1, 0, 2, 3, 4], "cycle": [4, 0, 1, 2, 3],
    "broadcast": [2, 2, 2, 2, 2], "chain": [1, 2, 3, 4, 4], "beam": [0, 0, 3, 3, 3], "nothing": [0, 1, 2, 3, 4],
    "all-free": [-1] * 5, "outside": [5, -7, 2**31 - 1, 3, -2**31], "moved": [-1, 0, 0, 1, -1],
}


@pytest.mark.parametrize("parent", list(CASES.values()), ids=list(CASES))
@pytest.mark.parametrize("v_res,bits,G,P", [(False, 2, 32, 64), (True, 4, 64, 128), (True, 2, 32, 64), (False, 4, 64, 64)])
def test_reorder_cases(parent, v_res, bits, G, P):
    t = Both(5, 4, 24, P, G=G, bits=bits, v_res=v_res)
    t.reserve([3 * P + 1, P, 2 * P + 40, 10, 1])
    t.m.lens = [3 * P, P - 1, 2 * P + 37, 10, 0]
    t.put()
    t.reorder(parent)
    t.reorder(parent)


@pytest.mark.parametrize("seed", range(8))
def test_random_calls(seed):
    rng = random.Random(100 + seed)
    B, P, maxp, Hkv = rng.choice([(6, 64, 4, 2), (20, 64, 3, 1), (3, 128, 6, 3)])
    t = Both(B, maxp, rng.choice([B * maxp, B * maxp // 2 + 1]), P, Hkv=Hkv, G=rng.choice([32, 64]),
             bits=rng.choice([2, 4]), v_res=rng.random() < 0.5, seed=seed)
    for _ in range(25):
        op = rng.randrange(3)
        if op == 0:
            t.reserve([rng.choice([0, 1, 30, 200]) for _ in range(B)])
            for b in range(B):
                held = next((j for j, x in enumerate(t.m.rows[b]) if x < 0), maxp) * P
                t.m.lens[b] = max(t.m.lens[b], rng.randrange(t.m.lens[b], held + 1) if held >= t.m.lens[b] else 0)
            t.c.seq_lens.copy_(torch.tensor(t.m.lens, dtype=torch.int32))
        elif op == 1:
            t.reorder([rng.choice([b, b, rng.randrange(-1, B)]) for b in range(B)])
        else:
            t.compact()


def test_reorder_large_batch():
    rng = random.Random(5)
    t = Both(512, 6, 4000, 64, Hkv=1, G=32)
    lens = [rng.randrange(0, 6 * 64 + 1) for _ in range(512)]
    t.reserve(lens)
    t.m.lens = lens
    t.put()
    t.reorder([rng.choice([b, rng.randrange(512), -1]) for b in range(512)])


def test_reorder_without_free_pages():
    """The copies that get no page end before their partly filled one; the lowest copies are served first."""
    t = Both(4, 2, 3, 64)
    t.reserve([100, 0, 0, 0])
    t.m.lens = [100, 0, 0, 0]
    t.put()
    t.reorder([0, 0, 0, 0])
    assert t.m.lens == [100, 100, 64, 64] and t.m.info == [1, 2, 3, 0]


def test_counts_of_pages_held_outside_the_table():
    """A caller's own reference keeps a page when the last sequence lets it go."""
    t = Both(2, 2, 4, 64)
    t.reserve([128, 0])
    t.m.lens = [128, 0]
    t.m.refs[1] += 1
    t.put()
    t.reorder([-1, 1])
    assert t.m.refs == [0, 1, 0, 0]
    t.compact()


@pytest.mark.parametrize("num,live", [(1, 0), (1, 1), (5, 2), (4096, 2000), (4097, 1), (4097, 4096), (33000, 12345)])
def test_compact_sizes(num, live):
    rng = random.Random(num + live)
    t = Both(4, max(1, min(num, 9000)), num, 64, Hkv=1, G=64)
    ids = rng.sample(range(num), live)
    for i, page in enumerate(ids):
        t.m.refs[page] = 1
        if i < 4 * t.m.max_pages:
            t.m.rows[i % 4][i // 4] = page
    if num > live:  # an entry of a page that is not in use
        dead = rng.choice([i for i in range(num) if t.m.refs[i] == 0])
        t.m.rows[3][-1], t.m.refs[dead] = dead, -2
    t.put()
    t.compact()
    if num > live:
        assert t.c.block_table[3, -1] == -1


def test_pool_offsets_past_32_bits():
    """Pages whose word offset passes 2^31, forked and moved."""
    num, Hkv, P, G = 140000, 32, 64, 32
    assert num * Hkv * P * 8 > 2**31
    c = kivi.PagedCache.allocate(2, Hkv, G, P, 2, num)
    pools = (c.k_codes, c.k_meta, c.v_codes, c.v_meta)
    for t in pools:
        t[num - 3:] = torch.randint(-2**31, 2**31 - 1, t[num - 3:].shape, dtype=torch.int32, device="cuda")
    refs = torch.ones(num, dtype=torch.int32, device="cuda")
    refs[num - 1] = 0
    refs[7:num - 3] = 0
    c.block_table.copy_(torch.tensor([[num - 2, num - 3], [-1, -1]], dtype=torch.int32))
    c.seq_lens.copy_(torch.tensor([100, 0], dtype=torch.int32))
    pool = kivi.PagePool.adopt(c, refs)
    refs[7:num - 3] = 1  # only the last page is free
    kivi.kivi_paged_reorder(c, pool, torch.tensor([0, 0], dtype=torch.int32, device="cuda"))
    assert c.block_table.tolist() == [[num - 2, num - 3], [num - 2, num - 1]]
    for t, used in zip(pools, (32, 1, 36, 36)):
        assert torch.equal(t[num - 1, :, :used], t[num - 3, :, :used])
    refs[7:num - 3] = 0
    want = [t[num - 3:].clone() for t in pools]
    new = kivi.kivi_paged_compact(c, pool)
    assert new[num - 3:].tolist() == [7, 8, 9] and c.block_table.tolist() == [[8, 7], [8, 9]]
    for t, w in zip(pools, want):
        assert torch.equal(t[7:10], w)


@pytest.mark.parametrize("P,Hkv", [(64, 1), (64, 3), (1024, 2), (8192, 1)])
def test_large_and_odd_pages(P, Hkv):
    t = Both(3, 2, 7, P, Hkv=Hkv, G=32)
    t.reserve([2 * P, P + 1, 5])
    t.m.lens = [2 * P - 3, P + 1, 5]
    t.put()
    t.reorder([0, 0, 1])
    t.reorder([0, -1, 2])
    t.compact()


def test_calls_in_a_graph():
    t = Both(4, 3, 12, 64)
    extra = torch.tensor([70, 0, 0, 10], dtype=torch.int32, device="cuda")
    parent = torch.tensor([0, 0, 3, 3], dtype=torch.int32, device="cuda")
    new_ids = torch.empty(12, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kivi.kivi_paged_reserve(t.c, t.pool, extra)
        kivi.kivi_paged_reorder(t.c, t.pool, parent)
        kivi.kivi_paged_compact(t.c, t.pool, new_ids)
    for lens in ([0, 0, 0, 0], [70, 0, 0, 10], [128, 70, 10, 10]):
        t.m.lens = list(lens)
        t.c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        t.m.reserve(extra.tolist())
        t.m.reorder(parent.tolist())
        assert new_ids.tolist() == t.m.compact()
        t.same()


def test_refusals_of_the_binding():
    t = Both(4, 3, 12, 64)
    with pytest.raises(TypeError):
        kivi.kivi_paged_reserve(t.c, t.pool, torch.zeros(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError):
        kivi.kivi_paged_reorder(t.c, t.pool, torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        kivi.kivi_paged_compact(t.c, t.pool, torch.zeros(12, dtype=torch.int32))
    with pytest.raises(TypeError):
        kivi.PagePool.adopt(t.c, torch.zeros(11, dtype=torch.int32, device="cuda"))


def test_a_serving_run():
    """Admission (reserve, packed attention, packed quantization), decoding with pages reserved step by
    step, a fork of two sequences, the end of another, a compaction and more decoding: every output against the
    oracle's own cache of that sequence."""
    Hq, Hkv, G, P, B = 4, 2, 32, 64, 5
    lens = [100, 64, 0, 31, 0]
    gen = torch.Generator().manual_seed(9)

    def normal(*shape):
        return torch.randn(shape, generator=gen).to(torch.float16)

    c = kivi.PagedCache.allocate(B, Hkv, G, P, 5, 22)
    pool = kivi.PagePool.allocate(c)
    T = sum(lens)
    q, k, v = normal(T, Hq, D), normal(T, Hkv, D), normal(T, Hkv, D)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
    kivi.kivi_paged_reserve(c, pool, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    out = kivi.kivi_prefill_attention_packed(q.cuda(), k.cuda(), v.cuda(), cu, 1 / math.sqrt(D))
    kivi.kivi_paged_prefill_packed(c, k.cuda(), v.cuda(), cu)
    orc, at = {}, 0
    for b, n in enumerate(lens):
        if n:
            kk, vv, qq = (t[at:at + n].transpose(0, 1).contiguous()[None].numpy() for t in (k, v, q))
            orc[b] = oracle.prefill(kk, vv, G, 320)
            ref = oracle.prefill_attention(qq, kk, vv, 1 / math.sqrt(D))
            assert_close(out[at:at + n].transpose(0, 1)[None], ref)
            at += n

    def step(live):
        qs, ks, vs = normal(B, Hq, D), normal(B, Hkv, D), normal(B, Hkv, D)
        kivi.kivi_paged_reserve(c, pool, torch.tensor([int(b in live) for b in range(B)], dtype=torch.int32).cuda())
        got = kivi.kivi_paged_decode_step(c, ks.cuda(), vs.cuda(), qs.cuda(), 1 / math.sqrt(D))
        # a row that is not live has no page: its token is dropped, and its length is put back
        idle = torch.tensor([b not in live for b in range(B)], device="cuda")
        c.seq_lens.masked_fill_(idle, 0)
        for b in live:
            oracle.append(orc[b], ks[b:b + 1].numpy(), vs[b:b + 1].numpy())
            assert_close(got[b:b + 1], oracle.attention(orc[b], qs[b:b + 1].numpy(), 1 / math.sqrt(D)))

    import copy
    for _ in range(5):
        step([0, 1, 3])
    kivi.kivi_paged_reorder(c, pool, torch.tensor([0, 1, 0, 3, 3], dtype=torch.int32).cuda())
    orc[2], orc[4] = copy.deepcopy(orc[0]), copy.deepcopy(orc[3])
    for _ in range(40):  # across a group and a page border
        step([0, 1, 2, 3, 4])
    kivi.kivi_paged_reorder(c, pool, torch.tensor([-1, 4, 2, 3, 4], dtype=torch.int32).cuda())
    orc[1] = copy.deepcopy(orc[4])
    del orc[0]
    kivi.kivi_paged_compact(c, pool)
    used = int(pool.info[2])
    table = c.block_table.cpu()
    assert int(table.max()) < used and (pool.ref_counts[used:] == 0).all()
    for _ in range(40):
        step([1, 2, 3, 4])
    assert c.seq_lens.tolist() == [0] + [orc[b].n for b in (1, 2, 3, 4)]

"""The packed quantizer where each of its CTAs takes a run of units: many heads, sequences and units,
in every form, bit for bit against the one-sequence call; clamped bounds, streams and graphs."""
from __future__ import annotations

import random

import pytest
import torch

from bit_asymmetric_kv_gb300 import build as kbuild
from bit_asymmetric_kv_gb300 import kivi
from test_gpu_packed_prefill import POOLS, pack, paged

pytestmark = pytest.mark.gpu
FORMS = [(G, P, bits, v_res) for G, P in ((32, 64), (64, 128)) for bits in (2, 4) for v_res in (False, True)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    kbuild.build()
    kivi.lib()


def rng_lens(count, most, seed):
    rng = random.Random(seed)
    return [rng.choice([0, 1, 63, 64, 65, most, rng.randrange(most + 1), rng.randrange(most + 1)]) for _ in range(count)]


BATCHES = {  # lengths, KV heads
    "long": ([20001, 0, 17000, 9999], 3),
    "32-sequences": (rng_lens(32, 3000, 1), 4),
    "33-sequences": (rng_lens(33, 3000, 2), 4),
    "200-sequences": (rng_lens(200, 500, 3), 5),
    "512-sequences": (rng_lens(512, 300, 4), 3),
}


def pair_of_caches(lens, Hkv, G, P, bits, v_res):
    B, maxp = len(lens), max(1, max(-(-n // P) for n in lens))
    held = [-(-n // P) for n in lens]
    num = sum(held) + 2
    ids = torch.randperm(num, generator=torch.Generator().manual_seed(2)).int()
    table, at = torch.full((B, maxp), -1, dtype=torch.int32), 0
    for b, m in enumerate(held):
        table[b, :m] = ids[at:at + m]
        at += m
    caches = [paged(B, Hkv, G, P, maxp, num, bits, v_res, 1) for _ in range(2)]
    for c in caches:
        c.block_table.copy_(table)
    return caches


def one_by_one(cache, k, v, bounds):
    for s, (a, b) in enumerate(bounds):
        if b > a:
            kivi.kivi_paged_prefill(cache, s, k[a:b].transpose(0, 1).contiguous(), v[a:b].transpose(0, 1).contiguous())


def assert_same(a, b, v_res):
    for name in POOLS[:6] + (("v_res",) if v_res else ()):
        assert torch.equal(getattr(a, name), getattr(b, name)), name


@pytest.mark.parametrize("batch", list(BATCHES))
@pytest.mark.parametrize("G,P,bits,v_res", FORMS)
def test_runs_of_units(batch, G, P, bits, v_res):
    lens, Hkv = BATCHES[batch]
    units = sum(-(-n // 64) for n in lens)
    ctas = 7 * torch.cuda.get_device_properties(0).multi_processor_count
    assert 2 * Hkv * units > 2 * ctas, "several units a CTA"
    (k, v), cu = pack(lens, [Hkv, Hkv], "tokens", 60 + bits, pad=13, lead=5)
    k[:, :, 7] *= 40
    a, b = pair_of_caches(lens, Hkv, G, P, bits, v_res)
    kivi.kivi_paged_prefill_packed(a, k, v, cu)
    bounds = cu.tolist()
    one_by_one(b, k, v, list(zip(bounds[:-1], bounds[1:])))
    assert_same(a, b, v_res)


@pytest.mark.parametrize("bounds,seqs", [
    ([-50, 90, 90, 2**31 - 1], [(0, 90), (90, 90), (90, 200)]),
    ([-2**31, -1, 70, 200], [(0, 0), (0, 70), (70, 200)]),
    ([200, 300, 2**31 - 1, 5], [(0, 0), (0, 0), (0, 0)]),
])
def test_clamped_bounds(bounds, seqs):
    (k, v), _ = pack([200], [2, 2], "tokens", 61)
    a, b = pair_of_caches([200, 200, 200], 2, 32, 64, 2, False)
    kivi.kivi_paged_prefill_packed(a, k, v, torch.tensor(bounds, dtype=torch.int32, device="cuda"))
    one_by_one(b, k, v, seqs)
    assert_same(a, b, False)


def test_in_a_graph_and_on_a_stream():
    """Captured once, replayed with other lengths; and on a stream that is not the current one."""
    lens = [150, 64, 1, 300]
    (k, v), cu = pack(lens, [3, 3], "tokens", 62)
    T = sum(lens)
    a, b = pair_of_caches([T] * 4, 3, 64, 128, 4, True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kivi.kivi_paged_prefill_packed(a, k, v, cu)
    for bounds in ([0, 150, 214, 215, T], [0, 0, 1, 500, T], [3, 3, 3, 3, 70]):
        cu.copy_(torch.tensor(bounds, dtype=torch.int32))
        g.replay()
        one_by_one(b, k, v, list(zip(bounds[:-1], bounds[1:])))
        assert_same(a, b, True)
    s = torch.cuda.Stream()
    cu.copy_(torch.tensor([0, 100, 100, 201, 400], dtype=torch.int32))
    s.wait_stream(torch.cuda.current_stream())
    kivi.kivi_paged_prefill_packed(a, k, v, cu, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    one_by_one(b, k, v, [(0, 100), (100, 100), (100, 201), (201, 400)])
    assert_same(a, b, True)

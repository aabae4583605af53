"""Read-back and appends on batches large enough that a warp reads several items, and a CTA quantizes several
units.  Each test asserts that its batch is that large."""
from __future__ import annotations

import random

import numpy as np
import pytest
import torch

from bit_asymmetric_kv_gb300 import build as kbuild
from bit_asymmetric_kv_gb300 import kivi
from paged_values import filled, tokens
from test_gpu_window_attention import pack
from test_gpu_window_cache import outputs, same, twins

pytestmark = pytest.mark.gpu
FORMS = [(G, bits, v_res) for G in (32, 64) for bits in (2, 4) for v_res in (False, True)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    kbuild.build()
    kivi.lib()


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ------------------------------------------------------------------------------ read
@pytest.mark.parametrize("G,bits,v_res,Hkv,layout", [(*f, 8, "tokens") for f in FORMS] + [
    (G, bits, v_res, Hkv, layout) for G, bits, v_res in ((32, 2, False), (64, 4, True)) for Hkv, layout in ((3, "heads"), (11, "gaps"))])
def test_reads_of_several_items_a_warp(G, bits, v_res, Hkv, layout):
    """Heads as many as a CTA's warps, fewer and more: a warp steps over heads, blocks and sequences."""
    rng, first = random.Random(Hkv), 70
    lens = [0, 1, 33, G, 2999] + [rng.randrange(3000) for _ in range(150 // Hkv)]
    c = filled(lens, Hkv, G, 128, bits, v_res, seed=24)
    c.block_table[4, 3], c.block_table[5, 0] = -1, c.dims.num_pages
    take = [n if i < 5 else rng.choice([n, max(0, n - 31), n * 3 // 4]) for i, n in enumerate(lens)]
    rooms = [t + rng.choice([0, 0, 5]) for t in take]
    # items (32 positions of a head) beyond what the grid's 4 CTAs an SM of 8 warps have at one each
    assert sum(-(-t // 32) for t in take) * Hkv > sms() * 32
    cu = torch.tensor([3] + [3 + x for x in np.cumsum(rooms)], dtype=torch.int32, device="cuda")
    k, v = outputs(int(cu[-1]) + 4, Hkv, layout)
    kivi.kivi_paged_read(c, cu, torch.tensor(take, dtype=torch.int32, device="cuda"), k, v, first=first)
    want = [np.full(tuple(t.shape), 7, np.float16) for t in (k, v)]
    bounds, table = cu.tolist(), c.block_table.cpu().numpy()
    for b, (n, m) in enumerate(zip(lens, take)):
        p = np.array(list(range(min(first, m))) + list(range(n - (m - min(first, m)), n)), dtype=np.int64)
        if m == 0:
            continue
        page = table[b, p // 128]
        held, late = (page >= 0) & (page < c.dims.num_pages), p >= n // G * G
        for w, t, kept in zip(want, tokens(c, b, p), (late, late & v_res)):
            t = np.clip(t.cpu().numpy(), -65504, 65504).astype(np.float16)
            t[~held & ~kept] = 0
            w[bounds[b]:bounds[b] + m] = t
    for name, w, t in zip("kv", want, (k, v)):
        bad = np.argwhere(t.cpu().numpy() != w)
        assert len(bad) == 0, (name, len(bad), bad[:4].tolist())


# ---------------------------------------------------------------------------- extend
@pytest.mark.parametrize("G,bits,v_res", FORMS)
@pytest.mark.parametrize("Hkv,layout", [(8, "tokens"), (5, "heads")])
def test_appends_of_several_units_a_cta(G, bits, v_res, Hkv, layout):
    """Bit for bit the whole prompts, with residuals before and behind."""
    rng = random.Random(G + bits + Hkv)
    old = [rng.choice([0, 1, G - 1, G, rng.randrange(300)]) for _ in range(34)]
    new = [rng.choice([0, 1, 500, 63, rng.randrange(1, 900), rng.randrange(1, 900)]) for _ in range(34)]
    # items (keys or values of 64 positions of a head) beyond a CTA's one: at most 7 CTAs an SM
    assert sum((o + n - 1) // 64 - o // 64 + 1 for o, n in zip(old, new) if n) * Hkv * 2 > sms() * 7
    a, b, kv = twins(max(o + n for o, n in zip(old, new)), 34, Hkv, G, 128, bits, v_res, 25)
    (k, v), cu = pack(new, [Hkv, Hkv], layout, 26, pad=70, lead=9)
    k[:, :, 7] *= 40
    bounds = cu.tolist()
    for s, n in enumerate(old):
        ks, vs = (t[:, :n].contiguous() for t in kv[s])
        if n:
            kivi.kivi_paged_prefill(a, s, ks, vs)
        if n + new[s]:
            lo, hi = bounds[s], bounds[s + 1]
            kivi.kivi_paged_prefill(b, s, torch.cat([ks, k[lo:hi].transpose(0, 1)], 1).contiguous(),
                                    torch.cat([vs, v[lo:hi].transpose(0, 1)], 1).contiguous())
    kivi.kivi_paged_extend_packed(a, k, v, cu)
    assert same(a, b) == ""

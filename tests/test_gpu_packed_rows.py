"""Packed attention row by row on the GPU: what a row's result may depend on."""
from __future__ import annotations

import math

import pytest
import torch

from bit_asymmetric_kv_gb300 import build as kbuild
from bit_asymmetric_kv_gb300 import kivi
from test_gpu_packed_prefill import pack

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    kbuild.build()
    kivi.lib()


def cu_of(*bounds):
    return torch.tensor(bounds, dtype=torch.int32, device="cuda")


HEADS = [(2, 2), (4, 1), (16, 1), (7, 1)]
BEHIND = {"ordinary": None, "large": 60000.0, "inf": math.inf, "-inf": -math.inf, "nan": math.nan}


@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("n", [5, 300, 1000])
@pytest.mark.parametrize("behind", list(BEHIND))
@pytest.mark.parametrize("as_prompt", [False, True])
def test_bits_do_not_depend_on_what_stands_behind(Hq, Hkv, n, behind, as_prompt):
    """The rows behind a prompt, padding or the next prompt, share its last tiles; the prompt's own bits are
    those that it has alone."""
    (q, k, v), _ = pack([n, 200], [Hq, Hkv, Hkv], "tokens", 20 + n)
    alone = kivi.kivi_prefill_attention_packed(q[:n], k[:n], v[:n], cu_of(0, n), 0.1)
    if BEHIND[behind] is not None:
        for t in (q, k, v):
            t[n:] = BEHIND[behind]
    cu = cu_of(0, n, n + 200) if as_prompt else cu_of(0, n)
    got = kivi.kivi_prefill_attention_packed(q, k, v, cu, 0.1)
    assert torch.equal(got[:n], alone)

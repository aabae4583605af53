"""Packed attention row by row on the GPU: what a row's result may depend on, how its weights hold
together over the whole range of scores, which rows clamped bounds give, and calls from other host threads.

Tolerance of the weights' test, before any run.  The scores are integers that fp32 holds exactly, at
most 9 apart, and every |v| is 1, so that sum_j p_j |v_j| / l = 1:
  - the output is rounded to fp16 once: 2^-11 |out| + 2^-25;
  - the probabilities enter the P.V product in fp16 (none is subnormal there): 2^-11;
  - an exponent is a difference of at most 9 log2(e) + 4 = 17 and a rescale's one of 13; scale and
    log2(e) are rounded to fp32 (2 * 2^-24 of the difference), the result once (2^-24 of it), an
    exponential is 2^-22 off: less than 2^-18 of a weight in all, numerator and denominator: 2^-17;
  - the sums over the keys in fp32: 2^-22 per step of 16 keys.
Nothing in it grows with the scores themselves.
"""
from __future__ import annotations

import math
import threading

import pytest
import torch

from bit_asymmetric_kv_gb300 import build as kbuild
from bit_asymmetric_kv_gb300 import kivi
from test_gpu_packed_prefill import check_attention, pack

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


# of each head: scores 256 k0 + a, and 9 more for the first key, whose tile comes last
SCORES = {
    "near": [(177, 24), (174, 10), (172, 31), (169, 17)],             # log2 just below 2^16
    "crossing-up": [(177, 107), (177, 109), (177, 110), (177, 112)],  # from below 2^16 to above
    "crossing-down": [(-178, 133), (-178, 136), (-178, 138), (-178, 141)],
    "beyond": [(250, 100), (500, 3), (-400, 5), (1000, 7)],
    "small": [(0, 0), (1, 3), (-2, 7), (40, 1)],
}


@pytest.mark.parametrize("kind", list(SCORES))
def test_weights_before_and_after_a_new_maximum_agree(kind):
    """Thousands of equal weights against one that is e^9 times as large and met last: the two sides' sums are
    alike, so that a mismatch between the weights before and after the jump shows."""
    n, heads = 8300, SCORES[kind]
    q = torch.zeros((n, len(heads), D), dtype=torch.float16, device="cuda")
    k, v = torch.zeros_like(q), torch.ones_like(q)
    q[:, :, 0], q[:, :, 1] = 256.0, 1.0
    for h, (k0, a) in enumerate(heads):
        k[:, h, 0], k[:, h, 1] = k0, a
        k[0, h, 1] = a + 9
    v[0] = -1.0
    out = kivi.kivi_prefill_attention_packed(q, k, v, cu_of(0, n), 1.0)
    i = torch.arange(n, dtype=torch.float64, device="cuda")[:, None, None]
    ref = (i - math.exp(9.0)) / (i + math.exp(9.0))
    tol = 2.0**-11 * ref.abs() + 2.0**-25 + 2.0**-11 + 2.0**-17 + (n / 16) * 2.0**-22
    worst = ((out.double() - ref).abs() - tol).amax((0, 2)).tolist()
    assert max(worst) <= 0, worst


@pytest.mark.parametrize("Hq,Hkv", [(2, 1), (2, 2)])
@pytest.mark.parametrize("bounds,seqs", [
    ([-50, 90, 60, 2**31 - 1], [(0, 90), None, (60, 200)]),            # rows 60 .. 89 in two: not looked at
    ([-2**31, 90, 90, 2**31 - 1], [(0, 90), None, (90, 200)]),
    ([-50, -1, 90, 200], [None, (0, 90), (90, 200)]),
    ([-3, 200, 200, 500], [(0, 200), None, None]),
    ([200, 2**31 - 1, 300, 1000], [None, None, None]),                 # all past the axis
    ([-9, -5, -5, 0], [None, None, None]),                             # all before it
])
def test_clamped_bounds(Hq, Hkv, bounds, seqs):
    """Starts are clamped to the axis and ends to [start, axis]: every row of one sequence has the bits that the
    sequence has alone, within the tolerance of the formula, and rows of none are left."""
    (q, k, v), _ = pack([200], [Hq, Hkv, Hkv], "tokens", 9)
    out = torch.full(q.shape, 3.0, dtype=torch.float16, device="cuda")
    kivi.kivi_prefill_attention_packed(q, k, v, cu_of(*bounds), 0.1, out=out)
    times = torch.zeros(200, dtype=torch.int32, device="cuda")
    for a, b in filter(None, seqs):
        times[a:b] += 1
    for a, b in filter(None, seqs):
        Q, K, V, cu = q[a:b], k[a:b], v[a:b], cu_of(0, b - a)
        alone = kivi.kivi_prefill_attention_packed(Q, K, V, cu, 0.1)
        check_attention(alone, Q, K, V, cu, 0.1)
        only = times[a:b] == 1
        assert only.any() and torch.equal(out[a:b][only], alone[only])
    assert (out[times == 0] == 3).all()


def test_a_thread_that_has_called_nothing_yet():
    """A host thread whose first CUDA call is this one."""
    (q, k, v), cu = pack([100, 44], [4, 2, 2], "tokens", 50)
    want = kivi.kivi_prefill_attention_packed(q, k, v, cu, 0.1)
    out, stream, seen = torch.zeros_like(want), torch.cuda.current_stream().cuda_stream, []

    def call():
        try:
            kivi.kivi_prefill_attention_packed(q, k, v, cu, 0.1, out=out, stream=stream)
        except Exception as e:  # noqa: BLE001
            seen.append(e)

    t = threading.Thread(target=call)
    t.start()
    t.join()
    assert not seen, seen
    torch.cuda.synchronize()
    assert torch.equal(out, want)

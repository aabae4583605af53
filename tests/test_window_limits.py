"""Dimensions at which window decode's unit counts leave 32 bits, refused on the host.  A whole context of n tokens
has at most n / 64 + 1 units; with a window, a sequence's units are counted with up to eight more than its n / 64
units of codes: four for the residual and four for a head's own work."""
from __future__ import annotations

import pytest

from bit_asymmetric_kv_gb300 import build as kbuild
from bit_asymmetric_kv_gb300 import kivi

FAKE = 1 << 20  # an aligned, never dereferenced address
UNSUPPORTED = 3


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kivi.lib()


def dims(B, max_pages):
    return kivi.kivi_paged_dims(B, 1, 128, 32, 2, 0, 64, max_pages, 20)


def calls(L, d):
    """Statuses of the whole-context calls and of the windows', all without a workspace."""
    c = kivi.kivi_paged_cache(FAKE, FAKE, FAKE, FAKE, FAKE, 0, FAKE, FAKE)
    rest = (FAKE, 0, 0, 0)
    whole = [L.kivi_paged_decode_attention(d, c, FAKE, 4, 0.1, *rest), L.kivi_paged_decode_step(d, c, FAKE, FAKE, FAKE, 4, 0.1, *rest)]
    window = [L.kivi_paged_decode_attention_window(d, c, FAKE, 4, 0.1, 5, 1, *rest),
              L.kivi_paged_decode_step_window(d, c, FAKE, FAKE, FAKE, 4, 0.1, 5, 1, *rest)]
    return whole, window


@pytest.mark.parametrize("B", [512, 511, 64, 63])
def test_counted_units_stay_in_32_bits(L, B):
    fits = (2**31 - 1) // B - 8       # pages of 64 tokens a sequence, a unit each
    cap = (2**31 - 1) // 64           # positions are 32 bits too
    for pages in (fits - 1, fits, fits + 1, fits + 6, fits + 7):
        if pages > cap:
            continue
        whole, window = calls(L, dims(B, pages))
        assert UNSUPPORTED not in whole, pages
        if pages <= fits:
            assert UNSUPPORTED not in window, pages
        else:
            assert window == [UNSUPPORTED] * 2, pages
    if fits + 8 <= cap:
        whole, window = calls(L, dims(B, fits + 8))
        assert whole == window == [UNSUPPORTED] * 2

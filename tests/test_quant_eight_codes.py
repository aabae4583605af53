"""The 4-bit codes' rule in the form that eight codes are checked in at once, against the rule as it is
written: rint(fl32(fl32(x - mn) / s)) with IEEE operations, for every fp16 scale and the values next to the
half-integers."""
from __future__ import annotations

import numpy as np


def f32(x):
    return np.asarray(x, dtype=np.float32)


def eight(d, s):
    """codes4_chunk8's arithmetic on fp32 d = fl(x - mn) and fp32 s of an fp16 scale."""
    rs = f32(1) / s
    q = d * rs
    r = np.rint(q)
    slow = (np.abs(q - r) > f32(0.5 - 2.0**-15)) | (q > f32(15.25))
    h = np.floor(q)
    m = h + f32(0.5)
    ms = m * s
    near = np.where(d > ms, h + 1, np.where(d < ms, h, np.rint(m)))
    exact = np.minimum(np.where(np.abs(q - m) < f32(2.0**-14), near, np.rint(q)), 15)
    return np.where(slow, exact, r).astype(np.int64)


def written(d, s):
    return np.clip(np.rint(d / s), 0, 15).astype(np.int64)


def test_next_to_the_half_integers():
    scales = np.arange(1, 0x7c00, dtype=np.uint16).view(np.float16).astype(np.float32)
    for h in range(16):
        mid = (f32(h) + f32(0.5)) * scales  # exact
        for step in (-3, -2, -1, 0, 1, 2, 3):
            d = mid
            for _ in range(abs(step)):
                d = np.nextafter(d, f32(np.inf if step > 0 else 0))
            assert np.array_equal(eight(d, scales), written(d, scales)), (h, step)


def test_random_differences():
    rng = np.random.default_rng(1)
    s = rng.integers(1, 0x7c00, 2_000_000).astype(np.uint16).view(np.float16).astype(np.float32)
    d = f32(rng.random(s.size) * 15.6) * s
    assert np.array_equal(eight(d, s), written(d, s))


def test_differences_of_fp16_values():
    """d as it comes about: x - mn of fp16 values of one group, with the group's scale."""
    rng = np.random.default_rng(2)
    x = (rng.standard_normal((40000, 32)) * 2.0 ** rng.integers(-14, 12, (40000, 1))).astype(np.float16)
    mn = x.min(1, keepdims=True).astype(np.float32)
    s = ((x.max(1, keepdims=True).astype(np.float32) - mn) / f32(15)).astype(np.float16).astype(np.float32)
    d = x.astype(np.float32) - mn
    keep = (s > 0)[:, 0]
    assert np.array_equal(eight(d[keep], s[keep]), written(d[keep], s[keep]))


def test_joined_codes_are_exact():
    c = np.random.default_rng(3).integers(0, 16, (1000, 8)).astype(np.float32)
    v = c[:, 1::2] * f32(16) + c[:, 0::2]
    lo, hi = (f32(v[:, i + 1] * f32(256) + v[:, i]) + f32(8388608) for i in (0, 2))
    word = (lo.view(np.uint32) & 0xFFFF) | (hi.view(np.uint32) << 16)
    want = sum(c[:, i].astype(np.uint32) << np.uint32(4 * i) for i in range(8))
    assert np.array_equal(word, want)

"""4-bit codes of values next to half-integers, where the packed quantizer's fast form gives way to the exact
comparison (within 2^-15), bit for bit against the definition: code = clamp(rint(fl32(fl32(x - mn) / s)), 0, 15), as prompts, and
as tokens appended behind a residual."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from bit_asymmetric_kv_gb300 import build as kbuild
from bit_asymmetric_kv_gb300 import kivi

D = 128


def scale_of(mn, mx):
    """fp32 value of the fp16 scale of fp16 minima and maxima."""
    return ((mx.astype(np.float32) - mn.astype(np.float32)) / np.float32(15)).astype(np.float16).astype(np.float32)


def on_halves(rng):
    """(mn, mx, x [.., 15]): ranges and, for each, the fp16 values on its half-integers, as often as they fill 15."""
    n = 100_000
    e = rng.integers(-12, 13, n)
    a = (rng.integers(1024, 2048, n) * 2.0 ** (e - 10)).astype(np.float16)
    # from zero, from the far side of zero, and from a value of the same size
    kind = rng.integers(0, 3, n)
    b = np.where(kind == 0, 0, np.where(kind == 1, -1, 0.5) * rng.integers(1, 2048, n) * 2.0 ** (e - 11)).astype(np.float16)
    mn, mx = np.minimum(a, b), np.maximum(a, b)
    s = scale_of(mn, mx).astype(np.float64)
    mn, mx, s = mn[s > 0], mx[s > 0], s[s > 0]
    at = mn.astype(np.float64)[:, None] + (np.arange(15) + 0.5) * s[:, None]
    x = at.astype(np.float16)
    on = (x == at) & (x >= mn[:, None]) & (x <= mx[:, None])
    some = on.any(1)
    x = np.take_along_axis(x[some], np.argsort(~on[some], axis=1, kind="stable"), 1)
    return mn[some], mx[some], np.take_along_axis(x, np.arange(15)[None] % on[some].sum(1)[:, None], 1)


def beside_halves(rng):
    """The same for ranges of which one half-integer lies next to zero, where fp16 is fine: values 2^-15 to 2^-21 of
    the scale beside it, on both sides."""
    n = 30_000
    s = (rng.integers(1024, 2048, n) * 2.0 ** (rng.integers(-6, 11, n) - 10)).astype(np.float16).astype(np.float64)
    h = rng.integers(0, 15, n) + 0.5
    mn = (-h * s).astype(np.float16)
    mx = (mn.astype(np.float64) + 15 * s).astype(np.float16)
    s = scale_of(mn, mx).astype(np.float64)
    step = np.sign(rng.random((n, 15)) - 0.5) * 2.0 ** rng.uniform(-21, -15.01, (n, 15))
    x = (mn.astype(np.float64)[:, None] + (h[:, None] + step) * s[:, None]).astype(np.float16)
    q = (x.astype(np.float64) - mn.astype(np.float64)[:, None]) / s[:, None]
    ok = ((np.abs(q - h[:, None]) < 2.0**-15) & (x >= mn[:, None]) & (x <= mx[:, None])).all(1)
    return mn[ok], mx[ok], x[ok]


def pool():
    """As many of the one kind as of the other."""
    rng = np.random.default_rng(11)
    a, b = on_halves(rng), beside_halves(rng)
    m = min(len(a[0]), len(b[0]))
    return [np.concatenate([x[:m], y[:m]]) for x, y in zip(a, b)]


def groups(count, size, seed):
    """fp16 [count, size]: groups of `size` values, each a range's ends and values next to its half-integers."""
    mn, mx, x = pool()
    rng = np.random.default_rng(seed)
    i = rng.integers(0, len(mn), count)
    g = x[i][:, rng.integers(0, 15, size)]
    ends = rng.permuted(np.tile(np.arange(size), (count, 1)), axis=1)[:, :2]
    rows = np.arange(count)
    g[rows, ends[:, 0]], g[rows, ends[:, 1]] = mn[i], mx[i]
    return g


def definition(x, axis):
    """Codes and {s, z} words."""
    mn, mx = x.min(axis, keepdims=True), x.max(axis, keepdims=True)
    s = scale_of(mn, mx)
    d = x.astype(np.float32) - mn.astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(s > 0, np.clip(np.rint(d / s), 0, 15), 0).astype(np.int64)
    z = np.where(mn == 0, np.float16(0), mn).astype(np.float16)
    word = s.astype(np.float16).view(np.uint16).astype(np.int64) | z.view(np.uint16).astype(np.int64) << 16
    return c, word.squeeze(axis)


def test_the_values_are_next_to_half_integers():
    mn, mx, x = pool()
    assert len(mn) > 4000
    s = scale_of(mn, mx)
    q = (x.astype(np.float32) - mn.astype(np.float32)[:, None]) / s[:, None]
    far = np.abs(q - np.floor(q) - np.float32(0.5))
    assert (far < 2.0**-14).all() and 0.4 < (far > 0).mean() < 0.6
    up = far * np.sign(q - np.floor(q) - np.float32(0.5))
    assert (up > 0).mean() > 0.15 and (up < 0).mean() > 0.15
    assert len(np.unique(np.floor(q[far > 0]))) == 15 and len(np.unique(np.floor(q[far == 0]))) == 15


def unpacked(words):
    w = words.cpu().numpy().astype(np.int64) & 0xFFFFFFFF
    return ((w[..., None] >> (4 * np.arange(8))) & 15).reshape(*w.shape[:-1], D)


@pytest.mark.gpu
@pytest.mark.parametrize("G,P", [(32, 64), (64, 128)])
@pytest.mark.parametrize("v_res", [False, True])
@pytest.mark.parametrize("appended", [False, True])
def test_codes_next_to_half_integers(G, P, v_res, appended):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    kbuild.build()
    B, Hkv, n = 3, 2, 8 * G
    k = groups(B * 8 * Hkv * D, G, 1).reshape(B, 8, Hkv, D, G).transpose(0, 1, 4, 2, 3).reshape(B, n, Hkv, D)
    v = groups(B * n * Hkv, D, 2).reshape(B, n, Hkv, D)
    kt, vt = (torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in (k, v))
    c = kivi.PagedCache.allocate(B, Hkv, G, P, n // P, B * (n // P), bits=4, value_residual=v_res)
    c.block_table.copy_(torch.randperm(B * (n // P), generator=torch.Generator().manual_seed(3)).view(B, -1))
    old = [0] * B
    if appended:  # the first group's rows come from the residual and from the call
        old = [G // 2 + 3, 2 * G + 1, 4 * G - 1]
        for b, m in enumerate(old):
            kivi.kivi_paged_prefill(c, b, kt[b, :m].transpose(0, 1).contiguous(), vt[b, :m].transpose(0, 1).contiguous())
    cu = torch.tensor([0] + list(np.cumsum([n - m for m in old])), dtype=torch.int32, device="cuda")
    rows = [torch.cat([t[b, m:] for b, m in enumerate(old)]) for t in (kt, vt)]
    (kivi.kivi_paged_extend_packed if appended else kivi.kivi_paged_prefill_packed)(c, *rows, cu)
    table = c.block_table.cpu().numpy()
    for b in range(B):
        want, word = definition(k[b].reshape(8, G, Hkv, D), 1)
        got = unpacked(c.k_codes[table[b].tolist()]).transpose(0, 2, 1, 3).reshape(8, G, Hkv, D)
        assert np.array_equal(got, want), np.argwhere(got != want)[:4].tolist()
        got = c.k_meta[table[b].tolist()].cpu().numpy().astype(np.int64).transpose(0, 2, 1, 3).reshape(8, Hkv, D) & 0xFFFFFFFF
        assert np.array_equal(got, word)
        want, word = definition(v[b], -1)
        got = unpacked(c.v_codes[table[b].tolist()]).transpose(0, 2, 1, 3).reshape(n, Hkv, D)
        assert np.array_equal(got, want), np.argwhere(got != want)[:4].tolist()
        got = c.v_meta[table[b].tolist()].cpu().numpy().astype(np.int64).transpose(0, 2, 1).reshape(n, Hkv) & 0xFFFFFFFF
        assert np.array_equal(got, word)
    assert c.seq_lens.tolist() == [n] * B

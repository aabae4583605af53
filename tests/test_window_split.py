"""The split of window decode's work between warps, on the host: the index arithmetic of the persistent grid where
there are more units than warps (counted units, empty ones among them), walked warp by warp.

Every unit with a visible token is taken once, by a warp that emits the head; the partials of a head fill the slots
that its header names, and no slot lies outside the workspace of n_warps + heads pairs."""
from __future__ import annotations

import bisect
import random

import pytest

UNIT = 64


def owner_warp(u, W, NW):
    return ((u + 1) * NW - 1) // W


def geometry(n, G, window, sinks):
    """(code units with a visible token, context units they are, whether there is a residual)."""
    NG = n // G
    nq, ncu = NG * G, -(-NG * G // UNIT)
    lo = max(n - window, 0)
    start = ncu if lo >= nq else lo // UNIT
    su = -(-min(sinks, nq) // UNIT)
    skip = max(start - su, 0)
    return ncu - skip, [u if u < su else u + skip for u in range(ncu - skip)], n > nq


def counted_units(R, codes, residual, counted):
    kResidual, kHead = (3 if R == 1 else 4), (2 if R == 1 else 3 if R == 2 else 4)
    if not counted:
        return codes + residual
    return codes + (kResidual if residual else 0) + (kHead if codes or residual else 0)


def walk(lens, Hkv, R, G, window, sinks, n_warps):
    geo = [geometry(n, G, window, sinks) for n in lens]
    for n, (codes, units, residual) in zip(lens, geo):
        vis = {t // UNIT for t in range(n // G * G) if t > n - 1 - window or t < sinks}
        assert sorted(vis) == units, (n, G, window, sinks)
    counted = sum(c + r for c, _, r in geo) * Hkv > n_warps
    U = [counted_units(R, c, r, counted) for c, _, r in geo]
    cum = [0]
    for u in U:
        cum.append(cum[-1] + u)
    W = Hkv * cum[-1]
    if W == 0:
        return counted
    NW = min(W, n_warps)
    taken, header, emitted = {}, {}, {}
    for gw in range(NW):
        u0, u1 = gw * W // NW, (gw + 1) * W // NW
        assert u0 < u1
        # the sequence of the first unit: the last with Hkv * cum <= u0
        b = bisect.bisect_right([Hkv * c for c in cum[:-1]], u0) - 1
        rel = u0 - Hkv * cum[b]
        kvh, uu = divmod(rel, U[b])
        assert kvh < Hkv
        worked = False
        for kk in range(u1 - u0):
            codes, _, residual = geo[b]
            last = codes if residual else codes - 1
            h = b * Hkv + kvh
            if uu == 0:
                start = Hkv * cum[b] + kvh * U[b]
                assert h not in header
                header[h] = (gw + h, owner_warp(start + last, W, NW) - gw + 1)
            if uu <= last:
                assert (h, uu) not in taken
                taken[h, uu] = gw
                worked = True
            if uu + 1 == U[b] or kk + 1 == u1 - u0:
                if worked:
                    emitted.setdefault(h, []).append(gw + h)
                worked = False
            uu += 1
            if uu == U[b]:
                uu, kvh = 0, kvh + 1
                if kvh == Hkv:
                    kvh, b = 0, b + 1
                    while b < len(lens) and cum[b + 1] == cum[b]:
                        b += 1
    assert set(taken) == {(b * Hkv + k, u) for b, (c, _, r) in enumerate(geo) for k in range(Hkv) for u in range(c + r)}
    slots = set()
    for h, (first, count) in header.items():
        assert emitted[h] == list(range(first, first + count)), (h, first, count, emitted[h])
        assert not slots & set(emitted[h]) and emitted[h][-1] < n_warps + len(lens) * Hkv
        slots |= set(emitted[h])
    assert set(emitted) == set(header)
    return counted


@pytest.mark.parametrize("seed", range(60))
def test_random_batches(seed):
    rng = random.Random(seed)
    B, Hkv, R, G = rng.choice([1, 3, 20, 64]), rng.choice([1, 2, 3, 8]), rng.choice([1, 2, 4]), rng.choice([32, 64])
    lens = [rng.choice([0, 1, G - 1, G, 64, rng.randrange(2000), rng.randrange(2000)]) for _ in range(B)]
    for window, sinks in ((1, 0), (rng.randrange(1, 200), rng.choice([0, 4, 70])), (rng.randrange(1, 3000), rng.randrange(300))):
        for n_warps in (12, 100, 1824):
            walk(lens, Hkv, R, G, window, sinks, n_warps)


@pytest.mark.parametrize("R", [1, 2, 4])
@pytest.mark.parametrize("G", [32, 64])
def test_full_batches(R, G):
    rng = random.Random(R * G)
    lens = [rng.choice([0, 5, 64, 200, rng.randrange(1, 2000), rng.randrange(1, 2000)]) for _ in range(64)]
    for window, sinks in ((400, 4), (1000, 70), (20, 0), (4096, 0)):
        assert walk(lens, 8, R, G, window, sinks, 300)  # a nonempty sequence has a unit at least: 8 heads of some 50
        assert not walk(lens[:4], 8, R, G, window, sinks, 1824)

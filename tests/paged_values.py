"""Plain readings of a paged cache, position by position and in 64 bits, for tests."""
from __future__ import annotations

import torch

D = 128


def _halves(w):
    h = w.contiguous().view(torch.float16).view(*w.shape, 2).double()
    return h[..., 0], h[..., 1]


def tokens(cache, b: int, positions):
    """(K, V) [len, Hkv, D] of sequence b at the given positions."""
    d = cache.dims
    n = min(max(int(cache.seq_lens[b]), 0), d.max_pages_per_seq * d.page_tokens)
    P, G, bits = d.page_tokens, d.G, d.bits
    p = torch.as_tensor(list(positions), dtype=torch.long, device=cache.k_codes.device)
    ch = torch.arange(D, device=p.device)
    page, row = cache.block_table[b].long()[p // P].clamp(0, d.num_pages - 1), p % P
    word, shift = ch * bits // 32, ch * bits % 32

    def codes(w):
        return ((w.long()[..., word] >> shift) & (2**bits - 1)).double()

    s, z = _halves(cache.k_meta[page, :, row // G])
    k = codes(cache.k_codes[page, :, row]) * s + z
    s, z = _halves(cache.v_meta[page, :, row])
    v = codes(cache.v_codes[page, :, row]) * s[..., None] + z[..., None]
    late = p >= n // G * G
    k[late] = cache.k_res[b][:, (p % G)[late]].transpose(0, 1).double()
    if cache.v_res is not None:
        v[late] = cache.v_res[b][:, (p % G)[late]].transpose(0, 1).double()
    return k, v


def seen(n: int, window: int, sinks: int):
    """Positions that the newest of n tokens sees."""
    return [t for t in range(n) if t > n - 1 - window or t < sinks]


def filled(lens, Hkv, G, P, bits, v_res, seed, spare=2, room=0):
    """A cache whose sequences hold prompts of the given lengths, in shuffled pages with pages for `room`
    more tokens; what no token was written to is full of ones (pages) or of -30000 (residuals)."""
    from bit_asymmetric_kv_gb300 import kivi

    gen = torch.Generator().manual_seed(seed)
    pages = [-(-(n + room) // P) for n in lens]
    maxp, num = max(1, max(pages)), sum(pages) + spare
    c = kivi.PagedCache.allocate(len(lens), Hkv, G, P, maxp, num, bits=bits, value_residual=v_res)
    for t in (c.k_codes, c.k_meta, c.v_codes, c.v_meta):
        t.fill_(-1)
    c.k_res.fill_(-30000.0)
    if v_res:
        c.v_res.fill_(-30000.0)
    ids = torch.randperm(num, generator=gen).tolist()
    table = torch.full((len(lens), maxp), -1, dtype=torch.int32)
    for b, m in enumerate(pages):
        for j in range(m):
            table[b, j] = ids.pop()
    c.block_table.copy_(table)
    for b, n in enumerate(lens):
        if n:
            k, v = (torch.randn((Hkv, n, D), generator=gen).to(torch.float16) for _ in "kv")
            k[:, :, 5] *= 30
            kivi.kivi_paged_prefill(c, b, k.cuda(), v.cuda())
    return c

"""Cases of the packed-prompt and page operators of the KIVI cache, for measuring them.

Operators:
  attention  causal attention over prompts of different lengths packed into one token axis
  quantize   the packed prompts' keys and values quantized into the pages of every sequence
  fork       sequences of a paged batch replaced by copies of others (a beam step)
  turnover   finished sequences freed and the pages of their successors reserved
  compact    the live pages moved to the low ids of the pool

`run` computes them in plain torch operations, or with `own` set by the library's calls.
"""
import math
import random

import torch

own = False

D = 128


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # three one-line prompts of a small model: launch latency
        dict(name="attention-few-tokens", op="attention", n_seqs=3, lo=1, hi=64, Hq=4, Hkv=1, layout="tokens", pad=0),
        # a full admission batch of chat turns, views of one fused projection, padded to a bucket
        dict(name="attention-short-prompts", op="attention", n_seqs=128, lo=1, hi=512, Hq=32, Hkv=8, layout="tokens",
             pad=100),
        # eight Llama-2-7B-shaped prompts of ragged lengths, head-major
        dict(name="attention-ragged-mha", op="attention", n_seqs=8, lo=700, hi=4113, Hq=32, Hkv=32, layout="heads",
             pad=0),
        # two long documents, Mistral-7B-shaped heads
        dict(name="attention-long-gqa", op="attention", n_seqs=2, lo=8200, hi=16384, Hq=32, Hkv=8, layout="tokens",
             pad=0),
        # a few small prompts into pages of 64 tokens
        dict(name="quantize-small", op="quantize", n_seqs=4, lo=1, hi=200, Hkv=2, G=32, P=64, bits=2, v_res=False,
             layout="tokens", pad=7),
        # an admission batch of long prompts
        dict(name="quantize-long", op="quantize", n_seqs=16, lo=500, hi=8192, Hkv=8, G=64, P=128, bits=2, v_res=False,
             layout="tokens", pad=0),
        # one small beam search
        dict(name="fork-small", op="fork", groups=1, beams=4, lo=90, hi=400, Hkv=1, G=32, P=64, v_res=False),
        # a beam step of a large batch
        dict(name="fork-beams", op="fork", groups=64, beams=4, lo=100, hi=4096, Hkv=8, G=32, P=64, v_res=False),
        # a small server's step
        dict(name="turnover-small", op="turnover", B=8, lo=20, hi=1000, P=64, spare=64),
        # a full server with a large pool
        dict(name="turnover-large", op="turnover", B=512, lo=100, hi=8192, P=64, spare=40000),
        # a small pool after a burst
        dict(name="compact-small", op="compact", B=8, lo=64, hi=900, Hkv=1, G=32, P=64, live=0.5),
        # a large pool, half of it holes
        dict(name="compact-large", op="compact", B=128, lo=500, hi=8192, Hkv=4, G=32, P=64, live=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "quantize", "fork", "turnover", "compact"])
    layout = rng.choice(["tokens", "heads"])
    if op == "attention":
        Hkv = rng.choice([1, 2, 4, 8, 32])
        R = rng.choice([1, 2, 4]) if Hkv < 32 else 1
        hi = _log(rng, 2, 12000)
        n_seqs = max(1, min(_log(rng, 1, 256), 40000 // hi))
        return dict(op=op, n_seqs=n_seqs, lo=max(1, int(hi * rng.random())), hi=hi, Hq=R * Hkv, Hkv=Hkv, layout=layout,
                    pad=rng.choice([0, 1, 63, 200]))
    G = rng.choice([32, 64])
    if op == "quantize":
        hi = _log(rng, 10, 8000)
        return dict(op=op, n_seqs=max(1, min(_log(rng, 1, 200), 60000 // hi)), lo=max(1, int(hi * rng.random())),
                    hi=hi, Hkv=rng.choice([1, 2, 3, 8]), G=G, P=rng.choice([64, 128, 256]), bits=rng.choice([2, 4]),
                    v_res=rng.random() < 0.3, layout=layout, pad=rng.choice([0, 5, 300]))
    if op == "fork":
        return dict(op=op, groups=_log(rng, 1, 48), beams=rng.choice([2, 3, 4, 5]), lo=rng.randrange(1, 400),
                    hi=_log(rng, 400, 4000), Hkv=rng.choice([1, 2, 4, 8]), G=G, P=rng.choice([64, 128]),
                    v_res=rng.random() < 0.3)
    if op == "turnover":
        return dict(op=op, B=_log(rng, 1, 512), lo=rng.randrange(1, 200), hi=_log(rng, 200, 8000),
                    P=rng.choice([64, 128, 256]), spare=_log(rng, 1, 40000))
    return dict(op=op, B=_log(rng, 1, 120), lo=rng.randrange(1, 400), hi=_log(rng, 400, 8000),
                Hkv=rng.choice([1, 2, 4]), G=G, P=rng.choice([64, 128]), live=rng.choice([0.2, 0.5, 0.9]))


def _lens(case, n):
    """The lengths of a case: its smallest and largest, the rest spread over their logarithm; one
    sequence in ten has no tokens."""
    r = random.Random("%d %d %d" % (n, case["lo"], case["hi"]))
    lens = [case["hi"], case["lo"]] + [_log(r, case["lo"], case["hi"]) for _ in range(n)]
    lens = [0 if i % 10 == 9 else x for i, x in enumerate(lens[:n])]
    r.shuffle(lens)
    return lens


def _groups(case):
    """(parent, lengths) of a beam step: survivors keep their rows, every other row of a group becomes
    a copy of one of the group's survivors."""
    r = random.Random("fork %d %d %d %d" % (case["groups"], case["beams"], case["lo"], case["hi"]))
    parent, lens = [], []
    for g in range(case["groups"]):
        n = _log(r, case["lo"], case["hi"])
        b0, beams = g * case["beams"], case["beams"]
        keep = sorted(r.sample(range(beams), r.randrange(1, beams)))
        for i in range(beams):
            parent.append(b0 + (i if i in keep else r.choice(keep)))
            lens.append(n)
    return parent, lens


def _page_bytes(case):
    """Bytes of one page of the pool."""
    P = case["P"]
    return case["Hkv"] * (2 * P * 32 * case.get("bits", 2) // 2 + P // case["G"] * 512 + 4 * P)


def work(case):
    op = case["op"]
    if op == "attention":
        lens = _lens(case, case["n_seqs"])
        T, pairs = sum(lens), sum(n * (n + 1) // 2 for n in lens)
        return {"bytes": 256 * T * 2 * (case["Hq"] + case["Hkv"]), "flops": 4 * D * case["Hq"] * pairs}
    if op == "quantize":
        lens, G, per = _lens(case, case["n_seqs"]), case["G"], 16 * case["bits"]
        out = 0
        for n in lens:
            nq = n // G * G
            nv = nq if case["v_res"] else n
            out += nq * per + nq // G * 512 + nv * (per + 4) + (n - nq) * 256 + (n - nv) * 256
        return {"bytes": case["Hkv"] * (512 * sum(lens) + out), "flops": 0}
    if op == "fork":
        parent, lens = _groups(case)
        P, G, moved = case["P"], case["G"], 0
        for b, p in enumerate(parent):
            if p != b:
                n = lens[p]
                r, rg = n % P, n % P // G * G
                moved += case["Hkv"] * (32 * rg + rg // G * 512 + 36 * (rg if case["v_res"] else r))
                moved += case["Hkv"] * (n % G) * 256 * (2 if case["v_res"] else 1)
                moved += 4 * -(-n // P)
        return {"bytes": 2 * moved + 8 * len(parent), "flops": 0}
    lens = _lens(case, case["B"])
    pages = sum(-(-n // case["P"]) for n in lens)
    if op == "turnover":
        gone = sum(-(-n // case["P"]) for b, n in enumerate(lens) if b % 4 == 1)
        return {"bytes": 8 * (pages + case["spare"]) + 16 * gone + 12 * len(lens), "flops": 0}
    num = max(pages + 1, int(pages / case["live"]))
    moved = pages * (num - pages) // num  # a live page lies above the live count with this chance
    return {"bytes": 2 * moved * _page_bytes(case) + 12 * num + 8 * pages, "flops": 0}


# ------------------------------------------------------------------------- inputs
def _packed(gen, T, heads, layout):
    """fp16 rows of a token axis of T for each of `heads` (name, count), as views [T, count, D]:
    of one fused projection ("tokens"), or head-major."""
    total = sum(c for _, c in heads)
    shape = (T, total, D) if layout == "tokens" else (total, T, D)
    buf = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.float16)
    if layout != "tokens":
        buf = buf.transpose(0, 1)
    out, at = {}, 0
    for name, c in heads:
        out[name] = buf[:, at:at + c]
        at += c
    return out


def _outliers(gen, k):
    """Two fixed outlier channels of every key head, as keys have them."""
    for h in range(k.shape[1]):
        c = torch.randperm(D, generator=gen, device="cuda")[:2]
        f = 20 + 20 * torch.rand(2, generator=gen, device="cuda")
        k[:, h, c] = (k[:, h, c].float() * f).to(torch.float16)


def _cu(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()


def _ceil(a, b):
    return -(-a // b)


def _pools(num, B, Hkv, G, P, bits, v_res, gen=None):
    W = D * bits // 32

    def words(*shape):
        if gen is None:
            return torch.zeros(shape, dtype=torch.int32, device="cuda")
        return torch.randint(-2**31, 2**31 - 1, shape, dtype=torch.int32, device="cuda", generator=gen)

    def rows():
        x = torch.zeros((B, Hkv, G, D), dtype=torch.float16, device="cuda")
        return x if gen is None else x.normal_(generator=gen)

    s = dict(k_codes=words(num, Hkv, P, W), k_meta=words(num, Hkv, P // G, D), v_codes=words(num, Hkv, P, W),
             v_meta=words(num, Hkv, P), k_res=rows(), v_res=rows() if v_res else None)
    s.update(num=num, B=B, Hkv=Hkv, G=G, P=P, bits=bits)
    return s


def prepare(case, seed):
    op = case["op"]
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    host = random.Random(int(seed) * 7919 + 18)
    s = {"op": op}
    if op == "attention":
        lens = _lens(case, case["n_seqs"])
        T = sum(lens) + case["pad"]
        s.update(_packed(gen, T, [("q", case["Hq"]), ("k", case["Hkv"]), ("v", case["Hkv"])], case["layout"]))
        _outliers(gen, s["k"])
        s["cu"], s["scale"] = _cu(lens), 1 / math.sqrt(D)
        out = torch.zeros((T, case["Hq"], D) if case["layout"] == "tokens" else (case["Hq"], T, D),
                          dtype=torch.float16, device="cuda")
        s["out"] = out if case["layout"] == "tokens" else out.transpose(0, 1)
        return s
    if op == "quantize":
        lens, P, B = _lens(case, case["n_seqs"]), case["P"], case["n_seqs"]
        T = sum(lens) + case["pad"]
        s.update(_packed(gen, T, [("k", case["Hkv"]), ("v", case["Hkv"])], case["layout"]))
        _outliers(gen, s["k"])
        maxp = max(1, max(_ceil(n, P) for n in lens))
        num = sum(_ceil(n, P) for n in lens) + 3
        s.update(_pools(num, B, case["Hkv"], case["G"], P, case["bits"], case["v_res"]))
        s["cu"] = _cu(lens)
        ids = list(range(num))
        host.shuffle(ids)
        table = [[ids.pop() for _ in range(_ceil(n, P))] for n in lens]
        s["table"] = torch.tensor([r + [-1] * (maxp - len(r)) for r in table], dtype=torch.int32).cuda()
        s["lens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        return s
    if op == "fork":
        parent, lens = _groups(case)
        P, B = case["P"], len(parent)
        maxp = max(_ceil(n, P) for n in lens) + 1
        held = sum(_ceil(lens[b], P) for b in range(B) if parent[b] == b)
        num = held + 2 * B
        s.update(_pools(num, B, case["Hkv"], case["G"], P, 2, case["v_res"], gen))
        ids = list(range(num))
        host.shuffle(ids)
        table = [[ids.pop() for _ in range(_ceil(lens[b], P))] if parent[b] == b else [] for b in range(B)]
        refs = [0] * num
        for row in table:
            for p in row:
                refs[p] = 1
        # the rows that are replaced hold what an earlier step forked into them
        table, refs, lens, _, _ = _fork_by_hand(table, refs, [n if parent[b] == b else 0 for b, n in enumerate(lens)],
                                                parent, P, maxp)
        _ids(s, table, refs, lens, maxp)
        s["parent"] = torch.tensor(parent, dtype=torch.int32).cuda()
        return s
    lens, P, B = _lens(case, case["B"]), case["P"], case["B"]
    maxp = max(_ceil(n, P) for n in lens) + 1
    pages = sum(_ceil(n, P) for n in lens)
    num = pages + case["spare"] if op == "turnover" else max(pages + 1, int(pages / case["live"]))
    ids = list(range(num))
    host.shuffle(ids)
    table = [[ids.pop() for _ in range(_ceil(n, P))] for n in lens]
    refs = [0] * num
    for row in table:
        for p in row:
            refs[p] = 1
    if op == "turnover":
        s.update(_pools(num, B, 1, 64, P, 2, False))
        _ids(s, table, refs, lens, maxp)
        gone = [b % 4 == 1 for b in range(B)]  # every fourth sequence is done; one of its length follows
        s["parent"] = torch.tensor([-1 if g else b for b, g in enumerate(gone)], dtype=torch.int32).cuda()
        s["extra"] = torch.tensor([n if g else 0 for n, g in zip(lens, gone)], dtype=torch.int32).cuda()
        return s
    s.update(_pools(num, B, case["Hkv"], case["G"], P, 2, False, gen))
    _ids(s, table, refs, lens, maxp)
    s["new_ids"] = torch.zeros(num, dtype=torch.int32, device="cuda")
    s["start"] = (s["table"].clone(), s["refs"].clone())
    return s


def _ids(s, table, refs, lens, maxp):
    s["table"] = torch.tensor([r + [-1] * (maxp - len(r)) for r in table], dtype=torch.int32).cuda()
    s["refs"] = torch.tensor(refs, dtype=torch.int32).cuda()
    s["lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
    s["info"] = torch.zeros(4, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------- plain forms
def _plain_attention(s):
    q, k, v, out = s["q"], s["k"], s["v"], s["out"]
    R = q.shape[1] // k.shape[1]
    cu = s["cu"].tolist()
    for a, b in zip(cu[:-1], cu[1:]):
        later = torch.ones((b - a, b - a), dtype=torch.bool, device=q.device).triu(1)
        for h in range(k.shape[1]):
            qs = q[a:b, h * R:(h + 1) * R].float().transpose(0, 1)
            x = (qs @ k[a:b, h].float().t()).mul_(s["scale"])
            x.masked_fill_(later, -math.inf)
            if b > a:
                x.sub_(x.amax(-1, keepdim=True)).exp_()
            o = (x @ v[a:b, h].float()) / x.sum(-1, keepdim=True)
            out[a:b, h * R:(h + 1) * R] = o.transpose(0, 1).to(torch.float16)
    return out


def _codes(x, dim, levels):
    """Codes and {scale, zero} words of the min/max quantizer over `dim` of fp32 x."""
    mn, mx = x.amin(dim, keepdim=True), x.amax(dim, keepdim=True)
    scale = ((mx - mn) / levels).to(torch.float16)
    zero = mn.to(torch.float16) + 0.0
    s = scale.float()
    c = torch.where(s > 0, ((x - mn) / torch.where(s > 0, s, 1.0)).round().clamp(0, levels), 0.0).to(torch.int64)
    word = scale.view(torch.int16).to(torch.int64) & 0xFFFF | (zero.view(torch.int16).to(torch.int64) & 0xFFFF) << 16
    return c, _int32(word).squeeze(dim)


def _int32(w):
    return torch.where(w >= 2**31, w - 2**32, w).to(torch.int32)


def _pack(codes, bits):
    per = 32 // bits
    c = codes.reshape(*codes.shape[:-1], D // per, per)
    return _int32((c << (bits * torch.arange(per, device=c.device))).sum(-1))


def _plain_quantize(s):
    k, v, P, G, bits = s["k"], s["v"], s["P"], s["G"], s["bits"]
    levels = 2**bits - 1
    dev = k.device
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    begin = s["cu"][:-1].long()
    B = n.numel()

    def rows(count):
        """(sequence, index) of count[b] rows of every sequence b."""
        b = torch.repeat_interleave(torch.arange(B, device=dev), count)
        return b, torch.arange(b.numel(), device=dev) - (count.cumsum(0) - count)[b]

    table = s["table"].long()
    gb, gi = rows(n // G)  # key groups
    x = k[(begin[gb] + gi * G)[:, None] + torch.arange(G, device=dev)].float()  # [groups, G, Hkv, D]
    c, meta = _codes(x, 1, levels)
    page, row = table[gb, gi * G // P], gi * G % P
    s["k_codes"][page[:, None], :, row[:, None] + torch.arange(G, device=dev)] = _pack(c, bits)
    s["k_meta"][page, :, row // G] = meta
    nv = n // G * G if s["v_res"] is not None else n
    vb, vi = rows(nv)  # values, token by token
    c, meta = _codes(v[begin[vb] + vi].float(), -1, levels)
    page = table[vb, vi // P]
    s["v_codes"][page, :, vi % P] = _pack(c, bits)
    s["v_meta"][page, :, vi % P] = meta
    rb, ri = rows(n % G)  # what fills no group
    at = begin[rb] + (n // G * G)[rb] + ri
    s["k_res"][rb, :, ri] = k[at]
    if s["v_res"] is not None:
        s["v_res"][rb, :, ri] = v[at]
    s["lens"].copy_(torch.where(n > 0, n.int(), s["lens"]))
    return _cache_out(s)


def _cache_out(s):
    out = {x: s[x] for x in ("k_codes", "k_meta", "v_codes", "v_meta", "k_res", "lens", "table")}
    if s["v_res"] is not None:
        out["v_res"] = s["v_res"]
    return out


def _plain_reorder(s):
    table, refs, lens, parent = s["table"].long(), s["refs"], s["lens"].long(), s["parent"].long()
    B, maxp = table.shape
    P, G, dev = s["P"], s["G"], table.device
    me, j = torch.arange(B, device=dev), torch.arange(maxp, device=dev)
    table = torch.where((table >= 0) & (table < s["num"]), table, -1)
    valid = (parent >= 0) & (parent < B)
    src = parent.clamp(0, B - 1)
    first = torch.full((B,), B, device=dev).scatter_reduce(0, src, torch.where(valid, me, B), "amin")
    heir = torch.where(parent == me, me, first)
    is_heir = valid & (heir[src] == me)
    n = lens.clamp(0, maxp * P)[src]
    full, r = n // P, n % P
    rows = table[src]
    new = torch.where(valid[:, None] & (is_heir[:, None] | (j < full[:, None])), rows, -1)
    last = rows[me, full.clamp(max=maxp - 1)]
    wants = valid & ~is_heir & (r > 0) & (last >= 0)
    changed = (parent != me)[:, None]
    before = refs > 0
    refs.index_add_(0, table.clamp(min=0).flatten(), -((table >= 0) & changed).int().flatten())
    refs.index_add_(0, new.clamp(min=0).flatten(), ((new >= 0) & changed).int().flatten())
    freed = (before & (refs <= 0)).sum()
    free = (refs <= 0).nonzero().flatten()
    k = wants.cumsum(0) - 1
    got = wants & (k < free.numel())
    b, to = me[got], free[k[got]]
    new[b, full[b]] = to
    refs[to] = 1
    rg = r // G * G
    rv = rg if s["v_res"] is not None else r
    row = torch.arange(P, device=dev)
    for name, used, at in (("k_codes", rg, row), ("k_meta", rg // G, row[:P // G]), ("v_codes", rv, row),
                           ("v_meta", rv, row)):
        x = s[name]
        take = (at < used[b][:, None])[:, None]
        take = take[..., None] if x.dim() == 4 else take
        x[to] = torch.where(take, x[last[b]], x[to])
    slot = (torch.arange(G, device=dev) < (n % G)[:, None]) & changed & valid[:, None]
    for name in ("k_res", "v_res"):
        if s[name] is not None:
            s[name].copy_(torch.where(slot[:, None, :, None], s[name][src], s[name]))
    n = torch.where(valid, torch.where(wants & ~got, full * P, n), 0)
    s["lens"].copy_(torch.where(changed[:, 0], n, lens))
    s["table"].copy_(new)
    s["info"].copy_(torch.stack([got.sum(), wants.sum() - got.sum(), (refs > 0).sum(), freed]))


def _plain_reserve(s):
    table, refs, P = s["table"], s["refs"], s["P"]
    B, maxp = table.shape
    want = torch.where(s["extra"] > 0, (s["lens"].clamp(min=0) + s["extra"]).clamp(max=maxp * P), 0)
    need = (torch.arange(maxp, device=table.device) < ((want + P - 1) // P)[:, None])
    need &= (table < 0) | (table >= s["num"])
    at = need.flatten().nonzero().flatten()
    free = (refs <= 0).nonzero().flatten()[:at.numel()]
    got = free.numel()
    table.view(-1)[at[:got]] = free.int()
    refs[free] = 1
    s["info"].copy_(torch.stack([torch.tensor(x, device=table.device) for x in (got, at.numel() - got)] +
                                [(refs > 0).sum(), torch.zeros_like(at.sum())]))


def _plain_compact(s):
    table, refs = s["table"], s["refs"]
    num, dev = s["num"], table.device
    live = refs > 0
    L = int(live.sum())
    ids = torch.arange(num, device=dev)
    movers, holes = (live & (ids >= L)).nonzero().flatten(), (~live & (ids < L)).nonzero().flatten()
    new = torch.where(live, ids, -1)
    new[movers] = holes
    for name in ("k_codes", "k_meta", "v_codes", "v_meta"):
        s[name][holes] = s[name][movers]
    refs[holes] = refs[movers]
    refs.copy_(torch.where(ids < L, refs, 0))
    inside = (table >= 0) & (table < num)
    table.copy_(torch.where(inside, new[table.clamp(0, num - 1).long()].int(), -1))
    s["new_ids"].copy_(new)
    s["info"].copy_(torch.tensor([movers.numel(), 0, L, 0]))


# --------------------------------------------------------------------------- a pass
def _handles(s):
    """The cache and pool handles that a serving loop keeps beside its buffers."""
    if "cache" not in s:
        from bit_asymmetric_kv_gb300 import kivi
        dims = kivi.make_paged_dims(s["B"], s["Hkv"], s["G"], s["P"], s["table"].shape[1], s["num"], bits=s["bits"],
                                    value_residual=s["v_res"] is not None)
        t = [s[x] for x in ("k_codes", "k_meta", "v_codes", "v_meta", "k_res")]
        c = kivi.kivi_paged_cache(*[x.data_ptr() for x in t], 0 if s["v_res"] is None else s["v_res"].data_ptr(),
                                  s["table"].data_ptr(), s["lens"].data_ptr())
        s["cache"] = kivi.PagedCache(dims, *t, s["table"], s["lens"], c, s["v_res"])
        if "refs" in s:
            s["pool"] = kivi.PagePool.adopt(s["cache"], s["refs"], s["info"])
    return s["cache"], s.get("pool")


def run(s):
    op = s["op"]
    if op == "attention":
        if own:
            from bit_asymmetric_kv_gb300 import kivi
            return kivi.kivi_prefill_attention_packed(s["q"], s["k"], s["v"], s["cu"], s["scale"], out=s["out"])
        return _plain_attention(s)
    if op == "quantize":
        if own:
            from bit_asymmetric_kv_gb300 import kivi
            kivi.kivi_paged_prefill_packed(_handles(s)[0], s["k"], s["v"], s["cu"])
            return _cache_out(s)
        return _plain_quantize(s)
    out = {x: s[x] for x in ("table", "refs", "lens", "info")}
    if op == "compact":  # the fragmented table and counts that every pass starts from
        s["table"].copy_(s["start"][0])
        s["refs"].copy_(s["start"][1])
    if own:
        from bit_asymmetric_kv_gb300 import kivi
        cache, pool = _handles(s)
        if op == "compact":
            kivi.kivi_paged_compact(cache, pool, s["new_ids"])
        else:
            kivi.kivi_paged_reorder(cache, pool, s["parent"])
            if op == "turnover":
                kivi.kivi_paged_reserve(cache, pool, s["extra"])
    elif op == "compact":
        _plain_compact(s)
    else:
        _plain_reorder(s)
        if op == "turnover":
            _plain_reserve(s)
    if op == "turnover":
        return out
    if op == "compact":
        out["new_ids"] = s["new_ids"]
    return {**out, **_cache_out(s)}


# ------------------------------------------------------------ the definition in 64 bits
def _fork_by_hand(table, refs, lens, parent, P, maxp):
    """The reorder of page ids, row by row: (table, refs, lens, info, copies), copies as
    (row, source row, from page, to page) with pages None where nothing is copied."""
    refs = list(refs)
    live = sum(r > 0 for r in refs)
    heirs = {}
    for b, p in enumerate(parent):
        if p == b:
            heirs[b] = b
    for b, p in enumerate(parent):
        if 0 <= p < len(parent):
            heirs.setdefault(p, b)
    new, new_lens, split = [], [], []
    for b, p in enumerate(parent):
        if not 0 <= p < len(parent):
            new.append([])
            new_lens.append(0)
            continue
        n = lens[p]
        new_lens.append(n)
        if heirs[p] == b:
            new.append(list(table[p]))
        else:
            new.append(list(table[p][:n // P]))
            if n % P and len(table[p]) > n // P:
                split.append(b)
    for b, p in enumerate(parent):
        if p != b:
            for x in table[b]:
                refs[x] -= 1
            for x in new[b]:
                refs[x] += 1
    freed = live - sum(r > 0 for r in refs)
    free = [i for i, r in enumerate(refs) if r <= 0]
    pages, got = {}, 0
    for b in split:
        p, n = parent[b], new_lens[b]
        if got < len(free):
            refs[free[got]] = 1
            new[b].append(free[got])
            pages[b] = (table[p][n // P], free[got])
            got += 1
        else:
            new_lens[b] = n // P * P
    copies = [(b, p) + pages.get(b, (None, None)) for b, p in enumerate(parent) if p != b and 0 <= p < len(parent)]
    info = [got, len(split) - got, sum(r > 0 for r in refs), freed]
    return new, refs, new_lens, info, copies


def _rows_of(t):
    return [[x for x in row if x >= 0] for row in t.tolist()]


def _exact_attention(case, s):
    q, k, v = (s[x].double() for x in "qkv")
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    R = case["Hq"] // case["Hkv"]
    cu = s["cu"].tolist()
    for i in range(len(cu) - 1):
        for r0 in range(cu[i], cu[i + 1], 1024):  # rows r0 .. r1 see the keys up to their own
            r1 = min(r0 + 1024, cu[i + 1])
            keys = torch.arange(cu[i], r1, device="cuda")
            seen = keys[None, :] <= torch.arange(r0, r1, device="cuda")[:, None]
            for h in range(case["Hq"]):
                x = torch.einsum("id,jd->ij", q[r0:r1, h], k[cu[i]:r1, h // R]) * s["scale"]
                w = torch.softmax(torch.where(seen, x, -torch.inf), -1)
                out[r0:r1, h] = torch.einsum("ij,jd->id", w, v[cu[i]:r1, h // R])
    return out


def _exact_quantize(case, s):
    """Sequence by sequence.  Every fp32 operation of the quantizer's definition is one operation in 64
    bits rounded to fp32, which gives the same value."""
    levels, bits, P, G = 2 ** case["bits"] - 1, case["bits"], case["P"], case["G"]

    def f32(x):
        return x.float().double()

    def quantized(x, dim):
        mn, mx = x.min(dim, keepdim=True).values, x.max(dim, keepdim=True).values
        sc = f32(f32(mx - mn) / levels).half()
        c = torch.round(f32(f32(x - mn) / sc.double().clamp_min(1e-30))).clamp(0, levels)
        c = torch.where(sc > 0, c, 0).long()
        z = torch.where(mn == 0, 0.0, mn).half()
        meta = (sc.view(torch.int16).long() & 65535) + ((z.view(torch.int16).long() & 65535) << 16)
        packed = torch.zeros((*x.shape[:-1], D * bits // 32), dtype=torch.int64, device=x.device)
        for ch in range(D):
            packed[..., ch * bits // 32] += c[..., ch] << (ch * bits % 32)
        return [torch.where(w > 2**31 - 1, w - 2**32, w).int() for w in (packed, meta.squeeze(dim))]

    cu, table = s["cu"].tolist(), s["table"].tolist()
    for b in range(case["n_seqs"]):
        n = cu[b + 1] - cu[b]
        ks, vs = s["k"][cu[b]:cu[b + 1]], s["v"][cu[b]:cu[b + 1]]
        for t0 in range(0, n, P):
            m, page = min(P, n - t0), table[b][t0 // P]
            g = m // G
            if g:
                x = ks[t0:t0 + g * G].double().reshape(g, G, case["Hkv"], D)
                c, meta = quantized(x, 1)
                s["k_codes"][page, :, :g * G] = c.reshape(g * G, case["Hkv"], -1).transpose(0, 1)
                s["k_meta"][page, :, :g] = meta.transpose(0, 1)
            m = g * G if case["v_res"] else m
            c, meta = quantized(vs[t0:t0 + m].double(), -1)
            s["v_codes"][page, :, :m] = c.transpose(0, 1)
            s["v_meta"][page, :, :m] = meta.transpose(0, 1)
        r = n % G
        if r:
            s["k_res"][b, :, :r] = ks[n - r:].transpose(0, 1)
            if case["v_res"]:
                s["v_res"][b, :, :r] = vs[n - r:].transpose(0, 1)
        if n:
            s["lens"][b] = n
    out = _cache_out(s)
    return {x: t.double() if t.is_floating_point() else t for x, t in out.items()}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "attention":
        return _exact_attention(case, s)
    if op == "quantize":
        return _exact_quantize(case, s)
    P, maxp = case["P"], s["table"].shape[1]
    table, refs, lens = _rows_of(s["table"]), s["refs"].tolist(), s["lens"].tolist()
    if op == "compact":
        live = [i for i, r in enumerate(refs) if r > 0]
        L = len(live)
        holes = iter([i for i, r in enumerate(refs) if r <= 0 and i < L])
        new = [-1] * s["num"]
        for i in live:
            new[i] = i if i < L else next(holes)
            if i >= L:
                for name in ("k_codes", "k_meta", "v_codes", "v_meta"):
                    s[name][new[i]] = s[name][i]
        counts = [0] * s["num"]
        for i in live:
            counts[new[i]] = refs[i]
        _ids(s, [[new[p] for p in row] for row in table], counts, lens, maxp)
        s["info"] = torch.tensor([sum(i >= L for i in live), 0, L, 0], dtype=torch.int32)
        s["new_ids"] = torch.tensor(new, dtype=torch.int32)
    else:
        parent = s["parent"].tolist()
        table, refs, lens, info, copies = _fork_by_hand(table, refs, lens, parent, P, maxp)
        old = s["k_res"].clone(), None if s["v_res"] is None else s["v_res"].clone()
        for b, p, a, z in copies:
            n, G = lens[p], case.get("G", 64)
            r, rg = n % P, n % P // G * G
            rv = rg if s["v_res"] is not None else r
            if z is not None:
                for name, used in (("k_codes", rg), ("k_meta", rg // G), ("v_codes", rv), ("v_meta", rv)):
                    s[name][z, :, :used] = s[name][a, :, :used]
            s["k_res"][b, :, :n % G] = old[0][p, :, :n % G]
            if s["v_res"] is not None:
                s["v_res"][b, :, :n % G] = old[1][p, :, :n % G]
        if op == "turnover":
            free = [i for i, r in enumerate(refs) if r <= 0]
            got = missing = 0
            for b, e in enumerate(s["extra"].tolist()):
                while e > 0 and len(table[b]) * P < lens[b] + e:
                    if got == len(free):
                        missing += 1
                        break
                    refs[free[got]] = 1
                    table[b].append(free[got])
                    got += 1
            info = [got, missing, sum(r > 0 for r in refs), 0]
        _ids(s, table, refs, lens, maxp)
        s["info"] = torch.tensor(info, dtype=torch.int32)
    out = {x: s[x] for x in ("table", "refs", "lens", "info")}
    if op == "turnover":
        return out
    if op == "compact":
        out["new_ids"] = s["new_ids"]
    out = {**out, **{x: t for x, t in _cache_out(s).items() if x not in out}}
    return {x: t.double() if t.is_floating_point() else t for x, t in out.items()}

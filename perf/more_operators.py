"""Cases of the sliding-window operators of the KIVI cache, for measuring them.

Operators (a query at position p sees position j when p - window < j <= p or j < sinks):
  attention  prompts, or chunks behind earlier tokens, packed into one token axis
  decode     one new token of every sequence over the quantized pages
  extend     chunks of new keys and values quantized into the pages behind what a sequence holds
  read       the newest tokens of every sequence (and its first ones) read back from the pages
  reserve    pages out of the window's reach given back, pages for the tokens to come handed out

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
        dict(name="attention-few-tokens", op="attention", n_seqs=3, lo=1, hi=64, olo=0, ohi=0, Hq=4, Hkv=1, window=32,
             sinks=4, layout="tokens", pad=0),
        # chunked prefill: the next chunk of every long prompt over the sinks, the window and itself
        dict(name="attention-chunks-gqa", op="attention", n_seqs=16, lo=200, hi=512, olo=500, ohi=4099, Hq=32, Hkv=8,
             window=4096, sinks=4, layout="tokens", pad=60),
        # ragged Llama-2-7B-shaped prompts, head-major, a short window and sinks
        dict(name="attention-ragged-mha", op="attention", n_seqs=8, lo=700, hi=4113, olo=0, ohi=0, Hq=32, Hkv=32,
             window=1024, sinks=4, layout="heads", pad=0),
        # two long documents, Mistral-7B-shaped heads and window
        dict(name="attention-long-gqa", op="attention", n_seqs=2, lo=8200, hi=16384, olo=0, ohi=0, Hq=32, Hkv=8,
             window=4096, sinks=0, layout="tokens", pad=0),
        # a step of a few chats on a small model
        dict(name="decode-small", op="decode", B=4, lo=10, hi=1500, Hq=8, Hkv=2, G=32, P=64, bits=2, v_res=False,
             window=256, sinks=4),
        # a step of a full Mistral-7B-shaped batch whose older pages are gone
        dict(name="decode-batch-gqa", op="decode", B=64, lo=100, hi=32808, Hq=32, Hkv=8, G=64, P=128, bits=2,
             v_res=False, window=4096, sinks=4),
        # 64 draft tokens' acceptance: a few tokens for every sequence
        dict(name="extend-drafts", op="extend", B=64, lo=1, hi=8, olo=30, ohi=2000, Hkv=8, G=32, P=64, bits=2,
             v_res=False, layout="tokens", pad=0),
        # the next chunk of long prompts, 4-bit codes
        dict(name="extend-chunks", op="extend", B=32, lo=500, hi=2048, olo=100, ohi=4000, Hkv=8, G=64, P=128, bits=4,
             v_res=False, layout="tokens", pad=0),
        # what a few short chats hold
        dict(name="read-small", op="read", B=4, lo=5, hi=300, Hkv=2, G=32, P=64, bits=2, v_res=True, take=256, first=4),
        # sinks and window of a full batch, for the next chunk's attention
        dict(name="read-window", op="read", B=32, lo=300, hi=16384, Hkv=8, G=64, P=128, bits=2, v_res=False, take=4099,
             first=4),
        # a small server's step
        dict(name="reserve-small", op="reserve", B=8, lo=20, hi=1000, P=64, window=256, sinks=4, step=1, spare=64),
        # a full server: chunks of 512 admitted, windows moved on
        dict(name="reserve-large", op="reserve", B=512, lo=100, hi=32768, P=64, window=4096, sinks=4, step=512,
             spare=4000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "decode", "decode", "extend", "read", "reserve"])
    layout = rng.choice(["tokens", "heads"])
    sinks = rng.choice([0, 1, 4, 4, 64, 100, 200])
    G, P, bits, v_res = rng.choice([32, 64]), rng.choice([64, 128, 256]), rng.choice([2, 4]), rng.random() < 0.3
    if op == "attention":
        Hkv = rng.choice([1, 2, 4, 8, 32])
        R = rng.choice([1, 2, 3, 4, 8]) if Hkv < 8 else rng.choice([1, 4]) if Hkv == 8 else 1
        hi = _log(rng, 2, 6000)
        ohi = rng.choice([0, 0, _log(rng, 1, 5000)])
        n_seqs = max(1, min(_log(rng, 1, 128), 24000 // hi, 48000 // (hi + ohi)))
        return dict(op=op, n_seqs=n_seqs, lo=max(1, int(hi * rng.random())), hi=hi, olo=int(ohi * rng.random()),
                    ohi=ohi, Hq=R * Hkv, Hkv=Hkv, window=_log(rng, 1, 8000), sinks=sinks, layout=layout,
                    pad=rng.choice([0, 1, 63, 200]))
    if op == "reserve":
        return dict(op=op, B=_log(rng, 1, 512), lo=rng.randrange(1, 200), hi=_log(rng, 200, 30000), P=P,
                    window=_log(rng, 1, 8000), sinks=sinks, step=_log(rng, 1, 512), spare=_log(rng, 1, 4000))
    B, Hkv = _log(rng, 1, 64), rng.choice([1, 2, 3, 8])
    if op == "decode":
        return dict(op=op, B=B, lo=rng.randrange(1, 400), hi=_log(rng, 400, 30000), Hq=Hkv * rng.choice([1, 2, 4]),
                    Hkv=Hkv, G=G, P=P, bits=bits, v_res=v_res, window=_log(rng, 1, 4096), sinks=sinks)
    if op == "extend":
        ohi = _log(rng, 2, 4000)
        hi = _log(rng, 1, 2000)
        return dict(op=op, B=max(1, min(B, 30000 // hi)), lo=max(1, int(hi * rng.random())), hi=hi,
                    olo=rng.randrange(1, ohi + 1), ohi=ohi, Hkv=Hkv, G=G, P=P, bits=bits, v_res=v_res, layout=layout,
                    pad=rng.choice([0, 5, 300]))
    return dict(op=op, B=min(B, 32), lo=rng.randrange(1, 300), hi=_log(rng, 300, 16000), Hkv=Hkv, G=G, P=P, bits=bits,
                v_res=v_res, take=_log(rng, 1, 4099), first=sinks)


def _lens(n, lo, hi, salt=""):
    """The smallest and the largest length, the rest spread over their logarithm; one sequence in ten
    has no tokens."""
    r = random.Random("%s %d %d %d" % (salt, n, lo, hi))
    lens = [hi, lo] + [_log(r, max(1, lo), max(1, hi)) for _ in range(n)]
    lens = [0 if i % 10 == 9 else x for i, x in enumerate(lens[:n])]
    r.shuffle(lens)
    return lens


def _chunks(case, n):
    """(new, earlier) tokens of every sequence."""
    return (_lens(n, case["lo"], case["hi"]),
            _lens(n, case["olo"], case["ohi"], "earlier") if case["ohi"] else [0] * n)


def _seen(p, window, sinks):
    """Positions that a query at position p sees."""
    return min(p + 1, window) + min(sinks, max(0, p + 1 - window))


def _dead(n, P, window, sinks):
    """Pages [a, b) of a sequence of n tokens that no token to come sees."""
    return -(-sinks // P), max(-(-sinks // P), max(0, n - window + 1) // P)


def work(case):
    op = case["op"]
    if op == "attention":
        new, old = _chunks(case, case["n_seqs"])
        pairs = sum(_seen(o + i, case["window"], case["sinks"]) for n, o in zip(new, old) for i in range(n))
        rows = sum(n + min(o, case["window"] - 1 + case["sinks"]) for n, o in zip(new, old) if n)
        return {"bytes": 256 * (2 * sum(new) * case["Hq"] + 2 * rows * case["Hkv"]), "flops": 4 * D * case["Hq"] * pairs}
    if op == "reserve":
        lens, P, entries = _lens(case["B"], case["lo"], case["hi"]), case["P"], 0
        for n in lens:
            a, b = _dead(n, P, case["window"], case["sinks"])
            entries += -(-(n + case["step"]) // P) - max(0, b - a)
        return {"bytes": 4 * entries + 4 * (entries + case["spare"]) + 12 * len(lens), "flops": 0}
    G, per = case["G"], 16 * case["bits"]
    held = 0

    def rows(a, n, res):
        """Bytes of what positions a .. n - 1 of a sequence of n tokens hold, keys and values."""
        nq = n // G * G
        nv = nq if res else n
        k, v = max(0, nq - a), max(0, nv - a)
        return k * per + -(-k // G) * 512 + v * (per + 4) + (n - max(a, nq)) * 256 + (n - max(a, nv)) * 256

    if op == "decode":
        lens, pairs = _lens(case["B"], case["lo"], case["hi"]), 0
        for n in lens:
            if n:
                seen = _seen(n - 1, case["window"], case["sinks"])
                tail = min(n, case["window"])
                pairs += seen
                held += rows(n - tail, n, case["v_res"]) + (seen - tail) * (2 * per + 4) + -(-(seen - tail) // G) * 512
        return {"bytes": case["Hkv"] * held + 512 * case["B"] * case["Hq"], "flops": 4 * D * case["Hq"] * pairs}
    if op == "extend":
        new, old = _chunks(case, case["B"])
        for n, o in zip(new, old):
            if n:
                q0, q1 = o // G * G, (o + n) // G * G
                used = (o - q0) * 256 if q1 > q0 else 0  # the residual that is quantized
                held += rows(q0, o + n, case["v_res"]) - ((o - q0) * (per + 4) if not case["v_res"] else 0)
                held += used * (2 if case["v_res"] else 1) + 512 * n - (0 if q1 > q0 else (o - q0) * 256 * (2 if case["v_res"] else 1))
        return {"bytes": case["Hkv"] * held, "flops": 0}
    for n in _lens(case["B"], case["lo"], case["hi"]):
        c = min(n, case["take"])
        f = min(case["first"], c) if c < n else 0
        held += rows(n - (c - f), n, case["v_res"]) + f * (2 * per + 4) + -(-f // G) * 512 + 512 * c
    return {"bytes": case["Hkv"] * held, "flops": 0}


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
    """Two fixed outlier channels of every head of keys [.., heads, .., D] (heads at axis 1)."""
    for h in range(k.shape[1]):
        c = torch.randperm(D, generator=gen, device="cuda")[:2]
        f = 20 + 20 * torch.rand(2, generator=gen, device="cuda")
        k[:, h, ..., c] = (k[:, h, ..., c].float() * f).to(torch.float16)


def _cu(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()


def _ceil(a, b):
    return -(-a // b)


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


def _cache(s, case, gen, host, lens, rooms, first_page, filled):
    """Pages, tables and residuals of sequences of `lens` tokens with table entries for `rooms` tokens;
    entries for which first_page(n) = (a, b) gives a <= entry < b hold no page.  Where `filled`, the pages
    hold quantized keys (with outlier channels) and values, else they are empty (zero)."""
    Hkv, G, P, bits, B = case["Hkv"], case["G"], case["P"], case["bits"], len(lens)
    maxp = max(1, max(_ceil(r, P) for r in rooms))
    rows = []
    for n, r in zip(lens, rooms):
        a, b = first_page(n)
        rows.append([0 if a <= j < b or j >= _ceil(r, P) else 1 for j in range(maxp)])
    num = sum(map(sum, rows)) + 3
    ids = list(range(num))
    host.shuffle(ids)
    s["table"] = torch.tensor([[ids.pop() if x else -1 for x in row] for row in rows], dtype=torch.int32).cuda()
    s["lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
    W = D * bits // 32
    for name, shape in (("k_codes", (num, Hkv, P, W)), ("k_meta", (num, Hkv, P // G, D)), ("v_codes", (num, Hkv, P, W)),
                        ("v_meta", (num, Hkv, P))):
        s[name] = torch.zeros(shape, dtype=torch.int32, device="cuda")
    scale = torch.ones((1, Hkv, 1, D), device="cuda")
    for h in range(Hkv):
        c = torch.randperm(D, generator=gen, device="cuda")[:2]
        scale[0, h, 0, c] = 20 + 20 * torch.rand(2, generator=gen, device="cuda")

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    s["k_res"] = (normal(B, Hkv, G, D) * scale).to(torch.float16)
    s["v_res"] = normal(B, Hkv, G, D).to(torch.float16) if case["v_res"] else None
    if filled:
        slab = max(1, (1 << 26) // (Hkv * P * D))
        for a in range(0, num, slab):
            m = min(slab, num - a)
            x = (normal(m, Hkv, P, D) * scale).half().float().view(m, Hkv, P // G, G, D)
            c, s["k_meta"][a:a + m] = _codes(x, 3, 2**bits - 1)
            s["k_codes"][a:a + m] = _pack(c, bits).view(m, Hkv, P, W)
            c, s["v_meta"][a:a + m] = _codes(normal(m, Hkv, P, D).half().float(), -1, 2**bits - 1)
            s["v_codes"][a:a + m] = _pack(c, bits)
    s.update(B=B, Hkv=Hkv, G=G, P=P, bits=bits, num=num)


def prepare(case, seed):
    op = case["op"]
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 23)
    host = random.Random(int(seed) * 7919 + 24)
    s = {"op": op}
    if op == "attention":
        new, old = _chunks(case, case["n_seqs"])
        T, pad, heads = sum(new), case["pad"], [("k", case["Hkv"]), ("v", case["Hkv"])]
        if case["ohi"]:
            s.update(_packed(gen, T + pad, [("q", case["Hq"])], case["layout"]))
            s.update(_packed(gen, T + sum(old) + pad, heads, case["layout"]))
        else:
            s.update(_packed(gen, T + pad, [("q", case["Hq"])] + heads, case["layout"]))
        _outliers(gen, s["k"])
        s["cu"], s["cu_kv"] = _cu(new), _cu([n + o for n, o in zip(new, old)]) if case["ohi"] else None
        s.update(window=case["window"], sinks=case["sinks"], scale=1 / math.sqrt(D), Lq=max(new),
                 Lk=max(n + o for n, o in zip(new, old)))
        shape = (T + pad, case["Hq"], D) if case["layout"] == "tokens" else (case["Hq"], T + pad, D)
        out = torch.zeros(shape, dtype=torch.float16, device="cuda")
        s["out"] = out if case["layout"] == "tokens" else out.transpose(0, 1)
        return s
    if op == "reserve":
        P, step = case["P"], case["step"]
        lens = _lens(case["B"], case["lo"], case["hi"])
        maxp = max(_ceil(n + step, P) for n in lens)
        # what the step before left: its window, ending at most one step earlier
        rows = []
        for n in lens:
            a, b = _dead(max(0, n - step), P, case["window"], case["sinks"])
            rows.append([j < _ceil(n, P) and not a <= j < b for j in range(maxp)])
        num = sum(map(sum, rows)) + case["spare"]
        ids = list(range(num))
        host.shuffle(ids)
        refs, table = [0] * num, []
        for row in rows:
            table.append([ids.pop() if x else -1 for x in row])
            for p in table[-1]:
                if p >= 0:
                    refs[p] = 1
        s["lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
        s["extra"] = torch.tensor([step if i % 16 else 0 for i in range(len(lens))], dtype=torch.int32).cuda()
        s["start"] = (torch.tensor(table, dtype=torch.int32).cuda(), torch.tensor(refs, dtype=torch.int32).cuda())
        s["table"], s["refs"] = s["start"][0].clone(), s["start"][1].clone()
        s["info"] = torch.zeros(4, dtype=torch.int32, device="cuda")
        s.update(B=len(lens), Hkv=1, G=64, P=P, bits=2, num=num, window=case["window"], sinks=case["sinks"], v_res=None)
        for name, shape in (("k_codes", (num, 1, P, 8)), ("k_meta", (num, 1, P // 64, D)), ("v_codes", (num, 1, P, 8)),
                            ("v_meta", (num, 1, P)), ("k_res", (len(lens), 1, 64, D))):
            s[name] = torch.zeros(shape, dtype=torch.float16 if name == "k_res" else torch.int32, device="cuda")
        return s
    if op == "decode":
        lens = _lens(case["B"], case["lo"], case["hi"])
        _cache(s, case, gen, host, lens, lens, lambda n: _dead(n - 1, case["P"], case["window"], case["sinks"]), True)
        s["q"] = torch.randn((case["B"], case["Hq"], D), generator=gen, device="cuda").to(torch.float16)
        s["out"] = torch.zeros_like(s["q"])
        s.update(window=case["window"], sinks=case["sinks"], scale=1 / math.sqrt(D))
        return s
    if op == "extend":
        new, old = _chunks(case, case["B"])
        _cache(s, case, gen, host, old, [n + o for n, o in zip(new, old)], lambda n: (0, 0), False)
        s.update(_packed(gen, sum(new) + case["pad"], [("k", case["Hkv"]), ("v", case["Hkv"])], case["layout"]))
        _outliers(gen, s["k"])
        s["cu"] = _cu(new)
        s["start"] = [(s[x], s[x].clone()) for x in ("lens", "k_res", "v_res") if s[x] is not None]
        return s
    lens = _lens(case["B"], case["lo"], case["hi"])
    took = [min(n, case["take"]) for n in lens]
    # the pages between the first tokens and the newest ones are gone
    _cache(s, case, gen, host, lens, lens,
           lambda n: (_ceil(case["first"], case["P"]), max(0, n - case["take"]) // case["P"]), True)
    s["cu"], s["take"] = _cu(took), torch.tensor(took, dtype=torch.int32).cuda()
    s["first"], s["T"] = case["first"], sum(took)
    s["k_out"], s["v_out"] = (torch.zeros((sum(took), case["Hkv"], D), dtype=torch.float16, device="cuda") for _ in "kv")
    return s


# ---------------------------------------------------------------------- plain forms
def _plain_attention(s):
    q, k, v, out, dev = s["q"], s["k"], s["v"], s["out"], s["q"].device
    R = q.shape[1] // k.shape[1]
    cu = s["cu"].long()
    ck = cu if s["cu_kv"] is None else s["cu_kv"].long()
    n, m = cu.diff(), ck.diff()
    i, j = torch.arange(s["Lq"], device=dev), torch.arange(s["Lk"], device=dev)
    pos = i + (m - n)[:, None]
    seen = (j <= pos[..., None]) & ((j > pos[..., None] - s["window"]) | (j < s["sinks"]))
    hidden = ~seen[:, None]
    b, at = (i < n[:, None]).nonzero(as_tuple=True)
    rows = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)
    keys = (ck[:-1, None] + j).clamp(max=k.shape[0] - 1)
    for h in range(k.shape[1]):
        qs = q[rows, h * R:(h + 1) * R].float().transpose(1, 2)             # [B, R, Lq, D]
        x = qs @ (k[keys, h].float().transpose(1, 2) * s["scale"])[:, None]  # [B, R, Lq, Lk]
        x.masked_fill_(hidden, -math.inf)
        x.sub_(x.amax(-1, keepdim=True).clamp(min=-1e38)).exp_()
        o = (x @ v[keys, h].float()[:, None]) / x.sum(-1, keepdim=True).clamp(min=1e-38)
        out[cu[b] + at, h * R:(h + 1) * R] = o.transpose(1, 2)[b, at].to(torch.float16)
    return out


def _tokens(s, b, p):
    """fp32 keys and values [.., Hkv, D] at positions p of sequences b."""
    P, G, bits, dev = s["P"], s["G"], s["bits"], s["table"].device
    shift = bits * torch.arange(32 // bits, device=dev, dtype=torch.int32)

    def halves(w):
        return (w & 0xFFFF).to(torch.int16).view(torch.float16).float(), (w >> 16).to(torch.int16).view(torch.float16).float()

    def codes(w):
        return ((w[..., None] >> shift) & (2**bits - 1)).flatten(-2).float()

    lens = s["lens"].long().clamp(min=0)
    page, row = s["table"].long()[b, p // P].clamp(min=0), p % P
    late = (p >= (lens // G * G)[b])[..., None, None]
    sc, z = halves(s["k_meta"][page, :, row // G])
    k = torch.where(late, s["k_res"][b, :, p % G].float(), codes(s["k_codes"][page, :, row]) * sc + z)
    sc, z = halves(s["v_meta"][page, :, row])
    v = codes(s["v_codes"][page, :, row]) * sc[..., None] + z[..., None]
    if s["v_res"] is not None:
        v = torch.where(late, s["v_res"][b, :, p % G].float(), v)
    return k, v


def _plain_decode(s):
    q, dev = s["q"], s["q"].device
    n, W, S = s["lens"].long()[:, None], s["window"], s["sinks"]
    W = min(W, s["table"].shape[1] * s["P"])
    p = torch.cat([torch.arange(S, device=dev).expand(n.shape[0], S), n - W + torch.arange(W, device=dev)], 1)
    first = torch.arange(S + W, device=dev) < S
    seen = torch.where(first, p < n, (p >= S) & (p >= 0))
    b = torch.arange(n.shape[0], device=dev)[:, None]
    k, v = _tokens(s, b, p.clamp(min=0).minimum((n - 1).clamp(min=0)))      # [B, L, Hkv, D]
    qs = q.float().view(n.shape[0], s["Hkv"], -1, D) * s["scale"]
    x = qs @ k.permute(0, 2, 3, 1)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True).clamp(min=-1e38)).exp_()
    o = (x @ v.transpose(1, 2)) / x.sum(-1, keepdim=True).clamp(min=1e-38)
    s["out"].copy_(o.view(q.shape))
    return s["out"]


def _rows(count):
    """(sequence, index) of count[b] rows of every sequence b."""
    b = torch.repeat_interleave(torch.arange(count.numel(), device=count.device), count)
    return b, torch.arange(b.numel(), device=count.device) - (count.cumsum(0) - count)[b]


def _plain_extend(s):
    k, v, P, G, bits = s["k"], s["v"], s["P"], s["G"], s["bits"]
    B, Hkv, T, dev = s["B"], s["Hkv"], k.shape[0], k.device
    levels = 2**bits - 1
    begin, m, n = s["cu"][:-1].long(), s["cu"].diff().long(), s["lens"].long()
    end = n + m
    table = s["table"].long()
    # every row that is used: the new ones, then the residuals'
    keys = torch.cat([k, s["k_res"].transpose(1, 2).reshape(B * G, Hkv, D)])
    values = v if s["v_res"] is None else torch.cat([v, s["v_res"].transpose(1, 2).reshape(B * G, Hkv, D)])

    def row(b, p):
        return torch.where(p >= n[b], begin[b] + p - n[b], T + b * G + p % G)

    gb, gi = _rows((end // G - n // G) * (m > 0))  # key groups that fill
    p = ((n // G)[gb] + gi) * G
    c, meta = _codes(keys[row(gb[:, None], p[:, None] + torch.arange(G, device=dev))].float(), 1, levels)
    page, at = table[gb, p // P], p % P
    s["k_codes"][page[:, None], :, at[:, None] + torch.arange(G, device=dev)] = _pack(c, bits)
    s["k_meta"][page, :, at // G] = meta
    if s["v_res"] is None:
        vb, p = _rows(m)
        p = p + n[vb]
    else:
        vb, p = _rows((end // G - n // G) * G * (m > 0))
        p = p + (n // G * G)[vb]
    c, meta = _codes(values[row(vb, p)].float(), -1, levels)
    page = table[vb, p // P]
    s["v_codes"][page, :, p % P] = _pack(c, bits)
    s["v_meta"][page, :, p % P] = meta
    rb, p = _rows(torch.minimum(m, end % G))  # new tokens that fill no group
    p = p + (end - torch.minimum(m, end % G))[rb]
    s["k_res"][rb, :, p % G] = k[begin[rb] + p - n[rb]]
    if s["v_res"] is not None:
        s["v_res"][rb, :, p % G] = v[begin[rb] + p - n[rb]]
    s["lens"].copy_(end)


def _plain_read(s):
    dev = s["table"].device
    take, n = s["take"].long(), s["lens"].long()
    b, i = _rows(take)
    p = torch.where(i < s["first"], i, n[b] - take[b] + i)
    k, v = _tokens(s, b, p)
    at = s["cu"].long()[b] + i
    s["k_out"][at] = k.clamp(-65504, 65504).to(torch.float16)
    s["v_out"][at] = v.clamp(-65504, 65504).to(torch.float16)
    return [s["k_out"], s["v_out"]]


def _plain_reserve(s):
    table, refs, P = s["table"], s["refs"], s["P"]
    maxp, dev = table.shape[1], table.device
    lens, go = s["lens"].clamp(min=0)[:, None], (s["extra"] > 0)[:, None]
    j = torch.arange(maxp, device=dev)
    inside = (table >= 0) & (table < s["num"])
    dead = go & (j * P >= s["sinks"]) & ((j + 1) * P <= lens - s["window"] + 1)
    before = (refs > 0).sum()
    refs.index_add_(0, table.clamp(0, s["num"] - 1).flatten(), -(inside & dead).int().flatten())
    table.masked_fill_(dead, -1)
    freed = before - (refs > 0).sum()
    want = torch.where(go, (lens + s["extra"][:, None]).clamp(max=maxp * P), 0)
    need = (j < (want + P - 1) // P) & ~dead & ~inside
    at = need.flatten()
    free = refs <= 0
    rank = at.cumsum(0) - 1
    have = free.sum()
    ids = free.nonzero().flatten()
    got = at & (rank < have)
    where = got.nonzero().flatten()
    table.view(-1)[where] = ids[:where.numel()].int()
    refs[ids[:where.numel()]] = 1
    s["info"].copy_(torch.stack([got.sum(), at.sum() - got.sum(), (refs > 0).sum(), freed]))


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
        if "q" in s:
            s["ws"] = kivi.paged_workspace(s["cache"], s["q"].shape[1])
    return s["cache"]


def run(s):
    op = s["op"]
    if op == "attention":
        if own:
            from bit_asymmetric_kv_gb300 import kivi
            return kivi.kivi_prefill_attention_window(s["q"], s["k"], s["v"], s["cu"], s["window"], s["sinks"],
                                                      s["scale"], cu_seqlens_kv=s["cu_kv"], out=s["out"])
        return _plain_attention(s)
    if op == "decode":
        if own:
            from bit_asymmetric_kv_gb300 import kivi
            cache = _handles(s)
            return kivi.kivi_paged_decode_attention_window(cache, s["q"], s["window"], s["sinks"], s["scale"],
                                                           out=s["out"], ws=s["ws"])
        return _plain_decode(s)
    if op == "read":
        if own:
            from bit_asymmetric_kv_gb300 import kivi
            kivi.kivi_paged_read(_handles(s), s["cu"], s["take"], s["k_out"], s["v_out"], first=s["first"])
            return [s["k_out"], s["v_out"]]
        return _plain_read(s)
    if op == "extend":
        for t, start in s["start"]:  # the lengths and residuals that every pass starts from
            t.copy_(start)
        if own:
            from bit_asymmetric_kv_gb300 import kivi
            kivi.kivi_paged_extend_packed(_handles(s), s["k"], s["v"], s["cu"])
        else:
            _plain_extend(s)
        return {x: s[x] for x in ("k_codes", "k_meta", "v_codes", "v_meta", "k_res", "v_res", "lens")
                if s[x] is not None}
    s["table"].copy_(s["start"][0])  # the table and counts that every pass starts from
    s["refs"].copy_(s["start"][1])
    if own:
        from bit_asymmetric_kv_gb300 import kivi
        kivi.kivi_paged_reserve_window(_handles(s), s["pool"], s["extra"], s["window"], s["sinks"])
    else:
        _plain_reserve(s)
    return {x: s[x] for x in ("table", "refs", "info")}


# ------------------------------------------------------------ the definition in 64 bits
def _halves(w):
    """(scale, zero) of {s, z} words, in 64 bits."""
    h = w.contiguous().view(torch.float16).view(*w.shape, 2).double()
    return h[..., 0], h[..., 1]


def _by_hand(s, b, p):
    """Keys and values [Hkv, len(p), D] of sequence b at the positions p (a range), channel by channel
    of the definition, in 64 bits."""
    n, P, G, bits = int(s["lens"][b]), s["P"], s["G"], s["bits"]
    k = torch.zeros((s["Hkv"], len(p), D), dtype=torch.float64, device="cuda")
    v = torch.zeros_like(k)
    ch = torch.arange(D, device="cuda")
    for t0 in sorted({t // P for t in p}):
        idx = [i for i, t in enumerate(p) if t // P == t0]
        page, rows = int(s["table"][b, t0]), torch.tensor([p[i] % P for i in idx], device="cuda")
        at = torch.tensor(idx, device="cuda")
        for name, out in (("k", k), ("v", v)):
            w = s[name + "_codes"][page][:, rows].long()
            c = (w[..., ch * bits // 32] >> (ch * bits % 32)) % 2**bits
            if name == "k":
                sc, z = (x[:, rows // G] for x in _halves(s["k_meta"][page]))
            else:
                sc, z = (x[:, rows, None] for x in _halves(s["v_meta"][page]))
            out[:, at] = c.double() * sc + z
    late = [i for i, t in enumerate(p) if t >= n // G * G]
    if late:
        slots = [p[i] % G for i in late]
        k[:, late] = s["k_res"][b][:, slots].double()
        if s["v_res"] is not None:
            v[:, late] = s["v_res"][b][:, slots].double()
    return k, v


def _exact_attention(case, s):
    q, k, v = (s[x].double() for x in "qkv")
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    R, W, S = case["Hq"] // case["Hkv"], case["window"], case["sinks"]
    new, old = _chunks(case, case["n_seqs"])
    qa = ka = 0
    for n, o in zip(new, old):
        for i0 in range(0, n, 512):  # queries i0 .. i1, at positions o + i0 ..: their window and the sinks
            i1 = min(n, i0 + 512)
            w0 = max(0, o + i0 - W + 1)
            j = list(range(min(S, w0))) + list(range(w0, o + i1))
            j = torch.tensor(j, device="cuda")
            p = torch.arange(o + i0, o + i1, device="cuda")[:, None]
            seen = (j <= p) & ((p - j < W) | (j < S))
            for h in range(case["Hkv"]):
                x = torch.einsum("ird,jd->rij", q[qa + i0:qa + i1, h * R:(h + 1) * R], k[ka + j, h]) * s["scale"]
                w = torch.softmax(torch.where(seen, x, -torch.inf), -1)
                out[qa + i0:qa + i1, h * R:(h + 1) * R] = torch.einsum("rij,jd->ird", w, v[ka + j, h])
        qa, ka = qa + n, ka + n + o
    return out


def _exact_decode(case, s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    R = case["Hq"] // case["Hkv"]
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        p = [t for t in range(n) if t < case["sinks"] or t > n - 1 - case["window"]]
        k, v = _by_hand(s, b, p)
        for h in range(case["Hq"]):
            w = torch.softmax((k[h // R] @ s["q"][b, h].double()) * s["scale"], 0)
            out[b, h] = w @ v[h // R]
    return out


def _quantized(x, dim, bits):
    """Codes (packed along the last axis) and {s, z} words.  Every fp32 operation of the quantizer's
    definition is one operation in 64 bits rounded to fp32, which gives the same value."""
    levels = 2**bits - 1

    def f32(y):
        return y.float().double()

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


def _exact_extend(case, s):
    P, G, bits = s["P"], s["G"], s["bits"]
    cu, table = s["cu"].tolist(), s["table"].tolist()
    for b, n in enumerate(s["lens"].tolist()):
        m = cu[b + 1] - cu[b]
        if m == 0:
            continue
        r, q0, end = n % G, n // G * G, n + m
        q1 = end // G * G
        ks = torch.cat([s["k_res"][b][:, :r], s["k"][cu[b]:cu[b + 1]].transpose(0, 1)], 1)  # from position q0 on
        vs = s["v"][cu[b]:cu[b + 1]].transpose(0, 1)
        if s["v_res"] is not None:
            vs = torch.cat([s["v_res"][b][:, :r], vs], 1)
        for g in range(q0, q1, G):
            page, at = table[b][g // P], g % P
            s["k_codes"][page, :, at:at + G], s["k_meta"][page, :, at // G] = _quantized(
                ks[:, g - q0:g - q0 + G].double(), 1, bits)
        v0, v1 = (q0, q1) if s["v_res"] is not None else (n, end)
        for t0 in range(v0 // P * P, v1, P):
            a, z, page = max(v0, t0), min(v1, t0 + P), table[b][t0 // P]
            if z > a:
                s["v_codes"][page, :, a - t0:z - t0], s["v_meta"][page, :, a - t0:z - t0] = _quantized(
                    vs[:, a - v0:z - v0].double(), -1, bits)
        if end > q1:
            s["k_res"][b, :, :end - q1] = ks[:, q1 - q0:].clone()
            if s["v_res"] is not None:
                s["v_res"][b, :, :end - q1] = vs[:, q1 - q0:].clone()
        s["lens"][b] = end
    out = {x: s[x] for x in ("k_codes", "k_meta", "v_codes", "v_meta", "k_res", "v_res", "lens") if s[x] is not None}
    return {x: t.double() if t.is_floating_point() else t for x, t in out.items()}


def _exact_read(case, s):
    k_out, v_out = torch.zeros_like(s["k_out"]).double(), torch.zeros_like(s["v_out"]).double()
    at = 0
    for b, c in enumerate(s["take"].tolist()):
        n = int(s["lens"][b])
        f = min(case["first"], c)
        if c:
            k, v = _by_hand(s, b, list(range(f)) + list(range(n - (c - f), n)))
            k_out[at:at + c], v_out[at:at + c] = k.transpose(0, 1), v.transpose(0, 1)
        at += c
    return [k_out.clamp(-65504, 65504), v_out.clamp(-65504, 65504)]


def _exact_reserve(case, s):
    table, refs, lens, extra = s["table"].tolist(), s["refs"].tolist(), s["lens"].tolist(), s["extra"].tolist()
    P, W, S = s["P"], case["window"], case["sinks"]
    live = sum(r > 0 for r in refs)
    wanted = []
    for b, row in enumerate(table):
        if extra[b] <= 0:
            continue
        for j, page in enumerate(row):
            seen = any(t < S or t > lens[b] - W for t in (j * P, j * P + P - 1))
            if not seen and page >= 0:
                refs[page] -= 1
            if not seen:
                row[j] = -1
            elif page < 0 and j * P < lens[b] + extra[b]:
                wanted.append((b, j))
    freed = live - sum(r > 0 for r in refs)
    free = [i for i, r in enumerate(refs) if r <= 0]
    for (b, j), page in zip(wanted, free):
        table[b][j] = page
        refs[page] = 1
    got = min(len(free), len(wanted))
    info = [got, len(wanted) - got, sum(r > 0 for r in refs), freed]
    return {"table": torch.tensor(table, dtype=torch.int32), "refs": torch.tensor(refs, dtype=torch.int32),
            "info": torch.tensor(info, dtype=torch.int32)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "decode": _exact_decode, "extend": _exact_extend, "read": _exact_read,
            "reserve": _exact_reserve}[case["op"]](case, s)

"""Cases of the packed-prompt and cache-eviction operators, with their plain forms.

The path they belong to: a batch of prompts of different lengths is prefilled in one call and
fills a cache; the attention weight each cached key receives is accumulated; the cache is cut
to a budget of slots by that weight; decoding goes on over the slots kept, each with the
position its key came from, and accumulates further.

    prefill   bifocal_prefill_packed   q, k, v [T, H, D], cu_seqlens [B + 1]
    weights   bifocal_key_weights      the last `obs` queries of each prompt
    evict     bifocal_cache_evict      paged cache -> `budget` slots on other pages
    decode    bifocal_decode_kept      one token per sequence over the kept slots

Definition, per sequence of length L with G = max(1, ceil(L / w_pretrained)): query i and key j <= i score
    scale <R(i w) q, R(j w) k>            if i - j < w0,
    scale <R(f(i)) q, R(f(j)) k>          otherwise, with f(p) = p w / G ("freq_interp") or floor(p / G) w ("pos_alias"),
where R rotates the pairs (d, d + D/2) by w_d = theta^(-2d/D) and scale = 1 / sqrt(D).
"""
import math

import torch

own = False

THETA = 1e6
BLOCK = 1 << 28  # scores held at a time by the plain forms


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a server's step of chat turns, most of them short: launches and latency count
        {"name": "prefill chat turns", "op": "prefill", "lens": "1,7,64,129,33,200,1,500,90,15,310,257", "hq": 32, "hkv": 8, "dim": 128,
         "dtype": "bf16", "mode": "freq_interp", "w0": 4096, "w_pre": 32768, "page": 16},
        # documents of ordinary lengths, some past the pretrained window (G = 1, 2 and 3 in one call)
        {"name": "prefill documents", "op": "prefill", "lens": "2300,5111,901,4099,1777", "hq": 32, "hkv": 8, "dim": 128,
         "dtype": "bf16", "mode": "freq_interp", "w0": 512, "w_pre": 2048, "page": 64},
        # one long prompt beside shorter ones, rows of the cache packed like the inputs
        {"name": "prefill long prompt", "op": "prefill", "lens": "16411,8190,411", "hq": 32, "hkv": 8, "dim": 128,
         "dtype": "bf16", "mode": "pos_alias", "w0": 4096, "w_pre": 8192, "page": 0},
        # a small model's heads in 32 bits, three query heads a key head, an empty prompt among them
        {"name": "prefill fp32 d64", "op": "prefill", "lens": "1,640,1023,0,2111", "hq": 12, "hkv": 4, "dim": 64,
         "dtype": "fp32", "mode": "freq_interp", "w0": 300, "w_pre": 512, "page": 0},
        # weights of a batch of prompts as its last 64 queries see them, before the first eviction
        {"name": "weights last 64", "op": "weights", "lens": "9001,3500,120,14777,63", "obs": 64, "hq": 32, "hkv": 8, "dim": 128,
         "dtype": "bf16", "mode": "freq_interp", "w0": 4096, "w_pre": 8192, "page": 16},
        # weights accumulated over every query of a prompt
        {"name": "weights all queries", "op": "weights", "lens": "6001", "obs": 1 << 30, "hq": 32, "hkv": 8, "dim": 128,
         "dtype": "bf16", "mode": "freq_interp", "w0": 1024, "w_pre": 2048, "page": 0},
        # the last 32 queries of a very long prompt
        {"name": "weights long prompt", "op": "weights", "lens": "100003", "obs": 32, "hq": 32, "hkv": 8, "dim": 128,
         "dtype": "bf16", "mode": "pos_alias", "w0": 4096, "w_pre": 32768, "page": 64},
        # one conversation over its budget
        {"name": "evict one", "op": "evict", "lens": "4099", "budget": 2048, "recent": 256, "sink": 4, "hkv": 8, "dim": 128, "page": 16},
        # a batch of long prompts cut to a budget, one of them below it
        {"name": "evict batch", "op": "evict", "lens": "32768,20011,16000,1500,9999,30001,12345,28000", "budget": 4096, "recent": 512,
         "sink": 4, "hkv": 8, "dim": 128, "page": 64},
        # a decode step of one conversation over its kept slots
        {"name": "decode one", "op": "decode", "lens": "2049", "stretch": 16, "hq": 32, "hkv": 8, "dim": 128,
         "mode": "freq_interp", "w0": 1024, "w_pre": 8192, "page": 16, "weights": True},
        # a batch at several lengths, as between two evictions
        {"name": "decode batch", "op": "decode", "lens": "4097,8192,1030,6011,4100,7777,5000,2222,4097,4111,8000,640,3999,6500,4222,5555",
         "stretch": 8, "hq": 32, "hkv": 8, "dim": 128, "mode": "freq_interp", "w0": 1024, "w_pre": 8192, "page": 64, "weights": True},
        # two very long caches of a small model, kept as a whole (no weights wanted)
        {"name": "decode long d64", "op": "decode", "lens": "60001,44444", "stretch": 2, "hq": 16, "hkv": 4, "dim": 64,
         "mode": "pos_alias", "w0": 4096, "w_pre": 32768, "page": 16, "weights": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["prefill", "weights", "evict", "decode"])
    hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8])
    mode, page = rng.choice(["freq_interp", "pos_alias"]), rng.choice([16, 32, 64, 128])
    c = {"op": op, "hkv": hkv, "dim": rng.choice([64, 128])}
    if op in ("prefill", "weights"):
        most = _log(rng, 8, 8192) if op == "prefill" else _log(rng, 64, 24000)
        lens = [_log(rng, 1, most) for _ in range(rng.randint(1, 8))]
        while sum(lens) > 24000:
            lens.pop()
        if rng.random() < 0.3:
            lens.insert(rng.randint(0, len(lens)), 0)
        c.update(hq=hkv * g, dtype=rng.choice(["bf16", "bf16", "fp32"]), page=rng.choice([0, page]))
        c.update(w0=rng.choice([0, _log(rng, 1, 4096)]), w_pre=_log(rng, 64, 32768), mode=mode)
        if op == "weights":
            c["obs"] = rng.choice([1, 16, 32, 64, 100, 1 << 30])
            if c["obs"] > 100:
                lens = [min(x, 4000) for x in lens]
    elif op == "evict":
        most = _log(rng, 16, 32768)
        lens = [_log(rng, 1, most) for _ in range(rng.randint(1, 8))]
        budget = _log(rng, 8, most)
        c.update(budget=budget, recent=rng.randint(0, budget // 2), sink=rng.randint(0, min(8, budget // 2)), page=page)
    else:
        most = _log(rng, 1, 60000)
        lens = [_log(rng, 1, most) for _ in range(rng.randint(1, 16))]
        while sum(lens) > 80000:
            lens.pop()
        c.update(hq=hkv * g, mode=mode, w0=rng.choice([0, _log(rng, 1, 4096)]), w_pre=_log(rng, 64, 32768), page=page,
                 stretch=rng.choice([1, 2, 8, 16]), weights=rng.random() < 0.75)
    c["lens"] = ",".join(map(str, lens or [1]))
    return c


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def work(case):
    lens, hkv, D = _lens(case), case["hkv"], case["dim"]
    T = sum(lens)
    if case["op"] == "prefill":
        e = 4 if case["dtype"] == "fp32" else 2
        pairs = sum(n * (n + 1) // 2 for n in lens)
        rows = T * D * ((case["hq"] + 2 * hkv) * e + case["hq"] * 2 + 2 * hkv * 2) + 4 * hkv * T
        return {"bytes": rows, "flops": 4 * D * case["hq"] * pairs}
    if case["op"] == "weights":
        e = 4 if case["dtype"] == "fp32" else 2
        seen = [min(n, case["obs"]) for n in lens]
        pairs = sum(n * (n + 1) // 2 - (n - m) * (n - m + 1) // 2 for n, m in zip(lens, seen))
        return {"bytes": T * hkv * (D * e + 4) + sum(seen) * case["hq"] * (D * e + 4), "flops": 2 * D * case["hq"] * pairs}
    if case["op"] == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": hkv * (8 * T + 2 * kept * (4 * D + 8)), "flops": 0}
    per = 4 * D + 4 + (8 if case["weights"] else 0)
    return {"bytes": T * hkv * per + len(lens) * D * 4 * (case["hq"] + hkv), "flops": 4 * D * case["hq"] * T}


# ------------------------------------------------------------------------------------ inputs
def _table(lens, page, gen, spare=3):
    """Block table with pages in a shuffled order, and the pages in all."""
    need = [(n + page - 1) // page for n in lens]
    pages = sum(need) + spare
    perm = torch.randperm(pages, generator=gen, device="cuda").int()
    table = torch.zeros(len(lens), max(1, max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        at += m
    return table, pages


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)

    lens, hkv, D, op = _lens(case), case["hkv"], case["dim"], case["op"]
    B, T = len(lens), sum(lens)
    s = {"op": op, "case": case, "lens": lens, "max_len": max(max(lens), 1)}
    if op in ("prefill", "weights"):
        dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
        s["q"], s["k"], s["v"] = randn(T, case["hq"], D, dtype=dt), randn(T, hkv, D, dtype=dt), randn(T, hkv, D, dtype=dt)
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
        rows, s["table"] = T, None
        if case["page"]:
            s["table"], pages = _table(lens, case["page"], gen)
            rows = pages * case["page"]
        if op == "prefill":
            s["kc"] = torch.zeros(rows, hkv, D, dtype=torch.bfloat16, device="cuda")
            s["vc"] = torch.zeros_like(s["kc"])
            s["kpos"] = torch.zeros(hkv, rows, dtype=torch.int32, device="cuda")
        else:
            s["kw"] = torch.zeros(hkv, rows, device="cuda")
            # the prefill's log-sum-exp; rows that no weight asks for hold its usual size
            s["lse"] = torch.log(torch.arange(1, T + 1, device="cuda").float()).expand(case["hq"], T).contiguous()
            _plain_lse(s)
        return s
    s["len_t"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["table"], pages = _table(lens, case["page"], gen)
    if op == "evict":
        kept = [min(n, case["budget"]) for n in lens]
        far, more = _table(kept, case["page"], gen)
        s["dst"] = far + pages  # pages of their own for what is kept
        pages += more
    rows = pages * case["page"]
    s["kc"], s["vc"] = randn(rows, hkv, D), randn(rows, hkv, D)
    # positions: every key's own, increasing with gaps (those between were evicted before); each head kept others
    n = s["max_len"]
    gaps = torch.randint(1, 2 * case.get("stretch", 1) + 1, (B, hkv, n), generator=gen, device="cuda")
    pos = gaps.cumsum(-1).int() - 1
    valid = torch.arange(n, device="cuda") < s["len_t"][:, None, None]
    s["newest"] = pos.masked_fill(~valid, 0).amax((1, 2)).int()
    # what keys have gathered so far: a few carry most of it, some nothing at all
    weight = torch.exp(2 * torch.randn(B, hkv, n, generator=gen, device="cuda")) * 0.05
    weight = weight * (torch.rand(B, hkv, n, generator=gen, device="cuda") > 0.02)
    s["kpos"] = torch.zeros(hkv, rows, dtype=torch.int32, device="cuda")
    s["kw"] = torch.zeros(hkv, rows, device="cuda")
    at = _rows(s["table"], case["page"], n)[valid[:, 0]]
    s["kpos"][:, at] = pos.transpose(0, 1)[:, valid[:, 0]]
    s["kw"][:, at] = weight.transpose(0, 1)[:, valid[:, 0]]
    if op == "decode":
        s["newest"] += 1
        s["q"], s["kn"], s["vn"] = randn(B, case["hq"], D), randn(B, hkv, D), randn(B, hkv, D)
    return s


# ------------------------------------------------------------------------------------ plain forms
def _rows(table, page, n):
    """Cache rows [B, n] of each sequence's first n slots."""
    slot = torch.arange(n, device="cuda")
    page_at = (slot // page).clamp(max=table.shape[1] - 1)
    return table[:, page_at].long() * page + slot % page


def _rotate(x, angle):
    """Pairs (d, d + D/2) of x turned by `angle` (64 bits: far positions), in 32 bits."""
    c, s = angle.cos().float(), angle.sin().float()
    a, b = x.float().chunk(2, -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _omega(dim):
    return THETA ** (-2.0 * torch.arange(dim // 2, device="cuda", dtype=torch.float64) / dim)


def _far(pos, factor, mode, omega):
    """Angles of the long-range branch; `factor` broadcasts against pos."""
    if mode == "freq_interp":
        return (pos.double() / factor)[..., None] * omega
    return torch.div(pos, factor, rounding_mode="floor").double()[..., None] * omega


def _row_blocks(s, b):
    """Rows of sequence b in blocks of bounded size: (first row of the sequence, its length, the block's row numbers)."""
    case, n = s["case"], s["lens"][b]
    lo = max(0, n - case.get("obs", n))
    step = max(1, BLOCK // (max(n, 1) * case["hq"]))
    return [torch.arange(i, min(i + step, n), device="cuda") for i in range(lo, n, step)]


def _forms(s, b):
    """One sequence's q [hkv, g, n, D] and k [hkv, 1, D, n] under both rotations."""
    case, n, at = s["case"], s["lens"][b], sum(s["lens"][:b])
    hkv, D = case["hkv"], case["dim"]
    factor = max(1, -(-n // case["w_pre"]))
    pos, omega = torch.arange(n, device="cuda"), _omega(D)
    near = (pos.double()[:, None] * omega)[:, None]
    far = _far(pos, factor, case["mode"], omega)[:, None]
    q, k = s["q"][at:at + n], s["k"][at:at + n]
    qs = [_rotate(q, x).view(n, hkv, case["hq"] // hkv, D).permute(1, 2, 0, 3) for x in (near, far)]
    ks = [_rotate(k, x).permute(1, 2, 0)[:, None] for x in (near, far)]
    return qs, ks


def _scores(s, forms, rows):
    """Scores of the rows against every key of the sequence, -inf beyond the row's own."""
    case = s["case"]
    (qo, ql), (ko, kl) = forms
    dist = rows[:, None] - torch.arange(ko.shape[-1], device="cuda")
    x = torch.where(dist < case["w0"], torch.matmul(qo[:, :, rows], ko), torch.matmul(ql[:, :, rows], kl))
    return (x / math.sqrt(case["dim"])).masked_fill(dist < 0, -math.inf)


def _plain_lse(s):
    for b, n in enumerate(s["lens"]):
        forms, at = _forms(s, b), sum(s["lens"][:b])
        for rows in _row_blocks(s, b):
            s["lse"][:, at + rows] = torch.logsumexp(_scores(s, forms, rows), -1).flatten(0, 1)


def _plain_prefill(s):
    case = s["case"]
    hkv, D, T = case["hkv"], case["dim"], s["q"].shape[0]
    out = torch.zeros(T, case["hq"], D, dtype=torch.bfloat16, device="cuda")
    for b, n in enumerate(s["lens"]):
        at = sum(s["lens"][:b])
        forms, v = _forms(s, b), s["v"][at:at + n].float().permute(1, 0, 2)[:, None]
        for rows in _row_blocks(s, b):
            x = _scores(s, forms, rows)
            p = torch.exp(x - x.amax(-1, keepdim=True))
            o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
            out[at + rows] = o.permute(2, 0, 1, 3).reshape(len(rows), -1, D).bfloat16()
        pos = torch.arange(n, device="cuda")
        to = at + pos if s["table"] is None else _rows(s["table"], case["page"], n)[b]
        s["kc"][to] = forms[1][0][:, 0].permute(2, 0, 1).bfloat16()
        s["vc"][to] = s["v"][at:at + n].bfloat16()
        s["kpos"][:, to] = pos.int()
    return out, s["kc"], s["vc"], s["kpos"]


def _plain_weights(s):
    case = s["case"]
    for b, n in enumerate(s["lens"]):
        at, forms = sum(s["lens"][:b]), _forms(s, b)
        total = torch.zeros(case["hkv"], n, device="cuda")
        for rows in _row_blocks(s, b):
            lse = s["lse"][:, at + rows].view(case["hkv"], -1, len(rows), 1)
            total += torch.exp(_scores(s, forms, rows) - lse).sum((1, 2))
        to = at + torch.arange(n, device="cuda") if s["table"] is None else _rows(s["table"], case["page"], n)[b]
        s["kw"][:, to] = total
    return s["kw"]


def _plain_evict(s):
    case, n, B = s["case"], s["max_len"], len(s["lens"])
    src = _rows(s["table"], case["page"], n)
    valid = (torch.arange(n, device="cuda") < s["len_t"][:, None])[:, None]
    pos, weight = s["kpos"][:, src].transpose(0, 1), s["kw"][:, src].transpose(0, 1)
    always = (pos < case["sink"]) | (pos > s["newest"][:, None, None] - case["recent"])
    rank = torch.where(always, math.inf, weight.nan_to_num(nan=-math.inf, posinf=3e38)).masked_fill(~valid, -math.inf)
    order = torch.argsort(rank, dim=-1, descending=True, stable=True)
    kept = torch.minimum(s["len_t"], torch.tensor(case["budget"], device="cuda", dtype=torch.int32))
    m = min(case["budget"], n)
    best = order[..., :m].masked_fill(torch.arange(m, device="cuda") >= kept[:, None, None], n)
    best = best.sort(-1)[0]  # in the order of their slots; n where fewer are kept
    b, h, i = (best < n).nonzero(as_tuple=True)
    old, new = src[b, best[b, h, i]], _rows(s["dst"], case["page"], m)[b, i]
    for pool in (s["kc"], s["vc"]):
        pool[new, h] = pool[old, h]
    for pool in (s["kpos"], s["kw"]):
        pool[h, new] = pool[h, old]
    return s["kc"], s["vc"], s["kpos"], s["kw"], kept


def _plain_decode(s):
    case, n, B = s["case"], s["max_len"], len(s["lens"])
    hkv, D = case["hkv"], case["dim"]
    omega = _omega(D)
    seq = torch.arange(B, device="cuda")
    src = _rows(s["table"], case["page"], n)
    last = src[seq, s["len_t"].long() - 1]
    near = s["newest"].double()[:, None, None] * omega
    s["kc"][last] = _rotate(s["kn"], near).bfloat16()
    s["vc"][last] = s["vn"]
    s["kpos"][:, last] = s["newest"]
    if case["weights"]:
        s["kw"][:, last] = 0
    factor = (s["newest"] + case["w_pre"]) // case["w_pre"]  # ceil((newest + 1) / w_pre)
    pos, k = s["kpos"][:, src].transpose(0, 1), s["kc"][src].float().transpose(1, 2)
    v = s["vc"][src].float().transpose(1, 2)
    by = factor[:, None, None]
    k_far = _rotate(k, _far(pos, by, case["mode"], omega) - pos.double()[..., None] * omega)
    q_far = _rotate(s["q"], _far(s["newest"], factor, case["mode"], omega)[:, None])
    q_near = _rotate(s["q"], near)
    x_near = torch.matmul(q_near.view(B, hkv, -1, D), k.transpose(2, 3))
    x_far = torch.matmul(q_far.view(B, hkv, -1, D), k_far.transpose(2, 3))
    x = torch.where((s["newest"][:, None, None] - pos < case["w0"])[:, :, None], x_near, x_far) / math.sqrt(D)
    valid = torch.arange(n, device="cuda") < s["len_t"][:, None]
    x = x.masked_fill(~valid[:, None, None], -math.inf)
    lse = torch.logsumexp(x, -1, keepdim=True)
    p = torch.exp(x - lse)
    out = torch.matmul(p, v).flatten(1, 2).bfloat16()
    if case["weights"]:
        at = src[valid]
        s["kw"][:, at] += p.sum(2).transpose(0, 1)[:, valid]
    return out, lse.flatten(1), s["kc"], s["vc"], s["kpos"], s["kw"]


# ------------------------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _own(s)
    return {"prefill": _plain_prefill, "weights": _plain_weights, "evict": _plain_evict, "decode": _plain_decode}[s["op"]](s)


def _own(s):
    import rope_context_extension_bifocal_b200 as bfl
    case = s["case"]
    if s["op"] == "evict":
        kept = bfl.bifocal_cache_evict(s["kc"], s["vc"], s["kpos"], s["kw"], case["page"], s["table"], s["len_t"], s["newest"],
                                       s["max_len"], case["budget"], recent=case["recent"], sink=case["sink"],
                                       dst_block_table=s["dst"])
        return s["kc"], s["vc"], s["kpos"], s["kw"], kept
    rope = dict(w0=case["w0"], w_pretrained=case["w_pre"], theta=THETA, mode=case["mode"])
    if s["op"] == "prefill":
        out, _ = bfl.bifocal_prefill_packed(s["q"], s["k"], s["v"], s["cu"], s["max_len"], kcache=s["kc"], vcache=s["vc"],
                                            kpos=s["kpos"], page_size=case["page"], block_table=s["table"], want_lse=False, **rope)
        return out, s["kc"], s["vc"], s["kpos"]
    if s["op"] == "weights":
        return bfl.bifocal_key_weights(s["q"], s["k"], s["lse"], s["cu"], s["max_len"], case["obs"], kweight=s["kw"],
                                       page_size=case["page"], block_table=s["table"], **rope)
    out, lse = bfl.bifocal_decode_kept(s["q"], s["kn"], s["vn"], s["kc"], s["vc"], s["kpos"], s["kw"] if case["weights"] else None,
                                       case["page"], s["table"], s["len_t"], s["newest"], s["max_len"], **rope)
    return out, lse, s["kc"], s["vc"], s["kpos"], s["kw"]


# ------------------------------------------------------------------------------------ 64 bits
def _turn(x, angle):
    """Rotation as a product of complex numbers, in 64 bits."""
    half = x.shape[-1] // 2
    z = torch.complex(x[..., :half].double(), x[..., half:].double()) * torch.polar(torch.ones_like(angle), angle)
    return torch.cat([z.real, z.imag], -1)


def _stretched(pos, factor, mode, dim):
    """Positions times frequencies of the far branch."""
    w = torch.exp(-math.log(THETA) * torch.arange(0, dim, 2, device="cuda", dtype=torch.float64) / dim)
    p = pos.double() / factor if mode == "freq_interp" else (pos // factor).double()
    return p[..., None] * w


def _exact_prompt(s, case):
    """Attention output, cached keys and gathered weights of every sequence, from the definition: one query head and a
    block of rows at a time."""
    D, g = case["dim"], case["hq"] // case["hkv"]
    T = s["q"].shape[0]
    out = torch.zeros(T, case["hq"], D, dtype=torch.float64, device="cuda")
    keys = torch.zeros(T, case["hkv"], D, dtype=torch.float64, device="cuda")
    gathered = torch.zeros(case["hkv"], T, dtype=torch.float64, device="cuda")
    first = 0
    for n in s["lens"]:
        span = slice(first, first + n)
        G = max(1, (n + case["w_pre"] - 1) // case["w_pre"])
        j = torch.arange(n, device="cuda")
        a1, a2 = _stretched(j, 1, "freq_interp", D), _stretched(j, G, case["mode"], D)
        start = max(0, n - case.get("obs", n))
        for h in range(case["hq"]):
            k, v = s["k"][span, h // g], s["v"][span, h // g].double()
            k1, k2 = _turn(k, a1), _turn(k, a2)
            keys[span, h // g] = k1
            for r in range(start, n, 4096):
                e = min(n, r + 4096)
                q = s["q"][first + r:first + e, h]
                d = j[r:e, None] - j[None, :e]
                x = torch.where(d >= case["w0"], _turn(q, a2[r:e]) @ k2[:e].T, _turn(q, a1[r:e]) @ k1[:e].T) * D ** -0.5
                x[d < 0] = -math.inf
                if case["op"] == "weights":
                    gathered[h // g, first:first + e] += torch.exp(x - s["lse"][h, first + r:first + e, None].double()).sum(0)
                else:
                    out[first + r:first + e, h] = torch.softmax(x, 1) @ v[:e]
        first += n
    return out, keys, gathered


def _places(s, case):
    """Cache row of every packed token."""
    if s["table"] is None:
        return torch.arange(s["q"].shape[0], device="cuda")
    table, page, got = s["table"].cpu(), case["page"], []
    for b, n in enumerate(s["lens"]):
        got += [int(table[b, j // page]) * page + j % page for j in range(n)]
    return torch.tensor(got, device="cuda", dtype=torch.long)


def exact(case, seed):
    s = prepare(case, seed)
    lens, D = s["lens"], case["dim"]
    if case["op"] == "evict":
        return None  # nothing is computed: rows are chosen and moved
    if case["op"] in ("prefill", "weights"):
        if sum(n * min(n, case.get("obs", n)) for n in lens) * case["hq"] * D > 3e12:
            return None
        out, keys, gathered = _exact_prompt(s, case)
        at = _places(s, case)
        if case["op"] == "weights":
            w = s["kw"].double()
            w[:, at] = gathered
            return w
        kc, vc = s["kc"].double(), s["vc"].double()
        kc[at], vc[at] = keys, s["v"].double()
        return out, kc, vc, None
    g, page = case["hq"] // case["hkv"], case["page"]
    out = torch.zeros(len(lens), case["hq"], D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(len(lens), case["hq"], dtype=torch.float64, device="cuda")
    kc, vc, kw = s["kc"].double(), s["vc"].double(), s["kw"].double()
    table = s["table"].cpu()
    for b, n in enumerate(lens):
        rows = torch.tensor([int(table[b, t // page]) * page + t % page for t in range(n)], device="cuda")
        now = s["newest"][b]
        G = max(1, (int(now) + case["w_pre"]) // case["w_pre"])
        here = _stretched(now, 1, "freq_interp", D)
        new = _turn(s["kn"][b], here.expand(case["hkv"], -1))
        kc[rows[-1]], vc[rows[-1]] = new, s["vn"][b].double()
        if case["weights"]:
            kw[:, rows[-1]] = 0
        for h in range(case["hkv"]):
            pos = s["kpos"][h, rows].clone()
            pos[-1] = now
            # the cache holds the new key in 16 bits, and attention reads it from there
            k = kc[rows, h].bfloat16().double()
            raw = _turn(k, -_stretched(pos, 1, "freq_interp", D))
            far = _turn(raw, _stretched(pos, G, case["mode"], D))
            for i in range(h * g, h * g + g):
                x1 = k @ _turn(s["q"][b, i], here)
                x2 = far @ _turn(s["q"][b, i], _stretched(now, G, case["mode"], D))
                x = torch.where(now - pos >= case["w0"], x2, x1) * D ** -0.5
                p = torch.softmax(x, 0)
                out[b, i], lse[b, i] = p @ vc[rows, h], torch.logsumexp(x, 0)
                if case["weights"]:
                    kw[h, rows] += p
    return out, lse, kc, vc, None, kw

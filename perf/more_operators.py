"""Cases of attention in serving: plain forms, the framework's calls, and 64-bit results.

Four calls around a cache of keys and values in pages: rows written into their pages (as they come or in 8 bits with a
scale for each row), pages read back into packed rows, attention of one new token of each stream over its pages, and
attention of packed prompts, whose keys may be more than the queries.  Query i of a sequence with n queries and m keys
stands at position i + m - n.
"""
import math
import random

import torch

own = False

TINY = 1e-30  # rows whose largest value is below this become zeros with scale 0


def listed():
    return [
        # the rows of one decoded byte of 32 streams, into caches of up to 8192: launch latency
        {"name": "write_step", "op": "write", "nseq": 32, "shortest": 1, "longest": 1, "before": 8191, "hkv": 4, "d": 128,
         "page": 64, "q8": False},
        # the global model's prompts, 32 x 2048 chunks, kept in 8 bits
        {"name": "write_q8_prompt", "op": "write", "nseq": 32, "shortest": 2048, "longest": 2048, "before": 0, "hkv": 4,
         "d": 128, "page": 64, "q8": True},
        # a few short streams read from an odd place on, three heads of 72, small pages
        {"name": "read_odd", "op": "read", "nseq": 7, "shortest": 0, "longest": 700, "before": 77, "hkv": 3, "d": 72,
         "page": 16, "q8": False},
        # 16 streams of 8192 bytes in 8 bits, to continue their prompts
        {"name": "read_q8_long", "op": "read", "nseq": 16, "shortest": 8192, "longest": 8192, "before": 0, "hkv": 4,
         "d": 128, "page": 64, "q8": True},
        # one chunk of one stream, 2048 chunks behind it: launch latency and the split over the length
        {"name": "step_one_stream", "op": "step", "nseq": 1, "shortest": 2048, "longest": 2048, "hq": 12, "hkv": 4,
         "d": 128, "page": 64, "q8": False, "window": 0, "prefix": 0, "cap": 0.0, "slopes": False},
        # a batch of streams of all ages on 8-bit pages
        {"name": "step_batch_q8", "op": "step", "nseq": 256, "shortest": 256, "longest": 2048, "hq": 12, "hkv": 4, "d": 128,
         "page": 64, "q8": True, "window": 0, "prefix": 0, "cap": 0.0, "slopes": False},
        # the byte encoder's window of 512 with its first bytes kept visible, capped scores, small pages
        {"name": "step_window_odd", "op": "step", "nseq": 61, "shortest": 0, "longest": 8192, "hq": 8, "hkv": 8, "d": 64,
         "page": 16, "q8": False, "window": 512, "prefix": 5, "cap": 30.0, "slopes": False},
        # few streams with 65536 positions each: bound by the cache's bytes
        {"name": "step_long", "op": "step", "nseq": 8, "shortest": 65536, "longest": 65536, "hq": 12, "hkv": 4, "d": 128,
         "page": 64, "q8": False, "window": 0, "prefix": 0, "cap": 0.0, "slopes": True},
        # a few short prompts arriving together, one of them empty
        {"name": "prompt_short", "op": "prompt", "nseq": 48, "shortest": 0, "longest": 100, "before": 0, "hq": 8, "hkv": 4,
         "d": 64, "causal": True, "window": 0, "prefix": 0, "cap": 0.0, "slopes": False},
        # the global model over 32 x 2048 chunks, 12 heads of 128 on 4 of keys: the largest product
        {"name": "prompt_chunks", "op": "prompt", "nseq": 32, "shortest": 2048, "longest": 2048, "before": 0, "hq": 12,
         "hkv": 4, "d": 128, "causal": True, "window": 0, "prefix": 0, "cap": 0.0, "slopes": False},
        # the byte encoder over ragged prompts of 1024 .. 8192 bytes, each byte seeing the last 512
        {"name": "prompt_window", "op": "prompt", "nseq": 16, "shortest": 1024, "longest": 8192, "before": 0, "hq": 8,
         "hkv": 8, "d": 64, "causal": True, "window": 512, "prefix": 0, "cap": 0.0, "slopes": False},
        # prompts continued in pieces over 4096 earlier keys, capped scores, distance bias, the first 100 keys seen by all
        {"name": "prompt_continue", "op": "prompt", "nseq": 8, "shortest": 64, "longest": 512, "before": 4096, "hq": 12,
         "hkv": 4, "d": 128, "causal": True, "window": 0, "prefix": 100, "cap": 30.0, "slopes": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "step", "step", "prompt", "prompt"])
    hkv, q8, page = _log(rng, 1, 8), rng.random() < 0.5, rng.choice([16, 32, 64, 128])
    if op in ("write", "read"):
        d = 16 * _log(rng, 2, 16)
        longest = _log(rng, 1, min(16384, 16 * 8192 * 4 * 128 // (hkv * d)))
        nseq = _log(rng, 1, max(1, min(256, 16 * 8192 * 4 * 128 // (longest * hkv * d))))
        if op == "write":
            nseq = max(1, nseq // 2)
        return {"op": op, "nseq": nseq, "shortest": rng.choice([0, longest // 4, longest]), "longest": longest,
                "before": rng.choice([0, _log(rng, 1, 1000)]), "hkv": hkv, "d": d, "page": page, "q8": q8}
    d, group = rng.choice([32, 64, 64, 96, 128, 128, 128, 256]), rng.choice([1, 1, 2, 3, 4, 8])
    case = {"op": op, "hq": hkv * group, "hkv": hkv, "d": d, "cap": rng.choice([0.0, 0.0, 30.0]),
            "slopes": rng.random() < 0.3, "prefix": rng.choice([0, 0, _log(rng, 1, 200)]), "window": 0}
    if op == "step":
        most = 8 * 65536 * 4 * 128 // (hkv * d)
        longest = _log(rng, 1, min(65536, most))
        nseq = _log(rng, 1, max(1, min(512, most // longest)))
        if rng.random() < 0.3:
            case["window"] = _log(rng, 1, 2048)
        return case | {"nseq": nseq, "shortest": rng.choice([0, longest // 4, longest]), "longest": longest, "page": page,
                       "q8": q8}
    before = rng.choice([0, 0, _log(rng, 1, 4096)])
    case["causal"] = rng.random() < 0.8
    most = 32 * 12 * 2048 * 2048 * 128 // (case["hq"] * max(d, 64))  # pairs of a query and a key
    longest = _log(rng, 1, 4096)
    while longest * (longest + before) > most:
        longest //= 2
    nseq = _log(rng, 1, max(1, min(64, most // (longest * (longest + before)), 262144 * 512 // (longest * case["hq"] * d))))
    if rng.random() < 0.3:
        case["window"] = _log(rng, 16, 1024)
    return case | {"nseq": nseq, "shortest": rng.choice([0, longest // 4, longest]), "longest": longest, "before": before}


def _lengths(case):
    # ragged lengths that go with the case, so that its outputs have one shape; both ends of the range are among them
    rng = random.Random(case["nseq"] * 1000003 + case["longest"])
    length = [rng.randint(case["shortest"], case["longest"]) for _ in range(case["nseq"])]
    return [case["longest"], case["shortest"], *length[2:]] if len(length) > 1 else [case["longest"]]


def _offsets(length):
    return torch.tensor([0] + length).cumsum(0).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, device="cuda", dtype=dtype, generator=gen)

    def slices(rows, *heads):  # column slices of one projection's output, as a block has them
        row = randn(rows, sum(heads) * d, dtype=torch.bfloat16)
        return [x.unflatten(1, (-1, d)) for x in row.split([h * d for h in heads], 1)]

    op, nseq, hkv, d = case["op"], case["nseq"], case["hkv"], case["d"]
    length = _lengths(case)
    s = {"case": case, "longest": max(length)}
    if op in ("step", "prompt"):
        hq = case["hq"]
        # bias by distance: slopes of 2^-1 .. 2^-8 over the heads
        s["slopes"] = (torch.exp2(-8.0 * torch.arange(1, hq + 1, device="cuda") / hq).float() if case["slopes"] else None)
        s["prefix"] = (torch.randint(0, case["prefix"] + 1, (nseq,), device="cuda", generator=gen, dtype=torch.int32)
                       if case["prefix"] else None)
    if op == "prompt":
        total = sum(length)
        s["offsets"], s["k_offsets"] = _offsets(length), None
        s["q"], s["k"], s["v"] = slices(total, hq, hkv, hkv)
        if case["before"]:  # keys and values of the earlier positions too, as read from their pages
            keys = [n + case["before"] for n in length]
            s["k_offsets"] = _offsets(keys)
            s["k"], s["v"] = (randn(sum(keys), hkv, d, dtype=torch.bfloat16) for _ in range(2))
        s["longest_k"] = s["longest"] + case["before"]
        return s
    # a pool with pages to spare, a stream's pages anywhere in it, -1 behind its last one
    page, before = case["page"], case.get("before", 0)
    cols = -(-(s["longest"] + before) // page)
    used = torch.tensor([-(-(n + before) // page) for n in length])
    npages = int(used.sum()) + 5
    there = torch.arange(cols)[None, :] < used[:, None]
    table = torch.full((nseq, cols), -1, dtype=torch.int32, device="cuda")
    table[there.cuda()] = torch.randperm(npages, device="cuda", generator=gen)[:int(used.sum())].to(torch.int32)
    s["table"] = table
    shape = (npages, hkv, page, d)
    for x in ("k", "v"):
        if case["q8"]:
            codes = torch.randint(-127, 128, shape, device="cuda", generator=gen, dtype=torch.int8)
            s[x + "_pages"], s[x + "_scale"] = codes, torch.exp(0.3 * randn(*shape[:3])) / 64.0
        else:
            s[x + "_pages"], s[x + "_scale"] = randn(*shape, dtype=torch.bfloat16), None
    if op == "step":
        s["q"] = slices(nseq, hq)[0]
        s["lengths"] = torch.tensor(length, dtype=torch.int32, device="cuda")
        return s
    s["total"] = sum(length)
    s["offsets"] = _offsets(length)
    s["start"] = (torch.randint(0, before + 1, (nseq,), device="cuda", generator=gen, dtype=torch.int32) if before else None)
    if op == "write":
        s["k"], s["v"] = slices(s["total"], hkv, hkv)
    return s


def _pairs(case):
    # visible pairs of a query and a key, without the prefix, which only adds to a window
    n = 0
    for length in _lengths(case):
        first, keys = case["before"], length + case["before"]
        lo = torch.arange(first, first + length, dtype=torch.int64)
        w = case["window"] or (1 << 40)
        hi = lo + 1 if case["causal"] else (lo + w).clamp(max=keys)
        n += int((hi - (lo - w + 1).clamp(min=0)).sum())
    return n


def work(case):
    length, hkv, d = _lengths(case), case["hkv"], case["d"]
    if case["op"] in ("write", "read"):
        rows = 2 * sum(length) * hkv
        pages = rows * (d + 4 if case["q8"] else 2 * d)
        # 8-bit pages are read back too, since they are compared as the values they stand for
        back = pages + rows * 2 * d if case["q8"] and case["op"] == "write" else 0
        return {"bytes": rows * 2 * d + pages + back, "flops": 0}
    hq = case["hq"]
    if case["op"] == "step":
        seen = sum(min(n, case["window"] or n) for n in length)
        return {"bytes": 2 * seen * hkv * (d + 4 if case["q8"] else 2 * d) + 4 * case["nseq"] * hq * d,
                "flops": 4 * seen * hq * d}
    total = sum(length)
    return {"bytes": 4 * total * hq * d + 4 * (total + case["nseq"] * case["before"]) * hkv * d,
            "flops": 4 * _pairs(case) * hq * d}


# ---------------------------------------------------------------- plain forms (32 bits)

def _places(s):
    # (page, position in it) of every packed row, and which rows have a page
    page, off = s["case"]["page"], s["offsets"]
    row = torch.arange(s["total"], device=off.device)
    seq = torch.searchsorted(off, row, right=True) - 1
    at = row - off[seq]
    if s["start"] is not None:
        at = at + s["start"][seq]
    return s["table"][seq, at // page].long(), at % page


def _codes(x):
    x = x.float()
    top = x.abs().amax(-1, keepdim=True)
    codes = (x * torch.where(top >= TINY, 127.0 / top, 0.0)).round().clamp(-127, 127).to(torch.int8)
    return codes, torch.where(top >= TINY, top / 127.0, 0.0)[..., 0]


def _rows(s, x, page, at):
    if s[x + "_scale"] is None:
        return s[x + "_pages"][page, :, at]
    return (s[x + "_pages"][page, :, at].float() * s[x + "_scale"][page, :, at][..., None]).to(torch.bfloat16)


def _plain_write(s):
    page, at = _places(s)
    if not s["case"]["q8"]:
        s["k_pages"][page, :, at] = s["k"]
        s["v_pages"][page, :, at] = s["v"]
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    s["k_pages"][page, :, at], s["k_scale"][page, :, at] = _codes(s["k"])
    s["v_pages"][page, :, at], s["v_scale"][page, :, at] = _codes(s["v"])
    return {"k": _rows(s, "k", page, at), "v": _rows(s, "v", page, at)}


def _plain_read(s):
    page, at = _places(s)
    return {"k": _rows(s, "k", page, at), "v": _rows(s, "v", page, at)}


def _weights(s, score, pos, key, there):
    # softmax of score [nseq, blocks, hkv, group, queries, keys] where `there` (the same without heads) holds
    c = s["case"]
    if c["cap"]:
        score.div_(c["cap"]).tanh_().mul_(c["cap"])
    if s["slopes"] is not None:
        far = (pos[..., :, None] - key[..., None, :]).abs()[:, :, None, None].float()
        score -= s["slopes"].view(c["hkv"], -1, 1, 1) * far
    score.masked_fill_(~there[:, :, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp_(min=-1e30)
    score.sub_(top).exp_()
    return score.div_(score.sum(-1, keepdim=True).clamp_(min=1e-30))


def _plain_step(s):
    c, page = s["case"], s["case"]["page"]
    n, w = s["lengths"].long()[:, None], c["window"] or s["longest"]
    band = n - w + torch.arange(w, device=n.device)  # the last w positions
    key, there = band, band >= 0
    if c["window"] and c["prefix"]:  # and those of the prefix in front of them
        first = torch.arange(c["prefix"], device=n.device).expand(c["nseq"], -1)
        key = torch.cat([first, band], 1)
        there = torch.cat([(first < s["prefix"].long()[:, None]) & (first < n - w), there], 1)
    inside = torch.where(there, key, 0)
    pages, at = s["table"].gather(1, inside // page).clamp_(min=0).long(), inside % page
    k, v = (s[x + "_pages"][pages, :, at].float() for x in ("k", "v"))  # [nseq, keys, hkv, d]
    if c["q8"]:
        k, v = k * s["k_scale"][pages, :, at][..., None], v * s["v_scale"][pages, :, at][..., None]
    q = s["q"].float().unflatten(1, (c["hkv"], -1))
    score = (q @ k.permute(0, 2, 3, 1)) * c["d"] ** -0.5
    p = _weights(s, score[:, None, :, :, None], n[:, None] - 1, key[:, None], there[:, None, None])
    return (p[:, 0, :, :, 0] @ v.transpose(1, 2)).flatten(1, 2).to(torch.bfloat16)


def _plain_prompt(s):
    # queries in blocks of a window's length, each with the keys that its window can reach; without one, one block
    c, off = s["case"], s["offsets"]
    k_off = off if s["k_offsets"] is None else s["k_offsets"]
    nq, nk = off.diff()[:, None, None], k_off.diff()[:, None, None]
    w, most = c["window"], s["longest_k"]
    size = min(w or s["longest"], s["longest"])
    blocks = -(-s["longest"] // size)
    query = torch.arange(blocks * size, device=off.device).view(1, blocks, size)
    pos = query + nk - nq
    if w:
        key = pos[:, :, :1] - w + 1 + torch.arange(size + (w if c["causal"] else 2 * w) - 1, device=off.device)
    else:
        key = torch.arange(most, device=off.device).expand(c["nseq"], blocks, most)

    def near(t, j):
        seen = (j <= t) if c["causal"] else torch.ones_like(j <= t)
        return seen & ((t - j).abs() < w) if w else seen

    there = near(pos[..., :, None], key[..., None, :])
    if c["prefix"]:
        first = s["prefix"].long()[:, None, None]
        there |= (key < first)[..., None, :]
        if w:  # keys of the prefix in front of the block's own
            more = torch.arange(c["prefix"], device=off.device).expand(c["nseq"], blocks, -1)
            add = (more < first) & ((more < key[..., :1]) | (more > key[..., -1:]))
            key = torch.cat([more, key], 2)
            there = torch.cat([add[:, :, None].expand(-1, -1, size, -1), there], 3)
    valid = (key >= 0) & (key < nk)
    there &= valid[..., None, :]
    at = k_off[:-1, None, None] + torch.where(valid, key, 0)
    at = at.clamp_(max=max(0, s["k"].shape[0] - 1))
    k, v = s["k"][at].float(), s["v"][at].float()  # [nseq, blocks, keys, hkv, d]
    row = torch.where(query < nq, off[:-1, None, None] + query, 0)
    q = s["q"][row].float().unflatten(3, (c["hkv"], -1)).permute(0, 1, 3, 4, 2, 5)  # [nseq, blocks, hkv, group, queries, d]
    score = (q.flatten(3, 4) @ k.permute(0, 1, 3, 4, 2)).unflatten(3, q.shape[3:5]).mul_(c["d"] ** -0.5)
    p = _weights(s, score, pos, key, there)
    o = (p.flatten(3, 4) @ v.transpose(2, 3)).unflatten(3, q.shape[3:5]).permute(0, 1, 4, 2, 3, 5).flatten(3, 4)
    out = torch.empty(s["q"].shape, dtype=torch.bfloat16, device=off.device)
    mine = (query < nq).expand(c["nseq"], -1, -1)
    out[row[mine]] = o[mine].to(torch.bfloat16)
    return out


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if not own:
        return {"write": _plain_write, "read": _plain_read, "step": _plain_step, "prompt": _plain_prompt}[case["op"]](s)
    import byte_level_lm_amd as B

    if case["op"] == "prompt":
        return B.attention(s["q"], s["k"], s["v"], s["offsets"], k_offsets=s["k_offsets"], causal=case["causal"],
                           window=case["window"] or None, cap=case["cap"] or None, slopes=s["slopes"], prefix=s["prefix"])
    scales = {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if case["op"] == "step":
        return B.attention_step(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lengths"], window=case["window"] or None,
                                cap=case["cap"] or None, slopes=s["slopes"], prefix=s["prefix"], **scales)
    if case["op"] == "write":
        offsets = None if case["longest"] == case["shortest"] == 1 else s["offsets"]  # one row of each stream
        B.kv_write(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], offsets=offsets, start=s["start"], **scales)
        if not case["q8"]:
            return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    # what the 8 bits stand for, where a case writes them
    k, v = B.kv_read(s["k_pages"], s["v_pages"], s["table"], s["offsets"], s["total"], start=s["start"], **scales)
    return {"k": k, "v": v}


# ---------------------------------------------------------------- 64 bits

def _exact_rows(s, seq, first, n, x):
    # rows of one stream's positions first .. first + n - 1, [n, hkv, d]
    page = s["case"]["page"]
    names = s["table"][seq].tolist()
    parts = []
    while n > 0:
        at = first % page
        m = min(n, page - at)
        part = s[x + "_pages"][names[first // page], :, at:at + m].double()
        if s[x + "_scale"] is not None:
            part = part * s[x + "_scale"][names[first // page], :, at:at + m, None].double()
        parts.append(part.transpose(0, 1))
        first, n = first + m, n - m
    return torch.cat(parts) if parts else torch.zeros(0, s["case"]["hkv"], s["case"]["d"], dtype=torch.float64, device="cuda")


def _exact_attend(s, q, k, v, seq, causal):
    # one sequence: q [n, hq, d], k, v [m, hkv, d] in 64 bits
    c = s["case"]
    n, m, group = q.shape[0], k.shape[0], c["hq"] // c["hkv"]
    out = torch.zeros_like(q)
    if not n or not m:
        return out
    here = torch.arange(m - n, m, device="cuda")[:, None]
    keys = torch.arange(m, device="cuda")[None, :]
    hidden = (keys > here) if causal else torch.zeros(n, m, dtype=torch.bool, device="cuda")
    if c["window"]:
        hidden = hidden | (keys <= here - c["window"]) | (keys >= here + c["window"])
    if s["prefix"] is not None:
        hidden = hidden & (keys >= int(s["prefix"][seq]))
    for h in range(c["hq"]):
        x = torch.mm(q[:, h], k[:, h // group].t()) / math.sqrt(c["d"])
        if c["cap"]:
            x = torch.tanh(x / c["cap"]) * c["cap"]
        if s["slopes"] is not None:
            x = x - s["slopes"][h].double() * (here - keys).abs()
        x = torch.where(hidden, -math.inf, x)
        out[:, h] = torch.mm(torch.softmax(x, 1).nan_to_num(0.0), v[:, h // group])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    length = _lengths(case)
    off = [sum(length[:i]) for i in range(len(length))] if case["nseq"] <= 4096 else None
    if case["op"] == "prompt":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        at = 0
        for i, n in enumerate(length):
            m = n + case["before"]
            out[off[i]:off[i] + n] = _exact_attend(s, s["q"][off[i]:off[i] + n].double(), s["k"][at:at + m].double(),
                                                   s["v"][at:at + m].double(), i, case["causal"])
            at += m
        return out
    if case["op"] == "step":
        return torch.cat([_exact_attend(s, s["q"][i:i + 1].double(), _exact_rows(s, i, 0, n, "k"),
                                        _exact_rows(s, i, 0, n, "v"), i, True) for i, n in enumerate(length)])
    start = s["start"].tolist() if s["start"] is not None else [0] * len(length)
    if case["op"] == "read":
        return {x: torch.cat([_exact_rows(s, i, start[i], n, x) for i, n in enumerate(length)]) for x in ("k", "v")}
    if case["q8"]:
        out = {}
        for x in ("k", "v"):
            rows = s[x].double()
            step = rows.abs().max(2, keepdim=True).values / 127.0
            out[x] = torch.round(rows / step) * step
        return out
    out = {x + "_pages": s[x + "_pages"].double() for x in ("k", "v")}
    names = s["table"].tolist()
    for i, n in enumerate(length):
        for t in range(n):
            there = start[i] + t
            for x in ("k", "v"):
                out[x + "_pages"][names[i][there // case["page"]], :, there % case["page"]] = s[x][off[i] + t].double()
    return out

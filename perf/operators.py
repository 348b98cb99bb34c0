"""The serving operators over paged caches: their calls as a user makes them, their plain forms, and what is measured.

Three operators that a server of the hybrid attention step runs together:

* "plan":   block tables and slot maps of one scheduler step, built on the GPU from the requests' lengths
            (csa_plan_pages),
* "write":  rows stored through a slot map, as bf16 or as FP8 codes with block exponents
            (csa_paged_write, csa_paged_write_fp8kv),
* "attend": dense attention over a paged cache of compressed entries plus a ring of window rows, for a batch whose
            requests share a long prefix (hca_attend_paged, hca_attend_paged_fp8kv).
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------------------------------------------- cases
def _attend(name, batch, nq, H, D, m, page, shared, suffix, W, ring, fp8=False, sinks=False, gain=False, rope=False,
            pad=0):
    return {"name": name, "op": "attend", "batch": batch, "nq": nq, "H": H, "D": D, "m": m, "page": page,
            "shared": shared, "suffix": suffix, "W": W, "ring": ring, "fp8": fp8, "sinks": sinks, "gain": gain,
            "rope": rope, "pad": pad}


def listed():
    return [
        # decode of 32 chats over one 1M-token document (m = 128), each with up to 24K tokens of its own
        _attend("attend_doc1m_b32", 32, 1, 128, 512, 128, 64, 8064, 192, 128, 128),
        # the same on FP8 pages, an odd batch
        _attend("attend_doc1m_b25_fp8", 25, 1, 128, 512, 128, 128, 7936, 150, 128, 128, fp8=True),
        # the decode batch of the headline benchmark: 8 requests over 128K shared tokens, small pages
        _attend("attend_128k_b8", 8, 1, 128, 512, 128, 16, 1024, 33, 128, 136),
        # four drafted tokens a request verified at once, every option of the attention, padded batch slots
        _attend("attend_verify_b16x4", 16, 4, 128, 512, 16, 32, 4096, 60, 128, 144, sinks=True, gain=True, rope=True,
                pad=3),
        # many requests of a small head count over a 64K-token prefix at m = 4
        _attend("attend_h16_b96", 96, 1, 16, 128, 4, 256, 16384, 200, 128, 128, sinks=True),
        # no shared prefix: long ragged requests in pages
        _attend("attend_ragged_b6", 6, 1, 128, 512, 128, 64, 0, 4001, 128, 131),
        # the tiny shape of the tests, where latency counts
        _attend("attend_tiny_b4", 4, 1, 8, 64, 4, 32, 480, 41, 16, 16),
        # one decode step of a batch
        {"name": "plan_decode_b256", "op": "plan", "batch": 256, "old": 131072, "new": 1, "m": 4, "page": 64, "ring": 128,
         "slack": 0},
        # prompts of up to 8K tokens, m = 4, with spare room in the outputs
        {"name": "plan_prefill_b48", "op": "plan", "batch": 48, "old": 3000, "new": 8190, "m": 4, "page": 64, "ring": 128,
         "slack": 1000},
        # the decode step of a very large batch at m = 1 (plain tokens)
        {"name": "plan_decode_b5000", "op": "plan", "batch": 5000, "old": 2000, "new": 3, "m": 1, "page": 16, "ring": 131,
         "slack": 17},
        # one decode step's new rows
        {"name": "write_decode_b256", "op": "write", "rows": 256, "D": 512, "slots": 65536, "fp8": False},
        # a prompt's rows, quantised on the way
        {"name": "write_prefill_fp8", "op": "write", "rows": 32770, "D": 512, "slots": 65536, "fp8": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _keys(case):
    return case["shared"] + case["suffix"] / 2 + case["W"]


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "plan", "write"])
    if op == "plan":
        batch = _log(rng, 1, 6000)
        new = _log(rng, 1, max(1, 390000 // batch)) if rng.random() < 0.6 else 1
        return {"op": "plan", "batch": batch, "old": _log(rng, 1, 200000), "new": min(new, 16384),
                "m": rng.choice([1, 4, 16, 128]), "page": rng.choice([16, 32, 48, 64, 128]),
                "ring": rng.choice([16, 128, 131, 160]), "slack": rng.choice([0, 0, 5, 400])}
    if op == "write":
        rows = _log(rng, 1, 32000)
        return {"op": "write", "rows": rows, "D": rng.choice([128, 256, 512]), "slots": min(65536, rows + _log(rng, 1, 40000)),
                "fp8": rng.random() < 0.5}
    while True:
        D = rng.choice([64, 128, 256, 512, 512])
        H = rng.choice([1, 8, 16, 40, 64, 128, 128])
        nq = rng.choice([1, 1, 1, 2, 4])
        batch = _log(rng, 1, 96)
        page = rng.choice([16, 32, 48, 64, 128])
        shared = 0 if rng.random() < 0.15 else page * max(1, _log(rng, 64, 12000) // page)
        suffix = _log(rng, 1, 400) if shared else _log(rng, 8, 4000)
        W = rng.choice([16, 128, 128])
        rope = rng.random() < 0.3
        case = {"op": "attend", "batch": batch, "nq": nq, "H": H, "D": D,
                "m": rng.choice([4, 16]) if rope else rng.choice([4, 16, 128]), "page": page, "shared": shared,
                "suffix": suffix, "W": W, "ring": W + nq - 1 + rng.choice([0, 0, 3, 32]),
                "fp8": D >= 128 and rng.random() < 0.4, "sinks": rng.random() < 0.4, "gain": rng.random() < 0.25,
                "rope": rope, "pad": rng.choice([0, 0, 1, 2]) if batch > 2 else 0}
        if batch * nq * H * D * _keys(case) <= 32 * 128 * 512 * 8200:
            return case


# ---------------------------------------------------------------------------------------------------- inputs
def _suffixes(case):
    """Entries of its own that each request holds (before the seed's permutation): spread over 0..suffix."""
    b, s = case["batch"], case["suffix"]
    return [s] if b == 1 else [(s * i) // (b - 1) for i in range(b)]


def _plan_lengths(case):
    """(tokens cached, tokens new) of each request before the seed's permutation: ragged up to old and new; one
    request in 16 is an empty slot of the batch."""
    b = case["batch"]
    old = [(case["old"] * (i % 97 + 1)) // 97 for i in range(b)]
    new = [case["new"] if case["new"] == 1 else 1 + ((case["new"] - 1) * (i % 31)) // 30 for i in range(b)]
    for i in range(15, b, 16):
        old[i] = new[i] = 0
    return old, new


def _gen(seed, k):
    return torch.Generator(device="cuda").manual_seed(seed * 1000 + k)


def _normal(shape, seed, k):
    return torch.randn(shape, generator=_gen(seed, k), device="cuda", dtype=torch.float32)


def _quantised(x):
    """Rows in the FP8 format of the cache: e4m3 codes, one UE8M0 exponent byte per 128 channels; the smallest power
    of two that brings a block's largest magnitude to 448 or less, an all-zero block at exponent 0."""
    blk = x.float().unflatten(-1, (-1, 128))
    amax = blk.abs().amax(-1)
    mant, ex = torch.frexp(amax)  # amax = mant * 2^ex, mant in [0.5, 1); 448 = 0.875 * 2^9
    k = torch.where(mant <= 0.875, ex - 9, ex - 8).clamp(-124, 119)
    k = torch.where(amax == 0, torch.zeros_like(k), k)
    scaled = torch.ldexp(blk, -k.unsqueeze(-1))
    codes = scaled.to(torch.float8_e4m3fn).view(torch.uint8)
    codes = torch.where(codes == 0x80, torch.zeros_like(codes), codes).flatten(-2)
    return codes, (k + 127).to(torch.uint8)


def _prepare_attend(case, seed):
    B, nq, H, D, m, page = (case[k] for k in ("batch", "nq", "H", "D", "m", "page"))
    rnd = random.Random(seed)
    suf = _suffixes(case)
    rnd.shuffle(suf)
    n_shared = case["shared"]
    max_pages = max(1, -(-(n_shared + case["suffix"]) // page))
    shared_pages = n_shared // page
    own_pages = [-(-s // page) for s in suf]
    n_pages = shared_pages + sum(own_pages) + 8
    ids = list(range(n_pages))
    rnd.shuffle(ids)
    table = torch.full((B, max_pages), -1, dtype=torch.int32)
    table[:, :shared_pages] = torch.tensor(ids[:shared_pages], dtype=torch.int32)
    at = shared_pages
    used = torch.zeros(n_pages, page, dtype=torch.bool)
    used[ids[:shared_pages]] = True
    for b in range(B):
        own_ids = ids[at:at + own_pages[b]]
        table[b, shared_pages:shared_pages + len(own_ids)] = torch.tensor(own_ids, dtype=torch.int32)
        at += len(own_ids)
        for j, p in enumerate(own_ids):
            used[p, :min(page, suf[b] - j * page)] = True
    # the newest query of a request sees exactly its entries: (t + 1) // m = shared + own
    t = [(n_shared + s) * m + rnd.randrange(m) - 1 for s in suf]
    pos = torch.tensor([[max(tb - nq + 1 + i, 0) for i in range(nq)] for tb in t], dtype=torch.int32)
    if case["pad"]:
        pos[B - case["pad"]:] = -1  # empty slots of the batch
    # compressed entries are RMSNorm'd rows; what no request holds is uninitialised memory (NaN here)
    pool = _normal((n_pages, page, D), seed, 1)
    pool = (pool * torch.rsqrt(pool.square().mean(-1, keepdim=True))).to(torch.bfloat16)
    win = _normal((B, case["ring"], D), seed, 2).to(torch.bfloat16)
    st = {"case": case, "q": _normal((B, nq, H, D), seed, 3).to(torch.bfloat16), "table": table.cuda(),
          "pos": pos.cuda(), "scale": D ** -0.5, "n_shared": n_shared,
          "sinks": _normal((H,), seed, 4) * 2 if case["sinks"] else None,
          "gain": 1 + 0.2 * _normal((D,), seed, 5) if case["gain"] else None, "rope": None}
    hole = ~used.cuda()
    if case["fp8"]:
        codes, exps = _quantised(pool)
        codes[hole] = 0x7F  # NaN
        exps[hole] = 255
        st["pool8"], st["pool8e"] = codes, exps
        st["win8"], st["win8e"] = _quantised(win)
    else:
        pool[hole] = float("nan")
        st["pool"], st["win"] = pool, win
    if case["rope"]:
        p = torch.arange(int(pos.max()) + 1, dtype=torch.float64, device="cuda")
        f = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
        a = p[:, None] * f
        st["rope"] = (a.cos().float(), a.sin().float())
    return st


def _prepare_plan(case, seed):
    old, new = _plan_lengths(case)
    rnd = random.Random(seed)
    order = list(range(case["batch"]))
    rnd.shuffle(order)
    old, new = [old[i] for i in order], [new[i] for i in order]
    m, page = case["m"], case["page"]
    max_pages = max(-(-((o + n) // m) // page) for o, n in zip(old, new)) + 6
    # up to four pages more in the past of every live request, by the seed: what is new stays as much
    old = [o + m * page * rnd.randrange(5) if o + n else 0 for o, n in zip(old, new)]
    held = [-(-(o // m) // page) for o in old]
    need = [-(-((o + n) // m) // page) for o, n in zip(old, new)]
    n_pages = sum(need) + 64
    ids = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed), dtype=torch.int64).to(torch.int32)
    table = torch.full((case["batch"], max_pages), -1, dtype=torch.int32)
    col = torch.arange(max_pages)
    mask = col[None] < torch.tensor(held)[:, None]
    table[mask] = ids[:int(mask.sum())]
    tokens = sum(new)
    entries = sum((o + n) // m - o // m for o, n in zip(old, new))
    return {"case": case, "old": torch.tensor(old, dtype=torch.int32, device="cuda"),
            "new": torch.tensor(new, dtype=torch.int32, device="cuda"),
            "free": ids[int(mask.sum()):].contiguous().cuda(), "table": table.cuda(),
            "max_tokens": tokens + case["slack"], "max_entries": entries + case["slack"]}


def _prepare_write(case, seed):
    n, slots, D = case["rows"], case["slots"], case["D"]
    perm = torch.randperm(slots, generator=_gen(seed, 1), device="cuda")[:n].to(torch.int64)
    perm[::17] = -1  # rows that no request asked to keep
    # rows of different sizes, as the streams of different tokens are
    rows = _normal((n, D), seed, 2) * torch.exp2(2 * _normal((n, 1), seed, 3))
    st = {"case": case, "rows": rows.to(torch.bfloat16), "slots": perm}
    if case["fp8"]:
        st["codes"] = torch.zeros((slots, D), dtype=torch.uint8, device="cuda")
        st["exps"] = torch.full((slots, D // 128), 127, dtype=torch.uint8, device="cuda")
    else:
        st["pool"] = torch.zeros((slots, D), dtype=torch.bfloat16, device="cuda")
    return st


def prepare(case, seed):
    return {"attend": _prepare_attend, "plan": _prepare_plan, "write": _prepare_write}[case["op"]](case, seed)


# ---------------------------------------------------------------------------------------------------- plain forms
def _dequantised(codes, exps):
    v = codes.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 128))
    return torch.ldexp(v, (exps.to(torch.int32) - 127).unsqueeze(-1)).flatten(-2)


def _rotate(x, cos, sin):
    """Rotate-half form on the trailing 64 channels; cos, sin broadcast against [..., 32]."""
    head, a, b = x[..., :-64], x[..., -64:-32], x[..., -32:]
    return torch.cat([head, a * cos - b * sin, b * cos + a * sin], -1)


def _plain_attend(st):
    case = st["case"]
    B, nq, H, D, m, page, W = (case[k] for k in ("batch", "nq", "H", "D", "m", "page", "W"))
    pos, table, n_shared, scale = st["pos"].long(), st["table"].long(), st["n_shared"], st["scale"]
    q = st["q"].float()
    q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + 1e-6)
    if st["gain"] is not None:
        q = q * st["gain"]
    if st["rope"] is not None:
        at = pos.clamp(min=0)
        cos, sin = st["rope"][0][at][:, :, None], st["rope"][1][at][:, :, None]
        q = _rotate(q, cos, sin)

    def rows(pages):  # the entries of the pages, in 32 bits; pages that are not there come as zeros
        at = pages.clamp(min=0)
        r = _dequantised(st["pool8"][at], st["pool8e"][at]) if case["fp8"] else st["pool"][at].float()
        return r.flatten(-3, -2)

    win = _dequantised(st["win8"], st["win8e"]) if case["fp8"] else st["win"].float()
    n_vis = torch.div(pos + 1, m, rounding_mode="floor").clamp(0, table.shape[1] * page)  # [B][nq]
    shared_pages = n_shared // page
    # the shared prefix: one product for the rows of all requests
    k_sh = rows(table[0, :shared_pages])
    j_sh = torch.arange(n_shared, device=q.device)
    s_sh = (q.reshape(-1, D) @ k_sh.T).mul_(scale).reshape(B, nq, H, n_shared)
    s_sh.masked_fill_((j_sh >= n_vis[..., None])[:, :, None], -math.inf)
    # every request's own entries and its window
    k_own = rows(table[:, shared_pages:])
    j_own = n_shared + torch.arange(k_own.shape[1], device=q.device)
    see_own = j_own < n_vis[..., None]  # [B][nq][n]
    k_own = torch.where(see_own.any(1)[..., None], k_own, 0.0)
    s_own = torch.einsum("bqhd,bnd->bqhn", q, k_own) * scale
    s_own = s_own.masked_fill(~see_own[:, :, None], -math.inf)
    u = pos[..., None] - torch.arange(W, device=q.device)  # positions of the window
    see_win = u >= 0
    k_win = win[torch.arange(B, device=q.device)[:, None, None], u.clamp(min=0) % case["ring"]]  # [B][nq][W][D]
    s_win = (torch.einsum("bqhd,bqwd->bqhw", q, k_win) * scale).masked_fill(~see_win[:, :, None], -math.inf)
    # one softmax over the three
    top = torch.cat([s.amax(-1, keepdim=True) for s in (s_sh, s_own, s_win) if s.shape[-1]], -1).amax(-1, keepdim=True)
    if st["sinks"] is not None:
        top = torch.maximum(top, st["sinks"][:, None])
    top = top.masked_fill(top == -math.inf, 0.0)
    p_sh, p_own, p_win = (s_sh.sub_(top).exp_(), (s_own - top).exp(), (s_win - top).exp())
    total = p_sh.sum(-1, keepdim=True) + p_own.sum(-1, keepdim=True) + p_win.sum(-1, keepdim=True)
    if st["sinks"] is not None:
        total = total + (st["sinks"][:, None] - top).exp()
    out = (p_sh.reshape(B * nq * H, n_shared) @ k_sh).reshape(q.shape) + torch.einsum("bqhn,bnd->bqhd", p_own, k_own) \
        + torch.einsum("bqhw,bqwd->bqhd", p_win, k_win)
    out = torch.where(total > 0, out / total, 0.0)
    if st["rope"] is not None:
        out = _rotate(out, cos, -sin)
    return out.to(torch.bfloat16)


def _plain_plan(st):
    case = st["case"]
    m, page, ring = case["m"], case["page"], case["ring"]
    old, new, table, free = st["old"].long(), st["new"].long(), st["table"], st["free"]
    B, max_pages = table.shape
    e0, e1 = torch.div(old, m, rounding_mode="floor"), torch.div(old + new, m, rounding_mode="floor")
    held = torch.div(e0 + page - 1, page, rounding_mode="floor")
    need = torch.div(e1 + page - 1, page, rounding_mode="floor")
    zero = torch.zeros(1, dtype=torch.int64, device=old.device)
    cu_tokens = torch.cat([zero, new.cumsum(0)])
    cu_entries = torch.cat([zero, (e1 - e0).cumsum(0)])
    cu_pages = torch.cat([zero, (need - held).cumsum(0)])
    col = torch.arange(max_pages, device=old.device)
    fresh = (col >= held[:, None]) & (col < need[:, None])
    ids = free[(cu_pages[:-1, None] + col - held[:, None]).clamp(0, free.numel() - 1)]
    table.copy_(torch.where(fresh, ids, table))

    def owner(cu, cap):  # (request, number within it, whether there is one) of every place of a packed output
        i = torch.arange(cap, device=old.device)
        b = torch.searchsorted(cu[1:], i, right=True).clamp(max=B - 1)
        return b, i - cu[b], i < cu[-1]

    b, i, there = owner(cu_entries, st["max_entries"])
    e = e0[b] + i
    pg = table[b, torch.div(e, page, rounding_mode="floor").clamp(max=max_pages - 1)].long()
    entry_slots = torch.where(there, pg * page + e % page, -1)
    b, i, there = owner(cu_tokens, st["max_tokens"])
    pos = old[b] + i
    tok_pos = torch.where(there, pos, -1).to(torch.int32)
    win_slots = torch.where(there & (pos >= (old + new)[b] - ring), b * ring + pos % ring, -1)
    counts = torch.stack([cu_tokens[-1], cu_entries[-1], cu_pages[-1], cu_pages[-1] * 0])
    return table, cu_tokens, cu_entries, entry_slots, tok_pos, win_slots, counts


def _plain_write(st):
    case, slots = st["case"], st["slots"]
    keep = slots >= 0
    at, rows = slots[keep], st["rows"][keep]
    if not case["fp8"]:
        st["pool"][at] = rows
        return st["pool"]
    st["codes"][at], st["exps"][at] = _quantised(rows)
    return st["codes"].view(torch.float8_e4m3fn), st["exps"]


# ---------------------------------------------------------------------------------------------------- the calls
def _own_run(st):
    import long_context_compressed_06_b200 as csa
    case = st["case"]
    if case["op"] == "plan":
        plan = csa.csa_plan_pages(st["old"], st["new"], st["free"], st["table"], case["m"], case["page"], case["ring"],
                                  st["max_tokens"], st["max_entries"])
        return (st["table"],) + tuple(plan)
    if case["op"] == "write":
        if case["fp8"]:
            csa.csa_paged_write_fp8kv(st["rows"], st["slots"], st["codes"], st["exps"])
            return st["codes"].view(torch.float8_e4m3fn), st["exps"]
        return csa.csa_paged_write(st["rows"], st["slots"], st["pool"])
    if case["fp8"]:
        return csa.hca_attend_paged_fp8kv(st["q"], st["pool8"], st["pool8e"], st["table"], case["m"], st["win8"],
                                          st["win8e"], st["pos"], case["W"], st["scale"], q_gain=st["gain"],
                                          n_shared=st["n_shared"], sinks=st["sinks"], rope=st["rope"])
    return csa.hca_attend_paged(st["q"], st["pool"], st["table"], case["m"], st["win"], st["pos"], case["W"],
                                st["scale"], q_gain=st["gain"], n_shared=st["n_shared"], sinks=st["sinks"],
                                rope=st["rope"])


def run(state):
    if own:
        return _own_run(state)
    return {"attend": _plain_attend, "plan": _plain_plan, "write": _plain_write}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------------- in 64 bits
def _exact_rows(codes, exps):
    """The values of FP8 rows, decoded from the bit fields."""
    c = codes.to(torch.int64)
    e, f = (c >> 3) & 15, c & 7
    mag = torch.where(e == 0, f.double() * 2.0 ** -9, (8 + f).double() * torch.exp2((e - 10).double()))
    v = torch.where(c >= 128, -mag, mag)
    return v * torch.exp2(exps.double() - 127).repeat_interleave(128, -1)


def _exact_attend(case, st):
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    D, m, page = case["D"], case["m"], case["page"]
    pos, table = st["pos"].tolist(), st["table"].long()
    for b in range(case["batch"]):
        last = max(pos[b])
        if last < 0:
            continue
        n = min((last + 1) // m, table.shape[1] * page)
        ids = table[b, :-(-n // page)]
        if case["fp8"]:
            k = _exact_rows(st["pool8"][ids], st["pool8e"][ids]).reshape(-1, D)[:n]
        else:
            k = st["pool"][ids].double().reshape(-1, D)[:n]
        for i, t in enumerate(pos[b]):
            if t < 0:
                continue
            at = torch.arange(max(0, t - case["W"] + 1), t + 1, device="cuda") % case["ring"]
            w = _exact_rows(st["win8"][b, at], st["win8e"][b, at]) if case["fp8"] else st["win"][b, at].double()
            x = torch.cat([k[:(t + 1) // m], w])
            q = st["q"][b, i].double()
            q = q / (q.pow(2).mean(1, keepdim=True) + 1e-6).sqrt()
            if st["gain"] is not None:
                q = q * st["gain"].double()
            if st["rope"] is not None:
                turn = torch.complex(st["rope"][0][t].double(), st["rope"][1][t].double())
                z = torch.complex(q[:, -64:-32], q[:, -32:]) * turn
                q = torch.cat([q[:, :-64], z.real, z.imag], 1)
            s = (q @ x.T) * st["scale"]
            if st["sinks"] is not None:
                s = torch.cat([s, st["sinks"].double()[:, None]], 1)
            p = torch.softmax(s, 1)[:, :x.shape[0]]
            o = p @ x
            if st["rope"] is not None:
                z = torch.complex(o[:, -64:-32], o[:, -32:]) * turn.conj()
                o = torch.cat([o[:, :-64], z.real, z.imag], 1)
            out[b, i] = o
    return out


def _exact_write(case, st):
    slots, rows = st["slots"].tolist(), st["rows"].double()
    keep = [(i, s) for i, s in enumerate(slots) if s >= 0]
    src, dst = torch.tensor([i for i, _ in keep], device="cuda"), torch.tensor([s for _, s in keep], device="cuda")
    if not case["fp8"]:
        out = torch.zeros((case["slots"], case["D"]), dtype=torch.float64, device="cuda")
        out[dst] = rows[src]
        return out
    values = torch.zeros((case["slots"], case["D"]), dtype=torch.float64, device="cuda")
    blk = rows[src].reshape(len(keep), -1, 128)
    amax = blk.abs().amax(2, keepdim=True)
    k = torch.ceil(torch.log2(amax / 448)).nan_to_num(neginf=0.0)
    k = torch.where(amax > 448 * torch.exp2(k), k + 1, torch.where(amax <= 448 * torch.exp2(k - 1), k - 1, k))
    x = blk / torch.exp2(torch.where(amax == 0, 0.0, k.clamp(-124, 119)))
    # to the nearest e4m3 value, ties to even: steps of 2^(e - 3) in [2^e, 2^(e + 1)), 2^-9 below 2^-6
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    values[dst] = (torch.round(x / step) * step).clamp(-448, 448).reshape(len(keep), -1)
    return values, None


def exact(case, seed):
    """The operators' definitions in 64 bits (whole numbers, as the plan's and the exponents, have no such value)."""
    if case["op"] == "plan":
        return None
    st = prepare(case, seed)
    return _exact_attend(case, st) if case["op"] == "attend" else _exact_write(case, st)


# ---------------------------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "plan":
        old, new = _plan_lengths(case)
        m, page = case["m"], case["page"]
        pages = sum(-(-((o + n) // m) // page) - (-(-(o // m) // page)) for o, n in zip(old, new))
        entries = sum((o + n) // m - o // m for o, n in zip(old, new))
        return {"bytes": 8 * case["batch"] + 8 * pages + 16 * (case["batch"] + 1) + 8 * (entries + case["slack"])
                + 12 * (sum(new) + case["slack"]), "flops": 0}
    if case["op"] == "write":
        kept = case["rows"] - -(-case["rows"] // 17)
        D = case["D"]
        out = D + D // 128 if case["fp8"] else 2 * D
        return {"bytes": 8 * case["rows"] + kept * (2 * D + out), "flops": 0}
    B, nq, H, D, m = (case[k] for k in ("batch", "nq", "H", "D", "m"))
    row = D + D // 128 if case["fp8"] else 2 * D
    # which requests are empty slots depends on the seed: the average request stands for each
    live = B - case["pad"]
    own_entries = sum(_suffixes(case)) * live / B
    keys = live * (case["shared"] + case["W"]) + own_entries
    entries = case["shared"] + own_entries + live * (case["W"] + nq - 1)
    return {"bytes": 4 * B * nq * H * D + entries * row, "flops": 4 * D * H * nq * keys}

"""GPU parity of the paged-cache operators against plain implementations in 64 bits.

Tolerance of the attention, element by element, from its roundings (bf16: half a step is 2^-8 of the value):
  * the output is rounded once:                                        2^-8 |o|
  * the weights p_j are rounded to bf16 for the second product:       2^-8 A,  A = sum_j p_j |x_j| / sum_j p_j
  * with a gain or RoPE the query is rounded to bf16 first, which moves every score by at most
    e = 2^-8 scale sum_d |q_d x_d| and the normalised weights by at most exp(2 e) - 1:  (exp(2 e) - 1) A
  * products and sums in 32 bits (512 terms, truncating tensor-core sums included): 2^-10 A
A rotated output mixes pairs of channels: their A enters by |cos| and |sin|.
"""
import numpy as np
import pytest
import torch

import long_context_compressed_06_b200 as csa_pkg  # noqa: F401
from long_context_compressed_06_b200 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


# ----------------------------------------------------------------------------- page plan
def plan_ref(old, new, free, table, m, page, ring, max_tokens, max_entries):
    table = table.copy()
    max_pages = table.shape[1]
    slots, pos, win, cu_t, cu_e = [], [], [], [0], [0]
    taken = cut = lacking = 0
    for b, (o, n) in enumerate(zip(old.tolist(), new.tolist())):
        if o < 0 or n < 0 or o + n > 2 ** 31 - 1:
            o = n = 0
        e0, e1 = o // m, (o + n) // m
        h, p = -(-e0 // page), -(-e1 // page)
        for j in range(h, p):
            if j >= max_pages:
                cut += 1
                continue
            if taken < len(free):
                table[b, j] = free[taken]
            else:
                table[b, j] = -1
                lacking += 1
            taken += 1
        for e in range(e0, e1):
            j = e // page
            pg = table[b, j] if j < max_pages else -1
            slots.append(pg * page + e % page if pg >= 0 else -1)
        for u in range(o, o + n):
            pos.append(u)
            win.append(b * ring + u % ring if u >= o + n - ring else -1)
        cu_t.append(len(pos))
        cu_e.append(len(slots))

    def pad(v, n, t):
        return np.array((v + [-1] * n)[:n], dtype=t)

    return (table, np.array(cu_t, np.int64), np.array(cu_e, np.int64), pad(slots, max_entries, np.int64),
            pad(pos, max_tokens, np.int32), pad(win, max_tokens, np.int64),
            np.array([cu_t[-1], cu_e[-1], taken, cut + lacking], np.int64))


def plan_case(batch, old_hi, new_hi, m, page, ring, seed, max_pages=None, free=None):
    rng = np.random.default_rng(seed)
    old = rng.integers(0, old_hi + 1, batch).astype(np.int32)
    new = rng.integers(0, new_hi + 1, batch).astype(np.int32)
    need = -(-((old.astype(np.int64) + new) // m) // page)
    held = -(-(old.astype(np.int64) // m) // page)
    if max_pages is None:
        max_pages = int(need.max()) + 2
    total = int(np.maximum(need, 1).sum()) + 8
    ids = rng.permutation(total).astype(np.int32)
    table = rng.integers(-5, 0, (batch, max_pages)).astype(np.int32)
    at = 0
    for b in range(batch):
        for j in range(min(held[b], max_pages)):
            table[b, j] = ids[at]
            at += 1
    fr = ids[at:] if free is None else ids[at:at + free]
    return old, new, fr, table


def check_plan(csa, old, new, fr, table, m, page, ring, max_tokens, max_entries):
    t = torch.tensor(table, device=DEV)
    args = [torch.tensor(x, device=DEV) for x in (old, new, fr)]
    ref = plan_ref(old, new, fr, table, m, page, ring, max_tokens, max_entries)
    got = None
    for _ in range(2):  # the second call finds the first one's pages noted: same answer
        got = csa.csa_plan_pages(*args, t, m, page, ring, max_tokens, max_entries, out=got)
        for name, g, r in zip(("table", "cu_tokens", "cu_entries", "entry_slots", "tok_pos", "win_slots", "counts"),
                              (t,) + tuple(got), ref):
            assert np.array_equal(g.cpu().numpy(), r), name


@pytest.mark.parametrize("batch,old,new,m,page,ring", [
    (1, 0, 1, 1, 1, 1),
    (1, 0, 5000, 4, 16, 7),
    (3, 130, 9, 4, 16, 128),
    (37, 1000, 1, 1, 16, 131),
    (97, 700, 300, 128, 3, 16),
    (513, 90, 40, 4, 5, 16),
    (6001, 9, 9, 3, 2, 5),
    (16384, 50, 3, 1, 16, 8),
    (16385, 50, 3, 1, 16, 8),     # the two-launch form
])
def test_plan_pages(cuda, batch, old, new, m, page, ring):
    o, n, fr, table = plan_case(batch, old, new, m, page, ring, batch + new)
    tokens = int(n.sum())
    entries = int(((o.astype(np.int64) + n) // m - o // m).sum())
    check_plan(cuda, o, n, fr, table, m, page, ring, tokens, entries)
    check_plan(cuda, o, n, fr, table, m, page, ring, tokens + 777, entries + 2500)
    check_plan(cuda, o, n, fr, table, m, page, ring, tokens // 2, entries // 3)   # cut
    check_plan(cuda, o, n, fr, table, m, page, ring, 0, 0)


def test_plan_pages_out_of_pages_and_columns(cuda):
    o, n, fr, table = plan_case(20, 400, 300, 4, 16, 128, 3, max_pages=9, free=5)
    check_plan(cuda, o, n, fr, table, 4, 16, 128, int(n.sum()), 3000)
    o, n, fr, table = plan_case(17000, 40, 30, 4, 2, 128, 4, max_pages=6, free=100)
    check_plan(cuda, o, n, fr, table, 4, 2, 128, int(n.sum()), 70000)


def test_plan_pages_bad_lengths_count_as_empty(cuda):
    o, n, fr, table = plan_case(9, 200, 100, 4, 16, 128, 5)
    o[2], n[4], o[6], n[6] = -1, -7, 2 ** 31 - 1, 5
    n[8] = 0
    check_plan(cuda, o, n, fr, table, 4, 16, 128, 600, 200)


def test_plan_pages_graph_replay_follows_the_lengths(cuda):
    o, n, fr, table = plan_case(33, 300, 60, 4, 16, 32, 6)
    t0 = torch.tensor(table, device=DEV)
    t = t0.clone()
    do, dn, df = (torch.tensor(x, device=DEV) for x in (o, n, fr))
    out = cuda.csa_plan_pages(do, dn, df, t, 4, 16, 32, 3000, 800)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cuda.csa_plan_pages(do, dn, df, t, 4, 16, 32, 3000, 800, out=out)
    n2 = (n // 2).astype(np.int32)
    dn.copy_(torch.tensor(n2))
    t.copy_(t0)
    g.replay()
    ref = plan_ref(o, n2, fr, table, 4, 16, 32, 3000, 800)
    for got, r in zip((t,) + tuple(out), ref):
        assert np.array_equal(got.cpu().numpy(), r)


# ----------------------------------------------------------------------------- paged writes
@pytest.mark.parametrize("n,d,slots", [(0, 64, 5), (1, 8, 1), (7, 72, 40), (300, 512, 301), (1025, 128, 4000)])
def test_paged_write(cuda, n, d, slots):
    rng = np.random.default_rng(n + d)
    rows = W.normal_bf16((n, d), 40 + n, DEV)
    at = rng.permutation(slots)[:n].astype(np.int64)
    at[::5] = -1
    at[1::11] = slots + 3
    at[2::13] = 2 ** 40
    pool = W.normal_bf16((slots, d), 41, DEV)
    ref = pool.clone()
    for i, s in enumerate(at.tolist()):
        if 0 <= s < slots:
            ref[s] = rows[i]
    got = cuda.csa_paged_write(rows, torch.tensor(at, device=DEV), pool)
    assert got is pool and torch.equal(pool.view(torch.int16), ref.view(torch.int16))


@pytest.mark.parametrize("n,d,slots", [(1, 128, 1), (5, 384, 9), (333, 512, 400), (1030, 256, 2000)])
def test_paged_write_fp8kv(cuda, n, d, slots):
    rng = np.random.default_rng(n + d)
    rows = W.normal_bf16((n, d), 50 + n, DEV) * torch.exp2(torch.randint(-20, 20, (n, 1), device=DEV).float()).bfloat16()
    rows[n // 2] = 0
    at = rng.permutation(slots)[:n].astype(np.int64)
    at[3::7] = -1
    codes = torch.randint(0, 127, (slots, d), dtype=torch.uint8, device=DEV)
    exps = torch.randint(0, 255, (slots, d // 128), dtype=torch.uint8, device=DEV)
    rc, re = codes.clone(), exps.clone()
    c, e = cuda.csa_quantize_fp8_kv(rows)
    for i, s in enumerate(at.tolist()):
        if s >= 0:
            rc[s], re[s] = c[i], e[i]
    cuda.csa_paged_write_fp8kv(rows, torch.tensor(at, device=DEV), codes, exps)
    assert torch.equal(codes, rc) and torch.equal(exps, re)


# ----------------------------------------------------------------------------- paged attention
def dequant(codes, exps):
    v = codes.cpu().view(torch.float8_e4m3fn).double().unflatten(-1, (-1, 128))
    return (v * torch.exp2(exps.cpu().double() - 127).unsqueeze(-1)).flatten(-2).numpy()


def attend_ref(q, pool, table, m, ring, pos, Wn, scale, eps, gain, sinks, rope):
    """-> (out, A, e): see the tolerance above.  pool and ring in 64 bits; rows outside the key sets may be NaN."""
    B, nq, H, D = q.shape
    n_pages, page = pool.shape[:2]
    out, mag, eps_s = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, nq, H, 1))
    for b in range(B):
        for i in range(nq):
            t = int(pos[b, i])
            if t < 0:
                continue
            ids = [(int(table[b, j // page]), j % page) for j in range(min((t + 1) // m, table.shape[1] * page))]
            rows = [pool[p, r] for p, r in ids if 0 <= p < n_pages]
            rows += [ring[b, u % ring.shape[1]] for u in range(max(0, t - Wn + 1), t + 1)]
            x = np.array(rows)
            y = q[b, i] / np.sqrt((q[b, i] ** 2).mean(-1, keepdims=True) + eps)
            if gain is not None:
                y = y * gain
            rot = rope is not None and t < rope[0].shape[0]
            if rot:
                c, s = rope[0][t], rope[1][t]
                u, v = y[:, -64:-32].copy(), y[:, -32:].copy()
                y[:, -64:-32], y[:, -32:] = u * c - v * s, v * c + u * s
            z = y @ x.T * scale
            top = z.max(-1, keepdims=True)
            if sinks is not None:
                top = np.maximum(top, sinks[:, None])
            p = np.exp(z - top)
            L = p.sum(-1, keepdims=True) + (np.exp(sinks[:, None] - top) if sinks is not None else 0)
            o, a = p @ x / L, p @ np.abs(x) / L
            if rot:
                u, v = o[:, -64:-32].copy(), o[:, -32:].copy()
                o[:, -64:-32], o[:, -32:] = u * c + v * s, v * c - u * s
                u, v = a[:, -64:-32].copy(), a[:, -32:].copy()
                a[:, -64:-32], a[:, -32:] = u * abs(c) + v * abs(s), v * abs(c) + u * abs(s)
            out[b, i], mag[b, i] = o, a
            if gain is not None or rope is not None:
                eps_s[b, i] = 2.0 ** -8 * abs(scale) * (np.abs(y) @ np.abs(x).T).max(-1, keepdims=True)
    return out, mag, eps_s


def tables(n):
    ang = np.arange(n)[:, None] * 10000.0 ** (-np.arange(32) / 32)
    return np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)


class Case:
    """Inputs of one call: ts[b][i] positions (-1: empty slot); the pool holds NaN wherever no query's key set reaches."""

    def __init__(self, ts, H, D, m, page, n_shared, Wn, ring_extra=0, fp8=False, gain=False, sinks=False, rope=False,
                 seed=1, drop=(), cols=1, nan=True, scale=None):
        ts = np.array(ts, np.int32)
        B, nq = ts.shape
        rng = np.random.default_rng(seed)
        self.m, self.Wn, self.n_shared, self.page = m, Wn, n_shared, page
        sp = n_shared // page
        vis = np.maximum((ts.max(1).astype(np.int64) + 1) // m, 0)
        own = [max(0, -(-int(v) // page) - sp) for v in vis]
        self.max_pages = max(1, sp + max(own) + cols)
        n_pages = sp + sum(own) + 3
        ids = rng.permutation(n_pages).astype(np.int32)
        table = np.full((B, self.max_pages), -1, np.int32)
        table[:, :sp] = ids[:sp]
        at = sp
        used = np.zeros((n_pages, page), bool)
        for j in range(min(n_shared, int(vis.max()))):
            used[ids[j // page], j % page] = True
        for b in range(B):
            for k in range(own[b]):
                table[b, sp + k] = ids[at]
                used[ids[at], :max(0, min(page, int(vis[b]) - (sp + k) * page))] = True
                at += 1
        for b, j, v in drop:  # pages that are not there
            if b is None:
                table[:, j] = v
            else:
                table[b, j] = v
        self.table = torch.tensor(table, device=DEV)
        self.q = W.normal_bf16((B, nq, H, D), seed + 100, DEV)
        pool = W.normal_bf16((n_pages, page, D), seed + 200, DEV)
        ring = W.normal_bf16((B, Wn + nq - 1 + ring_extra, D), seed + 300, DEV)
        rows = np.zeros(ring.shape[:2], bool)
        for b in range(B):
            for t in ts[b]:
                for u in range(max(0, int(t) - Wn + 1), int(t) + 1):
                    rows[b, u % ring.shape[1]] = True
        self.fp8 = fp8
        if fp8:
            self.pool, self.pe = csa_pkg.csa_quantize_fp8_kv(pool)
            self.ring, self.re = csa_pkg.csa_quantize_fp8_kv(ring)
            if nan:
                self.pool[torch.tensor(~used)] = 0x7F
                self.pe[torch.tensor(~used)] = 255
                self.ring[torch.tensor(~rows)] = 0x7F
            self.pool64, self.ring64 = dequant(self.pool, self.pe), dequant(self.ring, self.re)
        else:
            if nan:
                pool[torch.tensor(~used)] = float("nan")
                ring[torch.tensor(~rows)] = float("nan")
            self.pool, self.ring = pool, ring
            self.pool64, self.ring64 = f64(pool), f64(ring)
        self.pos = torch.tensor(ts, device=DEV)
        self.scale = D ** -0.5 if scale is None else scale
        self.gain = W.uniform_f32((D,), seed + 400, DEV) + 0.5 if gain else None
        self.sinks = W.uniform_f32((H,), seed + 500, DEV) * 4 - 1 if sinks else None
        self.rope = None
        if rope:
            self.rope_np = tables(int(ts.max()) + 1 if rope is True else rope)
            self.rope = tuple(torch.tensor(x, device=DEV) for x in self.rope_np)

    def run(self, csa, n_shared=None, **kw):
        kw = dict(q_gain=self.gain, sinks=self.sinks, rope=self.rope,
                  n_shared=self.n_shared if n_shared is None else n_shared, **kw)
        if self.fp8:
            return csa.hca_attend_paged_fp8kv(self.q, self.pool, self.pe, self.table, self.m, self.ring, self.re, self.pos,
                                              self.Wn, self.scale, **kw)
        return csa.hca_attend_paged(self.q, self.pool, self.table, self.m, self.ring, self.pos, self.Wn, self.scale, **kw)

    def ref(self):
        g = None if self.gain is None else f64(self.gain)
        s = None if self.sinks is None else f64(self.sinks)
        r = None if self.rope is None else tuple(x.astype(np.float64) for x in self.rope_np)
        return attend_ref(f64(self.q), self.pool64, self.table.cpu().numpy(), self.m, self.ring64, self.pos.cpu().numpy(),
                          self.Wn, self.scale, 1e-6, g, s, r)

    def check(self, got, ref=None):
        out, mag, e = ref or self.ref()
        tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + np.expm1(2 * e) + 2.0 ** -10) * mag
        err = np.abs(f64(got) - out)
        assert np.isfinite(f64(got)).all()
        assert (err <= tol).all(), (float((err - tol).max()), np.argwhere(err > tol)[:4].tolist())


CASES = {
    # positions, H, D, m, page, n_shared, W
    "one_token": dict(ts=[[0]], H=1, D=64, m=4, page=16, n_shared=0, Wn=4),
    "no_entries": dict(ts=[[2], [1]], H=8, D=128, m=4, page=16, n_shared=0, Wn=16),
    "own_only": dict(ts=[[399], [40], [-1], [1201]], H=8, D=64, m=4, page=32, n_shared=0, Wn=16),
    "own_h128": dict(ts=[[2100], [1300]], H=128, D=512, m=4, page=48, n_shared=0, Wn=128, sinks=True),
    "own_rope": dict(ts=[[2100, 2101], [1300, 1301]], H=64, D=128, m=4, page=16, n_shared=0, Wn=32, rope=True, gain=True),
    "shared_one_page": dict(ts=[[400], [70], [64]], H=8, D=64, m=4, page=16, n_shared=16, Wn=16),
    "shared_tile": dict(ts=[[600], [520], [511]], H=16, D=128, m=4, page=128, n_shared=128, Wn=16),
    "shared_odd": dict(ts=[[1003], [900], [800], [-1], [700]], H=40, D=128, m=4, page=48, n_shared=144, Wn=16, ring_extra=3),
    "shared_256": dict(ts=[[2600], [2500]], H=3, D=256, m=4, page=80, n_shared=560, Wn=16, sinks=True),
    "shared_512": dict(ts=[[1700], [1690], [1650]], H=128, D=512, m=4, page=32, n_shared=384, Wn=128),
    "shared_512_odd": dict(ts=[[700], [690], [650]], H=72, D=512, m=2, page=16, n_shared=304, Wn=8, gain=True),
    "shared_rope_64": dict(ts=[[700, 701], [690, 691]], H=24, D=64, m=2, page=16, n_shared=272, Wn=8, rope=True),
    "shared_rope_128": dict(ts=[[700, 701], [690, 691]], H=24, D=128, m=2, page=64, n_shared=320, Wn=8, rope=True, gain=True),
    "shared_rope_256": dict(ts=[[700], [690]], H=100, D=256, m=2, page=64, n_shared=320, Wn=8, rope=300, sinks=True),
    "shared_rope_512": dict(ts=[[700], [690]], H=128, D=512, m=2, page=64, n_shared=320, Wn=8, rope=True, gain=True,
                            sinks=True),
    # queries that see only part of the shared entries, none of them, entries that nobody sees (NaN)
    "part_seen": dict(ts=[[11], [399], [-1], [777]], H=40, D=128, m=4, page=16, n_shared=320, Wn=16),
    "part_seen_512": dict(ts=[[0], [333], [555]], H=128, D=512, m=1, page=64, n_shared=1024, Wn=16),
    "part_seen_256": dict(ts=[[0, 1, 2], [331, 332, 333]], H=20, D=256, m=1, page=32, n_shared=512, Wn=16),
    "none_seen": dict(ts=[[2], [1]], H=8, D=64, m=4, page=16, n_shared=64, Wn=16),
    "all_empty": dict(ts=[[-1], [-1]], H=8, D=64, m=4, page=16, n_shared=64, Wn=16),
    "row_tiles": dict(ts=[[900 + 3 * i] for i in range(37)], H=8, D=64, m=4, page=16, n_shared=208, Wn=16),
    # several row tiles per pair of SMs, shared and own tiles in turn
    "many_ranges_64": dict(ts=[[790 + 7 * i] for i in range(150)], H=64, D=64, m=2, page=16, n_shared=384, Wn=40),
    "many_ranges_128": dict(ts=[[790 + 7 * (i % 50)] for i in range(250)], H=40, D=128, m=2, page=32, n_shared=352, Wn=16),
    "many_ranges_256": dict(ts=[[700 + 9 * i] for i in range(80)], H=128, D=256, m=4, page=64, n_shared=128, Wn=30),
    "many_ranges_512": dict(ts=[[700 + 9 * i] for i in range(80)], H=128, D=512, m=4, page=16, n_shared=160, Wn=30),
    "many_ranges_fp8": dict(ts=[[700 + 9 * i] for i in range(80)], H=128, D=512, m=4, page=64, n_shared=128, Wn=30,
                            fp8=True),
    "long_own": dict(ts=[[1200], [9000], [300]], H=128, D=128, m=2, page=64, n_shared=128, Wn=128),
    "many_units": dict(ts=[[30000 + 100 * i] for i in range(3)], H=4, D=64, m=2, page=64, n_shared=14976, Wn=16),
    "many_units_128": dict(ts=[[25000 + 100 * i] for i in range(5)], H=64, D=128, m=8, page=16, n_shared=3056, Wn=16),
    "pages_missing": dict(ts=[[700], [690], [650]], H=16, D=128, m=2, page=16, n_shared=304, Wn=8,
                          drop=((None, 3, -1), (None, 9, 10 ** 6), (1, 19, -7))),
    "pages_missing_512": dict(ts=[[700], [690]], H=128, D=512, m=2, page=64, n_shared=320, Wn=8, drop=((None, 1, -1),)),
    "big_scale": dict(ts=[[900], [890]], H=16, D=128, m=2, page=16, n_shared=432, Wn=16, scale=3.0),
    "negative_scale": dict(ts=[[900], [890]], H=16, D=128, m=2, page=16, n_shared=432, Wn=16, scale=-0.3),
    "zero_scale": dict(ts=[[400], [890]], H=16, D=128, m=2, page=16, n_shared=432, Wn=16, scale=0.0),
    "fp8_own": dict(ts=[[700], [41], [-1]], H=16, D=128, m=2, page=16, n_shared=0, Wn=8, fp8=True),
    "fp8_shared": dict(ts=[[700], [690], [650]], H=40, D=128, m=2, page=16, n_shared=304, Wn=8, fp8=True,
                       drop=((None, 3, -1),)),
    "fp8_512": dict(ts=[[1700], [1690]], H=128, D=512, m=4, page=48, n_shared=384, Wn=64, fp8=True, sinks=True),
    "fp8_part_seen": dict(ts=[[0], [333]], H=16, D=256, m=1, page=16, n_shared=512, Wn=16, fp8=True, rope=True),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_attend_paged(cuda, name):
    c = Case(**CASES[name])
    ref = c.ref()
    for n_shared in sorted({0, c.n_shared}):
        got = c.run(cuda, n_shared=n_shared)
        assert cuda.csa_sync_status() == 0
        c.check(got, ref)
    empty = (c.pos < 0).cpu()
    assert (got.cpu()[empty] == 0).all()

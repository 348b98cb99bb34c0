"""GPU parity of the paged-cache operators against plain implementations in 64 bits.

Tolerance of the attention, element by element, from its roundings (bf16: half a step is 2^-8 of the value):
  * the output is rounded once:                                        2^-8 |o|
  * the weights p_j are rounded to bf16 for the second product:       2^-8 A,  A = sum_j p_j |x_j| / sum_j p_j
  * with a gain or RoPE the query is rounded first, to the sum of two bf16 numbers (query by query at D = 512: to
    one), which moves every score by at most e = 2^-16 (2^-8) scale sum_d |q_d x_d|, plus 2^-20 of it for the 32-bit
    arithmetic, and the normalised weights by at most exp(2 e) - 1:  (exp(2 e) - 1) A
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
    v = codes.view(torch.float8_e4m3fn).float().double().unflatten(-1, (-1, 128))
    return (v * torch.exp2(exps.double() - 127).unsqueeze(-1)).flatten(-2)


def attend_ref(q, pool, table, m, ring, pos, Wn, scale, eps, gain, sinks, rope):
    """-> (out, A, e): see the tolerance above.  64-bit tensors on the GPU; pool and ring rows outside the key sets may
    be NaN."""
    B, nq, H, D = q.shape
    n_pages, page = pool.shape[:2]
    out, mag, eps_s = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q[..., :1])
    for b in range(B):
        for i in range(nq):
            t = int(pos[b, i])
            if t < 0:
                continue
            j = torch.arange(min((t + 1) // m, table.shape[1] * page), device=DEV)
            ids = table[b].long()[j // page]
            there = (ids >= 0) & (ids < n_pages)
            u = torch.arange(max(0, t - Wn + 1), t + 1, device=DEV)
            x = torch.cat([pool[ids[there], j[there] % page], ring[b, u % ring.shape[1]]])
            y = q[b, i] / (q[b, i].pow(2).mean(-1, keepdim=True) + eps).sqrt()
            if gain is not None:
                y = y * gain
            rot = rope is not None and t < rope[0].shape[0]
            if rot:
                c, s = rope[0][t], rope[1][t]
                u, v = y[:, -64:-32].clone(), y[:, -32:].clone()
                y[:, -64:-32], y[:, -32:] = u * c - v * s, v * c + u * s
            z = y @ x.T * scale
            top = z.amax(-1, keepdim=True)
            if sinks is not None:
                top = torch.maximum(top, sinks[:, None])
            p = (z - top).exp()
            total = p.sum(-1, keepdim=True) + ((sinks[:, None] - top).exp() if sinks is not None else 0)
            o, a = p @ x / total, p @ x.abs() / total
            if rot:
                u, v = o[:, -64:-32].clone(), o[:, -32:].clone()
                o[:, -64:-32], o[:, -32:] = u * c + v * s, v * c - u * s
                u, v = a[:, -64:-32].clone(), a[:, -32:].clone()
                a[:, -64:-32], a[:, -32:] = u * c.abs() + v * s.abs(), v * c.abs() + u * s.abs()
            out[b, i], mag[b, i] = o, a
            if gain is not None or rope is not None:
                eps_s[b, i] = (2.0 ** -16 + 2.0 ** -20) * abs(scale) * (y.abs() @ x.abs().T).amax(-1, keepdim=True)
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
            self.pool64, self.ring64 = pool.double(), ring.double()
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

    def ref(self, at=slice(None)):
        def d(x):
            return None if x is None else x.double()
        return attend_ref(self.q[at].double(), self.pool64, self.table[at], self.m, self.ring64[at], self.pos[at].cpu(),
                          self.Wn, self.scale, 1e-6, d(self.gain), d(self.sinks),
                          None if self.rope is None else tuple(d(x) for x in self.rope))

    def check(self, got, ref=None, n_shared=None):
        out, mag, e = ref or self.ref()
        if self.q.shape[-1] == 512 and not self.by_row_tiles(n_shared):
            e = e * 256
        tol = 2.0 ** -8 * out.abs() + (2.0 ** -8 + torch.expm1(2 * e) + 2.0 ** -10) * mag
        err = (got.double() - out).abs()
        assert got.isfinite().all()
        assert (err <= tol).all(), (float((err - tol).max()), (err > tol).nonzero()[:4].tolist())

    def workspace_bytes(self, n_shared=None):
        return csa_pkg.attend_paged_workspace_bytes(*self.q.shape, self.page, self.max_pages,
                                                    self.n_shared if n_shared is None else n_shared, self.ring.shape[1],
                                                    self.Wn, self.fp8, self.rewrite())

    def rewrite(self):
        return self.gain is not None or self.rope is not None or self.scale < 0

    def by_row_tiles(self, n_shared=None):
        """Whether the call takes the kernel over row tiles of the whole batch: its workspace holds a partial per pair
        of SMs and row tile."""
        n_shared = self.n_shared if n_shared is None else n_shared
        B, nq, H, D = self.q.shape
        tiles = -(-B * nq * H // 128)
        parts = torch.cuda.get_device_properties(0).multi_processor_count // 2 + tiles
        want = [parts * 128 * max(D, 128) * 4, parts * 128 * 8, tiles * 8]
        if self.rewrite():
            want += [B * nq * H * D * 2, B * nq * H * D * 2, B * nq * H * 4]
        if self.fp8:
            want.append((n_shared + B * (self.max_pages * self.page - n_shared + self.ring.shape[1])) * D * 2)
        return self.workspace_bytes(n_shared) == sum(-(-w // 256) * 256 for w in want)


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
        c.check(got, ref, n_shared)
    empty = (c.pos < 0).cpu()
    assert (got.cpu()[empty] == 0).all()


def spread(lo, hi, n, nq=1, also=()):
    """n sequences' positions from lo to hi, every few of them one of `also`."""
    ts = [lo + (hi - lo) * ((i * 37) % n) // n for i in range(n)]
    for i, t in enumerate(also):
        ts[(i * 7 + 3) % n] = t
    return [[t - nq + 1 + k if t >= nq - 1 else (t if k == nq - 1 else -1) for k in range(nq)] for t in ts]


# Sizes at which the estimate prefers the kernel over row tiles; its tile edges, masks and hand-overs.
ROW_TILES = {
    "d64_h8": dict(ts=spread(4103, 4600, 64), H=8, D=64, m=2, page=16, n_shared=2048, Wn=16),
    "d64_h3": dict(ts=spread(4103, 4600, 150), H=3, D=64, m=2, page=48, n_shared=1968, Wn=5, sinks=True),
    "d64_h1": dict(ts=spread(4103, 4300, 200, nq=2), H=1, D=64, m=2, page=32, n_shared=2048, Wn=16),
    "d128_h16": dict(ts=spread(4103, 5600, 64), H=16, D=128, m=2, page=64, n_shared=2048, Wn=128, ring_extra=3),
    "d128_h40_rope": dict(ts=spread(2103, 2700, 60), H=40, D=128, m=1, page=80, n_shared=2080, Wn=16, rope=True),
    "d128_h64_nq4": dict(ts=spread(2103, 2700, 20, nq=4), H=64, D=128, m=1, page=16, n_shared=2000, Wn=33, gain=True,
                         sinks=True),
    "d256_h100": dict(ts=spread(2103, 2700, 40), H=100, D=256, m=1, page=32, n_shared=2016, Wn=16, rope=1000, gain=True),
    "d256_h64": dict(ts=spread(2103, 2700, 40), H=64, D=256, m=1, page=64, n_shared=1984, Wn=128),
    "d512_h128": dict(ts=spread(2103, 2700, 24), H=128, D=512, m=1, page=64, n_shared=2048, Wn=128),
    "d512_h128_page16": dict(ts=spread(2103, 2500, 24), H=128, D=512, m=1, page=16, n_shared=1936, Wn=100, ring_extra=7),
    "d512_h128_nq4": dict(ts=spread(2103, 2300, 8, nq=4), H=128, D=512, m=1, page=32, n_shared=2016, Wn=128, rope=True,
                          gain=True, sinks=True),
    "d512_h72": dict(ts=spread(2103, 2300, 40), H=72, D=512, m=1, page=128, n_shared=1920, Wn=16),
    "d512_own_only": dict(ts=spread(300, 3500, 24), H=128, D=512, m=1, page=64, n_shared=0, Wn=128),
    "d128_own_only": dict(ts=spread(300, 5500, 40, also=(-1, 0, 1, 15, 16)), H=64, D=128, m=1, page=16, n_shared=0, Wn=17),
    # few entries seen, or none; entries that nobody sees hold NaN
    "part_seen_128": dict(ts=spread(2103, 2300, 60, also=(-1, 0, 1, 127, 128, 129, 255, 1000, -1)), H=40, D=128, m=1, page=16,
                          n_shared=2000, Wn=16),
    "part_seen_512": dict(ts=spread(900, 1100, 40, also=(-1, 0, 1, 127, 128, 511)), H=128, D=512, m=1, page=64, n_shared=2048,
                          Wn=16),
    "part_seen_256": dict(ts=spread(900, 1100, 60, also=(-1, 0, 1, 127, 128, 511)), H=64, D=256, m=1, page=16, n_shared=1600,
                          Wn=16),
    "part_seen_64": dict(ts=spread(1000, 1200, 100, also=(-1, 0, 1, 127, 128, 511)), H=8, D=64, m=1, page=32, n_shared=3200,
                         Wn=16, sinks=True),
    "short_windows": dict(ts=spread(2048, 2060, 64, also=(0, 3, 14, 15)), H=16, D=128, m=1, page=16, n_shared=2048, Wn=100,
                          ring_extra=50),
    "missing_128": dict(ts=spread(2103, 2300, 60), H=40, D=128, m=1, page=16, n_shared=2000, Wn=16,
                        drop=((None, 3, -1), (None, 90, 10 ** 6), (1, 126, -7), (59, 128, 10 ** 6))),
    "missing_512": dict(ts=spread(2103, 2300, 24), H=128, D=512, m=1, page=64, n_shared=1984, Wn=16,
                        drop=((None, 1, -1), (5, 32, -1))),
    "big_scale": dict(ts=spread(2103, 2300, 60), H=40, D=128, m=1, page=16, n_shared=2000, Wn=16, scale=3.0),
    "negative_scale": dict(ts=spread(2103, 2300, 60), H=40, D=128, m=1, page=16, n_shared=2000, Wn=16, scale=-0.3, rope=True),
    "zero_scale": dict(ts=spread(2103, 2300, 60, also=(5,)), H=40, D=128, m=1, page=16, n_shared=2000, Wn=16, scale=0.0),
    "fp8_128": dict(ts=spread(1103, 1300, 60, also=(-1, 0, 100)), H=40, D=128, m=1, page=16, n_shared=1008, Wn=16, fp8=True,
                    drop=((None, 3, -1), (2, 65, -1))),
    "fp8_512": dict(ts=spread(2103, 2300, 24), H=128, D=512, m=2, page=48, n_shared=960, Wn=128, fp8=True, rope=True),
    "fp8_256_own": dict(ts=spread(300, 2300, 60), H=64, D=256, m=1, page=32, n_shared=0, Wn=30, fp8=True),
}


@pytest.mark.parametrize("name", sorted(ROW_TILES))
def test_attend_paged_row_tiles(cuda, name):
    c = Case(**ROW_TILES[name])
    assert c.by_row_tiles()
    # whatever workspace and output held before
    ws = torch.full((c.workspace_bytes(),), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full_like(c.q, float("nan"))
    got = c.run(cuda, workspace=ws, out=out)
    assert cuda.csa_sync_status() == 0
    assert got.data_ptr() == out.data_ptr()
    c.check(got)
    again = c.run(cuda)
    assert torch.equal(again.view(torch.int16), got.view(torch.int16))  # the same sums in the same order
    assert (got[c.pos < 0] == 0).all()


@pytest.mark.parametrize("kw", [
    CASES["own_only"], CASES["part_seen"], ROW_TILES["part_seen_128"], ROW_TILES["d128_own_only"], ROW_TILES["fp8_128"],
    dict(ROW_TILES["part_seen_512"], rope=True, gain=True, sinks=True), dict(ROW_TILES["part_seen_64"], gain=True)])
def test_attend_paged_empty_slots_hold_anything(cuda, kw):
    """The query of an empty slot of the batch may be NaN or infinite: its output is zero, the others' theirs."""
    c = Case(**kw)
    empty = c.pos < 0
    assert empty.any()
    c.q[empty] = torch.where(torch.arange(c.q.shape[-1], device=DEV) % 2 == 0, float("nan"), float("inf")).to(c.q.dtype)
    got = c.run(cuda)
    assert cuda.csa_sync_status() == 0
    assert (got[empty] == 0).all()
    c.check(got)


@pytest.mark.parametrize("name", ["d512_h128_nq4", "d256_h100", "part_rope"])
def test_attend_paged_tables_aligned_to_their_elements(cuda, name):
    """Gain and RoPE tables that start at an odd float; positions past the tables, and empty slots."""
    kw = ROW_TILES[name] if name in ROW_TILES else dict(ROW_TILES["part_seen_512"], rope=100, gain=True)
    c = Case(**kw)
    before = c.run(cuda)
    def odd(x):
        y = torch.empty(x.numel() + 1, dtype=x.dtype, device=DEV)[1:].view(x.shape)
        return y.copy_(x)
    c.gain, c.rope = odd(c.gain), tuple(odd(x) for x in c.rope)
    assert c.gain.data_ptr() % 16 == 4
    got = c.run(cuda)
    assert cuda.csa_sync_status() == 0
    assert torch.equal(got.view(torch.int16), before.view(torch.int16))
    c.check(got)


@pytest.mark.parametrize("kw", [
    dict(ts=[[0], [0], [-1], [0]], H=8, D=64, m=4, page=16, n_shared=0, Wn=4),
    dict(ts=[[0]] * 40, H=128, D=128, m=4, page=16, n_shared=0, Wn=16),
    dict(ts=[[0]] * 3, H=128, D=512, m=4, page=16, n_shared=0, Wn=16, gain=True),
    dict(ts=[[0]] * 3, H=128, D=512, m=4, page=16, n_shared=0, Wn=16, fp8=True)])
def test_attend_paged_one_key_is_its_value(cuda, kw):
    """A row with one key: the weight's rounding cancels, so the output is the key's value to the bit."""
    c = Case(**kw)
    got = c.run(cuda)
    assert cuda.csa_sync_status() == 0
    want = torch.where((c.pos >= 0)[..., None, None], c.ring64[:, :1, None].to(torch.bfloat16), 0.0).expand_as(got)
    assert torch.equal(got.float(), want.float())


def test_attend_paged_very_many_row_tiles(cuda):
    """More row tiles than the kernel counts at once."""
    c = Case(ts=[[390 + 11 * b + i for i in range(64)] for b in range(130)], H=128, D=64, m=8, page=16, n_shared=48, Wn=9)
    assert c.by_row_tiles()
    got = c.run(cuda)
    assert cuda.csa_sync_status() == 0
    assert got.isfinite().all()
    at = torch.tensor([0, 1, 63, 127, 128, 129], device=DEV)  # row tiles from 8192 on among them
    c.check(got[at], c.ref(at))


@pytest.mark.parametrize("D,nq,gain", [(64, 64, False), (128, 32, True), (256, 16, False), (512, 16, True)])
def test_attend_paged_many_short_row_tiles(cuda, D, nq, gain):
    """Many row tiles a pair of SMs with few keys each, time and again: no hand-over from one to the next may be missed
    (one in some 70,000 was, when a wait could look for a phase that was over)."""
    c = Case(ts=[[390 + 11 * b + i for i in range(nq)] for b in range(130)], H=128, D=D, m=8, page=16, n_shared=48, Wn=9,
             gain=gain)
    assert c.by_row_tiles()
    first = c.run(cuda)
    for _ in range(40):
        got = c.run(cuda)
        assert cuda.csa_sync_status() == 0
        assert torch.equal(got.view(torch.int16), first.view(torch.int16))


def test_attend_paged_fp8_beyond_the_copy(cuda):
    """Tables so wide that the FP8 rows are not copied: query by query."""
    c = Case(**ROW_TILES["fp8_512"], gain=True, cols=2900)
    assert not c.by_row_tiles()
    got = c.run(cuda)
    assert cuda.csa_sync_status() == 0
    c.check(got)


@pytest.mark.parametrize("kw", [ROW_TILES["d512_h128"], ROW_TILES["fp8_512"], CASES["shared_512"], CASES["fp8_512"]])
def test_attend_paged_in_a_large_pool(cuda, kw):
    """Pages whose rows lie past 2^31 elements and 2^32 bytes of the pool; the others are not initialised."""
    c = Case(**kw)
    ref = c.ref()
    before = c.run(cuda)
    first = (2 ** 32 + 2 ** 22) // (c.page * 512 * (1 if c.fp8 else 2))
    def moved(x):
        big = torch.empty((first + x.shape[0],) + x.shape[1:], dtype=x.dtype, device=DEV)
        big[first:] = x
        return big
    c.pool = moved(c.pool)
    if c.fp8:
        c.pe = moved(c.pe)
    c.table = torch.where(c.table >= 0, c.table + first, c.table)
    for n_shared in (c.n_shared, 0):
        got = c.run(cuda, n_shared=n_shared)
        assert cuda.csa_sync_status() == 0
        c.check(got, ref, n_shared)
    assert torch.equal(c.run(cuda).view(torch.int16), before.view(torch.int16))


@pytest.mark.parametrize("fp8", [False, True])
def test_paged_write_into_a_large_pool(cuda, fp8):
    d, n = 512, 40
    n_slots = (2 ** 32 + 2 ** 22) // (d if fp8 else 2 * d)
    rows = W.normal_bf16((n, d), 5, DEV)
    slots = torch.cat([torch.arange(n // 2), torch.arange(n_slots - n // 2, n_slots)]).to(DEV)
    if fp8:
        codes = torch.empty((n_slots, d), dtype=torch.uint8, device=DEV)
        exps = torch.empty((n_slots, d // 128), dtype=torch.uint8, device=DEV)
        cuda.csa_paged_write_fp8kv(rows, slots, codes, exps)
        c, e = cuda.csa_quantize_fp8_kv(rows)
        assert torch.equal(codes[slots], c) and torch.equal(exps[slots], e)
    else:
        pool = torch.empty((n_slots, d), dtype=torch.bfloat16, device=DEV)
        cuda.csa_paged_write(rows, slots, pool)
        assert torch.equal(pool[slots], rows)


@pytest.mark.parametrize("name", ["d512_h128", "d128_h16", "fp8_512", "d512_h128_nq4"])
def test_attend_paged_graph_follows_its_inputs(cuda, name):
    """Captured on a side stream, replayed with other positions, queries and pages; beside another graph of its own."""
    c, other = Case(**ROW_TILES[name]), Case(**dict(ROW_TILES["d64_h8"], seed=9))
    B = c.pos.shape[0]
    ws = torch.empty(c.workspace_bytes(), dtype=torch.uint8, device=DEV)
    out, out2 = torch.empty_like(c.q), torch.empty_like(other.q)
    c.run(cuda, workspace=ws, out=out)
    other.run(cuda, out=out2)
    torch.cuda.synchronize()
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s1):
        c.run(cuda, workspace=ws, out=out)
    with torch.cuda.graph(g2, stream=s2):
        other.run(cuda, out=out2)
    # fewer entries seen, other queries, the batch's rows in another order
    order = torch.randperm(B, device=DEV)
    c.q.copy_(torch.randn_like(c.q, dtype=torch.float32))
    c.table.copy_(c.table[order])
    c.ring.copy_(c.ring[order])
    if c.fp8:
        c.re.copy_(c.re[order])
    c.ring64 = c.ring64[order]
    c.pos.copy_(c.pos[order])
    out.fill_(float("nan"))
    out2.fill_(float("nan"))
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        g.replay()
        g.replay()
    with torch.cuda.stream(s2):
        g2.replay()
    torch.cuda.synchronize()
    assert cuda.csa_sync_status() == 0
    c.check(out)
    other.check(out2)


@pytest.mark.parametrize("kw", [
    CASES["own_only"], CASES["fp8_512"], CASES["shared_rope_128"], CASES["shared_rope_512"], ROW_TILES["d512_h128_nq4"],
    ROW_TILES["fp8_512"], ROW_TILES["negative_scale"], dict(CASES["own_only"], scale=-1.0, sinks=True)])
def test_native_marshalling_makes_the_same_call(cuda, kw):
    from long_context_compressed_06_b200 import binding
    c = Case(**kw)
    got = c.run(cuda)
    keep = binding._native
    assert keep.__name__.endswith("_native")
    args = (c.q, c.pool, c.pe if c.fp8 else None, c.table, c.m, c.ring, c.re if c.fp8 else None, c.pos, c.Wn, c.scale, 1e-6,
            c.gain, c.n_shared, c.sinks, c.rope)
    native = keep.attend_paged(*args)
    assert native.dtype == torch.bfloat16 and native.shape == c.q.shape and native.is_contiguous()
    try:
        binding._native = binding._Unbound
        long_way = c.run(cuda)
    finally:
        binding._native = keep
    for x in (native, long_way):
        assert torch.equal(x.view(torch.int16), got.view(torch.int16))
    class Sub(torch.Tensor):
        pass

    # not regular: another order of the rows, another type, another rank, a subclass, an odd number
    for i, x in ((0, c.q.transpose(1, 2)), (0, c.q.float()), (3, c.table.long()), (7, c.pos[0]), (0, c.q.as_subclass(Sub)),
                 (4, True), (4, 2 ** 40), (7, c.pos.cpu()), (14, (1, 2)), (12, c.page + 1)):
        assert keep.attend_paged(*args[:i], x, *args[i + 1:]) is None, i


def test_native_plan_and_write_make_the_same_calls(cuda):
    from long_context_compressed_06_b200 import binding
    keep = binding._native
    results = []
    for native in (True, False):
        old = torch.tensor([0, 5, 100, 63, 0], dtype=torch.int32, device=DEV)
        new = torch.tensor([70, 1, 0, 2, 0], dtype=torch.int32, device=DEV)
        free = torch.arange(9, 0, -1, dtype=torch.int32, device=DEV)
        table = torch.full((5, 6), -1, dtype=torch.int32, device=DEV)
        table[1, 0], table[2, :2], table[3, 0] = 20, torch.tensor([21, 22]), 23
        pool = torch.zeros((30 * 16, 128), dtype=torch.bfloat16, device=DEV)
        rows = W.normal_bf16((25, 128), 3, DEV)
        codes, exps = torch.zeros((480, 128), dtype=torch.uint8, device=DEV), torch.zeros((480, 1), dtype=torch.uint8, device=DEV)
        try:
            if not native:
                binding._native = binding._Unbound
            plan = cuda.csa_plan_pages(old, new, free, table, 4, 16, 32, 81, 25)
            assert cuda.csa_paged_write(rows, plan[2], pool) is pool
            assert cuda.csa_paged_write_fp8kv(rows, plan[2], codes, exps) == (codes, exps)
        finally:
            binding._native = keep
        assert [x.dtype for x in plan] == [torch.int64] * 3 + [torch.int32] + [torch.int64] * 2
        results.append([x.clone() for x in plan] + [table, pool, codes, exps])
        plan[3].fill_(7)                        # outputs of one allocation, each its own
        assert all(torch.equal(a, b) for k, (a, b) in enumerate(zip(plan, results[-1])) if k != 3)
    assert all(torch.equal(a, b) for a, b in zip(*results))
    # the outputs are tensors like any other, in inference mode too
    for mode in (torch.inference_mode(), torch.no_grad()):
        with mode:
            plan = cuda.csa_plan_pages(old, new, free, table, 4, 16, 32, 81, 25)
            plan[2].add_(1)
            assert torch.equal(plan[2].view(5, 5).t().contiguous().t().reshape(-1) - 1, results[0][2])
            assert plan[3].cpu().tolist() == results[0][3].tolist() and plan[0].clone().is_contiguous()
    # nothing appended, no room
    z = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = cuda.csa_plan_pages(z, z, z[:0], torch.full((1, 1), -1, dtype=torch.int32, device=DEV), 4, 16, 16, 0, 0)
    assert [x.numel() for x in out] == [2, 2, 0, 0, 0, 4] and out[5].tolist() == [0, 0, 0, 0]


def test_attend_paged_refusals(cuda):
    c = Case(**CASES["shared_tile"])
    def bad(exc, **kw):
        with pytest.raises(exc):
            c.run(cuda, **kw)
    bad(csa_pkg.CsaError, n_shared=64)          # not whole pages
    bad(csa_pkg.CsaError, n_shared=128 * 100)   # past the table
    bad(csa_pkg.CsaError, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    bad(TypeError, workspace=torch.empty(1 << 24, dtype=torch.uint8))  # host memory
    bad(ValueError, out=torch.empty_like(c.q[:1]))
    big = Case(**CASES["shared_tile"])
    big.pos = big.pos.cpu()
    with pytest.raises(TypeError):
        big.run(cuda)
    big = Case(**CASES["shared_tile"])
    big.ring = big.ring[:, :8].contiguous()     # fewer rows than the window
    with pytest.raises(csa_pkg.CsaError):
        big.run(cuda)
    big = Case(**CASES["shared_tile"])
    big.table = big.table[:1].contiguous()
    with pytest.raises(ValueError):
        big.run(cuda)
    big = Case(**CASES["shared_tile"])
    big.gain = torch.ones(3, device=DEV)
    with pytest.raises(ValueError):
        big.run(cuda)
    with pytest.raises(ValueError):             # one slot per row
        cuda.csa_paged_write(c.q[0, 0].contiguous(), torch.zeros(3, dtype=torch.int64, device=DEV), c.pool)
    with pytest.raises(TypeError):
        cuda.csa_plan_pages(*(torch.zeros(3, dtype=torch.int64, device=DEV),) * 3, c.table, 4, 16, 16, 9, 9)
    with pytest.raises(ValueError):             # negative room
        z = torch.zeros(3, dtype=torch.int32, device=DEV)
        cuda.csa_plan_pages(z, z, z, torch.zeros(3, 4, dtype=torch.int32, device=DEV), 4, 16, 16, -1, 9)


# ----------------------------------------------------------------------------- the operators as a server runs them
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("batch", [5, 40])
def test_prefill_and_decode_over_pages(cuda, batch, fp8):
    """Requests with a common prompt: its pages are written once and noted in every row of the table, then a ragged
    prefill and decode steps: plan, writes of the entries and of the window rows through its slot maps, attention."""
    H, D, m, page, Wn, ring_rows = 8, 128, 4, 16, 24, 40
    rng = np.random.default_rng(batch)
    prompt = 64 * page * m                       # tokens of the shared prompt: 64 pages
    total = prompt + 400
    streams = W.normal_bf16((batch, total, D), 70, DEV)                 # window rows of every position
    entries = W.normal_bf16((batch, total // m, D), 71, DEV)
    streams[:, :prompt], entries[:, :prompt // m] = streams[:1, :prompt], entries[:1, :prompt // m]
    n_pages = 64 + batch * 8 + 5
    pool = torch.full((n_pages, page, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    ring = torch.full((batch, ring_rows, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    if fp8:
        pool8 = [torch.full((n_pages, page, D), 0x7F, dtype=torch.uint8, device=DEV),
                 torch.full((n_pages, page, D // 128), 255, dtype=torch.uint8, device=DEV)]
        ring8 = [torch.full((batch, ring_rows, D), 0x7F, dtype=torch.uint8, device=DEV),
                 torch.full((batch, ring_rows, D // 128), 255, dtype=torch.uint8, device=DEV)]
        round_trip = lambda x: dequant(*cuda.csa_quantize_fp8_kv(x.contiguous()))  # noqa: E731
        streams64, entries64 = round_trip(streams), round_trip(entries)
    else:
        streams64, entries64 = streams.double(), entries.double()
    ids = torch.tensor(rng.permutation(n_pages).astype(np.int32), device=DEV)
    table = torch.full((batch, 80), -1, dtype=torch.int32, device=DEV)

    def write(rows, slots, dst, dst8):
        if fp8:
            cuda.csa_paged_write_fp8kv(rows, slots, *dst8)
        else:
            cuda.csa_paged_write(rows, slots, dst)

    def step(old, new, free):
        """One step of every request; returns the pages taken."""
        tokens, n_entries = int(new.sum()), int(((old + new) // m - old // m).sum())
        t = lambda x: torch.tensor(x.astype(np.int32), device=DEV)  # noqa: E731
        cu_t, cu_e, slots, pos, win, counts = cuda.csa_plan_pages(t(old), t(new), free, table, m, page, ring_rows,
                                                                  tokens + 3, n_entries + 5)
        assert counts.tolist()[:2] == [tokens, n_entries] and counts.tolist()[3] == 0
        cu_t, cu_e = cu_t.tolist(), cu_e.tolist()
        er = torch.cat([entries[b, old[b] // m:(old[b] + new[b]) // m] for b in range(len(old))] + [entries[0, :5]])
        sr = torch.cat([streams[b, old[b]:old[b] + new[b]] for b in range(len(old))] + [streams[0, :3]])
        write(er, slots, pool, pool8 if fp8 else None)
        write(sr, win, ring, ring8 if fp8 else None)
        assert pos.tolist()[:tokens] == [int(u) for b in range(len(old)) for u in range(old[b], old[b] + new[b])]
        return int(counts[2])

    # the prompt, by the first request; the others note its pages
    zero = np.zeros(batch, np.int64)
    first = zero.copy()
    first[0] = prompt
    used = step(zero, first, ids)
    assert used == 64
    table[1:, :64] = table[:1, :64]
    # the window rows of the prompt's end, for every request
    tail = torch.arange(prompt - Wn, prompt, device=DEV)
    slots = (torch.arange(batch, device=DEV)[:, None] * ring_rows + tail % ring_rows).flatten()
    write(streams[0, tail].repeat(batch, 1), slots, ring, ring8 if fp8 else None)
    cached = zero + prompt
    news = [rng.integers(1, 61, batch), np.ones(batch, np.int64), np.ones(batch, np.int64), rng.integers(0, 3, batch)]
    for new in news:
        used += step(cached, new, ids[used:])
        cached = cached + new
        q = torch.randn(batch, 1, H, D, device=DEV).to(torch.bfloat16)
        pos = torch.tensor((cached - 1).astype(np.int32)[:, None], device=DEV)
        for n_shared in (0, 64 * page):
            if fp8:
                out = cuda.hca_attend_paged_fp8kv(q, *pool8, table, m, *ring8, pos, Wn, D ** -0.5, n_shared=n_shared)
            else:
                out = cuda.hca_attend_paged(q, pool, table, m, ring, pos, Wn, D ** -0.5, n_shared=n_shared)
            assert cuda.csa_sync_status() == 0
            for b in range(batch):
                t = int(cached[b]) - 1
                x = torch.cat([entries64[b, :(t + 1) // m], streams64[b, max(0, t - Wn + 1):t + 1]])
                y = q[b, 0].double()
                y = y / (y.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()
                p = torch.softmax(y @ x.T * D ** -0.5, -1)
                o, a = p @ x, p @ x.abs()
                tol = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -10) * a
                assert ((out[b, 0].double() - o).abs() <= tol).all(), (b, t, n_shared)


def test_attend_paged_on_another_stream_and_two_at_once(cuda):
    cs = [Case(**dict(ROW_TILES["d128_h16"], seed=s)) for s in (1, 2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for c, s in zip(cs, streams):
        with torch.cuda.stream(s):
            outs.append(c.run(cuda))
    torch.cuda.synchronize()
    for c, o in zip(cs, outs):
        c.check(o)

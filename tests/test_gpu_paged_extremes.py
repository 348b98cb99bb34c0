"""hca_attend_paged at the ends of its inputs' range, against the formula in 64 bits: scores of any size, keys that are
not finite."""
import math

import pytest
import torch

import long_context_compressed_06_b200 as csa_pkg  # noqa: F401
from test_gpu_paged import CASES, DEV, ROW_TILES, Case, dequant

pytestmark = pytest.mark.gpu


def exact_scores(c, size, unit, seed=5):
    """Queries +-s by head parity, s a vector of signs; keys s * size but for 8 channels that hold s * unit * (0 or 1):
    every score is +-(size (D - 8) + unit n), n in 0..8, and exact in 32 bits, so that only the weights' and the
    output's roundings are left of the tolerance in test_gpu_paged.py."""
    g = torch.Generator().manual_seed(seed)
    D, H = c.q.shape[-1], c.q.shape[2]
    s = (torch.randint(0, 2, (D,), generator=g) * 2 - 1).to(torch.bfloat16).to(DEV)
    c.q = (s * (1 - 2 * (torch.arange(H, device=DEV) % 2)).to(torch.bfloat16)[:, None]).expand(c.q.shape).contiguous()

    def rows(old):  # unused rows stay what they are (NaN)
        x = torch.full(old.shape, float(size), dtype=torch.bfloat16, device=DEV)
        x[..., -8:] = unit * torch.randint(0, 2, (*old.shape[:-1], 8), generator=g).to(torch.bfloat16).to(DEV)
        return torch.where(old.isnan(), old, x * s)

    c.pool, c.ring = rows(c.pool), rows(c.ring)
    c.pool64, c.ring64 = c.pool.double(), c.ring.double()
    if c.gain is not None:  # (rows under a gain of 1 are the sum of two bf16 numbers exactly, too)
        c.gain = torch.ones_like(c.gain)


def exact_ref(c):
    out, mag, e = c.ref()
    return out, mag, torch.zeros_like(e)


# log2 of the largest score at D = 128: 14.0, 14.5, 15.6, 19.4
@pytest.mark.parametrize("size", [96, 136, 288, 4096])
@pytest.mark.parametrize("scale", [1.0, -1.0])
@pytest.mark.parametrize("name", ["d64_h8", "d128_h16", "d256_h64", "d512_h128", "d128_h64_nq4", "part_seen_128"])
def test_large_scores_over_row_tiles(cuda, name, size, scale):
    c = Case(**dict(ROW_TILES[name], scale=scale))
    exact_scores(c, size, 1.0)
    assert c.by_row_tiles()
    got = c.run(cuda)
    assert cuda.csa_sync_status() == 0
    c.check(got, exact_ref(c))


@pytest.mark.parametrize("size", [96, 136, 288])
@pytest.mark.parametrize("name", ["own_only", "shared_odd", "shared_512"])
def test_large_scores_query_by_query(cuda, name, size):
    c = Case(**dict(CASES[name], scale=1.0))
    exact_scores(c, size, 1.0)
    assert not c.by_row_tiles()
    out, mag, e = c.ref()
    # scores rounded to 32 bits here: off by 2^-24 of their size, with the factor's own rounding
    c.check(c.run(cuda), (out, mag, e + 2.0 ** -23 * size * c.q.shape[-1]))


# scores of 2^25 to 2^67, whose rounding to 32 bits alone moves them by more than 1.  Those below the largest are
# `unit` = size / 4096 away or more: their weights are next to nothing, whatever their rounding makes of them.
@pytest.mark.parametrize("size", [2.0 ** 18, 2.0 ** 22, 2.0 ** 26, 2.0 ** 60])
@pytest.mark.parametrize("name", ["d64_h8", "d128_h16", "d256_h64", "d512_h128", "d128_h64_nq4"])
def test_huge_scores_over_row_tiles(cuda, name, size):
    c = Case(**dict(ROW_TILES[name], scale=1.0))
    unit = size / 4096
    exact_scores(c, size, unit)
    assert c.by_row_tiles()
    got = c.run(cuda)
    assert cuda.csa_sync_status() == 0
    # Scores of up to z log2 units come in 32-bit steps of `step`.  A score is rounded by half a step and the reference
    # that all are taken from cut by up to 3, the same for every key: a key `unit` below the top stays unit / step - 1
    # steps below it at least (half a step for each of the two), each of them worth `step` units, or 16 where the kernel
    # takes a step for 16 (from 2^28 on).  All n of them weigh at most n times that, in a channel at most its largest
    # value.  (D = 512, the closest: unit is 2.9 steps at least.)
    z = size * c.q.shape[-1] / math.log(2)
    step = 2.0 ** (math.floor(math.log2(z)) - 23)
    away = (unit / math.log(2) / step - 1) * (step if z < 2.0 ** 28 else min(step, 16.0)) * math.log(2)
    n = c.max_pages * c.page + c.Wn
    extra = n * math.exp(-min(away, 700.0)) * torch.full((c.q.shape[-1],), size, dtype=torch.float64, device=DEV)
    extra[-8:] *= unit / size
    out, mag, e = exact_ref(c)
    assert away > 10
    c.check(got, (out, mag + 2.0 ** 8 * extra, e))


# ----------------------------------------------------------------------------- keys and queries that are not finite
NAN, INF = float("nan"), float("inf")


def shows_what_the_formula_does(c, got):
    """-> where the formula's result is not finite, there the kernel's is not either."""
    out = c.ref()[0]
    assert not (got.isfinite() & ~out.isfinite()).any()
    return ~out.isfinite()


# rows of one key, and of few: a NaN score is no maximum, and must not make the row one without keys
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("kw,by_row_tiles", [
    (CASES["one_token"], False), (CASES["no_entries"], False), (CASES["shared_odd"], False), (ROW_TILES["d128_own_only"], True),
    (dict(ROW_TILES["part_seen_512"], Wn=1), True), (dict(ROW_TILES["part_seen_64"], Wn=1), True)])
def test_a_key_that_is_not_finite_shows(cuda, kw, by_row_tiles, value):
    c = Case(**kw)
    assert c.by_row_tiles() == by_row_tiles
    b = int(torch.where(c.pos.amax(1) >= 0, c.pos.amax(1), 2 ** 30).argmin())
    c.ring[b, int(c.pos[b].max()) % c.ring.shape[1]] = value  # the newest token's row of the shortest request
    c.ring64 = c.ring.double()
    got = c.run(cuda)
    assert cuda.csa_sync_status() == 0
    hit = shows_what_the_formula_does(c, got)
    assert hit[b].any() and not hit[torch.arange(len(hit), device=DEV) != b].any()


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("name", ["one_token", "shared_odd", "own_rope", "shared_512", "d64_h8", "d128_h16", "d128_h64_nq4",
                                  "d256_h64", "d512_h128", "d128_own_only", "part_seen_512", "fp8_128"])
def test_a_query_that_is_not_finite_is_its_own_rows(cuda, name, value):
    c = Case(**(ROW_TILES.get(name) or CASES[name]))
    assert c.by_row_tiles() == (name in ROW_TILES)
    clean = c.run(cuda)
    live = (c.pos >= 0).nonzero().tolist()
    (b0, i0), (b1, i1) = live[0], live[-1]
    H, D = c.q.shape[2:]
    rows = torch.zeros(c.q.shape[:3], dtype=torch.bool, device=DEV)
    for b, i, h in ((b0, i0, 0), (b1, i1, H - 1)):
        c.q[b, i, h, D - 3] = value
        rows[b, i, h] = True
    got = c.run(cuda)
    assert cuda.csa_sync_status() == 0
    assert got[rows].isnan().all() and shows_what_the_formula_does(c, got)[rows].all()
    assert torch.equal(got[~rows].view(torch.int16), clean[~rows].view(torch.int16))


def key_places(c, where):
    """A key that some queries take and others do not: ("pool", page, row) or ("ring", request, row), and which
    queries' key sets it is in, [batch][nq]."""
    pos = c.pos.cpu().long()
    vis = torch.where(pos >= 0, (pos + 1) // c.m, 0)
    B = pos.shape[0]
    if where == "shared":  # an entry of the shared pages that only some of the queries see
        j = int(vis[(vis > 0) & (vis < c.n_shared)].min())
        return ("pool", int(c.table[0, j // c.page]), j % c.page), vis > j
    b = max(range(B // 3, B), key=lambda i: (int(vis[i].max()) > c.n_shared, -abs(i - B // 2)))
    of_b = (torch.arange(B) == b)[:, None]
    if where.endswith("entry"):
        j = c.n_shared if where == "first_entry" else int(vis[b].max()) - 1
        assert j >= c.n_shared and vis[b].max() > j
        return ("pool", int(c.table[b, j // c.page]), j % c.page), of_b & (vis > j)
    u = int(pos[b].max()) - (0 if where == "newest_token" else c.Wn // 2)
    return ("ring", b, u % c.ring.shape[1]), of_b & (pos >= u) & (u > pos - c.Wn)


def check_apart(cuda, c, where, value, whole):
    clean = c.run(cuda)
    (kind, i, r), takes = key_places(c, where)
    assert takes.any() and not takes.all()
    rows = getattr(c, kind)
    assert c.fp8 or rows[i, r].isfinite().all()
    D, H = c.q.shape[-1], c.q.shape[2]
    rows[i, r, slice(None) if whole else slice(D // 2 + 5, D // 2 + 6)] = value
    if c.fp8:
        c.pool64, c.ring64 = dequant(c.pool, c.pe), dequant(c.ring, c.re)
    else:
        c.pool64, c.ring64 = c.pool.double(), c.ring.double()
    got = c.run(cuda)
    assert cuda.csa_sync_status() == 0
    takes = takes.to(DEV)
    out, mag, e = c.ref()
    # who takes it shows it, wherever the formula does
    assert not out[takes].isfinite().all()
    assert not (got[takes].isfinite() & ~out[takes].isfinite()).any()
    # who does not take it is as right as ever, and as it was to the bit if no row beside its own in a tile of 128 does
    x = ~takes
    assert got[x].isfinite().all()
    tol = 2.0 ** -8 * out[x].abs() + (2.0 ** -8 + torch.expm1(2 * e[x] * (256 if D == 512 and not c.by_row_tiles() else 1))
                                      + 2.0 ** -10) * mag[x]
    assert ((got[x].double() - out[x]).abs() <= tol).all()
    row_takes = takes[:, :, None].expand(-1, -1, H).flatten()
    if c.by_row_tiles():
        tile_takes = torch.nn.functional.pad(row_takes, (0, -len(row_takes) % 128)).view(-1, 128).any(1)
        row_takes = tile_takes.repeat_interleave(128)[:len(row_takes)]
    same = (got.view(torch.int16) == clean.view(torch.int16)).flatten(0, 2).all(-1)
    assert same[~row_takes].all()


VALUES = [(NAN, False), (NAN, True), (INF, False), (-INF, True)]


@pytest.mark.parametrize("value,whole", VALUES)
@pytest.mark.parametrize("where", ["first_entry", "last_entry", "newest_token", "mid_window"])
@pytest.mark.parametrize("name", ["d64_h8", "d64_h1", "d128_h16", "d128_h40_rope", "d128_h64_nq4", "d256_h100", "d256_h64",
                                  "d512_h72", "d512_h128_nq4", "d128_own_only"])
def test_a_key_reaches_only_who_takes_it_over_row_tiles(cuda, name, where, value, whole):
    c = Case(**ROW_TILES[name])
    assert c.by_row_tiles()
    check_apart(cuda, c, where, value, whole)


@pytest.mark.parametrize("value,whole", VALUES)
@pytest.mark.parametrize("name", ["part_seen_64", "part_seen_128", "part_seen_256", "part_seen_512"])
def test_a_shared_key_reaches_only_who_sees_it_over_row_tiles(cuda, name, value, whole):
    c = Case(**ROW_TILES[name])
    assert c.by_row_tiles()
    check_apart(cuda, c, "shared", value, whole)


@pytest.mark.parametrize("where", ["first_entry", "newest_token"])
@pytest.mark.parametrize("name", ["fp8_128", "fp8_256_own", "fp8_512"])
def test_an_fp8_key_reaches_only_who_takes_it_over_row_tiles(cuda, name, where):
    c = Case(**ROW_TILES[name])
    assert c.by_row_tiles()
    check_apart(cuda, c, where, 0x7F, False)  # NaN


@pytest.mark.parametrize("value,whole", VALUES)
@pytest.mark.parametrize("name,where", [("own_only", "first_entry"), ("own_only", "newest_token"), ("shared_odd", "last_entry"),
                                        ("shared_rope_128", "newest_token"), ("part_seen", "shared"), ("shared_256", "mid_window")])
def test_a_key_reaches_only_who_takes_it_query_by_query(cuda, name, where, value, whole):
    c = Case(**CASES[name])
    assert not c.by_row_tiles()
    check_apart(cuda, c, where, value, whole)


# an infinite channel: heads whose query has its sign have a score of +inf, the others one of -inf, a weight of 0, and
# 0 x inf; with no other key, or no other in the partial row, 0 / 0
@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("value", [INF, -INF])
@pytest.mark.parametrize("kw,by_row_tiles", [
    (CASES["one_token"], False), (CASES["no_entries"], False), (dict(CASES["shared_512"], ts=[[1700], [1690], [0]], Wn=1), False),
    (dict(CASES["own_only"], Wn=1), False), (ROW_TILES["d128_own_only"], True), (dict(ROW_TILES["part_seen_512"], Wn=1), True),
    (dict(ROW_TILES["part_seen_64"], Wn=1), True), (dict(ROW_TILES["d512_h72"], Wn=1), True)])
def test_scores_of_minus_infinity_are_not_rows_without_keys(cuda, kw, by_row_tiles, value, sinks):
    c = Case(**dict(kw, sinks=sinks))
    assert c.by_row_tiles() == by_row_tiles
    b = int(torch.where(c.pos.amax(1) >= 0, c.pos.amax(1), 2 ** 30).argmin())
    r = int(c.pos[b].max()) % c.ring.shape[1]
    # every key of the query, where there are few; else its window
    for u in range(max(0, int(c.pos[b].max()) - c.Wn + 1), int(c.pos[b].max()) + 1):
        c.ring[b, u % c.ring.shape[1], 7] = value
    assert c.ring[b, r, 7] == value
    c.ring64 = c.ring.double()
    got = c.run(cuda)
    assert cuda.csa_sync_status() == 0
    hit = shows_what_the_formula_does(c, got)
    assert hit[b].any()
    rest = (torch.arange(len(hit), device=DEV) != b)
    assert not hit[rest].any() and got[rest].isfinite().all()


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_beside_a_key_that_is_not_finite_leave_out_missing_pages(cuda, fp8):
    """Keys that are all alike (values 1 to 1.4, so that an output is as large as its terms): an entry without a page
    that counted as a row of zeros would show, 160 of some 1100."""
    name = "fp8_128" if fp8 else "part_seen_128"
    c = Case(**dict(ROW_TILES[name], drop=[(None, 4 * i + 1, -1) for i in range(10)], seed=9))
    assert c.by_row_tiles()
    g = torch.Generator().manual_seed(3)

    def rows(old):
        codes = torch.randint(0x38, 0x3C, old.shape, generator=g).to(torch.uint8).to(DEV)
        if fp8:
            return torch.where(old == 0x7F, old, codes)
        return torch.where(old.isnan(), old, codes.view(torch.float8_e4m3fn).to(torch.bfloat16))

    c.pool, c.ring = rows(c.pool), rows(c.ring)
    if fp8:
        c.pe, c.re = torch.where(c.pe == 255, c.pe, 127), torch.where(c.re == 255, c.re, 127)
    (kind, i, r), takes = key_places(c, "newest_token")
    getattr(c, kind)[i, r, 9] = 0x7F if fp8 else NAN
    if fp8:
        c.pool64, c.ring64 = dequant(c.pool, c.pe), dequant(c.ring, c.re)
    else:
        c.pool64, c.ring64 = c.pool.double(), c.ring.double()
    got = c.run(cuda)
    assert cuda.csa_sync_status() == 0
    x = ~takes.to(DEV)
    out, mag, e = c.ref()
    assert got[x].isfinite().all() and (e == 0).all()
    assert ((got[x].double() - out[x]).abs() <= 2.0 ** -8 * out[x].abs() + (2.0 ** -8 + 2.0 ** -10) * mag[x]).all()

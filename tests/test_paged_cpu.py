"""Argument checks of the paged-cache calls that need no GPU: every refusal comes from the host, before any launch, and
the sizes of the workspaces are plain functions of the shapes."""
import ctypes

import pytest
import torch

import long_context_compressed_06_b200 as csa
from long_context_compressed_06_b200 import build as csa_build

A = ctypes.c_void_p(0x10000)    # an aligned fake device address (never dereferenced)
M8 = ctypes.c_void_p(0x10008)   # 8-byte aligned
M4 = ctypes.c_void_p(0x10004)   # 4-byte aligned
ODD = ctypes.c_void_p(0x10001)
INV, UNS, WS = csa.CSA_ERR_INVALID, csa.CSA_ERR_UNSUPPORTED, csa.CSA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    csa_build.build()
    return csa.load()


def call(fn, names, values, **changed):
    v = dict(zip(names, values))
    assert set(changed) <= set(names)
    v.update(changed)
    return fn(*[v[n] for n in names])


PLAN = ("old new batch m page ring free n_free table max_pages cu_t cu_e slots max_e pos win max_t counts ws wsb "
        "stream").split()
PLAN_OK = (A, A, 20000, 4, 16, 128, A, 10, A, 8, A, A, A, 5, A, A, 5, A, None, 0, None)


@pytest.mark.parametrize("changed", [
    dict(batch=0), dict(m=0), dict(page=0), dict(ring=0), dict(n_free=-1), dict(max_pages=0), dict(max_e=-1), dict(max_t=-1),
    dict(old=None), dict(new=ODD), dict(table=None), dict(cu_t=M4), dict(cu_e=None), dict(counts=M4), dict(free=None),
    dict(slots=M4), dict(slots=None), dict(pos=None), dict(win=M4)])
def test_plan_pages_refuses(lib, changed):
    assert call(lib.csa_plan_pages, PLAN, PLAN_OK, **changed) == INV


def test_plan_pages_limits_and_workspace(lib):
    assert call(lib.csa_plan_pages, PLAN, PLAN_OK, batch=2 ** 20 + 1) == UNS
    assert call(lib.csa_plan_pages, PLAN, PLAN_OK, max_e=2 ** 31) == UNS
    assert call(lib.csa_plan_pages, PLAN, PLAN_OK, max_t=2 ** 31) == UNS
    need = lib.csa_plan_workspace_bytes(20000)
    assert need > 0 and lib.csa_plan_workspace_bytes(16384) == 0 and lib.csa_plan_workspace_bytes(0) == 0
    assert call(lib.csa_plan_pages, PLAN, PLAN_OK) == WS
    assert call(lib.csa_plan_pages, PLAN, PLAN_OK, ws=A, wsb=need - 1) == WS
    assert call(lib.csa_plan_pages, PLAN, PLAN_OK, ws=M4, wsb=need) == WS


def test_paged_write_refuses(lib):
    f, names = lib.csa_paged_write, "rows slots n d pool n_slots stream".split()
    ok = (A, A, 4, 64, A, 10, None)
    for changed in (dict(n=-1), dict(d=0), dict(d=12), dict(n_slots=0), dict(rows=M8), dict(rows=None), dict(slots=M4),
                    dict(pool=M8), dict(pool=None)):
        assert call(f, names, ok, **changed) == INV, changed
    f, names = lib.csa_paged_write_fp8kv, "rows slots n d codes exps n_slots stream".split()
    ok = (A, A, 4, 128, A, A, 10, None)
    for changed in (dict(n=-1), dict(d=64), dict(d=200), dict(n_slots=0), dict(rows=M8), dict(slots=None), dict(codes=M8),
                    dict(exps=None)):
        assert call(f, names, ok, **changed) == INV, changed


BF = ("q gain sinks cos sin npos pool n_pages page table max_pages n_shared m ring ring_rows W pos batch nq H D scale eps "
      "out ws wsb stream").split()
BF_OK = (A, None, None, None, None, 0, A, 64, 16, A, 8, 32, 4, A, 130, 128, A, 2, 3, 16, 128, 0.1, 1e-6, A, A, 2 ** 40, None)
F8 = ("q gain sinks cos sin npos pool pool_e n_pages page table max_pages n_shared m ring ring_e ring_rows W pos batch nq H "
      "D scale eps out ws wsb stream").split()
F8_OK = (A, None, None, None, None, 0, A, A, 64, 16, A, 8, 32, 4, A, A, 130, 128, A, 2, 3, 16, 128, 0.1, 1e-6, A, A, 2 ** 40,
         None)
COMMON = [
    dict(q=M8), dict(q=None), dict(gain=ODD), dict(sinks=ODD), dict(cos=A), dict(sin=A), dict(cos=A, sin=A, npos=0),
    dict(cos=A, sin=ODD, npos=4), dict(pool=M8), dict(pool=None), dict(n_pages=0), dict(page=0), dict(page=8), dict(page=24),
    dict(table=None), dict(table=ODD), dict(max_pages=0), dict(n_shared=-16), dict(n_shared=40), dict(n_shared=144),
    dict(m=0), dict(ring=None), dict(ring_rows=129), dict(W=0), dict(pos=None), dict(batch=0), dict(nq=0), dict(H=0),
    dict(eps=-1.0), dict(eps=float("nan")), dict(out=M8)]


@pytest.mark.parametrize("changed", COMMON)
def test_attend_paged_refuses(lib, changed):
    assert call(lib.hca_attend_paged, BF, BF_OK, **changed) == INV
    assert call(lib.hca_attend_paged_fp8kv, F8, F8_OK, **changed) == INV


@pytest.mark.parametrize("changed", [
    dict(H=129), dict(D=96), dict(D=1024), dict(n_pages=2 ** 31 // 16 + 1), dict(max_pages=2 ** 31 // 16),
    dict(batch=2 ** 24, ring_rows=130), dict(batch=2 ** 23, nq=2, H=128, ring_rows=129),
    dict(batch=2 ** 30, nq=2 ** 30, ring_rows=2 ** 30 + 127)])
def test_attend_paged_unsupported(lib, changed):
    assert call(lib.hca_attend_paged, BF, BF_OK, **changed) == UNS
    assert call(lib.hca_attend_paged_fp8kv, F8, F8_OK, **changed) == UNS


def test_attend_paged_fp8_unsupported(lib):
    assert call(lib.hca_attend_paged_fp8kv, F8, F8_OK, D=64) == UNS
    assert call(lib.hca_attend_paged_fp8kv, F8, F8_OK, pool_e=None) == INV
    assert call(lib.hca_attend_paged_fp8kv, F8, F8_OK, ring_e=None) == INV


def test_attend_paged_workspace(lib):
    # (batch, nq, H, D, page, max_pages, n_shared, ring_rows, W, fp8)
    for shape in ((64, 1, 16, 128, 64, 300, 8192, 128, 128, False), (32, 1, 128, 512, 64, 129, 8064, 128, 128, True)):
        need = csa.attend_paged_workspace_bytes(*shape)
        assert need > 0
        batch, nq, H, D, page, max_pages, n_shared, ring_rows, Wn, fp8 = shape
        change = dict(batch=batch, nq=nq, H=H, D=D, page=page, max_pages=max_pages, n_shared=n_shared, ring_rows=ring_rows,
                      W=Wn, wsb=need - 1)
        fn, names, ok = (lib.hca_attend_paged_fp8kv, F8, F8_OK) if fp8 else (lib.hca_attend_paged, BF, BF_OK)
        assert call(fn, names, ok, **change) == WS
        assert call(fn, names, ok, **dict(change, wsb=need, ws=M8)) == WS
    # a gain, RoPE or a negative scale needs its own
    assert csa.attend_paged_workspace_bytes(64, 1, 16, 128, 64, 300, 8192, 128, 128, False, True) >= \
        csa.attend_paged_workspace_bytes(64, 1, 16, 128, 64, 300, 8192, 128, 128) + 2 * 64 * 16 * 128 * 2
    assert csa.attend_paged_workspace_bytes(0, 1, 16, 128, 64, 300, 8192, 128, 128) == 0
    assert csa.attend_paged_workspace_bytes(2, 1, 16, 100, 64, 300, 8192, 128, 128) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        csa.csa_paged_write(x[0], torch.zeros(16, dtype=torch.int64), x)
    with pytest.raises(TypeError):
        csa.csa_paged_write("rows", torch.zeros(16, dtype=torch.int64), None)
    with pytest.raises(TypeError):
        csa.hca_attend_paged(x, x, x, 4, x, x, 16, 0.1)


def test_native_marshalling_takes_regular_calls_only(lib):
    """What it does not take it leaves to the long way, which raises."""
    from long_context_compressed_06_b200 import binding
    n = binding._native
    x = torch.zeros(4, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    assert n.paged_write(x[0], torch.zeros(16, dtype=torch.int64), x) is None          # host memory
    assert n.paged_write() is None and n.paged_write(1, 2, 3) is None and n.paged_write(None, None, None, None) is None
    assert n.plan_pages(i, i, i, torch.zeros(4, 8, dtype=torch.int32), 4, 16, 16, 9, 9) is None
    assert n.plan_pages(i, i, i) is None and n.plan_pages(*[None] * 9) is None
    assert n.attend_paged(*[None] * 15) is None and n.attend_paged() is None
    assert n.attend_paged(x[None], x, None, i[:, None], 4, x, None, i[:, None], 16, 1.0, 1e-6, None, 0, None, None) is None
    with pytest.raises(RuntimeError):
        n.bind("/nowhere/libcsa.so")
    assert n.paged_write(x[0], torch.zeros(16, dtype=torch.int64), x) is None
    with pytest.raises(TypeError):
        csa.csa_plan_pages(i, i, i, torch.zeros(4, 8, dtype=torch.int32), 4, 16, 16, 9, 9)
    with pytest.raises(TypeError):
        csa.hca_attend_paged(x[None], x, i[:, None], 4, x, i[:, None], 16, 1.0)

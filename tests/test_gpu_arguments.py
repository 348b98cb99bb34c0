"""Arguments that the calls take in more than one form."""
import subprocess
import sys

import pytest
import torch

from long_context_compressed_06_b200 import build as csa_build
from long_context_compressed_06_b200 import workloads as W
from test_gpu_paged import Case, spread

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_workspace_may_be_a_view_with_gaps(cuda):
    """A workspace is memory: a view whose elements lie apart holds as many bytes from its first on."""
    q = W.normal_bf16((1, 1, 128, 512), 1, DEV)
    kv, win = W.normal_bf16((1, 4096, 512), 2, DEV), W.normal_bf16((1, 128, 512), 3, DEV)
    pos = torch.tensor([[16383]], dtype=torch.int32, device=DEV)
    need = cuda.attend_workspace_bytes(1, 1, 128, 512, 4096 + 128)
    assert need > 0

    def run(ws):
        return cuda.hca_attend(q, kv, 4, win, pos, 128, 512 ** -0.5, workspace=ws, win_pos0=16384 - 128)

    want = run(None)
    for ws in (torch.empty(2 * need, dtype=torch.uint8, device=DEV)[::2], torch.empty((need // 4 + 1, 2), device=DEV)[:, 0],
               torch.empty((need // 64 + 1, 64), dtype=torch.uint8, device=DEV).t()):
        assert not ws.is_contiguous()
        assert torch.equal(run(ws).view(torch.int16), want.view(torch.int16))
    # more elements than memory under them, memory of the host, no tensor
    for ws in (torch.empty(1, dtype=torch.uint8, device=DEV).expand(need), torch.empty(need, dtype=torch.uint8), need):
        with pytest.raises((TypeError, ValueError)):
            run(ws)


def test_status_is_the_first_call_of_a_process(cuda):
    r = subprocess.run([sys.executable, "-c", "import long_context_compressed_06_b200 as csa; assert csa.csa_sync_status() == 0\n"
                        "import torch; assert torch.zeros(3, device='cuda').sum().item() == 0"],
                       cwd=csa_build.ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("kw,extra", [
    (dict(ts=spread(2103, 2168, 32), H=128, D=512, m=1, page=64, n_shared=2048, Wn=128), 1920),
    (dict(ts=spread(4103, 4160, 64), H=16, D=128, m=1, page=64, n_shared=4096, Wn=128), 8064)])
def test_rings_much_longer_than_the_window_are_not_taken_whole(cuda, kw, extra):
    """The kernel over row tiles goes through every row of the rings: it is not the choice where that is most of it."""
    assert Case(**kw).by_row_tiles()
    c = Case(**kw, ring_extra=extra)
    assert not c.by_row_tiles()
    c.check(c.run(cuda))

"""GPU checks of the workspace that a caller of the adapters' binding gives: anything whose
bytes the kernels could not write is refused before a launch, any other is used."""

import pytest
import torch

from tests.test_gpu_lora import rows

import weight_only_int2_gb300 as wq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [3, 600])
def test_workspaces(M):
    x, A, B, base = rows((M, 64), 1), rows((2, 16, 64), 2), rows((2, 40, 16), 3), rows((M, 40), 4)
    ids = (torch.arange(M, device="cuda") % 3 - 1).int()
    need = wq.lora_workspace_bytes(M, 2, 16)
    call = lambda ws: wq.lora_gemm(x, A, B, ids, base, ws=ws)  # noqa: E731
    want = wq.lora_gemm(x, A, B, ids, base)
    for ws in (torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty((2, need // 4), device="cuda")):
        ws.view(-1).view(torch.uint8).fill_(255)  # NaN, were it read
        assert torch.equal(call(ws), want)
    one = torch.empty(1, dtype=torch.uint8, device="cuda")
    for ws, err, word in [
            (torch.empty(need, dtype=torch.uint8), ValueError, "must be a CUDA tensor"),
            (torch.empty(need, dtype=torch.uint8, pin_memory=True), ValueError, "must be a CUDA tensor"),
            (one.expand(need), ValueError, "contiguous"),  # `need` values, one byte
            (torch.empty((2 * need, 2), dtype=torch.uint8, device="cuda")[:, 0], ValueError, "contiguous"),
            (need, TypeError, "must be a torch.Tensor"), (one, wq.WQError, "too small")]:
        with pytest.raises(err, match=word):
            call(ws)

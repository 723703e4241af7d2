"""grouped_linear_bwd refuses outputs that share memory with anything that the call reads."""
import pytest
import torch

from quantized_lora_fine_b200 import api
from tests.block_helpers import normal

pytestmark = pytest.mark.gpu


def _case(dev):
    E, n, M = 2, 64, 6
    buf = torch.empty(E * n * n * 4, dtype=torch.uint8, device=dev)          # dW's bytes, the weight's in their first half
    W = buf[: E * n * n * 2].view(torch.bfloat16).view(E, n, n)
    W.copy_(normal((E, n, n), 1).to(dev))
    X, dY = normal((M, n), 2).to(dev), normal((M, n), 3).to(dev)
    offs = torch.tensor([0, 2, M], dtype=torch.int32, device=dev)
    return W, X, dY, offs, buf.view(torch.float32).view(E, n, n)


@pytest.mark.parametrize("need_dX", [True, False])
def test_dw_over_the_weight(cuda_device, need_dX):
    W, X, dY, offs, dW = _case(cuda_device)
    before = W.clone()
    with pytest.raises(ValueError, match="dW may not overlap"):
        api.grouped_linear_bwd(W, X, dY, offs, need_dX=need_dX, dW=dW)
    torch.cuda.synchronize()
    assert torch.equal(W, before)

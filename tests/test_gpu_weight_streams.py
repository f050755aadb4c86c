"""mx_weights on another stream than the current one: the matrices are not
laid into memory that the current stream may still use."""
import pytest
import torch

import shared_matrix_expert_amd as em
from oracle import operators as ops
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_weights_made_on_a_side_stream(handle):
    N, K = 2048, 2048                                     # codes of 2 MB: a block of their own in torch's pool
    dense = {k: torch.randn(1, N, K, device=DEV) for k in em._WEIGHT_KEYS[:12:2]}
    dense.update({k: None for k in em._WEIGHT_KEYS[12:16]})
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = [torch.empty(1, N, K // 2, dtype=torch.uint8, device=DEV) for _ in range(8)]
    at = {t.data_ptr() for t in freed}
    del freed                                             # the current stream's to give again
    W = em.mx_weights(dense, side.cuda_stream if handle else side)
    side.synchronize()
    assert not any(W[k].data_ptr() in at for k in em._WEIGHT_KEYS[:12:2])
    src = dense["b_dn"]
    codes, x = ops.quantize(src.cpu().double().numpy(), ops.FP4)
    assert torch.equal(W["b_dn"].cpu(), torch.from_numpy(ops.pack(codes, ops.FP4)))
    assert torch.equal(W["b_dn_scale"].cpu(), torch.from_numpy(ops.by_step(x)))

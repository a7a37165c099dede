"""Linear attention and the query / key norms (include/gdn_lin.h, gdn_layer.h) in calls that
lie at the edge of what their headers allow. Inputs and tolerances as in test_gpu_lin_ops."""
import pytest
import torch

from chunked_linear_recurrence_gated_gb300 import gdn
from test_gpu_lin_ops import DT, lin_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("decay", ["mid", "head"])
def test_no_tokens(dtype, packed, decay):
    """States pass through; a log-decay for each token has no elements, nor has its gradient
    (which torch gives as a null pointer)."""
    x = lin_inputs(1 if packed else 2, 0, 2, 64, 128, DT[dtype], decay, nseq=2)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda") if packed else None
    a = [x[i] for i in "qkvg"]
    o, S = gdn.gdn_lin_fwd(*a, x["S"], cu_seqlens=cu)
    assert o.numel() == 0 and torch.equal(S, x["S"])
    for dS, want in ((x["dS"], x["dS"]), (None, torch.zeros_like(x["dS"]))):
        r = gdn.gdn_lin_bwd(*a, x["S"], x["do"], dS, cu_seqlens=cu)
        torch.cuda.synchronize()
        assert torch.equal(r[4], want)
        assert r[3].shape == (x["g"].shape if decay == "mid" else (2,)) and (r[3] == 0).all()

"""Edges of the layer operators (include/gdn_layer.h) on the GPU: waits that run
out, open gates, small eps, empty batches, and the precision of fp32 calls."""
import pytest
import torch

from chunked_linear_recurrence_gated_gb300 import gdn
from test_gpu_layer_ops import gen, test_res_norm as check_res_norm

pytestmark = pytest.mark.gpu


# ------------------------------------------------- the exchange within a cluster
def test_exchange_sums_arrive():
    gdn.gdn_layer_status()
    sums = torch.zeros(4, device="cuda")
    assert gdn.diag_exchange(sums) == 0
    assert gdn.gdn_layer_status() == 0
    assert sums.tolist() == [256.0] * 4


@pytest.mark.parametrize("silent", range(4))
def test_exchange_wait_that_runs_out_is_reported(silent):
    """A CTA that sends nothing: every wait of its cluster runs out, the sums are
    NaN, the status says so once, and the context keeps computing."""
    gdn.gdn_layer_status()
    sums = torch.zeros(4, device="cuda")
    assert gdn.diag_exchange(sums, silent=silent, limit_log2=20) == 0
    assert gdn.gdn_layer_status() == 5  # GDN_ERR_TIMEOUT; reading resets it
    assert gdn.gdn_layer_status() == 0
    assert torch.isnan(sums).all()
    check_res_norm(("bf16", "f32"), True, True, 37, 8200)
    assert gdn.gdn_layer_status() == 0

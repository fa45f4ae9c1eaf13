"""GPU test of layer_norm_fwd over channels against the two other norms of that layout: the
oracle's layer_norm in 64 bits, and the pre-norm inside block_forward, which a block shows as
out - x where the layer passes its input on (K = 0, D = 1), the projection's values are its
input (identity) and its gates are open (sigmoid(40) = 1)."""
import numpy as np
import pytest
import torch

import oracle
from synth import make_generic_inputs
from test_gpu_block import TOL, run_block

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def s4():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import structured_state_space_dplr_amd as s4
    return s4


@pytest.mark.parametrize("H,L,batch", [(48, 64, 2), (128, 256, 2), (100, 128, 1)])
def test_agrees_with_the_oracle_and_the_block(s4, H, L, batch):
    x = make_generic_inputs(H=H, N=4, L=L, batch=batch, seed=H)
    gen = np.random.default_rng(H)
    gamma, beta = (1 + 0.3 * gen.standard_normal(H)).astype(np.float32), gen.standard_normal(H).astype(np.float32)
    u = torch.from_numpy(np.ascontiguousarray(x["u"], dtype=np.float32)).cuda()
    y = torch.empty_like(u)
    s4.layer_norm_fwd(u, torch.from_numpy(gamma).cuda(), torch.from_numpy(beta).cuda(), y, axis=1)
    y = y.cpu().numpy().astype(np.float64)
    want = oracle.layer_norm(x["u"], gamma, beta)
    # y follows fp32 sums of at most 256 values (2^-20 of their size) and a few roundings
    assert np.abs(y - want).max() <= 64 * 2.0 ** -24 * np.abs(want).max()
    x.update(B=np.zeros_like(x["B"]), C=np.zeros_like(x["C"]), D=np.ones_like(x["D"]))
    W = np.concatenate([np.eye(H), np.zeros((H, H))])
    bias = np.concatenate([np.zeros(H), np.full(H, 40.0)])
    out = run_block(s4, x, {"gamma": gamma, "beta": beta, "W": W, "bias": bias})
    assert np.abs(out - x["u"] - y).max() <= TOL * np.abs(out).max()

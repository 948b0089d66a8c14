"""GPU: calls in a workspace that was sized for a larger one give the same, bit for bit."""
import numpy as np
import pytest
import torch

from tests import ssm_reference as sr
from tests.test_gpu_ssm import Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bf16", [True, False])
def test_a_shorter_prompt(bf16):
    i = sr.make(7, 1, 4096, 32, 1, 32, 32, bf16, gate=False)
    a, b = Layer(i), Layer(i)
    ws = torch.full((a.gdn.ssm_prefill_workspace_bytes(a.d, 4160),), 0xFF, dtype=torch.uint8, device="cuda")
    a.prefill(ws=ws)
    b.prefill()
    torch.cuda.synchronize()
    assert torch.equal(a.y, b.y) and torch.equal(a.state, b.state) and torch.equal(a.tail, b.tail)


def test_a_smaller_selection():
    import gated_deltanet_decode_amd as gdn
    r = np.random.default_rng(8)
    K, V, S = 4, 128000, 4
    ws = torch.full((gdn.beam_select_workspace_bytes(30, K, V, S),), 0xFF, dtype=torch.uint8, device="cuda")
    lg = r.standard_normal((16, K, V)).astype(np.float32)
    sc = -r.random((16, K)).astype(np.float32)
    out = torch.zeros(16, S, device="cuda"), *(torch.zeros(16, S, dtype=torch.int32, device="cuda") for _ in range(2))
    gdn.beam_select(torch.from_numpy(lg).cuda(), torch.from_numpy(sc).cuda(), *out, ws)
    torch.cuda.synchronize()
    want = sr.select(lg, sc, S)
    assert np.array_equal(out[1].cpu().numpy(), want[1]) and np.array_equal(out[2].cpu().numpy(), want[2])

"""More tokens than a grid of chunks holds, against a handful of weight rows."""
import numpy as np
import pytest

import layer_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"


def test_gemm_of_millions_of_tokens():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_matmul_02_amd as bqm

    m, k, n = 4_300_000, 2048, 16         # 4.4 GB of codes; chunks of 48 tokens would be 89584
    g = torch.Generator(device=DEV).manual_seed(1)
    w = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    ws = torch.randint(118, 130, (n, k // 32), generator=g, device=DEV, dtype=torch.uint8)
    xq = torch.randint(0, 256, (m, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    xs = torch.randint(118, 130, (m, k // 32), generator=g, device=DEV, dtype=torch.uint8)
    y = torch.full((m, n), float("nan"), device=DEV)
    bqm.bqm_mxfp4_gemm(w, ws, xq, xs, y)
    assert bool(torch.isfinite(y).all())
    at = torch.tensor([0, 1, m // 4, m // 2, 65535 * 48, 65535 * 64 - 1, 65535 * 64, m - 2, m - 1], device=DEV)
    ref, T = layer_ref.mxfp4_matmul(w.cpu().numpy(), ws.cpu().numpy(),
                                    layer_ref.mxfp4_values(xq[at].cpu().numpy(), xs[at].cpu().numpy()))
    # the bound of the GEMM's own tests: three additions a 64-k step
    assert (np.abs(y[at].cpu().numpy() - ref) <= (3 * k / 64 + 2) * 2.0 ** -23 * T).all()

"""What the backward pass leaves of the error of a delta taken from the rounded O."""
import numpy as np
import pytest
import torch

from oracle import training as tr
from test_gpu_o_attn_train import Problem, _np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[2] * 200, [1, 2, 3, 5, 8] * 30, [33] * 20, [130, 200]])
def test_rows_of_dS_sum_to_zero(d, lens):
    """With one key vector k in every row of K, dQ_i = scale k sum_j dS_ij, whose exact value is 0: dQ shows what delta
    is off by.  Over a block of 128 queries its 2-norm is at most 2^-11 of that of sum_j |dS_ij|.
    Arithmetic: dP and delta are fp32 sums of d products ((d + 16) 2^-24 of the magnitude sum each), a dS is two bf16
    parts (2^-16 of it); the threshold and dQ are rounded (2^-8 of the error itself)."""
    import overlapped_tensor_gemm_gb300 as fo
    pb = Problem(1, 2, 1, d, [(n, n) for n in lens], True, 91 + len(lens))
    k = pb.k[0][:1].clone()
    pb.k[0].copy_(k.expand(pb.mk, d))
    O, LSE, dQ, dK, dV = pb.outputs()
    with fo.Context(0) as c:
        c.attn_forward(pb.q, pb.k, pb.v, O, LSE, **pb.kw)
        c.attn_backward(pb.q, pb.k, pb.v, O, LSE, pb.do, dQ, dK, dV, **pb.kw)
        torch.cuda.synchronize()
        c.poll()
    k = k[0].double().cpu().numpy()
    scale = d ** -0.5
    off = _np(dQ[0], 2, d) @ k / (scale * (k @ k))  # [queries, heads]
    for q, kk, v, do, qs, ks in pb.parts(0):
        _, _, w = tr.attn_forward(q, kk, v)
        for h in range(2):
            dp = do[:, h] @ v[:, 0].T
            ds = w[h] * (dp - (w[h] * dp).sum(1, keepdims=True))
            noise = 2 * (d + 16) * 2.0 ** -24 * (w[h] * (np.abs(do[:, h]) @ np.abs(v[:, 0]).T)).sum(1) * 2 + 2.0 ** -16 * np.abs(ds).sum(1)
            for b in range(0, q.shape[0], 128):
                rows = slice(b, b + 128)
                e = np.linalg.norm(off[qs][rows, h])
                size = np.linalg.norm(np.abs(ds[rows]).sum(1))
                assert e <= (2.0 ** -11 * size + np.linalg.norm(noise[rows])) * (1 + 2.0 ** -7), (qs, h, b, e / size)

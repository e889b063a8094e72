"""Workspaces of the training operators: a call that cannot have its own enqueues nothing, one that needs none asks for
none."""
import pytest
import torch

from test_gpu_o_attn_train import Problem, _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("packed", [False, True])
def test_a_capture_that_lacks_a_later_workspace_holds_nothing(packed):
    """32 query heads on one key/value head: dQ's walks are whole, dK's and dV's are cut into parts, whose sums need a
    workspace of their own.  A small call before has made the others, so the capture can lack that one alone (or, with
    packed sequences, the block table too)."""
    import overlapped_tensor_gemm_gb300 as fo
    small = Problem(1, 2, 2, 64, [(50, 50)], True, 81)
    big = Problem(1, 32, 1, 64, [(2048, 2048)], True, 82, packed=packed)
    O, LSE, dQ, dK, dV = big.outputs()
    with fo.Context(0) as c:
        _check(c, small)
        c.attn_forward(big.q, big.k, big.v, O, LSE, **big.kw)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            with pytest.raises(fo.FoError) as e:
                c.attn_backward(big.q, big.k, big.v, O, LSE, big.do, dQ, dK, dV, **big.kw)
            assert e.value.status == fo.FO_ERR_UNSUPPORTED and "capture" in str(e.value)
            mark = torch.ones(1, device="cuda") * 2  # the graph is not empty
        graph.replay()
        torch.cuda.synchronize()
        c.poll()
        assert mark.item() == 2
        for t in dQ + dK + dV:
            assert torch.isnan(t).all()
        # made once outside, the same call can be captured
        c.attn_backward(big.q, big.k, big.v, O, LSE, big.do, dQ, dK, dV, **big.kw)
        torch.cuda.synchronize()
        want = [t[0].clone() for t in (dQ, dK, dV)]
        for t in dQ + dK + dV:
            t.fill_(0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.attn_backward(big.q, big.k, big.v, O, LSE, big.do, dQ, dK, dV, **big.kw)
        graph.replay()
        torch.cuda.synchronize()
        c.poll()
        for a, b in zip(want, (dQ, dK, dV)):
            assert torch.equal(a, b[0])


def test_a_norm_without_vector_gradients_needs_no_workspace():
    """Residual and a gate per token, no norm: nothing is summed over tokens, so the first call can be captured."""
    import overlapped_tensor_gemm_gb300 as fo
    g = torch.Generator(device="cuda").manual_seed(7)
    R, Y, gate, dR_out = (torch.randn((50, 64), generator=g, device="cuda").to(torch.bfloat16) for _ in range(4))
    dR, dY, dgate = (torch.zeros_like(R) for _ in range(3))
    with fo.Context(0) as c:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.norm_residual_backward([R], [Y], None, [dR_out], [dR], [dY], gate=[gate], dgate=[dgate])
        graph.replay()
        torch.cuda.synchronize()
        c.poll()
    assert torch.equal(dR, dR_out)
    # one fp32 product each, rounded to bf16
    assert torch.equal(dY, (dR_out.float() * gate.float()).to(torch.bfloat16))
    assert torch.equal(dgate, (dR_out.float() * Y.float()).to(torch.bfloat16))

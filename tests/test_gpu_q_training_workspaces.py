"""Workspaces of the training operators: a call that cannot have its own enqueues nothing."""
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

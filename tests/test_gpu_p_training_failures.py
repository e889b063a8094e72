"""The training operators' kernels around a failure: with the abort word of an earlier call raised, and with limits
shorter than any wait, every call ends, the poll reports the failure, and the context computes correctly afterwards.

No wait of these kernels depends on another rank, so none can be made to run out from outside: a GB300 suspends a
waiting thread for longer than their copies and products take, and 20 of 20 calls with a limit of one microsecond
finish.  That a CTA which does give up leaves with no copy and no product in flight is by construction: the warps that
issue them wait for them before they leave, whatever the other warps did."""
import pytest
import torch

import fo_workloads as wl
from helpers import to_dev
from test_gpu_o_attn_train import Problem, _check

pytestmark = pytest.mark.gpu

# short packed sequences (walks shorter than the stages), one long sequence, walks cut into parts
SHAPES = [lambda d: Problem(1, 4, 2, d, [(n, n) for n in (1, 130, 300, 5, 256)] * 8, True, 71),
          lambda d: Problem(1, 4, 4, d, [(2500, 2500)], True, 72),
          lambda d: Problem(1, 8, 1, d, [(700, 700)], False, 73)]


@pytest.fixture()
def ctx():
    import overlapped_tensor_gemm_gb300 as fo
    c = fo.Context(0)
    yield c
    c.close()


def _step(ctx, pb, **kw):
    O, LSE, dQ, dK, dV = pb.outputs()
    ctx.attn_forward(pb.q, pb.k, pb.v, O, LSE, **pb.kw, **kw)
    ctx.attn_backward(pb.q, pb.k, pb.v, O, LSE, pb.do, dQ, dK, dV, **pb.kw, **kw)
    return O, LSE, dQ, dK, dV


def _fail(ctx):
    """A ring call whose hop the host leaves out: its wait runs out and raises the abort word."""
    P, m, K, N = 4, 128, 256, 256
    inp = wl.ag_inputs(P, m, K, N, 77, True)
    X, W = [to_dev(x) for x in inp["X_shards"]], [to_dev(w) for w in inp["W_col"]]
    Y = [torch.zeros((P * m, N), dtype=torch.bfloat16, device="cuda") for _ in range(P)]
    ctx.ag_gemm(X, W, Y, fault="skip_hop", timeout_us=20000)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_calls_behind_a_failed_one(ctx, shape, d):
    """Calls that find the abort word of an earlier failure end early or not, but they end; the poll reports that
    failure, and the same calls after it are right."""
    import overlapped_tensor_gemm_gb300 as fo
    pb = SHAPES[shape](d)
    _fail(ctx)
    for _ in range(3):
        _step(ctx, pb)
    torch.cuda.synchronize()
    with pytest.raises(fo.FoError) as e:
        ctx.poll()
    assert e.value.status == fo.FO_ERR_TIMEOUT
    _check(ctx, pb)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_limits_of_a_microsecond(ctx, shape, d):
    """Each call either gives up, which the poll says, or is right."""
    import overlapped_tensor_gemm_gb300 as fo
    pb = SHAPES[shape](d)
    want = _step(ctx, pb)
    torch.cuda.synchronize()
    ctx.poll()
    for _ in range(20):
        got = _step(ctx, pb, timeout_us=1)
        torch.cuda.synchronize()
        try:
            ctx.poll()
        except fo.FoError as e:
            assert e.status == fo.FO_ERR_TIMEOUT
        else:
            for a, b in zip(want, got):
                assert all(torch.equal(x.nan_to_num(7.0), y.nan_to_num(7.0)) for x, y in zip(a, b))
    _check(ctx, pb)


def test_contexts_of_several_threads_at_once():
    """A host thread may own a context: the first calls of four of them at the same time, each right."""
    import threading

    import overlapped_tensor_gemm_gb300 as fo
    pbs = [Problem(1, 4, 2, 64 if i % 2 else 128, [(400 + 37 * i,) * 2, (90, 90)], True, 90 + i) for i in range(4)]
    outs, wrong = [None] * 4, []
    torch.cuda.synchronize()
    start = threading.Barrier(4)

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()), fo.Context(0) as c:
                start.wait()
                for _ in range(5):
                    outs[i] = _step(c, pbs[i])
                torch.cuda.current_stream().synchronize()
                c.poll()
        except BaseException as e:  # noqa: BLE001
            wrong.append(e)
            start.abort()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
    with fo.Context(0) as c:
        for pb, got in zip(pbs, outs):
            want = _step(c, pb)
            torch.cuda.synchronize()
            c.poll()
            for a, b in zip(want, got):
                assert all(torch.equal(x.nan_to_num(7.0), y.nan_to_num(7.0)) for x, y in zip(a, b))

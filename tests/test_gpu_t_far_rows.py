"""Rows so far apart that a matrix spans more than 2^31 elements: the same bits as from contiguous matrices."""
import pytest
import torch

pytestmark = pytest.mark.gpu

LD = 65536
ROWS = 2 ** 31 // LD + 300  # the last rows lie behind 2^31 elements


@pytest.fixture(scope="module")
def ctx():
    import overlapped_tensor_gemm_gb300 as fo
    c = fo.Context(0)
    yield c
    c.close()


def _far(x):
    """The same matrix with its rows LD elements apart, between columns that nothing may touch."""
    base = torch.empty((x.shape[0], LD), dtype=x.dtype, device="cuda")
    view = base[:, 64:64 + x.shape[1]]
    view.copy_(x)
    return view


def _rnd(g, cols, dtype=torch.bfloat16):
    return torch.randn((ROWS, cols), generator=g, device="cuda").to(dtype)


def test_attention(ctx):
    """Packed sequences, the last of them behind 2^31 elements."""
    g = torch.Generator(device="cuda").manual_seed(3)
    d = 64
    off = torch.tensor([0, 500, ROWS - 700, ROWS - 150, ROWS], dtype=torch.int32, device="cuda")
    near = [_rnd(g, n * d) for n in (2, 1, 1, 2)]  # Q, K, V, dO
    kw = dict(heads=2, kv_heads=1, head_dim=d, q_offsets=off, causal=True)
    got = []
    for move in (lambda x: x, _far):
        Q, K, V, dO = (move(x) for x in near)
        O, dQ, dK, dV = (move(torch.zeros_like(x)) for x in (near[0], *near[:3]))
        LSE = torch.zeros((2, -(-ROWS // 4) * 4), device="cuda")[:, :ROWS]
        ctx.attn_forward([Q], [K], [V], [O], [LSE], **kw)
        ctx.attn_backward([Q], [K], [V], [O], [LSE], [dO], [dQ], [dK], [dV], **kw)
        torch.cuda.synchronize()
        ctx.poll()
        got.append([t.clone() for t in (O, LSE, dQ, dK, dV)])
        assert dK[-1].abs().sum() > 0
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [512, 333])
def test_norm_and_rope(ctx, dtype, cols):
    import overlapped_tensor_gemm_gb300 as fo
    g = torch.Generator(device="cuda").manual_seed(4)
    R, Y, dX, dR = (_rnd(g, cols, t) for t in (dtype, torch.bfloat16, torch.bfloat16, dtype))
    w = [torch.randn(cols, generator=g, device="cuda") for _ in range(3)]
    got = []
    for move in (lambda x: x, _far):
        pad = lambda x: torch.nn.functional.pad(x, (0, -x.shape[1] % 8))[:, :x.shape[1]]  # noqa: E731
        r, y, dx, dr = (move(x) if move is _far else pad(x) for x in (R, Y, dX, dR))
        ro, x, ndr, ndy = ((move if move is _far else pad)(torch.zeros_like(t)) for t in (R, Y, R, Y))
        dw = [torch.empty(cols, device="cuda") for _ in range(3)]
        ctx.norm_residual([r], [y], [ro], [x], w_post=w[0], gate=w[1], w_pre=w[2])
        ctx.norm_residual_backward([ro], [y], [dx], [dr], [ndr], [ndy], w_post=w[0], gate=w[1], w_pre=w[2],
                                   dw_post=dw[0], dgate=dw[1], dw_pre=dw[2])
        turned = (move if move is _far else pad)(torch.zeros_like(R))
        if cols % 64 == 0:
            ctx.rope([r], [turned], fo.RopeTable(64))
        torch.cuda.synchronize()
        ctx.poll()
        got.append([t.clone() for t in (ro, x, ndr, ndy, turned, *dw)])
        del r, y, dx, dr, ro, x, ndr, ndy, turned
        torch.cuda.empty_cache()
    for a, b in zip(*got):
        assert torch.equal(a, b)

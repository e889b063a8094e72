"""The 8-bit code of m, bit by bit, as elementary fp32 operations give it.  A random part decides a code, so that
a last bit of m, of its block's scale or of their quotient can move it by a whole step of e4m3 (up to an
eighth); such an element's weight leaves fp32's accuracy in the next step.  Hence nothing is left open: each
product and the sum of m are rounded once, the quotient as IEEE rounds it, and the codes are equal."""
import numpy as np
import pytest
import torch

from oracle import losses as ls

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
BETA1, BETA2 = 0.9, 0.95


@pytest.fixture(scope="module")
def ctx():
    import overlapped_tensor_gemm_gb300 as fo
    c = fo.Context(0)
    yield c
    c.close()


def _group(sizes, kind, seed):
    import overlapped_tensor_gemm_gb300 as fo
    param, grad, master = kind
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda n: torch.randn(n, generator=g, device="cuda")  # noqa: E731
    wide = [torch.exp2(3 * randn(-(-n // 256))) for n in sizes]  # rows of a weight differ in scale
    each = [x.repeat_interleave(256)[:n] for x, n in zip(wide, sizes)]
    s = {"w": [(0.02 * randn(n)).to(param) for n in sizes],
         "g": [(1e-3 * randn(n) * x).to(grad) for n, x in zip(sizes, each)],
         "v": [torch.randint(1, 256, (n,), generator=g, device="cuda").to(torch.uint8) for n in sizes]}
    s["master"] = [w.float() for w in s["w"]] if master else None
    s["m_scale"] = [3e-4 * x * torch.rand(x.shape, generator=g, device="cuda") / 100 for x in wide]
    s["m"] = [(120 * randn(n)).clamp(-448, 448).to(torch.float8_e4m3fn) for n in sizes]
    s["v_range"] = [torch.stack([2 * torch.log2(3e-4 * x), torch.full_like(x, 0.03)], 1).reshape(-1).contiguous() for x in wide]
    return s, fo.AdamWTensors(s["w"], s["g"], s["m"], s["v"], master=s["master"], m_scale=s["m_scale"], v_range=s["v_range"])


def _codes(q, scale, grad, factor, words):
    """(m as e4m3 values, scales) behind the step, for one tensor"""
    n, nb = q.numel(), scale.numel()
    blocks = lambda x: torch.nn.functional.pad(x, (0, nb * 256 - n)).view(nb, 256)  # noqa: E731
    b1, r1 = (torch.tensor(x, dtype=F32, device="cuda") for x in (BETA1, 1 - BETA1))
    old = blocks(q.float()) * scale[:, None]
    m = b1 * old + r1 * (blocks(grad.float()) * factor)
    top = m.abs().amax(1, keepdim=True)
    new = top * torch.tensor(1 / 448, dtype=F32, device="cuda")
    x = (m.abs() / new).double().clamp(max=448)
    # below 2^-6 steps are 2^-9; a step's part has 20 bits
    x = torch.where(x < 2.0 ** -6, torch.round(x * 2.0 ** 29) * 2.0 ** -29, x)
    step = torch.exp2(torch.floor(torch.log2(x.clamp(min=2.0 ** -6))) - 3)
    r = blocks(torch.from_numpy((words & np.uint64(0xFFFF)).astype(np.float64)).cuda()) / 65536
    code = torch.copysign(torch.floor(x / step + r) * step, m.double())
    return code.reshape(-1)[:n], new[:, 0]


@pytest.mark.parametrize("kind", [(BF, BF, True), (F32, F32, False), (BF, F32, False)], ids=["masters", "fp32", "bf16"])
@pytest.mark.parametrize("factor", [1.0, 0.37])
def test_codes_of_m(ctx, kind, factor):
    sizes, seed = [9000001, 700, 3, 2000256, 257, 4194304], 0x13579BDF02468
    s, group = _group(sizes, kind, 1)
    f = torch.tensor(factor, dtype=F32, device="cuda")
    want = [_codes(s["m"][i], s["m_scale"][i], s["g"][i], f, ls.words(seed, 12, i, n)) for i, n in enumerate(sizes)]
    ctx.adamw_step(group, 3e-4, 12, beta1=BETA1, beta2=BETA2, grad_scale=float(f.item()), seed=seed)
    torch.cuda.synchronize()
    ctx.poll()
    for i in range(len(sizes)):
        assert torch.equal(s["m_scale"][i], want[i][1]), i
        wrong = s["m"][i].float().double() != want[i][0]
        assert not wrong.any(), (i, int(wrong.sum()), s["m"][i].float()[wrong][:4], want[i][0][wrong][:4])

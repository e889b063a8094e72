"""Norm and unpacking of so many elements that a warp takes four blocks in a row, across tensors of odd sizes;
8-bit states of more tensors than a launch takes; the random rounding of bf16 weights, value by value."""
import numpy as np
import pytest
import torch

import test_gpu_v_adamw as adamw
from oracle import losses as ls

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
u = 2.0 ** -24
# 28 million elements: runs of four blocks begin at 16 blocks a warp, 152 x 4 x 8 warps, 256 elements a block
LONG = [9000001, 300, 7, 8448 + 5, 8000777, 1, 1280000, 700, 3000003, 257, 6710016]


@pytest.fixture(scope="module")
def ctx():
    import overlapped_tensor_gemm_gb300 as fo
    c = fo.Context(0)
    yield c
    c.close()


def _placed(n, dtype):
    """n elements 64 bytes into a buffer whose other bytes are 77, and a check of those"""
    size = torch.empty((), dtype=dtype).element_size()
    base = torch.full((n * size + 144,), 77, dtype=torch.uint8, device="cuda")

    def check():
        assert (base[:64] == 77).all() and (base[64 + n * size:] == 77).all()
    return base[64:64 + n * size].view(dtype), check


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_norm_of_runs_of_blocks(ctx, dtype):
    """About one element in a block is 1 or 2, the others 0: the squares' sum is a whole number (110 000 blocks, 2.5 in
    the mean), which twice fp32 holds exactly, and one missed or doubled element is 2e-6 of the norm."""
    import overlapped_tensor_gemm_gb300 as fo
    g = torch.Generator(device="cuda").manual_seed(1)
    grads, total = [], 0
    for n in LONG:
        t = torch.zeros(n, dtype=dtype, device="cuda")
        at = torch.randint(0, n, (max(1, n // 256),), generator=g, device="cuda")
        t[at] = torch.randint(1, 3, at.shape, generator=g, device="cuda").to(dtype)
        t[-1] = 1
        grads.append(t)
        total += int((t.double() ** 2).sum().item())
    w = [torch.zeros(n, dtype=BF, device="cuda") for n in LONG]
    m, v, _, _ = fo.adamw_states(w)
    norm = torch.zeros(1, device="cuda")
    ctx.grad_norm(fo.AdamWTensors(w, grads, m, v), norm)
    torch.cuda.synchronize()
    assert abs(norm.item() - total ** 0.5) <= 2 * u * total ** 0.5


def _random_states(sizes, seed):
    """8-bit states of any codes (m's but NaN), ranges as a training run has them; with the checks of their surroundings"""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = ([], [], [], [])
    for n in sizes:
        nb = -(-n // 256)
        q = torch.randint(0, 254, (n,), generator=g, device="cuda")
        q = torch.where(q >= 127, q + 1, q).to(torch.uint8)  # (127 and 255 are NaN)
        out[0].append(q.view(torch.float8_e4m3fn))
        out[1].append(torch.randint(0, 256, (n,), generator=g, device="cuda").to(torch.uint8))
        out[2].append(torch.exp2(torch.randn(nb, generator=g, device="cuda") - 12))
        low = -30 + 4 * torch.randn(nb, generator=g, device="cuda")
        gap = torch.rand(nb, generator=g, device="cuda") * (24 / 254)
        out[3].append(torch.stack([low, gap], 1).reshape(-1).contiguous())
    return out


def _check_unpacked(states, i, n, m, v, dtype):
    """Against the header's formula in 64 bits: two roundings of m and the output's; v is 2^x with x rounded to fp32 (two
    operations on numbers below 64) and an exponential of 2^-22"""
    block = torch.arange(n, device="cuda") // 256
    rm = states[0][i].float().double() * states[2][i].double()[block]
    low, gap = states[3][i].double().view(-1, 2).T
    code = states[1][i].double()
    rv = torch.where(code > 0, torch.exp2(low[block] + (code - 1) * gap[block]), 0.0)
    for got, ref in ((m, rm), (v, rv)):
        tol = (adamw.HALF[dtype] + 64 * u) * ref.abs() + 2.0 ** -149
        assert ((got.double() - ref).abs() <= tol).all(), i


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_unpacking_of_runs_of_blocks(ctx, dtype):
    import overlapped_tensor_gemm_gb300 as fo
    states = _random_states(LONG, 2)
    w = [torch.zeros(n, dtype=BF, device="cuda") for n in LONG]
    group = fo.AdamWTensors(w, w and [torch.zeros_like(x) for x in w], states[0], states[1], m_scale=states[2],
                            v_range=states[3])
    out = [[_placed(n, dtype) for n in LONG] for _ in range(2)]
    ctx.adamw_unpack(group, *[[t for t, _ in x] for x in out])
    torch.cuda.synchronize()
    for i, n in enumerate(LONG):
        _check_unpacked(states, i, n, out[0][i][0], out[1][i][0], dtype)
        out[0][i][1](), out[1][i][1]()


def test_8_bit_states_of_more_tensors_than_a_launch_takes(ctx):
    """900 tensors of three kinds with 8-bit states: step, codes (a tensor's place in the whole group enters the random
    words) and unpacking."""
    sizes = [1 + (i * 53) % 700 for i in range(900)]
    s = adamw.Set(sizes, [adamw.KINDS[3], adamw.KINDS[10], adamw.KINDS[4]], seed=15)
    before = [s.values(i) for i in range(len(sizes))]
    ctx.adamw_step(s.group, step=9, stochastic=True, seed=0x5555AAAA12345, **adamw.HYPER)
    out = [[torch.full((n,), 7.0, device="cuda") for n in sizes] for _ in range(2)]
    ctx.adamw_unpack(s.group, *out)
    torch.cuda.synchronize()
    ctx.poll()
    s.check_guards()
    adamw._check_step(s, before, 9, 1.0, True, 0x5555AAAA12345)
    for i, n in enumerate(sizes):
        for got, ref in zip((out[0][i], out[1][i]), s.values(i)[2:]):
            assert (np.abs(got.double().cpu().numpy() - ref) <= 65 * u * np.abs(ref) + 2.0 ** -149).all(), i


@pytest.mark.parametrize("which", [[2, 8], [5, 10]], ids=["32-bit", "8-bit"])
def test_random_rounding_of_weights_by_the_stated_word(ctx, which):
    """A bf16 weight without a master is the one of the two values around the new weight that the header's random word
    says.  The fp32 weight has 16 bits below bf16's; what is added to them is 16 bits of the word.  Where the sum is
    nearer to the next value than the weight's own error (that of the step's other tests) and its rounding to
    fp32, half of 2^-16 of a bf16 step, either neighbour will do."""
    hyper, step, seed = adamw.HYPER, 6, 0xFEDCBA9876543
    s = adamw.Set([1000, 70000, 3, 256, 5003, 257], [adamw.KINDS[k] for k in which], seed=16)
    before = [s.values(i) for i in range(len(s.sizes))]
    ctx.adamw_step(s.group, step=step, stochastic=True, seed=seed, **hyper)
    torch.cuda.synchronize()
    c64 = lambda x: float(np.float32(x))  # noqa: E731
    lr, eps, wd, b1, b2 = c64(hyper["lr"]), c64(hyper["eps"]), c64(hyper["weight_decay"]), hyper["beta1"], hyper["beta2"]
    decided = total = 0
    for i, n in enumerate(s.sizes):
        w, g, m, v = before[i]
        rw, rm, rv = ls.adamw(w, g, m, v, step, lr, b1, b2, eps, wd)
        root = np.sqrt(rv / (1 - b2 ** step)) + eps
        em = 4 * u * (np.abs(b1 * m) + np.abs((1 - b1) * g))
        ev = 6 * u * rv + (64 * u * v if which[0] == 5 else 0.0)
        update = np.abs(rm / (1 - b1 ** step)) / root
        ew = (4 * u * (np.abs(w) * (1 + lr * wd) + lr * update)
              + lr * (update * (ev / np.where(rv > 0, rv, 1) + 32 * u) + em / (1 - b1 ** step) / root))
        word = ls.words(seed, step, i, n) * np.uint64(0x9E3779B9) & np.uint64(0xFFFFFFFF)
        r = (word >> np.uint64(16)).astype(np.float64) / 65536
        size = np.exp2(np.floor(np.log2(np.abs(rw))) - 7)   # a bf16 step
        part = np.abs(rw) / size
        want = np.sign(rw) * np.floor(part + r) * size
        near = np.abs(part + r - np.round(part + r)) <= ew / size + 2.0 ** -16
        got = s.w[i].double().cpu().numpy()
        wrong = got != want
        assert not (wrong & ~near).any(), (i, int((wrong & ~near).sum()), got[wrong & ~near][:3], want[wrong & ~near][:3])
        assert (np.abs(got - want) <= size * 1.001).all()
        decided, total = decided + int((~near).sum()), total + n
    assert decided >= 0.9 * total  # (an error of 2^-12 of a step leaves all but one in a thousand)


def test_many_tensors_in_one_group_and_in_groups_of_their_own(ctx):
    """32-bit states: the same bits, whichever launch and place a tensor has."""
    import overlapped_tensor_gemm_gb300 as fo
    sizes = [1 + (i * 37) % 600 for i in range(900)]
    kinds = [adamw.KINDS[0], adamw.KINDS[1], adamw.KINDS[8]]
    s, t = adamw.Set(sizes, kinds, seed=17), adamw.Set(sizes, kinds, seed=17)
    ctx.adamw_step(s.group, step=7, **adamw.HYPER)
    for i in range(len(sizes)):
        one = fo.AdamWTensors(t.w[i:i + 1], t.g[i:i + 1], t.m[i:i + 1], t.v[i:i + 1], master=t.master[i:i + 1])
        ctx.adamw_step(one, step=7, **adamw.HYPER)
    torch.cuda.synchronize()
    for a, b in zip(s.state(), t.state()):
        assert torch.equal(a, b)

"""The barrier protocol of the attention training kernels, on the CPU.

A wait names a phase of its barrier by one bit, so it tells a phase that has completed from one that has not only
while the barrier is at most one phase ahead of it: a waiter that looks later than that waits for ever.  The roles
of a kernel are written down here as their waits and arrivals; the arrays' sizes come from the sources.  Nothing
that a role does can keep another one from going on, so the most phases that a barrier can complete while a wait is
still to be looked at are those of the run in which that one role stands still and all others go as far as they can."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "overlapped_tensor_gemm_gb300", "csrc")
N = 9  # blocks of a walk
WORKERS = 2  # of the warps that share a barrier: enough for one to be late


def _sizes(source, struct, **constants):
    """Barriers per field of a control block."""
    with open(os.path.join(CSRC, source)) as f:
        body = re.search(r"struct alignas\(8\) %s \{(.*?)\};" % struct, f.read(), re.S).group(1)
    out = {}
    for line in re.findall(r"uint64_t ([^;]*);", body):
        for name, size in re.findall(r"(\w+)(?:\[(\w+)\])?", line):
            out[name] = int(constants.get(size, size)) if size else 1
    return out


def _ring(size, i):
    return i % size, i // size


class Net:
    """Roles as lists of ("wait", barrier, phase) and ("arrive", barrier, ...); the arrivals of a copy or of the
    tensor pipe stand where they are issued.  A phase of -1: a wait that a fresh barrier passes."""

    def __init__(self):
        self.roles, self.needs = {}, {}

    def run(self, late=None):
        """Completed phases of every barrier once nothing moves any more, and the roles that are done; `late`: a
        (role, position) that is not passed."""
        at = dict.fromkeys(self.roles, 0)
        got = {}
        done = lambda b: got.get(b, 0) // self.needs.get(b, 1)  # noqa: E731
        moved = True
        while moved:
            moved = False
            for name, ops in self.roles.items():
                while at[name] < len(ops) and (name, at[name]) != late:
                    op = ops[at[name]]
                    if op[0] == "wait":
                        if done(op[1]) <= op[2]:
                            break
                    else:
                        for b in op[1:]:
                            got[b] = got.get(b, 0) + 1
                    at[name] += 1
                    moved = True
        return done, {n for n in self.roles if at[n] == len(self.roles[n])}

    def check(self):
        done, finished = self.run()
        assert finished == set(self.roles)
        for name, ops in self.roles.items():
            for pos, op in enumerate(ops):
                if op[0] != "wait":
                    continue
                done, _ = self.run(late=(name, pos))
                assert done(op[1]) <= op[2] + 1, (name, pos, op, "phases completed", done(op[1]))


def _wait(name, size, i):
    slot, phase = _ring(size, i)
    return ("wait", (name, slot), phase)


def _free(name, size, i):  # the slot's last use before i has been released
    slot, phase = _ring(size, i)
    return ("wait", (name, slot), phase - 1)


def _at(name, size, i):
    return (name, i % size)


def test_a_barrier_two_phases_ahead_is_found():
    net = Net()
    net.roles = {"fast": [("arrive", "b")] * 2, "late": [("wait", "b", 0), ("wait", "b", 1)]}
    with pytest.raises(AssertionError):
        net.check()


@pytest.mark.parametrize("dim", [64, 128])
def test_dkv(dim):
    z = _sizes("fo_attn_bwd.cu", "DkvCtl")
    bufs = 2 if dim == 64 else 1  # buffers of S^T
    weights = min(z["p_full"], bufs)
    load, mma, stats = [], [], []
    for i in range(N):
        load += [_free("empty", 2, i), ("arrive", _at("q_full", 2, i)), ("arrive", _at("do_full", 2, i))]
        stats += [_free("st_empty", 2, i), ("arrive", _at("st_full", 2, i))]
    mma += [_wait("q_full", 2, 0), ("arrive", ("s_full", 0)), _wait("do_full", 2, 0), ("arrive", ("dp_full", 0))]
    for i in range(N):
        more = i + 1 < N
        scores = [_wait("q_full", 2, i + 1), ("arrive", _at("s_full", bufs, i + 1))] if more else []
        if bufs == 2:
            mma += scores
        mma += [_wait("p_full", weights, i)]
        if bufs == 1:
            mma += scores
        mma += [_wait("ds_full", z["ds_full"], i), ("arrive", _at("empty", 2, i))]
        if more:
            mma += [_wait("do_full", 2, i + 1), ("arrive", ("dp_full", 0))]
    mma += [("arrive", ("acc_full", 0))]
    net = Net()
    net.roles = {"load": load, "mma": mma, "stats": stats}
    for w in range(WORKERS):
        ops = []
        for i in range(N):
            ops += [_wait("st_full", 2, i), _wait("s_full", bufs, i), ("arrive", _at("p_full", weights, i)),
                    _wait("dp_full", 1, i), ("arrive", _at("ds_full", z["ds_full"], i)), ("arrive", _at("st_empty", 2, i))]
        net.roles[f"work {w}"] = ops + [_wait("acc_full", 1, 0)]
    for b in [_at(n, z[n], i) for n in ("p_full", "ds_full", "st_empty") for i in range(2)]:
        net.needs[b] = WORKERS
    net.check()


def test_dq():
    z = _sizes("fo_attn_bwd.cu", "DqCtl", kKStages=3, kVStages=2)
    ks, vs, ds = z["k_full"], z["v_full"], z["ds_full"]
    load, scores, grad = [], [], []
    for i in range(N):
        load += [_free("k_empty", ks, i), ("arrive", _at("k_full", ks, i)), _free("v_empty", vs, i), ("arrive", _at("v_full", vs, i))]
        scores += [_wait("k_full", ks, i)] + ([_free("s_free", 2, i)] if i >= 2 else []) + [("arrive", _at("s_full", 2, i))]
        scores += [_wait("v_full", vs, i)] + ([_wait("dp_free", 1, i - 1)] if i >= 1 else [])
        scores += [("arrive", ("dp_full", 0), _at("v_empty", vs, i))]
        grad += [_wait("ds_full", ds, i), ("arrive", _at("s_free", 2, i), _at("k_empty", ks, i))]
    net = Net()
    net.roles = {"load": load, "scores": scores, "grad": grad + [("arrive", ("acc_full", 0))]}
    for w in range(WORKERS):
        ops = []
        for i in range(N):
            ops += [_wait("s_full", 2, i), _wait("dp_full", 1, i), ("arrive", ("dp_free", 0)), ("arrive", _at("ds_full", ds, i))]
        net.roles[f"work {w}"] = ops + [_wait("acc_full", 1, 0)]
    net.needs[("dp_free", 0)] = WORKERS
    for i in range(ds):
        net.needs[("ds_full", i)] = WORKERS
    net.check()


@pytest.mark.parametrize("dim,apart", [(64, True), (64, False), (128, False)])
@pytest.mark.parametrize("rescale", [False, True])
def test_forward(dim, apart, rescale):
    ks, vs = (4, 4) if dim == 64 else (2, 3)
    load = []
    for j in range(N):
        load += [_free("k_empty", ks, j), ("arrive", _at("k_full", ks, j)), _free("v_empty", vs, j), ("arrive", _at("v_full", vs, j))]
    mma = [_wait("k_full", ks, 0)] + [("arrive", ("s_full", t)) for t in range(2)] + [_wait("v_full", vs, 0)]
    for j in range(N):
        more = j + 1 < N
        for t in range(2):
            operands = [_wait("v_full" if t else "k_full", vs if t else ks, j + 1)] if more else []
            product = [("arrive", ("o_done", t))]
            mma += operands if apart else []
            mma += [("wait", ("p_full", t), j)]
            mma += [] if apart else product + operands
            mma += [("arrive", ("s_full", t))] if more else []
            mma += product if apart else []
            if t == 0:
                mma += [("arrive", _at("k_empty", ks, j))] + ([("arrive", _at("v_empty", vs, j - 1))] if j else [])
    net = Net()
    net.roles = {"load": load, "mma": mma}
    for t in range(2):
        net.needs[("p_full", t)] = WORKERS
        for w in range(WORKERS):
            ops = []
            for j in range(N):
                ops += [("wait", ("s_full", t), j)]
                ops += [("wait", ("o_done", t), j - 1)] if j and (apart or rescale) else []
                ops += [("arrive", ("p_full", t))]
            net.roles[f"softmax {t} {w}"] = ops + [("wait", ("o_done", t), N - 1)]
    net.check()

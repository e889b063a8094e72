"""Refusals of the training operators' entry points and their host-only parts, without a GPU: every
argument is checked before the context is, so a null context reaches the checks and is refused last."""
import ctypes
import math
import os
import types

import numpy as np
import pytest

import overlapped_tensor_gemm_gb300 as fo
from oracle import training as tr

NULL = ctypes.c_void_p()
PAGE = 1 << 20  # matrices of the tests lie this far apart (addresses that nothing reads)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fo.LIB_PATH):
        from overlapped_tensor_gemm_gb300 import _build
        _build.build()
    return fo.load()


def _mat(slot, rows, cols, dtype=fo.FO_BF16, ld=None, offset=0):
    ld = -(-cols // 8) * 8 if ld is None else ld
    return fo.FoMat((slot + 1) * PAGE + offset, dtype, 0, rows, cols, ld)


def _arr(*mats):
    return (fo.FoMat * len(mats))(*mats)


def _refused(status, want, text):
    msg = fo.load().fo_last_error_string().decode()
    assert status == want, (status, msg)
    assert text in msg, msg


# -- norms -----------------------------------------------------------------------------------
class Norm:
    """A valid call (m = 4, H = 24, P = 2) whose parts a test replaces."""

    def __init__(self):
        self.m, self.h = 4, 24
        two = lambda slot, dt=fo.FO_BF16: _arr(_mat(slot, 4, 24, dt), _mat(slot + 1, 4, 24, dt))  # noqa: E731
        self.R, self.Y, self.RO, self.X = two(0, fo.FO_F32), two(2), two(4, fo.FO_F32), two(6)
        self.dX, self.dRO, self.dR, self.dY = two(8), two(10, fo.FO_F32), two(12, fo.FO_F32), two(14)
        self.w_post, self.w_pre, self.gate = _arr(_mat(16, 1, 24)), _arr(_mat(17, 1, 24)), _arr(_mat(18, 1, 24))
        self.d_post, self.d_pre, self.d_gate = (_arr(_mat(20 + i, 1, 24, fo.FO_F32)) for i in range(3))
        self.token, self.alpha, self.eps, self.P = 0, 1.0, 1e-6, 2

    def params(self):
        ptr = lambda a: None if a is None else ctypes.cast(a, ctypes.POINTER(fo.FoMat))  # noqa: E731
        return (fo.FoNormParams(ptr(self.w_post), ptr(self.w_pre), ptr(self.gate), self.token, self.alpha, self.eps, 0),
                fo.FoNormGrads(ptr(self.d_post), ptr(self.d_pre), ptr(self.d_gate)))

    def forward(self):
        p, _ = self.params()
        return fo.load().fo_norm_residual(NULL, self.R, self.Y, self.P, ctypes.byref(p), self.RO, self.X, NULL)

    def backward(self):
        p, g = self.params()
        return fo.load().fo_norm_residual_backward(NULL, self.RO, self.Y, self.dX, self.dRO, self.P, ctypes.byref(p),
                                                   self.dR, self.dY, ctypes.byref(g), NULL)


def test_norm_valid_calls_reach_the_context(lib):
    c = Norm()
    _refused(c.forward(), fo.FO_ERR_INVALID_ARG, "null context")
    _refused(c.backward(), fo.FO_ERR_INVALID_ARG, "null context")
    c = Norm()
    c.RO, c.X = c.R, c.Y          # both in place
    _refused(c.forward(), fo.FO_ERR_INVALID_ARG, "null context")
    c = Norm()
    c.dR, c.dY = c.dRO, c.dX
    _refused(c.backward(), fo.FO_ERR_INVALID_ARG, "null context")
    c = Norm()
    c.Y = c.RO = c.w_post = c.gate = None  # the norm in front of the first block
    _refused(c.forward(), fo.FO_ERR_INVALID_ARG, "null context")


@pytest.mark.parametrize("change,want,text", [
    (lambda c: setattr(c, "P", 0), fo.FO_ERR_INVALID_ARG, "P=0"),
    (lambda c: setattr(c, "P", 9), fo.FO_ERR_INVALID_ARG, "P=9"),
    (lambda c: setattr(c, "R", None), fo.FO_ERR_INVALID_ARG, "null matrix"),
    (lambda c: setattr(c, "RO", None), fo.FO_ERR_INVALID_ARG, "R_out goes with"),
    (lambda c: setattr(c, "Y", None), fo.FO_ERR_INVALID_ARG, "need a block output"),
    (lambda c: setattr(c, "X", None), fo.FO_ERR_INVALID_ARG, "both or neither"),
    (lambda c: setattr(c, "w_pre", None), fo.FO_ERR_INVALID_ARG, "both or neither"),
    (lambda c: setattr(c, "eps", -1.0), fo.FO_ERR_INVALID_ARG, "eps"),
    (lambda c: setattr(c, "eps", math.nan), fo.FO_ERR_INVALID_ARG, "eps"),
    (lambda c: setattr(c, "alpha", math.inf), fo.FO_ERR_INVALID_ARG, "residual_scale"),
    (lambda c: setattr(c, "token", 2), fo.FO_ERR_INVALID_ARG, "gate_per_token"),
    (lambda c: setattr(c, "w_post", _arr(_mat(16, 1, 23))), fo.FO_ERR_SHAPE, "w_post"),
    (lambda c: setattr(c, "w_post", _arr(_mat(16, 1, 24, 7))), fo.FO_ERR_INVALID_ARG, "w_post"),
    (lambda c: setattr(c, "gate", _arr(_mat(18, 4, 24))), fo.FO_ERR_SHAPE, "gate"),
    (lambda c: setattr(c, "gate", _arr(_mat(18, 1, 24, fo.FO_F32))), fo.FO_ERR_UNSUPPORTED, "one type"),
    (lambda c: c.Y.__setitem__(1, _mat(3, 5, 24)), fo.FO_ERR_SHAPE, "Y[1]"),
    (lambda c: c.Y.__setitem__(1, _mat(3, 4, 24, fo.FO_F32)), fo.FO_ERR_INVALID_ARG, "Y[1]"),
    (lambda c: c.R.__setitem__(0, _mat(0, 4, 16400, fo.FO_F32)), fo.FO_ERR_UNSUPPORTED, "at most 16384"),
    (lambda c: c.X.__setitem__(0, _mat(6, 4, 24, offset=2)), fo.FO_ERR_UNSUPPORTED, "aligned"),
    (lambda c: c.X.__setitem__(0, _mat(6, 4, 24, ld=25)), fo.FO_ERR_UNSUPPORTED, "pitch"),
    (lambda c: c.X.__setitem__(0, _mat(2, 4, 24, offset=16)), fo.FO_ERR_INVALID_ARG, "overlaps"),
    (lambda c: c.X.__setitem__(0, _mat(3, 4, 24)), fo.FO_ERR_INVALID_ARG, "overlaps"),   # X[0] over Y[1]
    (lambda c: c.X.__setitem__(1, c.X[0]), fo.FO_ERR_INVALID_ARG, "overlaps"),
    (lambda c: c.RO.__setitem__(0, _mat(16, 4, 24, fo.FO_F32)), fo.FO_ERR_INVALID_ARG, "overlaps w_post"),
])
def test_norm_forward_refusals(lib, change, want, text):
    c = Norm()
    change(c)
    _refused(c.forward(), want, text)


@pytest.mark.parametrize("change,want,text", [
    (lambda c: (setattr(c, "dX", None), setattr(c, "dRO", None)), fo.FO_ERR_INVALID_ARG, "neither dX"),
    (lambda c: setattr(c, "dX", None), fo.FO_ERR_INVALID_ARG, "both or neither"),
    (lambda c: setattr(c, "dY", None), fo.FO_ERR_INVALID_ARG, "dY goes with"),
    (lambda c: setattr(c, "d_post", None), fo.FO_ERR_INVALID_ARG, "its gradient"),
    (lambda c: setattr(c, "w_post", None), fo.FO_ERR_INVALID_ARG, "its gradient"),
    (lambda c: setattr(c, "d_gate", _arr(_mat(22, 4, 24))), fo.FO_ERR_SHAPE, "dgate"),
    (lambda c: c.dR.__setitem__(0, _mat(4, 4, 24, fo.FO_F32)), fo.FO_ERR_INVALID_ARG, "overlaps R_out"),
    (lambda c: c.dY.__setitem__(0, _mat(2, 4, 24)), fo.FO_ERR_INVALID_ARG, "overlaps Y"),
    (lambda c: setattr(c, "d_pre", c.d_post), fo.FO_ERR_INVALID_ARG, "overlaps"),
])
def test_norm_backward_refusals(lib, change, want, text):
    c = Norm()
    change(c)
    _refused(c.backward(), want, text)


def test_views_of_one_matrix_do_not_overlap(lib):
    # R, Y, R_out and X as column ranges of one wide matrix: side by side is fine, one column shared is not
    c = Norm()
    col = lambda at, cols=24: _arr(_mat(0, 4, cols, ld=256, offset=2 * at))  # noqa: E731
    c.P, c.R, c.Y, c.RO, c.X = 1, col(0), col(24), col(48), col(72)
    _refused(c.forward(), fo.FO_ERR_INVALID_ARG, "null context")
    c.X = col(64)
    _refused(c.forward(), fo.FO_ERR_INVALID_ARG, "overlaps")
    c.X = _arr(_mat(0, 4, 24, ld=256, offset=2 * 240))  # its rows run into the next rows' R
    _refused(c.forward(), fo.FO_ERR_INVALID_ARG, "overlaps R")


# -- attention -------------------------------------------------------------------------------
class Attn:
    """A valid call (5 queries, 7 keys, 4 heads on 2, head_dim 64, P = 2) whose parts a test replaces."""

    def __init__(self):
        two = lambda slot, rows, cols, dt=fo.FO_BF16: _arr(_mat(slot, rows, cols, dt), _mat(slot + 1, rows, cols, dt))  # noqa: E731
        self.Q, self.K, self.V = two(0, 5, 256), two(2, 7, 128), two(4, 7, 128)
        self.O, self.LSE, self.dO = two(6, 5, 256), two(8, 4, 5, fo.FO_F32), two(10, 5, 256)
        self.dQ, self.dK, self.dV = two(12, 5, 256), two(14, 7, 128), two(16, 7, 128)
        self.P, self.heads, self.kv, self.dim = 2, 4, 2, 64
        self.mask = fo.FoAttnMask(1, 0, None, None, 0.0, 0)

    def forward(self):
        mask = None if self.mask is None else ctypes.byref(self.mask)
        return fo.load().fo_attn_forward(NULL, self.Q, self.K, self.V, self.P, self.heads, self.kv, self.dim, mask,
                                         self.O, self.LSE, None, NULL)

    def backward(self):
        mask = None if self.mask is None else ctypes.byref(self.mask)
        return fo.load().fo_attn_backward(NULL, self.Q, self.K, self.V, self.O, self.LSE, self.dO, self.P, self.heads,
                                          self.kv, self.dim, mask, self.dQ, self.dK, self.dV, None, NULL)


BAD, SHAPE, NO = fo.FO_ERR_INVALID_ARG, fo.FO_ERR_SHAPE, fo.FO_ERR_UNSUPPORTED


@pytest.mark.parametrize("change,want,text", [
    (lambda c: None, BAD, "null context"),
    (lambda c: (c.mask.__setattr__("num_seqs", 3), c.mask.__setattr__("q_offsets", PAGE),
                c.mask.__setattr__("k_offsets", PAGE)), BAD, "null context"),
    (lambda c: setattr(c, "P", 0), BAD, "P=0"),
    (lambda c: setattr(c, "Q", None), BAD, "null matrix"),
    (lambda c: setattr(c, "O", None), BAD, "null matrix"),
    (lambda c: setattr(c, "mask", None), BAD, "null matrix array or mask"),
    (lambda c: setattr(c, "kv", 3), BAD, "multiple of kv_heads"),
    (lambda c: setattr(c, "kv", 0), BAD, "multiple of kv_heads"),
    (lambda c: setattr(c, "dim", 96), NO, "head_dim"),
    (lambda c: setattr(c, "dim", 128), SHAPE, "Q[0]"),
    (lambda c: setattr(c, "heads", 6), SHAPE, "Q[0]"),
    (lambda c: c.mask.__setattr__("causal", 2), BAD, "causal"),
    (lambda c: c.mask.__setattr__("scale", -1.0), BAD, "scale"),
    (lambda c: c.mask.__setattr__("scale", math.nan), BAD, "scale"),
    (lambda c: c.mask.__setattr__("num_seqs", -1), BAD, "num_seqs"),
    (lambda c: c.mask.__setattr__("num_seqs", 1), BAD, "q_offsets"),
    (lambda c: c.mask.__setattr__("k_offsets", PAGE), BAD, "q_offsets"),
    (lambda c: (c.mask.__setattr__("num_seqs", 1), c.mask.__setattr__("q_offsets", PAGE)), SHAPE, "without k_offsets"),
    (lambda c: (c.mask.__setattr__("num_seqs", 1), c.mask.__setattr__("q_offsets", PAGE + 2)), NO, "4-byte"),
    (lambda c: c.V.__setitem__(1, _mat(5, 6, 128)), SHAPE, "V[1]"),
    (lambda c: c.K.__setitem__(1, _mat(3, 7, 128, fo.FO_F32)), BAD, "K[1]"),
    (lambda c: c.O.__setitem__(0, _mat(6, 5, 256, offset=8)), NO, "aligned"),
    (lambda c: c.LSE.__setitem__(0, _mat(8, 5, 4, fo.FO_F32)), SHAPE, "LSE[0]"),
    (lambda c: c.LSE.__setitem__(0, _mat(8, 4, 5)), BAD, "LSE[0]"),
])
def test_attention_refusals(lib, change, want, text):
    for run in (Attn.forward, Attn.backward):
        c = Attn()
        change(c)
        _refused(run(c), want, text)


def test_attention_refuses_bad_options(lib):
    c = Attn()
    o = fo.opts()
    o.order = 7
    st = fo.load().fo_attn_forward(NULL, c.Q, c.K, c.V, c.P, c.heads, c.kv, c.dim, ctypes.byref(c.mask), c.O, c.LSE,
                                   ctypes.byref(o), NULL)
    _refused(st, BAD, "order")


def test_attention_outputs_may_not_overlap(lib):
    c = Attn()
    c.O[1] = c.Q[0]
    _refused(c.forward(), BAD, "O[1] overlaps Q[0]")
    c = Attn()
    c.dQ = c.Q
    _refused(c.backward(), BAD, "dQ[0] overlaps Q[0]")
    c = Attn()
    c.dV = c.dK
    _refused(c.backward(), BAD, "overlaps")
    c = Attn()
    c.dK[0] = _mat(15, 9, 128)
    _refused(c.backward(), SHAPE, "dK[0]")
    # Q, K, V and their gradients as columns of one matrix each
    c = Attn()
    c.P = 1
    c.K, c.V = _arr(_mat(2, 5, 128)), _arr(_mat(2, 5, 128))
    for name, slot in (("", 0), ("d", 12)):
        for part, at, cols in (("Q", 0, 256), ("K", 256, 128), ("V", 384, 128)):
            setattr(c, name + part, _arr(_mat(slot, 5, cols, ld=512, offset=2 * at)))
    _refused(c.backward(), BAD, "null context")


# -- rotary positions ------------------------------------------------------------------------
def _rope(X=None, Y=None, P=1, table=None, head_dim=16, layout=0, positions=None):
    table = fo.RopeTable(8).c if table is None else table
    X = _arr(_mat(0, 4, 48)) if X is None else X
    Y = _arr(_mat(1, 4, 48)) if Y is None else Y
    return fo.load().fo_rope(NULL, X, P, ctypes.byref(table), head_dim, layout, positions, 0, 0, Y, NULL)


def test_rope_refusals(lib):
    bad, shape, no = fo.FO_ERR_INVALID_ARG, fo.FO_ERR_SHAPE, fo.FO_ERR_UNSUPPORTED
    _refused(_rope(), bad, "null context")
    same = _arr(_mat(0, 4, 48))
    _refused(_rope(X=same, Y=same), bad, "null context")  # in place
    _refused(_rope(table=fo.FoRopeTable()), bad, "not initialised")
    _refused(_rope(head_dim=6), shape, "below the table")
    _refused(_rope(head_dim=20), shape, "whole number of heads")
    _refused(_rope(layout=2), bad, "layout")
    _refused(_rope(P=0), bad, "P=0")
    _refused(_rope(Y=_arr(_mat(1, 5, 48))), shape, "one shape")
    _refused(_rope(Y=_arr(_mat(1, 4, 48, fo.FO_F32))), bad, "dtype")
    _refused(_rope(Y=_arr(_mat(0, 4, 48, offset=16))), bad, "overlaps")
    _refused(_rope(X=_arr(_mat(0, 4, 48, offset=2))), no, "aligned")
    _refused(_rope(positions=(ctypes.c_void_p * 1)(None)), bad, "positions[0]")
    _refused(_rope(positions=(ctypes.c_void_p * 1)(PAGE + 2)), no, "4-byte")
    two = _arr(_mat(1, 4, 48), _mat(1, 4, 48))
    _refused(_rope(X=_arr(_mat(0, 4, 48), _mat(2, 4, 48)), Y=two, P=2), bad, "overlaps Y[1]")
    st = fo.load().fo_rope_backward(NULL, None, 1, ctypes.byref(fo.RopeTable(8).c), 16, 0, None, 0, 0, same, NULL)
    _refused(st, bad, "null matrix")


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=514), dict(base=1.0),
                                dict(base=math.inf), dict(scaling="linear", factor=0.0),
                                dict(scaling="banded", factor=8.0), dict(scaling="banded", factor=8.0, original_length=8,
                                                                         low_factor=4.0, high_factor=4.0),
                                dict(scaling="ramped", factor=math.nan, original_length=8)])
def test_rope_table_refusals(lib, kw):
    with pytest.raises(fo.FoError) as e:
        fo.RopeTable(kw.pop("rot_dim", 64), **kw)
    assert e.value.status in (fo.FO_ERR_INVALID_ARG, fo.FO_ERR_UNSUPPORTED)


@pytest.mark.parametrize("kw,how", [
    (dict(), dict()),
    (dict(scaling="linear", factor=4.0), dict(scaling="linear", factor=4.0)),
    (dict(scaling="banded", factor=8.0, original_length=8192),
     dict(scaling="banded", factor=8.0, low=1.0, high=4.0, length=8192)),
    (dict(scaling="ramped", factor=16.0, original_length=4096),
     dict(scaling="ramped", factor=16.0, low=1.0, high=32.0, length=4096)),
    (dict(scaling="linear", factor=0.05), dict(scaling="linear", factor=0.05)),  # more than a turn per position
])
@pytest.mark.parametrize("rot,base", [(128, 10000.0), (64, 500000.0), (2, 10000.0), (512, 100.0)])
def test_rope_table_frequencies(lib, kw, how, rot, base):
    t = fo.RopeTable(rot, base=base, **kw)
    freq, amp = tr.rope_frequencies(rot, base, **how)
    assert t.rot_dim == rot and t.c.amplitude == np.float32(amp)
    got = np.array([t.c.turns[i] for i in range(rot // 2)], np.float64) / 2.0 ** 64
    want = freq / (2 * math.pi)
    want -= np.floor(want)
    # a few roundings in 64 bits (pow: 1 ulp; a frequency above one turn loses its whole turns' bits)
    assert np.abs(got - want).max() <= 16 * 2.0 ** -53 * max(1.0, freq.max())


def test_views_whose_rows_share_memory(lib):
    """An expanded gradient (the gradient of a sum, say) has rows 0 elements apart: read as if its rows lay one
    behind another, it would be read past its end."""
    torch = pytest.importorskip("torch")
    here = types.SimpleNamespace(device=-1)  # what get_device() says of the host
    for t in (torch.zeros(1, 16).expand(4, 16), torch.zeros(64).as_strided((4, 16), (8, 1)),
              torch.zeros(1, 4, 4).expand(4, 4, 4)):
        with pytest.raises(ValueError, match="share memory"):
            fo.mat(t)
        with pytest.raises(ValueError, match="share memory"):
            fo.Context._list(here, [t], 1, "dO")
    for t in (torch.zeros(1, 16), torch.zeros(64).as_strided((1, 16), (0, 1)), torch.zeros(0, 16),
              torch.zeros(4, 24)[:, :16]):
        m = fo.Context._list(here, [t], 1, "dO")[0]
        assert (m.ptr or 0, m.rows, m.cols) == (t.data_ptr(), *t.shape)
        assert m.ld == (24 if t.shape[0] == 4 else 16)

"""Refusals of the losses' and the optimizer's entry points, without a GPU: every argument is checked
before the context is, so a null context reaches the checks and is refused last."""
import ctypes
import math
import types

import pytest

import overlapped_tensor_gemm_gb300 as fo
from test_training_refusals import NULL, PAGE, _arr, _mat, _refused, lib  # noqa: F401

BAD, SHAPE, NO = fo.FO_ERR_INVALID_ARG, fo.FO_ERR_SHAPE, fo.FO_ERR_UNSUPPORTED


def _at(slot, offset=0):
    return (slot + 1) * PAGE + offset


class Loss:
    """A valid call (6 rows, 24 + 17 columns, P = 2) whose parts a test replaces."""

    def __init__(self):
        two = lambda slot, dt=fo.FO_BF16: _arr(_mat(slot, 6, 24, dt), _mat(slot + 1, 6, 17, dt))  # noqa: E731
        self.z, self.d, self.P = two(0), two(2, fo.FO_F32), 2
        self.y, self.logp, self.lse, self.ent, self.a, self.h = (_at(s) for s in range(4, 10))
        self.old, self.adv, self.ref, self.w, self.stats, self.off, self.margins = (_at(s) for s in range(10, 17))
        self.scale, self.pairs = 1.0, 2
        self.policy = fo.FoPolicyParams(1.0, 0.2, 0.2, 0.1, 0.0, 1)
        self.pref = fo.FoPreferenceParams(0, 0, 1.0, 0.1, 0.0, 0.0)

    def logprobs(self):
        return fo.load().fo_token_logprobs(NULL, self.z, self.P, self.y, self.scale, self.logp, self.lse, self.ent, NULL)

    def backward(self):
        return fo.load().fo_token_logprobs_backward(NULL, self.z, self.P, self.y, self.scale, self.lse, self.ent,
                                                    self.a, self.h, self.d, NULL)

    def policy_loss(self):
        self.policy.scale = self.scale if self.policy.scale == 1.0 else self.policy.scale
        return fo.load().fo_policy_loss(NULL, self.z, self.P, self.y, self.old, self.adv, self.ref, self.w,
                                        ctypes.byref(self.policy), self.logp, self.stats, self.d, NULL)

    def preference_loss(self):
        self.pref.scale = self.scale if self.pref.scale == 1.0 else self.pref.scale
        return fo.load().fo_preference_loss(NULL, self.z, self.P, self.y, self.off, self.pairs, self.ref,
                                            ctypes.byref(self.pref), self.logp, self.margins, self.stats, self.d, NULL)


ALL = (Loss.logprobs, Loss.backward, Loss.policy_loss, Loss.preference_loss)
GRAD = ALL[1:]


@pytest.mark.parametrize("change,want,text", [
    (lambda c: None, BAD, "null context"),
    (lambda c: setattr(c, "P", 0), BAD, "P=0"),
    (lambda c: setattr(c, "P", 9), BAD, "P=9"),
    (lambda c: setattr(c, "z", None), BAD, "null matrix"),
    (lambda c: setattr(c, "y", None), BAD, "targets: null"),
    (lambda c: setattr(c, "y", PAGE * 5 + 2), NO, "4-byte"),
    (lambda c: setattr(c, "scale", 0.0), BAD, "scale"),
    (lambda c: setattr(c, "scale", -1.0), BAD, "scale"),
    (lambda c: setattr(c, "scale", math.nan), BAD, "scale"),
    (lambda c: setattr(c, "scale", math.inf), BAD, "scale"),
    (lambda c: c.z.__setitem__(0, _mat(0, 6, 24, 7)), BAD, "logits[0]"),
    (lambda c: c.z.__setitem__(1, _mat(1, 6, 17, fo.FO_F32)), BAD, "logits[1]"),
    (lambda c: c.z.__setitem__(1, _mat(1, 5, 17)), SHAPE, "logits[1]"),
    (lambda c: c.z.__setitem__(1, _mat(1, 6, 17, ld=17)), NO, "pitch"),
    (lambda c: c.z.__setitem__(1, _mat(1, 6, 17, offset=8)), NO, "aligned"),
    (lambda c: setattr(c, "z", _arr(_mat(0, 6, 0, ld=8), _mat(1, 6, 0, ld=8)))
     or setattr(c, "d", _arr(_mat(2, 6, 0, ld=8), _mat(3, 6, 0, ld=8))), SHAPE, "at least one entry"),
    (lambda c: setattr(c, "z", _arr(_mat(0, 6, 1 << 30), _mat(1, 6, 17)))
     or setattr(c, "d", _arr(_mat(2, 6, 1 << 30), _mat(3, 6, 17))), NO, "vocabulary"),
])
@pytest.mark.parametrize("call", ALL, ids=lambda f: f.__name__)
def test_what_every_loss_refuses(lib, call, change, want, text):  # noqa: F811
    c = Loss()
    change(c)
    _refused(call(c), want, text)


@pytest.mark.parametrize("change,want,text", [
    (lambda c: c.d.__setitem__(0, _mat(2, 6, 25, fo.FO_F32)), SHAPE, "dlogits[0]"),
    (lambda c: c.d.__setitem__(1, _mat(3, 6, 17)), BAD, "dlogits[1]"),
    (lambda c: c.d.__setitem__(0, _mat(2, 6, 24, 5)), BAD, "dlogits[0]"),
    (lambda c: setattr(c, "d", _arr(_mat(0, 6, 24), _mat(1, 6, 17))), BAD, "null context"),   # over the logits
    (lambda c: setattr(c, "d", _arr(_mat(0, 6, 24, offset=16), _mat(1, 6, 17))), BAD, "overlaps"),
    (lambda c: setattr(c, "d", _arr(_mat(1, 6, 24), _mat(0, 6, 17))), BAD, "overlaps"),
    (lambda c: setattr(c, "d", _arr(_mat(0, 6, 24, fo.FO_F32, ld=16 * 3), _mat(3, 6, 17, fo.FO_F32))), BAD, "overlaps"),
    (lambda c: setattr(c, "y", _at(2, 64)), BAD, "overlaps"),
])
@pytest.mark.parametrize("call", GRAD, ids=lambda f: f.__name__)
def test_what_gradients_refuse(lib, call, change, want, text):  # noqa: F811
    c = Loss()
    change(c)
    _refused(call(c), want, text)


@pytest.mark.parametrize("call,change,want,text", [
    (Loss.logprobs, lambda c: (setattr(c, "logp", None), setattr(c, "lse", None), setattr(c, "ent", None)), BAD,
     "no output"),
    (Loss.logprobs, lambda c: (setattr(c, "logp", None), setattr(c, "lse", None)), BAD, "null context"),
    (Loss.logprobs, lambda c: setattr(c, "lse", c.logp + 4), BAD, "overlaps"),
    (Loss.logprobs, lambda c: setattr(c, "lse", c.y), BAD, "overlaps targets"),
    (Loss.backward, lambda c: setattr(c, "d", None), BAD, "null matrix"),
    (Loss.backward, lambda c: setattr(c, "lse", None), BAD, "lse: null"),
    (Loss.backward, lambda c: setattr(c, "a", None), BAD, "dlogp: null"),
    (Loss.backward, lambda c: setattr(c, "ent", None), BAD, "entropy: null"),
    (Loss.backward, lambda c: (setattr(c, "ent", None), setattr(c, "h", None)), BAD, "null context"),
    (Loss.policy_loss, lambda c: setattr(c, "adv", None), BAD, "advantages: null"),
    (Loss.policy_loss, lambda c: setattr(c, "stats", None), BAD, "stats: null"),
    (Loss.policy_loss, lambda c: setattr(c, "stats", c.logp), BAD, "overlaps"),
    (Loss.policy_loss, lambda c: setattr(c, "logp", c.old), BAD, "overlaps old_logp"),
    (Loss.policy_loss, lambda c: setattr(c, "ref", None), BAD, "kl_coef needs ref_logp"),
    (Loss.policy_loss, lambda c: (setattr(c, "ref", None), setattr(c.policy, "kl_coef", 0.0)), BAD, "null context"),
    (Loss.policy_loss, lambda c: [setattr(c, x, None) for x in ("old", "w", "logp", "d")] and None, BAD, "null context"),
    (Loss.policy_loss, lambda c: setattr(c.policy, "clip_low", -0.1), BAD, "clip_low"),
    (Loss.policy_loss, lambda c: setattr(c.policy, "clip_low", 1.5), BAD, "clip_low"),
    (Loss.policy_loss, lambda c: setattr(c.policy, "clip_high", math.inf), BAD, "clip_high"),
    (Loss.policy_loss, lambda c: setattr(c.policy, "entropy_coef", math.nan), BAD, "entropy_coef"),
    (Loss.policy_loss, lambda c: setattr(c.policy, "mean", 2), BAD, "mean"),
    (Loss.preference_loss, lambda c: setattr(c, "off", None), BAD, "offsets: null"),
    (Loss.preference_loss, lambda c: setattr(c, "stats", None), BAD, "loss: null"),
    (Loss.preference_loss, lambda c: [setattr(c, x, None) for x in ("ref", "margins", "logp", "d")] and None, BAD,
     "null context"),
    (Loss.preference_loss, lambda c: setattr(c, "pairs", 0), BAD, "num_pairs=0"),
    (Loss.preference_loss, lambda c: setattr(c, "margins", c.off), BAD, "overlaps"),
    (Loss.preference_loss, lambda c: setattr(c.pref, "kind", 3), BAD, "unknown kind"),
    (Loss.preference_loss, lambda c: setattr(c.pref, "average", 2), BAD, "average"),
    (Loss.preference_loss, lambda c: setattr(c.pref, "beta", 0.0), BAD, "beta"),
    (Loss.preference_loss, lambda c: setattr(c.pref, "label_smoothing", 1.5), BAD, "label_smoothing"),
    (Loss.preference_loss, lambda c: setattr(c.pref, "margin", math.inf), BAD, "margin"),
])
def test_what_one_loss_refuses(lib, call, change, want, text):  # noqa: F811
    c = Loss()
    change(c)
    _refused(call(c), want, text)


def test_losses_of_no_rows_need_no_vectors(lib):  # noqa: F811
    c = Loss()
    c.z = _arr(_mat(0, 0, 24), _mat(1, 0, 17))
    c.d = _arr(_mat(2, 0, 24), _mat(3, 0, 17))
    c.y = c.logp = c.lse = c.ent = c.a = c.old = c.adv = c.w = None
    for call in ALL:
        _refused(call(c), BAD, "null context")


# -- AdamW -----------------------------------------------------------------------------------
def _tensor(slot=0, n=1000, eight=False, has_master=True, ptype=fo.FO_BF16, gtype=fo.FO_BF16, **more):
    at = dict(param=_at(slot), grad=_at(slot + 1), master=_at(slot + 2) if has_master else None, m=_at(slot + 3),
              v=_at(slot + 4), m_scale=_at(slot + 5) if eight else None, v_range=_at(slot + 6) if eight else None)
    at.update(more)
    return fo.FoAdamWTensor(*at.values(), n, ptype, gtype)


def _create(*ts, count=None):
    h = ctypes.c_void_p()
    arr = (fo.FoAdamWTensor * max(len(ts), 1))(*ts)
    return fo.load().fo_adamw_group_create(arr, len(ts) if count is None else count, ctypes.byref(h)), h


@pytest.mark.parametrize("tensor,want,text", [
    (_tensor(param=None), BAD, "param[0]: null"),
    (_tensor(gtype=7), BAD, "grad[0]: unknown"),
    (_tensor(ptype=5), BAD, "param[0]: unknown"),
    (_tensor(ptype=fo.FO_F32), BAD, "fp32 parameter has none"),
    (_tensor(param=_at(0, 8)), NO, "aligned"),
    (_tensor(m=_at(3, 4)), NO, "m[0]"),
    (_tensor(eight=True, v_range=_at(6, 4)), NO, "v_range[0]"),
    (_tensor(eight=True, v_range=None), BAD, "go together"),
    (_tensor(n=-1), SHAPE, "negative"),
    (_tensor(v=_at(3)), BAD, "overlaps"),
    (_tensor(master=_at(0, 1984)), BAD, "overlaps"),      # 1000 bf16 end at 2000
    (_tensor(grad=_at(3, 3984)), BAD, "overlaps"),
    (_tensor(eight=True, m_scale=_at(4, 996)), BAD, "overlaps"),
], ids=range(13))
def test_group_refusals(lib, tensor, want, text):  # noqa: F811
    st, h = _create(tensor)
    _refused(st, want, text)
    assert not h.value


def test_group_refuses_counts_and_tensors_that_meet(lib):  # noqa: F811
    _refused(_create(_tensor(), count=-1)[0], BAD, "null tensor array")
    assert fo.load().fo_adamw_group_create(None, 0, None) == BAD
    _refused(_create(_tensor(0), _tensor(8), _tensor(0, m=_at(20), v=_at(21), master=_at(22)))[0], BAD, "overlaps")


def test_groups_of_nothing_and_of_shared_gradients(lib):  # noqa: F811
    for ts in ((), (_tensor(n=0, param=None),), (_tensor(0), _tensor(8, grad=_at(1))),
               tuple(_tensor(8 * i, eight=i % 2 == 0) for i in range(900))):
        st, h = _create(*ts)
        assert st == fo.FO_OK and h.value, fo.load().fo_last_error_string()
        assert fo.load().fo_adamw_group_destroy(h) == fo.FO_OK
    assert fo.load().fo_adamw_group_destroy(None) == fo.FO_OK


@pytest.mark.parametrize("change,want,text", [
    (dict(), BAD, "null context"),
    (dict(beta1=1.0), BAD, "beta1"),
    (dict(beta2=-0.1), BAD, "beta2"),
    (dict(eps=-1.0), BAD, "eps"),
    (dict(lr=math.nan), BAD, "lr"),
    (dict(lr=math.nan, lr_dev=_at(40)), BAD, "null context"),
    (dict(weight_decay=math.inf), BAD, "weight_decay"),
    (dict(step=0), BAD, "step=0"),
    (dict(step=0, step_dev=_at(40)), BAD, "null context"),
    (dict(step_dev=PAGE + 1), NO, "step_dev"),
    (dict(max_norm=1.0), BAD, "max_norm needs norm"),
    (dict(max_norm=1.0, norm=_at(40)), BAD, "null context"),
    (dict(norm=_at(0)), BAD, "norm overlaps param[0]"),
    (dict(lr_dev=_at(3, 3996)), BAD, "lr_dev overlaps m[0]"),
    (dict(lr_dev=_at(3, 4000)), BAD, "null context"),
    (dict(step_dev=_at(4)), BAD, "step_dev overlaps v[0]"),
    (dict(norm=_at(1)), BAD, "null context"),  # (a step only reads its gradients)
    (dict(stochastic=2), BAD, "stochastic"),
])
def test_step_refusals(lib, change, want, text):  # noqa: F811
    st, h = _create(_tensor())
    assert st == fo.FO_OK
    how = dict(beta1=0.9, beta2=0.999, lr=0.1, eps=1e-8, weight_decay=0.0, grad_scale=1.0, max_norm=0.0, stochastic=0,
               step=1, seed=0, lr_dev=None, step_dev=None, norm=None)
    how.update(change)
    _refused(fo.load().fo_adamw_step(NULL, h, ctypes.byref(fo.FoAdamWParams(**how)), NULL), want, text)
    fo.load().fo_adamw_group_destroy(h)


def test_norm_and_unpack_refusals(lib):  # noqa: F811
    st, h = _create(_tensor(eight=True), _tensor(8))
    f = fo.load()
    _refused(f.fo_grad_norm(NULL, None, PAGE, NULL), BAD, "null group")
    _refused(f.fo_grad_norm(NULL, h, None, NULL), BAD, "norm[0]: null")
    _refused(f.fo_grad_norm(NULL, h, _at(40), NULL), BAD, "null context")
    _refused(f.fo_grad_norm(NULL, h, _at(1, 1996), NULL), BAD, "norm overlaps grad[0]")
    _refused(f.fo_grad_norm(NULL, h, _at(12), NULL), BAD, "norm overlaps v[1]")
    _refused(f.fo_adamw_step(NULL, None, None, NULL), BAD, "null group")
    _refused(f.fo_adamw_step(NULL, h, None, NULL), BAD, "null parameters")
    ptr = lambda *a: (ctypes.c_void_p * 2)(*a)  # noqa: E731
    good, good_v, none = ptr(_at(40), None), ptr(_at(41), None), ptr(None, None)
    _refused(f.fo_adamw_unpack(NULL, h, good, good_v, 0, NULL), BAD, "null context")
    _refused(f.fo_adamw_unpack(NULL, h, good, good, 0, NULL), BAD, "overlaps")
    _refused(f.fo_adamw_unpack(NULL, h, good, ptr(_at(40, 2000), None), 0, NULL), BAD, "null context")
    _refused(f.fo_adamw_unpack(NULL, h, good, ptr(_at(40, 2000), None), 1, NULL), BAD, "v[0] overlaps m[0]")
    _refused(f.fo_adamw_unpack(NULL, h, good, ptr(_at(4, 16), None), 0, NULL), BAD, "v[0] overlaps the group's v[0]")
    _refused(f.fo_adamw_unpack(NULL, h, good, none, 0, NULL), BAD, "v[0]: null")
    _refused(f.fo_adamw_unpack(NULL, h, ptr(PAGE + 8, None), good, 1, NULL), NO, "m[0]")
    _refused(f.fo_adamw_unpack(NULL, h, good, good, 2, NULL), BAD, "dtype")
    f.fo_adamw_group_destroy(h)


# -- what the binding itself refuses ------------------------------------------------------------
def test_binding_refuses_what_it_cannot_marshal(lib):  # noqa: F811
    torch = pytest.importorskip("torch")
    ctx = types.SimpleNamespace(device=0)
    for name in ("_here", "_entries"):
        setattr(ctx, name, getattr(fo.Context, name).__get__(ctx))
    v = torch.zeros(4)
    with pytest.raises(ValueError, match="context on cuda:0"):
        ctx._entries(v, "logp", 4)
    assert ctx._entries(None, "logp", 4) is None
    with pytest.raises(ValueError, match="on one GPU"):
        fo.AdamWTensors([v], [v], [v], [v])
    with pytest.raises(ValueError, match="2 tensors for 1"):
        fo.AdamWTensors([v], [v, v], [v], [v])
    with pytest.raises(ValueError, match="m\\[0\\] is missing"):
        fo.AdamWTensors([v.cuda() if torch.cuda.is_available() else _Fake(v)],
                        [v.cuda() if torch.cuda.is_available() else _Fake(v)], [None], [v])
    with pytest.raises(ValueError, match="8 or 32"):
        fo.adamw_states([v], 16)
    m, s, scale, rng = fo.adamw_states([torch.zeros(3, 300)], 8)
    assert m[0].dtype == torch.float8_e4m3fn and m[0].shape == (3, 300) and s[0].dtype == torch.uint8
    assert scale[0].shape == (4,) and rng[0].shape == (8,)


class _Fake:
    """A tensor that says it is on cuda:0."""

    def __init__(self, t):
        self._t = t
        self.device = types.SimpleNamespace(type="cuda", index=0)

    def __getattr__(self, name):
        return getattr(self._t, name)


def test_struct_layouts_match_the_headers():
    assert ctypes.sizeof(fo.FoPolicyParams) == 24
    assert ctypes.sizeof(fo.FoPreferenceParams) == 24
    assert ctypes.sizeof(fo.FoAdamWTensor) == 8 * 8 + 2 * 4
    assert ctypes.sizeof(fo.FoAdamWParams) == 2 * 8 + 6 * 4 + 2 * 8 + 3 * 8

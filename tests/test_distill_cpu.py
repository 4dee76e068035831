"""The oracle of the distillation loss against torch's autograd and differences, and the host-side
argument checks of kron_topk_logits and the kron_distill calls (CPU only: nothing is launched)."""
import ctypes

import numpy as np
import pytest

from kronecker_factored_structured_amd import _lib
from oracle import distill as OD

BASE = 0x7f0000000000
MB = 1 << 20


def P(off=0):
    return ctypes.c_void_p(BASE + off)


def _case(seed, N=5, V=23, k=6, tail=False, T=1.7):
    g = np.random.default_rng(seed)
    z = g.standard_normal((N, V)) * 2
    ids = np.stack([g.permutation(V)[:k] for _ in range(N)])
    t = np.sort(g.standard_normal((N, k)) * 2, 1)[:, ::-1].copy()
    lse = np.log(np.exp(t / T).sum(1)) + 0.2 if tail else None
    return z, ids, t, lse, g.integers(0, V, N), g.uniform(0.1, 1, N)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("alpha", [0.0, 0.4, 1.0])
def test_oracle_matches_autograd(tail, alpha):
    torch = pytest.importorskip("torch")
    T = 1.7
    z, ids, t, lse, lab, w = _case(1, tail=tail, T=T)
    zt = torch.from_numpy(z).requires_grad_()
    lq = torch.log_softmax(zt / T, 1)
    if tail:
        p = torch.exp(torch.from_numpy(t) / T - torch.from_numpy(lse)[:, None])
        pt, mask = 1 - p.sum(1), torch.zeros_like(zt).scatter(1, torch.from_numpy(ids), 1.0)
        qt = (lq.exp() * (1 - mask)).sum(1)
        kd = (p * (p.log() - lq.gather(1, torch.from_numpy(ids)))).sum(1) + pt * (pt.log() - qt.log())
    else:
        p = torch.softmax(torch.from_numpy(t) / T, 1)
        kd = torch.nn.functional.kl_div(lq.gather(1, torch.from_numpy(ids)), p, reduction="none").sum(1)
    ce = torch.nn.functional.cross_entropy(zt, torch.from_numpy(lab), reduction="none")
    loss = (torch.from_numpy(w) * (alpha * T * T * kd + (1 - alpha) * ce)).sum()
    loss.backward()
    got, dz, _, _ = OD.loss_and_grad(z, ids, t, lse, lab, w, T, alpha)
    assert abs(got - loss.item()) <= 1e-12 * max(1, abs(got))
    assert np.abs(dz - zt.grad.numpy()).max() <= 1e-13


def test_oracle_matches_differences():
    z, ids, t, lse, lab, w = _case(2, tail=True)
    ids[0, 3] = ids[0, 1]          # a token given twice
    ids[1, 2] = -1                 # an unused slot
    f = lambda y: OD.loss_and_grad(y, ids, t, lse, lab, w, 1.7, 0.6)[0]
    dz = OD.loss_and_grad(z, ids, t, lse, lab, w, 1.7, 0.6)[1]
    for n, v in ((0, ids[0, 1]), (0, ids[0, 0]), (1, ids[1, 0]), (2, 4), (4, 20)):
        e = np.zeros_like(z)
        e[n, v] = 1e-5
        assert abs((f(z + e) - f(z - e)) / 2e-5 - dz[n, v]) <= 1e-9


def test_oracle_topk_order():
    z = np.array([[1.0, 3.0, 3.0, -np.inf, 2.0, 3.0]])
    ids, vals, lse = OD.topk(z, 4, 1.0)
    assert ids.tolist() == [[1, 2, 5, 4]] and vals.tolist() == [[3.0, 3.0, 3.0, 2.0]]
    assert abs(lse[0] - np.log(np.exp(1) + 3 * np.exp(3) + np.exp(2))) < 1e-14


def topk(N=8, V=1000, ld=1000, k=10, dt=0, T=1.0, z=P(0), ids=P(64 * MB), vals=P(65 * MB), lse=P(66 * MB)):
    return _lib.lib().kron_topk_logits(N, V, ld, k, dt, T, z, ids, vals, lse, None)


def test_topk_argument_errors():
    assert topk(N=0, z=None, ids=None, vals=None, lse=None) == 0
    assert topk(N=-1) == _lib.KRON_E_SHAPE
    assert topk(V=0) == _lib.KRON_E_SHAPE
    assert topk(k=0) == _lib.KRON_E_SHAPE
    assert topk(V=9, ld=9) == _lib.KRON_E_SHAPE                      # k > V
    assert topk(ld=999) == _lib.KRON_E_SHAPE
    assert topk(ld=1 << 62) == _lib.KRON_E_SHAPE
    assert topk(k=257) == _lib.KRON_E_UNSUPPORTED
    assert topk(V=262145, ld=262145) == _lib.KRON_E_UNSUPPORTED
    assert topk(dt=7) == _lib.KRON_E_DTYPE
    for T in (0.0, -1.0, float("nan"), float("inf")):
        assert topk(T=T) == _lib.KRON_E_ARG
    assert topk(z=None) == _lib.KRON_E_NULL
    assert topk(lse=None) == _lib.KRON_E_NULL
    assert topk(z=P(2)) == _lib.KRON_E_ALIGN                          # fp32 at two bytes
    assert topk(ids=P(64 * MB + 4)) == _lib.KRON_E_ALIGN
    assert topk(ids=P(16)) == _lib.KRON_E_ALIAS                       # ids in the logits
    assert topk(vals=P(64 * MB + 16)) == _lib.KRON_E_ALIAS            # vals over ids


def distill(mode=0, null=(), **kw):
    d = _lib.KronDistill(8, 1000, 10, 1000, 1008, 0, 0, 2.0, 0.5)
    a = dict(z=P(0), ids=P(64 * MB), t=P(65 * MB), tl=P(66 * MB), lab=P(67 * MB), w=P(68 * MB), loss=P(69 * MB),
             stats=P(70 * MB), gout=P(71 * MB), dz=P(128 * MB), ws=P(72 * MB), nb=None)
    for k, v in kw.items():
        if k in a:
            a[k] = v
        else:
            setattr(d, k, v)
    for k in null:
        a[k] = None
    L = _lib.lib()
    if a["nb"] is None:
        a["nb"] = L.kron_distill_workspace_bytes(ctypes.byref(d))
    common = (ctypes.byref(d), a["z"], a["ids"], a["t"], a["tl"], a["lab"], a["w"])
    if mode == 0:
        return L.kron_distill(*common, a["loss"], a["dz"], a["ws"], ctypes.c_size_t(a["nb"]), None)
    if mode == 1:
        return L.kron_distill_fwd(*common, a["loss"], a["stats"], a["ws"], ctypes.c_size_t(a["nb"]), None)
    return L.kron_distill_bwd(*common, a["stats"], a["gout"], a["dz"], None)


def test_distill_workspace():
    d = _lib.KronDistill(1000, 500, 10, 500, 500, 1, 0, 1.0, 1.0)
    nb = _lib.lib().kron_distill_workspace_bytes(ctypes.byref(d))
    assert nb >= 4000 and nb % 256 == 0
    d.V = 0
    assert _lib.lib().kron_distill_workspace_bytes(ctypes.byref(d)) == 0
    assert _lib.lib().kron_distill_workspace_bytes(None) == 0


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_distill_argument_errors(mode):
    E = _lib
    for kw, want in ((dict(N=-1), E.KRON_E_SHAPE), (dict(V=0), E.KRON_E_SHAPE), (dict(k=-1), E.KRON_E_SHAPE),
                     (dict(k=0), E.KRON_E_SHAPE), (dict(k=257), E.KRON_E_UNSUPPORTED),
                     (dict(V=262145, ld=262145, ldd=262145), E.KRON_E_UNSUPPORTED), (dict(ld=999), E.KRON_E_SHAPE),
                     (dict(ld=1 << 62), E.KRON_E_SHAPE),
                     (dict(dtype=3), E.KRON_E_DTYPE), (dict(flags=2), E.KRON_E_ARG),
                     (dict(temperature=0.0), E.KRON_E_ARG), (dict(temperature=float("nan")), E.KRON_E_ARG),
                     (dict(alpha=-0.1), E.KRON_E_ARG), (dict(alpha=1.1), E.KRON_E_ARG),
                     (dict(alpha=float("nan")), E.KRON_E_ARG),
                     (dict(null=("z",)), E.KRON_E_NULL), (dict(null=("ids",)), E.KRON_E_NULL),
                     (dict(null=("t",)), E.KRON_E_NULL), (dict(null=("lab",)), E.KRON_E_NULL),
                     (dict(z=P(2)), E.KRON_E_ALIGN), (dict(t=P(65 * MB + 4)), E.KRON_E_ALIGN)):
        assert distill(mode, **kw) == want, kw
    if mode != 1:
        assert distill(mode, ldd=999) == E.KRON_E_SHAPE
        assert distill(mode, null=("dz",)) == E.KRON_E_NULL
        assert distill(mode, dz=P(16)) == E.KRON_E_ALIAS              # shifted over the logits
        assert distill(mode, dz=P(0)) == E.KRON_E_ALIAS               # the logits, but another row stride
        assert distill(mode, dz=P(65 * MB)) == E.KRON_E_ALIAS         # over the teacher
    if mode != 2:
        assert distill(mode, null=("loss",)) == E.KRON_E_NULL
        assert distill(mode, null=("ws",)) == E.KRON_E_WORKSPACE
        assert distill(mode, nb=100) == E.KRON_E_WORKSPACE
        assert distill(mode, ws=P(72 * MB + 64)) == E.KRON_E_ALIGN
        assert distill(mode, loss=P(32)) == E.KRON_E_ALIAS
    if mode == 1:
        assert distill(mode, null=("stats",)) == E.KRON_E_NULL
        assert distill(mode, stats=P(68 * MB)) == E.KRON_E_ALIAS
    if mode == 2:
        assert distill(mode, null=("stats",)) == E.KRON_E_NULL
        assert distill(mode, null=("gout",)) == E.KRON_E_NULL
        assert distill(mode, N=0, null=("z", "ids", "t", "tl", "lab", "w", "stats", "dz")) == 0


def test_binding_refuses():
    torch = pytest.importorskip("torch")
    import kronecker_factored_structured_amd as K
    z = torch.zeros(3, 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        K.kron_topk_logits(z, 2)
    with pytest.raises(ValueError, match="unsupported dtype"):
        K.kron_topk_logits(z.double(), 2)
    with pytest.raises(ValueError, match="GPU tensor"):
        K.kron_distill(z, torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2))


def test_temperature_whose_reciprocal_overflows():
    """The kernels scale by log2(e) / T: below 4.3e-39 that is infinite, and 0 times it NaN."""
    for T in (1e-45, 1e-39, 4.2e-39):
        assert topk(T=T) == _lib.KRON_E_ARG
        for mode in (0, 1, 2):
            assert distill(mode, temperature=T) == _lib.KRON_E_ARG

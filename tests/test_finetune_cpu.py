"""The oracles of the vocabulary cross-entropy, the adapters and the orthogonalised update against torch's autograd,
differences and the singular values, and the host-side argument checks of their entry points (CPU only: nothing is
launched)."""
import ctypes

import numpy as np
import pytest

from kronecker_factored_structured_amd import _lib
from oracle import adapters as OA
from oracle import muon as OM
from oracle import vocab_ce as OV

BASE = 0x7f0000000000
MB = 1 << 20


def P(off=0):
    return ctypes.c_void_p(BASE + off)


def L():
    return _lib.lib()


# ------------------------------------------------------------------------------------------ oracles
def test_vocab_oracle_matches_autograd():
    torch = pytest.importorskip("torch")
    g = np.random.default_rng(0)
    h, W = g.standard_normal((9, 6)), g.standard_normal((13, 6))
    lab, w = g.integers(0, 13, 9), g.uniform(0.1, 1, 9)
    w[[2, 5]] = 0
    ht, Wt = torch.from_numpy(h).requires_grad_(), torch.from_numpy(W).requires_grad_()
    nll = torch.nn.functional.cross_entropy(ht @ Wt.T, torch.from_numpy(lab), reduction="none")
    loss = (torch.from_numpy(w) * nll).sum()
    (1.5 * loss).backward()
    o = OV.forward_backward(h, W, lab, w, gout=1.5)
    assert abs(o["loss"] - loss.item()) < 1e-12
    assert np.abs(o["dh"] - ht.grad.numpy()).max() < 1e-13 and np.abs(o["dW"] - Wt.grad.numpy()).max() < 1e-13
    assert np.all(o["nll"][[2, 5]] == 0)


def test_vocab_oracle_matches_differences():
    g = np.random.default_rng(1)
    h, W, lab = g.standard_normal((4, 3)), g.standard_normal((5, 3)), np.array([0, 4, 2, 2])
    o = OV.forward_backward(h, W, lab)
    for arr, grad in ((h, o["dh"]), (W, o["dW"])):
        for i in np.ndindex(arr.shape):
            keep, d = arr[i], 1e-5
            arr[i] = keep + d
            hi = OV.forward_backward(h, W, lab)["loss"]
            arr[i] = keep - d
            lo = OV.forward_backward(h, W, lab)["loss"]
            arr[i] = keep
            assert abs((hi - lo) / (2 * d) - grad[i]) < 1e-9


def test_adapters_oracle_matches_differences():
    g = np.random.default_rng(2)
    N, K, M, R, E = 7, 4, 3, 2, 3
    x, base, dy = g.standard_normal((N, K)), g.standard_normal((N, M)), g.standard_normal((N, M))
    D, U, s = g.standard_normal((E, R, K)), g.standard_normal((E, M, R)), g.uniform(0.5, 2, E)
    starts, ids = np.array([1, 3, 3, 6]), np.array([2, 0, 2])
    f = lambda: (dy * OA.forward(x, base, D, U, ids, starts, s)[0]).sum()
    o = OA.backward(x, dy, D, U, ids, starts, s)[0]
    for arr, grad in ((x, o["dx"]), (D, o["ddown"]), (U, o["dup"])):
        for i in np.ndindex(arr.shape):
            keep, d = arr[i], 1e-5
            arr[i] = keep + d
            hi = f()
            arr[i] = keep - d
            lo = f()
            arr[i] = keep
            assert abs((hi - lo) / (2 * d) - grad[i]) < 1e-8
    y = OA.forward(x, base, D, U, ids, starts, s)[0]
    assert np.array_equal(y[[0, 6]], base[[0, 6]])      # rows of no request
    assert np.all(o["ddown"][[0, 1]] == 0) and np.all(o["dup"][1] == 0)      # adapters without rows


@pytest.mark.parametrize("shape", [(5, 9), (9, 5), (1, 7), (6, 6)])
def test_muon_oracle_acts_on_singular_values(shape):
    g = np.random.default_rng(3)
    u = g.standard_normal(shape)
    o = OM.orthogonalise(u)
    P_, v, Q = np.linalg.svd(u / (np.sqrt((u ** 2).sum()) + 1e-7), full_matrices=False)
    a, b, c = OM.COEFFS
    for _ in range(5):
        v = a * v + b * v ** 3 + c * v ** 5
    assert np.abs(o - (P_ * v) @ Q).max() < 1e-10
    assert np.all(v < 1.3)      # (how far up a small one comes depends on where it started)


# ------------------------------------------------------------------------------------------ refusals
def vocab_fwd(N=4, K=8, V=16, dtype=0, h=P(), W=P(MB), labels=P(2 * MB), weights=None, loss=P(3 * MB), nll=P(4 * MB),
              stats=P(5 * MB), ws=P(64 * MB), nbytes=64 * MB):
    return L().kron_vocab_ce_fwd(N, K, V, dtype, h, W, labels, weights, loss, nll, stats, ws, nbytes, None)


def vocab_bwd(N=4, K=8, V=16, dtype=0, h=P(), W=P(MB), labels=P(2 * MB), weights=None, stats=P(5 * MB), gout=P(3 * MB),
              dh=P(6 * MB), dW=P(7 * MB), ws=P(64 * MB), nbytes=64 * MB):
    return L().kron_vocab_ce_bwd(N, K, V, dtype, h, W, labels, weights, stats, gout, dh, dW, ws, nbytes, None)


@pytest.mark.parametrize("f", [vocab_fwd, vocab_bwd])
def test_vocab_refusals(f):
    need = L().kron_vocab_ce_workspace_bytes(4, 8, 16, 0, 0, int(f is vocab_bwd))
    assert 0 < need <= 64 * MB
    for kw, want in ((dict(N=-1), "SHAPE"), (dict(K=0), "SHAPE"), (dict(V=0), "SHAPE"),
                     (dict(N=_lib.KRON_VOCAB_CE_MAX_ROWS + 1), "UNSUPPORTED"),
                     (dict(K=_lib.KRON_VOCAB_CE_MAX_WIDTH + 1), "UNSUPPORTED"),
                     (dict(V=_lib.KRON_VOCAB_MAX + 1), "UNSUPPORTED"), (dict(dtype=2), "DTYPE"),
                     (dict(h=None), "NULL"), (dict(W=None), "NULL"), (dict(labels=None), "NULL"), (dict(stats=None), "NULL"),
                     (dict(ws=None), "WORKSPACE"), (dict(nbytes=need - 1), "WORKSPACE"), (dict(ws=P(64 * MB + 16)), "ALIGN"),
                     (dict(h=P(4)), "ALIGN"), (dict(labels=P(2 * MB + 8)), "ALIGN"), (dict(weights=P(8 * MB + 4)), "ALIGN"),
                     (dict(ws=P(MB)), "ALIAS"), (dict(ws=P()), "ALIAS")):
        assert f(**kw) == getattr(_lib, "KRON_E_" + want), (kw, _lib.last_error())
    if f is vocab_fwd:
        more = ((dict(loss=None), "NULL"), (dict(nll=None), "NULL"), (dict(nll=P()), "ALIAS"), (dict(loss=P(4 * MB)), "ALIAS"))
    else:
        more = ((dict(gout=None), "NULL"), (dict(dh=P()), "ALIAS"), (dict(dW=P(MB)), "ALIAS"), (dict(dW=P(6 * MB)), "ALIAS"))
    for kw, want in more:
        assert f(**kw) == getattr(_lib, "KRON_E_" + want), (kw, _lib.last_error())
    assert vocab_bwd(dh=None, dW=None) == _lib.KRON_OK      # nothing asked, nothing launched


def test_vocab_workspace():
    ws = L().kron_vocab_ce_workspace_bytes
    assert ws(-1, 8, 16, 0, 0, 0) == 0 and ws(1, 8, 16, 7, 0, 0) == 0 and ws(1, 8, _lib.KRON_VOCAB_MAX + 1, 0, 0, 0) == 0
    # the logits are never held: far below their size, forward and backward
    for dtype in (0, 1):
        logits = 65536 * 131072 * 4
        assert ws(65536, 768, 131072, dtype, 0, 0) < logits / 20
        assert ws(65536, 768, 131072, dtype, 1, 1) < logits / 10


def sizes(**kw):
    d = dict(N=8, K=16, M=12, R=4, E=3, B=2, dtype=0)
    d.update(kw)
    return _lib.KronAdapters(**d)


def ada_fwd(d=None, x=P(), base=P(MB), down=P(2 * MB), up=P(3 * MB), ids=P(4 * MB), starts=P(5 * MB), scales=None, y=P(6 * MB), **kw):
    return L().kron_adapters_fwd(None if d == 0 else ctypes.byref(sizes(**kw)), x, base, down, up, ids, starts, scales, y, None)


def ada_bwd(d=None, x=P(), dy=P(MB), down=P(2 * MB), up=P(3 * MB), ids=P(4 * MB), starts=P(5 * MB), scales=None, dx_base=None,
            dx=P(6 * MB), ddown=P(7 * MB), dup=P(8 * MB), ws=P(64 * MB), nbytes=MB, **kw):
    return L().kron_adapters_bwd(None if d == 0 else ctypes.byref(sizes(**kw)), x, dy, down, up, ids, starts, scales, dx_base, dx,
                                 ddown, dup, ws, nbytes, None)


@pytest.mark.parametrize("f", [ada_fwd, ada_bwd])
def test_adapters_refusals(f):
    for kw, want in ((dict(d=0), "NULL"), (dict(N=-1), "SHAPE"), (dict(B=-1), "SHAPE"), (dict(K=0), "SHAPE"), (dict(M=0), "SHAPE"),
                     (dict(R=0), "SHAPE"), (dict(E=0), "SHAPE"), (dict(R=129), "UNSUPPORTED"), (dict(E=65536), "UNSUPPORTED"),
                     (dict(K=65537), "UNSUPPORTED"), (dict(M=65537), "UNSUPPORTED"), (dict(N=(1 << 24) + 1), "UNSUPPORTED"),
                     (dict(B=(1 << 20) + 1), "UNSUPPORTED"), (dict(dtype=9), "DTYPE"), (dict(x=None), "NULL"),
                     (dict(down=None), "NULL"), (dict(up=None), "NULL"), (dict(ids=None), "NULL"),
                     (dict(starts=None), "SHAPE"),      # two requests of one row each, but eight rows
                     (dict(x=P(8)), "ALIGN"), (dict(ids=P(4 * MB + 2)), "ALIGN"), (dict(starts=P(5 * MB + 1)), "ALIGN"),
                     (dict(scales=P(9 * MB + 4)), "ALIGN")):
        assert f(**kw) == getattr(_lib, "KRON_E_" + want), (kw, _lib.last_error())
    if f is ada_fwd:
        more = ((dict(base=None), "NULL"), (dict(y=None), "NULL"), (dict(y=P()), "ALIAS"), (dict(y=P(MB + 16)), "ALIAS"),
                (dict(y=P(4 * MB)), "ALIAS"), (dict(y=P(5 * MB)), "ALIAS"), (dict(y=P(2 * MB)), "ALIAS"))
    else:
        more = ((dict(dy=None), "NULL"), (dict(ddown=None), "NULL"), (dict(dup=None), "NULL"), (dict(dx=None, dx_base=P(9 * MB)), "NULL"),
                (dict(ws=None), "WORKSPACE"), (dict(nbytes=16), "WORKSPACE"), (dict(ws=P(64 * MB + 16)), "ALIGN"), (dict(dx=P()), "ALIAS"),
                (dict(dx_base=P(6 * MB + 16)), "ALIAS"), (dict(ddown=P(6 * MB)), "ALIAS"), (dict(dup=P(3 * MB)), "ALIAS"))
    for kw, want in more:
        assert f(**kw) == getattr(_lib, "KRON_E_" + want), (kw, _lib.last_error())
    assert ada_fwd(N=0, B=0, starts=None, x=None, base=None, y=None, ids=None) == _lib.KRON_OK      # nothing launched


@pytest.mark.parametrize("f", [ada_fwd, ada_bwd])
def test_adapters_requests(f):
    """ids belong to the requests, not to the rows: none of them is read without rows either, and all are without ids."""
    for kw, want in ((dict(N=0, x=None, ids=None), "NULL"), (dict(N=0, B=5, ids=None), "NULL"),
                     (dict(B=_lib.KRON_ADAPTERS_MAX_REQUESTS + 1), "UNSUPPORTED")):
        assert f(**kw) == getattr(_lib, "KRON_E_" + want), (kw, _lib.last_error())
    assert ada_fwd(N=0, B=0, ids=None) == _lib.KRON_OK      # nothing launched
    # (a refusal that comes after ids': no request, no ids)
    assert f(B=0, ids=None, x=P(8)) == _lib.KRON_E_ALIGN


def test_muon_refuses_what_fp32_does_not_hold():
    for kw in (dict(eps=1e-60), dict(lr=1e60), dict(momentum=1e39), dict(weight_decay=1e300), dict(b=-1e39), dict(lr=1e30, weight_decay=1e30),
               dict(eps=1e39)):
        assert muon(**kw) == _lib.KRON_E_ARG, kw


def muon(tensors=((P(), P(MB), P(2 * MB), 2, 8, 4),), dtype=0, hyper=None, ws=P(64 * MB), nbytes=64 * MB, n=None, **kw):
    d = dict(lr=0.02, momentum=0.95, weight_decay=0.0, a=3.4445, b=-4.775, c=2.0315, eps=1e-7, nesterov=1, steps=5)
    d.update(kw)
    k = len(tensors)
    arr = ctypes.c_void_p * max(k, 1)
    cols = list(zip(*tensors)) or [()] * 6
    ptr = [arr(*[t.value if t else None for t in c]) for c in cols[:3]]
    ints = [(ctypes.c_int64 * max(k, 1))(*cols[3]), (ctypes.c_int32 * max(k, 1))(*cols[4]), (ctypes.c_int32 * max(k, 1))(*cols[5])]
    h = None if hyper == 0 else ctypes.byref(_lib.KronMuon(**d))
    return L().kron_muon_step(h, k if n is None else n, dtype, *ptr, *ints, None, ws, nbytes, None)


def test_muon_refusals():
    one = lambda p=P(), g=P(MB), m=P(2 * MB), c=2, r=8, k=4: ((p, g, m, c, r, k),)
    big = one(c=1, r=128, k=128)
    need = L().kron_muon_workspace_bytes(1, (ctypes.c_int64 * 1)(1), (ctypes.c_int32 * 1)(128), (ctypes.c_int32 * 1)(128), 0)
    assert need > 0
    assert L().kron_muon_workspace_bytes(1, (ctypes.c_int64 * 1)(7), (ctypes.c_int32 * 1)(32), (ctypes.c_int32 * 1)(64), 0) == 0
    for kw, want in ((dict(hyper=0), "NULL"), (dict(n=-1), "ARG"), (dict(n=4097), "ARG"), (dict(dtype=3), "DTYPE"),
                     (dict(tensors=one(p=None)), "NULL"), (dict(tensors=one(g=None)), "NULL"), (dict(tensors=one(m=None)), "NULL"),
                     (dict(tensors=one(c=-1)), "SHAPE"), (dict(tensors=one(r=0)), "SHAPE"), (dict(tensors=one(k=0)), "SHAPE"),
                     (dict(tensors=one(r=_lib.KRON_MUON_MAX_SIDE + 1)), "UNSUPPORTED"), (dict(tensors=one(c=(1 << 20) + 1)), "UNSUPPORTED"),
                     (dict(lr=float("nan")), "ARG"), (dict(momentum=-0.1), "ARG"), (dict(eps=0.0), "ARG"), (dict(steps=0), "ARG"),
                     (dict(steps=_lib.KRON_MUON_MAX_STEPS + 1), "ARG"), (dict(a=float("inf")), "ARG"),
                     (dict(tensors=one(p=P(4))), "ALIGN"), (dict(tensors=one(m=P(2 * MB + 8))), "ALIGN"),
                     (dict(tensors=big, ws=None), "WORKSPACE"), (dict(tensors=big, nbytes=need - 1), "WORKSPACE"),
                     (dict(tensors=big, ws=P(64 * MB + 128)), "ALIGN"), (dict(tensors=big, ws=P(MB)), "ALIAS"),
                     (dict(tensors=one(g=P())), "ALIAS"), (dict(tensors=one(m=P(128))), "ALIAS"),
                     # one tensor given twice, one's momentum in another's gradient
                     (dict(tensors=one() + one(g=P(3 * MB), m=P(4 * MB))), "ALIAS"),
                     (dict(tensors=one() + one(p=P(5 * MB), g=P(3 * MB), m=P(MB))), "ALIAS")):
        assert muon(**kw) == getattr(_lib, "KRON_E_" + want), (kw, _lib.last_error())
    assert muon(tensors=()) == _lib.KRON_OK and muon(tensors=one(p=None, c=0)) == _lib.KRON_OK

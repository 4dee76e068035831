"""The oracle of the gated block against torch's autograd, and the host-side argument checks of
kron_glu_fwd / kron_glu_bwd (CPU only: nothing is launched)."""
import ctypes

import numpy as np
import pytest

from kronecker_factored_structured_amd import _lib
from kronecker_factored_structured_amd._lib import KronShape
from oracle import glu as OG

BASE = 0x7f0000000000
MB = 1 << 20


def P(off=0):
    return ctypes.c_void_p(BASE + off)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("with_S", [False, True])
def test_oracle_matches_autograd(act, with_S):
    torch = pytest.importorskip("torch")
    g = np.random.default_rng(3)
    N, p, q, m, n, r = 6, 3, 5, 4, 2, 3
    t = lambda *s: torch.from_numpy(g.standard_normal(s)).requires_grad_()
    x, A, B, bias, S = t(N, p * m), t(2, r, p, q), t(2, r, m, n), t(2, q * n), t(2, p, q)
    z = []
    for f in range(2):
        C = A[f] * S[f] if with_S else A[f]
        W = sum(torch.kron(C[i], B[f, i]) for i in range(r))
        z.append(x @ W + bias[f])
    fn = torch.nn.functional
    a = dict(silu=fn.silu, gelu=fn.gelu, gelu_tanh=lambda v: fn.gelu(v, approximate="tanh"), relu=fn.relu)[act](z[0])
    y = a * z[1]
    dy = torch.from_numpy(g.standard_normal((N, q * n)))
    y.backward(dy)
    args = [v.detach().numpy() for v in (x, S, A, B, bias)]
    if not with_S:
        args[1] = None
    assert np.abs(OG.forward(*args, act) - y.detach().numpy()).max() <= 1e-12
    got = OG.backward(*args, dy.numpy(), act)
    for k, v in (("dx", x), ("dA", A), ("dB", B), ("dbias", bias)) + ((("dS", S),) if with_S else ()):
        assert np.abs(got[k] - v.grad.numpy()).max() <= 1e-11, k


def test_workspace():
    L = _lib.lib()
    s = KronShape(100, 32, 64, 24, 32, 4, 0)
    nb = lambda dt, S, b: L.kron_glu_workspace_bytes(ctypes.byref(s), dt, S, b)
    assert nb(0, 0, 0) > 0 and nb(0, 0, 0) % 256 == 0
    assert nb(0, 0, 0) > nb(1, 1, 0) > nb(1, 0, 0)         # three parts of a value, two or one of C, one
    assert nb(1, 0, 1) > 100 * 2048 * 8
    assert nb(2, 0, 0) == 0
    for bad in (KronShape(-1, 4, 4, 4, 4, 1, 0), KronShape(1, 65, 4, 4, 4, 1, 0), KronShape(1, 4, 4, 4, 4, 17, 0),
                KronShape(1, 4, 4, 4, 4, 1, 1)):
        assert L.kron_glu_workspace_bytes(ctypes.byref(bad), 0, 0, 0) == 0


def call(back, shape=(8, 4, 6, 5, 3, 2, 0), act=0, dt=0, null=(), nb=None, **kw):
    s = KronShape(*shape)
    names = ("x", "S", "A", "B", "bias", "dy", "dx", "dS", "dA", "dB", "dbias", "y", "ws")
    a = {k: P(i * MB) for i, k in enumerate(names)}
    a.update(kw)
    for k in null:
        a[k] = None
    L = _lib.lib()
    if nb is None:
        nb = L.kron_glu_workspace_bytes(ctypes.byref(s), dt if dt in (0, 1) else 0, int(a["S"] is not None), int(back))
    ins = (ctypes.byref(s), act, dt, a["x"], a["S"], a["A"], a["B"], a["bias"])
    if not back:
        return L.kron_glu_fwd(*ins, a["y"], a["ws"], ctypes.c_size_t(nb), None)
    return L.kron_glu_bwd(*ins, a["dy"], a["dx"], a["dS"], a["dA"], a["dB"], a["dbias"], a["ws"], ctypes.c_size_t(nb), None)


@pytest.mark.parametrize("back", [False, True])
def test_argument_errors(back):
    E = _lib
    for kw, want in ((dict(shape=(-1, 4, 6, 5, 3, 2, 0)), E.KRON_E_SHAPE), (dict(shape=(8, 0, 6, 5, 3, 2, 0)), E.KRON_E_SHAPE),
                     (dict(shape=(8, 65, 6, 5, 3, 2, 0)), E.KRON_E_UNSUPPORTED),
                     (dict(shape=(8, 4, 6, 5, 65, 2, 0)), E.KRON_E_UNSUPPORTED),
                     (dict(shape=(8, 4, 6, 5, 3, 17, 0)), E.KRON_E_UNSUPPORTED),
                     (dict(shape=(8, 4, 6, 5, 3, 2, 1)), E.KRON_E_ARG), (dict(act=4), E.KRON_E_ARG),
                     (dict(act=-1), E.KRON_E_ARG), (dict(dt=5), E.KRON_E_DTYPE),
                     (dict(null=("A",)), E.KRON_E_NULL), (dict(null=("B",)), E.KRON_E_NULL), (dict(null=("x",)), E.KRON_E_NULL),
                     (dict(null=("ws",)), E.KRON_E_WORKSPACE), (dict(nb=255), E.KRON_E_WORKSPACE),
                     (dict(ws=P(12 * MB + 128)), E.KRON_E_ALIGN), (dict(x=P(8)), E.KRON_E_ALIGN),
                     (dict(bias=P(4 * MB + 8)), E.KRON_E_ALIGN), (dict(ws=P(0)), E.KRON_E_ALIAS)):
        assert call(back, **kw) == want, kw
    if back:
        assert call(True, null=("dy",)) == E.KRON_E_NULL
        assert call(True, null=("dA",)) == E.KRON_E_NULL
        assert call(True, null=("dS",)) == E.KRON_E_NULL          # S without dS
        assert call(True, null=("S",)) == E.KRON_E_NULL           # dS without S
        assert call(True, dx=P(0)) == E.KRON_E_ALIAS              # dx over x
        assert call(True, dB=P(8 * MB + 16)) == E.KRON_E_ALIAS    # dB over dA
        assert call(True, dbias=P(12 * MB + 256)) == E.KRON_E_ALIAS
    else:
        assert call(False, null=("y",)) == E.KRON_E_NULL
        assert call(False, y=P(16)) == E.KRON_E_ALIAS
        assert call(False, shape=(0, 4, 6, 5, 3, 2, 0), null=("x", "y")) == 0


def test_binding_refuses():
    torch = pytest.importorskip("torch")
    import kronecker_factored_structured_amd as K
    x, A, B = torch.zeros(2, 6), torch.zeros(2, 1, 2, 2), torch.zeros(2, 1, 3, 2)
    with pytest.raises(ValueError, match="GPU tensor"):
        K.kron_glu_fwd(x, None, A, B)
    with pytest.raises(ValueError, match="act must be"):
        K.kron_glu_fwd(x, None, A, B, act="tanh")
    with pytest.raises(ValueError, match="unsupported dtype"):
        K.kron_glu_fwd(x.half(), None, A, B)


def test_module_refuses_sizes_that_its_forward_would():
    pytest.importorskip("torch")
    import kronecker_factored_structured_amd as K
    for kw in (dict(in_features=65 * 4), dict(out_features=65 * 4), dict(in_features=65, m=65, n=4), dict(n=65, out_features=65),
               dict(r=17), dict(r=0), dict(in_features=0)):
        with pytest.raises(ValueError, match="must be in 1"):
            K.KronGLU(**{**dict(in_features=64, out_features=32, m=4, r=2), **kw})
    assert sum(p.numel() for p in K.KronGLU(64, 32, m=4, r=2).parameters()) == 2 * (16 * 8 * 3 + 2 * 16 + 32)


def test_stream_without_the_private_handle(monkeypatch):
    """A torch without the private call has its public one asked, of the tensors' device."""
    torch = pytest.importorskip("torch")
    from types import SimpleNamespace

    from kronecker_factored_structured_amd import api
    monkeypatch.setattr(api, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: SimpleNamespace(cuda_stream=0x1230 + d.index))
    assert api._stream(torch.device("cuda", 5)).value == 0x1235
    monkeypatch.setattr(api, "_raw_stream", lambda i: 0x4560 + i)
    assert api._stream(torch.device("cuda", 5)).value == 0x4565

"""GPU parity of the gated Kronecker block with the fp64 oracle on the same (rounded) inputs.

Tolerances.  fp32 outputs, the bf16 block's parameter gradients among them: the layer's bar, 1e-5 of the
largest value (a product drops parts below 2^-21 = 4.8e-7 of it, sums are fp32).  bf16 outputs: half a step of
the value (2^-8), and 2e-4 of the largest value for the intermediates, which are carried in two bf16 parts
(2^-16 = 1.5e-5 each, three of them in a row and at most four times as large as the result)."""
import numpy as np
import pytest

from _harness import TOL_F32, rel_err
from oracle import glu as OG

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def K():
    import kronecker_factored_structured_amd as mod
    return mod


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def inputs(seed, N, p, q, m, n, r, dtype, S=False, bias=False):
    g = torch.Generator().manual_seed(seed)
    t = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(dtype).cuda()
    mask = None
    if S:
        mask = (torch.rand(2, p, q, generator=g) * (torch.rand(2, p, q, generator=g) < 0.5)).to(dtype).cuda()
    return (t(N, p * m), mask, t(2, r, p, q, scale=p ** -0.5), t(2, r, m, n, scale=m ** -0.5),
            t(2, q * n, scale=0.3) if bias else None), t(N, q * n)


def same(got, want, name=""):
    got, want = (got if isinstance(got, tuple) else (got,)), want
    t = got[0]
    if t.numel() == 0:
        return
    g, top = f64(t), np.abs(want).max()
    if t.dtype == BF:
        bad = np.abs(g - want) > 2.0 ** -8 * np.abs(want) + 2e-4 * top
        assert not bad.any(), (name, np.argwhere(bad)[:3], g[bad][:3], want[bad][:3])
    else:
        assert rel_err(g, want) <= TOL_F32, (name, rel_err(g, want))


SHAPES = [
    (1, 1, 1, 1, 1, 1), (3, 2, 3, 5, 4, 2), (2, 16, 16, 64, 64, 2), (5, 17, 33, 31, 15, 1), (9, 32, 64, 24, 32, 4),
    (33, 25, 43, 30, 47, 3), (130, 32, 32, 32, 32, 4), (7, 64, 64, 64, 64, 2), (11, 64, 3, 2, 61, 5), (4, 3, 64, 63, 5, 16),
    (1027, 9, 17, 11, 13, 2), (6, 48, 49, 33, 34, 6), (257, 32, 64, 32, 64, 4)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N,p,q,m,n,r", SHAPES)
def test_glu(N, p, q, m, n, r, dtype):
    for k, (act, S, bias) in enumerate((("silu", False, False), ("gelu", True, True), ("gelu_tanh", True, False))):
        print(f"[glu] N={N} p={p} q={q} m={m} n={n} r={r} {dtype} {act} S={S} bias={bias}", flush=True)
        a, dy = inputs(N + k, N, p, q, m, n, r, dtype, S, bias)
        h = [f64(v) for v in a]
        same(K().kron_glu_fwd(*a, act=act), OG.forward(*h, act), "y")
        got = K().kron_glu_bwd(*a, dy, act=act)
        want = OG.backward(*h, f64(dy), act)
        for key in ("dx", "dA", "dB", "dS", "dbias"):
            if (key == "dS" and not S) or (key == "dbias" and not bias):
                assert got[key] is None
            else:
                same(got[key], want[key], key)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_glu_relu(dtype):
    """dy is zero where the gate's value is within rounding of the kink."""
    a, dy = inputs(5, 40, 9, 17, 11, 13, 2, dtype, True, True)
    h = [f64(v) for v in a]
    g = OG.project(*h)[0]
    dy[torch.from_numpy(np.abs(g) < 1e-3).cuda()] = 0
    same(K().kron_glu_fwd(*a, act="relu"), OG.forward(*h, "relu"), "y")
    got, want = K().kron_glu_bwd(*a, dy, act="relu"), OG.backward(*h, f64(dy), "relu")
    for key in ("dx", "dA", "dB", "dS", "dbias"):
        same(got[key], want[key], key)


def test_large_activations_stay_finite():
    """Gates of some hundreds either way: the activations saturate, nothing overflows."""
    a, dy = inputs(6, 50, 8, 8, 8, 8, 1, F32)
    a = (a[0] * 300,) + a[1:]
    h = [f64(v) for v in a]
    for act in ("silu", "gelu", "gelu_tanh"):
        with np.errstate(over="ignore"):
            same(K().kron_glu_fwd(*a, act=act), OG.forward(*h, act), act)
            want = OG.backward(*h, f64(dy), act)
        got = K().kron_glu_bwd(*a, dy, act=act)
        for key in ("dx", "dA", "dB"):
            same(got[key], want[key], key)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_empty_batch(dtype):
    a, dy = inputs(1, 0, 4, 6, 5, 3, 2, dtype, True, True)
    assert K().kron_glu_fwd(*a).shape == (0, 18)
    got = K().kron_glu_bwd(*a, dy)
    for key in ("dA", "dB", "dS", "dbias"):
        assert got[key].abs().max().item() == 0, key


def test_rows_are_independent_and_calls_repeat():
    """A row's output is the same bits in any batch it is part of, and a NaN stays in its row."""
    a, dy = inputs(2, 37, 32, 64, 24, 32, 4, BF, False, True)
    y, g = K().kron_glu_fwd(*a), K().kron_glu_bwd(*a, dy)
    assert torch.equal(y, K().kron_glu_fwd(*a))
    g2 = K().kron_glu_bwd(*a, dy)
    assert all(torch.equal(g[k], g2[k]) for k in g if g[k] is not None)
    assert torch.equal(K().kron_glu_fwd(a[0][5:6], *a[1:]), y[5:6])
    x = a[0].clone()
    x[3, 100] = float("nan")
    yn = K().kron_glu_fwd(x, *a[1:])
    keep = [i for i in range(37) if i != 3]
    assert torch.equal(yn[keep], y[keep]) and bool(torch.isnan(yn[3]).any())


def test_outputs_given_and_not_asked():
    a, dy = inputs(3, 12, 5, 6, 7, 8, 3, F32, True, True)
    ref = K().kron_glu_bwd(*a, dy)
    got = K().kron_glu_bwd(*a, dy, want_dx=False)
    assert got["dx"] is None and torch.equal(got["dA"], ref["dA"])
    outs = {k: torch.full_like(v, float("nan")) for k, v in ref.items()}
    outs["dbias"] = None
    got = K().kron_glu_bwd(*a, dy, outs=outs)
    assert got["dB"] is outs["dB"] and got["dbias"] is None
    assert all(torch.equal(got[k], ref[k]) for k in ("dx", "dA", "dB", "dS"))
    y = torch.empty(12, 48, device="cuda")
    assert K().kron_glu_fwd(*a, out=y) is y


def test_gradient_against_differences():
    """Central differences of sum(dy o y) along one direction of each input: off by h^2/6 of the third derivative
    (for a product of two functions linear in each factor, times silu: below 30 * the slope's scale here) and by
    the outputs' rounding over h."""
    a, dy = inputs(8, 20, 6, 7, 5, 4, 2, F32, True, True)
    got = K().kron_glu_bwd(*a, dy)
    f = lambda v: float((f64(K().kron_glu_fwd(*v)) * f64(dy)).sum())
    scale = float((np.abs(f64(K().kron_glu_fwd(*a))) * np.abs(f64(dy))).sum())
    h = 2.0 ** -6
    for i, key in enumerate(("dx", "dS", "dA", "dB", "dbias")):
        v = torch.randn(a[i].shape, generator=torch.Generator().manual_seed(i)).cuda()
        v /= v.norm()
        up, dn = list(a), list(a)
        up[i], dn[i] = a[i] + h * v, a[i] - h * v
        slope = (f(up) - f(dn)) / (2 * h)
        want = float((f64(got[key]) * f64(v)).sum())
        assert abs(slope - want) <= 30 * scale * h * h / 6 + TOL_F32 * scale / h, (key, slope, want)


def test_another_stream_and_a_captured_call():
    a, dy = inputs(4, 65, 32, 32, 32, 32, 4, BF, True, True)
    y, g = K().kron_glu_fwd(*a), K().kron_glu_bwd(*a, dy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            ys, gs = K().kron_glu_fwd(*a), K().kron_glu_bwd(*a, dy)
    s.synchronize()
    assert torch.equal(ys, y) and all(torch.equal(gs[k], g[k]) for k in g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yc, gc = K().kron_glu_fwd(*a), K().kron_glu_bwd(*a, dy)
    for i in range(3):
        a[0].copy_(torch.randn(a[0].shape, generator=torch.Generator().manual_seed(i)).to(BF))
        graph.replay()
        torch.cuda.synchronize()
        y, g = K().kron_glu_fwd(*a), K().kron_glu_bwd(*a, dy)
        assert torch.equal(yc, y) and all(torch.equal(gc[k], g[k]) for k in g), i


def test_binding_refusals():
    k = K()
    a, dy = inputs(1, 4, 4, 6, 5, 3, 2, F32, True, True)
    x, S, A, B, bias = a

    def bad(match, *args, fn=k.kron_glu_fwd, **kw):
        with pytest.raises(ValueError, match=match):
            fn(*args, **kw)

    bad("x must be", x[:, :-1].contiguous(), S, A, B, bias)
    bad("contiguous", x.t(), S, A, B, bias)
    bad("A must be", x, S, A[0], B, bias)
    bad("rank", x, S, A, B[:, :1].contiguous(), bias)
    bad("S must be", x, S[0], A, B, bias)
    bad("bias", x, S, A, B, bias[0].contiguous())
    bad("must be torch.float32", x, S, A.to(BF), B, bias)
    bad("act", x, S, A, B, bias, act="swish")
    bad("out", x, S, A, B, bias, out=torch.zeros(4, 17, device="cuda"))
    bad("dy", x, S, A, B, bias, dy[:3], fn=k.kron_glu_bwd)
    bad("dA", x, S, A, B, bias, dy, fn=k.kron_glu_bwd, outs={"dA": torch.zeros(2, 4, 6, device="cuda")})
    with pytest.raises(k._lib.KronError, match="exceeds 64"):
        big, _ = inputs(1, 2, 65, 2, 2, 2, 1, F32)
        k.kron_glu_fwd(*big)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("p,q,m,n,r", [(50, 20, 30, 28, 2), (20, 30, 28, 50, 3), (50, 40, 30, 28, 3), (50, 28, 20, 50, 1),
                                       (33, 20, 40, 33, 7), (20, 40, 50, 20, 2)])
def test_glu_sides_either_side_of_32(p, q, m, n, r, dtype):
    """One side of a factor above 32 and the other below, with S and without, over more rows than a pass holds."""
    for k, (N, S) in enumerate(((701, True), (300, False))):
        print(f"[glu 32] N={N} p={p} q={q} m={m} n={n} r={r} {dtype} S={S}", flush=True)
        a, dy = inputs(N + k, N, p, q, m, n, r, dtype, S, True)
        h = [f64(v) for v in a]
        same(K().kron_glu_fwd(*a), OG.forward(*h, "silu"), "y")
        got, want = K().kron_glu_bwd(*a, dy), OG.backward(*h, f64(dy), "silu")
        for key in ("dx", "dA", "dB", "dbias") + (("dS",) if S else ()):
            same(got[key], want[key], key)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_module(dtype):
    """KronGLU: leading dimensions, gradients of the input and of each parameter, no gradient asked of x."""
    k = K()
    torch.manual_seed(0)
    mod = k.KronGLU(4 * 5, 6 * 3, m=5, r=2, n=3, act="gelu", device="cuda", dtype=dtype)
    with torch.no_grad():
        mod.bias.normal_(std=0.3)
        mod.S.mul_(torch.rand_like(mod.S))
    x = torch.randn(3, 7, 20, device="cuda").to(dtype).requires_grad_()
    y = mod(x)
    dy = torch.randn(3, 7, 18, device="cuda").to(dtype)
    assert y.shape == (3, 7, 18) and y.dtype == dtype
    h = [f64(v) for v in (x.reshape(21, 20), mod.S, mod.A, mod.B, mod.bias)]
    same(y.reshape(21, 18), OG.forward(*h, "gelu"), "y")
    y.backward(dy)
    want = OG.backward(*h, f64(dy).reshape(21, 18), "gelu")
    for key, t in (("dx", x), ("dS", mod.S), ("dA", mod.A), ("dB", mod.B), ("dbias", mod.bias)):
        assert t.grad.shape == t.shape and t.grad.dtype == dtype
        same(t.grad.reshape(want[key].shape), want[key], key)
    y2 = mod(x.detach())
    y2.sum().backward()
    assert mod(x[:, :0]).shape == (3, 0, 18)
    plain = k.KronGLU(20, 18, m=5, r=1, n=3, with_S=False, bias=False, device="cuda")
    (g,) = torch.autograd.grad(plain(x.detach().float()).sum(), [plain.A])
    assert bool(g.abs().sum() > 0) and len(list(plain.parameters())) == 2


def test_module_refusals():
    k = K()
    with pytest.raises(ValueError, match="multiple of m"):
        k.KronGLU(21, 18, m=5, r=1, n=3, device="cuda")
    with pytest.raises(ValueError, match="act"):
        k.KronGLU(20, 18, m=5, r=1, n=3, act="tanh", device="cuda")
    with pytest.raises(ValueError, match="x must be"):
        k.KronGLU(20, 18, m=5, r=1, n=3, device="cuda")(torch.zeros(2, 19, device="cuda"))
    mod = k.KronGLU(20, 18, m=5, r=1, n=3, device="cuda")
    x = torch.randn(2, 20, device="cuda", requires_grad=True)
    (g,) = torch.autograd.grad(mod(x).sum(), [x], create_graph=True)
    with pytest.raises(RuntimeError):      # one derivative only
        g.sum().backward()


def test_more_rows_than_a_launch_takes():
    """2^24 + 9 rows of one value each, with factors of more ranks than fit a workgroup: the last rows are as
    right as the first."""
    N, r = 2 ** 24 + 9, 16
    print("[glu] many rows", flush=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy = (torch.randn(N, 1, device="cuda", generator=g) for _ in range(2))
    A, B = torch.randn(2, r, 1, 1, device="cuda", generator=g), torch.randn(2, r, 1, 1, device="cuda", generator=g)
    W = (A.double() * B.double()).sum((1, 2, 3))
    y = K().kron_glu_fwd(x, None, A, B, act="relu").double()
    xd, dyd = x.double(), dy.double()
    gate, up = xd * W[0], xd * W[1]
    want = torch.relu(gate) * up
    assert (y - want).abs().max() <= TOL_F32 * want.abs().max()
    got = K().kron_glu_bwd(x, None, A, B, None, dy, act="relu")
    dg, du = dyd * up * (gate > 0), dyd * torch.relu(gate)
    dx = dg * W[0] + du * W[1]
    assert (got["dx"].double() - dx).abs().max() <= TOL_F32 * dx.abs().max()
    dW = torch.stack([(xd * dg).sum(), (xd * du).sum()])
    # (a sum of N terms of either sign, each within the bar of its size)
    size = torch.stack([(xd * dg).abs().sum(), (xd * du).abs().sum()])
    for f in range(2):
        assert bool(((got["dA"][f].double() - B[f].double() * dW[f]).abs() <= TOL_F32 * B[f].double().abs() * size[f]).all())
        assert bool(((got["dB"][f].double() - A[f].double() * dW[f]).abs() <= TOL_F32 * A[f].double().abs() * size[f]).all())

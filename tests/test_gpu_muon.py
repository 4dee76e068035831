"""kron_muon_step against the fp64 oracle.

Tolerances.  The momentum is two fp32 roundings.  For the matrix X, a worst-case bound over five steps of three products is
of no use (the absolute sums grow with the sides' powers), so the bar is what plain arithmetic of the same precision
leaves on the same inputs, computed by the oracle: fp32 throughout for fp32 parameters; operands rounded to fp16 for
bf16 ones, whose kernels hold X, A and the polynomial of A in one fp16 part.  The kernel's error of X, as a
Frobenius norm, may be four times that, and at least 16 fp32 (fp16) roundings of X itself.  On top comes the parameter's own
rounding (fp32 2^-24 twice, bf16 2^-8)."""
import numpy as np
import pytest

from oracle import muon as OM

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
u = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def K():
    import kronecker_factored_structured_amd as k
    return k


def f64(t):
    return t.detach().cpu().double().numpy()


def tensors(seed, shapes, dtype, rank=None):
    g = torch.Generator().manual_seed(seed)
    W = [torch.randn(s, generator=g).to(dtype).cuda() for s in shapes]
    if rank is None:
        G = [(torch.randn(s, generator=g) * 0.01).to(dtype).cuda() for s in shapes]
    else:
        G = [(torch.randn(*s[:-1], rank, generator=g) @ torch.randn(*s[:-2], rank, s[-1], generator=g)).to(dtype).cuda() for s in shapes]
    m = [(torch.randn(s, generator=g) * 0.05 * (rank is None)).cuda() for s in shapes]
    return W, G, m


def half(v):
    """Rounded to fp16 in the range that the kernels' scale gives it."""
    return (v * 4096).astype(np.float16).astype(v.dtype) / 4096


def compare(W, G, m, lr=0.1, **kw):
    k = K()
    before = [[f64(t) for t in ts] for ts in (W, G, m)]
    args = dict(lr=lr, momentum=0.95, nesterov=True, weight_decay=0.0, steps=5, scales=None)
    args.update(kw)
    k.kron_muon_step(W, G, m, **args)
    bf = W[0].dtype == torch.bfloat16
    for i, (w0, g0, m0) in enumerate(zip(*before)):
        shape = w0.shape
        if w0.size == 0:
            continue
        scale = args["scales"][i] if args["scales"] else max(1.0, shape[-2] / shape[-1]) ** 0.5
        got_w, got_m = f64(W[i]).reshape(-1, *shape[-2:]), f64(m[i]).reshape(-1, *shape[-2:])
        for j, (w, g, mo) in enumerate(zip(*(v.reshape(-1, *shape[-2:]) for v in (w0, g0, m0)))):
            hyper = dict(mu=args["momentum"], nesterov=args["nesterov"], wd=args["weight_decay"], scale=scale, steps=args["steps"])
            want_w, want_m, o = OM.step(w, g, mo, lr, **hyper)
            assert np.all(np.abs(got_m[j] - want_m) <= 2 * u * (np.abs(want_m) + np.abs(0.95 * mo) + np.abs(g)))
            _, _, plain = OM.step(w, g, mo, lr, dtype=np.float32, part=half if bf else (lambda v: v), **hyper)
            err = max(4 * np.linalg.norm(plain - o), 16 * (2.0 ** -11 if bf else u) * np.linalg.norm(o))
            r = 2.0 ** -8 if bf else 3 * u
            off = np.abs(got_w[j] - want_w) - r * (np.abs(want_w) + np.abs(w))
            assert np.linalg.norm(np.maximum(off, 0)) <= lr * scale * err, (shape, j)


SMALL = [(1, 1), (1, 5), (5, 1), (3, 7), (16, 16), (17, 15), (32, 32), (2, 4, 32, 64), (3, 24, 32), (48, 24), (64, 64), (64, 300), (16, 1500),
         (2000, 9), (33, 500), (5, 63, 49)]
LARGE = [(65, 65), (65, 130), (200, 70), (128, 128), (64, 1000), (16, 3000), (3000, 16), (1, 5000), (3, 100, 260), (2, 300, 66)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SMALL + LARGE)
def test_values(shape, dtype):
    compare(*tensors(sum(shape), [shape], dtype))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kw", [dict(nesterov=False), dict(weight_decay=0.3), dict(steps=1), dict(steps=6), dict(momentum=0.0), dict(lr=0.0)])
def test_arguments(kw, dtype):
    args = dict(scales=[0.5, 2.0])
    args.update(kw)
    compare(*tensors(3, [(2, 20, 30), (90, 80)], dtype), **args)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_tensors(dtype):
    """More tensors than a launch takes, small and large, tall and wide of one size, one empty."""
    shapes = [(2, 8, 12)] * 30 + [(70, 90)] * 3 + [(90, 70)] * 2 + [(0, 8, 8)] + [(4, 4)] * 15 + [(70, 5, 66, 67)] + [(70, 90)] * 40
    compare(*tensors(4, shapes, dtype))


@pytest.mark.parametrize("shape", [(300, 280), (512, 512), (256, 700)])
def test_larger_tiles(shape):
    """Stacks large enough for the larger tiles."""
    compare(*tensors(5, [(6, *shape)], torch.float32))
    compare(*tensors(5, [(6, *shape)], torch.bfloat16))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(24, 40), (100, 120)])
def test_low_rank(shape, dtype):
    """Gradients of rank 1 and 3: singular values of zero stay next to zero."""
    for rank in (1, 3):
        compare(*tensors(rank, [shape], dtype, rank=rank), nesterov=False)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(3, 20, 30), (3, 80, 90)])
def test_zeros_and_non_finite(shape, dtype):
    """A matrix of zeros stays (X = 0); a NaN or an infinity spoils its own matrix and no other."""
    k = K()
    W, G, m = tensors(6, [shape], dtype)
    G[0][0], m[0][0] = 0, 0
    G[0][2, 1, 1] = float("nan")
    w0 = W[0].clone()
    k.kron_muon_step(W, G, m, lr=0.1)
    assert torch.equal(W[0][0], w0[0]) and torch.count_nonzero(m[0][0]) == 0
    assert torch.isfinite(W[0][1]).all() and not torch.equal(W[0][1], w0[1])
    assert torch.isnan(W[0][2]).all()


@pytest.mark.parametrize("shape", [(20, 30), (80, 90)])
@pytest.mark.parametrize("scale", [1e-18, 1e18])
def test_sizes_of_gradients(shape, scale):
    """The update does not depend on the gradient's size (eps aside: it counts beside norms of 1e-7)."""
    k = K()
    W, G, m = tensors(7, [shape], torch.float32)
    m[0].zero_()
    W2, m2 = [W[0].clone()], [torch.zeros_like(m[0])]
    k.kron_muon_step(W, G, m, lr=1.0, eps=1e-30)
    k.kron_muon_step(W2, [G[0] * scale], m2, lr=1.0, eps=1e-30)
    assert (W[0] - W2[0]).abs().max().item() < 1e-4


def test_repeatable_and_workspace_ignored():
    k = K()
    out = []
    for fill in (0, 255):
        W, G, m = tensors(8, [(100, 130), (3, 30, 20), (2, 130, 100)], torch.float32)
        ws = torch.full((1 << 23,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(3):
            k.kron_muon_step(W, G, m, lr=0.05, workspace=ws)
        out.append(W + m)
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_binding_refuses():
    k = K()
    W, G, m = tensors(9, [(4, 6), (8, 8)], torch.float32)
    for bad in (lambda: k.kron_muon_step(W, G[:1], m, lr=0.1), lambda: k.kron_muon_step(W, G, m, lr=0.1, scales=[1.0]),
                lambda: k.kron_muon_step([W[0], W[1].bfloat16()], G, m, lr=0.1), lambda: k.kron_muon_step(W, [G[0], G[1].t()[:4]], m, lr=0.1),
                lambda: k.kron_muon_step(W, G, [m[0], m[1].double()], lr=0.1), lambda: k.kron_muon_step([W[0].view(-1)], [G[0].view(-1)], [m[0].view(-1)], lr=0.1),
                lambda: k.kron_muon_step([W[1].t()], [G[1]], [m[1]], lr=0.1)):
        with pytest.raises(ValueError):
            bad()
    from kronecker_factored_structured_amd._lib import KronError
    with pytest.raises(KronError):
        k.kron_muon_step([W[0], W[0]], G[:1] * 2, m[:1] * 2, lr=0.1)
    with pytest.raises(KronError):
        k.kron_muon_step(W, G, m, lr=0.1, steps=0)
    k.kron_muon_step([], [], [], lr=0.1)

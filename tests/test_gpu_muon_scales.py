"""kron_muon_step where the default coefficients' bounds do not hold: other quintics, matrices that grow or shrink from step to
step, the smallest eps and gradients at both ends of fp32's range.

Tolerances as in test_gpu_muon.py: the error of X, as a Frobenius norm, may be four times what plain arithmetic of the same
precision leaves on the same inputs (fp32, or operands rounded to fp16's eleven bits), and at least sixteen roundings of X;
then the parameter's own rounding.  A step's product P X is off by 2^-22 of P, as much of X and as much for the product of
the second parts, 12 u in all; where the quintic is linear, P is a multiple of the identity whose rounding is the same
everywhere and in every step, so that steps * 12 u may add up (fp32; the plain arithmetic has no such parts).  `half` rounds to eleven bits whatever the matrix's size."""
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


def half(v):
    """Rounded to eleven bits, over the largest value as the kernels' scales have it."""
    up = 2.0 ** (12 - np.frexp(np.abs(v).max())[1]) if np.abs(v).max() > 0 else 1.0
    return (v * up).astype(np.float16).astype(v.dtype) / v.dtype.type(up)


def tensors(seed, shape, dtype):
    g = torch.Generator().manual_seed(seed)
    r = lambda s: torch.randn(shape, generator=g) * s
    return r(1.0).to(dtype).cuda(), r(0.01).to(dtype).cuda(), r(0.05).cuda()


def compare(shape, dtype, coeffs, steps, lr=0.1, seed=0):
    k = K()
    W, G, m = tensors(seed + sum(shape), shape, dtype)
    W.zero_()      # (X is what is left, however small)
    before = [f64(t).reshape(-1, *shape[-2:]) for t in (W, G, m)]
    k.kron_muon_step([W], [G], [m], lr=lr, coeffs=coeffs, steps=steps, scales=[1.0])
    bf = dtype == torch.bfloat16
    got = f64(W).reshape(-1, *shape[-2:])
    for j, (w, g, mo) in enumerate(zip(*before)):
        kw = dict(steps=steps, coeffs=coeffs)
        want, _, o = OM.step(w, g, mo, lr, **kw)
        _, _, plain = OM.step(w, g, mo, lr, dtype=np.float32, part=half if bf else (lambda v: v), **kw)
        err = max(4 * np.linalg.norm(plain - o), (16 * 2.0 ** -11 if bf else max(16, 12 * steps) * u) * np.linalg.norm(o))
        r = 2.0 ** -8 if bf else 3 * u
        off = np.abs(got[j] - want) - r * (np.abs(want) + np.abs(w))
        assert np.linalg.norm(np.maximum(off, 0)) <= lr * err, (shape, j, np.linalg.norm(o))


# a cubic and quintics that stay next to 1, a steep one of one step, ones that make every singular value larger or smaller
QUINTICS = [((1.5, -0.5, 0.0), 5), ((1.875, -1.25, 0.375), 6), ((8.28721201814563, -23.595886519098837, 17.300387312530933), 1),
            ((4.0, -6.0, 2.5), 3), ((2.0, 0.0, 0.0), 10), ((15.0, 0.0, 0.0), 1), ((1000.0, 0.0, 0.0), 1), ((12.0, -20.0, 9.0), 1),
            ((0.5, 0.0, 0.0), 6), ((0.5, 0.0, 0.0), 16), ((0.1, -0.05, 0.01), 6), ((0.001, 0.0, 0.0), 5), ((0.0, 0.01, 0.0), 2),
            ((0.0, 0.0, 0.0), 2), ((-2.0, 1.5, -0.5), 5), ((0.0, 0.0, 900.0), 1)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(20, 30), (90, 80), (80, 300), (2, 200, 70)])
@pytest.mark.parametrize("coeffs,steps", QUINTICS)
def test_other_quintics(coeffs, steps, shape, dtype):
    """Coefficients for which P, A or X leave fp16's range at the default's scale, on matrices that fit LDS and that do not."""
    compare(shape, dtype, coeffs, steps)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(1, 1), (5, 1), (3, 7), (17, 15), (2, 4, 32, 64), (48, 24), (64, 64), (64, 300), (16, 1500), (2000, 9), (5, 63, 49),
                                   (65, 65), (65, 130), (200, 70), (64, 1000), (16, 3000), (3001, 17), (1, 5000), (3, 100, 260), (2, 300, 66)])
def test_the_default(shape, dtype):
    """X alone (the rounding of parameters next to 1 would hide it)."""
    compare(shape, dtype, OM.COEFFS, 5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(20, 30), (90, 80)])
def test_rank_one_grows(shape, dtype):
    """The gradient of one sample: a singular value of 1, and the bound itself is reached."""
    k = K()
    g = torch.Generator().manual_seed(1)
    G = (torch.randn(shape[0], 1, generator=g) @ torch.randn(1, shape[1], generator=g)).to(dtype).cuda()
    for coeffs, steps in (((2.0, 0.0, 0.0), 10), ((8.0, -4.0, 1.0), 2), ((1000.0, 0.0, 0.0), 1), ((1.0, 1.0, 1.0), 2)):
        W, m = torch.zeros_like(G), torch.zeros(shape, device="cuda")
        k.kron_muon_step([W], [G], [m], lr=1.0, coeffs=coeffs, steps=steps, scales=[1.0], nesterov=False)
        o = OM.orthogonalise(f64(G), steps=steps, coeffs=coeffs)
        # P's roundings and the products', each relative to P's and X's bound: steps of at most sixteen (eight at 2^-11)
        tol = (8 * 2.0 ** -11 + 2.0 ** -8 if dtype == torch.bfloat16 else 32 * u) * steps * np.linalg.norm(o)
        assert np.linalg.norm(f64(W) + o) <= tol, (coeffs, steps)


def test_growth_beyond_the_limit_is_refused():
    """Matrices that do not fit LDS are held in 16-bit parts: a quintic that takes a singular value beyond what these
    hold is refused for them, before anything is launched; in LDS it is fp32 and runs."""
    k = K()
    from kronecker_factored_structured_amd._lib import KronError
    for coeffs, steps in (((8.28721201814563, -23.595886519098837, 17.300387312530933), 5), ((1e6, 0.0, 0.0), 1), ((2.0, 0.0, 0.0), 16),
                          ((1e38, 1e38, 1e38), 16), ((0.0, 0.0, -1e5), 2)):
        W, G, m = tensors(3, (80, 90), torch.float32)
        keep = [W.clone(), m.clone()]
        with pytest.raises(KronError):
            k.kron_muon_step([W], [G], [m], lr=0.1, coeffs=coeffs, steps=steps)
        assert torch.equal(W, keep[0]) and torch.equal(m, keep[1])
    compare((20, 30), torch.float32, (2.0, 0.0, 0.0), 16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(3, 20, 30), (3, 80, 90)])
@pytest.mark.parametrize("eps", [1e-30, 1e-36, 1e-40, 1.5e-45])
def test_zeros_and_the_smallest_eps(shape, dtype, eps):
    """A matrix of zeros stays where 1 / eps is beyond fp32."""
    k = K()
    W, G, m = tensors(6, shape, dtype)
    G[0], m[0] = 0, 0
    w0 = W.clone()
    k.kron_muon_step([W], [G], [m], lr=0.1, eps=eps)
    assert torch.equal(W[0], w0[0]) and torch.count_nonzero(m[0]) == 0
    assert torch.isfinite(W).all() and not torch.equal(W[1], w0[1])


@pytest.mark.parametrize("shape", [(20, 30), (80, 90), (300, 16)])
@pytest.mark.parametrize("up", [-130, -126, -120, 100, 119])
def test_gradients_at_the_ends_of_the_range(shape, up):
    """The update does not depend on the gradient's size, up to where fp32 itself ends: values of 2^-130 have 2^-149 / 2^-130 =
    2^-19 of rounding, which five steps of the quintic multiply by at most 3.45^5 = 489 where the singular value is small, so
    X, of values below 1.3, is off by at most 2^-19 * 489 * 2 as a norm over sqrt of the smaller side."""
    k = K()
    W, G, m = tensors(7, shape, torch.float32)
    G = G / G.abs().max()
    m.zero_()
    W2, m2 = W.clone(), torch.zeros_like(m)
    k.kron_muon_step([W], [G], [m], lr=1.0, eps=1.5e-45)
    small = torch.ldexp(G, torch.tensor(up // 2, device="cuda"))
    small = torch.ldexp(small, torch.tensor(up - up // 2, device="cuda"))
    k.kron_muon_step([W2], [small], [m2], lr=1.0, eps=1.5e-45)
    o = f64(W2) - f64(W)
    assert np.isfinite(o).all()
    tol = 2.0 ** -19 * 489 * 2 * min(shape) ** 0.5 if up < -100 else 1e-5 * min(shape) ** 0.5
    assert np.linalg.norm(o) <= tol

"""kron_muon_step on matrices of many tiles, against the same steps in 64 bits on the GPU.

Tolerances as in test_gpu_muon.py: the error of X, as a Frobenius norm, may be four times what plain arithmetic of the same
precision leaves on the same inputs (fp32; for bf16 parameters operands rounded to fp16's eleven bits), and at least sixteen
roundings of X; then the parameter's own rounding (bf16 2^-8, fp32 2^-24 twice and the product's)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
u = 2.0 ** -24
COEFFS = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def K():
    import kronecker_factored_structured_amd as k
    return k


def half(v):
    return (v * 4096).to(torch.float16).to(v.dtype) / 4096


def steps_of(x, steps, part=lambda v: v):
    """x: one matrix, its smaller side first, in the type of the arithmetic."""
    a, b, c = COEFFS
    eye = torch.eye(x.shape[0], device=x.device, dtype=x.dtype)
    for _ in range(steps):
        x = part(x)
        A = part(x @ x.t().contiguous())
        x = part(a * eye + b * A + c * (A @ A)) @ x
    return x


def tensors(seed, shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda s: torch.randn(shape, device="cuda", generator=g) * s
    return r(1.0).to(dtype), r(0.01).to(dtype), r(0.05)


def compare(shapes, dtype, steps=5, lr=0.1, only=None):
    """Every matrix of every tensor (only: the numbers of those that are looked at)."""
    k = K()
    T = [tensors(i + sum(s), s, dtype) for i, s in enumerate(shapes)]
    for W, _, _ in T:
        W.zero_()      # (the rounding of parameters next to 1 would hide most of X's)
    before = [(W.clone(), m.clone()) for W, _, m in T]
    k.kron_muon_step(*([t[i] for t in T] for i in range(3)), lr=lr, steps=steps)
    bf = dtype == torch.bfloat16
    r = 2.0 ** -8 if bf else 3 * u
    for (W, G, m), (w0, m0) in zip(T, before):
        rows, cols = W.shape[-2:]
        scale = max(1.0, rows / cols) ** 0.5
        views = [t.view(-1, rows, cols) for t in (W, G, m, w0, m0)]
        for j in only or range(views[0].shape[0]):
            w1, g, m1, w, mo = (t[j].double() for t in views)
            want_m = 0.95 * mo + g
            assert bool(((m1 - want_m).abs() <= 2 * u * (want_m.abs() + (0.95 * mo).abs() + g.abs())).all())
            x = g + 0.95 * want_m
            x = x / (x.norm() + 1e-7)
            x = (x.t() if rows > cols else x).contiguous()
            o = steps_of(x, steps)
            plain = steps_of(x.float(), steps, half if bf else (lambda v: v)).double()
            err = max(4 * (plain - o).norm().item(), 16 * (2.0 ** -11 if bf else u) * o.norm().item())
            want = w - lr * scale * (o.t() if rows > cols else o)
            off = (w1 - want).abs() - r * (want.abs() + w.abs())
            assert off.clamp(min=0).norm().item() <= lr * scale * err, (rows, cols, j)


def test_more_matrices_than_a_group_takes():
    """Seventeen of 4096 x 4096: sixteen share a workspace, the last one has it to itself."""
    compare([(17, 4096, 4096)], torch.bfloat16, steps=1, only=(0, 15, 16))


# What a product's tile follows from is the number of tiles of all matrices: 64 x 64 with four groups of wavefronts (one matrix),
# 64 x 64 with two steps in LDS, 128 x 128 and 256 x 256; ragged sides, wide and tall ones together
@pytest.mark.parametrize("shapes", [[(530, 700)], [(700, 530)], [(5, 700, 720)], [(3, 720, 700), (2, 700, 720)], [(9, 520, 530), (9, 530, 520)],
                                    [(40, 520, 530), (24, 530, 520)], [(4, 768, 2048)], [(2, 2048, 768), (2, 768, 2048)], [(1100, 1000)], [(2, 2100, 2000)]])
def test_fp32(shapes):
    compare(shapes, torch.float32)


@pytest.mark.parametrize("shapes", [[(1000, 1020)], [(1020, 1000)], [(5, 700, 720)], [(3, 720, 700), (2, 700, 720)], [(9, 520, 530), (9, 530, 520)],
                                    [(40, 520, 530), (24, 530, 520)], [(4, 768, 2048)], [(2, 2048, 768), (2, 768, 2048)], [(1001, 1015)], [(2, 2100, 2000)]])
def test_bf16(shapes):
    compare(shapes, torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_non_finite_matrices_stay_alone(dtype):
    """In tiles of 128 and 256, of one group each: the others are what they are without it."""
    k = K()
    for shape in ((18, 520, 530), (64, 520, 530)):
        W, G, m = tensors(3, shape, dtype)
        W2, m2 = W.clone(), m.clone()
        k.kron_muon_step([W2], [G], [m2], lr=0.1)
        G[7, 100, 3], G[11, 519, 529] = float("nan"), float("inf")
        G[13], m[13] = 0, 0
        w13 = W[13].clone()
        k.kron_muon_step([W], [G], [m], lr=0.1)
        keep = [i for i in range(shape[0]) if i not in (7, 11, 13)]
        assert torch.equal(W[keep], W2[keep]) and torch.equal(W[13], w13)
        assert torch.isnan(W[7]).all() and not torch.isfinite(W[11]).any()

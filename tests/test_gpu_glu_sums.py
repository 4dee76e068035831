"""Precision of the gated block where the largest value does not hide it: positive data, each output against its own size.

bf16 outputs: half a step of the value, and 2^-16 of the sum that it comes from for intermediates carried as two
rounded bf16 parts (off by half a unit of the second one: 2^-17 of a value, once in y and twice in dx; sums are
fp32, below 2^-17 for the 64 terms here)."""
import numpy as np
import pytest

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


def half_step(v):
    """Half a bf16 step at the size of v."""
    return 2.0 ** (np.floor(np.log2(np.abs(v))) - 8)


@pytest.mark.parametrize("S", [False, True])
@pytest.mark.parametrize("N,p,q,m,n", [(256, 8, 16, 8, 32), (4096, 1, 1, 8, 32)])
def test_bf16_intermediates_are_rounded(N, p, q, m, n, S):
    """u = 1 exactly, so y is the gate's sum of positive terms; dx of d = dy u, which bf16 does not hold, likewise."""
    g = torch.Generator().manual_seed(11)
    pos = lambda *s: (0.5 + torch.rand(*s, generator=g)).to(BF).cuda()
    x, A, B, dy = pos(N, p * m), pos(2, 1, p, q), pos(2, 1, m, n), pos(N, q * n)
    mask = pos(2, p, q) if S else None
    bias = torch.zeros(2, q * n, dtype=BF, device="cuda")
    bias[1] = 1
    A1 = A.clone()
    A1[1] = 0
    y = f64(K().kron_glu_fwd(x, mask, A1, B, bias, act="relu"))
    want = OG.forward(f64(x), f64(mask), f64(A1), f64(B), f64(bias), "relu")
    err = np.abs(y - want) - half_step(want)
    assert (err <= 2.0 ** -16 * want).all(), (err / want).max() * 2 ** 16
    got = f64(K().kron_glu_bwd(x, mask, A, B, bias, dy, act="relu")["dx"])
    want = OG.backward(f64(x), f64(mask), f64(A), f64(B), f64(bias), f64(dy), "relu")["dx"]
    err = np.abs(got - want) - half_step(want)
    assert (err <= 2.0 ** -16 * want).all(), (err / want).max() * 2 ** 16


def test_sums_over_many_rows_of_one_sign():
    """The same row four million times: every rounding of a running sum has the same sign.  At most 512 rows are
    summed in one run of at most six additions each (half a unit of the running sum, which grows evenly: 512 * 6 *
    2^-25 of the result), and the runs of a group, at most 256 here, in another (2^-17)."""
    N, r = 2 ** 22 + 5, 16
    print("[glu] many rows of one sign", flush=True)
    g = torch.Generator().manual_seed(3)
    pos = lambda *s: (0.5 + torch.rand(*s, generator=g)).cuda()
    x0, dy0, A, B, bias = pos(1, 1), pos(1, 2), pos(2, r, 1, 2), pos(2, r, 1, 1), pos(2, 2)
    x, dy = x0.expand(N, 1).contiguous(), dy0.expand(N, 2).contiguous()
    got = K().kron_glu_bwd(x, None, A, B, bias, dy, act="relu")
    want = OG.backward(*(f64(v) for v in (x0, None, A, B, bias, dy0)), "relu")
    for key in ("dA", "dB", "dbias"):
        err = np.abs(f64(got[key]) / (N * want[key]) - 1).max()
        assert err <= 512 * 6 * 2.0 ** -25 + 2.0 ** -17, (key, err)


def test_module_with_float32_parameters_and_a_bfloat16_input():
    """The products take the parameters rounded to bfloat16; their gradients are the float32 ones of those (the
    layer's bar, 1e-5 of the largest value), which bfloat16 could hold to 2^-8 alone."""
    from _harness import TOL_F32, rel_err
    torch.manual_seed(2)
    mod = K().KronGLU(8 * 6, 10 * 7, m=6, r=3, n=7, act="gelu", device="cuda")
    with torch.no_grad():
        mod.S.mul_(torch.rand_like(mod.S))
        mod.bias.normal_(std=0.3)
    x = torch.randn(5, 40, 48, device="cuda").to(BF).requires_grad_()
    dy = torch.randn(5, 40, 70, device="cuda").to(BF)
    y = mod(x)
    assert y.dtype == BF and y.shape == (5, 40, 70)
    y.backward(dy)
    h = [f64(x).reshape(200, 48)] + [f64(p.to(BF)) for p in (mod.S, mod.A, mod.B, mod.bias)]
    want = OG.backward(*h, f64(dy).reshape(200, 70), "gelu")
    for key, t in (("dS", mod.S), ("dA", mod.A), ("dB", mod.B), ("dbias", mod.bias)):
        assert t.grad.dtype == F32 and rel_err(f64(t.grad), want[key].reshape(t.shape)) <= TOL_F32, key
    assert x.grad.dtype == BF
    # the other way round stays refused: a float32 input of bfloat16 parameters
    with pytest.raises(ValueError, match="must be torch.float32"):
        mod.to(BF)(x.detach().float())


def test_float32_products():
    """Outputs of one product after another, x B and then C, beside their own size.  Of three bf16 parts the first is
    cut off the top bits and the second rounded: they leave less than 2^-7, at most 2^-16, and nothing, so the terms
    left out of a product are below 2 * 2^-23, and what is left is summed from the small terms up: one rounding of
    its size (2^-24, or 2^-23 if it is cut off)."""
    N = 512
    g = torch.Generator().manual_seed(12)
    pos = lambda *s: (1 + torch.rand(*s, generator=g)).cuda()
    x, A, B = pos(N, 1), pos(2, 1, 1, 64), pos(2, 1, 1, 64)
    A[1] = 0
    bias = torch.zeros(2, 64 * 64, device="cuda")
    bias[1] = 1
    want = OG.forward(*(f64(v) for v in (x, None, A, B, bias)), "relu")
    err = np.abs(f64(K().kron_glu_fwd(x, None, A, B, bias, act="relu")) / want - 1).max()
    assert err <= 2 * (2.0 ** -22 + 2.0 ** -23), err * 2 ** 24
    # the gradient of x through the gate alone: u = 1 (its weight is 0), d = dy, one term a sum
    x, A, B, dy = pos(N, 64 * 64), pos(2, 1, 64, 1), pos(2, 1, 64, 1), pos(N, 1)
    A[1] = 0
    bias = torch.zeros(2, 1, device="cuda")
    bias[1] = 1
    got = f64(K().kron_glu_bwd(x, None, A, B, bias, dy, act="relu")["dx"])
    want = f64(dy)[:, :, None] * (f64(A)[0, 0] * f64(B)[0, 0].T).reshape(1, 1, -1)
    err = np.abs(got / want.reshape(N, -1) - 1).max()
    assert err <= 2 * (2.0 ** -22 + 2.0 ** -23), err * 2 ** 24


def test_float32_values_up_to_the_largest():
    """Values that bf16 rounds to infinity (3.39e38 to fp32's largest) count as themselves."""
    top = torch.finfo(F32).max
    x = torch.tensor([[top, -top], [3.395e38, 1.0]], device="cuda")
    A = torch.tensor([2.0 ** -100, 0.0]).view(2, 1, 1, 1).cuda()
    B = torch.zeros(2, 1, 2, 2, device="cuda")
    B[0, 0] = torch.tensor([[1.0, 0.0], [0.0, 1.0]])
    bias = torch.tensor([[0.0, 0.0], [1.0, 1.0]], device="cuda")
    y = f64(K().kron_glu_fwd(x, None, A, B, bias, act="relu"))
    want = np.maximum(f64(x) * 2.0 ** -100, 0)
    assert (np.abs(y - want) <= 2 * (2.0 ** -22 + 2.0 ** -23) * np.abs(want)).all(), (y, want)

"""KronAdapters as a user's model holds it: converted to bfloat16 after it was made."""
import numpy as np
import pytest

from oracle import adapters as OA

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
u = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def f64(t):
    return t.detach().cpu().double().numpy()


def test_adapters_of_a_converted_model():
    """Forward and backward of a model that .bfloat16() made: y within (K + R + 16) u of the sum of the terms' sizes and a
    last rounding of 2^-8, gradients within (N + 32 + 16) u of theirs and the bf16 parameters' rounding."""
    import kronecker_factored_structured_amd as K
    torch.manual_seed(2)
    mod = torch.nn.Sequential(K.KronAdapters(torch.nn.Linear(32, 24, device="cuda"), 32, 24, rank=5, adapters=3, alpha=0.7, device="cuda"))
    with torch.no_grad():
        mod[0].up.normal_()
    mod.bfloat16()
    m = mod[0]
    x = torch.randn(40, 32, device="cuda").bfloat16().requires_grad_()
    y = mod(x)
    dy = torch.randn(40, 24, device="cuda").bfloat16()
    y.backward(dy)
    ids, starts, scales = np.zeros(1, int), np.array([0, 40]), np.full(3, np.float32(0.7 / 5), np.float64)
    args = (f64(m.down), f64(m.up), ids, starts, scales)
    want, size = OA.forward(f64(x), f64(m.projection(x)), *args)
    assert np.all(np.abs(f64(y) - want) <= 53 * u * size * 1.01 + 2.0 ** -8 * np.abs(want))
    g, size = OA.backward(f64(x), f64(dy), *args)
    for key, t in (("ddown", m.down.grad), ("dup", m.up.grad)):
        assert t.dtype == torch.bfloat16
        assert np.all(np.abs(f64(t) - g[key]) <= 88 * u * size[key] * 1.01 + 2.0 ** -8 * np.abs(g[key])), key

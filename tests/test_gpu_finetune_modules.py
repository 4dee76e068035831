"""KronAdapters and KronVocabCE as a user's model holds them: converted to bfloat16 after it was made, with weights that are
learnt."""
import numpy as np
import pytest

from oracle import adapters as OA
from oracle import vocab_ce as OV

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


def test_adapters_of_an_assigned_state():
    """load_state_dict(assign=True) puts a checkpoint's own tensors in the scales' place, bfloat16 ones too."""
    import kronecker_factored_structured_amd as K

    def model(device):
        return K.KronAdapters(torch.nn.Linear(16, 8, device=device), 16, 8, rank=2, adapters=2, alpha=3.0, device=device)

    torch.manual_seed(5)
    saved = model("cuda").bfloat16()
    with torch.no_grad():
        saved.up.normal_()
    state = {k: v.bfloat16() for k, v in saved.state_dict().items()}
    mod = model("meta")
    mod.load_state_dict(state, assign=True)
    x = torch.randn(5, 16, device="cuda").bfloat16()
    assert torch.equal(mod(x), saved(x))      # (3 / 2 is what bfloat16 holds)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_learnt_weights(dtype):
    """d loss / d weights[n] is the row's own nll; a row of weight 0 is left out, and so is its gradient (0), whatever it
    holds.  Weights of any shape, beside the gradients of h and W or alone."""
    import kronecker_factored_structured_amd as K
    g = torch.Generator().manual_seed(4)
    h, W = torch.randn(3, 7, 16, generator=g).to(dtype).cuda(), torch.randn(50, 16, generator=g).to(dtype).cuda()
    lab = torch.randint(0, 50, (3, 7), generator=g).cuda()
    raw = torch.rand(3, 7, generator=g).cuda()
    raw[1, 2:5] = 0
    h[1, 3], lab[1, 4] = float("nan"), -100
    _, nll, _ = K.kron_vocab_ce_fwd(h.view(21, 16), W, lab.view(21), weights=raw.view(21))
    for others in (False, True):
        leaf = raw.clone().requires_grad_()
        hh, WW = h.clone().requires_grad_(others), W.clone().requires_grad_(others)
        (K.KronVocabCE()(hh, WW, lab, 2 * leaf) * 3).backward()
        assert torch.equal(leaf.grad, 6 * nll.view(3, 7)) and torch.count_nonzero(leaf.grad[1, 2:5]) == 0
        assert (hh.grad is not None) == others and (WW.grad is not None) == others
    keep = torch.tensor([n for n in range(21) if n not in (9, 10, 11)])
    o = OV.forward_backward(f64(h.view(21, 16))[keep], f64(W), lab.view(21).cpu().numpy()[keep])
    # (eps_nll of test_gpu_vocab_ce.py)
    eps = 2 * 36 * u * o["zs"] + u * (4 * (o["z"].max(1) - o["z"].min(1)) + 3 * (50 / 2048 + 64) + 8) + u * (np.abs(o["z"]).max(1) + np.abs(o["nll"]))
    assert np.all(np.abs(f64(nll)[keep] - o["nll"]) <= eps)
    plain = raw.clone()      # (weights that need no gradient get none)
    WW = W.clone().requires_grad_()
    K.KronVocabCE()(h, WW, lab, plain).backward()
    assert plain.grad is None and WW.grad is not None

"""The top logits and the distillation loss over rows whose values are extreme against the temperature: large
maxima, tokens without mass off the kept ones, a teacher that keeps nothing, small temperatures.

Tolerances as for ordinary rows: q and p within REL = 600 * 2^-24 (three roundings of 2^-24 |argument|, the arguments
that leave any mass being below 150 here, and the sums), each gradient against the sum of its terms' sizes and half a
step of its type, the loss against its terms' sizes."""
import numpy as np
import pytest

from _harness import dev
from oracle import distill as OD

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

REL = 600 * 2.0 ** -24
F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def K():
    import kronecker_factored_structured_amd as mod
    return mod


def f64(t):
    return t.detach().cpu().double().numpy()


def within(loss, dz, oracle, dtype, extra=0.0):
    want, g, scale, lscale = oracle
    assert abs(f64(loss)[0] - want) <= (REL + extra) * lscale + 1e-30, (f64(loss)[0], want, lscale)
    half = torch.finfo(dtype).eps / 2
    tol = (REL + extra) * scale + half * (np.abs(g) + REL * scale) + 1e-37
    bad = ~(np.abs(f64(dz) - g) <= tol)      # (a NaN is bad)
    assert not bad.any(), (np.argwhere(bad)[:5], f64(dz)[bad][:5], g[bad][:5])


def check(z, ids, t, lse, lab, w, T, alpha, oracle, dtype, extra=0.0):
    """Loss and gradient in one call and in two, against the oracle's."""
    d = dict(teacher_lse=dev(lse), labels=dev(lab), weights=dev(w), temperature=T, alpha=alpha)
    gi, gt = dev(ids.astype(np.int32)), dev(t)
    out = K().kron_distill(z, gi, gt, **d)
    loss, stats = K().kron_distill_fwd(z, gi, gt, **d)
    dz = K().kron_distill_bwd(z, gi, gt, stats, torch.ones(1, device="cuda"), **d)
    within(out["loss"], out["dlogits"], oracle, dtype, extra)
    within(loss, dz, oracle, dtype, extra)


LARGE = [1e9, -1e9, 1e10, -1e10, -3e10, 1e12, -1e12, 1e20, -1e20, -1e30, 1e37, -1e37]


def large_rows(N, V, dtype):
    """Rows filled with one large value, one of them with the next smaller numbers between, one whose first half is
    far below the rest, one with a large value in ordinary ones."""
    z = torch.randn(N, V, generator=torch.Generator().manual_seed(5)) * 2
    for i, v in enumerate(LARGE):
        z[i] = v
    z[12] = (1 - torch.arange(V).remainder(40) * 2.0 ** -20) * 3e10
    z[13, :V // 2] = -1e30
    z[14, V // 3] = 2e10
    z[15, :V // 2] = 1e10
    z[15, V // 2:] = -1e10
    return z.to(dtype).cuda()


@pytest.mark.parametrize("N", [16, 600])
@pytest.mark.parametrize("T", [0.5, 1.0, 2.0, 30000.0])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_distill_rows_of_large_values(dtype, T, N):
    """Few rows go by chunks, many one to a workgroup (those without weight are not read)."""
    V, k, alpha = 9000, 4, 0.5
    print(f"[distill large] {dtype} T={T} N={N}", flush=True)
    z = large_rows(N, V, dtype)
    g = np.random.default_rng(1)
    ids = np.stack([g.permutation(V)[:k] for _ in range(N)])
    t = g.standard_normal((N, k)).astype(np.float32)
    lab = g.integers(0, V, N)
    lab[14] = V // 3
    ids[13] = V // 2 + ids[13] % (V // 2)
    lab[13] = V - 5
    w = np.zeros(N, np.float32)
    w[:16] = g.uniform(0.2, 1.0, 16)
    for rows, a in ((range(12), alpha), ((12, 13, 14, 15), alpha), ((12, 13, 14, 15), 1.0)):
        wr = np.zeros(N, np.float32)
        wr[list(rows)] = w[list(rows)]
        check(z, ids, t, None, lab, wr, T, a, OD.loss_and_grad(f64(z), ids, t, None, lab, wr, T, a), dtype)


@pytest.mark.parametrize("V", [9000, 131073])
@pytest.mark.parametrize("T", [0.5, 1.0, 2.0, 30000.0])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_topk_rows_of_large_values(dtype, T, V):
    print(f"[topk large] {dtype} T={T} V={V}", flush=True)
    z, k = large_rows(16, V, dtype), 30
    ids, vals, lse = K().kron_topk_logits(z, k, temperature=T)
    wi, wv, wl = OD.topk(f64(z), k, T)
    assert np.array_equal(ids.cpu().numpy(), wi) and np.array_equal(f64(vals), wv)
    assert np.all(np.abs(f64(lse) - wl) <= REL + 4 * 2.0 ** -24 * np.abs(wl)), (f64(lse), wl)

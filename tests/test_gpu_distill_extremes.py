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


@pytest.mark.parametrize("N,V", [(3, 9001), (600, 9001), (2, 140001)])
@pytest.mark.parametrize("T,alpha,gap", [(1.0, 1.0, 150.0), (1.0, 0.5, 150.0), (2.0, 0.5, 290.0), (1.5, 0.5, 200.0), (0.5, 0.7, 75.0)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_distill_kept_tokens_far_above_the_rest(dtype, T, alpha, gap, N, V):
    """The student's mass off the kept tokens is e^-gap/T of the row: no exponential beside the row's maximum holds
    it, but its logarithm and its tokens' shares of it are ordinary numbers."""
    k = 24
    print(f"[distill gap] {dtype} T={T} alpha={alpha} gap={gap} N={N} V={V}", flush=True)
    g = np.random.default_rng(2)
    z = torch.randn(N, V, generator=torch.Generator().manual_seed(5)) * 2
    ids = np.stack([g.permutation(V)[:k] for _ in range(N)])
    t = (g.standard_normal((N, k)) * 2 + 6).astype(np.float32)
    lse = (np.log(np.exp(t.astype(np.float64) / T).sum(1)) + g.uniform(0.01, 0.3, N)).astype(np.float32)
    lab = g.integers(0, V, N)
    lab[1] = ids[1, 3]
    z.scatter_(1, torch.from_numpy(ids), torch.gather(z, 1, torch.from_numpy(ids)) + gap)
    if N > 2:      # only one kept token stands out, and one of the others does as well
        z[2, torch.from_numpy(ids[2, 1:])] -= gap
        z[2, (ids[2, 0] + 1) % V] += 30
    z = z.to(dtype).cuda()
    w = np.zeros(N, np.float32)
    w[:3] = g.uniform(0.2, 1.0, min(N, 3))
    check(z, ids, t, lse, lab, w, T, alpha, OD.loss_and_grad(f64(z), ids, t, lse, lab, w, T, alpha), dtype)


@pytest.mark.parametrize("mask", ["infinity", "lowest", "large"])
@pytest.mark.parametrize("N,V", [(40, 9001), (600, 9001), (4, 140001)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_distill_teacher_and_student_masked_alike(dtype, N, V, mask):
    """Both models allow the same u < k tokens of a row: there is no tail, and what the rounded lse leaves of one is
    no mass.  The loss is the one over the kept tokens, with the teacher's sum off one by the rounding of lse."""
    k, u, T, alpha = 32, 20, 2.0, 0.5
    fill = dict(infinity=-float("inf"), lowest=torch.finfo(dtype).min, large=-1e30)[mask]
    print(f"[distill masked] {dtype} N={N} V={V} {mask}", flush=True)
    g = np.random.default_rng(7)
    gen = torch.Generator().manual_seed(5)
    zt, z = torch.full((N, V), fill), torch.full((N, V), fill)
    live = torch.from_numpy(np.stack([g.permutation(V)[:u] for _ in range(N)]))
    zt.scatter_(1, live, torch.randn(N, u, generator=gen) * 2 + 4)
    z.scatter_(1, live, torch.randn(N, u, generator=gen) * 2)
    zt, z = zt.to(dtype).cuda(), z.to(dtype).cuda()
    ids, vals, lse = K().kron_topk_logits(zt, k, temperature=T)
    ids, t, lse = ids.cpu().numpy(), vals.cpu().numpy(), lse.cpu().numpy()
    lab = live[:, 0].numpy()
    w = np.zeros(N, np.float32)
    w[:40] = g.uniform(0.2, 1.0, min(N, 40))
    want = OD.loss_and_grad(f64(z), ids[:, :u], t[:, :u], None, lab, w, T, alpha)
    # p is off by the rounding of lse and of its sum, below 2^-20 in all
    check(z, ids, t, lse, lab, w, T, alpha, want, dtype, extra=2.0 ** -20)


def test_distill_a_tail_that_the_student_cannot_have():
    """Every logit off the kept tokens is -infinity and the teacher's tail is not small: the loss is infinite, and the
    gradient a number."""
    N, V, k = 3, 500, 8
    z = torch.full((N, V), -float("inf"), device="cuda")
    z[:, :k] = torch.randn(N, k, generator=torch.Generator().manual_seed(1)).cuda()
    z[2] = torch.randn(V, generator=torch.Generator().manual_seed(2)).cuda()
    ids = torch.arange(k, device="cuda", dtype=torch.int32).repeat(N, 1)
    t = torch.zeros(N, k, device="cuda")
    lse = torch.full((N,), float(np.log(k)) + 0.1, device="cuda")
    a = K().kron_distill(z, ids, t, teacher_lse=lse)
    assert a["loss"].item() == float("inf")
    # M q - p on the kept tokens with M = 1, nothing elsewhere
    p = np.exp(-f64(lse)[:2, None]) * np.ones(k)
    q = torch.softmax(z[:2, :k].double(), 1).cpu().numpy()
    assert np.abs(f64(a["dlogits"])[:2, :k] - (q - p) / N).max() <= REL * 2 / N
    assert not a["dlogits"][:2, k:].any() and bool(torch.isfinite(a["dlogits"]).all())


@pytest.mark.parametrize("N", [2, 600])
def test_distill_a_teacher_without_any_value(N):
    """A row of -infinity as kron_topk_logits keeps it: values and lse are -infinity, every p is 0 and the rest of the
    vocabulary has all the mass, whatever lse is."""
    V, k, T = 3000, 6, 1.5
    z = torch.randn(N, V, generator=torch.Generator().manual_seed(4)).cuda()
    ids, vals, lse = K().kron_topk_logits(torch.full((N, V), -float("inf"), device="cuda"), k, temperature=T)
    assert bool((lse == -float("inf")).all())
    ids, t = ids.cpu().numpy(), vals.cpu().numpy()
    w = np.zeros(N, np.float32)
    w[:2] = 0.5
    want = OD.loss_and_grad(f64(z), ids, t, np.zeros(N, np.float32), None, w, T, 1.0)
    check(z, ids, t, lse.cpu().numpy(), None, w, T, 1.0, want, F32)


@pytest.mark.parametrize("N", [4, 600])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("T", [0.003, 0.02])
def test_distill_small_temperatures(T, tail, N):
    """The teacher's values over T are thousands: p = exp of their differences, not of a rounded quotient's.  (The
    calls take T as a 32-bit float; the oracle gets that number.)"""
    T = float(np.float32(T))
    V, k = 4000, 12
    g = np.random.default_rng(9)
    z = torch.randn(N, V, generator=torch.Generator().manual_seed(5)) * T
    ids = np.stack([g.permutation(V)[:k] for _ in range(N)])
    t = (g.standard_normal((N, k)) * T + 20).astype(np.float32)
    lse = None
    if tail:      # (the rounding of an lse of thousands is an input like any other)
        m = t.astype(np.float64).max(1)
        lse = (m / T + np.log(np.exp((t.astype(np.float64) - m[:, None]) / T).sum(1)) + g.uniform(0.1, 0.3, N)).astype(np.float32)
    w = np.zeros(N, np.float32)
    w[:4] = g.uniform(0.2, 1.0, 4)
    z = z.cuda()
    check(z, ids, t, lse, None, w, T, 1.0, OD.loss_and_grad(f64(z), ids, t, lse, None, w, T, 1.0), F32)


def test_loss_module_takes_a_single_row():
    """logits [V] with ids and teacher [k] and nothing before them: one row, as with a leading dimension of one."""
    V, k = 333, 12
    gen = torch.Generator().manual_seed(8)
    z = torch.randn(V, generator=gen).cuda().requires_grad_()
    ids, vals, lse = K().kron_topk_logits(torch.randn(1, V, generator=gen).cuda(), k)
    lab, w = torch.tensor(7, device="cuda"), torch.tensor(0.5, device="cuda")
    mod = K().KronDistillLoss(temperature=2.0, alpha=0.5)
    loss = mod(z, ids[0], vals[0], lse[0], lab, w)
    (g,) = torch.autograd.grad(loss, [z])
    want = mod(z.view(1, V), ids, vals, lse, lab.view(1), w.view(1))
    (gw,) = torch.autograd.grad(want, [z])
    assert loss.shape == () and torch.equal(loss, want) and g.shape == (V,) and torch.equal(g, gw)


@pytest.mark.parametrize("V", [7, 3000, 140000])
def test_topk_lse_of_one_value(V):
    """A row with one finite value z has lse z / T exactly: rounded once (and the quotient in 64 bits)."""
    T = 1.7
    z = torch.full((50, V), -float("inf"))
    v = torch.randn(50, generator=torch.Generator().manual_seed(6)) * 50
    z[:, V // 2] = v
    lse = K().kron_topk_logits(z.cuda(), 2, temperature=T)[2]
    want = v.double().numpy() / float(np.float32(T))
    assert np.all(np.abs(f64(lse) - want) <= 2.0 ** -24 * np.abs(want) * (1 + 2.0 ** -20))


@pytest.mark.parametrize("V,dtype", [(110003, BF), (60001, F32)])
def test_many_rows_of_a_long_vocabulary(V, dtype):
    """Rows that no workgroup's registers hold, more of them than one to a CU: chunks, in one call (in place too) and
    in two.  Most have no weight, so that the oracle has few to do."""
    N, k, T, alpha = 520, 40, 2.0, 0.5
    print(f"[distill long] V={V} {dtype}", flush=True)
    g = np.random.default_rng(3)
    z = (torch.randn(N, V, generator=torch.Generator().manual_seed(5)) * 2).to(dtype).cuda()
    ids = np.stack([g.permutation(V)[:k] for _ in range(N)])
    t = (g.standard_normal((N, k)) * 2 + 6).astype(np.float32)
    lse = (np.log(np.exp(t.astype(np.float64) / T).sum(1)) + g.uniform(0.01, 0.3, N)).astype(np.float32)
    lab = g.integers(0, V, N)
    w = np.zeros(N, np.float32)
    w[5::100] = g.uniform(0.2, 1.0, len(w[5::100]))
    z[105] = -1e10
    z[205, torch.from_numpy(ids[205]).cuda()] += 300
    check(z, ids, t, lse, lab, w, T, alpha, OD.loss_and_grad(f64(z), ids, t, lse, lab, w, T, alpha), dtype)
    args = dict(teacher_lse=dev(lse), labels=dev(lab), weights=dev(w), temperature=T, alpha=alpha)
    want = K().kron_distill(z, dev(ids.astype(np.int32)), dev(t), **args)
    got = K().kron_distill(z, dev(ids.astype(np.int32)), dev(t), out=z, **args)
    assert torch.equal(z, want["dlogits"]) and torch.equal(got["loss"], want["loss"])


def test_distill_a_teacher_without_any_value_far_above_the_rest():
    """teacher_lse of -infinity is no rounding: the rest has all the mass also where the student has next to none there."""
    V, k = 3000, 6
    z = torch.randn(2, V, generator=torch.Generator().manual_seed(4)).cuda()
    z[:, :k] += 150
    ids = np.tile(np.arange(k), (2, 1))
    t, lse = np.full((2, k), -np.inf, np.float32), np.full(2, -np.inf, np.float32)
    want = OD.loss_and_grad(f64(z), ids, t, np.zeros(2, np.float32), None, None, 1.0, 1.0)
    check(z, ids, t, lse, None, None, 1.0, 1.0, want, F32)


@pytest.mark.parametrize("N", [3, 600])
@pytest.mark.parametrize("T", [1.0, 2.0, 1.5])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_label_of_the_lowest_value(dtype, T, N):
    """The cross-entropy of a label that the type's lowest value masks is as large as that, and a number."""
    V, alpha = 700, 0.25
    z = torch.randn(N, V, generator=torch.Generator().manual_seed(3))
    z[1, 50:60] = torch.finfo(dtype).min
    z = z.to(dtype).cuda()
    ids, t = np.tile(np.arange(4), (N, 1)), np.zeros((N, 4), np.float32)
    lab = np.full(N, 55)
    w = np.zeros(N, np.float32)
    w[:3] = 0.25
    check(z, ids, t, None, lab, w, T, alpha, OD.loss_and_grad(f64(z), ids, t, None, lab, w, T, alpha), dtype)


@pytest.mark.parametrize("N,V", [(3, 5001), (600, 5001), (2, 140001)])
@pytest.mark.parametrize("gap", [26.0, 30.0, 50.0, 52.0, 70.0])
def test_distill_a_wide_rest_far_below(gap, N, V):
    """Off the kept tokens, themselves e^-gap of the row, logits spread over 45: e^-45 = 2^-65 of the rest's largest share
    is still a gradient of its own."""
    k = 24
    g = np.random.default_rng(6)
    z = torch.rand(N, V, generator=torch.Generator().manual_seed(5)) * 45
    ids = np.stack([g.permutation(V)[:k] for _ in range(N)])
    z.scatter_(1, torch.from_numpy(ids), 45 + gap + torch.rand(N, k, generator=torch.Generator().manual_seed(6)))
    t = (g.standard_normal((N, k)) * 2 + 6).astype(np.float32)
    lse = (np.log(np.exp(t.astype(np.float64)).sum(1)) + g.uniform(0.01, 0.3, N)).astype(np.float32)
    w = np.zeros(N, np.float32)
    w[:3] = g.uniform(0.2, 1.0, min(N, 3))
    z = z.cuda()
    check(z, ids, t, lse, None, w, 1.0, 1.0, OD.loss_and_grad(f64(z), ids, t, lse, None, w, 1.0, 1.0), F32)

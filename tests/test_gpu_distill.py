"""GPU parity of the teacher's top logits and the distillation loss with the fp64 oracle.

Tolerances.  q = exp((z - m) / T) / total: the exponent carries three roundings (1/T, log2 e and the
product) of 2^-24 |arg|, |arg| <= 60 here, and the exponential one unit; the total a sum of V positive
terms in at most 300 sequential additions.  Together below 600 * 2^-24 = 3.6e-5 of q; the same holds for p.
A gradient is a sum of such terms, so it is off by at most REL times the sum of their sizes, which the
oracle gives, plus half a step of its type."""
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


def rows(N, V, pad, dtype, seed, scale=2.0, off=0):
    """N x V logits in a buffer with `pad` more columns (NaN) and `off` elements before the first row."""
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((off + N * (V + pad),), float("nan"), dtype=dtype, device="cuda")
    z = buf[off:].view(N, V + pad)[:, :V]
    z.copy_((torch.randn(N, V, generator=g) * scale).to(dtype))
    return buf, z


@pytest.mark.parametrize("N,V,k,dtype,T,pad,off", [
    (1, 1, 1, F32, 1.0, 0, 0), (3, 7, 7, BF, 2.0, 1, 3), (4, 255, 200, F32, 1.0, 2, 1), (5, 1000, 256, BF, 1.5, 3, 5),
    (3, 50257, 64, BF, 2.0, 0, 0), (2, 50257, 20, F32, 1.0, 47, 0), (2, 70001, 256, F32, 1.0, 0, 1),
    (2, 140003, 100, BF, 1.0, 0, 0), (1, 262144, 256, F32, 4.0, 0, 0), (1, 262144, 256, BF, 4.0, 0, 0),
    (2, 131072, 33, BF, 1.0, 0, 0), (0, 100, 5, F32, 1.0, 0, 0)])
def test_topk(N, V, k, dtype, T, pad, off):
    print(f"[topk] N={N} V={V} k={k} {dtype} T={T} pad={pad} off={off}", flush=True)
    _, z = rows(N, V, pad, dtype, V + k, off=off)
    ids, vals, lse = K().kron_topk_logits(z, k, temperature=T)
    wi, wv, wl = OD.topk(f64(z), k, T)
    assert np.array_equal(ids.cpu().numpy(), wi)
    assert np.array_equal(f64(vals), wv)
    # the maximum's own rounding (2^-24 |m / T|) and the sum's relative error
    assert np.all(np.abs(f64(lse) - wl) <= REL + 4 * 2.0 ** -24 * np.abs(wl))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("V", [40, 5000, 90000, 200000])
def test_topk_rows_that_defeat_the_threshold(V, dtype):
    """Equal values everywhere, few distinct values, sorted rows, infinities, a block of large ones."""
    print(f"[topk ties] V={V} {dtype}", flush=True)
    k = min(V, 100)
    z = torch.zeros(8, V)
    z[1] = -0.0
    z[1, ::3] = 0.0                                          # zeros of both signs are equal
    z[2] = torch.randint(0, 3, (V,), generator=torch.Generator().manual_seed(1)).float()
    z[3] = torch.arange(V).float()
    z[4] = -torch.arange(V).float()
    z[5] = -float("inf")
    z[5, V // 2] = 1.0
    z[6] = -float("inf")                                     # nothing left
    z[7, 5:25] = torch.finfo(dtype).max
    z[7, 26:] = torch.finfo(dtype).min
    z = z.to(dtype)
    ids, vals, lse = K().kron_topk_logits(z.cuda(), k)
    with np.errstate(invalid="ignore"):
        wi, wv, wl = OD.topk(z.double().numpy(), k)
    assert np.array_equal(ids.cpu().numpy(), wi)
    assert np.array_equal(f64(vals), wv)
    wl[6] = -np.inf
    got = f64(lse)
    assert got[6] == -np.inf
    fin = np.isfinite(wl)
    assert np.all(np.abs(got[fin] - wl[fin]) <= REL + 4 * 2.0 ** -24 * np.abs(wl[fin]))


def test_topk_nan_and_infinity():
    z = torch.randn(3, 3000, generator=torch.Generator().manual_seed(3))
    z[0, 17] = float("nan")
    z[1, 21] = float("inf")
    ids, vals, lse = K().kron_topk_logits(z.cuda(), 4)
    assert ids[0, 0].item() == 17 and torch.isnan(vals[0, 0]) and torch.isnan(lse[0])
    assert ids[1, 0].item() == 21 and vals[1, 0].item() == float("inf") and lse[1].item() == float("inf")
    assert torch.isfinite(lse[2])


def teacher(N, V, k, seed, T, tail):
    g = np.random.default_rng(seed)
    ids = np.stack([g.permutation(V)[:k] for _ in range(N)]) if N else np.zeros((0, k), np.int64)
    t = (np.sort(g.standard_normal((N, k)) * 2, 1)[:, ::-1] + 6).astype(np.float32)
    lse = None
    if tail:
        lse = (np.log(np.exp(t.astype(np.float64) / T).sum(1)) + g.uniform(0.01, 0.3, N)).astype(np.float32)
    w = g.uniform(0.2, 1.0, N).astype(np.float32)
    return ids, t, lse, g.integers(0, V, N), w


def close(loss, dz, z, ids, t, lse, lab, w, T, alpha, dtype, up=1.0):
    want, g, scale, lscale = OD.loss_and_grad(f64(z), ids, t, lse, lab, w, T, alpha)
    if loss is not None:
        assert abs(f64(loss)[0] - want) <= REL * lscale + 1e-30, (f64(loss)[0], want)
    if dz is not None:
        # half a step of the output's type (1e-37 covers the fixed steps under the smallest normal)
        half = torch.finfo(dtype).eps / 2
        tol = REL * scale * up + half * (np.abs(g) + REL * scale) * up + 1e-37
        bad = np.abs(f64(dz) - up * g) > tol
        assert not bad.any(), (np.argwhere(bad)[:5], f64(dz)[bad][:5], up * g[bad][:5])


CASES = [
    (1, 1, 1, F32, 1.0, 1.0, False, 0, 0), (3, 5, 5, F32, 2.0, 0.5, True, 1, 1), (7, 257, 16, BF, 1.5, 1.0, True, 3, 0),
    (4, 1000, 256, F32, 1.0, 0.9, False, 0, 0), (3, 4099, 64, BF, 2.0, 0.5, True, 0, 1), (2, 16391, 7, F32, 4.0, 1.0, True, 2, 3),
    (3, 50257, 64, BF, 2.0, 0.5, True, 0, 0), (2, 50257, 64, F32, 1.0, 0.0, False, 47, 0), (2, 66001, 64, F32, 2.0, 0.5, True, 0, 1),
    (2, 131072, 256, BF, 1.0, 1.0, False, 0, 0), (1, 262144, 256, F32, 2.0, 0.5, True, 0, 0),
    (1, 262143, 256, BF, 2.0, 0.5, True, 1, 1), (0, 100, 4, F32, 1.0, 0.5, False, 0, 0)]


@pytest.mark.parametrize("N,V,k,dtype,T,alpha,tail,pad,off", CASES)
def test_distill(N, V, k, dtype, T, alpha, tail, pad, off):
    print(f"[distill] N={N} V={V} k={k} {dtype} T={T} alpha={alpha} tail={tail} pad={pad} off={off}", flush=True)
    buf, z = rows(N, V, pad, dtype, V, off=off)
    ids, t, lse, lab, w = teacher(N, V, k, k + V, T, tail)
    d = dict(teacher_lse=dev(lse), labels=dev(lab), weights=dev(w), temperature=T, alpha=alpha)
    gi = dev(ids.astype(np.int32))
    out = K().kron_distill(z, gi, dev(t), **d)
    close(out["loss"], out["dlogits"], z, ids, t, lse, lab, w, T, alpha, dtype)
    # 64-bit tokens, and the two calls with an upstream gradient
    loss, stats = K().kron_distill_fwd(z, dev(ids.astype(np.int64)), dev(t), **d)
    assert torch.equal(loss, out["loss"])
    up = torch.tensor([1.75], device="cuda")
    dz = K().kron_distill_bwd(z, gi, dev(t), stats, up, **d)
    close(None, dz, z, ids, t, lse, lab, w, T, alpha, dtype, up=1.75)
    one = K().kron_distill_bwd(z, gi, dev(t), stats, torch.ones(1, device="cuda"), **d)
    assert torch.equal(one, out["dlogits"])
    # in place, and the columns behind V stay as they are
    ref = buf.clone()
    got = K().kron_distill(z, gi, dev(t), out=z, **d)
    assert got["dlogits"] is z and torch.equal(z, out["dlogits"])
    behind = torch.ones_like(ref, dtype=torch.bool)
    behind[off:].view(N, V + pad)[:, :V] = False
    assert torch.equal(torch.isnan(buf[behind]), torch.isnan(ref[behind])) and bool(torch.isnan(buf[behind]).all())


@pytest.mark.parametrize("V,dtype,T,alpha,tail", [
    (700, BF, 2.0, 0.5, True), (20001, BF, 1.0, 0.5, False), (40000, BF, 1.5, 0.5, True), (50257, BF, 2.0, 1.0, True),
    (60001, BF, 2.0, 0.5, True), (100003, BF, 2.0, 0.5, False), (106489, BF, 1.0, 0.0, False), (7000, F32, 2.0, 0.5, True),
    (26600, F32, 1.5, 0.5, True), (53001, F32, 1.0, 1.0, False)])
def test_distill_many_rows(V, dtype, T, alpha, tail):
    """Enough rows for one workgroup per row; most of them without weight, so that the oracle has few to do."""
    N, k = 530, 48
    print(f"[distill rows] V={V} {dtype} T={T} alpha={alpha} tail={tail}", flush=True)
    _, z = rows(N, V, 3, dtype, V)
    ids, t, lse, lab, w = teacher(N, V, k, V, T, tail)
    w[np.arange(N) % 90 != 7] = 0
    ids[97, 5:9] = ids[97, 2]
    ids[187, ::2] = -1
    if tail:
        lse[97] += 3
    d = dict(teacher_lse=dev(lse), labels=dev(lab), weights=dev(w), temperature=T, alpha=alpha)
    gi = dev(ids.astype(np.int32))
    a = K().kron_distill(z, gi, dev(t), **d)
    close(a["loss"], a["dlogits"], z, ids, t, lse, lab, w, T, alpha, dtype)
    got = K().kron_distill(z, gi, dev(t), out=z, **d)      # in place
    assert torch.equal(z, a["dlogits"]) and torch.equal(got["loss"], a["loss"])


@pytest.mark.parametrize("N", [3, 600])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_distill_rows_of_the_lowest_and_largest_values(N, dtype):
    """Rows of the type's lowest value throughout, of its largest one among the lowest, of -infinity but for a few."""
    V, k, T = 9000, 4, 2.0
    _, z = rows(N, V, 0, dtype, 3)
    lo, hi = torch.finfo(dtype).min, torch.finfo(dtype).max
    z[0] = lo
    z[1] = lo
    z[1, 40] = z[1, 8999] = hi
    z[2] = -float("inf")
    z[2, 100:110] = 1.0
    ids = np.tile(np.array([100, 101, 102, 103]), (N, 1))
    ids[1] = [40, 8999, -1, -1]
    t = np.zeros((N, k), np.float32)
    w = np.zeros(N, np.float32)
    w[:3] = 0.5
    lab = np.full(N, 105)
    lab[1] = 40
    d = dict(labels=dev(lab), weights=dev(w), temperature=T, alpha=0.5)
    a = K().kron_distill(z, dev(ids.astype(np.int32)), dev(t), **d)
    close(a["loss"], a["dlogits"], z, ids, t, None, lab, w, T, 0.5, dtype)
    # nothing but -infinity has no distribution: NaN, in its own row only
    z[0] = -float("inf")
    b = K().kron_distill(z, dev(ids.astype(np.int32)), dev(t), **d)
    assert torch.isnan(b["loss"]).all() and torch.isnan(b["dlogits"][0]).all()
    assert torch.equal(b["dlogits"][1:], a["dlogits"][1:])
    # a NaN logit shows
    z[0] = 0
    z[0, 4321] = float("nan")
    b = K().kron_distill(z, dev(ids.astype(np.int32)), dev(t), **d)
    assert torch.isnan(b["loss"]).all() and torch.isnan(b["dlogits"][0]).any() and torch.equal(b["dlogits"][1:], a["dlogits"][1:])


@pytest.mark.parametrize("V", [300, 9001, 140001])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_slots(V, tail):
    """Unused slots, a row without any, a token given several times, a teacher of -infinity, logits of -infinity
    (the vocabulary's masked tokens) and of the lowest value, rows of weight 0 that hold NaN."""
    N, k, T, alpha = 8, 40, 2.0, 0.7
    print(f"[distill slots] V={V} tail={tail}", flush=True)
    _, z = rows(N, V, 5, F32, V)
    ids, t, lse, lab, w = teacher(N, V, k, V, T, tail)
    ids[1, 3:30] = -1
    ids[2] = -1
    ids[3, 20:23] = ids[3, 4]
    ids[3, 24] = ids[3, 5]
    lab[3] = ids[3, 4]
    t[4, 10:] = -np.inf
    free = np.setdiff1d(np.arange(V), np.append(ids[5], lab[5]))[:100]
    z[5, torch.from_numpy(free).cuda()] = -float("inf")
    z[6, torch.from_numpy(np.setdiff1d(np.arange(V), np.append(ids[6], lab[6]))[:50]).cuda()] = torch.finfo(F32).min
    w[7] = 0
    z[7] = float("nan")
    if tail:      # the kept mass of rows with dropped or repeated slots stays below one
        lse[3] += 3.0
    z0 = z.clone()
    zh = f64(z)
    zh[7] = 0
    d = dict(teacher_lse=dev(lse), labels=dev(lab), weights=dev(w), temperature=T, alpha=alpha)
    a = K().kron_distill(z, dev(ids.astype(np.int32)), dev(t), **d)
    close(a["loss"], a["dlogits"], torch.from_numpy(zh), ids, t, lse, lab, w, T, alpha, F32)
    assert not a["dlogits"][7].any()
    b = K().kron_distill(z, dev(ids.astype(np.int32)), dev(t), **d)
    assert torch.equal(a["loss"], b["loss"]) and torch.equal(a["dlogits"], b["dlogits"])
    assert torch.equal(torch.nan_to_num(z), torch.nan_to_num(z0))


def test_distill_all_teacher_values_minus_infinity():
    z = torch.randn(2, 50, device="cuda")
    t = torch.full((2, 4), -float("inf"), device="cuda")
    ids = torch.arange(4, device="cuda", dtype=torch.int32).repeat(2, 1)
    a = K().kron_distill(z, ids, t)
    assert a["loss"].item() == 0 and not a["dlogits"].any()


@pytest.mark.parametrize("what", ["id", "label"])
def test_distill_bad_token_gives_nan(what):
    N, V, k = 3, 777, 5
    _, z = rows(N, V, 0, F32, 1)
    ids, t, lse, lab, w = teacher(N, V, k, 1, 1.0, True)
    good = K().kron_distill(z, dev(ids.astype(np.int32)), dev(t), dev(lse), dev(lab), dev(w), 1.0, 0.5)
    if what == "id":
        ids[1, 2] = V
    else:
        lab[1] = -100
    a = K().kron_distill(z, dev(ids.astype(np.int32)), dev(t), dev(lse), dev(lab), dev(w), 1.0, 0.5)
    assert torch.isnan(a["loss"]).all() and torch.isnan(a["dlogits"][1]).all()
    assert torch.equal(a["dlogits"][0], good["dlogits"][0]) and torch.equal(a["dlogits"][2], good["dlogits"][2])
    loss, stats = K().kron_distill_fwd(z, dev(ids.astype(np.int32)), dev(t), dev(lse), dev(lab), dev(w), 1.0, 0.5)
    dz = K().kron_distill_bwd(z, dev(ids.astype(np.int32)), dev(t), stats, torch.ones(1, device="cuda"), dev(lse), dev(lab),
                              dev(w), 1.0, 0.5)
    assert torch.isnan(loss).all() and torch.isnan(dz[1]).all() and torch.equal(dz[0], good["dlogits"][0])


def test_cross_entropy_alone():
    """alpha = 0 needs no teacher: the mean cross-entropy over a vocabulary."""
    N, V = 9, 5001
    _, z = rows(N, V, 0, F32, 2)
    lab = np.random.default_rng(0).integers(0, V, N)
    a = K().kron_distill(z, None, None, labels=dev(lab), alpha=0.0)
    close(a["loss"], a["dlogits"], z, None, None, None, lab, None, 1.0, 0.0, F32)


def test_gradient_against_differences():
    """The loss along a direction v: (L(z + h v) - L(z - h v)) / 2h is off the slope by h^2 / 6 times the third
    derivative (below 4 here: T^2 = 2.25 times moments of softmax of at most 1, over T^3, v of unit entries) and by
    the losses' rounding (REL * lscale) / h."""
    N, V, k, T, alpha = 4, 400, 20, 1.5, 0.6
    _, z = rows(N, V, 0, F32, 5)
    ids, t, lse, lab, w = teacher(N, V, k, 5, T, True)
    d = dict(teacher_lse=dev(lse), labels=dev(lab), weights=dev(w), temperature=T, alpha=alpha)
    gi = dev(ids.astype(np.int32))
    v = torch.sign(torch.randn(N, V, generator=torch.Generator().manual_seed(9))).cuda()
    h = 2.0 ** -5
    up = K().kron_distill_fwd(z + h * v, gi, dev(t), **d)[0]
    dn = K().kron_distill_fwd(z - h * v, gi, dev(t), **d)[0]
    slope = (f64(up) - f64(dn))[0] / (2 * h)
    got = float((f64(K().kron_distill(z, gi, dev(t), **d)["dlogits"]) * f64(v)).sum())
    lscale = OD.loss_and_grad(f64(z), ids, t, lse, lab, w, T, alpha)[3]
    assert abs(slope - got) <= 4 * w.sum() * h * h / 6 + REL * lscale / h


def test_another_stream_and_a_captured_call():
    """The whole use of the set: the teacher's top logits, then loss and gradient, on a side stream and replayed
    from a graph, every replay against the eager result."""
    V, N, k = 8191, 33, 24
    _, zt = rows(N, V, 0, BF, 11)
    _, z = rows(N, V, 0, BF, 12)
    k_ = K()

    def step(dst=None):
        ids, vals, lse = k_.kron_topk_logits(zt, k, temperature=2.0)
        return k_.kron_distill(z, ids, vals, teacher_lse=lse, temperature=2.0, out=dst)

    ref = step()
    ids, vals, lse = (f64(v) for v in k_.kron_topk_logits(zt, k, temperature=2.0))
    close(ref["loss"], ref["dlogits"], z, ids.astype(int), vals, lse, None, None, 2.0, 1.0, BF)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = step()
        side = step()
    s.synchronize()
    assert torch.equal(side["loss"], ref["loss"]) and torch.equal(side["dlogits"], ref["dlogits"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = step()
    for i in range(3):
        z.copy_(torch.randn(N, V, generator=torch.Generator().manual_seed(i)).to(BF))
        g.replay()
        torch.cuda.synchronize()
        want = step()
        assert torch.equal(cap["loss"], want["loss"]) and torch.equal(cap["dlogits"], want["dlogits"]), i


def test_binding_refusals():
    k = K()
    z = torch.zeros(4, 50, device="cuda")
    ids, t = torch.zeros(4, 3, device="cuda", dtype=torch.int32), torch.zeros(4, 3, device="cuda")
    lab = torch.zeros(4, device="cuda", dtype=torch.int64)

    def bad(match, *a, **kw):
        with pytest.raises(ValueError, match=match):
            k.kron_distill(*a, **kw)

    bad("dense rows", z.t(), ids, t)
    bad("overlap", z[:1].expand(4, 50), ids, t)
    bad("unsupported dtype", z.half(), ids, t)
    bad("ids must be", z, ids[:3], t)
    bad("int32 or int64", z, ids.short(), t)
    bad("teacher", z, ids, t[:, :2].contiguous())
    bad("teacher_lse", z, ids, t, torch.zeros(3, device="cuda"))
    bad("labels are needed", z, ids, t, alpha=0.5)
    bad("labels", z, ids, t, labels=lab.int(), alpha=0.5)
    bad("needed when alpha", z, None, None)
    bad("weights", z, ids, t, weights=torch.zeros(4, 1, device="cuda"))
    bad("out must be", z, ids, t, out=torch.zeros(4, 50, device="cuda", dtype=BF))
    with pytest.raises(ValueError, match="k must be"):
        k.kron_topk_logits(z, 51)
    with pytest.raises(ValueError, match="stats"):
        k.kron_distill_bwd(z, ids, t, torch.zeros(4, 4, device="cuda"), torch.ones(1, device="cuda"))


@pytest.mark.parametrize("V,dtype,T,alpha,tail", [
    (900, F32, 1.5, 0.5, True), (32003, F32, 1.0, 1.0, True), (50257, BF, 2.0, 0.5, False), (106489, BF, 1.0, 0.0, False)])
def test_two_calls_over_many_rows(V, dtype, T, alpha, tail):
    """The forward of many rows keeps the statistics that the backward call takes."""
    N, k = 520, 30
    print(f"[distill two calls] V={V} {dtype} T={T} alpha={alpha} tail={tail}", flush=True)
    _, z = rows(N, V, 1, dtype, V)
    ids, t, lse, lab, w = teacher(N, V, k, V, T, tail)
    w[np.arange(N) % 90 != 7] = 0
    ids[97, 5:9] = ids[97, 2]
    ids[187, ::2] = -1
    if tail:
        lse[97] += 3
    d = dict(teacher_lse=dev(lse), labels=dev(lab), weights=dev(w), temperature=T, alpha=alpha)
    gi = dev(ids.astype(np.int32))
    loss, stats = K().kron_distill_fwd(z, gi, dev(t), **d)
    dz = K().kron_distill_bwd(z, gi, dev(t), stats, torch.tensor([0.5], device="cuda"), **d)
    close(loss, dz, z, ids, t, lse, lab, w, T, alpha, dtype, up=0.5)
    assert bool(torch.isfinite(stats).all()) and not dz[0].any()
    got = K().kron_distill_bwd(z, gi, dev(t), stats, torch.tensor([0.5], device="cuda"), out=z, **d)
    assert got is z and torch.equal(z, dz)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_topk_nan_and_infinity_in_long_rows(dtype):
    """In rows that are cut: a NaN, infinities in several parts, a part of -infinity, fewer than k finite values."""
    V, k = 200001, 50
    z = torch.randn(5, V, generator=torch.Generator().manual_seed(3)).to(dtype)
    z[0, V - 3] = float("nan")
    z[1, 21] = z[1, V - 1] = float("inf")
    z[2, :V // 2] = -float("inf")
    z[3] = -float("inf")
    z[3, [5, V // 2, V - 2]] = torch.tensor([1.0, 3.0, 2.0], dtype=dtype)
    z[4] = 7.0
    ids, vals, lse = K().kron_topk_logits(z.cuda(), k)
    assert ids[0, 0].item() == V - 3 and bool(torch.isnan(vals[0, 0])) and bool(torch.isnan(lse[0]))
    assert ids[1, :2].tolist() == [21, V - 1] and vals[1, 1].item() == float("inf") and lse[1].item() == float("inf")
    for r in range(2, 5):
        wi, wv, wl = OD.topk(f64(z[r:r + 1]), k)
        assert np.array_equal(ids[r].cpu().numpy(), wi[0]) and np.array_equal(f64(vals[r]), wv[0])
        assert abs(lse[r].item() - wl[0]) <= REL + 4 * 2.0 ** -24 * abs(wl[0])


def test_more_rows_than_a_launch_has_workgroups():
    """2^21 + 70 rows of a small vocabulary: the rows behind the first launch are as right as those in it."""
    N, V, k = 2 ** 21 + 70, 6, 2
    print("[rows] topk", flush=True)
    z = torch.randn(N, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    ids, vals, lse = K().kron_topk_logits(z, k)
    v, i = torch.sort(z, dim=1, descending=True, stable=True)
    assert torch.equal(vals, v[:, :k]) and torch.equal(ids, i[:, :k].int())
    assert bool(((lse - torch.logsumexp(z.double(), 1)).abs() <= REL + 4 * 2.0 ** -24 * lse.abs()).all())
    print("[rows] distill", flush=True)
    t = vals * 0.5
    out = K().kron_distill(z, ids, t)
    loss, stats = K().kron_distill_fwd(z, ids, t)
    dz = K().kron_distill_bwd(z, ids, t, stats, torch.ones(1, device="cuda"))
    p = torch.softmax(t.double(), 1)
    q = torch.softmax(z.double(), 1)
    want = q.clone().scatter_add_(1, ids.long(), -p) / N
    # (absolute sizes of a row's terms sum to two)
    for got in (out["dlogits"], dz):
        assert bool(((got.double() - want).abs() <= 2 * REL / N).all())
    kd = (p * (torch.log(p) - torch.log(torch.gather(q, 1, ids.long())))).sum(1)
    scale = (p * (torch.log(p).abs() + torch.log(torch.gather(q, 1, ids.long())).abs())).sum(1).mean()
    for got in (out["loss"], loss):
        assert abs(got.item() - kd.mean().item()) <= REL * float(scale)


@pytest.mark.parametrize("dtype,pad,off", [(F32, 47, 1), (BF, 47, 3), (BF, 0, 5), (F32, 200, 0)])
def test_gradient_rows_stand_like_the_logits(dtype, pad, off):
    """Without `out` the gradients' rows are as far apart and as aligned as the logits', or dense behind wide gaps."""
    N, V, k = 5, 150, 3
    _, z = rows(N, V, pad, dtype, 4, off=off)
    ids, t, _, _, w = teacher(N, V, k, 4, 1.0, False)
    a = K().kron_distill(z, dev(ids.astype(np.int32)), dev(t), weights=dev(w))
    close(a["loss"], a["dlogits"], z, ids, t, None, None, w, 1.0, 1.0, dtype)
    dz = a["dlogits"]
    assert dz.shape == z.shape and dz.stride(1) == 1 and dz.stride(0) == (V if pad >= V else V + pad)
    assert (dz.data_ptr() - z.data_ptr()) % 16 == 0


@pytest.mark.parametrize("dtype", [F32, BF])
def test_loss_module(dtype):
    """KronDistillLoss over a batch of sequences whose vocabulary is padded in memory: the loss and, behind another
    factor, the logits' gradient."""
    Bs, L, V, k, T, alpha = 2, 9, 333, 12, 2.0, 0.5
    _, z = rows(Bs * L, V, 7, dtype, 21)
    ids, t, lse, lab, w = teacher(Bs * L, V, k, 21, T, True)
    w[4] = 0
    leaf = z.view(Bs, L, V).detach().requires_grad_()
    mod = K().KronDistillLoss(temperature=T, alpha=alpha)
    shape = lambda a, *s: dev(a).view(Bs, L, *s)
    loss = mod(leaf, shape(ids.astype(np.int32), k), shape(t, k), shape(lse), shape(lab), shape(w))
    assert loss.shape == () and loss.dtype == F32
    (g,) = torch.autograd.grad(3 * loss, [leaf])
    close(loss.view(1), g.reshape(Bs * L, V), z, ids, t, lse, lab, w, T, alpha, dtype, up=3.0)
    ce = K().KronDistillLoss(alpha=0.0)(leaf, labels=shape(lab))
    close(ce.view(1), None, z, None, None, None, lab, None, 1.0, 0.0, dtype)


def test_loss_module_refusals():
    k = K()
    for kw in (dict(temperature=0.0), dict(alpha=1.5)):
        with pytest.raises(ValueError, match="temperature"):
            k.KronDistillLoss(**kw)
    with pytest.raises(ValueError, match="needed when alpha"):
        k.KronDistillLoss()(torch.zeros(2, 10, device="cuda", requires_grad=True))
    z = torch.randn(2, 10, device="cuda", requires_grad=True)
    ids, t = torch.zeros(2, 1, device="cuda", dtype=torch.int32), torch.zeros(2, 1, device="cuda")
    (g,) = torch.autograd.grad(k.KronDistillLoss()(z, ids, t), [z], create_graph=True)
    with pytest.raises(RuntimeError):      # one derivative only
        g.sum().backward()

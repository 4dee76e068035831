"""The vocabulary cross-entropy at sizes that take each tile of its products, against 64 bits on the GPU.

Tolerances as derived in test_gpu_vocab_ce.py and test_gpu_vocab_ce_extremes.py (u = 2^-24): a logit is off by
eps_z = (K + 20) u S, S = sum |h| |W|, a probability by eps = 2 eps_z + u (4 spread + 3 (V / 2048 + 64) + 8) of itself, the entry
of a row's own label by 4 u of the weight more; dz is rounded to bf16 (2^-8) or to two parts (2^-22, or 2^-50 of the weight, see
test_gpu_vocab_ce_extremes.py); dh and dW sum |dz| times |W| or |h| with (terms + 40) u and are rounded once."""
import pytest

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


def case(N, Kf, V, dtype, skip):
    g = torch.Generator(device="cuda").manual_seed(N + V)
    W = torch.randn(V, Kf, device="cuda", generator=g) * 2.5 * Kf ** -0.5
    lab = torch.randint(0, V, (N,), device="cuda", generator=g)
    h = torch.randn(N, Kf, device="cuda", generator=g) + W[lab] * 0.5
    w = None
    if skip:
        w = torch.rand(N, device="cuda", generator=g) + 0.1
        w[torch.rand(N, device="cuda", generator=g) < skip] = 0
        w[N - 1] = 0.5
        h[w == 0], lab[w == 0] = float("nan"), -1
    return h.to(dtype), W.to(dtype), lab, w


def compare(h, W, lab, w, gout=0.75):
    k = K()
    N, Kf, V = *h.shape, W.shape[0]
    loss, nll, stats = k.kron_vocab_ce_fwd(h, W, lab, weights=w)
    out = k.kron_vocab_ce_bwd(h, W, lab, stats, torch.tensor([gout], device="cuda"), weights=w)
    bf = h.dtype == torch.bfloat16
    wn = torch.full((N,), 1.0 / N, device="cuda", dtype=torch.float64) if w is None else w.double()
    used = torch.nonzero(wn != 0)[:, 0]
    rest = torch.nonzero(wn == 0)[:, 0]
    x, Wd, wn, lab = h[used].double(), W.double(), wn[used], lab[used]
    row = torch.arange(len(used), device="cuda")
    z = x @ Wd.t()
    lse = torch.logsumexp(z, 1)
    want = lse - z[row, lab]
    spread, most = z.max(1).values - z.min(1).values, z.abs().max(1).values
    S = (x.abs() @ Wd.abs().t()).max(1).values
    eps = 2 * (Kf + 20) * u * S + u * (4 * spread + 3 * (V / 2048 + 64) + 8)
    eps_nll = eps + u * (most + want.abs())
    assert bool(((nll[used].double() - want).abs() <= eps_nll).all())
    assert torch.count_nonzero(nll[rest]) == 0 and torch.count_nonzero(out["dh"][rest]) == 0
    assert abs(loss.item() - (wn * want).sum().item()) <= (wn * eps_nll).sum().item() + 2 * u * (wn * want.abs()).sum().item()
    dz = torch.exp(z - lse[:, None])
    del z
    off = dz * eps[:, None] + 2.0 ** -50
    off[row, lab] += 4 * u
    dz[row, lab] -= 1
    dz *= gout * wn[:, None]
    off = off * (gout * wn[:, None]) + dz.abs() * (2.0 ** -8 if bf else 2.0 ** -22)
    size = dz.abs() + off
    r = 2.0 ** -8 if bf else 2 * u
    for key, got, want, bound in (("dh", out["dh"][used], dz @ Wd, off @ Wd.abs() + (V + 40) * u * (size @ Wd.abs())),
                                  ("dW", out["dW"], dz.t() @ x, off.t() @ x.abs() + (N + 40) * u * (size.t() @ x.abs()))):
        assert bool(((got.double() - want).abs() <= bound * (1 + r) + r * want.abs() + 1e-37).all()), key


BF16 = [(63, 2952, 33584), (40, 1787, 51801), (50, 257, 66001), (64, 192, 40007), (3, 100, 52001),                # 256 x 64 and its rows' ends; dh in it
        (8473, 1634, 916), (5966, 500, 6437), (4324, 2114, 1984), (4171, 695, 5716),          # dh in 256 x 256 and 192 x 256, whole and in parts
        (1029, 1063, 1807), (4663, 467, 417), (700, 520, 20001), (6216, 143, 11018),           # dh in 128 x 128; dW in 256 x 256, whole lines, in parts
        (1540, 113, 73929)]                                                                    # two pieces
FP32 = [(100, 333, 30011), (64, 192, 40007), (32, 515, 9001), (8271, 1703, 443), (4171, 695, 5716), (7769, 1410, 1267), (7961, 138, 5122),
        (2738, 249, 1778), (3573, 685, 303), (1768, 168, 11257), (700, 520, 20001), (6657, 14, 20711)]


@pytest.mark.parametrize("skip", [0.0, 0.4])
@pytest.mark.parametrize("N,Kf,V", BF16)
def test_bf16(N, Kf, V, skip):
    compare(*case(N, Kf, V, torch.bfloat16, skip))


@pytest.mark.parametrize("skip", [0.0, 0.4])
@pytest.mark.parametrize("N,Kf,V", FP32)
def test_fp32(N, Kf, V, skip):
    compare(*case(N, Kf, V, torch.float32, skip))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wide_ranges(dtype):
    """More rows than W is taken as it is for: sizes of rows 2^15 apart, of tokens 2^10, of weights 2^30."""
    h, W, lab, _ = case(300, 40, 700, dtype, 0)
    h[::3] *= 2.0 ** -15
    W[::5] *= 2.0 ** -10
    w = torch.rand(300, device="cuda") + 0.5
    w[::7] *= 2.0 ** -30
    compare(h, W, lab, w)
    compare(h * 2.0 ** -60, W * 2.0 ** 60, lab, None)
    compare(h * 40, W, lab, w)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_non_finite_rows_stay_alone(dtype):
    k = K()
    h, W, lab, _ = case(300, 40, 700, dtype, 0)
    good = k.kron_vocab_ce_fwd(h, W, lab)[1]
    h[5, 3], h[70, 0], h[299, 39] = float("nan"), float("inf"), float("-inf")
    loss, nll, stats = k.kron_vocab_ce_fwd(h, W, lab)
    bad = torch.zeros(300, dtype=torch.bool, device="cuda")
    bad[[5, 70, 299]] = True
    assert torch.equal(torch.isfinite(nll), ~bad) and not torch.isfinite(loss).any()
    assert (nll[~bad] - good[~bad]).abs().max().item() <= 1e-4
    out = k.kron_vocab_ce_bwd(h, W, lab, stats, torch.ones(1, device="cuda"))
    assert torch.equal(torch.isfinite(out["dh"]).all(1), ~bad)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_labels_of_no_token(dtype):
    k = K()
    h, W, lab, _ = case(300, 40, 700, dtype, 0)
    for bad in (-1, 700, 1 << 35, -(1 << 50), -(1 << 63), (1 << 63) - 1):
        l2 = lab.clone()
        l2[257] = bad
        loss, nll, stats = k.kron_vocab_ce_fwd(h, W, l2)
        assert torch.isnan(loss).all() and torch.isnan(nll[257]) and torch.isnan(nll).sum() == 1
        out = k.kron_vocab_ce_bwd(h, W, l2, stats, torch.ones(1, device="cuda"))
        assert torch.isnan(out["dh"][257]).all() and torch.isnan(out["dh"]).any(1).sum() == 1
        assert torch.isnan(out["dW"]).all()


@pytest.mark.parametrize("N,dtype", [(128, torch.float32), (129, torch.float32), (300, torch.bfloat16)])
def test_tokens_at_minus_infinity(N, dtype):
    """A token of W at -infinity has probability 0 where W is taken as it is; from 129 rows on fp32 values are two parts, and an
    infinity has none: NaN."""
    k = K()
    h, W, lab, _ = case(N, 40, 300, torch.float32, 0)
    h[:, 0] = 1
    lab[lab == 7] = 8
    keep = torch.tensor([v for v in range(300) if v != 7], device="cuda")
    want = k.kron_vocab_ce_fwd(h.to(dtype), W[keep].to(dtype).contiguous(), lab - (lab > 7).long())[1]
    W[7], W[7, 0] = 0, float("-inf")
    h, W = h.to(dtype), W.to(dtype)
    loss, nll, stats = k.kron_vocab_ce_fwd(h, W, lab)
    out = k.kron_vocab_ce_bwd(h, W, lab, stats, torch.ones(1, device="cuda"))
    if dtype == torch.float32 and N > 128:
        assert torch.isnan(nll).all() and torch.isnan(loss).all()
        return
    assert (nll - want).abs().max().item() <= 1e-5 * want.abs().max().item() + 1e-5
    assert torch.count_nonzero(out["dW"][7]) == 0 and torch.isfinite(out["dW"]).all()
    assert torch.isnan(out["dh"][:, 0]).all() and torch.isfinite(out["dh"][:, 1:]).all()

"""Vocabulary cross-entropy, adapters and orthogonalised update on tensors of more than 2^31 values: what lies behind there is
what it would be on its own.

Tolerances: the bounds that the operators' own tests derive, u = 2^-24; where the same kernels run on a part of a stack, equal."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
u = 2.0 ** -24
LONG = 1 << 31


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of GPU memory")
    yield
    torch.cuda.empty_cache()


def K():
    import kronecker_factored_structured_amd as k
    return k


@pytest.mark.parametrize("N,dtype", [(3, torch.bfloat16), (150, torch.bfloat16), (3, torch.float32), (150, torch.float32)])
def test_vocabulary(N, dtype):
    """W and dW of 2.3e9 values: few rows, and tiles (fp32: of W's copy in two parts)."""
    k = K()
    V, Kf = 140001, 16384
    assert V * Kf > LONG
    g = torch.Generator(device="cuda").manual_seed(N)
    W = torch.randn(V, Kf, device="cuda", generator=g, dtype=dtype).mul_(2.0 * Kf ** -0.5)
    lab = torch.randint(V - 500, V, (N,), device="cuda", generator=g)
    h = (torch.randn(N, Kf, device="cuda", generator=g) + W[lab].float()).to(dtype)
    loss, nll, stats = k.kron_vocab_ce_fwd(h, W, lab)
    out = k.kron_vocab_ce_bwd(h, W, lab, stats, torch.ones(1, device="cuda"))
    hd, z = h.double(), torch.empty(N, V, device="cuda", dtype=torch.float64)
    S = torch.zeros(N, device="cuda", dtype=torch.float64)
    for v in range(0, V, 10000):
        w = W[v:v + 10000].double()
        z[:, v:v + 10000] = hd @ w.t()
        S = torch.maximum(S, (hd.abs() @ w.abs().t()).max(1).values)
    lse = torch.logsumexp(z, 1)
    row = torch.arange(N, device="cuda")
    want = lse - z[row, lab]
    eps = 2 * (Kf + 20) * u * S + u * (4 * (z.max(1).values - z.min(1).values) + 3 * (V / 2048 + 64) + 8)
    assert bool(((nll.double() - want).abs() <= eps + u * (z.abs().max(1).values + want.abs())).all())
    bf = dtype == torch.bfloat16
    r = 2.0 ** -8 if bf else 2 * u
    dz = torch.exp(z - lse[:, None]) / N
    off = dz * eps[:, None] + 2.0 ** -50 / N
    off[row, lab] += 4 * u / N
    dz[row, lab] -= 1.0 / N
    off += dz.abs() * (2.0 ** -8 if bf else 2.0 ** -22)
    size = dz.abs() + off
    dh, bound = torch.zeros_like(hd), torch.zeros_like(hd)
    for v in range(0, V, 10000):
        s = slice(v, v + 10000)
        w = W[s].double()
        dh += dz[:, s] @ w
        bound += off[:, s] @ w.abs() + (V + 40) * u * (size[:, s] @ w.abs())
        if v + 20000 > V or v == 0 or v == 70000:      # both ends of dW, and some of its middle
            want = dz[:, s].t() @ hd
            b = off[:, s].t() @ hd.abs() + (N + 40) * u * (size[:, s].t() @ hd.abs())
            assert bool(((out["dW"][s].double() - want).abs() <= b * (1 + r) + r * want.abs()).all()), v
    assert bool(((out["dh"].double() - dh).abs() <= bound * (1 + r) + r * dh.abs()).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_adapters(dtype):
    """x, dx and y of 2.2e9 values each, y in place: the last request's rows, and its part of the adapter's gradient, beside those
    in front of it."""
    k = K()
    N, Kf, M, R = 540000, 4096, 4000, 20
    assert N * M > LONG
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g, dtype=dtype)
    down, up = r(3, R, Kf), r(3, M, R)
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    ids, starts = [0, 1, 2, -1, 1], [0, 20, 530000, 539000, 539100, 539990]
    x, y = r(N, Kf), r(N, M)
    rows, behind = slice(539100, 539990), slice(539990, N)
    xd, D, U = x[rows].double(), down[1].double(), up[1].double()
    last = 2.0 ** -8 if dtype == torch.bfloat16 else u

    def near(got, want, size, n, rr):
        return bool(((got.double() - want).abs() <= (n + 16) * u * size * (1 + rr) + rr * want.abs()).all())

    want = y[rows].double() + xd @ D.t() @ U.t()
    size = y[rows].double().abs() + xd.abs() @ D.abs().t() @ U.abs().t()
    keep = y[behind].clone()
    k.kron_adapters_fwd(x, y, down, up, dev(ids), dev(starts), out=y)
    assert near(y[rows], want, size, Kf + R, last) and torch.equal(y[behind], keep)
    dy, dyd = y, y[rows].double()
    out = k.kron_adapters_bwd(x, dy, down, up, dev(ids), dev(starts))
    assert near(out["dx"][rows], dyd @ U @ D, dyd.abs() @ U.abs() @ D.abs(), M + R, last)
    assert torch.count_nonzero(out["dx"][behind]) == 0
    # all of adapter 1's rows
    for key, n in (("dup", Kf + N), ("ddown", M + N)):
        want, size = (torch.zeros(out[key].shape[1:], device="cuda", dtype=torch.float64) for _ in range(2))
        for i in [*range(20, 530000, 10000), 539100]:
            s = slice(i, 539990 if i == 539100 else min(i + 10000, 530000))
            for f, total in ((lambda t: t.double(), want), (lambda t: t.double().abs(), size)):
                a, b, d, q = f(x[s]), f(dy[s]), f(down[1]), f(up[1])
                total += b.t() @ (a @ d.t()) if key == "dup" else (b @ q).t() @ a
        assert near(out[key][1], want, size, n, u), key


@pytest.mark.parametrize("shape", [(540000, 64, 63), (540, 2000, 2000)])
def test_update(shape):
    """540,000 matrices in LDS, 540 in groups of tiles: the last ones are those of a stack of them alone."""
    k = K()
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda: torch.randn(*shape, device="cuda", generator=g, dtype=torch.bfloat16)
    W, G = r(), r()
    assert W.numel() > LONG
    m = torch.zeros(shape, device="cuda")
    n = 100 if shape[0] > 1000 else 28      # (540 = 8 groups of 64 and one of 28: the same tiles)
    parts = [t[-n:].clone() for t in (W, G, m)]
    one = [t[:1].clone() for t in (W, G, m)]
    k.kron_muon_step([W], [G], [m], lr=0.1, steps=2)
    k.kron_muon_step(*([t] for t in parts), lr=0.1, steps=2)
    assert torch.equal(W[-n:], parts[0]) and torch.equal(m[-n:], parts[2])
    k.kron_muon_step(*([t] for t in one), lr=0.1, steps=2)
    assert (W[:1].double() - one[0].double()).abs().max().item() <= 0.1 * 16 * 2.0 ** -11 + 2 * 2.0 ** -8 * 6

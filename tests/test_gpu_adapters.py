"""kron_adapters_fwd / kron_adapters_bwd against the fp64 oracle.

Tolerances: every product and sum is fp32 (u = 2^-24): an output that sums n terms in all, inner products among them, is
off by at most (n + 16) u of the sum of the terms' absolute values (the oracle's `size`), and rounded once to its type
(bf16 2^-8)."""
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


def K():
    import kronecker_factored_structured_amd as k
    return k


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def case(seed, N, Kf, M, R, E, lens, dtype, first=0, none=True):
    """Requests of the given lengths from row `first` on."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()
    starts = None if lens is None else torch.tensor(np.cumsum([first, *lens]), dtype=torch.int32).cuda()
    B = N if lens is None else len(lens)
    ids = torch.randint(-1 if none else 0, E, (B,), generator=g).int().cuda()
    return dict(x=r(N, Kf), base=r(N, M), dy=r(N, M), dxb=r(N, Kf), down=r(E, R, Kf), up=r(E, M, R), ids=ids, starts=starts,
                scales=(torch.rand(E, generator=g) + 0.2).cuda())


def compare(c, scales=True, with_base=True):
    k = K()
    sc = c["scales"] if scales else None
    bf = c["x"].dtype == torch.bfloat16
    r = 2.0 ** -8 if bf else u
    N, Kf, M, R = c["x"].shape[0], c["x"].shape[1], c["base"].shape[1], c["down"].shape[1]
    st = None if c["starts"] is None else c["starts"].cpu().numpy()
    ids = c["ids"].cpu().numpy()
    y = k.kron_adapters_fwd(c["x"], c["base"], c["down"], c["up"], c["ids"], c["starts"], sc)
    want, size = OA.forward(f64(c["x"]), f64(c["base"]), f64(c["down"]), f64(c["up"]), ids, st, f64(sc))
    tol = (Kf + R + 16) * u * size
    assert np.all(np.abs(f64(y) - want) <= tol * (1 + r) + r * np.abs(want))
    g = k.kron_adapters_bwd(c["x"], c["dy"], c["down"], c["up"], c["ids"], c["starts"], sc, dx_base=c["dxb"] if with_base else None)
    want, size = OA.backward(f64(c["x"]), f64(c["dy"]), f64(c["down"]), f64(c["up"]), ids, st, f64(sc), f64(c["dxb"]) if with_base else None)
    for key, n, rr in (("dx", M + R, r), ("ddown", M + N, u), ("dup", Kf + N, u)):
        tol = (n + 16) * u * size[key]
        assert np.all(np.abs(f64(g[key]) - want[key]) <= tol * (1 + rr) + rr * np.abs(want[key])), key
    return y, g


LENS = [[1], [0, 1, 0], [16], [17, 15], [5, 0, 33, 2, 16, 1], [100, 3], [1] * 40]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("Kf,M,R", [(16, 16, 16), (7, 9, 3), (130, 70, 20)])
def test_values(lens, Kf, M, R, dtype):
    compare(case(sum(lens) + R, sum(lens), Kf, M, R, 4, lens, dtype))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Kf,M,R", [(1, 1, 1), (768, 2048, 16), (750, 2021, 5), (64, 4096, 33), (2000, 100, 128), (256, 256, 64), (60, 68, 17), (100, 300, 8)])
def test_sizes(Kf, M, R, dtype):
    compare(case(R, 50, Kf, M, R, 3, [20, 1, 29], dtype), scales=R % 2 == 0, with_base=R % 2 == 1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [1, 2, 63, 300])
def test_single_tokens(N, dtype):
    """One row a request, without borders, gives what borders of one row each give."""
    c = case(N, N, 128, 200, 16, 5, None, dtype)
    y, g = compare(c)
    c["starts"] = torch.arange(N + 1, dtype=torch.int32).cuda()
    y2, g2 = compare(c)
    assert torch.equal(y, y2) and torch.equal(g["dx"], g2["dx"])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_requests_and_adapters(dtype):
    g = np.random.default_rng(1)
    lens = list(g.integers(0, 9, 700))
    compare(case(2, sum(lens), 40, 48, 8, 90, lens, dtype))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_adapter_many_rows(dtype):
    """Few columns and many rows: the gradients' rows are shared among workgroups."""
    compare(case(3, 5000, 64, 32, 8, 1, [2999, 2001], dtype, none=False))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Kf,M", [(24, 40), (25, 39)])
def test_rows_of_no_request(Kf, M, dtype):
    """Rows before the first and behind the last request and of requests without an adapter: base's, and left as they are
    in place; nothing of x is read there."""
    k = K()
    c = case(4, 90, Kf, M, 6, 3, [10, 20, 7], dtype, first=13)
    c["ids"] = torch.tensor([1, -1, 2], dtype=torch.int32).cuda()
    out = torch.ones(90, dtype=torch.bool, device="cuda")
    out[13:23] = False
    out[43:50] = False
    y, _ = compare(c)
    assert torch.equal(y[out], c["base"][out])
    c["x"][out] = float("nan")
    c["dy"][out] = float("nan")
    buf = c["base"].clone()
    got = k.kron_adapters_fwd(c["x"], buf, c["down"], c["up"], c["ids"], c["starts"], c["scales"], out=buf)
    assert got is buf and torch.equal(buf, y)
    dx = c["dxb"].clone()
    args = (c["x"], c["dy"], c["down"], c["up"], c["ids"], c["starts"], c["scales"])
    g = k.kron_adapters_bwd(*args, dx_base=dx, outs=dict(dx=dx))
    assert torch.equal(dx[out], c["dxb"][out]) and torch.isfinite(dx).all()
    assert torch.isfinite(g["ddown"]).all() and torch.isfinite(g["dup"]).all() and torch.count_nonzero(g["dup"][0]) == 0
    g2 = k.kron_adapters_bwd(*args, want_dx=False)
    assert g2["dx"] is None and torch.equal(g2["ddown"], g["ddown"]) and torch.equal(g2["dup"], g["dup"])
    g3 = k.kron_adapters_bwd(*args)
    assert torch.count_nonzero(g3["dx"][out]) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ids_of_no_adapter(dtype):
    k = K()
    c = case(5, 40, 16, 24, 4, 3, [10, 20, 10], dtype)
    c["ids"] = torch.tensor([0, 3, 1 << 30], dtype=torch.int32).cuda()
    y = k.kron_adapters_fwd(c["x"], c["base"], c["down"], c["up"], c["ids"], c["starts"], c["scales"])
    assert torch.isnan(y[10:]).all() and torch.isfinite(y[:10]).all()
    g = k.kron_adapters_bwd(c["x"], c["dy"], c["down"], c["up"], c["ids"], c["starts"], c["scales"])
    assert torch.isnan(g["dx"][10:]).all() and torch.isfinite(g["dx"][:10]).all()
    assert torch.isfinite(g["ddown"]).all() and torch.count_nonzero(g["dup"][1:]) == 0


def test_starts_beyond_the_rows():
    """Bounds outside [0, N] count as the nearer one (a batch padded for a captured step)."""
    k = K()
    c = case(6, 32, 16, 16, 4, 3, [8, 8, 8, 8], torch.float32, none=False)
    args = (c["x"], c["base"], c["down"], c["up"], c["ids"])
    want = k.kron_adapters_fwd(*args, c["starts"])
    c["starts"][0], c["starts"][-1] = -100, 1 << 30
    assert torch.equal(k.kron_adapters_fwd(*args, c["starts"]), want)


def test_no_rows():
    k = K()
    c = case(7, 0, 8, 8, 2, 2, [0, 0], torch.float32)
    assert k.kron_adapters_fwd(c["x"], c["base"], c["down"], c["up"], c["ids"], c["starts"]).shape == (0, 8)
    g = k.kron_adapters_bwd(c["x"], c["dy"], c["down"], c["up"], c["ids"], c["starts"])
    assert torch.count_nonzero(g["ddown"]) == 0 and torch.count_nonzero(g["dup"]) == 0


def test_no_requests():
    """Rows of no request at all: y = base, gradients of nothing."""
    k = K()
    c = case(7, 20, 8, 12, 2, 2, [20], torch.float32)
    none, starts = c["ids"][:0], c["starts"][:1]
    assert torch.equal(k.kron_adapters_fwd(c["x"], c["base"], c["down"], c["up"], none, starts), c["base"])
    g = k.kron_adapters_bwd(c["x"], c["dy"], c["down"], c["up"], none, starts)
    assert torch.count_nonzero(g["dx"]) == 0 and torch.count_nonzero(g["ddown"]) == 0 and torch.count_nonzero(g["dup"]) == 0


def test_repeatable():
    k = K()
    c = case(8, 3000, 96, 64, 16, 2, [1700, 1300], torch.bfloat16, none=False)
    args = (c["x"], c["dy"], c["down"], c["up"], c["ids"], c["starts"], c["scales"])
    a = k.kron_adapters_bwd(*args)
    need = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")
    b = k.kron_adapters_bwd(*args, workspace=need)
    for key in a:
        assert torch.equal(a[key], b[key]), key


def test_binding_refuses():
    k = K()
    c = case(9, 20, 8, 12, 4, 3, [10, 10], torch.float32)
    ok = dict(x=c["x"], base=c["base"], down=c["down"], up=c["up"], ids=c["ids"], starts=c["starts"], scales=c["scales"])
    k.kron_adapters_fwd(**ok)
    for key, bad in (("x", c["x"].bfloat16()), ("x", c["x"][:, :7]), ("base", c["base"][:19]), ("down", c["down"][:2]), ("up", c["up"][:, :, :3]),
                     ("ids", c["ids"].long()), ("ids", c["ids"][:1]), ("starts", c["starts"].long()), ("starts", c["starts"][:0]),
                     ("starts", None), ("scales", c["scales"][:1]), ("scales", c["scales"].cpu())):
        with pytest.raises(ValueError):
            k.kron_adapters_fwd(**{**ok, key: bad})
    with pytest.raises(ValueError):
        k.kron_adapters_bwd(c["x"], c["dy"][:, :3], c["down"], c["up"], c["ids"], c["starts"])

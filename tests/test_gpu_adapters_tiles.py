"""kron_adapters_fwd / kron_adapters_bwd over many rows, where a bf16 tile is 32 rows, against 64 bits on the GPU.

Tolerances as in test_gpu_adapters.py: products and sums are fp32, an output of n terms is off by (n + 16) u of the sum of
their absolute values, and rounded once to its type (bf16 2^-8)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
u = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def exact(x, base, dy, down, up, ids, starts, scales, sign):
    """y, dx (from nothing), ddown, dup in 64 bits; of the absolute values where `sign` is false."""
    f = (lambda t: t.double()) if sign else (lambda t: t.double().abs())
    x, dy, down, up, scales, y = f(x), f(dy), f(down), f(up), f(scales), f(base).clone()
    dx, dd, du = torch.zeros_like(x), torch.zeros_like(down), torch.zeros_like(up)
    for i, e in enumerate(ids):
        r = slice(starts[i], starts[i + 1])
        if e < 0 or starts[i] == starts[i + 1]:
            continue
        t, g = scales[e] * (x[r] @ down[e].t()), scales[e] * (dy[r] @ up[e])
        y[r] += t @ up[e].t()
        dx[r] += g @ down[e]
        dd[e] += g.t() @ x[r]
        du[e] += dy[r].t() @ t
    return dict(y=y, dx=dx, ddown=dd, dup=du)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Kf,M,R", [(64, 96, 16), (130, 75, 24), (75, 130, 17), (256, 264, 64), (200, 72, 33), (40, 56, 5), (96, 64, 128)])
def test_many_rows(Kf, M, R, dtype):
    """8,192 rows and more: requests of one row, of none, of a tile and of thousands, some without an adapter, rows before the
    first and behind the last."""
    import kronecker_factored_structured_amd as K
    lens = [33, 0, 1, 32, 31, 64, 4000, 1, 0, 700, 2999, 500, 17, 1]
    first, N, E = 5, sum(lens) + 5 + 11, 4
    g = torch.Generator(device="cuda").manual_seed(R)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g).to(dtype)
    x, base, dy, dxb, down, up = r(N, Kf), r(N, M), r(N, M), r(N, Kf), r(E, R, Kf), r(E, M, R)
    scales = torch.rand(E, device="cuda", generator=g) + 0.2
    starts = [int(v) for v in np.cumsum([first, *lens])]
    ids = [0, 1, 2, -1, 0, 3, 1, 1, 2, -1, 0, 0, 3, 2]
    assert N >= 8192
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    args = (down, up, dev(ids), dev(starts), scales)
    got = K.kron_adapters_bwd(x, dy, *args, dx_base=dxb)
    got["y"] = K.kron_adapters_fwd(x, base, *args)
    want, size = (exact(x, base, dy, down, up, ids, starts, scales, s) for s in (True, False))
    want["dx"] += dxb.double()
    size["dx"] += dxb.double().abs()
    last = 2.0 ** -8 if dtype == torch.bfloat16 else u
    for key, n, rr in (("y", Kf + R, last), ("dx", M + R, last), ("ddown", M + N, u), ("dup", Kf + N, u)):
        off = (got[key].double() - want[key]).abs()
        assert bool((off <= (n + 16) * u * size[key] * (1 + rr) + rr * want[key].abs()).all()), key
    none = torch.ones(N, dtype=torch.bool, device="cuda")
    for i, e in enumerate(ids):
        none[starts[i]:starts[i + 1]] = e < 0
    assert torch.equal(got["y"][none], base[none]) and torch.equal(got["dx"][none], dxb[none])
    # in place, with nothing of the rows without an adapter read
    x[none], dy[none] = float("nan"), float("nan")
    buf, dx = base.clone(), dxb.clone()
    assert torch.equal(K.kron_adapters_fwd(x, buf, *args, out=buf), got["y"])
    again = K.kron_adapters_bwd(x, dy, *args, dx_base=dx, outs=dict(dx=dx))
    for key in ("dx", "ddown", "dup"):
        assert torch.equal(again[key], got[key]), key


def test_ids_of_no_adapter():
    import kronecker_factored_structured_amd as K
    r = lambda *s: torch.randn(*s, device="cuda").bfloat16()
    x, base, dy, down, up = r(8300, 40), r(8300, 56), r(8300, 56), r(3, 20, 40), r(3, 56, 20)
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    args = (down, up, dev([0, 3, 1]), dev([0, 4001, 4100, 8300]))
    bad = torch.zeros(8300, dtype=torch.bool, device="cuda")
    bad[4001:4100] = True
    y = K.kron_adapters_fwd(x, base, *args)
    g = K.kron_adapters_bwd(x, dy, *args)
    for t in (y, g["dx"]):
        assert torch.isnan(t[bad]).all() and torch.isfinite(t[~bad]).all()
    assert torch.isfinite(g["ddown"]).all() and torch.count_nonzero(g["dup"][2]) == 0

"""The vocabulary cross-entropy in fp32 where the gradients' terms are small, tokens that every row finds unlikely, and where
h and W lie at opposite ends of fp32's range.

Tolerances as derived in test_gpu_vocab_ce.py, entry by entry: a logit is off by eps_z = (K + 20) u S, S = sum |h| |W|, and a
probability by eps = 2 eps_z + u (4 spread + 3 (V / 2048 + 64) + 8) of itself.  The entry of a row's own label is a difference,
off by 4 u of the weight more; every other entry of dz is off by eps of itself and its two parts' rounding, 2^-22 of itself or
2^-50 of the weight: a second part that is subnormal is off by 2^-25 over 2^15 and 2^11, 2^-51, and as much is left out with the
product of both second parts, where dz's is at most 2^-25 over 2^15 (its first one is subnormal) and h's 2^-11 of h.  dW sums N
of them times h with (N + 40) u, dh V of them times W."""
import numpy as np
import pytest

from oracle import vocab_ce as OV

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
    return t.detach().cpu().double().numpy()


def compare(h, W, lab, w, g=0.75):
    k = K()
    loss, nll, stats = k.kron_vocab_ce_fwd(h, W, lab, weights=w)
    out = k.kron_vocab_ce_bwd(h, W, lab, stats, torch.tensor([g], device="cuda"), weights=w)
    o = OV.forward_backward(f64(h), f64(W), lab.cpu().numpy(), None if w is None else f64(w), gout=g)
    N, Kf, V = h.shape[0], h.shape[1], W.shape[0]
    used, wn = o["used"], np.abs(o["w"][o["used"]])
    spread = o["z"].max(1) - o["z"].min(1)
    eps = 2 * (Kf + 20) * u * o["zs"] + u * (4 * spread + 3 * (V / 2048 + 64) + 8)
    assert np.all(np.abs(f64(nll)[used] - o["nll"][used]) <= eps + u * (np.abs(o["z"]).max(1) + np.abs(o["nll"][used])))
    label = np.arange(V) == lab.cpu().numpy()[used][:, None]
    ddz = abs(g) * wn[:, None] * (o["p"] * eps[:, None] + 4 * u * label + 2.0 ** -50) + np.abs(o["dz"]) * 2.0 ** -22
    sz = np.abs(o["dz"]) + ddz
    bound = ddz @ np.abs(f64(W)) + (V + 40) * u * (sz @ np.abs(f64(W)))
    assert np.all(np.abs(f64(out["dh"])[used] - o["dh"][used]) <= bound * (1 + 2 * u) + 2 * u * np.abs(o["dh"][used]))
    bound = ddz.T @ np.abs(o["x"]) + (N + 40) * u * (sz.T @ np.abs(o["x"]))
    off = np.abs(f64(out["dW"]) - o["dW"])
    assert np.all(off <= bound * (1 + 2 * u) + 2 * u * np.abs(o["dW"]) + 1e-37), (off / bound).max()
    return o, off


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("N,Kf,V", [(5, 24, 300), (40, 24, 700), (100, 24, 500), (200, 24, 700), (700, 24, 400)])
def test_unlikely_tokens(N, Kf, V, weights):
    """Half of the vocabulary lies 10 to 30 below the rest in every row, at probabilities of 1e-6 to 1e-14: their dW has
    its own digits.  (h's first value is 8 and W's lowers them by it, so that the sums S stay small.)"""
    g = torch.Generator().manual_seed(N + V)
    W = torch.randn(V, Kf, generator=g) * 0.3 * Kf ** -0.5
    h = torch.randn(N, Kf, generator=g)
    h[:, 0] = 8
    low = torch.arange(V) % 2 == 1
    W[:, 0] = 0
    W[low, 0] = -(1.25 + 2.5 * torch.rand(int(low.sum()), generator=g))
    lab = torch.randint(0, V // 2, (N,), generator=g) * 2
    w = None
    if weights:
        w = torch.rand(N, generator=g) + 0.1
        w[torch.rand(N, generator=g) < 0.3] = 0
        w[0] = 1
        w = w.cuda()
    o, off = compare(h.cuda(), W.cuda(), lab.cuda(), w)
    # of a token's largest gradient: 2e-3 down to probabilities of 1e-12 (2^-50 is 8.9e-4 of that, eps up to 2e-4)
    likely = o["p"].max(0)
    rows = np.abs(o["dW"]).max(1)
    assert (likely < 1e-9).any() and (likely < 1e-11).any()
    assert np.all((off.max(1) <= 2e-3 * rows)[likely > 1e-12])


@pytest.mark.parametrize("N", [20, 60, 110, 200])
@pytest.mark.parametrize("up", [-121, -100, 100, 121])
def test_operands_at_the_ends_of_the_range(N, up):
    """h 2^up and W 2^-up: the logits and the losses are those of h and W, bit by bit; dh is 2^-up of theirs, dW 2^up.  (Every
    scale is a power of two; gradients that fp32 has no normal number for are left out.)"""
    k = K()
    g = torch.Generator().manual_seed(N)
    h, W = torch.randn(N, 40, generator=g).cuda(), (torch.randn(300, 40, generator=g) * 0.4).cuda()
    h, W = (torch.where(t.abs() < 2.0 ** -5, torch.full_like(t, 0.25), t) for t in (h, W))      # (normal at either end)
    lab, gout = torch.randint(0, 300, (N,), generator=g).cuda(), torch.ones(1, device="cuda")

    def times(t, e):
        return torch.ldexp(torch.ldexp(t, torch.tensor(e // 2, device="cuda")), torch.tensor(e - e // 2, device="cuda"))

    outs = []
    for a, b in ((h, W), (times(h, up), times(W, -up))):
        loss, nll, stats = k.kron_vocab_ce_fwd(a, b, lab)
        outs.append((nll, k.kron_vocab_ce_bwd(a, b, lab, stats, gout)))
    assert torch.equal(outs[0][0], outs[1][0])
    for key, e in (("dh", -up), ("dW", up)):
        want, got = times(outs[0][1][key].double(), e), outs[1][1][key].double()
        there = want.abs() >= 2.0 ** -100
        assert bool(torch.isfinite(got).all())
        assert torch.equal(got[there], want[there]), key
        assert bool((got[~there].abs() < 2.0 ** -99).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [40, 200])
@pytest.mark.parametrize("heavier,up", [(100, 0), (-100, 0), (120, -60), (125, -90), (-100, 60), (-90, 100)])
def test_weights_at_the_ends_of_the_range(N, heavier, up, dtype):
    """Weights 2^heavier, h 2^up and W 2^-up: dh is 2^(heavier - up) and dW 2^(heavier + up) of what they are without, bit by bit,
    where that is within the range."""
    k = K()
    g = torch.Generator().manual_seed(N)
    h, W = torch.randn(N, 40, generator=g).cuda(), (torch.randn(300, 40, generator=g) * 0.4).cuda()
    h, W = (torch.where(t.abs() < 2.0 ** -5, torch.full_like(t, 0.25), t).to(dtype) for t in (h, W))
    w = (torch.rand(N, generator=g) + 0.5).cuda()
    lab, gout = torch.randint(0, 300, (N,), generator=g).cuda(), torch.ones(1, device="cuda")

    def times(t, e):
        return (t.double() * 2.0 ** e).to(t.dtype)

    outs = []
    for a, b, c in ((h, W, w), (times(h, up), times(W, -up), times(w, heavier))):
        _, _, stats = k.kron_vocab_ce_fwd(a, b, lab, weights=c)
        outs.append(k.kron_vocab_ce_bwd(a, b, lab, stats, gout, weights=c))
    for key, e in (("dh", heavier - up), ("dW", heavier + up)):
        want, got = outs[0][key].double() * 2.0 ** e, outs[1][key].double()
        there = (want.abs() >= 2.0 ** -100) & (want.abs() < 2.0 ** 127)
        assert torch.equal(got[there], want[there]), key

"""kron_vocab_ce_fwd / kron_vocab_ce_bwd against the fp64 oracle.

Tolerances, derived from the roundings (u = 2^-24).  An fp32 operand as two fp16 parts is off by at most 2^-22 of it
(two roundings of 2^-11), and the product of the two second parts, at most 2^-22 of the terms', is left out: 3 * 2^-22
= 12 u of sum |h| |W|; bf16 operands are exact.  The sums over K are fp32: at most (K + 8) u more of the same sum, S.  So
a logit is off by eps_z = (K + 20) u S.  The exponential takes the rounded product with log2(e): a relative error of
2 u |z - max| + 4 u.  The sums of a row take the tile's values one after the other (at most 32), then join tiles: at
most V / 2048 + 64 additions in a row, each of which may also rescale by an exponential (2 more roundings):
  eps_nll = 2 eps_z + u (4 spread + 3 (V / 2048 + 64) + 8) + u (|max| + |nll|)      (spread: of the row's logits)
and a probability is off by that much of itself.  dz = w (p - [label]) is then off by w p eps_nll + 2 u w, and rounded: to
bf16 (2^-8) or to two parts (2^-22).  dh and dW sum |dz| times |W| or |h| with (terms + 20) u, and are rounded once to
their type.  (dz of the row's label is a difference: its bound goes by w, not by dz.)"""
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


def case(seed, N, Kf, V, dtype, skip=0.0, scale=2.5):
    g = torch.Generator().manual_seed(seed)
    W = torch.randn(V, Kf, generator=g) * scale * Kf ** -0.5
    lab = torch.randint(0, V, (N,), generator=g)
    h = torch.randn(N, Kf, generator=g) + W[lab] * 0.5
    w = None
    if skip:
        w = torch.rand(N, generator=g) + 0.1
        w[torch.rand(N, generator=g) < skip] = 0
        w = w.cuda()
    return h.to(dtype).cuda(), W.to(dtype).cuda(), lab.cuda(), w


def compare(h, W, lab, w, g=0.75, dead=False):
    """Forward and backward against the oracle within the bounds above."""
    k = K()
    loss, nll, stats = k.kron_vocab_ce_fwd(h, W, lab, weights=w)
    out = k.kron_vocab_ce_bwd(h, W, lab, stats, torch.tensor([g], device="cuda"), weights=w)
    hh = f64(h)
    if dead:
        hh = np.where(np.isnan(hh), 0, hh)
    labs = lab.cpu().numpy()
    o = OV.forward_backward(hh, f64(W), np.where((labs < 0) | (labs >= W.shape[0]), 0, labs) if dead else labs, None if w is None else f64(w), gout=g)
    bf, N, Kf, V = h.dtype == torch.bfloat16, h.shape[0], h.shape[1], W.shape[0]
    used, wn = o["used"], np.abs(o["w"][o["used"]])
    spread = o["z"].max(1) - o["z"].min(1) if len(used) else np.zeros(0)
    eps = 2 * (Kf + 20) * u * o["zs"] + u * (4 * spread + 3 * (V / 2048 + 64) + 8) + u * (np.abs(o["z"]).max(1, initial=0) + np.abs(o["nll"][used]))
    assert np.all(np.abs(f64(nll)[used] - o["nll"][used]) <= eps)
    rest = np.setdiff1d(np.arange(N), used)
    assert np.all(f64(nll)[rest] == 0)
    lsize = (wn * np.abs(o["nll"][used])).sum()
    assert abs(loss.item() - o["loss"]) <= (wn * eps).sum() + 2 * u * lsize
    ddz = abs(g) * wn[:, None] * (o["p"] * eps[:, None] + 4 * u) + np.abs(o["dz"]) * (2.0 ** -8 if bf else 2.0 ** -22)
    sz = np.abs(o["dz"]) + ddz
    out_r = 2.0 ** -8 if bf else 2 * u
    bound = ddz @ np.abs(f64(W)) + (V + 40) * u * (sz @ np.abs(f64(W)))
    dh = f64(out["dh"])
    assert np.all(np.abs(dh[used] - o["dh"][used]) <= bound * (1 + out_r) + out_r * np.abs(o["dh"][used]) + 1e-37)
    assert np.all(dh[rest] == 0)
    bound = ddz.T @ np.abs(o["x"]) + (N + 40) * u * (sz.T @ np.abs(o["x"]))
    assert np.all(np.abs(f64(out["dW"]) - o["dW"]) <= bound * (1 + out_r) + out_r * np.abs(o["dW"]) + 1e-37)
    return loss, nll, out


SHAPES = [(1, 1, 1), (1, 8, 2), (3, 5, 7), (2, 64, 256), (37, 64, 500), (64, 100, 257), (65, 128, 255), (64, 750, 1003),
          (129, 96, 1025), (257, 768, 513), (300, 66, 3001)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,Kf,V", SHAPES)
def test_values(N, Kf, V, dtype):
    compare(*case(N * 7 + V, N, Kf, V, dtype))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,Kf,V,skip", [(3, 5, 7, 0.5), (64, 64, 300, 0.5), (130, 100, 600, 0.9), (700, 64, 1500, 0.1), (1100, 72, 400, 0.6)])
def test_rows_left_out(N, Kf, V, skip, dtype):
    """Rows of weight 0 hold NaN and labels of no token: nothing of them is used."""
    h, W, lab, w = case(N, N, Kf, V, dtype, skip)
    w[0] = 0
    h[w == 0] = float("nan")
    lab[w == 0] = 1 << 40
    compare(h, W, lab, w, dead=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_no_row_left(dtype):
    k = K()
    h, W, lab, _ = case(0, 70, 24, 90, dtype)
    w = torch.zeros(70, device="cuda")
    loss, nll, stats = k.kron_vocab_ce_fwd(h, W, lab, weights=w)
    out = k.kron_vocab_ce_bwd(h, W, lab, stats, torch.ones(1, device="cuda"), weights=w)
    for t in (loss, nll, out["dh"], out["dW"]):
        assert torch.count_nonzero(t) == 0
    loss, nll, stats = k.kron_vocab_ce_fwd(h[:0], W, lab[:0])
    out = k.kron_vocab_ce_bwd(h[:0], W, lab[:0], stats, torch.ones(1, device="cuda"))
    assert loss.item() == 0 and nll.numel() == 0 and out["dh"].shape == (0, 24) and torch.count_nonzero(out["dW"]) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_several_pieces(dtype):
    """A vocabulary in more than one piece: the gradient of all of it is over the workspace's bound."""
    N, Kf, V = (4100, 40, 70000) if dtype == torch.bfloat16 else (2100, 40, 70000)
    k = K()
    assert k.kron_vocab_ce_workspace_bytes(N, Kf, V, dtype, False, True) < N * V * 2 * (2 if dtype == torch.float32 else 1)
    h, W, lab, _ = case(5, N, Kf, V, dtype)
    hd, Wd = h.double(), W.double()
    z = hd @ Wd.t()
    lse = torch.logsumexp(z, 1)
    row = torch.arange(N, device="cuda")
    nll_want = lse - z[row, lab]
    dz = torch.exp(z - lse[:, None])
    dz[row, lab] -= 1
    dz /= N
    loss, nll, stats = k.kron_vocab_ce_fwd(h, W, lab)
    out = k.kron_vocab_ce_bwd(h, W, lab, stats, torch.ones(1, device="cuda"))
    zs = (hd.abs() @ Wd.abs().t()).max().item()
    eps = 2 * (Kf + 20) * u * zs + u * (4 * 40 + 3 * (V / 2048 + 64) + 60)
    assert (nll.double() - nll_want).abs().max().item() <= eps
    r = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -22
    size = dz.abs() * (r + eps + 40 * u) + 4 * u / N
    out_r = 2.0 ** -8 if dtype == torch.bfloat16 else 2 * u
    for got, want, bound in ((out["dh"], dz @ Wd, (size + V * u * dz.abs()) @ Wd.abs()), (out["dW"], dz.t() @ hd, (size + N * u * dz.abs()).t() @ hd.abs())):
        assert bool(((got.double() - want).abs() <= 1.01 * bound + out_r * want.abs()).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_labels_of_no_token(dtype):
    k = K()
    h, W, lab, _ = case(3, 20, 16, 50, dtype)
    good, _, _ = k.kron_vocab_ce_fwd(h, W, lab)
    for bad in (-1, 50, 1 << 35, -(1 << 50)):
        l2 = lab.clone()
        l2[7] = bad
        loss, nll, stats = k.kron_vocab_ce_fwd(h, W, l2)
        assert torch.isnan(loss).all() and torch.isnan(nll[7]) and torch.isnan(nll).sum() == 1
        out = k.kron_vocab_ce_bwd(h, W, l2, stats, torch.ones(1, device="cuda"))
        assert torch.isnan(out["dh"][7]).all() and torch.isnan(out["dh"]).any(1).sum() == 1
        assert torch.isnan(out["dW"]).all()
    assert torch.isfinite(good).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_non_finite_rows_stay_alone(dtype):
    k = K()
    h, W, lab, _ = case(4, 80, 16, 300, dtype)
    h[5, 3], h[70, 0] = float("nan"), float("inf")
    loss, nll, stats = k.kron_vocab_ce_fwd(h, W, lab)
    bad = torch.zeros(80, dtype=torch.bool, device="cuda")
    bad[[5, 70]] = True
    assert torch.equal(torch.isfinite(nll), ~bad)
    out = k.kron_vocab_ce_bwd(h, W, lab, stats, torch.ones(1, device="cuda"))
    assert torch.equal(torch.isfinite(out["dh"]).all(1), ~bad)
    o = OV.forward_backward(f64(h[~bad]), f64(W), lab[~bad].cpu().numpy())
    assert np.abs(f64(nll[~bad]) - o["nll"]).max() <= 1e-4


def test_tokens_at_minus_infinity():
    """A token whose logit is -infinity in every row has probability 0 (its row of W is -infinity where h is 1)."""
    k = K()
    h, W, lab, _ = case(6, 33, 16, 40, torch.float32)
    h[:, 0] = 1
    W[7, 0] = float("-inf")
    W[7, 1:] = 0
    lab[lab == 7] = 8
    loss, nll, stats = k.kron_vocab_ce_fwd(h.bfloat16(), W.bfloat16(), lab)
    keep = torch.tensor([v for v in range(40) if v != 7], device="cuda")
    o = OV.forward_backward(f64(h.bfloat16()), f64(W[keep].bfloat16()), (lab - (lab > 7).long()).cpu().numpy())
    assert np.abs(f64(nll) - o["nll"]).max() <= 1e-5 * max(1, np.abs(o["nll"]).max())
    dW = k.kron_vocab_ce_bwd(h.bfloat16(), W.bfloat16(), lab, stats, torch.ones(1, device="cuda"))["dW"]
    assert torch.count_nonzero(dW[7]) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wide_ranges(dtype):
    """Logits in the hundreds, rows and tokens whose sizes lie 2^40 apart, weights 2^30 apart."""
    compare(*case(8, 90, 32, 300, dtype, scale=60.0))
    h, W, lab, _ = case(9, 90, 32, 300, dtype)
    h[::3] *= 2.0 ** -30
    W[::5] *= 2.0 ** -10
    w = torch.rand(90, device="cuda") + 0.5
    w[::7] *= 2.0 ** -30
    compare(h, W, lab, w)
    compare(h * 2.0 ** -60, W * 2.0 ** 60, lab, None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_repeatable_and_workspace_ignored(dtype):
    k = K()
    h, W, lab, w = case(10, 200, 72, 900, dtype, 0.3)
    g = torch.ones(1, device="cuda")
    first = None
    for fill in (0, 255, 127):
        def ws(b):
            return torch.full((k.kron_vocab_ce_workspace_bytes(200, 72, 900, dtype, True, b),), fill, dtype=torch.uint8, device="cuda")
        loss, nll, stats = k.kron_vocab_ce_fwd(h, W, lab, weights=w, workspace=ws(False))
        out = k.kron_vocab_ce_bwd(h, W, lab, stats, g, weights=w, workspace=ws(True))
        got = [loss, nll, out["dh"], out["dW"]]
        first = first or got
        for a, b in zip(first, got):
            assert torch.equal(a, b)
    only = k.kron_vocab_ce_bwd(h, W, lab, stats, g, weights=w, want_dh=False)
    assert only["dh"] is None and torch.equal(only["dW"], first[3])
    only = k.kron_vocab_ce_bwd(h, W, lab, stats, g, weights=w, want_dW=False)
    assert only["dW"] is None and torch.equal(only["dh"], first[2])


def test_many_rows_against_blocks_of_them():
    """Rows' results do not depend on the rows beside them: 5000 at once, in another order and in blocks (bf16: the operands
    are not scaled).  Another number of rows may take other tiles, whose sums of exponentials come in another order: each
    of the two is within eps_nll (above) of the exact value, so they are within 2 eps_nll of each other."""
    k = K()
    h, W, lab, _ = case(11, 5000, 64, 700, torch.bfloat16)
    _, nll, _ = k.kron_vocab_ce_fwd(h, W, lab)
    order = torch.randperm(5000, generator=torch.Generator().manual_seed(1)).cuda()
    assert torch.equal(k.kron_vocab_ce_fwd(h[order].contiguous(), W, lab[order].contiguous())[1], nll[order])
    parts = [k.kron_vocab_ce_fwd(h[i:i + 1250].contiguous(), W, lab[i:i + 1250].contiguous())[1] for i in range(0, 5000, 1250)]
    z = h.double() @ W.double().t()
    zs = (h.double().abs() @ W.double().abs().t()).max(1).values
    eps = 2 * (64 + 20) * u * zs + u * (4 * (z.max(1).values - z.min(1).values) + 3 * (700 / 2048 + 64) + 8) \
        + u * (z.abs().max(1).values + nll.double().abs())
    assert bool(((nll.double() - torch.cat(parts).double()).abs() <= 2 * eps).all())


def test_equal_weights_are_not_rounded():
    """bf16: weights of 1 / N each, and none at all, give the same gradients, and so do weights of any size but for their
    size: what is rounded to bf16 is (softmax - [label]) over the largest weight, the same in all three.  c dW is then off
    from c times dW by the last roundings alone, half a step of each."""
    k = K()
    N = 300
    h, W, lab, _ = case(13, N, 64, 700, torch.bfloat16)
    g = torch.ones(1, device="cuda")
    outs = []
    for w in (None, torch.full((N,), 1 / N, device="cuda"), torch.full((N,), 0.77, device="cuda")):
        _, _, stats = k.kron_vocab_ce_fwd(h, W, lab, weights=w)
        outs.append(k.kron_vocab_ce_bwd(h, W, lab, stats, g, weights=w))
    for key in ("dh", "dW"):
        assert torch.equal(outs[0][key], outs[1][key])
        a, b = outs[0][key].double() * (0.77 * N), outs[2][key].double()
        assert bool(((a - b).abs() <= (2.0 ** -8 + 8 * u) * (a.abs() + b.abs())).all())


def test_binding_refuses():
    k = K()
    h, W, lab, w = case(12, 10, 8, 20, torch.float32, 0.2)
    for bad in (lambda: k.kron_vocab_ce_fwd(h.cpu(), W, lab), lambda: k.kron_vocab_ce_fwd(h, W.bfloat16(), lab),
                lambda: k.kron_vocab_ce_fwd(h, W[:, :4], lab), lambda: k.kron_vocab_ce_fwd(h, W, lab.int()),
                lambda: k.kron_vocab_ce_fwd(h, W, lab[:3]), lambda: k.kron_vocab_ce_fwd(h, W, lab, weights=w.double()),
                lambda: k.kron_vocab_ce_fwd(h.t(), W, lab), lambda: k.kron_vocab_ce_fwd(h.half(), W.half(), lab)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ValueError):
        k.kron_vocab_ce_bwd(h, W, lab, torch.zeros(10, 3, device="cuda"), torch.ones(1, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,Kf,V", [(1, 7, 31), (1, 70, 4000), (15, 33, 129), (16, 130, 127), (17, 333, 700), (33, 36, 2000), (50, 257, 1100),
                                    (64, 1001, 300), (65, 68, 900), (100, 190, 515), (128, 65, 3001)])
def test_few_rows(N, Kf, V, dtype):
    compare(*case(N + Kf, N, Kf, V, dtype))
    h, W, lab, w = case(N + V, N, Kf, V, dtype, 0.4)
    h[w == 0] = float("nan")
    compare(h, W, lab, w, dead=True)


def test_few_rows_of_any_address_are_refused():
    """Operands that start one value into their storage: addresses are multiples of 16 bytes, rows of any width."""
    k = K()
    h, W, lab, _ = case(9, 9, 77, 400, torch.float32)
    moved = torch.zeros(h.numel() + 1, device="cuda")[1:].view(h.shape)
    with pytest.raises(k._lib.KronError):
        k.kron_vocab_ce_fwd(moved, W, lab)


def test_few_rows_and_tokens_at_infinity():
    """A token of W at -infinity changes no other token's logit, whatever K is."""
    k = K()
    h, W, lab, _ = case(16, 33, 45, 200, torch.float32)
    h[:, 0] = 1
    W[7], W[7, 0] = 0, float("-inf")
    lab[lab == 7] = 8
    keep = torch.tensor([v for v in range(200) if v != 7], device="cuda")
    for t in (torch.float32, torch.bfloat16):
        _, nll, _ = k.kron_vocab_ce_fwd(h.to(t), W.to(t), lab)
        o = OV.forward_backward(f64(h.to(t)), f64(W[keep].to(t)), (lab - (lab > 7).long()).cpu().numpy())
        assert np.abs(f64(nll) - o["nll"]).max() <= 1e-5 * max(1, np.abs(o["nll"]).max())

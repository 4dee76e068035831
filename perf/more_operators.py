"""Cases of the vocabulary head's cross-entropy, the adapters of many requests and the orthogonalised update:
what a pass reads, computes and returns, in elementary torch operations and in the library's calls.

The three are what a step of fine-tuning a language model of Kronecker layers needs next to the layers: low-rank
adapters beside a projection (and the same adapters in serving, many requests of different adapters at once), the
loss through a large vocabulary from the hidden states, and the update of factors, adapters and dense matrices.
Sizes: the 768-wide GPT-2 small block and the 1024-wide layers of the benchmark, GPT-2's vocabulary, a generic
one, and the factors of those layers.
"""
import math

import torch

own = False

COEFFS = (3.4445, -4.7750, 2.0315)      # of the quintic of one Newton-Schulz step


# ---------------------------------------------------------------------------------- cases
def _head(name, op, N, K, V, dtype, skip=0.0):
    return dict(name=name, op=op, N=N, K=K, V=V, dtype=dtype, skip=skip)


def _adapt(name, op, N, B, E, K, M, R, dtype, none=0.0):
    return dict(name=name, op=op, N=N, B=B, E=E, K=K, M=M, R=R, dtype=dtype, none=none)


def _muon(name, shapes, copies, dtype, nesterov=True, decay=0.0):
    return dict(name=name, op="muon", shapes=shapes, copies=copies, dtype=dtype, nesterov=nesterov, decay=decay)


def listed():
    return [
        # the likelihood of a short text under GPT-2 small's head: a few ragged rows
        _head("head fwd 37 x 768 x 50257", "head_fwd", 37, 768, 50257, "bf16"),
        # scoring a batch of texts in fp32 (a generic vocabulary), every tenth position is padding
        _head("head fwd 2050 x 1024 x 32003", "head_fwd", 2050, 1024, 32003, "f32", skip=0.1),
        # loss and gradients of a training batch of 8 x 1024 tokens, GPT-2 small's head
        _head("head train 8192 x 768 x 50257", "head_train", 8192, 768, 50257, "bf16"),
        # fine-tuning on answers: half of the positions are the prompt's and have no weight; fp32, odd width
        _head("head train 1001 x 750 x 32003", "head_train", 1001, 750, 32003, "f32", skip=0.5),
        # one token of one request through its adapter, as a served model calls it: latency counts
        _adapt("adapters one token", "adapters_fwd", 1, 1, 8, 768, 2048, 16, "bf16"),
        # a step of 64 requests with 32 adapters, one new token each, some without an adapter
        _adapt("adapters 64 tokens", "adapters_fwd", 64, 64, 32, 1024, 4096, 16, "bf16", none=0.1),
        # prompts of 24 requests, 8192 tokens together, in fp32 with a rank that fills no tile
        _adapt("adapters prompts", "adapters_fwd", 8192, 24, 8, 1024, 1024, 24, "f32", none=0.1),
        # gradients of eight adapters trained at once on one batch of 32 texts
        _adapt("adapters bwd 8192 x 768-2048", "adapters_bwd", 8192, 32, 8, 768, 2048, 16, "bf16"),
        # gradients over a few short texts, odd widths
        _adapt("adapters bwd 301 x 750-2021", "adapters_bwd", 301, 7, 3, 750, 2021, 5, "f32", none=0.2),
        # the factors of twelve gated blocks, 768 -> 2048 in four ranks: many small matrices
        _muon("muon factors", "2x4x32x64+2x4x24x32", 12, "f32"),
        # one dense projection of the 1024-wide model
        _muon("muon 1024 x 1024", "1024x1024", 1, "f32", decay=0.01),
        # feed-forward matrices and an adapter's pair, parameters and gradients in bf16, tall and wide
        _muon("muon bf16 set", "768x2048+2048x768+16x768+2048x16", 2, "bf16", nesterov=False, decay=0.1),
    ]


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


_MOST = {}


def draw(rng):
    """One more case of the same ranges; its rows (or matrices) are cut until it costs no more than the largest listed
    case of its operator."""
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("head_fwd", "head_train", "adapters_fwd", "adapters_bwd", "muon", "muon"))
    dtype = rng.choice(("bf16", "f32"))
    if op.startswith("head"):
        c = dict(op=op, N=log(1, 8192), K=log(48, 2048), V=log(500, 131072), dtype=dtype, skip=rng.choice((0.0, 0.1, 0.5)))
    elif op.startswith("adapters"):
        N = log(1, 8192)
        c = dict(op=op, N=N, B=min(N, log(1, 256)), E=log(1, 64), K=log(24, 4096), M=log(24, 4096), R=log(1, 64), dtype=dtype,
                 none=rng.choice((0.0, 0.1, 0.5)))
    else:
        kind = rng.choice(("factors", "dense", "adapter"))
        if kind == "factors":
            shapes = "%dx%dx%d" % (rng.randint(1, 8), log(3, 64), log(3, 64))
        elif kind == "dense":
            shapes = "%dx%d" % (log(65, 1024), log(65, 2048))
        else:
            r, k = log(1, 64), log(65, 4096)
            shapes = rng.choice(("%dx%d" % (r, k), "%dx%d" % (k, r)))
        c = dict(op=op, shapes=shapes, copies=rng.randint(1, 24 if kind == "factors" else 3), dtype=dtype, nesterov=rng.random() < 0.5,
                 decay=rng.choice((0.0, 0.01, 0.1)))
    if not _MOST:
        for x in listed():
            _MOST[x["op"]] = max(_MOST.get(x["op"], 0), _cost(x))
    cut = "copies" if op == "muon" else "N"
    while c[cut] > 1 and _cost(c) > _MOST[op]:
        c[cut] = c[cut] * 7 // 8
        if "B" in c:
            c["B"] = min(c["B"], c["N"])
    return c


def _shapes(c):
    return [tuple(int(v) for v in s.split("x")) for s in c["shapes"].split("+")] * c["copies"]


def work(case):
    c, es = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"].startswith("head"):
        N, K, V = c["N"], c["K"], c["V"]
        used = max(1, round(N * (1 - c["skip"])))
        if c["op"] == "head_fwd":      # labels and weights in, the rows' losses out
            return dict(bytes=es * (used * K + V * K) + 16 * N, flops=2 * used * K * V)
        # the logits and the two products of their gradient
        return dict(bytes=es * (used * K + N * K + 2 * V * K) + 16 * N, flops=6 * used * K * V)
    if c["op"].startswith("adapters"):
        N, E, K, M, R = (c[k] for k in ("N", "E", "K", "M", "R"))
        rows = max(1, round(N * (1 - c["none"])))
        params = min(E, c["B"]) * R * (K + M)
        if c["op"] == "adapters_fwd":
            return dict(bytes=es * (rows * K + 2 * N * M + params), flops=2 * rows * R * (K + M))
        # x, dy and the projection's dx in, dx and the adapters' gradients (fp32) out; the two inner products
        # again, dx, and both gradients
        return dict(bytes=es * (rows * (K + M) + 2 * N * K + params) + 4 * E * R * (K + M), flops=2 * rows * R * (3 * K + 2 * M))
    total = dict(bytes=0, flops=0)
    for s in _shapes(c):
        n = math.prod(s)
        a, l = min(s[-2:]), max(s[-2:])
        # parameters and momentum in and out, gradients in; per step two symmetric products and a whole one
        total["bytes"] += n * (3 * es + 8)
        total["flops"] += 5 * (n // (a * l)) * (3 * a * a * l + a * a * a)
    return total


# ---------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dt)

    if c["op"].startswith("head"):
        N, K, V = c["N"], c["K"], c["V"]
        # logits of about 2.5, the label's raised by about 5; the frequent tokens have the low numbers
        W = normal(V, K, scale=2.5 * K ** -0.5)
        labels = (torch.rand(N, device="cuda", generator=g) ** 3 * V).long().clamp(max=V - 1)
        h = torch.randn(N, K, device="cuda", generator=g) + W[labels].float() * 0.8
        s = dict(case=c, h=h.to(dt), W=W, labels=labels, w=None, up=torch.rand(1, device="cuda", generator=g) + 0.5)
        if c["skip"]:
            w = (torch.rand(N, device="cuda", generator=g) >= c["skip"]).float()
            w[0] = 1.0
            s["w"] = w / w.sum()
        return s
    if c["op"].startswith("adapters"):
        N, B, E, K, M, R = (c[k] for k in ("N", "B", "E", "K", "M", "R"))
        s = dict(case=c, x=normal(N, K), down=normal(E, R, K, scale=K ** -0.5), up=normal(E, M, R, scale=R ** -0.5),
                 scales=torch.rand(E, device="cuda", generator=g) * 2 + 0.1)
        ids = torch.randint(0, E, (B,), device="cuda", generator=g)
        ids = torch.where(torch.rand(B, device="cuda", generator=g) < c["none"], torch.full_like(ids, -1), ids)
        s["ids"], s["starts"] = ids.int(), None
        if N != B:      # requests of uneven lengths; a step of single tokens needs no borders
            cut = torch.sort(torch.randint(0, N + 1, (B - 1,), device="cuda", generator=g))[0]
            end = torch.tensor([0, N], device="cuda")
            s["starts"] = torch.cat([end[:1], cut, end[1:]]).int()
        if c["op"] == "adapters_fwd":
            s["base"] = normal(N, M)
        else:
            s["dy"], s["base"] = normal(N, M), normal(N, K)
        return s
    s = dict(case=c, W=[], G=[], m=[])
    for shape in _shapes(c):
        rows, cols = shape[-2:]
        k = max(1, min(rows, cols) // 4)
        # a gradient: a part of low rank, as a batch gives it, and noise
        low = torch.randn(*shape[:-2], rows, k, device="cuda", generator=g) @ torch.randn(*shape[:-2], k, cols, device="cuda", generator=g).contiguous()
        s["W"].append(normal(*shape, scale=rows ** -0.5))
        s["G"].append((low * (1e-3 * k ** -0.5) + torch.randn(*shape, device="cuda", generator=g) * 3e-4).to(dt))
        s["m"].append(torch.randn(*shape, device="cuda", generator=g) * 3e-3)
    return s


LR, MU = 0.02, 0.95


def _gain(shape):
    return math.sqrt(max(1.0, shape[-2] / shape[-1]))


# ---------------------------------------------------------------------------------- plain forms
def _plain_head(s):
    c = s["case"]
    h, W, lab = s["h"].float(), s["W"].float(), s["labels"][:, None]
    N = h.shape[0]
    w = s["w"] if s["w"] is not None else torch.full((N,), 1.0 / N, device=h.device)
    z = h @ W.t()
    top = z.max(1, keepdim=True)[0]
    at = torch.gather(z, 1, lab) - top
    z = torch.exp(z - top)
    total = z.sum(1, keepdim=True)
    nll = (torch.log(total) - at)[:, 0] * (w != 0)
    loss = (w * nll).sum().reshape(1)
    if c["op"] == "head_fwd":
        return dict(loss=loss, nll=nll)
    dz = (z / total).scatter_add(1, lab, -torch.ones_like(total)) * (w * s["up"])[:, None]
    return dict(loss=loss, nll=nll, dh=(dz @ W).to(s["h"].dtype), dW=(dz.t() @ h).to(s["W"].dtype))


def _plain_adapters(s):
    c = s["case"]
    N, E, R = c["N"], c["E"], c["R"]
    x, D, U = s["x"].float(), s["down"].float(), s["up"].float()
    row = torch.arange(N, device=x.device)
    at = row if s["starts"] is None else torch.searchsorted(s["starts"][1:].contiguous(), row.int(), right=True)
    ids = s["ids"].long()[at]
    # every adapter's products, and a row's own of them: scale where the adapter is the row's, else 0
    mine = ((ids[:, None] == torch.arange(E, device=x.device)) * s["scales"])[:, :, None]
    D = D.reshape(E * R, -1)
    U = U.permute(0, 2, 1).reshape(E * R, -1)
    t = ((x @ D.t()).reshape(N, E, R) * mine).reshape(N, E * R)
    if c["op"] == "adapters_fwd":
        return (s["base"].float() + t @ U).to(s["x"].dtype)
    dy = s["dy"].float()
    g = ((dy @ U.t()).reshape(N, E, R) * mine).reshape(N, E * R)
    return dict(dx=(s["base"].float() + g @ D).to(s["x"].dtype), ddown=(g.t() @ x).reshape(E, R, -1),
                dup=(dy.t() @ t).reshape(-1, E, R).permute(1, 0, 2).contiguous())


def _plain_muon(s):
    c = s["case"]
    a, b, k = COEFFS
    for W, G, m in zip(s["W"], s["G"], s["m"]):
        grad = G.float()
        m.mul_(MU).add_(grad)
        u = grad + MU * m if c["nesterov"] else m
        tall = u.shape[-2] > u.shape[-1]
        X = (u.transpose(-1, -2) if tall else u).reshape(-1, *sorted(u.shape[-2:])).contiguous()
        X = X / (torch.sqrt((X * X).sum((1, 2), keepdim=True)) + 1e-7)
        for _ in range(5):
            A = X @ X.transpose(1, 2).contiguous()
            X = a * X + (b * A + k * (A @ A)) @ X
        X = (X.transpose(1, 2) if tall else X).reshape(u.shape)
        W.copy_(W.float() * (1 - LR * c["decay"]) - (LR * _gain(W.shape)) * X)
    return dict(W=s["W"], m=s["m"])


# ---------------------------------------------------------------------------------- one pass
def run(state):
    s, c = state, state["case"]
    if not own:
        return (_plain_head if c["op"].startswith("head") else _plain_adapters if c["op"].startswith("adapters") else _plain_muon)(s)
    import kronecker_factored_structured_amd as K
    if c["op"].startswith("head"):
        loss, nll, stats = K.kron_vocab_ce_fwd(s["h"], s["W"], s["labels"], weights=s["w"])
        if c["op"] == "head_fwd":
            return dict(loss=loss, nll=nll)
        g = K.kron_vocab_ce_bwd(s["h"], s["W"], s["labels"], stats, s["up"], weights=s["w"])
        return dict(loss=loss, nll=nll, dh=g["dh"], dW=g["dW"])
    if c["op"] == "adapters_fwd":
        return K.kron_adapters_fwd(s["x"], s["base"], s["down"], s["up"], s["ids"], starts=s["starts"], scales=s["scales"])
    if c["op"] == "adapters_bwd":
        return K.kron_adapters_bwd(s["x"], s["dy"], s["down"], s["up"], s["ids"], starts=s["starts"], scales=s["scales"], dx_base=s["base"])
    K.kron_muon_step(s["W"], s["G"], s["m"], lr=LR, momentum=MU, nesterov=c["nesterov"], weight_decay=c["decay"],
                     scales=[_gain(w.shape) for w in s["W"]])
    return dict(W=s["W"], m=s["m"])


# ---------------------------------------------------------------------------------- 64 bits
def _exact_head(s):
    c, lab = s["case"], s["labels"]
    N, V = lab.shape[0], c["V"]
    W = s["W"].double()
    w = torch.full((N,), 1.0 / N, device=W.device, dtype=torch.float64) if s["w"] is None else s["w"].double()
    nll, dh, dW = [], [], torch.zeros_like(W)
    step = max(1, (1 << 27) // V)
    for i in range(0, N, step):
        h, l, v = s["h"][i:i + step].double(), lab[i:i + step], w[i:i + step]
        logp = torch.log_softmax(h @ W.t(), 1)
        row = torch.arange(l.shape[0], device=l.device)
        nll.append(-logp[row, l] * (v != 0))
        if c["op"] == "head_train":
            # d nll / d logit = softmax - the label's indicator
            dz = torch.exp(logp)
            dz[row, l] -= 1
            dz *= (v * s["up"].double())[:, None]
            dh.append(dz @ W)
            dW += dz.t() @ h
    nll = torch.cat(nll)
    out = dict(loss=(w * nll).sum().reshape(1), nll=nll)
    return out if c["op"] == "head_fwd" else dict(out, dh=torch.cat(dh), dW=dW)


def _exact_adapters(s):
    """Request by request: y = base + scale (x D^T) U^T, and the gradients of sum(dy y)."""
    c = s["case"]
    out = s["base"].double().clone()
    dD, dU = torch.zeros_like(s["down"], dtype=torch.float64), torch.zeros_like(s["up"], dtype=torch.float64)
    borders = list(range(c["N"] + 1)) if s["starts"] is None else s["starts"].tolist()
    for i, e in enumerate(s["ids"].tolist()):
        rows = slice(borders[i], borders[i + 1])
        if e < 0 or borders[i] == borders[i + 1]:
            continue
        x, D, U, f = s["x"][rows].double(), s["down"][e].double(), s["up"][e].double(), s["scales"][e].double()
        t = x @ D.t()
        if c["op"] == "adapters_fwd":
            out[rows] += f * (t @ U.t())
            continue
        dy = s["dy"][rows].double()
        dt = f * (dy @ U)
        out[rows] += dt @ D
        dD[e] += dt.t() @ x
        dU[e] += f * (dy.t() @ t)
    return out if c["op"] == "adapters_fwd" else dict(dx=out, ddown=dD, dup=dU)


def _exact_muon(s):
    """The steps act on the singular values alone: X = P diag(v) Q^T becomes P diag(f(..f(v))) Q^T with
    f(v) = a v + b v^3 + c v^5, here through the eigenvectors of X X^T."""
    c = s["case"]
    if sum(math.prod(v) * min(v[-2:]) for v in _shapes(c)) > 6e9:
        return None
    out = dict(W=[], m=[])
    for W, G, m in zip(s["W"], s["G"], s["m"]):
        grad = G.double()
        m = MU * m.double() + grad
        u = (grad + MU * m if c["nesterov"] else m).cpu()
        tall = u.shape[-2] > u.shape[-1]
        x = (u.mT if tall else u).reshape(-1, *sorted(u.shape[-2:]))
        x = x / (torch.linalg.matrix_norm(x, keepdim=True) + 1e-7)
        lam, P = torch.linalg.eigh(x @ x.mT)
        lam = lam.clamp(min=0)
        q = torch.ones_like(lam)
        for _ in range(5):
            f = COEFFS[0] + lam * (COEFFS[1] + lam * COEFFS[2])
            q, lam = q * f, lam * f * f
        o = (P * q[:, None, :]) @ (P.mT @ x)
        o = (o.mT if tall else o).reshape(u.shape).to(W.device)
        out["W"].append(W.double() * (1 - LR * c["decay"]) - LR * _gain(W.shape) * o)
        out["m"].append(m)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return (_exact_head if op.startswith("head") else _exact_adapters if op.startswith("adapters") else _exact_muon)(s)

"""Timed cases of the operators that train a draft head beside its plain matrix
products: the embedding lookup with its gradient, the gated block's two
projections with their product, and the cross entropy of an output layer whose
logits are never kept.

`run` makes either the library's calls (`own`) or the same computation in
elementary torch operations in float32, rounded once at the end.  `exact` has
the definitions in float64.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_TORCH = {BF16: torch.bfloat16, F32: torch.float32}
_SIZE = {BF16: 2, F32: 4}
PAD = -1  # token of a padded position


# ------------------------------------------------------------------- cases
def _embedding(name, tokens, vocab, width, dtype, scale, pad, backward):
    return {"name": name, "op": "embedding", "tokens": tokens, "vocab": vocab, "width": width,
            "dtype": dtype, "scale": scale, "pad": pad, "backward": backward}


def _gated(name, m, n, k, dtype, act, backward):
    return {"name": name, "op": "gated", "m": m, "n": n, "k": k, "dtype": dtype, "act": act,
            "backward": backward}


def _entropy(name, m, vocab, k, dtype, bias, masked, pad, lse, backward):
    return {"name": name, "op": "entropy", "m": m, "vocab": vocab, "k": k, "dtype": dtype,
            "bias": bias, "masked": masked, "pad": pad, "lse": lse, "backward": backward}


def listed():
    return [
        # one request's K+1 = 6 verify positions: the smallest call, where
        # latency counts
        _embedding("embedding_one_request", 6, 128256, 4096, BF16, 1.0, 0.0, False),
        # a training batch of packed sequences, embeddings scaled by the root
        # of their width; the gradient is a whole table
        _embedding("embedding_training", 16384, 128256, 4096, BF16, 64.0, 0.1, True),
        # fp32, an odd vocabulary and an odd width
        _embedding("embedding_f32_odd", 3001, 50257, 777, F32, 1.0, 0.2, True),
        # a gated block's projections for one token
        _gated("gated_one_token", 1, 14336, 4096, BF16, "silu", False),
        # the same for the verify positions of 32 requests with 5 drafts
        _gated("gated_verify_batch", 192, 14336, 4096, BF16, "silu", False),
        # in training
        _gated("gated_training", 8192, 14336, 4096, BF16, "silu", True),
        # odd sizes, fp32
        _gated("gated_f32_odd", 301, 1001, 777, F32, "gelu", True),
        # scoring one verified request's tokens
        _entropy("entropy_one_request", 6, 128256, 4096, BF16, False, 0.0, 0.0, False, False),
        # a training batch over the benchmark's vocabulary, prompt positions
        # padded, with a penalty on the log of the softmax sum
        _entropy("entropy_training", 8192, 128256, 4096, BF16, False, 0.0, 0.1, True, True),
        # a smaller head on packed sequences, most of whose positions are prompt
        _entropy("entropy_small_head", 2048, 32000, 1024, BF16, False, 0.0, 0.6, False, True),
        # an odd vocabulary, its bias masking tokens that may not be sampled
        _entropy("entropy_masked_odd", 1001, 50257, 768, BF16, True, 0.2, 0.1, True, True),
        # odd sizes, fp32
        _entropy("entropy_f32_odd", 77, 32001, 515, F32, True, 0.0, 0.1, False, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["embedding", "gated", "entropy"])
    dtype = rng.choice([BF16, BF16, F32])
    whole = rng.random() < 0.6  # the usual widths: whole 64s
    if op == "embedding":
        width, vocab = _log_int(rng, 64, 8192), _log_int(rng, 1000, 262144)
        if whole:
            width = -(-width // 64) * 64
        vocab = max(1000, min(vocab, 500000000 // width))
        n = _log_int(rng, 1, min(32768, 130000000 // width))
        return {"op": op, "tokens": n, "vocab": vocab, "width": width, "dtype": dtype,
                "scale": rng.choice([1.0, math.sqrt(width), 0.5]), "pad": rng.choice([0.0, 0.1, 0.5]),
                "backward": rng.random() < 0.6}
    most = 1.0e12 if dtype == BF16 else 5e10
    m, k = _log_int(rng, 1, 8192), _log_int(rng, 64, 8192)
    if whole:
        k = -(-k // 64) * 64
    backward = rng.random() < 0.6
    if op == "gated":
        n = _log_int(rng, 64, 28672)
        n = max(64, min(n, int(0.4 * most / (m * k))))
        if whole:
            n = -(-n // 64) * 64
        # relu's slope jumps at 0: in float32 a sum of products that rounds to
        # the other side of 0 moves the gradients by more than rounding does
        acts = ["silu", "silu", "gelu", "none"] + ([] if backward else ["relu"])
        return {"op": op, "m": m, "n": n, "k": k, "dtype": dtype, "act": rng.choice(acts),
                "backward": backward}
    vocab = _log_int(rng, 1000, 262144)
    vocab = max(1000, min(vocab, int(most / (m * k)), 500000000 // k))
    if whole:
        vocab = -(-vocab // 64) * 64
    bias = rng.random() < 0.4
    return {"op": op, "m": m, "vocab": vocab, "k": k, "dtype": dtype, "bias": bias,
            "masked": rng.choice([0.0, 0.2]) if bias else 0.0, "pad": rng.choice([0.0, 0.1, 0.6]),
            "lse": rng.random() < 0.5, "backward": backward}


def work(case):
    e = _SIZE[case["dtype"]]
    if case["op"] == "embedding":
        n, h = case["tokens"], case["width"]
        live = n * (1 - case["pad"])
        # rows that are looked up are read once each; of tokens that come as
        # these do about a third of the calls' positions are the first of theirs
        nbytes = n * 4 + n * h * e + min(live, case["vocab"]) * h * e / 3
        if case["backward"]:
            nbytes += live * h * e + case["vocab"] * h * e
        return {"bytes": nbytes, "flops": n * h * (2 if case["backward"] else 1)}
    if case["op"] == "gated":
        m, n, k = case["m"], case["n"], case["k"]
        nbytes = (m * k + 2 * n * k + m * n) * e
        flops = 4.0 * m * n * k
        if case["backward"]:  # the gradient of y is read, those of x and both weights written
            nbytes += (m * n + m * k + 2 * n * k) * e
            flops *= 3
        return {"bytes": nbytes, "flops": flops}
    m, v, k = case["m"] * (1 - case["pad"]), case["vocab"], case["k"]
    nbytes = (m * k + v * k + (v if case["bias"] else 0)) * e + case["m"] * 12
    flops = 2.0 * m * v * k
    if case["backward"]:
        nbytes += (case["m"] * k + v * k + (v if case["bias"] else 0)) * e
        flops *= 3
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------ inputs
def _tokens(g, n, vocab, pad):
    """Tokens as text has them, the i-th most frequent about 1 / i of the time,
    their numbers in no order of frequency; some positions padded."""
    rank = torch.exp(torch.rand(n, generator=g, device="cuda", dtype=torch.float64) * math.log(vocab + 1))
    rank = (rank.long() - 1).clamp_(0, vocab - 1)
    at = (rank * 48271 + 11) % vocab
    gone = torch.rand(n, generator=g, device="cuda") < pad
    return at.masked_fill(gone, PAD).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = _TORCH[case["dtype"]]
    s = dict(case)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "embedding":
        n, vocab, width = case["tokens"], case["vocab"], case["width"]
        s["weight"] = randn(vocab, width).div_(math.sqrt(width)).to(dt)
        s["ids"] = _tokens(g, n, vocab, case["pad"])
        if case["backward"]:
            s["weight"].requires_grad_()
            s["g_y"] = randn(n, width).to(dt)
        return s
    if case["op"] == "gated":
        m, n, k = case["m"], case["n"], case["k"]
        s["x"] = randn(m, k).to(dt)
        s["gate"] = randn(n, k).div_(math.sqrt(k)).to(dt)
        s["up"] = randn(n, k).div_(math.sqrt(k)).to(dt)
        if case["backward"]:
            s["g_y"] = randn(m, n).to(dt)
            for t in (s["x"], s["gate"], s["up"]):
                t.requires_grad_()
        return s
    m, vocab, k = case["m"], case["vocab"], case["k"]
    w = randn(vocab, k).mul_(2.2 / math.sqrt(k))
    s["ids"] = _tokens(g, m, vocab, case["pad"])
    # hidden states that lean to their token's row, as a trained head's do
    lean = torch.rand(m, 1, generator=g, device="cuda") * 6
    s["x"] = randn(m, k).add_(lean * w[s["ids"].long().clamp_min(0)]).to(dt)
    s["weight"] = w.to(dt)
    s["b"] = None
    if case["bias"]:
        b = randn(vocab) * 0.5
        if case["masked"]:
            hide = torch.rand(vocab, generator=g, device="cuda") < case["masked"]
            hide[s["ids"].long().clamp_min(0)] = False
            b.masked_fill_(hide, -math.inf)
        s["b"] = b.to(dt)
    if case["backward"]:
        s["g_loss"] = torch.rand(m, generator=g, device="cuda") + 0.5
        s["g_lse"] = randn(m) * 0.1 if case["lse"] else None
        for t in (s["x"], s["weight"], s["b"]):
            if t is not None:
                t.requires_grad_()
    return s


# --------------------------------------------------------- the library's calls
def _run_own(s):
    import draft_verification_row_amd as sv
    if s["op"] == "embedding":
        y = sv.spec_embedding(s["weight"], s["ids"], scale=s["scale"])
        out = {"y": y}
        if s["backward"]:
            out["grad_weight"], = torch.autograd.grad([y], [s["weight"]], [s["g_y"]])
        return out
    if s["op"] == "gated":
        y = sv.spec_gated_linear(s["x"], s["gate"], s["up"], activation=s["act"])
        out = {"y": y}
        if s["backward"]:
            names = ("x", "gate", "up")
            grads = torch.autograd.grad([y], [s[n] for n in names], [s["g_y"]])
            out.update(("grad_" + n, t) for n, t in zip(names, grads))
        return out
    r = sv.spec_cross_entropy(s["x"], s["weight"], s["ids"], s["b"])
    out = {"loss": r.loss, "lse": r.lse}
    if s["backward"]:
        names = [n for n in ("x", "weight", "b") if s[n] is not None]
        ends, weights = [r.loss], [s["g_loss"]]
        if s["lse"]:
            ends, weights = ends + [r.lse], weights + [s["g_lse"]]
        grads = torch.autograd.grad(ends, [s[n] for n in names], weights)
        out.update(("grad_" + n, t) for n, t in zip(names, grads))
    return out


# ----------------------------------------------------------------- plain forms
def _plain_embedding(s):
    ids = s["ids"].long()
    live = (ids != PAD)[:, None]
    w = s["weight"].detach()
    y = torch.where(live, w[ids.clamp_min(0)].float() * s["scale"], 0.0)
    out = {"y": y.to(w.dtype)}
    if s["backward"]:
        grad = torch.zeros(w.shape, dtype=torch.float32, device=w.device)
        part = torch.where(live, s["g_y"].float(), 0.0)
        grad.index_add_(0, ids.clamp_min(0), part)
        out["grad_weight"] = (grad * s["scale"]).to(w.dtype)
    return out


def _act(z, name):
    if name == "relu":
        return torch.where(z > 0, z, 0.0)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        cdf = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return cdf + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return sig * (1 + z * (1 - sig))
    return torch.ones_like(z)


def _plain_gated(s):
    dt = s["x"].dtype
    x, wg, wu = (s[n].detach().float() for n in ("x", "gate", "up"))
    gate, up = x @ wg.t(), x @ wu.t()
    a = _act(gate, s["act"])
    out = {"y": (a * up).to(dt)}
    if s["backward"]:
        gy = s["g_y"].float()
        d_up = gy * a
        d_gate = gy * up * _act_grad(gate, s["act"])
        out["grad_x"] = (d_gate @ wg + d_up @ wu).to(dt)
        out["grad_gate"] = (d_gate.t() @ x).to(dt)
        out["grad_up"] = (d_up.t() @ x).to(dt)
    return out


def _plain_entropy(s):
    dt = s["x"].dtype
    x, w = s["x"].detach().float(), s["weight"].detach().float()
    ids = s["ids"].long()
    live = ids != PAD
    at = ids.clamp_min(0)[:, None]
    z = x @ w.t()
    if s["b"] is not None:
        z = z + s["b"].detach().float()
    top = z.amax(-1, keepdim=True)
    picked = (z.gather(1, at) - top)[:, 0]
    e = torch.exp(z - top)
    del z
    total = e.sum(-1, keepdim=True)
    log_total = torch.log(total)[:, 0]
    out = {"loss": torch.where(live, log_total - picked, 0.0),
           "lse": torch.where(live, top[:, 0] + log_total, 0.0)}
    if s["backward"]:
        gl = torch.where(live, s["g_loss"], 0.0)
        both = gl + torch.where(live, s["g_lse"], 0.0) if s["lse"] else gl
        dz = e.mul_((both / total[:, 0])[:, None])
        dz.scatter_add_(1, at, -gl[:, None])
        out["grad_x"] = (dz @ w).to(dt)
        out["grad_weight"] = (dz.t() @ x).to(dt)
        if s["b"] is not None:
            out["grad_b"] = dz.sum(0).to(dt)
    return out


_PLAIN = {"embedding": _plain_embedding, "gated": _plain_gated, "entropy": _plain_entropy}


def run(state):
    if own:
        return _run_own(state)
    return _PLAIN[state["op"]](state)


# ------------------------------------------------------- definitions, 64 bits
_PIECE = 1 << 28  # elements of a matrix taken into float64 at a time


def _exact_embedding(s):
    w = s["weight"].detach()
    n, (vocab, width) = s["tokens"], w.shape
    keep = s["ids"] >= 0
    y = torch.zeros(n, width, dtype=torch.float64, device=w.device)
    y[keep] = w[s["ids"][keep].long()].double() * s["scale"]
    out = {"y": y}
    if s["backward"]:
        # positions sorted by token, so that each token's rows are added together
        order = torch.argsort(s["ids"].long(), stable=True)
        grad = torch.zeros(vocab, width, dtype=torch.float64, device=w.device)
        ids = s["ids"].long()[order]
        rows = s["g_y"][order].double()
        some = ids >= 0
        grad.index_put_((ids[some],), rows[some], accumulate=True)
        out["grad_weight"] = grad.mul_(s["scale"])
    return out


def _exact_gated(s):
    x, wg, wu = (s[n].detach().double() for n in ("x", "gate", "up"))
    a, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
    normal = lambda v: 0.5 * torch.erfc(-v / math.sqrt(2.0))  # noqa: E731
    act = s["act"]
    f = {"none": lambda v: v, "relu": lambda v: v.clamp_min(0.0), "gelu": lambda v: v * normal(v),
         "silu": lambda v: v * torch.sigmoid(v)}[act](a)
    out = {"y": f * u}
    if s["backward"]:
        if act == "relu":
            slope = (a > 0).double()
        elif act == "gelu":
            slope = normal(a) + a * torch.exp(-a * a / 2) * (1 / math.sqrt(2 * math.pi))
        elif act == "silu":
            sg = torch.sigmoid(a)
            slope = sg + a * sg * torch.sigmoid(-a)
        else:
            slope = torch.ones_like(a)
        dy = s["g_y"].double()
        da, du = dy * u * slope, dy * f
        out["grad_x"] = torch.mm(da, wg) + torch.mm(du, wu)
        out["grad_gate"] = torch.mm(da.t(), x)
        out["grad_up"] = torch.mm(du.t(), x)
    return out


def _exact_entropy(s):
    m, vocab = s["m"], s["vocab"]
    x, w = s["x"].detach().double(), s["weight"].detach().double()
    b = None if s["b"] is None else s["b"].detach().double()
    keep = (s["ids"] >= 0).double()
    ids = s["ids"].long().clamp_min(0)
    loss, lse = [], []
    if s["backward"]:
        gx, gw = torch.empty_like(x), torch.zeros_like(w)
        gb = None if b is None else torch.zeros_like(b)
    step = max(1, _PIECE // vocab)
    for r in range(0, m, step):
        z = torch.mm(x[r:r + step], w.t())
        if b is not None:
            z += b
        k, at = keep[r:r + step], ids[r:r + step, None]
        n = torch.logsumexp(z, -1)
        loss.append((n - z.gather(1, at)[:, 0]) * k)
        lse.append(n * k)
        if s["backward"]:
            one = s["g_loss"][r:r + step].double() * k
            two = s["g_lse"][r:r + step].double() * k if s["lse"] else torch.zeros_like(one)
            d = torch.exp(z.sub_(n[:, None])).mul_((one + two)[:, None])
            d.scatter_add_(1, at, -one[:, None])
            gx[r:r + step] = torch.mm(d, w)
            gw += torch.mm(d.t(), x[r:r + step])
            if gb is not None:
                gb += d.sum(0)
    out = {"loss": torch.cat(loss), "lse": torch.cat(lse)}
    if s["backward"]:
        out["grad_x"], out["grad_weight"] = gx, gw
        if gb is not None:
            out["grad_b"] = gb
    return out


_EXACT = {"embedding": _exact_embedding, "gated": _exact_gated, "entropy": _exact_entropy}


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))

"""Measured cases of the training operators: group norm with an activation
(channels last), bias + dropout + residual with a counter-based mask, and the
router's balance loss, each with its backward.

``listed()`` names the cases, ``draw()`` gives further ones of the same ranges,
``prepare()`` makes a case's inputs from a seed, ``run()`` makes one pass:
in elementary torch operations, or, where ``own`` is true, through the
library's entry points. ``exact()`` states the same results in 64 bits and
``work()`` the bytes and operations a pass cannot do without.
"""
import math

import torch

own = False

EPS = 1e-5
COEF = 0.01


def listed():
    return [
        # the lowest resolution of an image model while it samples, two samples for guidance: latency counts
        {"name": "groupnorm_small", "op": "groupnorm", "B": 2, "S": 64, "C": 1280, "G": 32, "pad": 0,
         "act": "silu", "dtype": "bf16"},
        # a decoder's last blocks on one 512 x 512 image: one long sample
        {"name": "groupnorm_image", "op": "groupnorm", "B": 1, "S": 262144, "C": 128, "G": 32, "pad": 0,
         "act": "silu", "dtype": "bf16"},
        # training in fp32 on a 33 x 35 crop, 11 channels a group, rows of a wider tensor
        {"name": "groupnorm_backward_odd", "op": "groupnorm_backward", "B": 3, "S": 1155, "C": 330, "G": 30,
         "pad": 5, "act": "gelu_tanh", "dtype": "f32"},
        # training at 64 x 64, 10 channels a group
        {"name": "groupnorm_backward_train", "op": "groupnorm_backward", "B": 32, "S": 4096, "C": 320, "G": 32,
         "pad": 0, "act": "silu", "dtype": "bf16"},
        # one short sequence of a small fp32 model
        {"name": "dropout_small", "op": "dropout", "M": 128, "N": 768, "pad": 0, "p": 0.1, "bias": True,
         "residual": True, "dtype": "f32"},
        # the end of a block on a training batch of 16384 tokens
        {"name": "dropout_large", "op": "dropout", "M": 16384, "N": 8192, "pad": 0, "p": 0.1, "bias": True,
         "residual": True, "dtype": "bf16"},
        # ragged rows that start at no vector's border
        {"name": "dropout_backward_odd", "op": "dropout_backward", "M": 4001, "N": 4097, "pad": 0, "p": 0.25,
         "bias": True, "dtype": "bf16"},
        # the same batch of 16384 tokens, backwards, with the bias's gradient
        {"name": "dropout_backward_large", "op": "dropout_backward", "M": 16384, "N": 8192, "pad": 0, "p": 0.1,
         "bias": True, "dtype": "bf16"},
        # a short sequence through a router of 8 experts, two of them chosen
        {"name": "balance_small", "op": "balance", "T": 64, "E": 8, "K": 2, "pad": 0, "padded": 0.0, "dtype": "f32"},
        # a training batch of 131072 tokens through a router of 256 experts, eight of them chosen
        {"name": "balance_large", "op": "balance", "T": 131072, "E": 256, "K": 8, "pad": 0, "padded": 0.0,
         "dtype": "f32"},
        # a padded batch, 60 experts, bf16 logits
        {"name": "balance_backward_odd", "op": "balance_backward", "T": 5003, "E": 60, "K": 6, "pad": 0,
         "padded": 0.2, "dtype": "bf16"},
        # the training batch, backwards
        {"name": "balance_backward_large", "op": "balance_backward", "T": 131072, "E": 256, "K": 8, "pad": 0,
         "padded": 0.0, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["groupnorm", "groupnorm_backward", "dropout", "dropout_backward", "balance", "balance_backward"])
    dtype = rng.choice(["f32", "bf16"])
    pad = rng.choice([0, 0, 0, 8, 3])
    if op.startswith("groupnorm"):
        G = rng.choice([1, 4, 8, 16, 30, 32])
        C = G * _log(rng, 1, 48)
        S = _log(rng, 16, 65536)
        B = min(_log(rng, 1, 32), max(1, (1 << 24) // (S * C)))
        S = min(S, (1 << 24) // C)
        act = rng.choice(["none", "silu", "silu", "gelu", "gelu_tanh"])
        return {"op": op, "B": B, "S": S, "C": C, "G": G, "pad": pad, "act": act, "dtype": dtype}
    if op.startswith("dropout"):
        N = _log(rng, 16, 16384)
        M = min(_log(rng, 1, 65536), max(1, (1 << 26) // N))
        case = {"op": op, "M": M, "N": N, "pad": pad, "p": rng.choice([0.0, 0.1, 0.25, 0.5]),
                "bias": rng.random() < 0.7, "dtype": dtype}
        if op == "dropout":
            case["residual"] = rng.random() < 0.7
        return case
    E = _log(rng, 2, 512)
    T = min(_log(rng, 1, 131072), (1 << 25) // E)
    return {"op": op, "T": T, "E": E, "K": rng.randint(1, min(8, max(1, E // 2))), "pad": pad,
            "padded": rng.choice([0.0, 0.0, 0.2]), "dtype": dtype}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _place(v, case):
    """v in the case's type, as rows of a tensor that is `pad` columns wider."""
    rows = torch.empty(v.shape[:-1] + (v.shape[-1] + case["pad"],), dtype=_dtype(case), device=v.device)
    rows[..., : v.shape[-1]] = v
    return rows[..., : v.shape[-1]]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    s = dict(case)
    if case["op"].startswith("groupnorm"):
        B, S, C, G = case["B"], case["S"], case["C"], case["G"]
        # activations: every channel with an offset and a spread of its own
        s["x"] = _place(normal(B, S, C) * (0.5 + torch.rand(C, generator=g, device="cuda")) + 0.5 * normal(C), case)
        s["w"] = (1 + 0.2 * normal(C)).to(_dtype(case))
        s["b"] = (0.1 * normal(C)).to(_dtype(case))
        if case["op"] == "groupnorm_backward":
            s["dy"] = _place(normal(B, S, C), case)
            # what the forward pass left: mean and 1 / sqrt(var + eps) of every sample's groups
            v = s["x"].double().reshape(B, S, G, C // G)
            mean = v.mean(dim=(1, 3))
            var = (v - mean[:, None, :, None]).square().mean(dim=(1, 3))
            s["stats"] = torch.stack([mean, 1 / (var + EPS).sqrt()], dim=2).float().contiguous()
    elif case["op"].startswith("dropout"):
        M, N = case["M"], case["N"]
        s["x"] = _place(normal(M, N), case)
        s["bias"] = (0.1 * normal(N)).to(_dtype(case)) if case["bias"] else None
        s["residual"] = _place(normal(M, N), case) if case.get("residual") else None
        s["seed"], s["offset"] = 0x9E3779B97F4A7C15 ^ seed, 1000 * seed + 7
    else:
        T, E, K = case["T"], case["E"], case["K"]
        logits = normal(T, E) + normal(E)
        s["logits"] = _place(logits, case)
        s["experts"] = logits.topk(K, dim=1).indices
        s["mask"] = torch.rand(T, generator=g, device="cuda") >= case["padded"] if case["padded"] else None
        if case["op"] == "balance_backward":
            s["dloss"] = 1 + 0.1 * normal(1)
            s["counts"] = _counts(s)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _run_own(s)
    return _PLAIN[s["op"]](s)


def _run_own(s):
    import row_wise_reduction_gb300 as ro

    op = s["op"]
    if op == "groupnorm":
        return ro.rowops_groupnorm_act(s["x"], s["G"], s["w"], s["b"], EPS, s["act"])
    if op == "groupnorm_backward":
        return ro.rowops_groupnorm_act_backward(s["x"], s["dy"], s["stats"], s["G"], s["w"], s["b"], s["act"])
    if op == "dropout":
        return ro.rowops_bias_dropout_residual(s["x"], s["residual"], s["bias"], s["p"], s["seed"], s["offset"])
    if op == "dropout_backward":
        dx, dbias = ro.rowops_bias_dropout_residual_backward(s["x"], s["p"], s["seed"], s["offset"],
                                                             bias_grad=s["bias"] is not None)
        return (dx, dbias) if s["bias"] is not None else (dx,)
    if op == "balance":
        return ro.rowops_router_balance_loss(s["logits"], s["experts"], COEF, s["mask"])
    return ro.rowops_router_balance_loss_backward(s["logits"], s["counts"], s["K"], s["dloss"], COEF, s["mask"])


def _act(z, act):
    if act == "none":
        return z
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.7071067811865476))
    return 0.5 * z * (1 + torch.tanh(0.79788456 * (z + 0.044715 * z * z * z)))


def _act_grad(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "silu":
        q = 1 / (1 + torch.exp(-z))
        return q * (1 + z * (1 - q))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.7071067811865476)) + z * 0.3989422804014327 * torch.exp(-0.5 * z * z)
    t = torch.tanh(0.79788456 * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * 0.79788456 * (1 + 3 * 0.044715 * z * z)


def _groupnorm(s):
    B, S, C = s["x"].shape
    G = s["G"]
    v = s["x"].float().reshape(B, S, G, C // G)
    n = S * (C // G)
    mean = v.sum(dim=(1, 3), keepdim=True) / n
    d = v - mean
    var = (d * d).sum(dim=(1, 3), keepdim=True) / n
    z = (d / torch.sqrt(var + EPS)).reshape(B, S, C) * s["w"].float() + s["b"].float()
    return _act(z, s["act"]).to(s["x"].dtype)


def _groupnorm_backward(s):
    B, S, C = s["x"].shape
    G = s["G"]
    n = S * (C // G)
    mean, rstd = (s["stats"][:, None, :, k, None] for k in (0, 1))
    xh = ((s["x"].float().reshape(B, S, G, C // G) - mean) * rstd).reshape(B, S, C)
    w = s["w"].float()
    dz = s["dy"].float() * _act_grad(xh * w + s["b"].float(), s["act"])
    db = dz.sum(dim=1)
    dw = (dz * xh).sum(dim=1)
    c1 = (db * w).reshape(B, 1, G, C // G).sum(dim=3, keepdim=True) / n
    c2 = (dw * w).reshape(B, 1, G, C // G).sum(dim=3, keepdim=True) / n
    dx = rstd * ((dz * w).reshape(B, S, G, C // G) - c1 - xh.reshape(B, S, G, C // G) * c2)
    return dx.reshape(B, S, C).to(s["x"].dtype), dw.sum(dim=0), db.sum(dim=0)


def _mulhilo(a, b):
    """High and low word of a * b, both below 2^32, in int64 without overflow."""
    low = a * (b & 0xFFFF)
    up = a * (b >> 16) + (low >> 16)
    return up >> 16, ((up & 0xFFFF) << 16) | (low & 0xFFFF)


def _keep(M, N, p, seed, offset, device):
    """Where the mask keeps: 16 random bits of Philox4x32-10 for each element,
    counter (column / 8, row, offset), key seed; kept where they reach
    round(65536 p). And the scale of what is kept."""
    drop = round(p * 65536)
    c0 = torch.arange((N + 7) // 8, device=device, dtype=torch.int64).expand(M, -1)
    c1 = torch.arange(M, device=device, dtype=torch.int64)[:, None].expand_as(c0)
    c2, c3 = (torch.full_like(c0, v) for v in (offset & 0xFFFFFFFF, offset >> 32))
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        h0, l0 = _mulhilo(0xD2511F53, c0)
        h1, l1 = _mulhilo(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    bits = torch.stack([h for c in (c0, c1, c2, c3) for h in (c & 0xFFFF, c >> 16)], dim=2)
    return bits.reshape(M, -1)[:, :N] >= drop, (65536 / (65536 - drop) if drop < 65536 else 0.0)


def _dropout(s):
    M, N = s["x"].shape
    keep, scale = _keep(M, N, s["p"], s["seed"], s["offset"], s["x"].device)
    v = s["x"].float()
    if s["bias"] is not None:
        v = v + s["bias"].float()
    v = torch.where(keep, v * scale, 0.0)
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v.to(s["x"].dtype)


def _dropout_backward(s):
    M, N = s["x"].shape
    keep, scale = _keep(M, N, s["p"], s["seed"], s["offset"], s["x"].device)
    v = torch.where(keep, s["x"].float() * scale, 0.0)
    dx = v.to(s["x"].dtype)
    return (dx, v.sum(dim=0)) if s["bias"] is not None else (dx,)


def _softmax(s):
    v = s["logits"].float()
    e = torch.exp(v - v.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _counts(s):
    """Assignments of every expert, and the tokens that take part."""
    T, E = s["logits"].shape
    mask = s["mask"] if s["mask"] is not None else torch.ones(T, dtype=torch.bool, device=s["logits"].device)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=s["logits"].device)
    counts.scatter_add_(0, s["experts"].reshape(-1), mask[:, None].expand(T, s["K"]).reshape(-1).long())
    counts[E] = mask.sum()
    return counts


def _balance(s):
    E = s["E"]
    counts = _counts(s)
    p = _softmax(s)
    if s["mask"] is not None:
        p = torch.where(s["mask"][:, None], p, 0.0)
    n = counts[E].double().clamp(min=1)
    loss = COEF * E / (n * n * s["K"]) * (counts[:E].double() * p.double().sum(dim=0)).sum()
    return loss.float().reshape(1), counts


def _balance_backward(s):
    E = s["E"]
    n = s["counts"][E].double().clamp(min=1)
    f = (COEF * E / (n * n * s["K"]) * s["dloss"].double() * s["counts"][:E].double()).float()
    p = _softmax(s)
    d = p * (f - (p * f).sum(dim=1, keepdim=True))
    if s["mask"] is not None:
        d = torch.where(s["mask"][:, None], d, 0.0)
    return d.to(s["logits"].dtype)


_PLAIN = {"groupnorm": _groupnorm, "groupnorm_backward": _groupnorm_backward, "dropout": _dropout,
          "dropout_backward": _dropout_backward, "balance": _balance, "balance_backward": _balance_backward}


# ---------------------------------------------------------------------------
# the same results in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))


def _phi(z):
    """The activations and their derivatives in 64 bits, by name."""
    def tanh_form():
        u = 0.79788456 * (z + 0.044715 * z ** 3)
        q = torch.sigmoid(2 * u)  # 0.5 (1 + tanh(u))
        return z * q, q + 2 * z * q * (1 - q) * 0.79788456 * (1 + 0.134145 * z ** 2)

    def exact_form():
        q = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * q, q + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)

    def silu():
        q = torch.sigmoid(z)
        return z * q, q + z * q * torch.sigmoid(-z)

    return {"none": lambda: (z, torch.ones_like(z)), "silu": silu, "gelu": exact_form, "gelu_tanh": tanh_form}


def _grouped(t, G):
    """(B, S, C) in 64 bits as (B, G, C / G, S)."""
    B, S, C = t.shape
    return t.double().permute(0, 2, 1).reshape(B, G, C // G, S)


def _ungrouped(t):
    B, G, L, S = t.shape
    return t.reshape(B, G * L, S).permute(0, 2, 1)


def _exact_groupnorm(s):
    G = s["G"]
    v = _grouped(s["x"], G)
    var, mean = torch.var_mean(v, dim=(2, 3), keepdim=True, correction=0)
    w, b = (s[k].double().reshape(1, G, -1, 1) for k in ("w", "b"))
    return _ungrouped(_phi((v - mean) * (var + EPS) ** -0.5 * w + b)[s["act"]]()[0])


def _exact_groupnorm_backward(s):
    G = s["G"]
    v, dy = _grouped(s["x"], G), _grouped(s["dy"], G)
    w, b = (s[k].double().reshape(1, G, -1, 1) for k in ("w", "b"))
    mean, rstd = (s["stats"].double()[:, :, k, None, None] for k in (0, 1))
    xh = (v - mean) * rstd
    dz = dy * _phi(xh * w + b)[s["act"]]()[1]
    dxh = dz * w
    dx = rstd * (dxh - dxh.mean(dim=(2, 3), keepdim=True) - xh * (dxh * xh).mean(dim=(2, 3), keepdim=True))
    return _ungrouped(dx), (dz * xh).sum(dim=(0, 3)).reshape(-1), dz.sum(dim=(0, 3)).reshape(-1)


def _exact_scale(s):
    """1 / (1 - p) where the mask keeps and 0 elsewhere: the mask's bits from
    products that wrap at 64 bits, both halves of a round taken from one."""
    M, N = s["x"].shape
    W = 1 << 32

    def every(v):
        return torch.zeros(M, (N + 7) // 8, dtype=torch.int64, device="cuda") + v

    x = [every(torch.arange((N + 7) // 8, device="cuda")), every(torch.arange(M, device="cuda")[:, None]),
         every(s["offset"] % W), every(s["offset"] // W)]
    key = [s["seed"] % W, s["seed"] // W]
    for r in range(10):
        a, b = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57
        up = [(v >> 32) & (W - 1) for v in (a, b)]
        x = [up[1] ^ x[1] ^ (key[0] + r * 0x9E3779B9) % W, b & (W - 1),
             up[0] ^ x[3] ^ (key[1] + r * 0xBB67AE85) % W, a & (W - 1)]
    u = torch.empty(M, (N + 7) // 8, 8, dtype=torch.int64, device="cuda")
    for i, v in enumerate(x):
        u[..., 2 * i], u[..., 2 * i + 1] = v % 65536, v // 65536
    drop = int(math.floor(s["p"] * 65536 + 0.5))
    kept = (u.reshape(M, -1)[:, :N] >= drop).double()
    return kept / (1 - drop / 65536) if drop < 65536 else kept


def _exact_dropout(s):
    v = s["x"].double()
    if s["bias"] is not None:
        v = v + s["bias"].double()
    v = v * _exact_scale(s)
    return v + s["residual"].double() if s["residual"] is not None else v


def _exact_dropout_backward(s):
    v = s["x"].double() * _exact_scale(s)
    return (v, v.sum(dim=0)) if s["bias"] is not None else (v,)


def _exact_counts(s):
    chosen = s["experts"] if s["mask"] is None else s["experts"][s["mask"]]
    return torch.bincount(chosen.reshape(-1), minlength=s["E"])


def _exact_balance(s):
    p = torch.exp(torch.log_softmax(s["logits"].double(), dim=1))
    if s["mask"] is not None:
        p = p[s["mask"]]
    f = _exact_counts(s)
    n = p.shape[0]
    loss = COEF * s["E"] * (f.double() / (n * s["K"]) * p.mean(dim=0)).sum() if n else torch.zeros((), device="cuda")
    return loss.double().reshape(1), torch.cat([f, torch.tensor([n], device="cuda")])


def _exact_balance_backward(s):
    E, n = s["E"], int(s["counts"][s["E"]])
    p = torch.exp(torch.log_softmax(s["logits"].double(), dim=1))
    f = s["counts"][:E].double()
    d = p * (f - p @ f[:, None]) * (COEF * E * s["dloss"].double() / (max(n, 1) ** 2 * s["K"]))
    return d if s["mask"] is None else d * s["mask"][:, None]


_EXACT = {"groupnorm": _exact_groupnorm, "groupnorm_backward": _exact_groupnorm_backward, "dropout": _exact_dropout,
          "dropout_backward": _exact_dropout_backward, "balance": _exact_balance,
          "balance_backward": _exact_balance_backward}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op.startswith("groupnorm"):
        n, C = case["B"] * case["S"] * case["C"], case["C"]
        if op == "groupnorm":  # x in, y out; w, b
            return {"bytes": 2 * n * es + 2 * C * es, "flops": 12 * n}
        # x, dy in, dx out; w, b, the statistics; dw, db
        return {"bytes": 3 * n * es + 2 * C * es + 8 * case["B"] * case["G"] + 8 * C, "flops": 30 * n}
    if op.startswith("dropout"):
        n, N = case["M"] * case["N"], case["N"]
        if op == "dropout":  # x, the residual in, y out; the bias
            return {"bytes": (2 + bool(case["residual"])) * n * es + (N * es if case["bias"] else 0), "flops": 3 * n}
        return {"bytes": 2 * n * es + (4 * N if case["bias"] else 0), "flops": 2 * n}
    n, E, T = case["T"] * case["E"], case["E"], case["T"]
    mask = T if case["padded"] else 0
    if op == "balance":  # the logits, the chosen experts; the counts and the loss
        return {"bytes": n * es + 8 * T * case["K"] + mask + 8 * (E + 1) + 4, "flops": 5 * n}
    return {"bytes": 2 * n * es + mask + 8 * (E + 1) + 4, "flops": 8 * n}

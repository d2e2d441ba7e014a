"""Measured cases of the serving step's operators: RMSNorm (with the residual's
addition) with an output in 8 bits and scales, attention of one new token over a
paged key-value cache, and sampling from logits.

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
E4M3_MAX = 448.0


def listed():
    return [
        # the step of four sequences: one scale a row, latency counts
        {"name": "norm_quant_small", "op": "norm_quant", "M": 4, "N": 4096, "pad": 0, "residual": True, "group": 0,
         "dtype": "bf16"},
        # the step of 256 sequences, a scale for every 128 columns
        {"name": "norm_quant_step", "op": "norm_quant", "M": 256, "N": 8192, "pad": 0, "residual": True, "group": 128,
         "dtype": "bf16"},
        # fp32 rows of odd length out of a wider tensor, the last group of each cut short, no residual
        {"name": "norm_quant_odd", "op": "norm_quant", "M": 1501, "N": 4099, "pad": 3, "residual": False,
         "group": 64, "dtype": "f32"},
        # a prompt batch of 16384 tokens
        {"name": "norm_quant_large", "op": "norm_quant", "M": 16384, "N": 8192, "pad": 0, "residual": True,
         "group": 128, "dtype": "bf16"},
        # one conversation of some hundred tokens: latency counts
        {"name": "attention_small", "op": "attention", "B": 1, "heads": 32, "kv_heads": 8, "D": 128, "page": 16,
         "longest": 512, "shortest": 512, "window": 0, "layout": "slots", "dtype": "bf16"},
        # a serving batch of 64 sequences of every length up to 8192
        {"name": "attention_batch", "op": "attention", "B": 64, "heads": 32, "kv_heads": 8, "D": 128, "page": 16,
         "longest": 8192, "shortest": 64, "window": 0, "layout": "slots", "dtype": "bf16"},
        # two long documents: few rows, so the cache's length is what can be shared out
        {"name": "attention_long", "op": "attention", "B": 2, "heads": 64, "kv_heads": 8, "D": 128, "page": 64,
         "longest": 131072, "shortest": 100000, "window": 0, "layout": "heads", "dtype": "bf16"},
        # fp32, 5 heads to a key head, head dimension 80, pages of 24 slots, a sliding window, an empty sequence
        {"name": "attention_odd", "op": "attention", "B": 9, "heads": 15, "kv_heads": 3, "D": 80, "page": 24,
         "longest": 5000, "shortest": 0, "window": 1999, "layout": "slots", "dtype": "f32"},
        # one sequence, the usual knobs together: latency counts
        {"name": "sample_small", "op": "sample", "T": 1, "V": 32000, "pad": 0, "knobs": "all", "dtype": "bf16"},
        # a batch of 256 sequences cut by mass
        {"name": "sample_top_p", "op": "sample", "T": 256, "V": 131072, "pad": 0, "knobs": "top_p", "dtype": "bf16"},
        # fp32 logits of an odd vocabulary in padded rows; every row has knobs of its own, some rows are greedy
        {"name": "sample_mixed", "op": "sample", "T": 61, "V": 50021, "pad": 3, "knobs": "mixed", "dtype": "f32"},
        # a large batch without a cut: temperature alone
        {"name": "sample_plain", "op": "sample", "T": 512, "V": 131072, "pad": 0, "knobs": "temperature",
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_quant", "attention", "sample"])
    dtype = rng.choice(["f32", "bf16", "bf16"])
    if op == "norm_quant":
        N = _log(rng, 64, 16384)
        if rng.random() < 0.6:
            N = max(64, N // 64 * 64)
        M = min(_log(rng, 1, 32768), (1 << 26) // N)
        return {"op": op, "M": M, "N": N, "pad": rng.choice([0, 0, 0, 8, 3]), "residual": rng.random() < 0.6,
                "group": rng.choice([0, 0, 32, 64, 128, 128, 256]), "dtype": dtype}
    if op == "attention":
        kv = rng.choice([1, 2, 3, 4, 8, 8, 16])
        heads = kv * rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8, 8, 12, 16])
        D = rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256])
        most = (1 << 28) // (kv * D)  # positions of all sequences together
        longest = min(_log(rng, 1, 65536), most)
        B = min(_log(rng, 1, 128), max(1, most // longest))
        shortest = rng.choice([0, 1, longest // 2, longest])
        window = rng.choice([0, 0, 0, max(1, longest // 3)])
        return {"op": op, "B": B, "heads": heads, "kv_heads": kv, "D": D, "page": rng.choice([8, 16, 16, 24, 32, 64, 128]),
                "longest": longest, "shortest": shortest, "window": window, "layout": rng.choice(["slots", "heads"]),
                "dtype": dtype}
    V = _log(rng, 100, 200000)
    T = min(_log(rng, 1, 1024), (1 << 25) // V)
    return {"op": op, "T": T, "V": V, "pad": rng.choice([0, 0, 0, 8, 3]),
            "knobs": rng.choice(["temperature", "top_k", "top_p", "min_p", "all", "mixed"]), "dtype": dtype}


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


def _lengths(case):
    """The sequences' lengths: the same ones for every seed, from the shortest to the longest."""
    B, lo, hi = case["B"], case["shortest"], case["longest"]
    return [hi - (hi - lo) * i // max(1, B - 1) for i in range(B)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype)

    s = dict(case)
    if case["op"] == "norm_quant":
        M, N = case["M"], case["N"]
        # a residual stream: some columns far larger than the rest
        spread = 1 + 8 * (torch.rand(N, generator=g, device="cuda") > 0.99)
        s["x"] = _place(normal(M, N), case)
        s["residual"] = _place(normal(M, N) * spread, case) if case["residual"] else None
        s["w"] = (1 + 0.2 * normal(N)).to(_dtype(case))
    elif case["op"] == "attention":
        B, H, K, D, page = (case[k] for k in ("B", "heads", "kv_heads", "D", "page"))
        lengths = _lengths(case)
        order = torch.randperm(B, generator=g, device="cuda")
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")[order]
        # every sequence's pages lie anywhere in the pool; what a sequence has no page for is -1
        width = max(1, -(-case["longest"] // page))
        used = torch.arange(width, device="cuda") * page < s["lengths"][:, None]
        pool = sum(-(-n // page) for n in lengths) + 3
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        table[used] = torch.randperm(pool, generator=g, device="cuda")[: pool - 3].int()
        s["table"] = table
        shape = (pool, page, K, D) if case["layout"] == "slots" else (pool, K, page, D)
        for name in ("k", "v"):
            cache = normal(*shape, dtype=_dtype(case))
            s[name] = cache if case["layout"] == "slots" else cache.transpose(1, 2)
        s["q"] = normal(B, H, D).to(_dtype(case))
        s["scale"] = D ** -0.5
    else:
        T, V = case["T"], case["V"]
        # a language model's logits: a wide bulk, and some tokens far above it, in some rows more than in others
        logits = 2.0 * normal(T, V)
        near = torch.randint(V, (T, 24), generator=g, device="cuda")
        lift = 4 + 10 * torch.rand(T, 24, generator=g, device="cuda") * torch.rand(T, 1, generator=g, device="cuda")
        s["logits"] = _place(logits.scatter_add_(1, near, lift), case)
        s["u"] = torch.rand(T, generator=g, device="cuda")
        knobs = case["knobs"]
        temperature = 0.5 + torch.rand(T, generator=g, device="cuda")
        top_k = torch.randint(1, 200, (T,), generator=g, device="cuda", dtype=torch.int32)
        top_p = 0.5 + 0.49 * torch.rand(T, generator=g, device="cuda")
        min_p = 0.02 + 0.1 * torch.rand(T, generator=g, device="cuda")
        if knobs == "mixed":
            on = torch.rand(4, T, generator=g, device="cuda") < 0.5
            temperature, top_k = torch.where(on[0], temperature, 0.0), torch.where(on[1], top_k, 0)
            top_p, min_p = torch.where(on[2], top_p, 1.0), torch.where(on[3], min_p, 0.0)
        every = knobs in ("all", "mixed")
        s["temperature"] = temperature
        s["top_k"] = top_k if every or knobs == "top_k" else None
        s["top_p"] = top_p if every or knobs == "top_p" else None
        s["min_p"] = min_p if every or knobs == "min_p" else None
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

    if s["op"] == "norm_quant":
        q, scales, residual_out = ro.rowops_rmsnorm_quant(s["x"], s["residual"], s["w"], EPS, s["group"])
        return (q, scales) if residual_out is None else (q, scales, residual_out)
    if s["op"] == "attention":
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=s["q"].device)
        out = ro.rowops_paged_attention(s["q"], s["k"], s["v"], s["table"], s["lengths"], s["scale"], s["window"],
                                        lse=lse)
        return out, lse
    knobs = {k: s[k] for k in ("temperature", "top_k", "top_p", "min_p") if s[k] is not None}
    logprob = torch.empty(s["T"], dtype=torch.float32, device=s["u"].device)
    tokens = ro.rowops_sample(s["logits"], s["u"], **knobs, logprob=logprob)
    return tokens, logprob


def _norm_quant(s):
    M, N = s["x"].shape
    v = s["x"].float()
    if s["residual"] is not None:
        residual_out = (v + s["residual"].float()).to(s["x"].dtype)
        v = residual_out.float()
    y = v / torch.sqrt((v * v).sum(dim=1, keepdim=True) / N + EPS) * s["w"].float()
    group = s["group"] or N
    groups = -(-N // group)
    padded = torch.zeros(M, groups * group, device=y.device)
    padded[:, :N] = y
    cut = padded.reshape(M, groups, group)
    scales = (cut.abs().amax(dim=2) / E4M3_MAX).clamp(min=2.0 ** -126)
    q = (cut / scales[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).reshape(M, -1)[:, :N].to(torch.float8_e4m3fn)
    return (q, scales) if s["residual"] is None else (q, scales, residual_out)


def _attention(s):
    B, H, D = s["q"].shape
    K = s["k"].shape[2]
    table = s["table"].long().clamp(min=0)
    k, v = (s[n][table].reshape(B, -1, K, D).float() for n in ("k", "v"))
    q = s["q"].float().reshape(B, K, H // K, D)
    scores = torch.einsum("bkgd,bnkd->bkgn", q, k) * s["scale"]
    at, n = torch.arange(k.shape[1], device=k.device), s["lengths"].long()[:, None]
    attended = at < n
    if s["window"]:
        attended = attended & (at >= n - s["window"])
    scores = torch.where(attended[:, None, None, :], scores, -math.inf)
    top = scores.amax(dim=3, keepdim=True).clamp(min=-3e38)
    e = torch.exp(scores - top)
    total = e.sum(dim=3, keepdim=True)
    v = torch.where(attended[:, :, None, None], v, 0.0)
    out = torch.einsum("bkgn,bnkd->bkgd", e, v) / total.clamp(min=1e-30)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)
    return out.reshape(B, H, D).to(s["q"].dtype), lse.reshape(B, H)


def _sample(s):
    x = s["logits"].double()  # in 64 bits: a cut or a draw is next to a border in some row
    T, V = x.shape
    temperature = s["temperature"].double()[:, None]
    warm = temperature > 0
    sorted_x, order = torch.sort(x, dim=1, descending=True, stable=True)
    w = torch.exp((sorted_x - sorted_x[:, :1]) / torch.where(warm, temperature, 1.0))
    rank = torch.arange(V, device=x.device)
    keep = warm | (rank == 0)
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        keep = keep & ((rank < k) | (k <= 0))
    w = torch.where(keep, w, 0.0)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        mass = torch.cumsum(w, dim=1)
        keep = keep & ((mass - w < p * mass[:, -1:]) | (p >= 1) | (rank == 0))
    if s["min_p"] is not None:
        keep = keep & (w >= s["min_p"].double()[:, None])
    w = torch.zeros_like(x).scatter_(1, order, torch.where(keep, w, 0.0))
    mass = torch.cumsum(w, dim=1)
    total = mass[:, -1:]
    token = (mass <= s["u"].double()[:, None] * total).sum(dim=1)
    logprob = torch.log(w.gather(1, token[:, None]) / total)[:, 0].float()
    return token, logprob


_PLAIN = {"norm_quant": _norm_quant, "attention": _attention, "sample": _sample}


# ---------------------------------------------------------------------------
# the same results in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))


def _exact_norm_quant(s):
    """q as the numbers that are rounded to 8 bits."""
    x = s["x"].double()
    if s["residual"] is not None:
        x = (x + s["residual"].double()).to(s["x"].dtype).double()
    y = x * (x.square().mean(dim=1, keepdim=True) + EPS).rsqrt() * s["w"].double()
    N = y.shape[1]
    group = s["group"] or N
    column = torch.arange(N, device=y.device) // group
    largest = torch.zeros(y.shape[0], -(-N // group), dtype=torch.float64, device=y.device)
    largest.scatter_reduce_(1, column.expand_as(y), y.abs(), "amax")
    scales = torch.maximum(largest / E4M3_MAX, torch.tensor(2.0 ** -126, dtype=torch.float64, device=y.device))
    q = y / scales[:, column]
    return (q, scales) if s["residual"] is None else (q, scales, x)


def _exact_attention(s):
    """Sequence by sequence, over the positions that it attends to."""
    B, H, D = s["q"].shape
    K, page = s["k"].shape[2], s["k"].shape[1]
    out = torch.zeros(B, H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lengths"].tolist()):
        first = max(0, n - s["window"]) if s["window"] else 0
        if n == first:
            continue
        at = torch.arange(first, n, device="cuda")
        pages, slots = s["table"][b].long()[at // page], at % page
        for h in range(K):
            heads = slice(h * (H // K), (h + 1) * (H // K))
            k, v = (s[name][pages, slots, h].double() for name in ("k", "v"))
            scores = s["q"][b, heads].double() @ k.T * s["scale"]
            lse[b, heads] = torch.logsumexp(scores, dim=1)
            out[b, heads] = torch.softmax(scores, dim=1) @ v
    return out, lse


def _exact_sample(s):
    """Row by row: the candidates from the largest down, cut, and the draw among them by index."""
    tokens, logprobs = [], []
    knobs = {k: s[k].tolist() if s[k] is not None else None for k in ("temperature", "top_k", "top_p", "min_p")}
    for t, u in enumerate(s["u"].tolist()):
        x = s["logits"][t].double()
        temperature = knobs["temperature"][t]
        if temperature <= 0:
            tokens.append((x == x.max()).nonzero()[0, 0])
            logprobs.append(x.new_zeros(()))
            continue
        p = torch.softmax(x / temperature, dim=0)
        largest_first = torch.argsort(-x, stable=True)
        n = x.numel()
        if knobs["top_k"] is not None and knobs["top_k"][t] > 0:
            n = min(n, knobs["top_k"][t])
        if knobs["top_p"] is not None and knobs["top_p"][t] < 1:
            c = p[largest_first[:n]].cumsum(0)
            n = 1 + int((c[:-1] < knobs["top_p"][t] * c[-1]).sum())
        if knobs["min_p"] is not None:
            n = min(n, int((p >= knobs["min_p"][t] * p.max()).sum()))
        among = largest_first[:n].sort().values
        c = p[among].cumsum(0)
        chosen = torch.searchsorted(c, (u * c[-1]).reshape(1), right=True)[0].clamp(max=n - 1)
        tokens.append(among[chosen])
        logprobs.append((p[among[chosen]] / c[-1]).log())
    return torch.stack(tokens), torch.stack(logprobs)


_EXACT = {"norm_quant": _exact_norm_quant, "attention": _exact_attention, "sample": _exact_sample}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm_quant":
        n, N = case["M"] * case["N"], case["N"]
        scales = case["M"] * -(-N // (case["group"] or N))
        # x in, q out, w, the scales; the residual in and out
        return {"bytes": n * (es + 1 + (2 * es if case["residual"] else 0)) + N * es + 4 * scales, "flops": 8 * n}
    if case["op"] == "attention":
        B, H, K, D = (case[k] for k in ("B", "heads", "kv_heads", "D"))
        attended = sum(min(n, case["window"] or n) for n in _lengths(case))
        # the keys and values attended to, q, out, lse, the pages' numbers and the lengths
        return {"bytes": 2 * attended * K * D * es + 2 * B * H * D * es + 4 * B * H + 4 * (attended // case["page"] + B)
                + 4 * B, "flops": 4 * attended * H * D}
    T, V = case["T"], case["V"]
    return {"bytes": T * V * es + T * (4 + 16 + 12), "flops": 5 * T * V}

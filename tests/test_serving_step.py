"""The serving operators together, as a decoding step uses them: one layer's norm into 8
bits, its products, the new keys and values written into a paged cache, attention over
it, the norm before the logits, and the draw of the next token, which the next step begins
with. Every operator's result is held to its 64-bit form on the inputs that it got; a
captured step replays to the same tokens, and so do steps on other streams, side by side."""
import numpy as np
import pytest
import torch

import row_wise_reduction_gb300 as ro
from oracle import serving as O
from tests import _compare as C
from tests import gpu_util as gu
from tests.test_parity_paged_attention import hold as hold_attention
from tests.test_parity_rmsnorm_quant import hold as hold_norm

pytestmark = [pytest.mark.gpu, gu.requires_gpu]

B, H, K, D, N, V, PAGE = 5, 8, 2, 32, 256, 1000, 8
KNOBS = dict(temperature=0.9, top_k=60, top_p=0.95, min_p=0.01)


class Decoder:
    """Weights, a cache and the step's own buffers; `width` pages a sequence."""

    def __init__(self, dtype, width, seed=3):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std=1.0):
            return (std * torch.randn(shape, generator=g, device="cuda")).to(dtype)

        self.embedding = normal(V, N)
        self.w1, self.w2 = 1 + normal(N, std=0.1), 1 + normal(N, std=0.1)
        self.qkv, self.proj, self.head = normal(N, (H + 2 * K) * D, std=N**-0.5), normal(H * D, N, std=(H * D) ** -0.5), \
            normal(N, V, std=3 * N**-0.5)
        self.k, self.v = (torch.full((B * 6, PAGE, K, D), float("nan"), device="cuda", dtype=dtype) for _ in range(2))
        pages = torch.randperm(B * 6, generator=g, device="cuda").int().view(B, 6)
        self.table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        self.table[:, :6] = pages
        self.lengths = torch.tensor([0, 3, 7, 8, 20], dtype=torch.int32, device="cuda")
        at = torch.arange(20, device="cuda")
        for b, n in enumerate(self.lengths.tolist()):  # the prompts' keys and values
            for c in (self.k, self.v):
                c[pages[b, at[:n] // PAGE].long(), at[:n] % PAGE] = normal(n, K, D)
        self.token = torch.arange(B, device="cuda")
        self.u = torch.zeros(B, device="cuda")
        self.logprob, self.lse = torch.empty(B, device="cuda"), torch.empty(B, H, device="cuda")
        need = ro.rowops_paged_attention_workspace_bytes(B, H, K, D, PAGE, width, 0, dtype)
        self.ws = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")

    @staticmethod
    def product(q, scales, group, w):
        """As a product in 8 bits has it: e4m3 numbers, scaled."""
        return ((q.float().view(B, -1, group) * scales[:, :, None]).view(B, N) @ w.float()).to(w.dtype)

    def step(self, check=False):
        x = self.embedding[self.token]
        q1, s1, _ = ro.rowops_rmsnorm_quant(x, None, self.w1, 1e-5, 64)
        qkv = self.product(q1, s1, 64, self.qkv)
        q, k, v = qkv.split([H * D, K * D, K * D], dim=1)
        at = self.lengths.long()
        where = self.table.gather(1, (at // PAGE)[:, None])[:, 0].long()
        self.k[where, at % PAGE] = k.unflatten(1, (K, D))
        self.v[where, at % PAGE] = v.unflatten(1, (K, D))
        self.lengths.add_(1)
        heads = q.unflatten(1, (H, D))  # rows of the wider qkv
        out = ro.rowops_paged_attention(heads, self.k, self.v, self.table, self.lengths, lse=self.lse, workspace=self.ws)
        a = out.flatten(1) @ self.proj
        q2, s2, x2 = ro.rowops_rmsnorm_quant(a, x, self.w2, 1e-5, 0)
        logits = self.product(q2, s2, N, self.head)
        ro.rowops_sample(logits, self.u, **KNOBS, token=self.token, logprob=self.logprob)
        if check:
            hold_norm(q1, s1, C.to_f64(x), C.to_f64(self.w1), 64)
            hold_attention(out, self.lse, heads, self.k, self.v, self.table, self.lengths)
            assert torch.equal(x2, (a.float() + x.float()).to(a.dtype))
            hold_norm(q2, s2, C.to_f64(x2), C.to_f64(self.w2), 0)
            knobs = {n: float(np.float32(v)) if n != "top_k" else v for n, v in KNOBS.items()}
            for b in range(B):
                want, lp, margin = O.sample_row(C.to_f64(logits[b]), float(self.u[b]), **knobs)
                if margin >= 2.0**-28:
                    assert int(self.token[b]) == want and abs(float(self.logprob[b]) - lp) <= 2.0**-20


def numbers(steps):
    return torch.rand(steps, B, generator=torch.Generator().manual_seed(9)).cuda()


def eager(dtype, width, steps=12, check=True):
    d, tokens = Decoder(dtype, width), []
    for u in numbers(steps):
        d.u.copy_(u)
        d.step(check)
        tokens.append(d.token.clone())
    return torch.stack(tokens)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("width", [6, 60000])  # attention in one kernel, and in two with a workspace
def test_steps_eager_captured_and_on_streams(dtype, width):
    want = eager(dtype, width)
    assert len(want.unique()) > 10
    us = numbers(12)

    # captured once, replayed with new numbers
    d = Decoder(dtype, width)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        d.u.copy_(us[0])
        d.step()
    torch.cuda.current_stream().wait_stream(s)
    tokens = [d.token.clone()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d.step()
    for u in us[1:]:
        d.u.copy_(u)
        g.replay()
        tokens.append(d.token.clone())
    assert torch.equal(torch.stack(tokens), want)

    # two at once, each on a stream of its own
    streams, decoders, got = [torch.cuda.Stream() for _ in range(2)], [Decoder(dtype, width) for _ in range(2)], [[], []]
    torch.cuda.synchronize()
    for u in us:
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                decoders[i].u.copy_(u)
                decoders[i].step()
                got[i].append(decoders[i].token.clone())
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(torch.stack(got[i]), want)

"""The training operators together, as a block of a mixture-of-experts image
model uses them: group norm + SiLU, a projection, bias + dropout + residual, the
router's logits and its balance loss, with the gradient of all of it.

Against 64-bit autograd in the 2-norm. Every operator and every product (taken
in 64 bits and rounded once) is off by at most 2^-18 of its result in that norm
(64 roundings of 2^-24: sums by threads and trees); a gradient passes at most 12
of them, and a map in between stretches an error by at most 4 (1.5 from w, 1.13
from the activation, 1.25 from dropout, weights of norm about 2 beside a skip).
Errors that pass several maps come back small against the skip connection's own
share, so 12 * 4 * 2^-18 < 2^-12 is allowed."""
import numpy as np
import pytest
import torch

import row_wise_reduction_gb300 as ro
from oracle import training as O
from tests import gpu_util as gu

pytestmark = [pytest.mark.gpu, gu.requires_gpu]

G, K, P, SEED, COEF = 8, 2, 0.2, 77, 0.5


class Block:
    def __init__(self, B, S, C, E, padded, seed=1):
        g = torch.Generator().manual_seed(seed)

        def rnd(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g) * scale).cuda()

        self.B, self.S, self.C, self.E = B, S, C, E
        T = B * S
        self.x, self.dr = rnd(B, S, C), rnd(T, C)
        self.w, self.b, self.bias = 1 + rnd(C, scale=0.1), rnd(C, scale=0.1), rnd(C)
        self.W, self.R = rnd(C, C, scale=C**-0.5), rnd(C, E, scale=C**-0.5)
        self.mask = None
        if padded:
            self.mask = torch.rand(T, generator=g).cuda() < 0.7
        self.one = torch.full((1,), 40.0 * T, device="cuda")  # a gradient of the size of dr's

    def mm(self, a, b):
        return (a.double() @ b.double()).float()

    def step(self, at=None, stream=None, ws=None):
        T, C = self.B * self.S, self.C
        ws = ws or {}
        stats = torch.empty(self.B, G, 2, device="cuda")
        h = ro.rowops_groupnorm_act(self.x, G, self.w, self.b, 1e-5, "silu", stats=stats, workspace=ws.get("gn"),
                                    stream=stream).view(T, C)
        x2 = self.x.view(T, C)
        r = ro.rowops_bias_dropout_residual(self.mm(h, self.W), x2, self.bias, P, SEED, 5, device_offset=at,
                                            stream=stream)
        logits = self.mm(r, self.R)
        experts = logits.topk(K, dim=1).indices
        loss, counts = ro.rowops_router_balance_loss(logits, experts, COEF, self.mask, workspace=ws.get("balance"),
                                                     stream=stream)
        dlogits = ro.rowops_router_balance_loss_backward(logits, counts, K, self.one, COEF, self.mask, stream=stream)
        dr = self.dr + self.mm(dlogits, self.R.t())
        dz, dbias = ro.rowops_bias_dropout_residual_backward(dr, P, SEED, 5, device_offset=at,
                                                             workspace=ws.get("dropout"), stream=stream)
        dh = self.mm(dz, self.W.t()).view_as(self.x)
        dx, dw, db = ro.rowops_groupnorm_act_backward(self.x, dh, stats, G, self.w, self.b, "silu",
                                                      workspace=ws.get("gn_backward"), stream=stream)
        out = dict(r=r, loss=loss, counts=counts, dx=dx + dr.view_as(self.x), dw=dw, db=db, dbias=dbias,
                   dW=self.mm(h.t(), dz), dR=self.mm(r.t(), dlogits))
        return out, experts

    def workspaces(self):
        T, f = self.B * self.S, torch.float32

        def of(n):
            return torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")

        return dict(gn=of(ro.rowops_groupnorm_act_workspace_bytes(self.B, self.S, self.C, G, f)),
                    gn_backward=of(ro.rowops_groupnorm_act_backward_workspace_bytes(self.B, self.S, self.C, G, f)),
                    dropout=of(ro.rowops_bias_dropout_residual_backward_workspace_bytes(T, self.C, f)),
                    balance=of(ro.rowops_router_balance_loss_workspace_bytes(T, self.E, f)))

    def reference(self, experts, at=0):
        """The same values by 64-bit autograd, for the same mask and choices."""
        T, C, E = self.B * self.S, self.C, self.E
        leaf = {k: getattr(self, k).double().cpu().requires_grad_() for k in ("x", "w", "b", "bias", "W", "R")}
        v = leaf["x"].view(self.B, self.S, G, C // G)
        mean = v.mean(dim=(1, 3), keepdim=True)
        xh = ((v - mean) / (v.var(dim=(1, 3), keepdim=True, correction=0) + 1e-5).sqrt()).view(T, C)
        z = xh * leaf["w"] + leaf["b"]
        keep = torch.from_numpy(O.dropout_keep(np.arange(T), C, P, SEED, 5 + at))
        r = leaf["x"].view(T, C) + keep * O.dropout_scale(P) * ((z * torch.sigmoid(z)) @ leaf["W"] + leaf["bias"])
        prob = torch.softmax(r @ leaf["R"], dim=1)
        rows = torch.ones(T, dtype=torch.bool) if self.mask is None else self.mask.cpu()
        chosen = torch.bincount(experts.cpu()[rows].reshape(-1), minlength=E)
        n = int(rows.sum())
        loss = COEF * E * (chosen / (n * K) * prob[rows].sum(dim=0) / n).sum()
        ((r * self.dr.double().cpu()).sum() + loss * self.one.double().cpu()).sum().backward()
        grads = {"d" + k: t.grad for k, t in leaf.items()}
        return dict(grads, r=r.detach(), loss=loss.detach().view(1), counts=torch.cat([chosen, torch.tensor([n])]))


def near(got, want):
    for k, ref in want.items():
        if k == "counts":
            assert torch.equal(got[k].cpu(), ref)
            continue
        err = (got[k].double().cpu().view(ref.shape) - ref).norm() / ref.norm()
        assert err <= 2.0**-12, f"{k}: off by {float(err):.3g}"


def same(a, b):
    for k in a:
        assert torch.equal(a[k], b[k]), k


SHAPES = [(2, 64, 64, 8), (3, 77, 40, 5), (1, 1, 16, 4), (2, 2500, 128, 64)]


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("form", ["", "stream"])
@pytest.mark.parametrize("B,S,C,E", SHAPES)
def test_block_against_64_bit_autograd(B, S, C, E, form, padded, monkeypatch):
    if form:
        monkeypatch.setenv("ROWOPS_GROUPNORM", form)
    if padded and B * S == 1:
        return  # its only row would be left out or kept: the other case
    m = Block(B, S, C, E, padded)
    got, experts = m.step()
    near(got, m.reference(experts))


@pytest.mark.parametrize("form", ["", "stream"])
def test_block_captured_and_replayed(form, monkeypatch):
    """Two graphs of two blocks that share one set of workspaces, replayed in
    turn with new masks, against eager runs: the same bits."""
    if form:
        monkeypatch.setenv("ROWOPS_GROUPNORM", form)
    blocks = [Block(2, 600, 64, 8, True, seed=s) for s in (1, 2)]
    ws = blocks[0].workspaces()
    at = torch.zeros(1, dtype=torch.int64, device="cuda")
    graphs, outs = [], []
    for m in blocks:
        m.step(at, ws=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(m.step(at, ws=ws)[0])
        graphs.append(g)
    for k in (0, 3, -1):
        at.fill_(k)
        for g in graphs:
            g.replay()
        for m, o in zip(blocks, outs):
            eager, experts = m.step(at)
            same(o, eager)
        near(o, m.reference(experts, k))


def test_block_on_streams_of_its_own():
    """On another current stream, and with the stream as an argument: the bits
    of the default stream. Two blocks at the same time, with their own workspaces."""
    blocks = [Block(2, 600, 64, 8, True, seed=s) for s in (1, 2)]
    want = [m.step()[0] for m in blocks]
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    got = []
    for m, s in zip(blocks, streams):
        with torch.cuda.stream(s):
            got.append([m.step(ws=m.workspaces())[0] for _ in range(3)])
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for o in runs:
            same(w, o)
    with torch.cuda.stream(streams[0]):  # the products' stream, named for the operators
        named = blocks[0].step(stream=streams[0])[0]
        raw = blocks[0].step(stream=streams[0].cuda_stream)[0]
    torch.cuda.synchronize()
    same(want[0], named)
    same(want[0], raw)

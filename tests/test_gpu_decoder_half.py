"""The operators together, as a training step runs them: residual and norm, the gated block, its last projection, residual and
norm, a quantized output head, log probabilities with entropy; and backwards through all of them, against float64
autograd on the dequantized weights.

Tolerance: a value passes at most 12 roundings to bf16 between the inputs and an output or gradient (outputs of the calls, T and G of
the adapters, the sums of the residual stream), each at most 2^-8 of it: 12 * 2^-8 < 0.05 of the norm."""
import pytest
import torch

import bit_nf4_quantized_11_amd as Q
from helpers import log, require_gpu

pytestmark = pytest.mark.gpu

TOL = 0.05
D, N, V, R, S, EPS = 256, 704, 1000, 16, 0.5, 1e-5


def _bf(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen) * std).bfloat16().cuda()


class Model:
    """Weights on the GPU; names of the projections: gate, up, down, head."""
    sizes = {"gate": (N, D), "up": (N, D), "down": (D, N), "head": (V, D)}

    def __init__(self, seed):
        gen = torch.Generator().manual_seed(seed)
        self.w = {k: Q.qlora_quantize_nf4(_bf(gen, *s, std=0.06)) for k, s in self.sizes.items()}
        self.A = {k: _bf(gen, s[1], R, std=0.06) for k, s in self.sizes.items()}
        self.B = {k: _bf(gen, R, s[0], std=0.06) for k, s in self.sizes.items()}
        self.n1, self.n2 = ((1 + 0.2 * _bf(gen, D).float()).bfloat16() for _ in range(2))

    def linear(self, x, k):
        return Q.qlora_linear_fwd(x, self.w[k], self.A[k], self.B[k], S)

    def linear_bwd(self, d, x, T, k, grads):
        dx, grads["A_" + k], grads["B_" + k] = Q.qlora_linear_bwd(d, x, T, self.w[k], self.A[k], self.B[k], S)
        return dx

    def step(self, x, res, token, dlp, dent):
        """(outputs, gradients): the library's calls alone, but for the sum of the two gradients of the block's input."""
        y, h = Q.qlora_rms_norm(x, self.n1, res, EPS)
        H, G, U, Tg, Tu = Q.qlora_gated_fwd(y, self.w["gate"], self.w["up"], self.A["gate"], self.B["gate"], self.A["up"],
                                            self.B["up"], S)
        d, Td = self.linear(H, "down")
        y2, h2 = Q.qlora_rms_norm(d, self.n2, h, EPS)
        logits, Th = self.linear(y2, "head")
        lp, stats, ent, _, _ = Q.qlora_token_logprob(logits, token, entropy=True)
        g = {}
        dl = Q.qlora_token_logprob_bwd(logits, token, stats, dlp, ent, dent)
        dy2 = self.linear_bwd(dl, y2, Th, "head", g)
        dh2, g["n2"] = Q.qlora_rms_norm_bwd(dy2, h2, self.n2, eps=EPS)
        H = Q.qlora_gated_bwd(None, G, U, H=True)[2]      # (the forward's is not kept)
        dH = self.linear_bwd(dh2, H, Td, "down", g)
        dG, dU, _ = Q.qlora_gated_bwd(dH, G, U, dG=G, dU=U)
        dy = self.linear_bwd(dG, y, Tg, "gate", g) + self.linear_bwd(dU, y, Tu, "up", g)
        g["x"], g["n1"] = Q.qlora_rms_norm_bwd(dy, h, self.n1, dh2, eps=EPS)
        return {"h": h, "h2": h2, "logits": logits, "lp": lp, "entropy": ent}, g

    def exact(self, x, res, token, dlp, dent):
        leaf = lambda t: t.double().cpu().requires_grad_()
        p = {"x": leaf(x), "n1": leaf(self.n1), "n2": leaf(self.n2)}
        for k in self.sizes:
            p["A_" + k], p["B_" + k] = leaf(self.A[k]), leaf(self.B[k])
        W = {k: Q.qlora_dequant(w).double().cpu() for k, w in self.w.items()}
        lin = lambda t, k: t @ W[k].t() + S * (t @ p["A_" + k]) @ p["B_" + k]
        norm = lambda t, w: torch.nn.functional.rms_norm(t, (D,), w, EPS)
        h = p["x"] + res.double().cpu()
        y = norm(h, p["n1"])
        h2 = h + lin(torch.nn.functional.silu(lin(y, "gate")) * lin(y, "up"), "down")
        logits = lin(norm(h2, p["n2"]), "head")
        all_lp = torch.log_softmax(logits, -1)
        t = token.cpu()
        lp = torch.where(t >= 0, all_lp.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
        ent = -(all_lp.exp() * all_lp).sum(-1)
        loss = (lp * dlp.double().cpu()).sum() + (ent * dent.double().cpu()).sum()
        names = list(p)
        grads = dict(zip(names, torch.autograd.grad(loss, [p[k] for k in names])))
        return {"h": h, "h2": h2, "logits": logits, "lp": lp, "entropy": ent}, grads


@pytest.mark.parametrize("M", [1, 20, 200, 1300])
def test_training_step(M):
    require_gpu()
    model = Model(M)
    gen = torch.Generator().manual_seed(M + 1)
    x, res = _bf(gen, M, D), _bf(gen, M, D, std=2.0)
    token = torch.randint(0, V, (M,), generator=gen).cuda()
    if M > 2:
        token[1] = -100
    dlp, dent = (torch.randn(M, generator=gen) / M).cuda(), (0.3 * torch.randn(M, generator=gen) / M).cuda()
    got = model.step(x, res, token, dlp, dent)
    want = model.exact(x, res, token, dlp, dent)
    for a, b in zip(got, want):
        assert set(a) == set(b)
        for k in a:
            ref = b[k].detach()
            off = (a[k].double().cpu() - ref).norm() / ref.norm()
            log("decoder half", M, k, f"{off:.2e}")
            assert off <= TOL, (k, off)
    # the same bits again
    again = model.step(x, res, token, dlp, dent)
    for a, b in zip(got, again):
        assert all(torch.equal(a[k], b[k]) for k in a)


def test_captured_step_follows_its_inputs():
    """A whole step captured once and replayed on other inputs, eager steps and synchronizations between: their bits."""
    require_gpu()
    M = 70
    model = Model(3)
    gen = torch.Generator().manual_seed(9)
    new = lambda: [_bf(gen, M, D), _bf(gen, M, D), torch.randint(0, V, (M,), generator=gen).cuda(),
                   (torch.randn(M, generator=gen) / M).cuda(), (torch.randn(M, generator=gen) / M).cuda()]
    args = new()
    model.step(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, grads = model.step(*args)
    for _ in range(3):
        for a, b in zip(args, new()):
            a.copy_(b)
        eager, eg = model.step(*args)
        eager, eg = ({k: t.clone() for k, t in d.items()} for d in (eager, eg))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], eager[k]) for k in out) and all(torch.equal(grads[k], eg[k]) for k in grads)

"""Quantisation-aware training of routed experts on one GPU.

A small routed layer learns a fixed one of the same shape.  Every step uses the
operators together as a trainer would:

  route_qb               scores, balanced top-k and mixture weights
  balance_loss           per-expert counts and the auxiliary loss of the routes
  mxfp4_quantize         fp32 master weights and bf16 activations to MXFP4
  mxfp4_matmul           gate, up and output products of all experts
  mxfp4_matmul_backward  gradients of their rows and weights, passed straight
                         through the quantisation to the masters
  router_backward        gradient of the router logits from the mixture weights
                         and from the balance loss

    python examples/qat_experts.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantile_balanced_routing_gb300 as qb  # noqa: E402


def situ_glu(g, u, beta1=4.0, beta2=25.0):
    a = beta1 * torch.tanh(g / beta1)
    return a * torch.sigmoid(a) * (beta2 * torch.tanh(u / beta2))


def dispatch(idx, n):
    """Routes in expert order: each one's token and place in [T, k], and the experts' offsets."""
    T, k = idx.shape
    order = torch.argsort(idx.flatten(), stable=True)
    offsets = torch.zeros(n + 1, dtype=torch.int32, device=idx.device)
    offsets[1:] = torch.cumsum(torch.bincount(idx.flatten(), minlength=n), 0)
    return order // k, order, offsets


class RoutedExperts:
    """Router and SiTU-GLU experts with fp32 master weights."""

    def __init__(self, d, n, k, m, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        new = lambda *s: torch.randn(*s, generator=g, device="cuda") / s[-1] ** 0.5  # noqa: E731
        self.n, self.k = n, k
        self.masters = dict(router=new(n, d), gate=new(n, m, d), up=new(n, m, d), out=new(n, d, m))

    def step(self, x, target, balance=0.01):
        """(task loss, balance loss, gradients of the masters) for tokens x [T, d] bf16."""
        w = self.masters
        T, n, k = x.shape[0], self.n, self.k
        logits = x.float() @ w["router"].t()
        _, _, idx, mix, _ = qb.route_qb(logits, k, qb_sweeps=0)
        aux = qb.balance_loss(logits, idx)
        token, place, offsets = dispatch(idx, n)
        wq = {name: qb.mxfp4_quantize(w[name]) for name in ("gate", "up", "out")}

        rows = qb.mxfp4_quantize(x[token])
        g = qb.mxfp4_matmul(rows, wq["gate"], offsets).requires_grad_()
        u = qb.mxfp4_matmul(rows, wq["up"], offsets).requires_grad_()
        act = situ_glu(g.float(), u.float()).bfloat16()
        act_q = qb.mxfp4_quantize(act.detach())
        e = qb.mxfp4_matmul(act_q, wq["out"], offsets).float()
        share = mix.flatten()[place][:, None]
        y = torch.zeros(T, x.shape[1], device=x.device).index_add_(0, token, share * e)

        err = y - target
        dy = err[token] * (2.0 / err.numel())
        # the mixture weights are in route order: back to [T, k]
        d_mix = torch.empty(T * k, device=x.device)
        d_mix[place] = (dy * e).sum(1)
        d_act, d_out = qb.mxfp4_matmul_backward((dy * share).bfloat16(), act_q, wq["out"], offsets)
        d_g, d_u = torch.autograd.grad(act, (g, u), d_act)
        _, d_gate = qb.mxfp4_matmul_backward(d_g, rows, wq["gate"], offsets, need_dx=False)
        _, d_up = qb.mxfp4_matmul_backward(d_u, rows, wq["up"], offsets, need_dx=False)
        d_logits = qb.router_backward(logits, idx, dw=d_mix.view(T, k), dloss=torch.full_like(aux.loss, balance),
                                      counts=aux.counts, tokens=aux.tokens)
        grads = dict(router=d_logits.t() @ x.float(), gate=d_gate, up=d_up, out=d_out)
        return float(err.square().mean()), float(aux.loss.mean()), grads


def train(steps=60, tokens=512, d=256, n=16, k=2, m=128, lr=3e-3, seed=0, log=print):
    teacher, student = RoutedExperts(d, n, k, m, seed), RoutedExperts(d, n, k, m, seed)
    for name, w in student.masters.items():      # start near the teacher: fine-tuning, not pre-training
        w += 0.3 * w.std() * torch.randn(w.shape, generator=torch.Generator(device="cuda").manual_seed(seed + 1),
                                         device="cuda")
    opt = torch.optim.Adam(list(student.masters.values()), lr=lr)
    history = []
    data = torch.Generator(device="cuda").manual_seed(seed + 2)
    for i in range(steps):
        x = torch.randn(tokens, d, generator=data, device="cuda").bfloat16()
        logits = x.float() @ teacher.masters["router"].t()
        _, _, idx, mix, _ = qb.route_qb(logits, k, qb_sweeps=0)
        token, place, offsets = dispatch(idx, n)
        target = torch.zeros(tokens, d, device="cuda")
        for e in range(n):                       # the teacher in fp32, without quantisation
            a, b = int(offsets[e]), int(offsets[e + 1])
            r = x[token[a:b]].float()
            h = situ_glu(r @ teacher.masters["gate"][e].t(), r @ teacher.masters["up"][e].t())
            target.index_add_(0, token[a:b], mix.flatten()[place[a:b]][:, None] * (h @ teacher.masters["out"][e].t()))
        task, aux, grads = student.step(x, target)
        for name, w in student.masters.items():
            w.grad = grads[name]
        opt.step()
        history.append((task, aux))
        if log and (i % 10 == 0 or i == steps - 1):
            log(f"step {i:3d}  task loss {task:.5f}  balance loss {aux:.4f}")
    if qb.qbmoe_status(None, None):
        raise RuntimeError("a kernel reported a device status")
    return history


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 60)

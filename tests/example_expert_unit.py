"""A unit of experts trained in 8 bits, as a file that runs: tokens sorted by expert and written to their experts' rows,
the experts' MLPs by grouped products, their results brought back weighted, the backward pass the same way, and one
clipped AdamW step over the experts' matrices with states in 8 bits.  No count of tokens comes to the host, so a whole
step can be captured into a graph.  run() returns the loss before every step.
"""

import torch

import fsdp_sharded_optimizer_flatparameter_gb300 as zs

HP = {"lr": 3e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.0}
ALIGN = 128                     # rows of an expert, for the weight gradients' sums


class ExpertUnit:
    """`experts` MLPs of width c and inner width f (a multiple of 128) for m tokens with k choices each."""

    def __init__(self, m, k, experts, c, f, seed=0):
        self.m, self.k, self.experts, self.c, self.f = m, k, experts, c, f
        rows = self.rows = zs.expert_rows(m, k, experts, ALIGN)
        q, b = zs.q8_empty, lambda *shape: torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        i32 = lambda *shape: torch.empty(shape, dtype=torch.int32, device="cuda")  # noqa: E731
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda sigma, *shape: torch.randn(*shape, generator=gen, device="cuda") * sigma  # noqa: E731
        # parameters and their optimizer's arrays: per expert gate and up (2 f x c) and down (c x f)
        self.w_in, self.w_out = b(experts * 2 * f, c), b(experts * c, f)
        self.g_in, self.g_out = b(experts * 2 * f, c), b(experts * c, f)
        mats = lambda x: list(x.view(experts, -1))  # noqa: E731
        params, grads = mats(self.w_in) + mats(self.w_out), mats(self.g_in) + mats(self.g_out)
        self.master = [rand(c ** -0.5, 2 * f * c) for _ in range(experts)] + [rand(f ** -0.5, c * f) for _ in range(experts)]
        states = [(zs.state_zeros(p.numel()), zs.state_zeros(p.numel())) for p in params]
        for p, w in zip(params, self.master):
            p.copy_(w)
        self.tensors = zs.TensorList(grads, self.master, [s[0][0] for s in states], [s[1][0] for s in states], params=params,
                                     m_scales=[s[0][1] for s in states], v_scales=[s[1][1] for s in states])
        self.norm, self.partials = torch.empty(2, device="cuda"), torch.empty(1216, device="cuda")
        # operands of the products: the weights as they are and, per expert, transposed
        self.in8, self.in8_t, self.out8, self.out8_t = q(experts * 2 * f, c), q(experts * c, 2 * f), q(experts * c, f), q(experts * f, c)
        # places of the tokens and what is kept for the backward pass
        self.row_of, self.starts, self.counts = i32(m, k), i32(experts + 1), i32(experts)
        self.y, self.gate, self.up, self.h, self.dy, self.d = q(rows, c), q(rows, f), q(rows, f), q(rows, f), q(rows, c), q(rows, 2 * f)
        self.y_t, self.h_t, self.dy_t, self.d_t = q(c, rows), q(f, rows), q(c, rows), q(2 * f, rows)
        self.gu, self.o, self.dh, self.dn = b(rows, 2 * f), b(rows, c), b(rows, f), b(rows, c)
        self.out, self.dx, self.dweights = b(m, c), b(m, c), torch.empty(m, k, device="cuda")

    def forward(self, x, ids, weights):
        """x (bf16 [m, c]) + the weighted results of the experts ids (int32 or int64 [m, k]; weights fp32)."""
        f, c = self.f, self.c
        part = lambda q, n, e: (q[0][n * e:n * (e + 1)], q[1][n * e:n * (e + 1)])  # noqa: E731
        for e in range(self.experts):
            zs.zs_q8_encode(self.w_in[2 * f * e:2 * f * (e + 1)], part(self.in8, 2 * f, e), part(self.in8_t, c, e))
            zs.zs_q8_encode(self.w_out[c * e:c * (e + 1)], part(self.out8, c, e), part(self.out8_t, f, e))
        zs.zs_expert_sort(ids, ALIGN, self.row_of, self.starts, self.counts)
        zs.zs_expert_dispatch(x, self.row_of, self.starts, self.counts, y=self.y)
        zs.zs_q8_matmul_experts(self.y, self.in8, self.starts, self.gu)
        zs.zs_swiglu_q8(self.gu[:, :f], self.gu[:, f:], self.h, self.gate, self.up)
        zs.zs_q8_matmul_experts(self.h, self.out8, self.starts, self.o)
        zs.zs_expert_combine(self.o, self.row_of, weights, self.out, residual=x)
        return self.out

    def backward(self, dout, weights):
        """Gradients of x (returned), of the weights (dweights) and of the experts' matrices (g_in, g_out)."""
        f, nb = self.f, self.f // 128
        d, d_t = self.d, self.d_t
        zs.zs_expert_combine_backward(dout, self.o, self.row_of, weights, self.starts, self.counts, self.dweights, dy=self.dy)
        zs.zs_q8_matmul_experts(self.dy, self.out8_t, self.starts, self.dh)
        zs.zs_swiglu_backward_q8(self.dh, self.gate, self.up, (d[0][:, :f], d[1][:, :nb]), (d[0][:, f:], d[1][:, nb:]),
                                 (d_t[0][:f], d_t[1][:f]), (d_t[0][f:], d_t[1][f:]), self.h_t)
        zs.zs_q8_transpose(self.dy, self.dy_t)
        zs.zs_q8_matmul_experts_grad(self.dy_t, self.h_t, self.starts, self.g_out)
        zs.zs_q8_matmul_experts(self.d, self.in8_t, self.starts, self.dn)
        zs.zs_q8_transpose(self.y, self.y_t)
        zs.zs_q8_matmul_experts_grad(self.d_t, self.y_t, self.starts, self.g_in)
        zs.zs_expert_combine(self.dn, self.row_of, None, self.dx, residual=dout)
        return self.dx

    def step(self, t, max_norm=1.0):
        zs.zs_grad_norm(self.tensors, max_norm, self.partials, self.norm)
        zs.zs_adamw_tensors(self.tensors, HP, t, factor=self.norm[1:], seed=t)


def run(steps=20, m=512, k=2, experts=8, c=256, f=256):
    unit = ExpertUnit(m, k, experts, c, f)
    gen = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    x = rand(m, c).to(torch.bfloat16)
    weights, ids = rand(m, experts).softmax(1).topk(k, dim=1)
    target = x.float() + (x.float() @ (rand(c, c) * c ** -0.5)).tanh()
    losses = []
    for t in range(1, steps + 1):
        err = unit.forward(x, ids, weights.contiguous()).float() - target
        losses.append(err.square().mean())
        unit.backward((err * (2.0 / err.numel())).to(torch.bfloat16), weights.contiguous())
        unit.step(t)
    return [float(v) for v in losses]


if __name__ == "__main__":
    got = run()
    print("loss %.4f -> %.4f in %d steps" % (got[0], got[-1], len(got)))

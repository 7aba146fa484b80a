"""A transformer MLP unit trained in 8 bits between the ZeRO-3 gather and the sharded step, as a file that runs.

Each simulated rank borrows the unit's full parameters (zs_zero3_gather_unit), runs its own batch forward and
backward with the 8-bit operators straight on the flat buffers - weights are read and weight gradients written
at their places in them - and the unit's gradients are reduce-scattered and stepped (zs_zero3_rs_step_unit).
Between forward and backward only 8-bit activations are kept.  run() returns the loss before every step.
"""

import torch

import fsdp_sharded_optimizer_flatparameter_gb300 as zs

EPS = 1e-5


class Unit:
    """One rank's buffers for a unit of width c and inner width f (a multiple of 128) and m tokens."""

    def __init__(self, m, c, f):
        self.m, self.c, self.f = m, c, f
        q, b = zs.q8_empty, lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        self.w_in, self.w_in_t, self.w_out, self.w_out_t = q(2 * f, c), q(c, 2 * f), q(c, f), q(f, c)
        self.y, self.s_q8, self.gate, self.up, self.h = q(m, c), q(m, c), q(m, f), q(m, f), q(m, f)      # kept (but h)
        self.dy, self.dy_t, self.y_t, self.h_t = q(m, c), q(c, m), q(c, m), q(f, m)
        self.d, self.d_t = q(m, 2 * f), q(2 * f, m)
        self.gu, self.out, self.dh, self.dn, self.dx = b(m, 2 * f), b(m, c), b(m, f), b(m, c), b(m, c)
        self.s, self.rstd = b(m, c), torch.empty(m, device="cuda")
        self.partials = torch.empty(304, c, device="cuda")

    def views(self, plan, flat):
        """The norm's weight, the gate and up weight and the down weight inside a unit buffer."""
        at = [(plan.param(k)[1], plan.param(k)[2]) for k in range(3)]
        w = [flat[o:o + n] for o, n in at]
        return w[0], w[1].view(2 * self.f, self.c), w[2].view(self.c, self.f)

    def forward(self, weights, x, residual):
        norm, w_in, w_out = weights
        zs.zs_q8_encode(w_in, self.w_in, self.w_in_t)                       # both operand forms in one pass
        zs.zs_q8_encode(w_out, self.w_out, self.w_out_t)
        zs.zs_rmsnorm_q8(x, residual, norm, EPS, self.y, s=self.s, rstd=self.rstd, s_q8=self.s_q8)
        zs.zs_q8_matmul(self.y, self.w_in, self.gu)
        zs.zs_swiglu_q8(self.gu[:, :self.f], self.gu[:, self.f:], self.h, self.gate, self.up)
        zs.zs_q8_matmul(self.h, self.w_out, self.out)
        return self.out                                                     # the next unit's x; self.s its residual

    def backward(self, weights, grads, dout, ds, scale, first):
        """dout: gradient of the unit's output; ds: of the residual stream past it.  grads: the views of a flat
        gradient buffer; scale and first as in zs_accumulate_grad.  Returns the gradient of x and residual."""
        f, nb = self.f, self.f // 128
        half = lambda q, rows: ((q[0][:f], q[1][:f]), (q[0][f:], q[1][f:])) if rows else (  # noqa: E731
            (q[0][:, :f], q[1][:, :nb]), (q[0][:, f:], q[1][:, nb:]))
        zs.zs_q8_encode(dout, self.dy, self.dy_t)
        zs.zs_q8_matmul(self.dy, self.w_out_t, self.dh)
        zs.zs_swiglu_backward_q8(self.dh, self.gate, self.up, *half(self.d, False), *half(self.d_t, True), self.h_t)
        zs.zs_q8_matmul(self.dy_t, self.h_t, grads[2], scale, first)
        zs.zs_q8_matmul(self.d, self.w_in_t, self.dn)
        zs.zs_q8_transpose(self.y, self.y_t)
        zs.zs_q8_matmul(self.d_t, self.y_t, grads[1], scale, first)
        zs.zs_rmsnorm_backward(self.dn, self.s_q8, weights[0], self.rstd, self.dx, grads[0], self.partials, ds=ds, scale=scale,
                               first=first)
        return self.dx


def run(steps=20, n_d=2, m=512, c=256, f=512):
    plan = zs.Plan([(c,), (2 * f, c), (c, f)], n_d=n_d, stage=zs.ZS_STAGE_ZERO3)
    P = plan.padded
    gen = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    master = torch.zeros(P, device="cuda")
    for k, (shape, sigma) in enumerate(zip(plan.shapes, (0.0, c ** -0.5, f ** -0.5))):
        _, o, n = plan.param(k)
        master[o:o + n] = sigma * rand(n) if sigma else 1.0
    m1, v1 = torch.zeros_like(master), torch.zeros_like(master)
    shards = master.to(torch.bfloat16)
    full = [torch.empty(P, dtype=torch.bfloat16, device="cuda") for _ in range(n_d)]
    grads = [torch.zeros(P, dtype=torch.bfloat16, device="cuda") for _ in range(n_d)]
    hp = {"lr": 3e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.0}
    units = [Unit(m, c, f) for _ in range(n_d)]
    batch = [(rand(m, c).mul(0.3).to(torch.bfloat16), rand(m, c).to(torch.bfloat16)) for _ in range(n_d)]
    mix = rand(c, c) * c ** -0.5
    target = [((x.float() + r.float()) @ mix).tanh() for x, r in batch]
    losses = []
    for t in range(1, steps + 1):
        zs.zs_zero3_gather_unit(plan, 0, shards, full)
        loss = 0.0
        for q, unit in enumerate(units):
            weights = unit.views(plan, full[q])
            out = unit.forward(weights, *batch[q])
            err = out.float() - target[q]
            loss = loss + err.square().mean() / n_d
            dout = (err * (2.0 / err.numel())).to(torch.bfloat16)
            unit.backward(weights, unit.views(plan, grads[q]), dout, None, 1.0, True)
        zs.zs_zero3_rs_step_unit(plan, 0, grads, master, m1, v1, shards, hp, t)
        losses.append(loss)
    return [float(x) for x in losses]


if __name__ == "__main__":
    got = run()
    print("loss %.4f -> %.4f in %d steps" % (got[0], got[-1], len(got)))

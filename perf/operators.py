"""Cases of the 8-bit training operators: what they are given, what they compute, and in what sizes.

A transformer MLP unit trained next to the sharded step: its residual sum and root-mean-square norm leave
8-bit codes, its linear layers multiply 8-bit codes, and what the backward pass needs of the forward pass
is kept in 8 bits.  The operators, by the `kind` of a case:

  norm       residual addition and RMS norm, output in 8 bits (and the sum kept in 8 bits)
  norm_back  its backward pass, from the kept sum
  product    matrix product of two 8-bit matrices, bf16 result
  gate       silu(gate) * up in 8 bits, gate and up kept in 8 bits
  gate_back  its backward pass from the kept gate and up: the gradients and the recomputed output as the
             next products' 8-bit operands
  encode     a bf16 matrix to 8 bits, as it is and transposed
  turn       a kept 8-bit matrix to its transposed 8-bit form, for the weight gradient's product

Format: a matrix of R x C values is codes (R x C, e4m3) and scales (R x ceil(C / 128), e8m0, powers of
two); value = code * scale of its row's block of 128 columns.  A block's scale is the smallest 2^e with
max|value| <= 448 * 2^e, e >= -127 (a block of zeros: e = -127).

`own` selects the framework's kernels; otherwise run() computes in elementary 32-bit torch operations.
"""

import math

import torch

own = False

BLOCK = 128
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
PARTIALS = 304        # rows of the caller's buffer for partial sums over tokens
EPS = 1e-5


def listed():
    return [
        # one token through a 2048-wide layer: latency
        {"name": "norm_token", "kind": "norm", "rows": 1, "cols": 2048, "keep": False},
        # a long training batch at width 4096, the sum also kept in 8 bits for the backward pass
        {"name": "norm_batch", "kind": "norm", "rows": 16384, "cols": 4096, "keep": True},
        # a ragged batch of an odd width (rows that start at odd 2-byte addresses), sum kept in bf16
        {"name": "norm_back_ragged", "kind": "norm_back", "rows": 999, "cols": 2047, "kept": "bf16", "ds": False},
        # the long training batch's backward pass, from the 8-bit sum, with the residual path's gradient
        {"name": "norm_back_batch", "kind": "norm_back", "rows": 16384, "cols": 4096, "kept": "q8", "ds": True},
        # one token through gate and up of a 4096 / 11008 layer: the weights' bytes are the work
        {"name": "product_token", "kind": "product", "m": 1, "n": 22016, "k": 4096},
        # a few tokens through its down layer
        {"name": "product_few", "kind": "product", "m": 37, "n": 4096, "k": 11008},
        # a training batch through gate and up: the largest
        {"name": "product_batch", "kind": "product", "m": 8192, "n": 22016, "k": 4096},
        # weight gradient of gate and up at 2048 / 5504 over a ragged number of tokens
        {"name": "product_grad_ragged", "kind": "product", "m": 11008, "n": 2048, "k": 5003},
        # a training batch's activation at 11008
        {"name": "gate_batch", "kind": "gate", "rows": 8192, "cols": 11008},
        # a ragged batch's activation backward at 5504
        {"name": "gate_back_ragged", "kind": "gate_back", "rows": 5003, "cols": 5504},
        # a step's weights into both operand forms
        {"name": "encode_weights", "kind": "encode", "rows": 22016, "cols": 4096},
        # a kept batch into the weight gradient's operand
        {"name": "turn_kept", "kind": "turn", "rows": 8192, "cols": 4096},
    ]


def _size(rng, lo, hi, odd=0.3):
    """A size from lo to hi, spread over its logarithm; a multiple of 16 (where it can be) or any number."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() >= odd and n >= 16:
        n = n // 16 * 16
    return min(max(n, lo), hi)


def draw(rng):
    kind = rng.choice(["norm", "norm_back", "product", "product", "gate", "gate_back", "encode", "turn"])
    if kind == "product":
        while True:
            c = {"kind": kind, "m": _size(rng, 1, 8192), "n": _size(rng, 256, 22016), "k": _size(rng, 128, 11008)}
            if c["m"] * c["n"] * c["k"] <= 8192 * 22016 * 4096:
                return c
    if kind in ("norm", "norm_back"):
        c = {"kind": kind, "rows": _size(rng, 1, 16384), "cols": _size(rng, 512, 4096)}
        if kind == "norm":
            return dict(c, keep=rng.random() < 0.5)
        return dict(c, kept=rng.choice(["bf16", "q8"]), ds=rng.random() < 0.5)
    if kind in ("gate", "gate_back"):
        return {"kind": kind, "rows": _size(rng, 1, 8192), "cols": _size(rng, 512, 11008)}
    return {"kind": kind, "rows": _size(rng, 16, 22016 if kind == "encode" else 8192), "cols": _size(rng, 256, 4096)}


# ------------------------------------------------------------------ buffers and inputs

def _up(n, m):
    return -(-n // m) * m


def _q8(rows, cols, device):
    """An empty 8-bit matrix: codes with rows 16 bytes apart or a multiple, scales packed."""
    codes = torch.zeros(rows, _up(cols, 16), dtype=torch.uint8, device=device)[:, :cols]
    return codes.view(E4M3), torch.zeros(rows, _up(cols, BLOCK) // BLOCK, dtype=torch.uint8, device=device).view(E8M0)


def _normal(gen, rows, cols, sigma, spiky=0.0):
    """bf16 values ~ N(0, sigma^2); `spiky` of the columns are 20 times larger, as outlier channels are."""
    x = torch.randn(rows, cols, generator=gen, device="cuda", dtype=torch.float32).mul_(sigma)
    if spiky:
        x[:, torch.rand(cols, generator=gen, device="cuda") < spiky] *= 20.0
    return x.to(torch.bfloat16)


def _gradient(gen, rows, cols):
    """bf16 gradients ~ N(0, 5e-4^2), 0.1 % of the entries 100 times larger."""
    x = torch.randn(rows, cols, generator=gen, device="cuda", dtype=torch.float32).mul_(5e-4)
    x.mul_(1.0 + 99.0 * (torch.rand(rows, cols, generator=gen, device="cuda") < 1e-3))
    return x.to(torch.bfloat16)


def _encoded(x):
    """An 8-bit matrix made from x, in rows 16 bytes apart or a multiple."""
    q = _q8(x.shape[0], x.shape[1], x.device)
    codes, scales = _encode(x.float())
    q[0].copy_(codes)
    q[1].copy_(scales)
    return q


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    kind, s = case["kind"], {"case": case}
    if kind == "product":
        s["a"] = _encoded(_normal(gen, case["m"], case["k"], 1.0, 0.005))
        s["b"] = _encoded(_normal(gen, case["n"], case["k"], 0.02))
        s["out"] = torch.empty(case["m"], case["n"], dtype=torch.bfloat16, device="cuda")
        return s
    R, C = case["rows"], case["cols"]
    if kind == "norm":
        s.update(x=_normal(gen, R, C, 0.3), residual=_normal(gen, R, C, 1.0, 0.005),
                 weight=(1.0 + 0.1 * torch.randn(C, generator=gen, device="cuda")).to(torch.bfloat16),
                 y=_q8(R, C, "cuda"), s=torch.empty(R, C, dtype=torch.bfloat16, device="cuda"),
                 rstd=torch.empty(R, device="cuda"), s_q8=_q8(R, C, "cuda") if case["keep"] else None)
    elif kind == "norm_back":
        kept = _normal(gen, R, C, 1.0, 0.005)
        s.update(dy=_gradient(gen, R, C), ds=_gradient(gen, R, C) if case["ds"] else None,
                 weight=(1.0 + 0.1 * torch.randn(C, generator=gen, device="cuda")).to(torch.bfloat16),
                 rstd=torch.rsqrt(kept.float().square().mean(1) + EPS),
                 s=_encoded(kept) if case["kept"] == "q8" else kept,
                 dx=torch.empty(R, C, dtype=torch.bfloat16, device="cuda"),
                 dw=torch.empty(C, dtype=torch.bfloat16, device="cuda"),
                 partials=torch.empty(PARTIALS, C, device="cuda"))
    elif kind == "gate":
        both = _normal(gen, R, 2 * C, 1.0)          # the gate and up product's result: its two halves
        s.update(gate=both[:, :C], up=both[:, C:], h=_q8(R, C, "cuda"), gate_q=_q8(R, C, "cuda"),
                 up_q=_q8(R, C, "cuda"))
    elif kind == "gate_back":
        s.update(gate_q=_encoded(_normal(gen, R, C, 1.0)), up_q=_encoded(_normal(gen, R, C, 1.0)),
                 dh=_gradient(gen, R, C), dgate=_q8(R, C, "cuda"), dup=_q8(R, C, "cuda"),
                 dgate_t=_q8(C, R, "cuda"), dup_t=_q8(C, R, "cuda"), h_t=_q8(C, R, "cuda"))
    elif kind == "encode":
        s.update(x=_normal(gen, R, C, 0.02), q=_q8(R, C, "cuda"), q_t=_q8(C, R, "cuda"))
    else:
        s.update(q=_encoded(_normal(gen, R, C, 1.0, 0.005)), q_t=_q8(C, R, "cuda"))
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import fsdp_sharded_optimizer_flatparameter_gb300 as zs
    kind = s["case"]["kind"]
    if kind == "norm":
        zs.zs_rmsnorm_q8(s["x"], s["residual"], s["weight"], EPS, s["y"], s=s["s"], rstd=s["rstd"], s_q8=s["s_q8"])
        out = {"y": s["y"], "s": s["s"], "rstd": s["rstd"]}
        return dict(out, s_q8=s["s_q8"]) if s["s_q8"] is not None else out
    if kind == "norm_back":
        zs.zs_rmsnorm_backward(s["dy"], s["s"], s["weight"], s["rstd"], s["dx"], s["dw"], s["partials"], ds=s["ds"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if kind == "product":
        zs.zs_q8_matmul(s["a"], s["b"], s["out"])
        return {"out": s["out"]}
    if kind == "gate":
        zs.zs_swiglu_q8(s["gate"], s["up"], s["h"], s["gate_q"], s["up_q"])
        return {"h": s["h"], "gate_q": s["gate_q"], "up_q": s["up_q"]}
    if kind == "gate_back":
        zs.zs_swiglu_backward_q8(s["dh"], s["gate_q"], s["up_q"], s["dgate"], s["dup"], s["dgate_t"], s["dup_t"],
                                 s["h_t"])
        return {k: s[k] for k in ("dgate", "dup", "dgate_t", "dup_t", "h_t")}
    if kind == "encode":
        zs.zs_q8_encode(s["x"], s["q"], s["q_t"])
        return {"q": s["q"], "q_t": s["q_t"]}
    zs.zs_q8_transpose(s["q"], s["q_t"])
    return {"q_t": s["q_t"]}


def _blocks(v):
    """[R, C] -> [R, blocks, 128], zeros past the last column."""
    pad = _up(v.shape[1], BLOCK) - v.shape[1]
    return (torch.nn.functional.pad(v, (0, pad)) if pad else v).reshape(v.shape[0], -1, BLOCK)


def _encode(v):
    """fp32 [R, C] -> codes [R, C] and scales [R, blocks]."""
    b = _blocks(v)
    mant, ex = torch.frexp(b.abs().amax(2))                       # max = mant * 2^ex, mant in [0.5, 1) or 0
    e = torch.where(mant > 0.875, ex - 8, ex - 9).clamp_(min=-127)          # 448 = 0.875 * 2^9
    e = torch.where(mant == 0, torch.full_like(e, -127), e)
    inverse = ((127 - e) << 23).to(torch.int32).view(torch.float32)         # 2^-e
    codes = (b * inverse[:, :, None]).to(E4M3).reshape(v.shape[0], -1)
    return codes[:, :v.shape[1]], (e + 127).to(torch.uint8).view(E8M0)


def _decode(q):
    codes, scales = q
    wide = scales.float().repeat_interleave(BLOCK, dim=1)[:, :codes.shape[1]]
    return codes.float() * wide


def _plain(s):
    kind = s["case"]["kind"]
    if kind == "norm":
        total = s["x"].float() + s["residual"].float()
        rstd = torch.rsqrt(total.square().mean(1) + EPS)
        out = {"y": _encode(total * rstd[:, None] * s["weight"].float()), "s": total.to(torch.bfloat16), "rstd": rstd}
        return dict(out, s_q8=_encode(total)) if s["s_q8"] is not None else out
    if kind == "norm_back":
        kept = _decode(s["s"]) if s["case"]["kept"] == "q8" else s["s"].float()
        xhat, dy = kept * s["rstd"][:, None], s["dy"].float()
        g = dy * s["weight"].float()
        dx = s["rstd"][:, None] * (g - xhat * (g * xhat).mean(1, keepdim=True))
        if s["ds"] is not None:
            dx = dx + s["ds"].float()
        return {"dx": dx.to(torch.bfloat16), "dw": (dy * xhat).sum(0).to(torch.bfloat16)}
    if kind == "product":
        return {"out": (_decode(s["a"]) @ _decode(s["b"]).T).to(torch.bfloat16)}
    if kind == "gate":
        g, u = s["gate"].float(), s["up"].float()
        return {"h": _encode(g / (1.0 + torch.exp(-g)) * u), "gate_q": _encode(g), "up_q": _encode(u)}
    if kind == "gate_back":
        g, u, dh = _decode(s["gate_q"]), _decode(s["up_q"]), s["dh"].float()
        sig = 1.0 / (1.0 + torch.exp(-g))
        dg, du = dh * u * sig * (1.0 + g * (1.0 - sig)), dh * g * sig
        return {"dgate": _encode(dg), "dup": _encode(du), "dgate_t": _encode(dg.T), "dup_t": _encode(du.T),
                "h_t": _encode((g * sig * u).T)}
    if kind == "encode":
        v = s["x"].float()
        return {"q": _encode(v), "q_t": _encode(v.T)}
    return {"q_t": _encode(_decode(s["q"]).T)}


# ------------------------------------------------------------------ the definition in 64 bits

def _grid64(v):
    """The 8-bit form of v in 64 bits: (codes' values, scales' values), each block of 128 columns by itself."""
    R, C = v.shape
    nb = (C + 127) // 128
    b = torch.zeros(R, nb * 128, dtype=torch.float64, device=v.device)
    b[:, :C] = v
    b = b.view(R, nb, 128)
    top = b.abs().max(dim=2).values
    e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448.0))
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e))
    e = e.clamp(min=-127.0)
    scale = torch.exp2(e)
    t = b / scale[:, :, None]
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3.0)   # 3 bits of mantissa from 2^-6 up
    codes = torch.round(t / step) * step                                          # ties to even
    return codes.view(R, -1)[:, :C].contiguous(), scale


def _wide64(q):
    codes, scales = q[0].float().double(), q[1].float().double()
    column = torch.arange(codes.shape[1], device=codes.device) // 128
    return codes * scales[:, column]


def exact(case, seed):
    s, kind = prepare(case, seed), case["kind"]
    if kind == "norm":
        total = s["x"].double() + s["residual"].double()
        rstd = (total.pow(2).sum(1) / total.shape[1] + EPS).pow(-0.5)
        out = {"y": _grid64(total * rstd[:, None] * s["weight"].double()), "s": total, "rstd": rstd}
        if case["keep"]:
            out["s_q8"] = _grid64(total)
        return out
    if kind == "norm_back":
        kept = _wide64(s["s"]) if case["kept"] == "q8" else s["s"].double()
        r, dy = s["rstd"].double()[:, None], s["dy"].double()
        g = dy * s["weight"].double()
        along = (g * kept).sum(1, keepdim=True) / kept.shape[1]
        dx = r * g - r.pow(3) * kept * along
        if s["ds"] is not None:
            dx += s["ds"].double()
        return {"dx": dx, "dw": (dy * kept * r).sum(0)}
    if kind == "product":
        return {"out": torch.matmul(_wide64(s["a"]), _wide64(s["b"]).t())}
    if kind == "gate":
        g, u = s["gate"].double(), s["up"].double()
        return {"h": _grid64(g * torch.sigmoid(g) * u), "gate_q": _grid64(g), "up_q": _grid64(u)}
    if kind == "gate_back":
        g, u, dh = _wide64(s["gate_q"]), _wide64(s["up_q"]), s["dh"].double()
        p = torch.sigmoid(g)
        dg, du = dh * u * (p + g * p * (1.0 - p)), dh * g * p
        return {"dgate": _grid64(dg), "dup": _grid64(du), "dgate_t": _grid64(dg.t()), "dup_t": _grid64(du.t()),
                "h_t": _grid64((g * p * u).t())}
    if kind == "encode":
        v = s["x"].double()
        return {"q": _grid64(v), "q_t": _grid64(v.t())}
    return {"q_t": _grid64(_wide64(s["q"]).t())}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    kind = case["kind"]
    if kind == "product":
        m, n, k = case["m"], case["n"], case["k"]
        nb = -(-k // BLOCK)
        return {"bytes": (m + n) * (k + nb) + 2 * m * n, "flops": 2 * m * n * k}
    R, C = case["rows"], case["cols"]
    n, by_row, by_col = R * C, R * -(-C // BLOCK), C * -(-R // BLOCK)
    if kind == "norm":
        keep = 1 if case["keep"] else 0
        return {"bytes": n * (7 + keep) + by_row * (1 + keep) + 4 * R + 2 * C, "flops": n * (6 + 3 * keep)}
    if kind == "norm_back":
        kept = n + by_row if case["kept"] == "q8" else 2 * n
        return {"bytes": kept + 4 * n + (2 * n if case["ds"] else 0) + 4 * R + 4 * C, "flops": 10 * n}
    if kind == "gate":
        return {"bytes": 7 * n + 3 * by_row, "flops": 14 * n}
    if kind == "gate_back":
        return {"bytes": 9 * n + 4 * by_row + 3 * by_col, "flops": 30 * n}
    if kind == "encode":
        return {"bytes": 4 * n + by_row + by_col, "flops": 6 * n}
    return {"bytes": 2 * n + by_row + by_col, "flops": 6 * n}

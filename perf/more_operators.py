"""Cases of the operators of an expert unit's training step: what they are given, what they compute, in what sizes.

A unit of experts trained next to the sharded step: every token chooses some experts, its row goes to each of
them as the 8-bit operand of their products, comes back weighted, and the experts' many matrices are stepped in
one pass, with the optimizer's states in 8 or in 32 bits.  The operators, by the `kind` of a case:

  dispatch      tokens sorted by expert (every expert's rows start at a multiple of `align`), each token's row
                encoded in 8 bits and written to its places
  combine       the experts' rows back at their tokens: weighted sum, plus a residual
  combine_back  its backward pass: the rows' gradients in 8 bits at their places, the weights' gradients
  product       the experts' products: rows of expert e times expert e's matrix
  product_grad  the experts' weight gradients: a product per expert, summed over its rows
  adamw         AdamW over many tensors at once, after their gradients' norm where it is clipped

8-bit matrices are those of perf/operators.py: e4m3 codes, a power-of-two scale per row and 128 columns.

8-bit states of a tensor of n elements: e4m3 codes of m and of r = sqrt(v), and a 32-bit scale per 256 elements,
value = code * scale, scale = largest magnitude of the block / 448 (a block with none of 2^-100 or more is all
zeros).  A magnitude between two codes goes up with the probability of its distance from the lower one, by 16
random bits of its own: m's are the lower and r's the upper 16 of h(i), with
    mix(x) = murmur3's finalizer;  h(i) = mix(i ^ mix(mix(seed + 0x9e3779b9 * (t + 1)) + (i >> 32)))
for element i of tensor t, in 32 bits; r > 0 is never rounded to 0, so that a state that vanished beside its block's
largest cannot make a step large.

`own` selects the framework's kernels; otherwise run() computes in elementary 32-bit torch operations.
"""

import math

import torch

own = False

BLOCK, STATE_BLOCK = 128, 256
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
HP = {"lr": 1e-4, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1}
MAX_NORM = 1.0


def listed():
    return [
        # one token to 8 of 64 experts of width 2048: latency
        {"name": "dispatch_token", "kind": "dispatch", "tokens": 1, "choices": 8, "experts": 64, "cols": 2048, "align": 1},
        # a long training batch's tokens to 8 of 64 experts, rows of every expert at multiples of 128 for the
        # weight gradients' products
        {"name": "dispatch_batch", "kind": "dispatch", "tokens": 16384, "choices": 8, "experts": 64, "cols": 2048, "align": 128},
        # a ragged batch of an odd width (rows that start at odd 2-byte addresses) back from 2 of 8 experts
        {"name": "combine_ragged", "kind": "combine", "tokens": 999, "choices": 2, "experts": 8, "cols": 2047, "align": 128,
         "residual": True},
        # the long training batch back from its experts
        {"name": "combine_batch", "kind": "combine", "tokens": 16384, "choices": 8, "experts": 64, "cols": 2048, "align": 128,
         "residual": False},
        # a ragged batch's backward pass at width 4096
        {"name": "combine_back_ragged", "kind": "combine_back", "tokens": 1003, "choices": 2, "experts": 8, "cols": 4096, "align": 128},
        # the long training batch's backward pass
        {"name": "combine_back_batch", "kind": "combine_back", "tokens": 16384, "choices": 8, "experts": 64, "cols": 2048, "align": 128},
        # a few tokens through 16 experts of 4096 to 2048: the weights' bytes are the work
        {"name": "product_few", "kind": "product", "tokens": 37, "choices": 2, "experts": 16, "n": 2048, "k": 4096, "align": 1},
        # the long training batch through its 64 experts
        {"name": "product_batch", "kind": "product", "tokens": 16384, "choices": 8, "experts": 64, "n": 2048, "k": 2048, "align": 128},
        # the weight gradients of 8 experts of 5504 and 2048 over a ragged number of tokens
        {"name": "product_grad_ragged", "kind": "product_grad", "tokens": 3001, "choices": 2, "experts": 8, "m": 5504, "n": 2048},
        # those of the long training batch
        {"name": "product_grad_batch", "kind": "product_grad", "tokens": 16384, "choices": 8, "experts": 64, "m": 2048, "n": 2048},
        # a unit of 96 expert matrices of 2048 x 2048, and the vectors beside them, with states in 8 bits, clipped
        {"name": "adamw_experts", "kind": "adamw", "bits": 8, "big": 2048 * 2048, "n_big": 96, "small": 2048, "n_small": 4, "shift": 0,
         "grads": "bf16", "clip": True},
        # the matrices of 2048 x 5504 of a few dense layers with many odd small tensors, states in 32 bits
        {"name": "adamw_layers", "kind": "adamw", "bits": 32, "big": 2048 * 5504, "n_big": 12, "small": 2047, "n_small": 64, "shift": 0,
         "grads": "bf16", "clip": False},
    ]


def _size(rng, lo, hi, odd=0.3):
    """A size from lo to hi, spread over its logarithm; a multiple of 16 (where it can be) or any number."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() >= odd and n >= 16:
        n = n // 16 * 16
    return min(max(n, lo), hi)


def draw(rng):
    kind = rng.choice(["dispatch", "combine", "combine_back", "product", "product_grad", "adamw", "adamw"])
    if kind == "adamw":
        while True:
            c = {"kind": kind, "bits": rng.choice([8, 32]), "big": _size(rng, 1000, 1 << 26), "n_big": _size(rng, 1, 512, 1.0),
                 "small": _size(rng, 1, 5000), "n_small": _size(rng, 1, 64, 1.0), "shift": rng.choice([0, 0, rng.randrange(1, 8)]),
                 "grads": rng.choice(["bf16", "bf16", "fp32"]), "clip": rng.random() < 0.5}
            if c["big"] * c["n_big"] * (2 if c["bits"] == 32 else 1) <= 96 << 22:
                return c
    experts = _size(rng, 4, 128, 1.0)
    c = {"kind": kind, "tokens": _size(rng, 1, 16384), "choices": rng.randrange(1, min(8, experts) + 1), "experts": experts}
    if kind in ("dispatch", "combine", "combine_back"):
        c.update(cols=_size(rng, 256, 2048), align=rng.choice([1, 16, 128]))
        return dict(c, residual=rng.random() < 0.5) if kind == "combine" else c
    c.update({"n": _size(rng, 128, 2048), "k": _size(rng, 128, 2048), "align": rng.choice([1, 16, 128])} if kind == "product"
             else {"m": _size(rng, 128, 2048), "n": _size(rng, 128, 2048)})
    return c


# ------------------------------------------------------------------ buffers and inputs

def _up(n, m):
    return -(-n // m) * m


def _q8(rows, cols, device):
    """An 8-bit matrix of zeros: codes with rows 16 bytes apart or a multiple, scales packed."""
    codes = torch.zeros(rows, max(16, _up(cols, 16)), dtype=torch.uint8, device=device)[:, :cols]
    return codes.view(E4M3), torch.zeros(rows, _up(cols, BLOCK) // BLOCK, dtype=torch.uint8, device=device).view(E8M0)


def _capacity(case):
    """Rows that hold every choice with each expert's rows from a multiple of align on."""
    pairs, align = case["tokens"] * case["choices"], case.get("align", BLOCK)
    return _up(pairs + min(case["experts"], pairs) * (align - 1), align)


def _choices(gen, case):
    """The experts of each token, without repetition, the liked ones several times as often; 1 % of the choices dropped."""
    T, K, E = case["tokens"], case["choices"], case["experts"]
    liking = torch.randn(E, generator=gen, device="cuda") * 0.7
    score = liking - torch.log(-torch.log(torch.rand(T, E, generator=gen, device="cuda").clamp_(1e-9, 1 - 1e-7)))
    ids = score.topk(K, dim=1).indices.to(torch.int32)
    ids.masked_fill_(torch.rand(T, K, generator=gen, device="cuda") < 0.01, -1)
    return ids.contiguous()


def _normal(gen, rows, cols, sigma, spiky=0.0):
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
    q = _q8(x.shape[0], x.shape[1], x.device)
    codes, scales = _encode(x.float())
    q[0].copy_(codes)
    q[1].copy_(scales)
    return q


def _sizes(case):
    """The tensors' sizes: the small ones spread among the big ones."""
    every = max(1, case["n_big"] // case["n_small"])
    sizes, left = [], case["n_small"]
    for i in range(case["n_big"]):
        sizes.append(case["big"])
        if left and i % every == 0:
            sizes.append(case["small"])
            left -= 1
    return sizes + [case["small"]] * left


def _prepare_adamw(case, gen):
    """Tensors as views of flat buffers, each from a multiple of 256 elements on (plus `shift`), zeros between them."""
    sizes, shift, q = _sizes(case), case["shift"], case["bits"] == 8
    first, at = [], 0
    for n in sizes:
        first.append(at)
        at += _up(n, STATE_BLOCK)
    dev = "cuda"
    blocks = torch.tensor([_up(n, STATE_BLOCK) // STATE_BLOCK for n in sizes], device=dev)
    tensor_of = torch.repeat_interleave(torch.arange(len(sizes), device=dev), blocks)
    start = torch.tensor(first, device=dev)[tensor_of]
    inner = torch.arange(at // STATE_BLOCK, device=dev) * STATE_BLOCK - start        # a block's first element in its tensor
    real = torch.tensor(sizes, device=dev)[tensor_of] - inner                        # elements of the tensor from there on
    live = (torch.arange(STATE_BLOCK, device=dev) < real[:, None]).reshape(-1)

    def flat(dtype, values=None):
        t = torch.zeros(at + shift, dtype=dtype, device=dev)
        if values is not None:
            t[shift:].copy_(values)
        return t

    def normal(sigma):
        return torch.randn(at, generator=gen, device=dev).mul_(sigma).mul_(live)

    # gradients and states of blocks of different sizes, as rows of a matrix have them; 0.1 % far larger gradients
    level = torch.exp(torch.randn(at // STATE_BLOCK, generator=gen, device=dev)).repeat_interleave(STATE_BLOCK)
    grad_type = torch.float32 if case["grads"] == "fp32" else torch.bfloat16
    g = normal(2e-5).mul_(level)
    g.mul_(1.0 + 30.0 * (torch.rand(at, generator=gen, device=dev) < 1e-3))
    s = {"grad": flat(grad_type, g.to(grad_type)), "master": flat(torch.float32, normal(0.05)), "param": flat(torch.bfloat16)}
    del g
    m = normal(4e-6).mul_(level)
    v = normal(1.0).square_().add_(0.1).mul_(4e-10).mul_(level).mul_(level).mul_(live)
    if q:
        zero = torch.zeros((), dtype=torch.int32, device=dev)
        for name, x in (("m", m), ("v", v.sqrt_())):
            codes, scale = _state(x, zero, False)
            s[name] = flat(torch.uint8, codes.view(torch.uint8)).view(E4M3)
            s[name + "_scale"] = scale
    else:
        s.update(m=flat(torch.float32, m), v=flat(torch.float32, v))
    del m, v, level
    s.update(tensor_of=tensor_of, inner=inner, step=1000, out=torch.zeros(2, device=dev), partials=torch.empty(1216, device=dev))
    if own:          # the list of tensors that a training program makes once, next to its parameters
        import fsdp_sharded_optimizer_flatparameter_gb300 as zs
        view = lambda name: [s[name][shift + o:shift + o + n] for o, n in zip(first, sizes)]  # noqa: E731
        scale = lambda name: [s[name][o // 256:(o + n + 255) // 256] for o, n in zip(first, sizes)] if q else None  # noqa: E731
        s["tensors"] = zs.TensorList(view("grad"), view("master"), view("m"), view("v"), params=view("param"),
                                  m_scales=scale("m_scale"), v_scales=scale("v_scale"))
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    kind, s = case["kind"], {"case": case}
    if kind == "adamw":
        return dict(s, **_prepare_adamw(case, gen))
    T, K, E, rows = case["tokens"], case["choices"], case["experts"], _capacity(case)
    ids = _choices(gen, case)
    sort = {"row_of": torch.empty(T, K, dtype=torch.int32, device="cuda"), "starts": torch.empty(E + 1, dtype=torch.int32, device="cuda"),
            "counts": torch.empty(E, dtype=torch.int32, device="cuda")}
    if kind == "dispatch":
        return dict(s, **sort, ids=ids, x=_normal(gen, T, case["cols"], 1.0, 0.005), y=_q8(rows, case["cols"], "cuda"))
    # what comes after the sorting has its results
    row_of, starts, counts = _sort(ids, E, case.get("align", BLOCK))
    s.update(row_of=row_of, starts=starts, counts=counts)
    if kind in ("combine", "combine_back"):
        C = case["cols"]
        s.update(y=_normal(gen, rows, C, 1.0, 0.005), weights=torch.rand(T, K, generator=gen, device="cuda").softmax(1))
        if kind == "combine":
            return dict(s, residual=_normal(gen, T, C, 1.0) if case["residual"] else None,
                        out=torch.empty(T, C, dtype=torch.bfloat16, device="cuda"))
        return dict(s, dout=_gradient(gen, T, C), dy=_q8(rows, C, "cuda"), dweights=torch.empty(T, K, device="cuda"))
    held = (torch.arange(rows, device="cuda")[:, None] - starts[:-1]).ge(0).sum(1) - 1        # each row's expert
    held = torch.arange(rows, device="cuda") < (starts[:-1] + counts)[held]                    # and whether it holds a token
    s["bounds"] = starts.tolist()                # for the plain form, which goes expert by expert
    if kind == "product":
        n, k = case["n"], case["k"]
        x = _normal(gen, rows, k, 1.0, 0.005).mul_(held[:, None])
        return dict(s, a=_encoded(x), b=_encoded(_normal(gen, E * n, k, 0.02)),
                    out=torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda"))
    m, n = case["m"], case["n"]
    return dict(s, a=_encoded(_gradient(gen, m, rows).mul_(held)), b=_encoded(_normal(gen, n, rows, 1.0).mul_(held)),
                out=torch.empty(E * m, n, dtype=torch.bfloat16, device="cuda"))


# ------------------------------------------------------------------ one pass

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import fsdp_sharded_optimizer_flatparameter_gb300 as zs
    case, kind = s["case"], s["case"]["kind"]
    if kind == "dispatch":
        zs.zs_expert_sort(s["ids"], case["align"], s["row_of"], s["starts"], s["counts"])
        zs.zs_expert_dispatch(s["x"], s["row_of"], s["starts"], s["counts"], y=s["y"])
        return {k: s[k] for k in ("row_of", "starts", "counts", "y")}
    if kind == "combine":
        zs.zs_expert_combine(s["y"], s["row_of"], s["weights"], s["out"], residual=s["residual"])
        return {"out": s["out"]}
    if kind == "combine_back":
        zs.zs_expert_combine_backward(s["dout"], s["y"], s["row_of"], s["weights"], s["starts"], s["counts"], s["dweights"], dy=s["dy"])
        return {"dy": s["dy"], "dweights": s["dweights"]}
    if kind == "product":
        zs.zs_q8_matmul_experts(s["a"], s["b"], s["starts"], s["out"])
        return {"out": s["out"]}
    if kind == "product_grad":
        zs.zs_q8_matmul_experts_grad(s["a"], s["b"], s["starts"], s["out"])
        return {"out": s["out"]}
    s["step"] += 1
    factor = None
    if case["clip"]:
        zs.zs_grad_norm(s["tensors"], MAX_NORM, s["partials"], s["out"])
        factor = s["out"][1:]
    zs.zs_adamw_tensors(s["tensors"], HP, s["step"], factor=factor, seed=s["step"])
    return _adamw_outputs(s)


def _adamw_outputs(s):
    names = ["master", "param", "m", "v"] + (["m_scale", "v_scale"] if s["case"]["bits"] == 8 else []) + (["out"] if s["case"]["clip"] else [])
    return {k: s[k] for k in names}


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


def _sort(ids, experts, align):
    """(row of every choice or -1, first rows of the experts and the last one's end, their choices)."""
    flat = ids.reshape(-1).long()
    flat = torch.where((flat < 0) | (flat >= experts), torch.full_like(flat, experts), flat)
    counts = torch.bincount(flat, minlength=experts + 1)
    padded = (counts[:experts] + align - 1) // align * align
    starts = torch.cat([torch.zeros_like(padded[:1]), padded.cumsum(0)])
    order = torch.sort(flat, stable=True).indices
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(flat.numel(), device=flat.device) - (counts.cumsum(0) - counts)[flat[order]]
    row = torch.where(flat < experts, starts[flat] + rank, torch.full_like(flat, -1))
    return row.reshape(ids.shape).int(), starts.int(), counts[:experts].int()


def _scatter(q, values, row_of):
    """Encoded rows ([T, K] or [T, 1] of them) to their places; zeros in the rows beside them."""
    codes, scales = _encode(values)
    T, K = row_of.shape
    per = values.shape[0] // T
    src = torch.arange(T * K, device=row_of.device) // (K if per == 1 else 1)
    rows = row_of.reshape(-1).long()
    kept = rows >= 0
    for to, what in ((q[0].view(torch.uint8), codes.view(torch.uint8)), (q[1].view(torch.uint8), scales.view(torch.uint8))):
        to.zero_()
        to[rows[kept]] = what[src[kept]]


def _bits(s):
    """The 32 random bits of every element, as int64."""
    def mix(x):
        x = (x ^ (x >> 16)) * 0x85ebca6b & 0xffffffff
        x = (x ^ (x >> 13)) * 0xc2b2ae35 & 0xffffffff
        return x ^ (x >> 16)
    key = mix((s["step"] + 0x9e3779b9 * (s["tensor_of"] + 1)) & 0xffffffff)
    key = mix((key + (s["inner"] >> 32)) & 0xffffffff)
    at = s["inner"][:, None] + torch.arange(STATE_BLOCK, device=key.device)
    return mix((at & 0xffffffff) ^ key[:, None]).reshape(-1)


def _state(x, bits, positive):
    """fp32 values (whole blocks) in 8 bits: codes and scales.  bits: 16 random ones each."""
    b = x.view(-1, STATE_BLOCK)
    top = b.abs().amax(1)
    top = torch.where(top >= 2.0 ** -100, top, torch.zeros_like(top))
    inverse = torch.where(top > 0, 448.0 / top, torch.zeros_like(top))
    t = (b * inverse[:, None]).reshape(-1)
    code = ((t.abs() * 2.0 ** -120).view(torch.int32) + (bits << 4)) >> 20          # e4m3's bits are at fp32's 20 and up
    code.clamp_(max=0x7e)
    if positive:
        code = torch.maximum(code, (t > 0).int())
    code |= (torch.signbit(t).int() << 7)
    return code.to(torch.uint8).view(E4M3), top * (1.0 / 448.0)


def _scalars(step):
    lr, b1, b2, eps, wd = (float(torch.tensor(HP[k], dtype=torch.float32)) for k in ("lr", "beta1", "beta2", "eps", "weight_decay"))
    return b1, b2, eps, 1.0 - lr * wd, 1.0 - b1, 1.0 - b2, lr / (1.0 - b1 ** step), math.sqrt(1.0 - b2 ** step)


def _plain(s):
    case, kind = s["case"], s["case"]["kind"]
    if kind == "dispatch":
        s["row_of"], s["starts"], s["counts"] = _sort(s["ids"], case["experts"], case["align"])
        _scatter(s["y"], s["x"].float(), s["row_of"])
        return {k: s[k] for k in ("row_of", "starts", "counts", "y")}
    if kind in ("combine", "combine_back"):
        T, K = s["row_of"].shape
        kept = (s["row_of"] >= 0)[:, :, None]
        y = s["y"][s["row_of"].clamp(min=0).long().reshape(-1)].reshape(T, K, -1).float()
        w = s["weights"][:, :, None]
        if kind == "combine":
            out = (torch.where(kept, y, torch.zeros_like(y)) * w).sum(1)
            if s["residual"] is not None:
                out = out + s["residual"].float()
            return {"out": out.to(torch.bfloat16)}
        d = s["dout"].float()[:, None, :]
        _scatter(s["dy"], (d * w).reshape(T * K, -1), s["row_of"])
        dw = (y * d).sum(2)
        return {"dy": s["dy"], "dweights": torch.where(kept[:, :, 0], dw, torch.zeros_like(dw))}
    if kind in ("product", "product_grad"):
        a, b, spans = _decode(s["a"]), _decode(s["b"]), list(zip(s["bounds"], s["bounds"][1:]))
        if kind == "product":
            n = case["n"]
            done = torch.cat([a[lo:hi] @ b[e * n:(e + 1) * n].T for e, (lo, hi) in enumerate(spans)])
            s["out"][:done.shape[0]] = done.to(torch.bfloat16)
        else:
            s["out"].copy_(torch.cat([a[:, lo:hi] @ b[:, lo:hi].T for lo, hi in spans]))
        return {"out": s["out"]}
    # adamw, over the flat buffers that hold the tensors
    s["step"] += 1
    b1, b2, eps, decay, c1, c2, size, root = _scalars(s["step"])
    q, shift = case["bits"] == 8, case["shift"]
    g, p, m, v = (s[k][shift:] for k in ("grad", "master", "m", "v"))
    g = g.float()
    if case["clip"]:
        norm = g.double().square().sum().sqrt().float()
        s["out"][0] = norm
        s["out"][1] = (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)
        g = g * s["out"][1]
    if q:
        wide = lambda name: s[name + "_scale"].repeat_interleave(STATE_BLOCK)  # noqa: E731
        m1 = b1 * (m.float() * wide("m")) + c1 * g
        v1 = b2 * (v.float() * wide("v")).square() + c2 * (g * g)
    else:
        m1, v1 = b1 * m + c1 * g, b2 * v + c2 * (g * g)
    r = v1.sqrt()
    p.copy_(p * decay - size * (m1 / (r / root + eps)))
    s["param"][shift:].copy_(p)
    if q:
        h = _bits(s)
        for name, x, bits in (("m", m1, h & 0xffff), ("v", r, h >> 16)):
            codes, s[name + "_scale"] = _state(x, bits.int(), name == "v")
            s[name][shift:].view(torch.uint8).copy_(codes.view(torch.uint8))
    else:
        m.copy_(m1)
        v.copy_(v1)
    return _adamw_outputs(s)


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


def _placed64(rows, cols, row_of, values):
    """Rows of the 8-bit form of values at row_of among rows of zeros."""
    codes = torch.zeros(rows, cols, dtype=torch.float64, device=values.device)
    scales = torch.full((rows, (cols + 127) // 128), 2.0 ** -127, dtype=torch.float64, device=values.device)
    at = row_of.reshape(-1).long()
    c, e = _grid64(values)
    codes[at[at >= 0]], scales[at[at >= 0]] = c[at >= 0], e[at >= 0]
    return codes, scales


def _rows64(ids, experts, align):
    """Where each choice goes, by counting the choices before it that have the same expert."""
    flat = ids.reshape(-1).cpu()
    rows, first = torch.full(flat.shape, -1, dtype=torch.int64), 0
    for e in range(experts):
        mine = (flat == e).nonzero()[:, 0]
        rows[mine] = first + torch.arange(len(mine))
        first += -(-len(mine) // align) * align
    return rows.reshape(ids.shape).to(ids.device)


def _random64(seed, tensor, first, n, device):
    """The random bits of elements first .. first + n of a tensor."""
    word = 1 << 32

    def scramble(k):
        k = (k ^ (k >> 16)) * 2246822507 % word
        k = (k ^ (k >> 13)) * 3266489909 % word
        return k ^ (k >> 16)

    k = scramble(scramble((seed + 2654435769 * (tensor + 1)) % word) + (first >> 32))
    return scramble(torch.arange(first, first + n, dtype=torch.int64, device=device) % word ^ k)


def _code64(x, bits, positive):
    """One tensor's values in 8 bits, 64-bit arithmetic: the codes' values and the blocks' scales."""
    n = x.numel()
    b = torch.zeros(_up(n, 256), dtype=torch.float64, device=x.device)
    b[:n] = x
    top = b.view(-1, 256).abs().max(1).values
    top = top * (top >= 2.0 ** -100)
    t = (b.view(-1, 256) * (448.0 / top.clamp(min=1e-200))[:, None] * (top > 0)[:, None]).view(-1)[:n]
    a = t.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3.0)
    code = (torch.floor(a / step + bits.double() / 65536.0) * step).clamp(max=448.0)
    if positive:
        code = torch.where((a > 0) & (code == 0), torch.full_like(code, 2.0 ** -9), code)
    return torch.sign(t) * code, top / 448.0


def _exact_adamw(s):
    case, shift = s["case"], s["case"]["shift"]
    b1, b2, eps, decay, c1, c2, size, root = (float(torch.tensor(x, dtype=torch.float32)) for x in _scalars(s["step"] + 1))
    names = ["master", "param", "m", "v"] + (["m_scale", "v_scale"] if case["bits"] == 8 else [])
    out = {k: torch.zeros(s[k].shape, dtype=torch.float64, device="cuda") for k in names}
    factor = 1.0
    if case["clip"]:
        norm = math.sqrt(sum(float(x.double().pow(2).sum()) for x in s["grad"].split(1 << 26)))
        factor = min(1.0, MAX_NORM / (norm + 1e-6))
        out["out"] = torch.tensor([norm, factor], dtype=torch.float64, device="cuda")
    at = 0
    for t, n in enumerate(_sizes(case)):
        here, blocks = slice(shift + at, shift + at + n), slice(at // 256, (at + n + 255) // 256)
        of_block = torch.arange(n, device="cuda") // 256
        g, p, m, v = (s[k][here].float().double() for k in ("grad", "master", "m", "v"))
        g = g * factor
        if case["bits"] == 8:
            m, v = m * s["m_scale"][blocks].double()[of_block], (v * s["v_scale"][blocks].double()[of_block]) ** 2
        m, v = b1 * m + c1 * g, b2 * v + c2 * g * g
        p = p * decay - size * m / (torch.sqrt(v) / root + eps)
        out["master"][here], out["param"][here] = p, p
        if case["bits"] == 8:
            bits = _random64(s["step"] + 1, t, 0, n, "cuda")
            out["m"][here], out["m_scale"][blocks] = _code64(m, bits % 65536, False)
            out["v"][here], out["v_scale"][blocks] = _code64(torch.sqrt(v), bits // 65536, True)
        else:
            out["m"][here], out["v"][here] = m, v
        at += _up(n, 256)
    return out


def exact(case, seed):
    s, kind = prepare(case, seed), case["kind"]
    if kind == "adamw":
        return _exact_adamw(s)
    if kind == "dispatch":
        rows = _rows64(s["ids"], case["experts"], case["align"])
        values = s["x"].double()[:, None, :].expand(-1, case["choices"], -1).reshape(-1, case["cols"])
        return {"row_of": None, "starts": None, "counts": None, "y": _placed64(_capacity(case), case["cols"], rows, values)}
    if kind in ("combine", "combine_back"):
        T, K = s["row_of"].shape
        y, w = s["y"].double(), s["weights"].double()
        if kind == "combine":
            out = torch.zeros(T, case["cols"], dtype=torch.float64, device="cuda") if s["residual"] is None else s["residual"].double()
            for j in range(K):
                got = s["row_of"][:, j].long()
                out[got >= 0] += w[got >= 0, j, None] * y[got[got >= 0]]
            return {"out": out}
        d, dw = s["dout"].double(), torch.zeros(T, K, dtype=torch.float64, device="cuda")
        for j in range(K):
            got = s["row_of"][:, j].long()
            dw[got >= 0, j] = torch.einsum("tc,tc->t", d[got >= 0], y[got[got >= 0]])
        values = (w[:, :, None] * d[:, None, :]).reshape(T * K, -1)
        return {"dy": _placed64(_capacity(case), case["cols"], s["row_of"], values), "dweights": dw}
    a, b, at = _wide64(s["a"]), _wide64(s["b"]), s["bounds"]
    if kind == "product":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            out[at[e]:at[e + 1]] = torch.matmul(a[at[e]:at[e + 1]], b[e * case["n"]:(e + 1) * case["n"]].t())
        return {"out": out}
    return {"out": torch.cat([torch.matmul(a[:, at[e]:at[e + 1]], b[:, at[e]:at[e + 1]].t()) for e in range(case["experts"])])}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    kind = case["kind"]
    if kind == "adamw":
        n = sum(_sizes(case))
        blocks = sum(-(-x // STATE_BLOCK) for x in _sizes(case))
        grad = 4 if case["grads"] == "fp32" else 2
        states = 4 * n + 16 * blocks if case["bits"] == 8 else 16 * n
        return {"bytes": n * (grad * (2 if case["clip"] else 1) + 8 + 2) + states, "flops": n * (16 + (2 if case["clip"] else 0))}
    T, K, E = case["tokens"], case["choices"], case["experts"]
    pairs = T * K
    if kind in ("dispatch", "combine", "combine_back"):
        C, coded = case["cols"], case["cols"] + -(-case["cols"] // BLOCK)
        if kind == "dispatch":
            return {"bytes": 8 * pairs + 8 * E + 2 * T * C + pairs * coded, "flops": 3 * T * C}
        if kind == "combine":
            return {"bytes": 8 * pairs + 2 * pairs * C + (4 if case["residual"] else 2) * T * C, "flops": 2 * pairs * C}
        return {"bytes": 12 * pairs + 2 * T * C + pairs * (2 * C + coded), "flops": 6 * pairs * C}
    if kind == "product":
        n, k = case["n"], case["k"]
        used = min(E, pairs)                     # experts whose matrices are read
        return {"bytes": (pairs + used * n) * (k + -(-k // BLOCK)) + 2 * pairs * n, "flops": 2 * pairs * n * k}
    m, n = case["m"], case["n"]
    return {"bytes": (m + n) * (pairs + -(-pairs // BLOCK)) + 2 * E * m * n, "flops": 2 * pairs * m * n}

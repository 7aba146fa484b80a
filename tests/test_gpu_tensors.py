"""AdamW over many tensors and the gradients' norm: states of 32 bits bit for bit as in the flat step, states of 8 bits
against the 64-bit oracle, at sizes, addresses and values where they can go wrong."""

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_gb300 as zs
from oracle import q8, steps, tensors
from q8_helpers import U16, U32

pytestmark = pytest.mark.gpu

HP = {"lr": 3e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1}
SIZES = [1, 7, 8, 255, 256, 257, 0, 512, 1000, 4096, 5, 70001]


class Arrays:
    """Tensors of the given sizes `shift` elements into sentinel-filled buffers, the arrays of a list."""

    def __init__(self, sizes, bits, grad=torch.bfloat16, shift=0, seed=0, params=True, gap=32):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.sizes, self.bits = sizes, bits
        at = np.cumsum([0] + [-(-n // 32) * 32 + gap for n in sizes]).tolist()
        self.bufs = {}

        def make(name, dtype, fill):
            buf = torch.full((at[-1] + shift + 64,), fill, dtype=dtype, device="cuda")
            self.bufs[name] = (buf, fill)
            return [buf[o + shift:o + shift + n] for o, n in zip(at, sizes)]

        rand = lambda n: torch.randn(n, generator=g, device="cuda")  # noqa: E731
        self.grad, self.master = make("grad", grad, 5.0), make("master", torch.float32, 5.0)
        self.param = make("param", torch.bfloat16, 5.0) if params else None
        self.m, self.v = (make(k, torch.uint8 if bits == 8 else torch.float32, 0x55 if bits == 8 else 5.0) for k in "mv")
        self.ms = self.vs = None
        if bits == 8:
            self.ms, self.vs = (make(k, torch.float32, 5.0) for k in ("ms", "vs"))
            self.ms, self.vs = ([x[:-(-n // 256)] for x, n in zip(xs, sizes)] for xs in (self.ms, self.vs))
        for i, n in enumerate(sizes):
            self.grad[i].copy_(rand(n) * 1e-3 * torch.exp(rand(n)))
            self.master[i].copy_(rand(n))
            if bits == 8:
                for codes, scale, top in ((self.m[i], self.ms[i], 256), (self.v[i], self.vs[i], 127)):
                    c = torch.randint(0, top, (n,), generator=g, device="cuda")
                    codes.copy_(torch.where((c & 0x7f) == 0x7f, c - 1, c))
                    scale.copy_(1e-6 * torch.rand(len(scale), generator=g, device="cuda"))
            else:
                self.m[i].copy_(rand(n) * 1e-4)
                self.v[i].copy_(rand(n).square() * 1e-7)

    def list(self, **kw):
        return zs.TensorList(self.grad, self.master, self.m, self.v, params=self.param, m_scales=self.ms, v_scales=self.vs, **kw)

    def numpy(self):
        get = lambda xs: [x.double().cpu().numpy() if x.is_floating_point() else x.cpu().numpy() for x in xs]  # noqa: E731
        return {k: get(getattr(self, k)) for k in ("grad", "master", "m", "v") + (("param",) if self.param else ()) +
                (("ms", "vs") if self.bits == 8 else ())}

    def snapshot(self):
        torch.cuda.synchronize()
        return {k: b.clone() for k, (b, _) in self.bufs.items()}

    def assert_untouched_outside(self):
        for name, (buf, fill) in self.bufs.items():
            copy = buf.clone()
            base = buf.data_ptr()
            for x in getattr(self, name):
                o = (x.data_ptr() - base) // x.element_size()
                copy[o:o + x.numel()] = fill
            assert bool((copy == fill).all()), name


def _f32(x):
    return x.astype(np.float32)


@pytest.mark.parametrize("shift", [0, 1, 8, 13])
@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("params", [True, False])
def test_states_of_32_bits_are_the_flat_steps(shift, grad, params):
    a = Arrays(SIZES, 32, grad, shift, params=params)
    before = a.numpy()
    decays = [i % 3 != 1 for i in range(len(SIZES))]
    zs.zs_adamw_tensors(a.list(no_decay=[not d for d in decays]), HP, 7)
    after = a.numpy()
    for i, n in enumerate(SIZES):
        g = _f32(before["grad"][i])
        s = steps.adamw_scalars(dict(HP, weight_decay=HP["weight_decay"] if decays[i] else 0.0), 7)
        m = s["beta1"] * _f32(before["m"][i]) + s["c1"] * g
        v = s["beta2"] * _f32(before["v"][i]) + s["c2"] * (g * g)
        p = _f32(before["master"][i]) * s["decay"] - s["step_size"] * (m / (np.sqrt(v) / s["sqrt_bc2"] + s["eps"]))
        for k, w in (("m", m), ("v", v), ("master", p)):
            assert np.array_equal(_f32(after[k][i]), w), (k, n)
        if params:
            assert torch.equal(a.param[i], a.master[i].to(torch.bfloat16))
        assert np.array_equal(after["grad"][i], before["grad"][i])
    a.assert_untouched_outside()


def test_the_same_bits_as_zs_adamw_shard_step():
    n = 5000
    a = Arrays([n], 32, seed=3)
    plan = zs.Plan([(n,)], 1, stage=2)
    copy = [x.clone() for x in (a.grad[0], a.master[0], a.m[0], a.v[0])]
    out = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    for t in range(1, 4):
        zs.zs_adamw_tensors(a.list(), HP, t)
        zs.zs_adamw_shard_step(plan, -1, [copy[0]], zs.ZS_SHARDED, *copy[1:], [out], zs.ZS_SHARDED, HP, t)
    assert all(torch.equal(x, y) for x, y in zip((a.master[0], a.m[0], a.v[0], a.param[0]), (*copy[1:], out)))


def _check_state(codes, scale, x, err, random, positive):
    """Codes and scales of a state whose values are x, each known to err."""
    n = len(x)
    lo, hi = tensors.block_tops(np.maximum(np.abs(x) - err, 0)), tensors.block_tops(np.abs(x) + err)
    assert np.all(scale >= lo / 448 * (1 - 2 * U32)) and np.all(scale <= hi / 448 * (1 + 2 * U32)), "a block's scale"
    wide = np.repeat(scale, 256)[:n]
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.where(wide > 0, x / wide, 0.0)
        # the scale, its inverse (division within 2 units), the product, and what 2^-120 cuts off subnormal codes
        off = np.where(wide > 0, err / wide, 0.0) + 12 * U32 * np.abs(t) + 2.0 ** -29
    rank = lambda c: np.where(c & 0x80, -(c & 0x7f).astype(int), c.astype(int))  # noqa: E731
    a, b, got = (rank(c) for c in (tensors.codes(np.clip(t - off, -448, 448), random, False), tensors.codes(np.clip(t + off, -448, 448), random, False), codes))
    # a magnitude's random bits raise it whatever its sign, so the codes of an interval around 0 lie between those of its ends
    a, b = np.minimum(a, b), np.maximum(a, b)
    if positive:
        a, b = np.maximum(a, (x > err).astype(int) * (wide > 0)), np.maximum(b, (wide > 0).astype(int))
    assert np.all((got >= a) & (got <= b)), "a code: %s" % np.nonzero((got < a) | (got > b))[0][:5]


@pytest.mark.parametrize("shift", [0, 1, 8, 13])
@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("factor", [None, 0.37])
def test_states_of_8_bits(shift, grad, factor):
    a = Arrays(SIZES, 8, grad, shift, seed=1)
    before, f = a.numpy(), torch.tensor([9.0, factor or 0.0, 9.0], device="cuda")
    seed = 0x1234567
    zs.zs_adamw_tensors(a.list(), HP, 12, factor=None if factor is None else f[1:2], seed=seed)
    after = a.numpy()
    b1, b2, eps, decay, c1, c2, size, root = tensors.scalars(HP, 12)
    for i, n in enumerate(SIZES):
        g, p = before["grad"][i], before["master"][i]
        m, r = tensors.decode(before["m"][i], before["ms"][i]), tensors.decode(before["v"][i], before["vs"][i])
        x = g * (float(np.float32(factor)) if factor else 1.0)
        want, m1, v1 = tensors.adamw(g, p, m, r * r, HP, 12, float(np.float32(factor)) if factor else 1.0)
        # m: three roundings of its two parts; v: positive parts, five roundings, halved by the root, which has two more
        m_err, r1 = 4 * U32 * (np.abs(b1 * m) + np.abs(c1 * x)), np.sqrt(v1)
        random = tensors.random_bits(seed, i, n)
        _check_state(after["m"][i], after["ms"][i], m1, m_err, random & 0xffff, False)
        _check_state(after["v"][i], after["vs"][i], r1, 6 * U32 * r1, random >> 16, True)
        den = r1 / root + eps
        err = 3 * U32 * np.abs(p) + size * (m_err + 16 * U32 * np.abs(m1)) / den
        assert np.all(np.abs(after["master"][i] - want) <= err)
        assert np.all(np.abs(after["param"][i] - after["master"][i]) <= U16 * np.abs(after["master"][i]))
    a.assert_untouched_outside()


def test_the_place_in_the_list_and_the_address_do_not_matter_to_a_state():
    """The same tensor aligned and not, whole and strided blocks: the same bits; another place or seed: other bits."""
    sizes = [3000, 3000]
    runs = []
    for shift, seed in ((0, 5), (3, 5), (0, 6)):
        a = Arrays(sizes, 8, shift=shift, seed=9)
        zs.zs_adamw_tensors(a.list(), HP, 2, seed=seed)
        runs.append([x.clone() for x in (*a.m, *a.v, *a.ms, *a.master)])
    assert all(torch.equal(x, y) for x, y in zip(runs[0], runs[1]))
    assert not torch.equal(runs[0][0], runs[2][0]) and torch.equal(runs[0][6], runs[2][6])
    a = Arrays(sizes, 8, seed=9)
    for k in (a.grad, a.master, a.m, a.v, a.ms, a.vs):
        k[1].copy_(k[0])
    zs.zs_adamw_tensors(a.list(), HP, 2, seed=5)
    assert not torch.equal(a.m[0], a.m[1]) and torch.equal(a.master[0], a.master[1])


@pytest.mark.parametrize("count", [47, 48, 49, 447, 448, 449, 1000])
@pytest.mark.parametrize("bits", [8, 32])
def test_lists_longer_than_a_table(count, bits):
    """Every launch's part of the list, tensors of no elements among them; the norm over all of them."""
    rng = np.random.default_rng(count)
    sizes = rng.choice([0, 1, 3, 256, 300], count).tolist()
    a, one = Arrays(sizes, bits, seed=count), Arrays(sizes, bits, seed=count)
    zs.zs_adamw_tensors(a.list(), HP, 3, seed=11)
    partials, out = torch.empty(500, device="cuda"), torch.empty(2, device="cuda")
    zs.zs_grad_norm(a.list(), 0.5, partials, out)
    norm, factor = tensors.grad_norm([g.double().cpu().numpy() for g in a.grad], 0.5)
    # squares rounded and eight in a chain, three more additions, halved by the root; a rounding each of the root and the norm
    assert abs(float(out[0]) - norm) <= 8 * U32 * norm and abs(float(out[1]) - factor) <= 12 * U32 * factor
    # the oracle of the update: each tensor's own, in the same place of a list of its own
    key = {}
    for i in rng.choice(count, 12).tolist():
        part = [n if j == i else 0 for j, n in enumerate(sizes)]
        b = zs.TensorList([x if j == i else x[:0] for j, x in enumerate(one.grad)], *[[x if n else x[:0] for x, n in zip(xs, part)] for xs in (one.master, one.m, one.v)],
                          params=[x if n else x[:0] for x, n in zip(one.param, part)],
                          m_scales=one.ms and [x if n else x[:0] for x, n in zip(one.ms, part)], v_scales=one.vs and [x if n else x[:0] for x, n in zip(one.vs, part)])
        if i not in key:
            zs.zs_adamw_tensors(b, HP, 3, seed=11)
            key[i] = True
        for xs, ys in ((a.master, one.master), (a.m, one.m), (a.v, one.v), (a.param, one.param)):
            assert torch.equal(xs[i], ys[i])
    a.assert_untouched_outside()


def test_steps_from_zero_follow_states_of_32_bits():
    """40 steps of noisy gradients from states of zeros: the masters stay near those of 32-bit states.  An update is a sum
    over steps of m / r, each with roundings of m and r of at most 2^-3 and no bias but the root's, below 2^-6 of r: the way
    travelled differs by well under a tenth of its length."""
    n, gen = 20000, torch.Generator(device="cuda").manual_seed(3)
    base = torch.randn(n, generator=gen, device="cuda")
    size = torch.exp(torch.randn(n, generator=gen, device="cuda"))
    runs = []
    for bits in (8, 32):
        master, grad = base.clone(), torch.empty(n, device="cuda")
        if bits == 8:
            (m, ms), (v, vs) = zs.state_zeros(n), zs.state_zeros(n)
            ts = zs.TensorList([grad], [master], [m], [v], m_scales=[ms], v_scales=[vs])
        else:
            ts = zs.TensorList([grad], [master], [torch.zeros(n, device="cuda")], [torch.zeros(n, device="cuda")])
        noise = torch.Generator(device="cuda").manual_seed(4)
        for t in range(1, 41):
            grad.copy_(size * (0.3 + torch.randn(n, generator=noise, device="cuda")))
            zs.zs_adamw_tensors(ts, HP, t, seed=t)
        runs.append(master - base)
    assert float((runs[0] - runs[1]).norm()) <= 0.1 * float(runs[1].norm())


def test_the_stochastic_rounding_lets_an_average_move():
    """v starts at 1 and its gradients are 0: r falls by sqrt(beta2) a step, far below half a code; after 200 steps the mean
    over the elements is where it belongs (200 roundings of up to 2^-3 over 10^5 elements: a deviation of under 1 %)."""
    n, hp = 1 << 17, dict(HP, beta2=0.999)
    r = torch.rand(n, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") * 0.9 + 0.05
    r[::256] = 1.0
    scale = torch.full((n // 256,), 1.0 / 448, device="cuda")
    v = (r * 448).to(torch.float8_e4m3fn)
    start = v.float() / 448
    m, ms = zs.state_zeros(n)
    ts = zs.TensorList([torch.zeros(n, device="cuda", dtype=torch.bfloat16)], [torch.zeros(n, device="cuda")], [m], [v], m_scales=[ms], v_scales=[scale])
    for t in range(1, 201):
        zs.zs_adamw_tensors(ts, hp, t, seed=t)
    now = v.float() * scale.repeat_interleave(256)
    want = 0.999 ** 100
    live = torch.ones(n, dtype=torch.bool, device="cuda")
    live[::256] = False
    assert abs(float(now[live].mean() / start[live].mean()) / want - 1) <= 0.01
    assert not ms.any() and not m.float().any()


@pytest.mark.parametrize("bits", [8, 32])
def test_values_that_are_not_finite(bits):
    a = Arrays([600, 300], bits, seed=2)
    b = Arrays([600, 300], bits, seed=2)
    a.grad[0][5], a.grad[0][300], a.grad[0][599] = float("nan"), float("inf"), float("-inf")
    b.grad[0][5], b.grad[0][300], b.grad[0][599] = 0.0, 0.0, 0.0
    for x in (a, b):
        if bits == 8:
            x.m[0][[5, 300, 599]], x.v[0][[5, 300, 599]] = 0, 0
        zs.zs_adamw_tensors(x.list(), HP, 2, seed=1)
    hit = torch.zeros(600, dtype=torch.bool, device="cuda")
    hit[[5, 300, 599]] = True
    assert bool((~torch.isfinite(a.master[0][hit])).all()) and torch.equal(a.master[0][~hit], b.master[0][~hit])
    for x, y in ((a.m, b.m), (a.v, b.v)):
        assert torch.equal(x[0][~hit], y[0][~hit]) and torch.equal(x[1], y[1])
        assert bool((x[0][hit] == 0x7f).all()) if bits == 8 else not bool(torch.isfinite(x[0][hit]).any())
    if bits == 8:
        assert all(torch.equal(x, y) for x, y in zip(a.ms + a.vs, b.ms + b.vs))


def test_blocks_of_nothing_and_of_tiny_values():
    """States and gradients of zeros stay zeros; values below 2^-100 too; a root that is not zero keeps a code."""
    n = 1024
    grad = torch.zeros(n, device="cuda")
    grad[256:512] = 1e-32
    grad[512:768] = 1e-9
    grad[512] = 1.0
    (m, ms), (v, vs) = zs.state_zeros(n), zs.state_zeros(n)
    master = torch.ones(n, device="cuda")
    ts = zs.TensorList([grad], [master], [m], [v], m_scales=[ms], v_scales=[vs])
    zs.zs_adamw_tensors(ts, dict(HP, weight_decay=0.0), 1, seed=3)
    assert ms[[0, 1, 3]].tolist() == [0, 0, 0] and vs[[0, 1, 3]].tolist() == [0, 0, 0]
    assert not m.view(torch.uint8)[:512].any() and bool((v.view(torch.uint8)[513:768] == 1).all())
    assert bool((master[:256] == 1).all()) and bool((master[768:] == 1).all()) and bool(torch.isfinite(master).all())


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_norm_that_is_not_finite_leaves_the_step_out(bits, bad):
    a = Arrays([5000, 33], bits, seed=4)
    a.grad[1][32] = bad
    before = a.snapshot()
    partials, out = torch.empty(64, device="cuda"), torch.empty(2, device="cuda")
    zs.zs_grad_norm(a.list(), 1.0, partials, out)
    assert not bool(torch.isfinite(out[0])) and bool(torch.isnan(out[1]))
    zs.zs_adamw_tensors(a.list(), HP, 5, factor=out[1:], seed=5)
    assert all(torch.equal(x.view(torch.uint8), before[k].view(torch.uint8)) for k, x in a.snapshot().items())


@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n_partials", [2, 7, 5000])
@pytest.mark.parametrize("shift", [0, 5])
def test_norm(grad, n_partials, shift):
    a = Arrays(SIZES + [3000001], 32, grad, shift, seed=8)
    partials = torch.full((n_partials + 2,), -7.0, device="cuda")
    for max_norm in (1e-4, 1e4):
        out = torch.full((4,), -7.0, device="cuda")
        zs.zs_grad_norm(a.list(), max_norm, partials[1:-1], out[1:3])
        norm, factor = tensors.grad_norm([g.double().cpu().numpy() for g in a.grad], max_norm)
        assert abs(float(out[1]) - norm) <= 8 * U32 * norm and abs(float(out[2]) - factor) <= 12 * U32 * factor
        assert float(out[0]) == -7 and float(out[3]) == -7 and float(partials[0]) == -7 and float(partials[-1]) == -7
        again = torch.empty(2, device="cuda")
        zs.zs_grad_norm(a.list(), max_norm, partials[1:-1], again)
        assert torch.equal(again, out[1:3])


def test_lists_of_nothing():
    out = torch.full((2,), 5.0, device="cuda")
    empty = zs.TensorList([], [], [], [])
    zs.zs_adamw_tensors(empty, HP, 1)
    zs.zs_grad_norm(empty, 1.0, torch.empty(3, device="cuda"), out)
    assert out.tolist() == [0.0, 1.0]
    none = [torch.empty(0, device="cuda")]
    zs.zs_adamw_tensors(zs.TensorList(none, none, none, none), HP, 1)
    zs.zs_grad_norm(zs.TensorList(none, none, none, none), 1.0, torch.empty(3, device="cuda"), out)
    assert out.tolist() == [0.0, 1.0]


def test_streams_graphs_and_gradients_that_move():
    a, b = Arrays([70000, 31], 8, seed=6), Arrays([70000, 31], 8, seed=6)
    partials, out = torch.empty(100, device="cuda"), torch.empty(2, device="cuda")

    def step(x, t):
        zs.zs_grad_norm(t, 0.01, partials, out)
        zs.zs_adamw_tensors(t, HP, 4, factor=out[1:], seed=4)

    step(a, a.list())
    want = a.snapshot()
    t = b.list()
    moved = [g.clone() for g in b.grad]
    t.set_grads(moved)
    kept = b.snapshot()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(b, t)
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[k]) for k, x in b.snapshot().items())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b, t)
    for k, (buf, _) in b.bufs.items():
        buf.copy_(kept[k])
    graph.replay()
    assert all(torch.equal(x, want[k]) for k, x in b.snapshot().items())


def test_a_tensor_past_two_to_the_32():
    """Elements past 2^32: the last block's random bits take their upper part from the index."""
    n = (1 << 32) + 300
    grad, master = torch.zeros(n, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, device="cuda")
    (m, ms), (v, vs) = zs.state_zeros(n), zs.state_zeros(n)
    tail = 556                                                       # from the last block before 2^32
    g = torch.randn(tail, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    grad[-tail:] = g.to(torch.bfloat16)
    zs.zs_adamw_tensors(zs.TensorList([grad], [master], [m], [v], m_scales=[ms], v_scales=[vs]), HP, 1, seed=77)
    x = 0.1 * grad[-tail:].double().cpu().numpy()
    key = tensors.mix((77 + 0x9e3779b9) & 0xffffffff)
    random = np.array([tensors.mix((i & 0xffffffff) ^ tensors.mix((key + (i >> 32)) & 0xffffffff)) for i in range(n - tail, n)])
    b1, _, _, _, c1, _, _, _ = tensors.scalars(HP, 1)
    x = c1 * grad[-tail:].double().cpu().numpy()
    _check_state(m[-tail:].view(torch.uint8).cpu().numpy(), ms[-3:].double().cpu().numpy(), x, 2 * U32 * np.abs(x), random & 0xffff, False)
    assert bool((master[-tail:] != 0).any()) and not bool((master[:1 << 20] != 0).any())


def test_decoded_codes_are_the_formats():
    """Every code as m and as r: what the step reads of it."""
    n = 256
    codes = torch.arange(256, dtype=torch.uint8, device="cuda")
    m, ms = codes.clone(), torch.ones(1, device="cuda")
    v, vs = (codes & 0x7f).clone(), torch.ones(1, device="cuda")
    v[127] = v[255] = 1
    master, grad = torch.zeros(n, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    hp = dict(HP, weight_decay=0.0)
    zs.zs_adamw_tensors(zs.TensorList([grad], [master], [m], [v], m_scales=[ms], v_scales=[vs]), hp, 9, seed=1)
    c = codes.cpu().numpy()
    mv, rv = q8.VALUES[c], np.abs(q8.VALUES[np.where((c & 0x7f) == 127, 1, c & 0x7f)])
    want = tensors.adamw(np.zeros(n), np.zeros(n), mv, rv ** 2, hp, 9)[0]
    got = master.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = ~np.isnan(want)
    assert np.all(np.abs(got[fine] - want[fine]) <= 16 * U32 * np.abs(want[fine]))


def test_no_decay_of_states_of_8_bits():
    sizes = [3000, 3000, 77, 77]
    a = Arrays(sizes, 8, seed=5)
    before = a.numpy()
    zs.zs_adamw_tensors(a.list(no_decay=[True, False, True, False]), HP, 3, seed=1)
    for i, n in enumerate(sizes):
        m, r = tensors.decode(before["m"][i], before["ms"][i]), tensors.decode(before["v"][i], before["vs"][i])
        hp = dict(HP, weight_decay=0.0 if i % 2 == 0 else HP["weight_decay"])
        want, m1, v1 = tensors.adamw(before["grad"][i], before["master"][i], m, r * r, hp, 3)
        size = tensors.scalars(hp, 3)[6]
        err = 3 * U32 * np.abs(before["master"][i]) + 24 * U32 * size * (np.abs(m) + np.abs(before["grad"][i])) / (np.sqrt(v1) / tensors.scalars(hp, 3)[7] + HP["eps"])
        assert np.all(np.abs(a.master[i].double().cpu().numpy() - want) <= err)


@pytest.mark.parametrize("bits", [8, 32])
def test_steps_in_a_row_do_not_need_plain_launches(bits):
    """Launches that overlap the one before and launches that do not: the same bits after many steps without a wait,
    over tensors whose tiles and scales change hands between the SMs."""
    sizes, runs = [3 << 20, 5000, 1 << 20, 77777], []
    for dependent in (1, 0):
        a = Arrays(sizes, bits, seed=12)
        ts = a.list()
        partials, out = torch.empty(1216, device="cuda"), torch.empty(2, device="cuda")
        torch.cuda.synchronize()
        zs.zs_set_dependent_launch(dependent)
        try:
            for t in range(1, 13):
                zs.zs_grad_norm(ts, 0.01, partials, out)
                zs.zs_adamw_tensors(ts, HP, t, factor=out[1:], seed=t)
        finally:
            zs.zs_set_dependent_launch(1)
        runs.append(a.snapshot())
    assert all(torch.equal(runs[0][k], runs[1][k]) for k in runs[0])


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
def test_waits_that_run_out(bits, grad):
    """The call reports it, leaves nothing under way, writes nothing outside, and the next call on fresh arrays is right."""
    sizes = [1 << 20, 3000, 1 << 19]
    want = Arrays(sizes, bits, grad, seed=3)
    zs.zs_adamw_tensors(want.list(), HP, 2, seed=2)
    want = want.snapshot()
    try:
        for limit in (0, 0, 0, 1, 300, 3000):
            a = Arrays(sizes, bits, grad, seed=3)
            torch.cuda.synchronize()
            zs.zs_set_q8_wait_limit(limit)
            zs.zs_adamw_tensors(a.list(), HP, 2, seed=2)
            torch.cuda.synchronize()
            assert zs.zs_device_status(clear=True) in ((zs.ZS_DEVERR_TENSORS_WAIT,) if limit == 0 else (zs.ZS_DEVERR_NONE, zs.ZS_DEVERR_TENSORS_WAIT))
            a.assert_untouched_outside()
            zs.zs_set_q8_wait_limit()
            a = Arrays(sizes, bits, grad, seed=3)
            zs.zs_adamw_tensors(a.list(), HP, 2, seed=2)
            assert all(torch.equal(x, want[k]) for k, x in a.snapshot().items())
            assert zs.zs_device_status() == zs.ZS_DEVERR_NONE
    finally:
        zs.zs_set_q8_wait_limit()


def test_an_eps_that_is_subnormal_or_none():
    """Elements without a gradient and states of zeros: 0 / eps is 0 for any eps above 0."""
    grad = torch.zeros(512, device="cuda")
    grad[:256] = torch.randn(256, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    for eps in (1e-42, 1e-38, 1e-30):
        (m, ms), (v, vs) = zs.state_zeros(512), zs.state_zeros(512)
        master = torch.ones(512, device="cuda")
        zs.zs_adamw_tensors(zs.TensorList([grad], [master], [m], [v], m_scales=[ms], v_scales=[vs]), dict(HP, eps=eps, weight_decay=0.0), 1)
        assert bool((master[256:] == 1).all()) and bool(torch.isfinite(master).all()) and bool((master[:256] != 1).all())


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
def test_any_offset_of_any_array(bits, grad):
    """Each array at an offset of its own, tensors of many tiles, with values that are not finite, far too large and of zero
    in some blocks: the same bits as at aligned addresses, and nothing written beside them."""
    n, rng = 25000, np.random.default_rng(bits)
    names = ["grad", "master", "m", "v", "param"]
    a = Arrays([n], bits, grad, seed=7)
    for where, value in ((3000, float("nan")), (9000, float("inf")), (12345, 1e9), (24999, -1e9), (0, 1e5)):
        a.grad[0][where] = value
    a.grad[0][5000:7000] = 0.0
    for run in range(6):
        b = Arrays([n], bits, grad, seed=7)
        shifts = {k: int(rng.integers(0, 16)) for k in names}
        moved, bufs = {}, {}
        for k in names:
            x, fill = getattr(a, k)[0], 3
            bufs[k] = torch.full((n + 64,), fill, dtype=x.dtype, device="cuda")
            moved[k] = bufs[k][16 + shifts[k]:16 + shifts[k] + n]
            moved[k].copy_(x)
        scales = [[a.ms[0].clone()], [a.vs[0].clone()]] if bits == 8 else [None, None]
        ts = zs.TensorList([moved["grad"]], [moved["master"]], [moved["m"]], [moved["v"]], params=[moved["param"]], m_scales=scales[0], v_scales=scales[1])
        for k in ("master", "m", "v"):
            getattr(b, k)[0].copy_(getattr(a, k)[0])
        b.grad[0].copy_(a.grad[0])
        if bits == 8:
            b.ms[0].copy_(a.ms[0])
            b.vs[0].copy_(a.vs[0])
        for t in (1, 2):
            zs.zs_adamw_tensors(ts, HP, t, seed=t)
            zs.zs_adamw_tensors(b.list(), HP, t, seed=t)
        for k in names[1:]:
            # a NaN is a NaN, whichever
            x, y = (v if v.dtype == torch.uint8 else torch.nan_to_num(v, nan=7.5) for v in (moved[k], getattr(b, k)[0]))
            assert torch.equal(x, y), (k, shifts)
            outside = bufs[k].clone()
            outside[16 + shifts[k]:16 + shifts[k] + n] = 3
            assert bool((outside == 3).all()), (k, shifts)
        if bits == 8:
            assert torch.equal(scales[0][0], b.ms[0]) and torch.equal(scales[1][0], b.vs[0])


def test_waits_that_run_out_in_shifted_tiles():
    sizes = [1 << 19, 3000]
    want = Arrays(sizes, 8, shift=3, seed=3)
    zs.zs_adamw_tensors(want.list(), HP, 2, seed=2)
    want = want.snapshot()
    try:
        for limit in (0, 0, 1, 300, 3000, 30000):
            a = Arrays(sizes, 8, shift=3, seed=3)
            torch.cuda.synchronize()
            zs.zs_set_q8_wait_limit(limit)
            zs.zs_adamw_tensors(a.list(), HP, 2, seed=2)
            torch.cuda.synchronize()
            assert zs.zs_device_status(clear=True) in (zs.ZS_DEVERR_NONE, zs.ZS_DEVERR_TENSORS_WAIT)
            a.assert_untouched_outside()
            zs.zs_set_q8_wait_limit()
            a = Arrays(sizes, 8, shift=3, seed=3)
            zs.zs_adamw_tensors(a.list(), HP, 2, seed=2)
            assert all(torch.equal(x, want[k]) for k, x in a.snapshot().items())
            assert zs.zs_device_status() == zs.ZS_DEVERR_NONE
    finally:
        zs.zs_set_q8_wait_limit()


@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n_partials", [2, 5000])
@pytest.mark.parametrize("sizes", [[100000, 3, 70001], [300] * 500])
def test_norm_of_gradients_near_their_bound(grad, n_partials, sizes):
    """Gradients up to 2e18: the sum of their squares is far past fp32's range, their norm is not, and the step is taken."""
    a = Arrays(sizes, 32, grad, 5, seed=8)
    gen = torch.Generator(device="cuda").manual_seed(3)
    for g in a.grad:
        g.copy_(1.9e18 * (1 - 0.5 * torch.rand(len(g), generator=gen, device="cuda")))
    partials, out = torch.empty(n_partials, device="cuda"), torch.empty(2, device="cuda")
    zs.zs_grad_norm(a.list(), 1.0, partials, out)
    norm, factor = tensors.grad_norm([g.double().cpu().numpy() for g in a.grad], 1.0)
    assert norm > 2.0 ** 64
    # as in test_norm
    assert abs(float(out[0]) - norm) <= 8 * U32 * norm and abs(float(out[1]) - factor) <= 12 * U32 * factor
    before = [x.clone() for x in a.master]
    zs.zs_adamw_tensors(a.list(), HP, 2, factor=out[1:])
    assert all(bool(torch.isfinite(x).all()) and not torch.equal(x, y) for x, y in zip(a.master, before))


@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
def test_norm_of_tiny_gradients(grad):
    """Near fp32's least number a sum of squares is off by half of it for every square besides what is relative, so the root
    by that over the norm; gradients below 2^-75 have no square."""
    a = Arrays([50000, 7], 32, grad, 3, seed=8)
    partials, out = torch.empty(64, device="cuda"), torch.empty(2, device="cuda")
    for scale in (1e-17, 1e-18):                                     # of gradients of about 1e-3
        for g in a.grad:
            g.copy_(g.float() * scale)
        zs.zs_grad_norm(a.list(), 1e-7, partials, out)
        norm, factor = tensors.grad_norm([g.double().cpu().numpy() for g in a.grad], 1e-7)
        assert abs(float(out[0]) - norm) <= 8 * U32 * norm + 50007 * 2.0 ** -150 / norm
        assert abs(float(out[1]) - factor) <= 12 * U32 * factor
        for g in a.grad:
            g.copy_(g.float() / scale)
    for g in a.grad:
        g.fill_(2.5e-23)
    zs.zs_grad_norm(a.list(), 1e-7, partials, out)
    assert float(out[0]) == 0 and abs(float(out[1]) - 0.1) <= 4 * U32 * 0.1


@pytest.mark.parametrize("shift", [0, 1])
def test_a_root_of_zero_has_the_code_of_zero(shift):
    """v = 0 is the code 0 without a sign, whichever path stores it: in blocks of nothing, beside other elements, beside one
    that is not finite, in whole tiles and parts of one; a code 0x80 that is there already is read as 0."""
    n = 3 * 2048 + 100
    a = Arrays([n], 8, shift=shift, seed=3)
    a.m[0].zero_()
    a.v[0].zero_()
    a.v[0][::7] = 0x80
    a.grad[0][::3] = 0.0
    a.grad[0][3000:5000] = 0.0
    a.grad[0][5001] = float("inf")
    zs.zs_adamw_tensors(a.list(), HP, 2, seed=1)
    none = a.grad[0] == 0
    assert not bool(a.v[0][none].any()) and not bool((a.m[0][none] & 0x7f).any())
    assert bool((a.v[0][~none] > 0).all()) and bool((a.v[0] < 0x80).all())


@pytest.mark.parametrize("beta2", [0.0, 0.3, 0.95])
def test_a_block_beside_a_value_that_is_not_finite_keeps_its_bits(beta2):
    """A block with an infinity or NaN takes another path, with the library's root: its other elements have the same bits, for
    gradients of every exponent whose squares are not zero, 2^23 - 2^15 significands of each, squares below fp32's normal
    numbers among them."""
    n = 1 << 23
    hp = dict(lr=1.0, beta1=0.0, beta2=beta2, eps=0.0, weight_decay=0.0)
    significands = 1 + torch.arange(n, device="cuda", dtype=torch.float64) / n
    for e in range(-74, 14):
        runs = []
        for special in (0.0, float("inf")):
            grad = (significands * 2.0 ** e).float()
            grad[::256] = special
            (m, ms), (v, vs) = zs.state_zeros(n), zs.state_zeros(n)
            master = torch.zeros(n, device="cuda")
            zs.zs_adamw_tensors(zs.TensorList([grad], [master], [m], [v], m_scales=[ms], v_scales=[vs]), hp, 1, seed=e & 0xff)
            runs.append([x.view(torch.uint8).view(n // 256, -1) for x in (master, m, v, ms, vs)])
        for name, x, y, skip in zip(("master", "m", "v", "m's scales", "v's scales"), *runs, (4, 1, 1, 0, 0)):
            assert torch.equal(x[:, skip:], y[:, skip:]), (name, e)


def test_small_codes_beside_a_value_that_is_not_finite():
    """Blocks whose magnitudes span 2^20, so that many codes are subnormal: the same bits with and without an infinity."""
    n = 1 << 26
    hp = dict(lr=1.0, beta1=0.0, beta2=0.0, eps=0.0, weight_decay=0.0)
    gen = torch.Generator(device="cuda").manual_seed(5)
    for seed in range(6):
        small = torch.exp2(-20 * torch.rand(n, generator=gen, device="cuda")) * 2.0 ** (4 * seed - 12)
        runs = []
        for special in (0.0, float("inf")):
            grad = small.clone()
            grad[::256] = special
            (m, ms), (v, vs) = zs.state_zeros(n), zs.state_zeros(n)
            zs.zs_adamw_tensors(zs.TensorList([grad], [torch.zeros(n, device="cuda")], [m], [v], m_scales=[ms], v_scales=[vs]), hp, 1, seed=seed)
            runs.append([m.view(torch.uint8).view(-1, 256)[:, 1:], v.view(torch.uint8).view(-1, 256)[:, 1:], ms, vs])
        assert [int((x != y).sum()) for x, y in zip(*runs)] == [0, 0, 0, 0]


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("shift", [0, 3])
def test_a_step_that_gives_up_has_stepped_a_block_or_left_it(bits, shift):
    """A limit of 0 is reported; at any limit a block's arrays are all as before the step or all as after it.  Tensors of 19
    tiles and a part: some CTAs begin with a tile that the warps read themselves, while the next one arrives."""
    sizes = [20 * 2048 - 256] * 448
    blocks = lambda a, k: torch.cat([x.view(len(x) // 256 if len(x) > 200 else len(x), -1) for x in getattr(a, k)])  # noqa: E731
    names = ["master", "param", "m", "v"] + (["ms", "vs"] if bits == 8 else [])
    a = Arrays(sizes, bits, shift=shift, seed=3)
    kept = {k: b.clone() for k, (b, _) in a.bufs.items()}
    left = [blocks(a, k) for k in names]
    zs.zs_adamw_tensors(a.list(), HP, 2, seed=2)
    stepped = [blocks(a, k) for k in names]
    assert bool((left[0] != stepped[0]).any(1).all())
    try:
        for limit in (0,) * 12 + (1, 100, 1000, 3000, 10000, 30000) * 2:
            for k, (b, _) in a.bufs.items():
                b.copy_(kept[k])
            ts = a.list()
            torch.cuda.synchronize()
            zs.zs_set_q8_wait_limit(limit)
            zs.zs_adamw_tensors(ts, HP, 2, seed=2)
            torch.cuda.synchronize()
            code = zs.zs_device_status(clear=True)
            assert code in ((zs.ZS_DEVERR_TENSORS_WAIT,) if limit == 0 else (zs.ZS_DEVERR_NONE, zs.ZS_DEVERR_TENSORS_WAIT))
            now = [blocks(a, k) for k in names]
            new, old = ([(x == y).all(1) for x, y in zip(now, ref)] for ref in (stepped, left))
            new, old = torch.stack(new).all(0), torch.stack(old).all(0)
            assert bool((new | old).all()), "%d of %d blocks in part, limit %d" % (int((~(new | old)).sum()), len(new), limit)
            assert code != zs.ZS_DEVERR_NONE or bool(new.all())
            a.assert_untouched_outside()
    finally:
        zs.zs_set_q8_wait_limit()

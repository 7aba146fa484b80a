"""Tokens to their experts' rows and back against the 64-bit oracle: sorting, dispatch, combine and its gradient, at the
sizes, strides, choices and values where they can go wrong."""

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_gb300 as zs
from oracle import experts, q8
from q8_helpers import SENTINEL, U16, U32, Bf16Matrix, Q8Matrix, check_close, check_encoded, to64

pytestmark = pytest.mark.gpu

LAYOUTS = [dict(lead=0, pad=0), dict(lead=16, pad=16), dict(lead=1, pad=0), dict(lead=3, pad=5)]


@pytest.fixture(autouse=True)
def _status_stays_clear():
    yield
    torch.cuda.synchronize()
    assert zs.zs_device_status(clear=True) == zs.ZS_DEVERR_NONE


def _ids(rng, tokens, choices, n_experts, dropped=0.1):
    """Choices with repetitions, some experts liked far more, some never chosen, some choices dropped."""
    like = rng.random(n_experts) ** 4 * (rng.random(n_experts) < 0.8) + 1e-9
    ids = rng.choice(n_experts, (tokens, choices), p=like / like.sum())
    out = rng.random((tokens, choices)) < dropped
    return np.where(out, rng.choice([-1, n_experts, -2 ** 31, 2 ** 31 - 1], (tokens, choices)), ids)


class Sorted:
    """A sort's results on the GPU, between sentinels."""

    def __init__(self, ids, n_experts, align, dtype=torch.int32):
        t, k = ids.shape
        make = lambda n: torch.full((n + 2,), -77, dtype=torch.int32, device="cuda")  # noqa: E731
        self.bufs = make(t * k), make(n_experts + 1), make(n_experts)
        self.row_of, self.starts, self.counts = (b[1:-1] for b in self.bufs)
        self.row_of = self.row_of.view(t, k)
        zs.zs_expert_sort(torch.from_numpy(ids).to(dtype).cuda(), align, self.row_of, self.starts, self.counts)

    def check(self, ids, n_experts, align):
        for got, want in zip((self.row_of, self.starts, self.counts), experts.sort(ids, n_experts, align)):
            assert np.array_equal(got.cpu().numpy(), want)
        assert all(int(b[0]) == -77 and int(b[-1]) == -77 for b in self.bufs)
        return self


# ------------------------------------------------------------------ sort

SORTS = [(1, 1, 1, 1), (1, 8, 64, 128), (5, 2, 3, 1), (33, 1, 2, 16), (700, 3, 8, 128), (1000, 32, 5, 7), (4097, 1, 1024, 128),
         (2049, 2, 1000, 1), (2048, 2, 33, 128), (9001, 7, 129, 100), (40000, 6, 300, 128)]


@pytest.mark.parametrize("tokens,choices,n_experts,align", SORTS)
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort_is_exact(tokens, choices, n_experts, align, dtype):
    rng = np.random.default_rng(tokens + choices + n_experts)
    ids = _ids(rng, tokens, choices, n_experts)
    Sorted(ids, n_experts, align, dtype).check(ids, n_experts, align)


@pytest.mark.parametrize("what", ["one", "none", "rising", "falling"])
@pytest.mark.parametrize("tokens", [40, 5000])
def test_sort_of_unusual_choices(what, tokens):
    n_experts, i = 37, np.arange(tokens * 2).reshape(tokens, 2)
    ids = {"one": i * 0 + 36, "none": i * 0 - 1, "rising": i % 37, "falling": 36 - i * 37 // (2 * tokens)}[what]
    Sorted(ids, n_experts, 128).check(ids, n_experts, 128)


def test_sort_of_ids_past_32_bits():
    ids = np.array([[2 ** 32, 1], [2 ** 40 + 1, 0], [-2 ** 33, 1]])
    Sorted(ids, 2, 4, torch.int64).check(ids, 2, 4)


def test_sort_of_no_tokens():
    starts, counts = torch.full((6,), 9, dtype=torch.int32, device="cuda"), torch.full((5,), 9, dtype=torch.int32, device="cuda")
    none = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    zs.zs_expert_sort(none, 8, none, starts, counts)
    assert not starts.any() and not counts.any()


# ------------------------------------------------------------------ dispatch

ROWS = [(1, 1, 4, 1, 1), (3, 2, 4, 128, 128), (5, 2, 3, 16, 129), (40, 3, 8, 1, 520), (17, 4, 2, 7, 77), (130, 8, 16, 16, 1000),
        (70, 2, 5, 128, 2047), (9, 32, 40, 1, 300), (300, 1, 6, 32, 2048)]


@pytest.mark.parametrize("tokens,choices,n_experts,align,cols", ROWS)
@pytest.mark.parametrize("layout", LAYOUTS)
def test_dispatch_is_exact(tokens, choices, n_experts, align, cols, layout):
    rng = np.random.default_rng(tokens * 7 + cols)
    ids = _ids(rng, tokens, choices, n_experts)
    s = Sorted(ids, n_experts, align).check(ids, n_experts, align)
    row_of, starts, counts = experts.sort(ids, n_experts, align)
    rows = zs.expert_rows(tokens, choices, n_experts, align) + 3
    x = Bf16Matrix(tokens, cols, **layout)
    v = x.fill(rng.standard_normal((tokens, cols)) * np.exp(rng.uniform(-20, 20, (tokens, 1))))
    token, zero = experts.written(starts, counts, rows)
    want = experts.dispatch(v, row_of, rows)
    codes, scales = q8.encode(want)
    both = Q8Matrix(rows, cols), Bf16Matrix(rows, cols, **layout)
    for y, b in ((both[0], None), (None, both[1]), both):
        zs.zs_expert_dispatch(x.t, s.row_of, s.starts, s.counts, y=y and y.pair, y_bf16=b and b.t)
        if y:
            got = y.numpy()
            for g, w, nothing in ((got[0], codes, SENTINEL), (got[1], scales, SENTINEL)):
                assert np.array_equal(g[token], w[token]) and not g[zero].any() and (g[~token & ~zero] == nothing).all()
            y.assert_untouched_outside()
        if b:
            got = to64(b.t)
            assert np.array_equal(got[token], want[token]) and not got[zero].any() and (got[~token & ~zero] == -3).all()
            b.assert_untouched_outside()


def test_dispatch_of_values_at_the_edges():
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    x[0, 3], x[1, 200], x[2] = float("inf"), float("nan"), 3.3895313892515355e38
    row_of = torch.tensor([[3, 0], [1, -1], [2, -1], [-1, -1]], dtype=torch.int32, device="cuda")
    starts, counts = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 4], [4]))
    y = Q8Matrix(4, 256)
    zs.zs_expert_dispatch(x, row_of, starts, counts, y=y.pair)
    want = q8.encode(to64(x)[[0, 1, 2, 0]])
    a, b = q8.VALUES[y.numpy()[0]], q8.VALUES[want[0]]
    assert np.array_equal(y.numpy()[1], want[1]) and np.array_equal(np.isnan(a), np.isnan(b))
    assert np.array_equal(a[~np.isnan(a)], b[~np.isnan(b)])


def test_rows_past_the_matrix_are_left_out():
    """A matrix with fewer rows than the sort gave: nothing is written behind it, and nothing read from there."""
    rng = np.random.default_rng(3)
    tokens, choices, cols, rows = 50, 2, 200, 61
    ids = rng.integers(0, 4, (tokens, choices))
    s = Sorted(ids, 4, 16)
    row_of = experts.sort(ids, 4, 16)[0]
    x = torch.from_numpy(rng.standard_normal((tokens, cols))).to(torch.bfloat16).cuda()
    y, b = Q8Matrix(rows, cols), Bf16Matrix(rows, cols)
    zs.zs_expert_dispatch(x, s.row_of, s.starts, s.counts, y=y.pair, y_bf16=b.t)
    y.assert_untouched_outside()
    b.assert_untouched_outside()
    assert np.array_equal(to64(b.t), experts.dispatch(to64(x), row_of, rows))
    w = torch.rand(tokens, choices, device="cuda")
    out = torch.empty_like(x)
    zs.zs_expert_combine(b.t, s.row_of, w, out)
    want = experts.combine(to64(b.t), row_of, to64(w))
    check_close(to64(out), want, U16 * np.abs(want) + 4 * U32 * np.abs(want) + 1e-30, "out")
    dw = torch.full((tokens, choices), 5.0, device="cuda")
    zs.zs_expert_combine_backward(x, b.t, s.row_of, w, s.starts, s.counts, dweights=dw, dy=y.pair)
    y.assert_untouched_outside()
    assert np.array_equal(to64(dw) == 0, row_of >= rows)


# ------------------------------------------------------------------ combine

def _sum_bound(y, row_of, w, res, want):
    # one rounding to bf16; a chain of `choices` fused additions in fp32, each to half a step of at most the sum of magnitudes
    most = experts.combine(np.abs(y), row_of, None if w is None else np.abs(w), None if res is None else np.abs(res))
    return U16 * np.abs(want) + (row_of.shape[1] + 1) * U32 * most


@pytest.mark.parametrize("tokens,choices,n_experts,align,cols", ROWS)
@pytest.mark.parametrize("layout", LAYOUTS)
def test_combine(tokens, choices, n_experts, align, cols, layout):
    rng = np.random.default_rng(tokens * 5 + cols)
    ids = _ids(rng, tokens, choices, n_experts)
    row_of, starts, counts = experts.sort(ids, n_experts, align)
    rows = zs.expert_rows(tokens, choices, n_experts, align)
    y, res, out = Bf16Matrix(rows, cols, **layout), Bf16Matrix(tokens, cols, **layout), Bf16Matrix(tokens, cols, **layout)
    yv, rv = y.fill(rng.standard_normal((rows, cols))), res.fill(rng.standard_normal((tokens, cols)))
    nothing = np.ones(rows, bool)
    nothing[row_of[row_of >= 0]] = False
    y.t[torch.from_numpy(nothing).cuda()] = float("nan")               # rows without a token are not read
    yv[nothing] = 0
    w = torch.from_numpy(rng.standard_normal((tokens, choices)).astype(np.float32)).cuda()
    at = torch.from_numpy(row_of).int().cuda()
    for weights in (None, w):
        for r in (None, res):
            out.t.fill_(float("nan"))
            zs.zs_expert_combine(y.t, at, weights, out.t, residual=None if r is None else r.t)
            wv, rr = None if weights is None else to64(w), None if r is None else rv
            want = experts.combine(yv, row_of, wv, rr)
            check_close(to64(out.t), want, _sum_bound(yv, row_of, wv, rr, want), "out")
            out.assert_untouched_outside()
    zs.zs_expert_combine(y.t, at, w, res.t, residual=res.t)             # in place
    assert torch.equal(res.t, out.t)


@pytest.mark.parametrize("tokens,choices,n_experts,align,cols", ROWS + [(60, 3, 4, 8, 5000), (5, 5, 3, 1, 9001)])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_combine_backward(tokens, choices, n_experts, align, cols, layout):
    rng = np.random.default_rng(tokens * 3 + cols)
    ids = _ids(rng, tokens, choices, n_experts)
    s = Sorted(ids, n_experts, align)
    row_of, starts, counts = experts.sort(ids, n_experts, align)
    rows = zs.expert_rows(tokens, choices, n_experts, align) + 2
    token, zero = experts.written(starts, counts, rows)
    y, dout = Bf16Matrix(rows, cols, **layout), Bf16Matrix(tokens, cols, **layout)
    yv = y.fill(rng.standard_normal((rows, cols)))
    dv = dout.fill(rng.standard_normal((tokens, cols)) * np.exp(rng.uniform(-10, 10, (tokens, 1))))
    y.t[torch.from_numpy(~token).cuda()] = float("nan")
    yv[~token] = 0
    w = torch.from_numpy(rng.standard_normal((tokens, choices)).astype(np.float32)).cuda()
    w[0] = 0.0
    for weights in (w, None):
        wv = None if weights is None else to64(w)
        dy, dw = experts.combine_backward(dv, yv, row_of, wv)
        q, b = Q8Matrix(rows, cols), Bf16Matrix(rows, cols, **layout)
        got = torch.full((tokens, choices), float("nan"), device="cuda")
        zs.zs_expert_combine_backward(dout.t, y.t, s.row_of, weights, s.starts, s.counts, dweights=got, dy=q.pair, dy_bf16=b.t)
        # a lane's chain of 8, one addition of its two halves, 5 over the lanes, the chunks of 512, up to 8 warps
        terms = 8 + 1 + 5 + -(-cols // 512) + 8
        bound = terms * U32 * experts.combine_backward(np.abs(dv), np.abs(yv), row_of, None)[1]
        check_close(to64(got), dw, bound + 1e-38, "dweights")
        codes, scales = q.numpy()
        check_encoded((codes[token], scales[token]), dy[token], U32)
        assert not codes[zero].any() and not scales[zero].any() and (codes[~token & ~zero] == SENTINEL).all()
        q.assert_untouched_outside()
        check_close(to64(b.t)[token], dy[token], (U16 + U32) * np.abs(dy[token]), "dy")
        assert not to64(b.t)[zero].any() and (to64(b.t)[~token & ~zero] == -3).all()
        b.assert_untouched_outside()
        # each output by itself
        q1, b1, dw1 = Q8Matrix(rows, cols), Bf16Matrix(rows, cols, **layout), torch.empty_like(got)
        zs.zs_expert_combine_backward(dout.t, None, s.row_of, weights, s.starts, s.counts, dy=q1.pair)
        zs.zs_expert_combine_backward(dout.t, None, s.row_of, weights, s.starts, s.counts, dy_bf16=b1.t)
        zs.zs_expert_combine_backward(dout.t, y.t, s.row_of, weights, s.starts, s.counts, dweights=dw1)
        assert torch.equal(q1.codes, q.codes) and torch.equal(q1.scales, q.scales) and torch.equal(b1.t, b.t)
        assert torch.equal(dw1, got)


def test_combine_backward_of_values_at_the_edges():
    """Infinities and NaN in the gradient and in the weights, products that pass fp32: codes NaN, scales of the rest."""
    dout = torch.ones(6, 300, dtype=torch.bfloat16, device="cuda")
    dout[0, 5], dout[1, 140], dout[2, :] = float("inf"), float("nan"), 3e38
    w = torch.tensor([[1.0], [2.0], [4.0], [float("nan")], [float("inf")], [1e-30]], device="cuda")
    row_of = torch.arange(6, dtype=torch.int32, device="cuda").view(6, 1)
    starts, counts = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 6], [6]))
    dy = Q8Matrix(6, 300)
    zs.zs_expert_combine_backward(dout, None, row_of, w, starts, counts, dy=dy.pair)
    with np.errstate(over="ignore", invalid="ignore"):
        v = (to64(dout).astype(np.float32) * w.cpu().numpy()).astype(np.float64)
    want = q8.encode(v)
    a, b = q8.VALUES[dy.numpy()[0]], q8.VALUES[want[0]]
    assert np.array_equal(dy.numpy()[1], want[1]) and np.array_equal(np.isnan(a), np.isnan(b))
    assert np.array_equal(a[~np.isnan(a)], b[~np.isnan(b)])


def test_nothing_to_bring_back():
    """All choices dropped: the residual, or zeros; no tokens: nothing."""
    at = torch.full((5, 2), -1, dtype=torch.int32, device="cuda")
    y, res = torch.full((4, 100), float("nan"), dtype=torch.bfloat16, device="cuda"), torch.randn(5, 100, device="cuda").to(torch.bfloat16)
    out, dw = torch.empty_like(res), torch.full((5, 2), 3.0, device="cuda")
    zs.zs_expert_combine(y, at, torch.ones(5, 2, device="cuda"), out, residual=res)
    assert torch.equal(out, res)
    zs.zs_expert_combine(y, at, None, out)
    assert not out.any()
    starts, counts = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    zs.zs_expert_combine_backward(res, y, at, None, starts, counts, dweights=dw)
    assert not dw.any()
    zs.zs_expert_combine(y[:0], at, None, out, residual=res)
    assert torch.equal(out, res)
    zs.zs_expert_combine(y, at[:0], None, out[:0])
    zs.zs_expert_dispatch(res[:0], at[:0], starts, counts, y_bf16=y)
    assert torch.isnan(y).all()


def test_rows_past_four_gigabytes():
    """Rows 2^30 elements apart: the last ones past 2^32 bytes of codes and of bf16."""
    ld = 1 << 30
    codes = torch.as_strided(torch.zeros(5 * ld + 4096, dtype=torch.uint8, device="cuda"), (6, 300), (ld, 1))
    scales = torch.zeros(6, 3, dtype=torch.uint8, device="cuda")
    wide = torch.as_strided(torch.zeros(5 * ld + 4096, dtype=torch.bfloat16, device="cuda"), (6, 300), (ld, 1))
    x = torch.randn(3, 300, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    at = torch.tensor([[0, 5], [3, 2], [4, -1]], dtype=torch.int32, device="cuda")
    starts, counts = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 1, 6], [1, 4]))
    zs.zs_expert_dispatch(x, at, starts, counts, y=(codes, scales), y_bf16=wide)
    row_of = at.cpu().numpy()
    want = experts.dispatch(to64(x), row_of, 6)
    assert np.array_equal(to64(wide), want)
    assert np.array_equal(codes.cpu().numpy(), q8.encode(want)[0])
    out = torch.empty_like(x)
    zs.zs_expert_combine(wide, at, None, out)
    assert torch.equal(out.float(), x.float() * torch.tensor([[2.0], [2.0], [1.0]], device="cuda"))


def test_many_tokens():
    """Several tokens per warp and CTA, every row checked."""
    T, K, E, C = 20000, 4, 50, 640
    gen = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.randint(0, E, (T, K), generator=gen, device="cuda")
    row_of, starts, counts = (torch.empty(n, dtype=torch.int32, device="cuda") for n in ((T, K), (E + 1,), (E,)))
    zs.zs_expert_sort(ids, 128, row_of, starts, counts)
    assert np.array_equal(row_of.cpu().numpy(), experts.sort(ids.cpu().numpy(), E, 128)[0])
    rows = zs.expert_rows(T, K, E, 128)
    x = torch.randn(T, C, generator=gen, device="cuda").to(torch.bfloat16)
    y = torch.full((rows, C), 7.0, dtype=torch.bfloat16, device="cuda")
    q = zs.q8_empty(rows, C)
    zs.zs_expert_dispatch(x, row_of, starts, counts, y=q, y_bf16=y)
    flat = row_of.reshape(-1).long()
    want = torch.zeros_like(y)
    want[flat] = x.repeat_interleave(K, 0)
    want[int(starts[-1]):] = 7.0
    assert torch.equal(y, want)
    enc = zs.q8_empty(rows, C)
    zs.zs_q8_encode(want, enc)
    n = int(starts[-1])
    assert all(torch.equal(a[:n].view(torch.uint8), b[:n].view(torch.uint8)) for a, b in zip(q, enc))
    w, out, dw = torch.rand(T, K, generator=gen, device="cuda"), torch.empty_like(x), torch.empty(T, K, device="cuda")
    zs.zs_expert_combine(y, row_of, w, out)
    total = x.double() * w.double().sum(1, keepdim=True)
    assert bool(((out.double() - total).abs() <= total.abs() * (U16 + 8 * U32)).all())
    zs.zs_expert_combine_backward(x, y, row_of, w, starts, counts, dweights=dw, dy=q)
    want = x.double().square().sum(1, keepdim=True).expand(T, K)
    assert bool(((dw.double() - want).abs() <= 30 * U32 * want).all())
    dy = torch.zeros(rows, C, device="cuda")
    dy[flat] = x.float().repeat_interleave(K, 0) * w.reshape(-1, 1)
    have = zs.q8_empty(rows, C)
    back = q[0][:n].float() * q[1][:n].float().repeat_interleave(128, 1)[:, :C]
    top = torch.nn.functional.pad(dy[:n].abs(), (0, 0)).view(n, -1, 128).amax(2).repeat_interleave(128, 1)
    assert bool(((back - dy[:n]).abs() <= dy[:n].abs() * 2.0 ** -4 + top * 2.0 ** -17).all())
    del have

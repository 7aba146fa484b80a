"""The experts' 8-bit products against the 64-bit oracle: groups of every size, sums over an expert's rows, and starts that no
sort gives."""

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_gb300 as zs
from oracle import experts, q8
from q8_helpers import U16, U32, Bf16Matrix, Q8Matrix, check_close, encoded, to64

pytestmark = pytest.mark.gpu

LAYOUTS = [dict(lead=0, pad=0), dict(lead=3, pad=5)]


@pytest.fixture(autouse=True)
def _status_stays_clear():
    zs.zs_device_status(clear=True)
    yield
    zs.zs_set_q8_wait_limit()
    torch.cuda.synchronize()
    assert zs.zs_device_status(clear=True) == zs.ZS_DEVERR_NONE


def _bound(size, want, k):
    # as for the plain product: one rounding to bf16, products exact, an addition per 32 columns and those inside
    return U16 * np.abs(want) + (k / 8 + 16) * 2 * U32 * size


def _starts(sizes):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")


ROWS = [([1], 1, 1), ([3, 0, 5], 40, 100), ([0, 0, 7], 128, 128), ([256, 1, 255, 257], 300, 513), ([128] * 5, 256, 640),
        ([0, 600, 0, 3, 1, 0], 129, 1100), (list(range(40)), 65, 200), ([5] * 100, 24, 385), ([2000, 3], 1000, 300),
        ([1] * 1024, 17, 130), ([70, 900, 20], 700, 1),
        ([300, 0, 0, 0, 2], 300, 600), ([1, 31, 33, 64, 0, 129], 513, 385), ([17] * 9, 1000, 2048), ([130, 0, 60, 96], 70, 300), ([0, 0], 5, 10)]


@pytest.mark.parametrize("sizes,n,k", ROWS)
def test_rows(sizes, n, k):
    rng = np.random.default_rng(n * 3 + k)
    E, m = len(sizes), sum(sizes) + 5                              # five rows of nobody
    a, av = encoded(rng, m, k)
    b, bv = encoded(rng, E * n, k, 0.02)
    starts = _starts(sizes)
    host = starts.tolist()
    want, size = experts.product(av, bv, host), experts.product(np.abs(av), np.abs(bv), host)
    for layout in LAYOUTS:
        out = Bf16Matrix(m, n, **layout)
        out.t.fill_(9.0)
        zs.zs_q8_matmul_experts(a.pair, b.pair, starts, out.t)
        got = to64(out.t)
        check_close(got[:m - 5], want[:m - 5], _bound(size, want, k)[:m - 5], "out")
        assert (got[m - 5:] == 9).all()
        out.assert_untouched_outside()
        before = out.fill(rng.standard_normal((m, n)) * np.abs(want).max())
        zs.zs_q8_matmul_experts(a.pair, b.pair, starts, out.t, scale=-0.25, first=False)
        both = before - 0.25 * want
        check_close(to64(out.t)[:m - 5], both[:m - 5], (_bound(size, want, k) + U16 * np.abs(both) + 2 * U32 * np.abs(before))[:m - 5], "added")
        assert np.array_equal(to64(out.t)[m - 5:], before[m - 5:])


SUMS = [([128], 1, 1), ([128, 0, 256], 40, 100), ([0, 0, 1280], 128, 128), ([256, 128, 2304, 128], 300, 513), ([0] * 6 + [128], 70, 30),
        ([128] * 60, 65, 200), ([640, 0] * 9, 257, 300), ([2048, 128, 128, 0], 600, 1100), ([0, 0, 0], 300, 70)]


@pytest.mark.parametrize("sizes,m,n", SUMS)
def test_sums(sizes, m, n):
    rng = np.random.default_rng(m * 3 + n)
    E, k = len(sizes), sum(sizes) + 128 + 7                        # columns of nobody, NaN in them
    a, av = encoded(rng, m, k)
    b, bv = encoded(rng, n, k)
    for q, v in ((a, av), (b, bv)):
        q.codes[:, k - 135:] = 0x7f
        v[:, k - 135:] = 0
    starts = _starts(sizes)
    host = starts.tolist()
    want, size = experts.product_grad(av, bv, host), experts.product_grad(np.abs(av), np.abs(bv), host)
    for layout in LAYOUTS:
        out = Bf16Matrix(E * m, n, **layout)
        out.t.fill_(float("nan"))
        zs.zs_q8_matmul_experts_grad(a.pair, b.pair, starts, out.t)
        check_close(to64(out.t), want, _bound(size, want, max(sizes)) + 1e-38, "out")
        out.assert_untouched_outside()
        before = out.fill(rng.standard_normal((E * m, n)) * np.abs(want).max())
        out.t[0, 0] = -0.0
        before[0, 0] = 0.0
        zs.zs_q8_matmul_experts_grad(a.pair, b.pair, starts, out.t, scale=0.5, first=False)
        both = before + 0.5 * want
        check_close(to64(out.t), both, _bound(size, want, max(sizes)) + U16 * np.abs(both) + 2 * U32 * np.abs(before), "added")
        empty = np.repeat(np.array(sizes) == 0, m)
        assert np.array_equal(to64(out.t)[empty], before[empty])     # an expert without rows leaves its gradient
        out.assert_untouched_outside()


@pytest.mark.parametrize("k", [128, 300, 640, 1100])
def test_every_block_has_its_own_scales(k):
    """Groups of one block of rows and of many, every block of the sum with its own scale, sums of different lengths in
    turn: each tile's products read their own scales."""
    rng = np.random.default_rng(k)
    sizes = [300, 20, 1100, 0, 700, 128, 513]
    E, m, n, nb = len(sizes), sum(sizes), 900, -(-k // 128)

    def operand(rows, cols):
        codes = rng.integers(0, 0x50, (rows, cols)).astype(np.uint8)
        scales = rng.integers(117, 138, (rows, -(-cols // 128))).astype(np.uint8)
        return Q8Matrix(rows, cols).fill(codes, scales), q8.decode(codes, scales)

    a, av = operand(m, k)
    b, bv = operand(E * n, k)
    starts = _starts(sizes)
    out = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    for _ in range(3):
        zs.zs_q8_matmul_experts(a.pair, b.pair, starts, out)
    want = experts.product(av, bv, starts.tolist())
    check_close(to64(out), want, _bound(want, want, k), "rows")     # codes and scales here are positive
    sums = [128, k // 128 * 128, 0, 128 * 17, 128, 256, 128 * 9, 128 * 4, 128 * 5] * 2
    a, av = operand(700, sum(sums))
    b, bv = operand(600, sum(sums))
    starts = _starts(sums)
    out = torch.full((len(sums) * 700, 600), float("nan"), dtype=torch.bfloat16, device="cuda")
    for _ in range(3):
        zs.zs_q8_matmul_experts_grad(a.pair, b.pair, starts, out)
    want = experts.product_grad(av, bv, starts.tolist())
    check_close(to64(out), want, _bound(want, want, max(sums)), "sums")


def test_starts_that_no_sort_gives():
    """Out of order, out of range, overlapping: nothing outside out is written, and the next call is right."""
    rng = np.random.default_rng(8)
    m, n, k, E = 500, 200, 256, 6
    a, av = encoded(rng, m, k)
    b, bv = encoded(rng, E * n, k)
    x, xv = encoded(rng, 200, m)
    good = [0, 100, 100, 250, 300, 301, 500]
    out, grad = Bf16Matrix(m, n), Bf16Matrix(E * 200, 200)
    for bad in ([-5, 100, 2 ** 31 - 1, 50, -2 ** 31, 400, 600], [500, 400, 300, 200, 100, 50, 0], [0, 500, 0, 500, 0, 500, 0],
                [2 ** 31 - 1] * 7, [0, 2 ** 31 - 1, 0, 2 ** 31 - 1, 0, 2 ** 31 - 1, 2 ** 31 - 1]):
        starts = torch.tensor(bad, dtype=torch.int32, device="cuda")
        zs.zs_q8_matmul_experts(a.pair, b.pair, starts, out.t)
        zs.zs_q8_matmul_experts_grad(x.pair, x.pair, starts, grad.t)
        out.assert_untouched_outside()
        grad.assert_untouched_outside()
        zs.zs_q8_matmul_experts(a.pair, b.pair, torch.tensor(good, dtype=torch.int32, device="cuda"), out.t)
        want = experts.product(av, bv, good)
        check_close(to64(out.t), want, _bound(experts.product(np.abs(av), np.abs(bv), good), want, k), "out")


@pytest.mark.parametrize("grad", [False, True])
def test_waits_that_run_out(grad):
    g = torch.Generator(device="cuda").manual_seed(2)
    sizes = [256, 0, 640, 128, 1280, 896]

    def filled(rows, cols):
        q = zs.q8_empty(rows, cols)
        zs.zs_q8_encode(torch.randn(rows, cols, generator=g, device="cuda").to(torch.bfloat16), q)
        return q

    starts, total = _starts(sizes), sum(sizes)
    if grad:
        a, b, out = filled(1000, total), filled(900, total), torch.empty(6000, 900, dtype=torch.bfloat16, device="cuda")
    else:
        a, b, out = filled(total, 700), filled(6 * 900, 700), torch.empty(total, 900, dtype=torch.bfloat16, device="cuda")
    call = lambda: (zs.zs_q8_matmul_experts_grad if grad else zs.zs_q8_matmul_experts)(a, b, starts, out)  # noqa: E731
    call()
    want = out.clone()
    for limit in (0, 0, 0, 1, 300, 3000):
        zs.zs_set_q8_wait_limit(limit)
        call()
        torch.cuda.synchronize()
        assert zs.zs_device_status(clear=True) in ((zs.ZS_DEVERR_MATMUL_WAIT,) if limit == 0 else (zs.ZS_DEVERR_NONE, zs.ZS_DEVERR_MATMUL_WAIT))
        zs.zs_set_q8_wait_limit()
        call()
        assert torch.equal(out, want)


@pytest.mark.parametrize("n", [1, 7, 20, 31, 33, 44, 97, 230, 700])
@pytest.mark.parametrize("align", [8, 16])
@pytest.mark.parametrize("grad", [False, True])
def test_out_as_the_first_columns_of_wider_rows(grad, align, n):
    """Rows of out that start on 16 or 32 bytes and end inside them: the columns beside keep what they hold."""
    rng = np.random.default_rng(n + align)
    k = 384 if grad else 200
    sizes = [128, 0, 256] if grad else [300, 0, 160, 500]          # past the few rows of an expert
    E, starts = len(sizes), _starts(sizes)
    rows = 300 if grad else sum(sizes)
    a, av = encoded(rng, rows, k)
    b, bv = encoded(rng, n if grad else E * n, k)
    oracle, call = (experts.product_grad, zs.zs_q8_matmul_experts_grad) if grad else (experts.product, zs.zs_q8_matmul_experts)
    host = starts.tolist()
    want, size = oracle(av, bv, host), oracle(np.abs(av), np.abs(bv), host)
    for more in (0, align):
        out = Bf16Matrix(len(want), n, pad=-n % align + more)
        out.t.fill_(float("nan"))
        for _ in range(3):
            call(a.pair, b.pair, starts, out.t)
        check_close(to64(out.t), want, _bound(size, want, k) + 1e-38, "out")
        out.assert_untouched_outside()

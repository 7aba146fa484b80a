"""Tokens to their experts' rows and back in 64-bit floating point, and the experts' products, straight from their
definitions (include/zs.h, "experts").  Matrices are numpy arrays of float64; row_of has -1 for a dropped choice."""

import numpy as np


def sort(ids, n_experts, align):
    """(row_of, starts, counts): choice by choice."""
    counts = [0] * n_experts
    for e in ids.reshape(-1):
        if 0 <= e < n_experts:
            counts[e] += 1
    starts = [0]
    for c in counts:
        starts.append(starts[-1] + -(-c // align) * align)
    row_of, seen = np.full(ids.size, -1, np.int64), [0] * n_experts
    for i, e in enumerate(ids.reshape(-1)):
        if 0 <= e < n_experts:
            row_of[i] = starts[e] + seen[e]
            seen[e] += 1
    return row_of.reshape(ids.shape), np.array(starts), np.array(counts)


def written(starts, counts, rows):
    """(rows that hold a token, rows that hold zeros), as masks over the matrix's rows."""
    token, zero = np.zeros(rows, bool), np.zeros(rows, bool)
    for e, c in enumerate(counts):
        token[starts[e]:min(starts[e] + c, rows)] = True
        zero[starts[e] + c:min(starts[e + 1], rows)] = True
    return token, zero


def dispatch(x, row_of, rows):
    """x's rows at their places among rows of zeros."""
    y = np.zeros((rows, x.shape[1]))
    for t in range(row_of.shape[0]):
        for r in row_of[t]:
            if 0 <= r < rows:
                y[r] = x[t]
    return y


def dispatch_backward(dy, row_of):
    return combine(dy, row_of, None)


def combine(y, row_of, weights, residual=None):
    out = np.zeros((row_of.shape[0], y.shape[1])) if residual is None else residual.copy()
    for t in range(row_of.shape[0]):
        for j, r in enumerate(row_of[t]):
            if 0 <= r < y.shape[0]:
                out[t] += y[r] * (1.0 if weights is None else weights[t, j])
    return out


def combine_backward(dout, y, row_of, weights):
    """(dy, dweights)."""
    dy, dw = np.zeros_like(y), np.zeros(row_of.shape)
    for t in range(row_of.shape[0]):
        for j, r in enumerate(row_of[t]):
            if 0 <= r < y.shape[0]:
                dy[r] = dout[t] * (1.0 if weights is None else weights[t, j])
                dw[t, j] = dout[t] @ y[r]
    return dy, dw


def product(a, b, starts):
    """Rows of expert e of a times the transpose of expert e's rows of b; zeros in the other rows."""
    n_experts = len(starts) - 1
    n = b.shape[0] // n_experts
    out = np.zeros((a.shape[0], n))
    for e in range(n_experts):
        out[starts[e]:starts[e + 1]] = a[starts[e]:starts[e + 1]] @ b[e * n:(e + 1) * n].T
    return out


def product_grad(a, b, starts):
    """Per expert the product over its columns of a and b, one after another."""
    return np.concatenate([a[:, lo:hi] @ b[:, lo:hi].T for lo, hi in zip(starts, starts[1:])])

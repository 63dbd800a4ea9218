"""Pins of the oracle's draft-tree and eviction functions: closed forms, explicit
loops and torch in float64."""
import math

import numpy as np
import pytest
import torch

import oracle


def bits(x):
    return x.bfloat16().view(torch.int16).numpy().view(np.uint16)


def values(x):
    return x.bfloat16().double()


def problem(n, G, L, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, G, 128, generator=g), torch.randn(L, 128, generator=g), torch.randn(L, 128, generator=g)


@pytest.mark.parametrize("n,L", [(1, 1), (1, 40), (5, 5), (5, 33)])
def test_chain_is_causal_softmax(n, L):
    q, K, V = problem(n, 2, L, n * 100 + L)
    z = oracle.tree_scores(bits(q), bits(K), oracle.tree_chain(n), 0.1)
    O, lse = oracle.softmax_rows(z, bits(V))
    s = torch.einsum("tgd,ld->tgl", values(q), values(K)) * 0.1
    hidden = torch.arange(L)[None] > torch.arange(n)[:, None] + L - n
    s = s.masked_fill(hidden[:, None], -math.inf)
    np.testing.assert_allclose(O, (torch.softmax(s, -1) @ values(V)).numpy(), atol=1e-13)
    np.testing.assert_allclose(lse, torch.logsumexp(s, -1).numpy(), atol=1e-13)


def test_tree_by_explicit_loops():
    # a root with two children, the second with one child: depths 0, 1, 1, 2
    q, K, V = problem(4, 1, 9, 3)
    words = [0b0001, 0b0011, 0b0101, 0b1101]
    slopes, cap, window = [0.25], 2.0, (1, 4)
    z = oracle.tree_scores(bits(q), bits(K), words, 0.2, cap, slopes, window)
    seen, depth, ctx = [[0], [0, 1], [0, 2], [0, 2, 3]], [0, 1, 1, 2], 5
    for t in range(4):
        for i in range(9):
            pos = i if i < ctx else ctx + depth[i - ctx]
            ok = i < ctx or i - ctx in seen[t]
            ok = ok and (pos < 1 or pos > ctx + depth[t] - 4)
            want = -math.inf
            if ok:
                s = float(values(q)[t, 0] @ values(K)[i]) * 0.2
                want = cap * math.tanh(s / cap) + 0.25 * (pos - (ctx + depth[t]))
            assert z[t, 0, i] == want or abs(z[t, 0, i] - want) < 1e-12


def test_empty_rows_and_unattended_values():
    q, K, V = problem(2, 1, 2, 4)
    z = oracle.tree_scores(bits(q), bits(K), [0, 0b10], 1.0)
    V[0] = float("nan")  # token 0 is seen by no row
    O, lse = oracle.softmax_rows(z, bits(V))
    assert lse[0, 0] == -np.inf and np.all(O[0] == 0)
    np.testing.assert_allclose(O[1, 0], values(V)[1].numpy())


def test_mass_of_a_row_sums_to_its_weight():
    q, K, V = problem(3, 2, 20, 5)
    z = oracle.tree_scores(bits(q), bits(K), oracle.tree_chain(3), 0.1)
    _, lse = oracle.softmax_rows(z, bits(V))
    m = oracle.key_mass(z, lse, [1.0, 0.0, 0.5])
    assert abs(m.sum() - 2 * 1.5) < 1e-12
    assert m[18] > 0 and abs(m[19] - 0.5 * np.exp(z[2, :, 19] - lse[2]).sum()) < 1e-15


def test_evict_keep_examples():
    nan = float("nan")
    m = np.array([5.0, 1.0, 2.0, 2.0, -0.0, 0.0, nan, 9.0])
    assert list(oracle.evict_keep(m, 3, 0, 0)) == [0, 2, 7]           # 9, 5, the first 2
    assert list(oracle.evict_keep(m, 4, 1, 1)) == [0, 2, 3, 7]
    assert list(oracle.evict_keep(m, 6, 0, 0)) == [0, 1, 2, 3, 4, 7]  # -0 ties with +0: the lower index
    assert list(oracle.evict_keep(m, 7, 0, 0)) == [0, 1, 2, 3, 4, 5, 7]
    assert list(oracle.evict_keep(m, 8, 0, 0)) == list(range(8))
    assert list(oracle.evict_keep(m[:2], 5, 2, 3)) == [0, 1]
    assert list(oracle.evict_keep(m, 4, 2, 2)) == [0, 1, 6, 7]

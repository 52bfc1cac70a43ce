"""Pins of the oracle's log probabilities: closed forms and special cases, not its own formula."""

import math

import numpy as np
import pytest
from scipy.special import logsumexp
from scipy.stats import entropy as shannon

import oracle


@pytest.mark.parametrize("V,scale", [(1, 1.0), (2, 0.5), (7, 1.0), (300, 2.0), (4096, 0.7)])
def test_row_against_scipy(V, scale):
    x = np.random.default_rng(V).normal(size=V) * 3
    lse, h, logp = oracle.row_logprobs(x, scale)
    assert lse == pytest.approx(logsumexp(scale * x), abs=1e-12)
    p = np.exp(scale * x - logsumexp(scale * x))
    assert h == pytest.approx(shannon(p), abs=1e-11)
    assert np.exp(logp).sum() == pytest.approx(1.0, abs=1e-12)


def test_uniform_and_certain_rows():
    lse, h, logp = oracle.row_logprobs(np.full(64, -3.0e38), 1.0)   # the lowest values are logits
    assert h == pytest.approx(math.log(64), abs=1e-9)
    x = np.full(100, -math.inf)
    x[37] = 2.0
    lse, h, logp = oracle.row_logprobs(x, 1.0)
    assert (lse, h, logp[37]) == (2.0, 0.0, 0.0) and logp[36] == -math.inf
    lse, h, logp = oracle.row_logprobs(np.full(5, -math.inf), 1.0)
    assert lse == -math.inf and h == 0.0 and np.all(logp == -math.inf)


def test_order_breaks_ties_by_id_and_lists_no_masked_token():
    x = np.array([1.0, -math.inf, 3.0, 1.0, 3.0, -0.0, 0.0])
    assert oracle.row_order(x).tolist() == [2, 4, 0, 3, 5, 6]
    assert oracle.row_order(np.array([1.0, math.nan])).size == 0


def test_batch_places_tokens_on_their_nodes():
    rng = np.random.default_rng(3)
    x = rng.normal(size=(2, 3, 11))
    tokens = np.array([[4, 5, 6, 7], [0, -1, 10, 3]])
    nodes = np.array([[-1, 0, 2, 2], [1, 1, 0, -5]])
    r = oracle.token_logprobs(x, tokens, nodes, 1.0, 4)
    for b in range(2):
        for i in range(4):
            want = 0.0 if nodes[b, i] < 0 or tokens[b, i] < 0 else \
                x[b, nodes[b, i], tokens[b, i]] - logsumexp(x[b, nodes[b, i]])
            assert r["logprobs"][b, i] == pytest.approx(want, abs=1e-12)
    assert np.array_equal(r["target"], x.argmax(2))
    assert np.array_equal(r["top_ids"], np.argsort(-x, axis=2)[..., :4])
    short = oracle.token_logprobs(x[:, :, :2], n_top=3)
    assert np.all(short["top_ids"][..., 2] == -1) and np.all(short["top_logprobs"][..., 2] == -math.inf)

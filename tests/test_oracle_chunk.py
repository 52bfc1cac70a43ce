"""Pins of the oracle's chunk and beam rules: against complex rotation, token-by-token decoding as chain
trees, compression from scratch, and brute force over all continuations."""

import itertools
import math

import numpy as np
import pytest

import oracle
from oracle import beam, chunk


@pytest.mark.parametrize("pairs", [0, 1])
def test_rotation_is_a_complex_product_and_keeps_relative_angles(pairs):
    rng = np.random.default_rng(1)
    d, r = 10, 6
    f = (10.0 ** -np.arange(3)).astype(np.float32)
    rows = rng.standard_normal((4, d))
    pos = [0, 1, 77, 100003]
    got = chunk.rotate(rows, pos, r, pairs, f)
    tail = rows[:, 4:]
    z = tail[:, 0::2] + 1j * tail[:, 1::2] if pairs else tail[:, :3] + 1j * tail[:, 3:]
    z = z * np.exp(1j * np.outer(pos, f.astype(np.float64)))
    want = rows.copy()
    if pairs:
        want[:, 4::2], want[:, 5::2] = z.real, z.imag
    else:
        want[:, 4:7], want[:, 7:] = z.real, z.imag
    np.testing.assert_allclose(got, want, atol=1e-9)
    assert np.array_equal(got[0], rows[0])
    # the product of two rotated rows depends on the difference of their positions
    a, b = rng.standard_normal(d), rng.standard_normal(d)
    dot = lambda p, q: float(chunk.rotate(a[None], [p], r, pairs, f)[0]
                             @ chunk.rotate(b[None], [q], r, pairs, f)[0])
    assert abs(dot(5, 3) - dot(1005, 1003)) < 1e-9 and abs(dot(5, 3) - dot(5, 4)) > 1e-3


def _cache(rng, cap, d, ms):
    return (rng.standard_normal((cap, d)), rng.standard_normal((cap, d)),
            {m: (np.zeros((cap // m, d)), np.zeros((cap // m, d))) for m in ms})


@pytest.mark.parametrize("ms", [(4,), (128,), (4, 128)])
def test_appending_in_parts_is_compressing_from_scratch(ms):
    rng = np.random.default_rng(2)
    d, n = 8, 300
    g = {m: rng.standard_normal(d) for m in ms}
    K, V = rng.standard_normal((n, d)), rng.standard_normal((n, d))
    rawK, rawV, comp = _cache(rng, 300, d, ms)
    L = 0
    for part in (1, 2, 0, 125, 1, 100, 71):
        L = chunk.append_request(rawK, rawV, comp, L, K[L:L + part], V[L:L + part], g, "f64")
    assert L == n and np.array_equal(rawK, K) and np.array_equal(rawV, V)
    for m in ms:
        ck, cv = oracle.compress_prefix(K, V, n, m, g[m], "f64")
        assert np.array_equal(comp[m][0], ck) and np.array_equal(comp[m][1], cv)


@pytest.mark.parametrize("W,tail,ms", [(128, "window", (4, 128)), (5, "window", (4,)),
                                       (0, "remainder", (4, 128)), (0, "window", (128,))])
def test_a_chunk_is_a_chain_of_tree_nodes(W, tail, ms):
    # the same tokens as a chain tree behind the prefix give the same outputs
    rng = np.random.default_rng(3)
    d, H, L, n = 8, 3, 250, 9
    g = {m: rng.standard_normal(d) for m in ms}
    rawK, rawV, comp = _cache(rng, 300, d, ms)
    for m in ms:
        ck, cv = oracle.compress_prefix(rawK, rawV, L, m, g[m], "f64")
        comp[m][0][:L // m], comp[m][1][:L // m] = ck, cv
    K, V, Q = (rng.standard_normal((n, d)), rng.standard_normal((n, d)),
               rng.standard_normal((n, H, d)))
    cfg = oracle.VerifyConfig(H=H, d=d, ms=ms, W=W, tail_mode=tail, store="f64")
    O, lse, _, _ = oracle.tree_verify_attn_request(cfg, list(range(-1, n - 1)), L, Q, comp, None, rawK,
                                                   rawV, K, V, g)
    end = chunk.append_request(rawK, rawV, comp, L, K, V, g, "f64")
    got, got_lse, _, _ = chunk.attend_request(Q, end, rawK, rawV, comp, W, tail, 1 / math.sqrt(d))
    np.testing.assert_allclose(got, O, atol=1e-12)
    np.testing.assert_allclose(got_lse, lse, atol=1e-12)


@pytest.mark.parametrize("seed", range(6))
def test_selection_is_the_best_of_all_continuations(seed):
    rng = np.random.default_rng(seed)
    width, V, eos, scale = 3, 5, 2, 0.75
    x = np.round(rng.standard_normal((width, V)) * 2)      # with ties
    x[rng.random((width, V)) < 0.2] = -math.inf
    scores = list(np.round(rng.standard_normal(width)))
    done = [0, int(rng.random() < 0.5), 0]
    code, rows = beam.select_group(x, scores, done, eos, scale)
    every = []
    for w, t in itertools.product(range(width), range(V)):
        if done[w]:
            if t == 0:
                every.append((scores[w], -w, -eos))
        elif x[w, t] > -math.inf:
            z = np.log(np.sum(np.exp(scale * x[w])))
            every.append((round(scores[w] + scale * x[w, t] - z, 9), -w, -t))
    best = sorted(every, reverse=True)[:width]
    by_rank = sorted((r[4], r) for r in rows if r[0] >= 0)
    assert code == 0 and len(by_rank) == len(best)
    for (k, r), (s, w, t) in zip(by_rank, best):
        assert (r[0], r[1]) == (-w, -t) and abs(r[2] - s) < 1e-8
        assert r[3] == int(done[-w] or -t == eos)
    # a beam that goes on keeps its best continuation in its own slot: tv_pages_fork can reorder
    for slot, r in enumerate(rows):
        if r[0] >= 0:
            assert rows[r[0]][0] == r[0]
            assert rows[r[0]][4] <= r[4]


def test_running_out_of_candidates_and_bad_values():
    x = np.full((3, 4), -math.inf)
    x[1, 3] = 0.5
    code, rows = beam.select_group(x, [0.0, -1.0, -math.inf], [0, 0, 0], 0, 1.0)
    assert code == 0 and rows == [(-1, -1, -math.inf, 0, -1), (1, 3, -1.0, 0, 0), (-1, -1, -math.inf, 0, -1)]
    x[0, 0] = math.nan
    assert beam.select_group(x, [0.0, -1.0, -math.inf], [0, 0, 0], 0, 1.0)[0] == -11
    assert beam.select_group(x, [0.0, -1.0, -math.inf], [1, 0, 0], 0, 1.0)[0] == 0
    assert beam.select_group(x, [-math.inf, -1.0, math.inf], [0, 0, 0], 0, 1.0)[0] == -11

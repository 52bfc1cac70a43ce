"""Pins of the oracle's page rules: hand-worked states and invariants over random histories."""

import numpy as np
import pytest

from oracle import pages


def _state(table, refs, L, P=4, d=2, seed=0):
    rng = np.random.default_rng(seed)
    pools = {1: tuple(rng.normal(size=(len(refs), P, d)) for _ in range(2))}
    return dict(table=[list(r) for r in table], refs=list(refs), L=list(L), pools=pools)


def test_fork_worked_example():
    # slot 0: 6 tokens in pages 3, 1; slot 1 becomes a copy, slot 2 is released
    s = _state([[3, 1, -1], [0, -1, -1], [4, -1, -1]], [1, 1, 0, 1, 1], [6, 2, 3])
    K = s["pools"][1][0].copy()
    assert pages.fork(s, 4, [0, 0, -1]) == 0
    assert s["table"] == [[3, 1, -1], [3, 0, -1], [-1, -1, -1]]   # page 0 freed and taken again
    assert s["refs"] == [1, 1, 0, 2, 0] and s["L"] == [6, 6, 0]
    assert np.array_equal(s["pools"][1][0][0, :2], K[1, :2])
    assert np.array_equal(s["pools"][1][0][0, 2:], K[0, 2:])      # rows past the valid ones stay


def test_truncation_into_a_shared_page_copies_it():
    s = _state([[0, 1], [0, 2]], [2, 1, 1, 0, 0], [6, 7])
    assert pages.fork(s, 4, [0, 1], [3, -1]) == 0
    # page 1, released behind the new length, is the lowest free one and takes the copy
    assert s["table"] == [[1, -1], [0, 2]] and s["refs"] == [1, 1, 1, 0, 0] and s["L"] == [3, 7]
    s = _state([[0, 1], [5, 2]], [1, 1, 1, 0, 0, 1], [6, 7])       # not shared: kept in place
    assert pages.fork(s, 4, [0, 1], [3, -1]) == 0
    assert s["table"] == [[0, -1], [5, 2]] and s["refs"] == [1, 0, 1, 0, 0, 1]


def test_failures_leave_the_state():
    s = _state([[0, 1], [2, -1]], [1, 1, 1], [6, 1])
    before = (list(map(list, s["table"])), list(s["refs"]), list(s["L"]))
    assert pages.fork(s, 4, [1, 0]) == pages.ERR_ARG          # neither source stays
    assert (s["table"], s["refs"], s["L"]) == before
    s = _state([[0, 1], [0, -1]], [2, 1], [6, 3])
    before = (list(map(list, s["table"])), list(s["refs"]), list(s["L"]))
    assert pages.fork(s, 4, [0, 0]) == pages.ERR_CAPACITY     # one page too few
    assert (s["table"], s["refs"], s["L"]) == before
    assert pages.reserve(s, 4, [0, 2]) == pages.ERR_CAPACITY
    assert pages.reserve(s, 4, [3, 0]) == pages.ERR_CAPACITY  # past the capacity
    assert (s["table"], s["refs"], s["L"]) == before


def test_reserve_and_compact_worked_example():
    s = _state([[5, -1, -1], [2, 4, -1]], [0, 0, 1, 1, 1, 1, 0], [4, 5])   # page 3: held outside
    assert pages.reserve(s, 4, [1, 4]) == 0
    assert s["table"] == [[5, 0, -1], [2, 4, 1]] and s["refs"] == [1, 1, 1, 1, 1, 1, 0]
    s = _state([[5, -1, -1], [2, 6, -1]], [0, 0, 1, 1, 0, 1, 1], [4, 5])
    K = s["pools"][1][0].copy()
    code, remap, n = pages.compact(s, 4)
    assert (code, n, remap) == (0, 4, [-1, -1, 2, 3, -1, 0, 1])
    assert s["table"] == [[0, -1, -1], [2, 1, -1]] and s["refs"] == [1, 1, 1, 1, 0, 0, 0]
    assert np.array_equal(s["pools"][1][0][0], K[5]) and np.array_equal(s["pools"][1][0][1, :1], K[6, :1])
    assert np.array_equal(s["pools"][1][0][1, 1:], K[1, 1:])


@pytest.mark.parametrize("seed", range(5))
def test_random_histories_keep_every_request_s_tokens(seed):
    # the token sequence seen through the table never changes but by commits, forks, truncations
    rng = np.random.default_rng(seed)
    B, G, P, n = 5, 6, 4, 24
    s = _state([[-1] * G for _ in range(B)], [0] * n, [0] * B)
    seq = [[] for _ in range(B)]
    K = s["pools"][1][0]
    for _ in range(60):
        op = rng.integers(3)
        if op == 0:      # a round: reserve, append
            if pages.reserve(s, P, [3] * B) == 0:
                for b in range(B):
                    for _ in range(int(rng.integers(1, 4))):
                        x = rng.normal(size=2)
                        K[s["table"][b][s["L"][b] // P], s["L"][b] % P] = x
                        seq[b].append(x)
                        s["L"][b] += 1
        elif op == 1:
            src = [int(x) for x in rng.integers(-1, B, size=B)]
            src = [b if src[b] == b or rng.random() < 0.5 else src[b] for b in range(B)]
            keep = [int(x) for x in rng.integers(-1, 18, size=B)]
            want = []
            for b in range(B):
                if src[b] == -1:
                    want.append([])
                elif src[src[b]] != src[b]:
                    want.append(list(seq[b]))
                else:
                    ks = [k for k in (keep[src[b]], keep[b]) if k >= 0]
                    want.append(seq[src[b]][:min([len(seq[src[b]])] + ks)])
            if pages.fork(s, P, src, keep) != pages.ERR_CAPACITY:
                seq = want
        else:
            pages.compact(s, P)
        held = [0] * n
        for b in range(B):
            assert s["L"][b] == len(seq[b])
            for i, x in enumerate(seq[b]):
                assert np.array_equal(K[s["table"][b][i // P], i % P], x)
            for p in s["table"][b]:
                if p >= 0:
                    held[p] += 1
        assert held == s["refs"]

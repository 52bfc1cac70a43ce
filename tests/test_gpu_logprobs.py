"""tv_token_logprobs on the GPU against the fp64 oracle.  Ids and targets are exact (they are decided
on the stored logits); the fp32 values are held to the rounding of their formulas.

Tolerances.  u = 2^-24.  A term e^{y}, y = scale (x - m), is formed as 2^{fl((x - m) c)} or, the same
to within one rounding, 2^{fl(x c - b)} with b = fl(m c) taken out again at the end; c = fl(scale
log2 e): the difference, the product and c each round by u relative to y, log2 e once more, so e^{y}
is off by a factor within 4 u |y| + 2^-22 (two ulp of the exponential); weighted by the terms, the sum S is off by 4 u E|y| + 2^-22, E|y| = ln S - entropy <= ln V, plus its additions: one thread adds at most
V / 256 + 8 terms in a row, the joins at most 16 more sums with a factor each (u for the sum,
2^-22 + 4 u for the factor's exponential).  ln S adds two ulp of itself.  So
  dS   = 4 u lnV + 2^-22 + (V / 256 + 24) u + 16 (2^-22 + 4 u) ... relative error of S and T
  logp = dS + 2 u |ln S| + 3 u |y|,  lse = dS + 2 u |ln S| + 2 u |scale m| + u |lse|
  entropy = ln S - T / S: dS + 2 u lnV for ln S, and 2 dS E|y| + 8 u E|y| for the quotient.
"""

import math

import numpy as np
import pytest
import torch

import oracle
from tree_speculative_verify_gb300 import _lib, engine, workloads

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _dS(V):
    return 4 * U * math.log(max(V, 2)) + 2 ** -22 + (V / 256 + 24) * U + 16 * (2 ** -22 + 4 * U)


def _shape(B, D):
    return _lib.make_shape(B=B, D=D, H=1, d=8, comp_mask=_lib.TV_COMP_C4)


def _run(x, tokens=None, nodes=None, scale=1.0, n_top=0, stream=None):
    """x: CUDA logits [B][D][V]; fills every output with garbage first."""
    B, D = x.shape[:2]
    f = lambda *s: torch.full(s, 7e7, dtype=torch.float32, device="cuda")
    i = lambda *s: torch.full(s, -77, dtype=torch.int32, device="cuda")
    n = 0 if tokens is None else tokens.shape[1]
    t = lambda a: None if a is None else torch.as_tensor(a, dtype=torch.int32).cuda()
    out = dict(lse=f(B, D), entropy=f(B, D), logprobs=f(B, n) if n else None,
               top_ids=i(B, D, n_top) if n_top else None,
               top_logprobs=f(B, D, n_top) if n_top else None, target=i(B, D))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tk, nd = t(tokens), t(nodes)
    torch.cuda.synchronize()
    _lib.tv_token_logprobs(_shape(B, D), x, tk, nd, scale, out["lse"], out["entropy"],
                           out["logprobs"], out["top_ids"], out["top_logprobs"], out["target"],
                           status, stream)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in out.items() if v is not None}, int(status.item())


def _close(got, want, tol, what):
    got = got.astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), what
    fine = np.isfinite(want)
    assert np.all(np.isfinite(got[fine])), what
    err = np.abs(got[fine] - want[fine])
    tol = np.broadcast_to(tol, want.shape)[fine]
    bad = err > tol
    assert not bad.any(), f"{what}: error {err[bad][:4]} over {tol[bad][:4]}"


def _check(x, got, tokens=None, nodes=None, scale=1.0, n_top=0):
    xs = x.detach().float().cpu().numpy()
    scale = float(np.float32(scale))
    want = oracle.token_logprobs(xs, tokens, nodes, scale, n_top)
    V = xs.shape[2]
    dS, lnV = _dS(V), math.log(max(V, 2))
    assert np.array_equal(got["target"], want["target"])
    top = np.where(np.isfinite(xs), np.abs(xs), 0).max(axis=2) if V else 0
    _close(got["lse"], want["lse"], dS + 2 * U * lnV + 2 * U * scale * top
           + U * np.where(np.isfinite(want["lse"]), np.abs(want["lse"]), 0), "lse")
    _close(got["entropy"], want["entropy"], dS + 2 * U * lnV + (2 * dS + 8 * U) * lnV, "entropy")
    lp_tol = lambda w: dS + 2 * U * lnV + 3 * U * (np.where(np.isfinite(w), np.abs(w), 0) + lnV)
    if n_top:
        assert np.array_equal(got["top_ids"], want["top_ids"])
        _close(got["top_logprobs"], want["top_logprobs"], lp_tol(want["top_logprobs"]), "top_logprobs")
    if tokens is not None:
        _close(got["logprobs"], want["logprobs"], lp_tol(want["logprobs"]), "logprobs")
    return want


def _logits(B, D, V, dtype, seed, pad=0, sigma=3.0):
    g = torch.Generator().manual_seed(seed)
    store = (torch.randn((B, D, V + pad), generator=g) * sigma).to(dtype).cuda()
    return store[:, :, :V]


BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("B,D,V,pad,dtype,K,n_tok,scale", [
    (1, 1, 1, 0, BF, 1, 1, 1.0), (1, 1, 1, 0, F32, 4, 0, 1.0), (2, 3, 2, 5, BF, 3, 4, 2.0),
    (1, 2, 7, 0, BF, 7, 3, 1.0), (3, 1, 8, 0, BF, 2, 1, 0.25), (1, 64, 9, 0, F32, 1, 64, 1.0),
    (2, 5, 31, 1, BF, 32, 9, 1.0), (1, 3, 33, 0, F32, 32, 2, 3.0), (2, 2, 257, 3, BF, 5, 7, 1.0),
    (4, 2, 1000, 0, F32, 0, 0, 1.0), (2, 8, 2047, 1, BF, 8, 8, 0.8), (2, 8, 2048, 0, BF, 8, 8, 1.0),
    (2, 8, 2049, 7, F32, 8, 8, 1.0), (3, 5, 4097, 2, BF, 20, 100, 1.0), (1, 1, 8191, 0, F32, 31, 3, 1.0),
    (1, 7, 16383, 0, BF, 32, 7, 1.3), (8, 8, 32000, 0, BF, 8, 8, 1.0), (2, 3, 50001, 2, BF, 5, 7, 1.25),
    (40, 8, 1024, 0, BF, 4, 8, 1.0), (1, 1, 131075, 0, BF, 32, 1, 1.0), (1, 2, 262144, 0, F32, 10, 1024, 0.6),
    (200, 1, 3001, 0, BF, 2, 1, 1.0), (1300, 1, 1501, 1, F32, 8, 1, 1.0),
    (160, 8, 2600, 3, BF, 32, 8, 1.1), (1217, 1, 70, 0, F32, 5, 1, 1.0), (620, 1, 9001, 0, F32, 20, 1, 1.0), (1, 6, 200000, 0, F32, 32, 6, 1.0),
])
def test_rows_match_oracle(B, D, V, pad, dtype, K, n_tok, scale):
    x = _logits(B, D, V, dtype, seed=V + B, pad=pad)
    rng = np.random.default_rng(V)
    tokens = nodes = None
    if n_tok:
        tokens = rng.integers(-1, V, size=(B, n_tok)).astype(np.int32)
        nodes = rng.integers(-1, D, size=(B, n_tok)).astype(np.int32)
    got, status = _run(x, tokens, nodes, scale, K)
    assert status == 0
    _check(x, got, tokens, nodes, scale, K)


def test_null_nodes_put_entry_i_on_node_i():
    x = _logits(3, 6, 700, F32, 1)
    tokens = np.random.default_rng(2).integers(0, 700, size=(3, 4)).astype(np.int32)
    got, status = _run(x, tokens, None, 1.0, 2)
    assert status == 0
    _check(x, got, tokens, None, 1.0, 2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [40, 5000, 33000])
def test_masked_rows(V, dtype):
    # rows of -inf only, one token left, every 97th left, the type's lowest value as the mask, all
    # logits at the lowest value, a lone token at the row's very end or start
    x = _logits(1, 8, V, dtype, 5).contiguous()
    low = torch.finfo(dtype).min
    keep = torch.arange(V, device="cuda") % 97 == 0
    x[0, 0] = -math.inf
    x[0, 1] = -math.inf
    x[0, 1, V // 2] = 1.5
    x[0, 2].masked_fill_(~keep, -math.inf)
    x[0, 3].masked_fill_(~keep, low)
    x[0, 4] = low
    x[0, 5] = -math.inf
    x[0, 5, V - 1] = -2.0
    x[0, 6] = -math.inf
    x[0, 6, 0] = low
    tokens = np.array([[0, V // 2, V // 2 + 1, 1, 97 % V, 3, V - 1, 0, 1]], dtype=np.int32)
    nodes = np.array([[0, 1, 1, 2, 3, 4, 5, 6, 6]], dtype=np.int32)
    got, status = _run(x, tokens, nodes, 1.0, 12)
    assert status == 0
    want = _check(x, got, tokens, nodes, 1.0, 12)
    assert got["target"][0, 0] == -1 and got["entropy"][0, 0] == 0 and got["lse"][0, 0] == -math.inf
    assert (want["top_ids"][0, 1] >= 0).sum() == 1


@pytest.mark.parametrize("dtype,copies,V", [(BF, 1, 20011), (F32, 1, 20011), (BF, 60, 20011),
                                            (BF, 140, 9011), (F32, 140, 5011)])
def test_ties_and_orders_that_defeat_a_threshold(dtype, copies, V):
    # (many copies of the rows: the thread counts that many rows take)
    x = torch.zeros((1, 9, V), dtype=dtype, device="cuda")
    ramp = torch.arange(V, device="cuda").float()
    x[0, 0] = 0.0                                        # all equal
    x[0, 1, ::2] = -0.0                                  # -0 and +0 are equal
    x[0, 2] = (ramp / 64).to(dtype)                      # ascending (bf16: long runs of ties)
    x[0, 3] = (-ramp / 64).to(dtype)                     # descending
    x[0, 4] = (ramp % 7).to(dtype)                       # thousands of ties at the top
    x[0, 5] = -math.inf
    x[0, 5, -40:] = 1.0                                  # the candidates at the end, tied
    x[0, 6] = -5.0
    x[0, 6, 100:4000] = 2.0                              # a run of ties within one stretch
    x[0, 7] = torch.randint(0, 3, (V,), generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    x[0, 8] = torch.finfo(dtype).min
    many = x.expand(copies, 9, V).contiguous()
    for K in (0, 1, 5, 32):
        got, status = _run(many, n_top=K)
        assert status == 0
        # copies start at other alignments: the same ids, and sums within the same tolerances
        for b in sorted({0, copies // 2, copies - 1}):
            _check(x, {k: v[b:b + 1] for k, v in got.items()}, n_top=K)
        for k in ("target", "top_ids"):
            if k in got:
                assert np.array_equal(got[k], np.broadcast_to(got[k][:1], got[k].shape))


def test_nan_and_inf_rows_are_reported_and_the_others_are_right():
    x = _logits(1, 6, 3000, F32, 9).contiguous()
    x[0, 1, 2999] = math.nan
    x[0, 3, 0] = math.inf
    x[0, 4] = math.nan
    x[0, 5] = -math.inf
    x[0, 5, 17] = math.nan
    tokens = np.array([[5, 5, 5, 5, 5, 5]], dtype=np.int32)
    got, status = _run(x, tokens, None, 1.0, 3)
    assert status == -11
    _check(x, got, tokens, None, 1.0, 3)
    for v in (1, 3, 4, 5):
        assert np.all(got["top_ids"][0, v] == -1) and math.isnan(got["lse"][0, v])
    clean = x[:, [0, 2]].contiguous()
    a, status = _run(clean, tokens[:, [0, 2]], None, 1.0, 3)
    assert status == 0
    for k in ("lse", "entropy", "target", "top_ids", "top_logprobs"):
        assert np.array_equal(a[k][0], got[k][0][[0, 2]]), k


def test_tokens_and_nodes_out_of_range_are_reported():
    x = _logits(2, 3, 500, BF, 4)
    tokens = np.array([[1, 500, 3], [1, 2, 3]], dtype=np.int32)
    nodes = np.array([[0, 1, 2], [0, 3, 2]], dtype=np.int32)
    got, status = _run(x, tokens, nodes, 1.0, 1)
    assert status == -1
    assert got["logprobs"][0, 1] == 0 and got["logprobs"][1, 1] == 0
    ok_t, ok_n = tokens.copy(), nodes.copy()
    ok_t[0, 1] = ok_n[1, 1] = -1
    _check(x, got, ok_t, ok_n, 1.0, 1)


def test_peaked_rows_keep_small_probabilities():
    x = _logits(1, 4, 9000, F32, 6).contiguous()
    x[0, 0, 5] = 60.0
    x[0, 1, 8999] = 1e4
    x[0, 2, 0] = 1e30
    x[0, 3] *= 1e-6
    tokens = np.array([[5, 6, 8999, 1, 0, 1, 7]], dtype=np.int32)
    nodes = np.array([[0, 0, 1, 1, 2, 2, 3]], dtype=np.int32)
    got, status = _run(x, tokens, nodes, 1.0, 3)
    assert status == 0
    _check(x, got, tokens, nodes, 1.0, 3)


@pytest.mark.parametrize("dtype,T", [(BF, 128), (F32, 256), (BF, 256)])
def test_largest_logits_in_one_thread_s_reach(dtype, T):
    # the pass gives thread i of T the vectors i, i + T, ...: all large logits in one of those columns,
    # and more of them than the candidate list holds, so that neither the bound nor the second scan
    # can keep the list short
    kvec = 8 if dtype == BF else 4
    V, rows = 80000, 1 if T == 256 else 600
    x = torch.full((rows, 1, V), -3.0, dtype=dtype, device="cuda")
    i = torch.arange(V, device="cuda")
    col = (i // kvec) % T == 5
    vals = torch.linspace(1.0, 200.0, int(col.sum()), device="cuda").to(dtype)
    x[0, 0, col] = vals[torch.randperm(len(vals), generator=torch.Generator().manual_seed(2)).cuda()]
    x[-1, 0, col] = vals
    got, status = _run(x, n_top=32)
    assert status == 0
    pick = [0, rows - 1]
    want = oracle.token_logprobs(x[pick].float().cpu().numpy(), n_top=32)
    assert np.array_equal(got["top_ids"][pick], want["top_ids"])
    assert np.array_equal(got["target"][pick], want["target"])


@pytest.mark.parametrize("scale", [1e-6, 0.01, 30.0, 1e6])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_extreme_temperatures(scale, dtype):
    # flat and one-token distributions, the exponents' far form (largest logit times scale beyond
    # thousands) and logits that straddle it
    x = _logits(1, 3, 5003, dtype, 21).contiguous()
    x[0, 1] += 300.0
    x[0, 2] -= 5000.0
    tokens = np.array([[0, 1, 2, 3, 4, 5]], dtype=np.int32)
    nodes = np.array([[0, 0, 1, 1, 2, 2]], dtype=np.int32)
    got, status = _run(x, tokens, nodes, scale, 6)
    assert status == 0
    _check(x, got, tokens, nodes, scale, 6)


def test_rows_beyond_32_bit_offsets():
    # rows 2^26 + 3 elements apart: the later ones start past 2^31 elements and 2^32 bytes
    D, V, ld = 64, 1003, (1 << 26) + 3
    store = torch.empty(D * ld, dtype=BF, device="cuda")
    x = store.as_strided((1, D, V), (D * ld, ld, 1))
    x.copy_(_logits(1, D, V, BF, 8))
    got, status = _run(x, n_top=4)
    assert status == 0
    _check(x, got, n_top=4)


def test_another_stream_and_a_captured_replay():
    x = _logits(2, 4, 6000, BF, 10).contiguous()
    want, _ = _run(x, n_top=5)
    got, status = _run(x, n_top=5, stream=torch.cuda.Stream())
    assert status == 0
    for k in want:
        assert np.array_equal(got[k], want[k]), k
    B, D, K = 2, 4, 5
    f = lambda *s: torch.zeros(s, dtype=torch.float32, device="cuda")
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    o = [f(B, D), f(B, D), i(B, D, K), f(B, D, K), i(B, D), i(1)]
    buf = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _lib.tv_token_logprobs(_shape(B, D), buf, None, None, 1.0, o[0], o[1], None, o[2], o[3], o[4], o[5])
    for seed in (10, 11):
        y = _logits(2, 4, 6000, BF, seed).contiguous()
        buf.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        want, _ = _run(y, n_top=K)
        for k, t in zip(("lse", "entropy", "top_ids", "top_logprobs", "target"), o):
            assert np.array_equal(t.cpu().numpy(), want[k]), k


def test_unwanted_outputs_and_no_rows():
    x = _logits(1, 3, 4000, BF, 12)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    target = torch.full((1, 3), -9, dtype=torch.int32, device="cuda")
    _lib.tv_token_logprobs(_shape(1, 3), x, None, None, 1.0, None, None, None, None, None, target, status)
    want, _ = _run(x)
    assert np.array_equal(target.cpu().numpy(), want["target"])
    empty = torch.zeros((0, 3, 10), dtype=BF, device="cuda")
    _lib.tv_token_logprobs(_shape(0, 3), empty, None, None, 1.0, None, None, None, None, None, None, status)


def test_binding_refuses_wrong_tensors():
    x = _logits(2, 3, 100, BF, 1)
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device="cuda")
    i32 = torch.int32
    st, sh = z(1, dt=i32), _shape(2, 3)
    call = lambda x=x, tokens=None, lse=None, ids=None, lps=None, scale=1.0, nodes=None, lp=None: \
        _lib.tv_token_logprobs(sh, x, tokens, nodes, scale, lse, None, lp, ids, lps, None, st)
    with pytest.raises(ValueError):
        call(x=x[:, :2])
    with pytest.raises(TypeError):
        call(x=x.half())
    with pytest.raises(ValueError):
        call(x=x.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError):
        call(x=x.cpu())
    with pytest.raises(ValueError):
        call(lse=z(5))
    with pytest.raises(TypeError):
        call(tokens=z(2, 3, dt=torch.int64), lp=z(2, 3))
    for kw, code in ((dict(scale=0.0), -1), (dict(scale=math.inf), -1), (dict(scale=math.nan), -1),
                     (dict(ids=z(2, 3, 33, dt=i32), lps=z(2, 3, 33)), -2),
                     (dict(tokens=z(2, 4, dt=i32), lp=z(2, 4)), -1)):
        with pytest.raises(_lib.TreeVerifyError) as e:
            call(**kw)
        assert e.value.code == code


def test_scored_round_feeds_the_acceptance_walk():
    # targets taken from logits that favour the workload's own targets: the round accepts the same
    wl = workloads.small()
    shape = engine.shape_for(wl)
    st, rb = engine.alloc_state(wl), engine.alloc_round(wl, shape)
    engine.prefill(shape, st, rb)
    st2, rb2 = st.clone(), engine.alloc_round(wl, shape)
    torch.cuda.synchronize()
    engine.verify_round(shape, st, rb)
    engine.alloc_scores(rb2, shape, workloads.VOCAB, n_top=4)
    rb2.logits.normal_(generator=torch.Generator(device="cuda").manual_seed(3))
    rb2.logits.scatter_(2, rb2.target.long().unsqueeze(2), 9.0)
    rb2.target.fill_(-5)
    L0 = st2.L.clone()
    graph = engine.RoundGraph(shape, st2, rb2, scored=True, prologue=lambda: st2.L.copy_(L0))
    rb2.target.fill_(-5)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert int(rb2.status.item()) == 0
        for k in ("target", "accept_len", "path", "bonus", "committed", "O"):
            assert torch.equal(getattr(rb, k), getattr(rb2, k)), k
        assert torch.equal(rb2.top_ids[:, :, 0], rb2.target)
        assert torch.equal(st.L, st2.L)
    want = oracle.token_logprobs(rb2.logits.float().cpu().numpy(), wl.draft, wl.parents)
    err = np.abs(rb2.draft_logprobs.cpu().numpy() - want["logprobs"]).max()
    assert err <= _dS(workloads.VOCAB) + 5 * U * (np.abs(want["logprobs"]).max() + 12)


@pytest.mark.parametrize("V", [900, 20011, 400000])
@pytest.mark.parametrize("scale,at", [(1.0, 6931.4487), (1.0, -6931.4487), (100.0, 69.31449),
                                      (100.0, -69.31449), (0.001, 6931448.7)])
def test_logits_on_both_sides_of_the_far_exponents(V, scale, at):
    # comparable weights whose scaled logits lie a few tenths of a nat to either side of where the
    # exponents take their far form (|logit * scale * log2 e| = 10^4): in one thread, in different
    # threads and in different CTAs of a row (400000 logits), the larger one first and last
    x = torch.full((1, 8, V), at - 300.0 / scale, dtype=F32, device="cuda")
    near, far = at - 0.19 / scale, at + 0.23 / scale
    gaps = (1, 4, 130, 4096 % V, V // 2, V - 9, 517, 8)
    for r, gap in enumerate(gaps):
        lo, hi = (near, far) if r % 2 else (far, near)
        first = 4 if gap + 8 < V else 0
        x[0, r, first] = lo
        x[0, r, first + gap] = hi
        x[0, r, (first + gap + 2) % V] = at + 0.01 / scale
    tokens = np.array([[4, 5, 8, 4 + gaps[2], 4 + gaps[3], 4 + gaps[4], 0, 4]], dtype=np.int32)
    nodes = np.array([[0, 0, 1, 2, 3, 4, 5, 7]], dtype=np.int32)
    got, status = _run(x, tokens, nodes, scale, 3)
    assert status == 0
    _check(x, got, tokens, nodes, scale, 3)


@pytest.mark.parametrize("B", [1, 12])
def test_acceptance_walk_takes_the_targets_of_the_call_in_front(B):
    # other logits before every round, and targets left over that no draft token equals: the walk
    # follows what the call just in front of it has written, called one by one and replayed
    wl = workloads.serving(B=B, L=(300, 900))
    shape = engine.shape_for(wl)
    st, rb = engine.alloc_state(wl), engine.alloc_round(wl, shape)
    engine.prefill(shape, st, rb)
    engine.alloc_scores(rb, shape, workloads.VOCAB, n_top=1)
    L0 = st.L.clone()
    graph = engine.RoundGraph(shape, st, rb, scored=True, prologue=lambda: st.L.copy_(L0))
    rng = np.random.default_rng(B)
    lengths = set()
    for k in range(24):
        want = rng.integers(0, workloads.VOCAB, size=(B, wl.D)).astype(np.int32)
        for b in range(B):
            for v in range(1, wl.D):       # half of the nodes lead on to one of their children
                if rng.random() < 0.5:
                    want[b, wl.parents[b, v]] = wl.draft[b, v]
        logits = torch.zeros_like(rb.logits)
        logits.scatter_(2, torch.as_tensor(want).cuda().long().unsqueeze(2), 9.0)
        rb.logits.copy_(logits)
        rb.target.fill_(-5)
        st.L.copy_(L0)
        torch.cuda.synchronize()
        graph.replay() if k % 2 else engine.verify_round(shape, st, rb, scored=True)
        torch.cuda.synchronize()
        assert int(rb.status.item()) == 0
        assert np.array_equal(rb.target.cpu().numpy(), want)
        for b in range(B):
            n, path, bonus = oracle.accept_walk(wl.parents[b], wl.draft[b], want[b])
            assert int(rb.accept_len[b]) == n and int(rb.bonus[b]) == bonus
            assert rb.path[b, :n].tolist() == list(path)[:n]
            lengths.add(n)
    assert len(lengths) > 1


@pytest.mark.parametrize("dtype,T,rows,V,ranks,columns", [
    (F32, 256, 104, 140003, 1, 1), (BF, 256, 104, 140003, 1, 1), (F32, 128, 600, 70003, 1, 1),
    (BF, 128, 600, 70003, 1, 1), (F32, 64, 1300, 8191, 1, 8), (BF, 64, 1300, 16384, 1, 8),
    (F32, 256, 1, 2200000, 16, 1), (BF, 256, 2, 2300000, 16, 1)])
def test_more_large_logits_in_few_threads_than_the_list_holds(dtype, T, rows, V, ranks, columns):
    # all large logits of a CTA's share (T threads, `ranks` CTAs per row) in the vectors of fewer threads
    # than there are alternatives, and more of them than the 512 candidates: the bound stays at the
    # others' value, the list overflows twice, and every alternative takes a scan of its own
    kvec = 8 if dtype == BF else 4
    n_vec = -(-V // kvec)
    per = -(-n_vec // ranks)
    i = torch.arange(V, device="cuda") // kvec
    col = (i % per) % T < columns
    assert int(col[: min(V, (per - T) * kvec)].sum()) > 512
    x = torch.full((rows, 1, V), -3.0, dtype=dtype, device="cuda")
    vals = torch.linspace(1.0, 200.0, int(col.sum()), device="cuda")
    order = torch.randperm(len(vals), generator=torch.Generator().manual_seed(2)).cuda()
    x[0, 0, col] = vals[order].to(dtype)
    x[-1, 0, col] = vals.to(dtype)
    tokens = np.full((rows, 1), 20, dtype=np.int32)
    pick = sorted({0, rows - 1})
    for K in (32, 2):
        got, status = _run(x, tokens, None, 1.0, K)
        assert status == 0
        _check(x[pick], {k: v[pick] for k, v in got.items()}, tokens[pick], None, 1.0, K)


def test_scored_rounds_at_a_temperature():
    wl = workloads.small()
    shape = engine.shape_for(wl)
    outs = []
    for graphed in (False, True):
        st, rb = engine.alloc_state(wl), engine.alloc_round(wl, shape)
        engine.prefill(shape, st, rb)
        engine.alloc_scores(rb, shape, workloads.VOCAB, n_top=2)
        rb.logits.normal_(generator=torch.Generator(device="cuda").manual_seed(4))
        if graphed:
            engine.RoundGraph(shape, st, rb, scored=True, inv_temperature=2.5).replay()
        else:
            engine.verify_round(shape, st, rb, scored=True, inv_temperature=2.5)
        torch.cuda.synchronize()
        assert int(rb.status.item()) == 0
        outs.append([t.cpu().numpy() for t in (rb.logits_lse, rb.entropy, rb.draft_logprobs, rb.top_logprobs)])
    for a, b in zip(*outs):
        assert np.array_equal(a, b)
    got = dict(zip(("lse", "entropy", "logprobs", "top_logprobs"), outs[0]), target=rb.target.cpu().numpy(),
               top_ids=rb.top_ids.cpu().numpy())
    _check(rb.logits, got, wl.draft, wl.parents, 2.5, 2)

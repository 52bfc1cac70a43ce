"""Calls that write the cache meet a page table with holes: what lies on the missing page is left out
and reported, nothing else is lost, and no row of another page changes."""

import numpy as np
import pytest
import torch

from tree_speculative_verify_gb300 import _lib, engine, workloads

pytestmark = pytest.mark.gpu

TV_ERR_ARG = -1


def test_prefill_of_a_long_prefix_with_a_page_missing():
    # more than 2 * 65535 C128 entries, so that a cluster computes three, the second of which lies on
    # the missing page: the entries around it come out as in the prefill of the whole prefix
    P, G, d = 1 << 20, 17, 8
    L = 128 * (2 * 65535 + 40)
    gen = torch.Generator(device="cuda").manual_seed(3)
    rawK, rawV = (torch.randn((G, P, d), generator=gen, device="cuda").bfloat16() for _ in range(2))
    g = torch.randn(d, generator=gen, device="cuda")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    missing = 8                                # entries 65536 .. 73727
    order = [(5 * k + 2) % G for k in range(G)]
    runs = []
    for hole in (False, True):
        table = list(order)
        if hole:
            table[missing] = -1
        pt, status = i32([table]), i32([0])
        shape = _lib.make_shape(B=1, D=1, H=1, d=d, comp_mask=_lib.TV_COMP_C128, raw_cap=G * P,
                                c4_cap=G * P // 4, c128_cap=G * P // 128, page_tokens=P, max_pages=G,
                                n_pool_pages=G, page_table=pt)
        c128K, c128V = (torch.full((G, P // 128, d), 7.0, dtype=torch.bfloat16, device="cuda")
                        for _ in range(2))
        _lib.tv_prefill_compress(shape, rawK, rawV, i32([L]), None, g, None, None, c128K, c128V, status)
        torch.cuda.synchronize()
        runs.append((c128K, c128V, int(status.item())))
    (wholeK, wholeV, ok), (K, V, code) = runs
    assert ok == 0 and code == TV_ERR_ARG
    for whole, part, raw in ((wholeK, K, rawK), (wholeV, V, rawV)):
        for p in range(G):
            want = torch.full_like(whole[p], 7.0) if p == order[missing] else whole[p]
            assert torch.equal(part[p], want), p
        # and those are the entries: the gated sum of their 128 rows, in fp64
        for logical in (0, 7, 9, 16):
            p, n = order[logical], min(P // 128, L // 128 - logical * P // 128)
            z = (rawK[p].double() @ g.double()).view(-1, 128)
            w = torch.softmax(z, 1)[:, :, None]
            ref = (w * raw[p].double().view(-1, 128, d)).sum(1)[:n]
            # (2^-8: the rounding of the stored entry; fp32 weights and sums are far below 1e-5)
            assert bool(((part[p, :n].double() - ref).abs() <= ref.abs() * 2 ** -8 + 1e-5).all()), logical


@pytest.mark.parametrize("ms", [(4, 128), (4,), (128,)])
def test_prefill_with_a_page_missing(ms):
    wl = workloads.make_workload("hole", B=3, D=4, H=2, d=64, W=128, tail_mode="window", ms=ms, dtype="f32",
                                 L=(1500, 2000), k=2, steps=3, p_match=0.5, seed=4, kv_scale=0.5)
    runs = []
    for hole in (False, True):
        shape, st = engine.alloc_paged(wl, 512, seed=1)
        rb = engine.alloc_round(wl, shape)
        for t in (st.c4K, st.c4V, st.c128K, st.c128V):
            t.fill_(7.0)
        gone = int(st.page_table[1, 1])
        if hole:
            st.page_table[1, 1] = -1
        engine.prefill(shape, st, rb)
        torch.cuda.synchronize()
        assert int(rb.status.item()) == (TV_ERR_ARG if hole else 0)
        runs.append(st)
    for m, names in ((4, ("c4K", "c4V")), (128, ("c128K", "c128V"))):
        for name in names if m in ms else ():
            whole, part = getattr(runs[0], name), getattr(runs[1], name)
            for p in range(whole.shape[0]):
                want = torch.full_like(whole[p], 7.0) if p == gone else whole[p]
                assert torch.equal(part[p], want), (name, p)


@pytest.mark.parametrize("L", [511, 512, 505])
def test_staging_with_a_page_missing(L):
    # request 0 has no page behind its first: what its cached chain would stage there is left out and
    # reported, the rows that still fit its first page are staged, the other request's are too
    wl = workloads.serving(B=2, L=(600, 600))
    wl.L[0] = L
    shape, st = engine.alloc_pool(wl, 512, 4, stage_chain=1)
    rb = engine.alloc_round(wl, shape)
    engine.prefill(shape, st, rb)
    engine.plan(shape, st, rb)
    torch.cuda.synchronize()
    before = {k: getattr(st, k).clone() for k in ("rawK", "rawV", "c4K", "c4V", "c128K", "c128V")}
    engine.branch_compress(shape, st, rb)
    torch.cuda.synchronize()
    table = st.page_table.tolist()
    want = {k: t.clone() for k, t in before.items()}
    left_out = False
    for b in range(2):
        v, depth = 0, 0
        while v is not None:
            pos = int(wl.L[b]) + depth
            page = table[b][pos // 512]
            if page < 0:
                left_out = True
            else:
                for raw, tree, c4, scr in (("rawK", rb.treeK, "c4K", rb.scrK4),
                                           ("rawV", rb.treeV, "c4V", rb.scrV4)):
                    want[raw][page, pos % 512] = tree[b, v]
                    if (pos + 1) % 4 == 0:
                        want[c4][page, pos % 512 // 4] = scr[b, v]
            kids = [u for u in range(1, wl.D) if wl.parents[b][u] == v]
            v, depth = (kids[0] if kids else None), depth + 1
    assert int(rb.status.item()) == (TV_ERR_ARG if left_out else 0)
    assert left_out or L == 505
    for k, t in want.items():
        assert torch.equal(getattr(st, k), t), k
    assert np.array_equal(st.L.cpu().numpy(), wl.L)

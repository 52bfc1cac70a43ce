"""The chunk calls at the ends of their ranges: work lists and batches that 32 or 16 bits do not count."""

import math

import numpy as np
import pytest
import torch

from oracle import chunk
from test_gpu_chunk import Batch
from tree_speculative_verify_gb300 import _lib

pytestmark = pytest.mark.gpu


def np64(t):
    return t.detach().double().cpu().numpy()


def test_a_work_list_of_more_than_2_31_half_tiles():
    """2^20 requests of one token, all behind the same page of 2^19: 2054 places each, on the tensor cores (the
    C128 entries, of which such a batch could have too many, are not active).  Sixteen queries and three
    lengths, so that every row can be compared.  Tolerances: as in test_gpu_chunk.py, and as these sums are
    long, a step (2^-23 of the partial sum) per product of 16 entries, 8192 of them, in O, and half a step
    per tile and CTA, 1100 at most, in the sum of the probabilities."""
    B, P, d, W = 1 << 20, 1 << 19, 128, 128
    g = torch.Generator().manual_seed(31)
    pool = [(0.5 * torch.randn((1, rows, d), generator=g)).bfloat16() for rows in (P, P, P // 4, P // 4)]
    rawK, rawV, c4K, c4V = (t.cuda() for t in pool)
    table = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    shape = _lib.make_shape(B=B, D=1, H=1, d=d, W=W, comp_mask=_lib.TV_COMP_C4, dtype=_lib.TV_BF16,
                            tail_mode=_lib.TV_TAIL_WINDOW, raw_cap=P, c4_cap=P // 4, c128_cap=P // 128,
                            attn_kernel=_lib.TV_ATTN_TCGEN05, page_tokens=P, max_pages=1, n_pool_pages=1,
                            page_table=table)
    kinds = (2.0 * torch.randn((16, 1, d), generator=g)).bfloat16()
    b = torch.arange(B, device="cuda")
    Q, L = kinds.cuda()[b % 16].contiguous(), (P - b % 3).to(torch.int32)
    starts = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    O, lse = torch.full_like(Q, 7.0), torch.full((B, 1), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.full((_lib.tv_chunk_workspace_size(shape, B),), 0xff, dtype=torch.uint8, device="cuda")
    scale = 1 / math.sqrt(d)
    _lib.tv_chunk_attn(shape, starts, Q, c4K, c4V, None, None, rawK, rawV, L, scale, O, lse, ws, status)
    torch.cuda.synchronize()
    assert status.item() == 0
    comp = {4: (np64(c4K[0]), np64(c4V[0]))}
    raw = np64(rawK[0]), np64(rawV[0])
    for less in range(3):
        want = chunk.attend_request(np64(kinds).reshape(1, 16, d), P - less, *raw, comp, W, "window", scale)
        want, want_lse, spread, size = (x[0] for x in want)
        e = 2 * d * 2.0 ** -24 * size
        long = 8192 * 2.0 ** -23 + 1100 * 2.0 ** -24
        tol = (2 * e[:, None] + 2.0 ** -8 + 2.0 ** -20 + long) * spread + 2.0 ** -8 * np.abs(want)
        tol_lse = e + 2.0 ** -20 * (np.abs(want_lse) + 1) + 1100 * 2.0 ** -24
        want, tol, want_lse, tol_lse = (torch.from_numpy(x).cuda() for x in (want, tol, want_lse, tol_lse))
        rows = (b % 3 == less).nonzero()[:, 0]
        for part in rows.split(1 << 16):
            kind = part % 16
            assert ((O[part, 0].double() - want[kind]).abs() <= tol[kind]).all()
            assert ((lse[part, 0].double() - want_lse[kind]).abs() <= tol_lse[kind]).all()


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (512, "bf16"), (64, "f32")])
def test_more_requests_than_a_grid_has_rows(d, dtype):
    """Page pools of 70000 slots, six of them in use, before and behind the 65535 that a grid's y takes."""
    B, at = 70000, [0, 7, 65534, 65535, 65536, 69999]
    s = Batch([700, 0, 1000, 511, 300, 129], [1, 3, 2, 1, 150, 1], H=4, d=d, dtype=dtype, P=512, rope=16,
              q_std=2.0, seed=d)
    table = torch.full((B, s.table.shape[1]), -1, dtype=torch.int32)
    table[at] = s.table
    table, L, starts = table.cuda(), torch.full((B,), 77, dtype=torch.int32), torch.zeros(B + 1, dtype=torch.int32)
    L[at] = torch.tensor(s.before, dtype=torch.int32)
    starts[1:][at] = torch.tensor(s.news, dtype=torch.int32)
    s.L, s.gpu_starts = L.cuda(), starts.cumsum(0).to(torch.int32).cuda()
    s.shape.B, s.shape.page_table = B, table.data_ptr()
    s.ws = torch.full((_lib.tv_chunk_workspace_size(s.shape, s.n),), 0xff, dtype=torch.uint8, device="cuda")
    old = [s.oracle_caches(b) for b in range(s.B)]
    s.append(s.Q, s.Qr)
    s.attend()
    torch.cuda.synchronize()
    assert s.status.item() == 0
    idle = torch.ones(B, dtype=torch.bool)
    idle[at] = False
    assert torch.all(s.L.cpu()[idle] == 77)
    s.L = s.L[at]
    s.check_append(old, s.Qr)
    s.check_attend()

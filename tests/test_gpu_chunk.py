"""tv_chunk_append and tv_chunk_attn on the GPU against the oracle, contiguous and paged.

Tolerances, from the roundings each side makes (u(t) = half a step of type t relative to the value:
bf16 2^-8, fp32 2^-24):
* a rotated element: u(t) of the result, and in fp32 the two products, their sum, cos and sin (2^-22
  relative each) on |x| + |y|: 2^-21 (|x| + |y|);
* an entry: its weights come from logits z = K.g summed in fp32, off by at most d u(fp32) sum |K_i g_i|
  =: e, so a weight is off by a factor of 1 +- 2e, the entry by 2e (max - min of the block's values),
  plus u(t) of the result and 2^-20 of the largest value for the sums;
* attention: a logit is off by at most e = 2 d u(fp32) max_j sum_i |q_i k_ji| scale (tensor-core sums
  may truncate: a whole step per addition), a probability by a factor of 1 +- 2e, on tensor cores also by
  u(bf16) of its rounding; so O by (2e + u + 2^-20) sum_j p_j |v_j| and u(t) |O|; lse by e + 2^-20 (|lse|
  + 1) (2^-20: base-2 exponentials and logarithms, the sums of up to some thousand terms).
"""

import math

import numpy as np
import pytest
import torch

from oracle import chunk
from tree_speculative_verify_gb300 import _lib, engine, workloads

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
NAMES = ("rawK", "rawV", "c4K", "c4V", "c128K", "c128V")


def np64(t):
    return t.detach().double().cpu().numpy()


class Batch:
    """A ragged batch: caches of `before` tokens per request, `news` new ones, on GPU and for the oracle."""

    def __init__(self, before, news, *, H=4, d=64, dtype="f32", P=0, W=128, tail="window", ms=(4, 128),
                 rope=0, pairs=0, pad_front=0, pad_back=0, ld=0, seed=0, cap=None, q_std=1.0, attn=0):
        g = torch.Generator().manual_seed(seed)
        self.before, self.news, self.H, self.d, self.P, self.W = list(before), list(news), H, d, P, W
        self.tail, self.ms, self.rope, self.pairs, self.dtype = tail, ms, rope, pairs, dtype
        B = self.B = len(before)
        dt = self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        randn = lambda *s: torch.randn(s, generator=g)
        most = max([b + n for b, n in zip(before, news)] + [1])
        unit = P or 128
        G = -(-(cap or most) // unit)
        self.cap = G * unit
        table = None
        if P:
            self.pool = B * G + 3
            self.table = torch.randperm(self.pool, generator=g)[:B * G].reshape(B, G).to(torch.int32)
            table = self.table.cuda()
        self.t = {}
        for name, m in zip(NAMES, (1, 1, 4, 4, 128, 128)):
            if m == 1 or m in ms:
                size = (self.pool, P // m, d) if P else (B, self.cap // m, d)
                self.t[name] = (0.5 * randn(*size)).to(dt).cuda()
        self.gates = {m: randn(d) / math.sqrt(d) for m in (4, 128)}
        self.starts = np.concatenate([[pad_front], pad_front + np.cumsum(news)]).astype(np.int32)
        self.n = int(self.starts[-1]) + pad_back
        wide = max(ld, d)
        self.KV = [(0.5 * randn(self.n, wide)).to(dt).cuda()[:, :d] for _ in range(2)]
        self.Q = (q_std * randn(self.n, H, d)).to(dt).cuda()
        self.inv_freq = (100.0 ** (-torch.arange(rope // 2) / max(rope // 2, 1))).float()
        mask = (_lib.TV_COMP_C4 if 4 in ms else 0) | (_lib.TV_COMP_C128 if 128 in ms else 0)
        paged = dict(page_tokens=P, max_pages=G, n_pool_pages=self.pool, page_table=table) if P else {}
        self.gpu_table = table
        self.shape = _lib.make_shape(
            B=B, D=1, H=H, d=d, W=W, comp_mask=mask,
            tail_mode=_lib.TV_TAIL_WINDOW if tail == "window" else _lib.TV_TAIL_REMAINDER,
            dtype=_lib.TV_BF16 if dtype == "bf16" else _lib.TV_F32, raw_cap=self.cap,
            c4_cap=self.cap // 4, c128_cap=self.cap // 128, attn_kernel=attn, **paged)
        i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32).cuda()
        self.L, self.gpu_starts, self.status = i32(before), i32(self.starts), i32([0])
        self.O = torch.full((self.n, H, d), 7.0, dtype=dt).cuda()
        self.lse = torch.full((self.n, H), 7.0).cuda()
        self.Qr = torch.full((self.n, H, d), 7.0, dtype=dt).cuda()
        size = _lib.tv_chunk_workspace_size(self.shape, self.n)
        self.ws = torch.full((max(size, 256),), 0xff, dtype=torch.uint8, device="cuda")

    def append(self, Q=None, Qr=None, stream=None):
        dev = {m: v.cuda() for m, v in self.gates.items()}
        f = self.inv_freq.cuda() if self.rope else None
        torch.cuda.synchronize()
        _lib.tv_chunk_append(self.shape, self.gpu_starts, *self.KV, Q, self.rope, self.pairs, f, dev[4],
                             dev[128], Qr, *[self.t.get(k) for k in NAMES], self.L, self.status, stream)
        torch.cuda.synchronize()

    def attend(self, stream=None, scale=None):
        t = self.t
        _lib.tv_chunk_attn(self.shape, self.gpu_starts, self.Q, t.get("c4K"), t.get("c4V"),
                           t.get("c128K"), t.get("c128V"), t["rawK"], t["rawV"], self.L,
                           scale or 1 / math.sqrt(self.d), self.O, self.lse, self.ws, self.status, stream)

    # ---- the oracle's view of the caches: per request, logical rows
    def rows(self, name, m, b, count):
        x = self.t[name]
        if not self.P:
            return np64(x[b, :count])
        per = self.P // m
        pages = self.table[b, :-(-count // per)].long()
        return np64(x[pages.cuda()].reshape(-1, self.d)[:count])

    def oracle_caches(self, b, cap=None):
        cap = cap or self.cap
        comp = {m: (self.rows(f"c{m}K", m, b, cap // m), self.rows(f"c{m}V", m, b, cap // m))
                for m in self.ms}
        return self.rows("rawK", 1, b, cap), self.rows("rawV", 1, b, cap), comp

    def check_append(self, old, Qr=None, bad=()):
        """`old`: every request's oracle caches before the call."""
        L = self.L.tolist()
        for b in range(self.B):
            lo, hi, start = int(self.starts[b]), int(self.starts[b + 1]), self.before[b]
            rawK, rawV, comp = old[b]
            newK, newV, new = self.oracle_caches(b)
            n = 0 if b in bad else hi - lo
            assert L[b] == start + n
            pos = range(start, start + n)
            K, V = np64(self.KV[0][lo:lo + n]), np64(self.KV[1][lo:lo + n])
            want = chunk.rotate(K, pos, self.rope, self.pairs, self.inv_freq.numpy())
            got = newK[start:start + n]
            self._rotated(got, want, K)
            if Qr is not None and n:
                Q = np64(self.Q[lo:hi])
                self._rotated(np64(Qr[lo:hi]), chunk.rotate(Q, pos, self.rope, self.pairs,
                                                            self.inv_freq.numpy()), Q)
            assert np.array_equal(newV[start:start + n], V)
            keep = np.r_[0:start, start + n:self.cap]
            assert np.array_equal(newK[keep], rawK[keep]) and np.array_equal(newV[keep], rawV[keep])
            for m in self.ms:
                first, end = start // m, (start + n) // m
                for side, (have, was, raw) in enumerate(((new[m][0], comp[m][0], newK),
                                                         (new[m][1], comp[m][1], newV))):
                    keep = np.r_[0:first, end:self.cap // m]
                    assert np.array_equal(have[keep], was[keep]), (b, m, side)
                    for j in range(first, end):
                        bk, bv = newK[m * j:m * j + m], raw[m * j:m * j + m]
                        g = self.gates[m].double().numpy()
                        z = bk @ g
                        w = np.exp(z - z.max())
                        e = self.d * 2.0 ** -24 * (np.abs(bk) @ np.abs(g)).max()
                        exact = (w / w.sum()) @ bv
                        tol = (2 * e * (bv.max(0) - bv.min(0)) + HALF[self.dtype] * np.abs(exact)
                               + 2.0 ** -20 * np.abs(bv).max(0))
                        assert np.all(np.abs(have[j] - exact) <= tol), (b, m, j, side)

    def _rotated(self, got, want, rows):
        both = np.zeros_like(want)
        if self.rope:
            tail = np.abs(rows[..., -self.rope:])
            half = self.rope // 2
            pair = (np.repeat(tail[..., 0::2] + tail[..., 1::2], 2, axis=-1) if self.pairs
                    else np.concatenate([tail[..., :half] + tail[..., half:]] * 2, axis=-1))
            both[..., -self.rope:] = pair
        tol = HALF[self.dtype] * np.abs(want) + 2.0 ** -21 * both
        tol[..., :self.d - self.rope] = 0
        assert np.all(np.abs(got - want) <= tol)

    def check_attend(self, bad=(), requests=None, scale=None):
        O, lse = np64(self.O), np64(self.lse)
        used = np.zeros(self.n, bool)
        on_tc = self.dtype == "bf16"
        for b in range(self.B):
            lo, hi = int(self.starts[b]), int(self.starts[b + 1])
            if b in bad or lo == hi:
                continue
            used[lo:hi] = True
            if requests is not None and b not in requests:
                continue
            L = self.before[b] + hi - lo
            rawK, rawV, comp = self.oracle_caches(b, cap=-(-L // 128) * 128)
            want, want_lse, spread, size = chunk.attend_request(
                np64(self.Q[lo:hi]), L, rawK, rawV, comp, self.W, self.tail,
                scale or 1 / math.sqrt(self.d))
            e = 2 * self.d * 2.0 ** -24 * size
            u = HALF["bf16"] if on_tc else 0.0
            tol = ((2 * e[..., None] + u + 2.0 ** -20) * spread + HALF[self.dtype] * np.abs(want))
            assert np.all(np.abs(O[lo:hi] - want) <= tol), (b, np.abs(O[lo:hi] - want).max())
            assert np.all(np.abs(lse[lo:hi] - want_lse) <= e + 2.0 ** -20 * (np.abs(want_lse) + 1)), b
        assert np.all(O[~used] == 7.0) and np.all(lse[~used] == 7.0)   # rows of no request


SHAPES = [  # d, dtype, H
    (64, "f32", 8), (8, "f32", 1), (72, "bf16", 3), (512, "bf16", 4), (256, "f32", 2)]


@pytest.mark.parametrize("d,dtype,H", SHAPES)
@pytest.mark.parametrize("P", [0, 512, 1536])
@pytest.mark.parametrize("ms", [(4, 128), (4,), (128,)])
def test_append_writes_rows_entries_and_lengths(d, dtype, H, P, ms):
    r = min(d, 64) // 2 * 2
    s = Batch([0, 0, 3, 127, 128, 500, 511, 1000, 1535, 40], [1, 300, 1, 1, 130, 20, 1, 0, 2, 600], H=H, d=d,
              dtype=dtype, P=P, ms=ms, rope=r, pairs=d % 16 == 0, seed=d + P)
    old = [s.oracle_caches(b) for b in range(s.B)]
    s.append(s.Q, s.Qr)
    assert s.status.item() == 0
    s.check_append(old, s.Qr)


@pytest.mark.parametrize("pairs", [0, 1])
@pytest.mark.parametrize("rope", [0, 2, 62, 64])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_strided_rows_padding_and_queries_in_place(rope, pairs, dtype):
    s = Batch([10, 60000, 0], [7, 3, 5], H=3, d=64, dtype=dtype, rope=rope, pairs=pairs, pad_front=2,
              pad_back=3, ld=96, seed=rope)
    old = [s.oracle_caches(b) for b in range(s.B)]
    t = {k: v.clone() for k, v in s.t.items()}
    s.append(s.Q, s.Qr)
    s.check_append(old, s.Qr)
    assert torch.all(s.Qr[:2] == 7) and torch.all(s.Qr[-3:] == 7)
    again = s.Q.clone()
    s.t, s.L = t, torch.tensor(s.before, dtype=torch.int32).cuda()
    s.append(again, again)
    assert torch.equal(again[2:-3], s.Qr[2:-3]) and torch.equal(again[:2], s.Q[:2])
    assert torch.equal(again[-3:], s.Q[-3:]) and s.status.item() == 0


@pytest.mark.parametrize("d,dtype", [(512, "bf16"), (64, "f32"), (128, "bf16")])
def test_entries_equal_prefill_however_the_tokens_are_split(d, dtype):
    whole = Batch([0, 5], [900, 777], d=d, dtype=dtype, P=512, rope=32, seed=3)
    parts = Batch([0, 5], [900, 777], d=d, dtype=dtype, P=512, rope=32, seed=3)
    whole.append()
    done = [0, 0]
    rng = np.random.default_rng(0)
    K, V = parts.KV
    lo = parts.starts.copy()
    while done != [900, 777]:
        step = [int(min(rng.choice([0, 1, 2, 3, 60, 128, 129]), n - k)) for n, k in zip((900, 777), done)]
        pick = np.concatenate([lo[b] + done[b] + np.arange(step[b]) for b in range(2)]).astype(np.int64)
        parts.KV = [x[torch.from_numpy(pick).cuda()] for x in (K, V)]
        parts.gpu_starts = torch.tensor([0, step[0], sum(step)], dtype=torch.int32).cuda()
        parts.append()
        done = [k + n for k, n in zip(done, step)]
    assert parts.L.tolist() == whole.L.tolist() == [900, 782] and parts.status.item() == 0
    for k in NAMES:
        assert torch.equal(parts.t[k], whole.t[k]), k
    # and prefill writes the same entries from the rows (its first entry of request 1 is of old rows)
    again = {k: v.clone() for k, v in whole.t.items()}
    dev = {m: v.cuda() for m, v in whole.gates.items()}
    _lib.tv_prefill_compress(whole.shape, again["rawK"], again["rawV"], whole.L, dev[4], dev[128],
                             again["c4K"], again["c4V"], again["c128K"], again["c128V"], whole.status)
    old = Batch([0, 5], [900, 777], d=d, dtype=dtype, P=512, rope=32, seed=3)
    page = int(whole.table[1, 0])
    for k in ("c4K", "c4V"):
        again[k][page, 0] = old.t[k][page, 0]
    for k in NAMES:
        assert torch.equal(again[k], whole.t[k]), k


def test_append_refuses_requests_one_by_one():
    P = 512
    s = Batch([100, 500, -3, 1020, 7, 0], [5, 30, 2, 10, 4, 3], d=64, P=P, seed=4, cap=1024)
    table = s.table.clone()
    table[1, 1] = -1         # the second page of request 1's new rows is missing
    table[5, 0] = 10 ** 6
    s.gpu_table.copy_(table.cuda())
    before = {k: v.clone() for k, v in s.t.items()}
    s.append()
    assert s.L.tolist() == [105, 500, -3, 1020, 11, 0] and s.status.item() in (-1, -4)
    good = Batch([100, 500, -3, 1020, 7, 0], [5, 30, 2, 10, 4, 3], d=64, P=P, seed=4, cap=1024)
    for k in NAMES:
        changed = (s.t[k] != before[k]).flatten(1).any(1).nonzero()[:, 0].tolist()
        allowed = {int(good.table[0, 0]), int(good.table[4, 0])}
        assert set(changed) <= allowed, k


@pytest.mark.parametrize("starts", [[0, 5, 3, 8], [-1, 2, 4, 8], [0, 3, 6, 99]])
def test_append_with_malformed_starts_changes_only_good_requests(starts):
    s = Batch([10, 20, 30], [3, 3, 2], d=64, seed=5)
    before = {k: v.clone() for k, v in s.t.items()}
    s.gpu_starts = torch.tensor(starts, dtype=torch.int32).cuda()
    s.append()
    bad = [b for b in range(3) if not 0 <= starts[b] <= starts[b + 1] <= s.n]
    assert bad and s.status.item() == -1
    for b in bad:
        assert s.L[b].item() == s.before[b]
        for k in NAMES:
            assert torch.equal(s.t[k][b], before[k][b]), k
    s.attend()      # nor does attention touch rows it cannot place
    torch.cuda.synchronize()


DESCENDING = [[0, 1000, 100, 300, 300], [0, 1000, 3, 500, 1000], [0, 900, 900, 900, 3, 3, 3, 3, 1000],
              [700, 700, 0, 1000], [0, 127, 1, 1000]]


@pytest.mark.parametrize("starts", DESCENDING + [None] * 6, ids=lambda s: "random" if s is None else None)
@pytest.mark.parametrize("P", [0, 512])
def test_append_with_descending_starts_takes_requests_whole_or_not_at_all(starts, P, request):
    """Enough tokens for the kernel that searches the starts: a request whose length advances has all its rows
    and entries, any other none."""
    rng = np.random.default_rng(len(request.node.name) * 7 + P)
    for _ in range(1 if starts else 8):
        at = starts or np.sort(rng.integers(0, 1001, rng.integers(3, 40))).tolist()
        if not starts:
            for i in rng.integers(0, len(at), 3):
                at[i] = int(rng.integers(-50, 1100))
        B = len(at) - 1
        s = Batch(rng.integers(0, 300, B).tolist(), [1000] + [0] * (B - 1), d=64, dtype="f32", P=P, rope=16,
                  seed=len(at), cap=1536)
        old = [s.oracle_caches(b) for b in range(B)]
        s.starts = np.array(at)
        s.gpu_starts = torch.tensor(at, dtype=torch.int32).cuda()
        s.append()
        bad = [b for b in range(B) if s.L[b].item() == s.before[b]]
        s.check_append(old, bad=bad)
        for b in range(B):
            if not 0 <= at[b] <= at[b + 1] <= s.n:
                assert b in bad and s.status.item() == -1


# ---- attention ------------------------------------------------------------------------------------
ATTEND = [  # before, news
    ([0], [1]), ([0, 0, 0], [1, 5, 130]), ([127, 128, 129, 3], [1, 1, 1, 1]), ([1000], [1]),
    ([700, 0, 5, 2000], [70, 3, 0, 1]), ([511, 512, 513], [2, 1, 33]), ([3500], [9])]


@pytest.mark.parametrize("d,dtype,H", [(64, "f32", 8), (512, "bf16", 64), (512, "bf16", 24), (128, "bf16", 5),
                                       (256, "f32", 3), (8, "f32", 1), (72, "bf16", 2), (512, "f32", 2)])
@pytest.mark.parametrize("P", [0, 512, 1536])
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attend_matches_the_oracle(d, dtype, H, P, case):
    before, news = ATTEND[case]
    s = Batch(before, news, H=H, d=d, dtype=dtype, P=P, q_std=2.0, seed=case, pad_front=case % 2,
              pad_back=3 * (case % 3))
    s.append()
    s.attend()
    torch.cuda.synchronize()
    assert s.status.item() == 0
    s.check_attend()


@pytest.mark.parametrize("W,tail,ms", [(0, "window", (4, 128)), (1, "window", (4,)), (37, "window", (128,)),
                                       (300, "window", (4, 128)), (1024, "window", (4,)),
                                       (0, "remainder", (4, 128)), (0, "remainder", (128,))])
@pytest.mark.parametrize("d,dtype,H", [(512, "bf16", 64), (64, "f32", 4), (128, "bf16", 16)])
@pytest.mark.parametrize("P", [0, 1024])
def test_attend_windows_and_compressors(W, tail, ms, d, dtype, H, P):
    s = Batch([1100, 0, 60], [40, 9, 1], H=H, d=d, dtype=dtype, P=P, W=W, tail=tail, ms=ms, q_std=2.0,
              seed=W)
    s.append()
    s.attend()
    torch.cuda.synchronize()
    assert s.status.item() == 0
    s.check_attend()


@pytest.mark.parametrize("d,H", [(512, 64), (512, 128), (512, 24), (512, 1), (384, 16), (256, 11), (128, 64),
                                 (128, 3)])
@pytest.mark.parametrize("P", [0, 1024])
@pytest.mark.parametrize("W", [0, 128, 300])
def test_attend_decoding_batches(d, H, P, W):
    # requests of no, one and two tokens at lengths around every tile boundary
    before = [0, 3, 4, 63, 64, 126, 127, 128, 255, 511, 512, 600, 1023, 1024, 1500, 2047, 3000, 5, 900]
    news = [1, 1, 1, 1, 0, 1, 1, 2, 1, 1, 1, 1, 1, 2, 1, 0, 1, 1, 1]
    s = Batch(before, news, H=H, d=d, dtype="bf16", P=P, W=W, q_std=2.0, seed=W + H)
    s.append()
    s.attend()
    torch.cuda.synchronize()
    assert s.status.item() == 0
    s.check_attend()


@pytest.mark.parametrize("d,H,before,n", [(512, 64, 40000, 1), (512, 64, 9000, 2), (512, 16, 20000, 5),
                                          (128, 8, 5000, 150), (256, 16, 100, 90)])
def test_attend_long_requests(d, H, before, n):
    s = Batch([before], [n], H=H, d=d, dtype="bf16", P=2048, q_std=2.0, seed=n)
    s.append()
    s.attend()
    torch.cuda.synchronize()
    assert s.status.item() == 0
    s.check_attend()


@pytest.mark.parametrize("H,P,W,ms,news", [
    (64, 1024, 128, (4, 128), [161, 3, 0, 40]), (128, 512, 100, (4, 128), [90, 33]), (24, 0, 0, (4,), [600]),
    (64, 1536, 300, (128,), [200, 1, 1]), (16, 512, 37, (4, 128), [900]), (40, 0, 1024, (4, 128), [128, 200])])
def test_attend_many_rows(H, P, W, ms, news):
    # enough rows for the kernel that shares a tile among 256 of them; the last items are split
    before = [1900, 130, 7, 511][:len(news)]
    s = Batch(before, news, H=H, d=512, dtype="bf16", P=P, W=W, ms=ms, q_std=2.0, seed=H + W, pad_front=1,
              pad_back=2)
    s.append()
    s.attend()
    torch.cuda.synchronize()
    assert s.status.item() == 0
    s.check_attend()


@pytest.mark.parametrize("d,dtype,H,P,W", [(512, "bf16", 1024, 512, 1024), (128, "bf16", 1000, 0, 1024),
                                           (64, "f32", 1024, 512, 1023), (72, "bf16", 333, 0, 1024),
                                           (512, "bf16", 2, 512, 1024), (512, "f32", 3, 512, 1024)])
def test_most_heads_and_widest_windows(d, dtype, H, P, W):
    s = Batch([1500, 3, 1020], [2, 1, 5], H=H, d=d, dtype=dtype, P=P, W=W, rope=8, q_std=2.0, seed=H + d)
    old = [s.oracle_caches(b) for b in range(s.B)]
    s.append(s.Q, s.Qr)
    s.check_append(old, s.Qr)
    s.attend()
    torch.cuda.synchronize()
    assert s.status.item() == 0
    s.check_attend()


def test_attend_growing_maxima():
    # logits that grow by hundreds from tile to tile: every tile rescales what is there
    s = Batch([6000, 6000], [1, 1], H=64, d=512, dtype="bf16", P=512, q_std=0.0, seed=13)
    s.append()
    ramp = torch.linspace(0, 1, s.t["c4K"].shape[1], device="cuda")
    for b in range(2):
        for g, page in enumerate(s.table[b].tolist()):
            s.t["c4K"][page] = ((g + ramp) / 12).bfloat16()[:, None] * (1 if b == 0 else -1)
    s.Q[:] = 1.0
    s.attend(scale=1.0)
    torch.cuda.synchronize()
    assert s.status.item() == 0
    s.check_attend(scale=1.0)


def test_attend_equals_one_token_at_a_time():
    # a chunk sees what its tokens would have seen one by one (up to the order of sums)
    s = Batch([900, 0], [37, 5], H=64, d=512, dtype="bf16", P=512, seed=6)
    s.append()
    s.attend()
    torch.cuda.synchronize()
    whole, lse = s.O.clone(), s.lse.clone()
    for i in range(37):
        one = [1 if i < n else 0 for n in s.news]
        at = [int(s.starts[b]) + i for b in range(2)]
        Q = torch.cat([s.Q[a:a + 1] for a, k in zip(at, one) if k])
        L = torch.tensor([b + i + 1 for b in s.before], dtype=torch.int32).cuda()
        starts = torch.tensor([0, one[0], sum(one)], dtype=torch.int32).cuda()
        O, l1 = torch.empty_like(Q), torch.empty((len(Q), 64), device="cuda")
        _lib.tv_chunk_attn(s.shape, starts, Q, s.t["c4K"], s.t["c4V"], s.t["c128K"], s.t["c128V"],
                           s.t["rawK"], s.t["rawV"], L, 1 / math.sqrt(512), O, l1, s.ws, s.status)
        torch.cuda.synchronize()
        for j, (a, k) in enumerate((x for x in zip(at, one) if x[1])):
            # two roundings of probabilities and outputs to bf16, on values below 0.5 * 5
            assert (O[j].float() - whole[a].float()).abs().max() <= 4 * 2.0 ** -8 * whole[a].abs().max()
            assert (l1[j] - lse[a]).abs().max() <= 1e-4
    assert s.status.item() == 0


def test_attend_extreme_logits():
    # one key far above all others, equal keys, and logits of hundreds: no overflow, weights to 1 and 0
    s = Batch([300, 300], [6, 1], H=8, d=512, dtype="bf16", q_std=0.0, seed=7)
    s.append()
    s.Q[:3] = 40.0 * s.t["rawK"][0, 301]
    s.Q[3:6] = -40.0 * s.t["rawK"][0, 250]
    s.attend(scale=1.0)
    torch.cuda.synchronize()
    assert s.status.item() == 0 and torch.isfinite(s.O.float()).all()
    s.check_attend(scale=1.0)


def test_attend_refuses_requests_one_by_one():
    s = Batch([100, 50, 3000], [5, 4, 6], H=4, d=512, dtype="bf16", seed=8)
    s.append()
    s.L[1] = 2                # shorter than its chunk
    s.L[2] = s.cap + 1
    s.attend()
    torch.cuda.synchronize()
    assert s.status.item() in (-1, -4)
    s.check_attend(bad=(1, 2))


@pytest.mark.parametrize("d,dtype", [(512, "bf16"), (64, "f32")])
def test_a_missing_page_is_reported_and_nothing_else_suffers(d, dtype):
    s = Batch([1500, 1500], [3, 3], H=8, d=d, dtype=dtype, P=512, seed=9)
    s.append()
    s.gpu_table[1, 0] = -1
    s.attend()
    torch.cuda.synchronize()
    assert s.status.item() == -1
    s.check_attend(requests=(0,))


@pytest.mark.parametrize("d,dtype,P", [(512, "bf16", 512), (512, "bf16", 0), (64, "f32", 512)])
def test_captured_and_replayed_on_another_stream(d, dtype, P):
    s = Batch([60, 1000, 0], [9, 1, 150], H=16, d=d, dtype=dtype, P=P, rope=16, seed=10)
    dev = {m: v.cuda() for m, v in s.gates.items()}
    f, L0, t0 = s.inv_freq.cuda(), s.L.clone(), {k: v.clone() for k, v in s.t.items()}

    def step():
        s.L.copy_(L0)
        _lib.tv_chunk_append(s.shape, s.gpu_starts, *s.KV, s.Q, 16, 0, f, dev[4], dev[128], s.Qr,
                             *[s.t[k] for k in NAMES], s.L, s.status)
        _lib.tv_chunk_attn(s.shape, s.gpu_starts, s.Qr, s.t["c4K"], s.t["c4V"], s.t["c128K"],
                           s.t["c128V"], s.t["rawK"], s.t["rawV"], s.L, 1 / math.sqrt(d), s.O, s.lse,
                           s.ws, s.status)

    step()
    torch.cuda.synchronize()
    O, lse, rows = s.O.clone(), s.lse.clone(), {k: v.clone() for k, v in s.t.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for k, v in t0.items():
            s.t[k].copy_(v)
        s.O.zero_()
        s.ws.fill_(0xff)
        graph.replay()
        torch.cuda.synchronize()
        used = slice(int(s.starts[0]), int(s.starts[-1]))
        assert torch.equal(s.O[used], O[used]) and torch.equal(s.lse[used], lse[used])
        assert all(torch.equal(s.t[k], rows[k]) for k in NAMES)
    other = torch.cuda.Stream()
    for k, v in t0.items():
        s.t[k].copy_(v)
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        step()
    other.synchronize()
    assert torch.equal(s.O[used], O[used]) and all(torch.equal(s.t[k], rows[k]) for k in NAMES)
    assert s.status.item() == 0


@pytest.mark.parametrize("d,dtype,H,n", [(512, "bf16", 64, 8), (512, "bf16", 64, 150), (64, "f32", 4, 40)])
def test_one_capture_serves_any_starts(d, dtype, H, n):
    """A graph captured for n new tokens, replayed with other splits of up to n: each replay is what eager
    calls on caches of its own give, and the rows of no request stay as they are."""
    cut = n // 3
    s = Batch([500, 1000, 0], [n - 2, 1, 1], H=H, d=d, dtype=dtype, P=512, rope=16, seed=21, cap=3000)
    dev = {m: v.cuda() for m, v in s.gates.items()}
    f = s.inv_freq.cuda()

    def step(t, L, Qr, O, lse, ws, status):
        _lib.tv_chunk_append(s.shape, s.gpu_starts, *s.KV, s.Q, 16, 0, f, dev[4], dev[128], Qr,
                             *[t[k] for k in NAMES], L, status)
        _lib.tv_chunk_attn(s.shape, s.gpu_starts, Qr, t["c4K"], t["c4V"], t["c128K"], t["c128V"],
                           t["rawK"], t["rawV"], L, 1 / math.sqrt(d), O, lse, ws, status)

    copy = lambda: ({k: v.clone() for k, v in s.t.items()}, s.L.clone(), s.Qr.clone(), s.O.clone(),
                    s.lse.clone(), s.ws.clone(), s.status.clone())
    captured, eager = copy(), copy()
    step(*copy())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*captured)
    for starts in ([0, n - 2, n - 1, n], [0, 1, 2, 3], [2, 2, 2 + cut, 2 + 2 * cut], [0, 0, 0, 0],
                   [0, 0, n, n]):
        s.gpu_starts.copy_(torch.tensor(starts, dtype=torch.int32))
        for x in captured[2:5] + eager[2:5]:
            x.fill_(7.0)
        graph.replay()
        step(*eager)
        torch.cuda.synchronize()
        assert captured[6].item() == 0 and eager[6].item() == 0
        assert all(torch.equal(captured[0][k], eager[0][k]) for k in NAMES)
        used = torch.zeros(n, dtype=torch.bool)
        used[starts[0]:starts[-1]] = True
        for x, y in zip(captured[1:5], eager[1:5]):
            assert torch.equal(x, y)
        for x in captured[2:5]:
            assert torch.all(x[~used.cuda()] == 7.0)
    news = np.diff(starts)
    s.before = [int(x - y) for x, y in zip(captured[1].tolist(), news)]
    s.news, s.starts, s.t, s.L, s.O, s.lse = news, np.array(starts), *captured[:2], *captured[3:5]
    s.Q = captured[2]
    s.check_attend()


def test_nothing_to_do():
    s = Batch([5, 0], [0, 0], H=4, d=64, pad_back=2)
    before = {k: v.clone() for k, v in s.t.items()}
    s.append(s.Q, s.Qr)
    s.attend()
    torch.cuda.synchronize()
    assert s.L.tolist() == [5, 0] and s.status.item() == 0
    assert all(torch.equal(s.t[k], before[k]) for k in NAMES) and torch.all(s.O == 7)
    assert torch.all(s.Qr == 7)


def test_many_requests():
    rng = np.random.default_rng(11)
    B = 3000
    before = rng.integers(0, 40, B).tolist()
    news = rng.choice([0, 1, 1, 2, 5], B).tolist()
    s = Batch(before, news, H=2, d=64, dtype="f32", seed=11)
    s.append()
    s.attend()
    torch.cuda.synchronize()
    assert s.status.item() == 0
    assert s.L.tolist() == [b + n for b, n in zip(before, news)]
    s.check_attend(requests=set(rng.integers(0, B, 60).tolist()))


def test_many_requests_on_tensor_cores():
    rng = np.random.default_rng(12)
    B = 2500
    before = rng.integers(0, 20, B).tolist()
    news = rng.choice([0, 1, 1, 2], B).tolist()
    s = Batch(before, news, H=8, d=512, dtype="bf16", seed=12, ms=(4,))
    s.append()
    s.attend()
    torch.cuda.synchronize()
    assert s.status.item() == 0
    s.check_attend(requests=set(rng.integers(0, B, 40).tolist()))


def test_more_requests_than_a_cta_keeps_starts_of():
    """64-row items on tensor cores, more requests than their starts fit into shared memory."""
    rng = np.random.default_rng(13)
    B = 4500
    before = rng.integers(0, 20, B).tolist()
    news = rng.choice([0, 1, 1, 3], B).tolist()
    s = Batch(before, news, H=3, d=128, dtype="bf16", seed=13, ms=(4,))
    s.append()
    s.attend()
    torch.cuda.synchronize()
    assert s.status.item() == 0
    s.check_attend(requests=set(rng.integers(0, B, 60).tolist()))


def test_many_requests_on_clusters():
    """More requests than the clusters count the items of, 281600 rows in 44 of them."""
    B = 2100
    before = [b % 19 for b in range(B)]
    news = [50 if b % 48 == 7 else 0 for b in range(B)]
    s = Batch(before, news, H=128, d=512, dtype="bf16", seed=14, ms=(4,))
    assert s.n * 128 > 128 * B
    s.append()
    s.attend()
    torch.cuda.synchronize()
    assert s.status.item() == 0
    s.check_attend(requests={7, 7 + 48 * 20, 7 + 48 * 43})


@pytest.mark.parametrize("d,dtype,rope,pairs", [(64, "f32", 64, 0), (64, "f32", 62, 0), (64, "f32", 30, 1),
                                                (128, "bf16", 64, 0), (128, "bf16", 24, 0)])
def test_append_long_streams_of_queries(d, dtype, rope, pairs):
    """More rows than four waves of CTAs, of requests that share CTAs; into other memory and in place."""
    s = Batch([5, 0, 300], [1200, 7, 1239], H=128, d=d, dtype=dtype, rope=rope, pairs=pairs, pad_front=1,
              pad_back=2, seed=15, ms=(4,))
    old = [s.oracle_caches(b) for b in range(s.B)]
    Q = s.Q.clone()
    s.append(Q, s.Qr)
    assert s.status.item() == 0
    s.check_append(old, s.Qr)
    assert torch.all(s.Qr[0] == 7) and torch.all(s.Qr[-2:] == 7)
    s.L.copy_(torch.tensor(s.before, dtype=torch.int32))
    s.append(Q, Q)
    assert torch.equal(Q[1:-2], s.Qr[1:-2])
    assert torch.equal(Q[0], s.Q[0]) and torch.equal(Q[-2:], s.Q[-2:])


@pytest.mark.parametrize("news,tile", [([1] * 40, 0), ([1] * 40, 1), ([2] * 3, 0), ([300], 1)])
def test_a_wait_that_runs_out_reports_timeout_and_the_context_stays_usable(news, tile):
    """The producers leave out the K copies of a tile, so the wait for it expires after 200 us; what was
    issued is drained, and the next call is right again."""
    before = [3000 - 7 * b for b in range(len(news))]
    s = Batch(before, news, H=64, d=512, dtype="bf16", P=512, seed=16)
    s.append()
    _lib.tv_debug_attn_timeout(200_000, tile)
    try:
        s.attend()
        torch.cuda.synchronize()
    finally:
        _lib.tv_debug_attn_timeout(2_000_000_000, -1)
    assert s.status.item() == -8
    s.status.zero_()
    s.O.fill_(7.0)
    s.lse.fill_(7.0)
    s.attend()
    torch.cuda.synchronize()
    assert s.status.item() == 0
    s.check_attend(requests={0, len(news) - 1})


@pytest.mark.parametrize("d,dtype,H", [(512, "bf16", 64), (128, "bf16", 4), (64, "f32", 3)])
@pytest.mark.parametrize("news", [[1, 1, 2], [90, 1, 100]])
@pytest.mark.parametrize("caps", [(201, 50, 1), (127, 31, 0), (250, 62, 1)])
def test_odd_capacities(d, dtype, H, news, caps):
    """Contiguous layers whose rows per request are no multiple of a tile, full to the last row."""
    raw, c4, c128 = caps
    before = [raw - n for n in news]
    s = Batch(before, news, H=H, d=d, dtype=dtype, seed=raw, q_std=2.0)
    for k, rows in zip(NAMES, (raw, raw, c4, c4, max(c128, 1), max(c128, 1))):
        s.t[k] = s.t[k][:, :rows].contiguous()
    s.shape.raw_cap, s.shape.c4_cap, s.shape.c128_cap = caps
    s.cap = raw
    s.ws = torch.full((max(_lib.tv_chunk_workspace_size(s.shape, s.n), 256),), 0xff, dtype=torch.uint8,
                      device="cuda")
    if c128 == 0:
        s.t["c128K"].fill_(9.0)
    s.append()
    s.attend()
    torch.cuda.synchronize()
    assert s.status.item() == 0 and s.L.tolist() == [raw] * 3
    assert c128 > 0 or torch.all(s.t["c128K"] == 9.0)
    s.check_attend()


@pytest.mark.parametrize("d,H,n", [(512, 64, 1), (512, 64, 250), (64, 4, 2)])
def test_offsets_past_32_bits(d, H, n):
    """The same batch in a small pool and at the far end of one of more than 2^32 elements: the same bits."""
    P = 1024
    s = Batch([3000, 5], [n, 1], H=H, d=d, dtype="bf16", P=P, seed=19, rope=16)
    big_pages = 2 ** 32 // (P * d) + s.pool + 1
    far = {}
    for k, m in zip(NAMES, (1, 1, 4, 4, 128, 128)):
        far[k] = torch.zeros((big_pages, P // m, d), dtype=s.dt, device="cuda")
        far[k][-s.pool:] = s.t[k]
    table = s.gpu_table
    s.append(s.Q, s.Qr)
    s.attend()
    torch.cuda.synchronize()
    near, O, lse, Qr = s.t, s.O.clone(), s.lse.clone(), s.Qr.clone()
    s.t = far
    s.far_table = table + (big_pages - s.pool)
    s.shape.n_pool_pages = big_pages
    s.shape.page_table = s.far_table.data_ptr()
    s.L.copy_(torch.tensor(s.before, dtype=torch.int32))
    for x in (s.O, s.lse, s.Qr):
        x.fill_(7.0)
    s.append(s.Q, s.Qr)
    s.attend()
    torch.cuda.synchronize()
    assert s.status.item() == 0
    assert torch.equal(s.O, O) and torch.equal(s.lse, lse) and torch.equal(s.Qr, Qr)
    for k in NAMES:
        assert torch.equal(far[k][-s.pool:], near[k]), k
        assert not far[k][:-s.pool].any(), k


@pytest.mark.parametrize("d,dtype,H,n", [(512, "bf16", 64, 1), (512, "bf16", 64, 200), (128, "bf16", 8, 3),
                                         (64, "f32", 4, 2)])
def test_idle_requests_need_no_pages(d, dtype, H, n):
    """A request without new tokens whose pages are elsewhere (its length stands) is no error."""
    s = Batch([900, 2000, 40], [n, 0, 1], H=H, d=d, dtype=dtype, P=512, seed=20)
    s.table[1] = -1
    s.gpu_table[1] = -1
    s.append(s.Q, s.Qr)
    s.attend()
    torch.cuda.synchronize()
    assert s.status.item() == 0 and s.L.tolist() == [900 + n, 2000, 41]
    s.check_attend()


def test_two_streams_at_once():
    """Two batches of their own, on two streams: bit for bit what each gives alone."""
    batches = [Batch([900, 40, 7000], [n, 1, 1], H=64, d=512, dtype="bf16", P=512, seed=17 + n)
               for n in (1, 250)]
    want = []
    for s in batches:
        s.append()
        s.attend()
        torch.cuda.synchronize()
        want.append((s.O.clone(), s.lse.clone()))
    streams = [torch.cuda.Stream() for _ in batches]
    for _ in range(20):
        for s, stream in zip(batches, streams):
            s.attend(stream)
    torch.cuda.synchronize()
    for s, (O, lse) in zip(batches, want):
        assert s.status.item() == 0 and torch.equal(s.O, O) and torch.equal(s.lse, lse)


def test_prompts_in_chunks_and_rounds_on_one_pool():
    """A prompt appended in two parts behind an empty pool gives the cache that prefill makes, and verify
    rounds go on from it bit for bit as from a prefilled one."""
    wl = workloads.make_workload("chunked", B=2, D=6, H=64, d=512, W=128, tail_mode="window", ms=(4, 128),
                                 dtype="bf16", L=[700, 1030], k=2, steps=3, p_match=0.6, seed=2,
                                 kv_scale=0.5)
    shape, st = engine.alloc_pool(wl, page_tokens=512, n_pool_pages=8)
    rb = engine.alloc_round(wl, shape)
    engine.prefill(shape, st, rb)
    shape2, st2 = engine.clone_pool(shape, st)
    rb2 = engine.alloc_round(wl, shape2)
    for x in (st2.rawK, st2.rawV, st2.c4K, st2.c4V, st2.c128K, st2.c128V, st2.L):
        x.zero_()
    O = lse = None
    for lo, hi in ((0, [300, 1]), ([300, 1], [700, 1030])):
        lo = [lo, lo] if isinstance(lo, int) else lo
        K = torch.cat([wl.rawK[b, lo[b]:hi[b]] for b in range(2)]).cuda()
        V = torch.cat([wl.rawV[b, lo[b]:hi[b]] for b in range(2)]).cuda()
        n = [hi[b] - lo[b] for b in range(2)]
        starts = torch.tensor([0, n[0], n[0] + n[1]], dtype=torch.int32).cuda()
        engine.append(shape2, st2, rb2, starts, K, V)
        Q = torch.randn((len(K), 64, 512), device="cuda").bfloat16()
        ws = engine.alloc_chunk(shape2, len(K))
        O, lse = engine.chunk_attention(shape2, st2, rb2, starts, Q, ws)
    torch.cuda.synchronize()
    assert rb2.status.item() == 0 and torch.isfinite(O.float()).all() and torch.isfinite(lse).all()
    assert torch.equal(st2.L, st.L)
    for b in range(2):
        for m, k in ((1, "rawK"), (1, "rawV"), (4, "c4K"), (4, "c4V"), (128, "c128K"), (128, "c128V")):
            pages = st.page_table[b][st.page_table[b] >= 0].long()
            n = int(wl.L[b]) // m
            a, c = (getattr(x, k)[pages].reshape(-1, 512)[:n] for x in (st, st2))
            assert torch.equal(a, c), (b, k)
    for _ in range(2):
        engine.verify_round(shape, st, rb)
        engine.verify_round(shape2, st2, rb2)
        torch.cuda.synchronize()
        for k in ("O", "lse", "accept_len", "path", "bonus", "committed"):
            assert torch.equal(getattr(rb, k), getattr(rb2, k)), k
        assert torch.equal(st.L, st2.L)
    assert rb.status.item() == 0 and rb2.status.item() == 0

"""Device buffers and the five-call verify round (allocation and marshalling only).

``DeviceState`` holds one batch's persistent cache (raw K/V, C4 and C128 entries, committed
lengths); ``RoundBuffers`` holds one round's inputs (tree, tokens, queries, tree K/V), the plan,
the scratch pad and the outputs.  ``verify_round`` enqueues tv_build_ancestor_mask,
tv_branch_compress, tv_tree_verify_attn, tv_accept_walk and tv_refresh_commit on one stream with
no host synchronisation, as "Adapting Tree-Structured Speculative Decoding to DeepSeek-V4 for
Efficient Inference" §4.1/§4.4 describe one target-verify stage.  Every step runs in the CUDA
library; PyTorch only allocates memory.
"""

import math
from dataclasses import dataclass, fields

import torch

from . import _lib


def shape_for(wl, attn_kernel=_lib.TV_ATTN_AUTO, B=None, stage_chain=0):
    comp = 0
    if 4 in wl.ms:
        comp |= _lib.TV_COMP_C4
    if 128 in wl.ms:
        comp |= _lib.TV_COMP_C128
    return _lib.make_shape(
        B=wl.B if B is None else B, D=wl.D, H=wl.H, d=wl.d, W=wl.W,
        tail_mode=_lib.TV_TAIL_WINDOW if wl.tail_mode == "window" else _lib.TV_TAIL_REMAINDER,
        comp_mask=comp, dtype=_lib.TV_F32 if wl.dtype == "f32" else _lib.TV_BF16,
        n_sel=wl.n_sel, attn_kernel=attn_kernel, raw_cap=wl.raw_cap,
        c4_cap=wl.cap4 if 4 in wl.ms else 0, c128_cap=wl.cap128 if 128 in wl.ms else 0,
        stage_chain=stage_chain)


@dataclass
class DeviceState:
    rawK: torch.Tensor
    rawV: torch.Tensor
    c4K: torch.Tensor
    c4V: torch.Tensor
    c128K: torch.Tensor
    c128V: torch.Tensor
    L: torch.Tensor
    k_idx: torch.Tensor = None    # [B][c4_cap][64] bf16 indexer keys (sparse C4 path only)
    page_table: torch.Tensor = None   # [B][max_pages] int32 (paged pools only)
    page_refs: torch.Tensor = None    # [n_pool_pages] int32 holders (managed pools only)
    page_ws: torch.Tensor = None      # workspace of the tv_pages_* calls (managed pools only)

    def clone(self):
        """A copy of the cache.  The indexer keys and the page table, which a round only reads, stay
        shared; of a managed pool, whose calls write both, ``clone_pool`` makes the copy."""
        if self.page_refs is not None:
            raise ValueError("the copy of a managed pool needs a shape with its own page table: "
                             "use engine.clone_pool(shape, state)")
        return DeviceState(*(t.clone() for t in (self.rawK, self.rawV, self.c4K, self.c4V,
                                                 self.c128K, self.c128V, self.L)),
                           k_idx=self.k_idx, page_table=self.page_table)


@dataclass
class RoundBuffers:
    parents: torch.Tensor
    draft: torch.Tensor
    target: torch.Tensor
    Q: torch.Tensor
    treeK: torch.Tensor
    treeV: torch.Tensor
    sel: torch.Tensor
    g4: torch.Tensor
    g128: torch.Tensor
    anc: torch.Tensor
    depth: torch.Tensor
    raw_lo: torch.Tensor
    vis4: torch.Tensor
    vis128: torch.Tensor
    scrK4: torch.Tensor
    scrV4: torch.Tensor
    scrK128: torch.Tensor
    scrV128: torch.Tensor
    O: torch.Tensor
    lse: torch.Tensor
    accept_len: torch.Tensor
    path: torch.Tensor
    bonus: torch.Tensor
    committed: torch.Tensor
    status: torch.Tensor
    workspace: torch.Tensor
    q_idx: torch.Tensor = None    # [B][64] bf16 indexer queries (sparse C4 path only)
    idx_ws: torch.Tensor = None   # indexer score workspace
    need: torch.Tensor = None     # [B] int32 positions to reserve per round, 0 for empty slots
                                  # (managed pools only)
    logits: torch.Tensor = None   # [B][D][vocab] the model's logits (scored rounds, alloc_scores)
    logits_lse: torch.Tensor = None     # [B][D] fp32
    entropy: torch.Tensor = None        # [B][D] fp32, nats
    draft_logprobs: torch.Tensor = None  # [B][D] fp32, every draft token under its parent
    top_ids: torch.Tensor = None        # [B][D][n_top] int32
    top_logprobs: torch.Tensor = None   # [B][D][n_top] fp32


def alloc_state(wl, device="cuda"):
    """Persistent cache of the workload on the device: raw rows uploaded, compressed rows zero."""
    dt = wl.torch_dtype
    z = lambda n: torch.zeros((wl.B, max(n, 1), wl.d), dtype=dt, device=device)
    return DeviceState(
        rawK=wl.rawK.to(device), rawV=wl.rawV.to(device),
        c4K=z(wl.cap4 if 4 in wl.ms else 0), c4V=z(wl.cap4 if 4 in wl.ms else 0),
        c128K=z(wl.cap128 if 128 in wl.ms else 0), c128V=z(wl.cap128 if 128 in wl.ms else 0),
        L=torch.as_tensor(wl.L, dtype=torch.int32).to(device),
        k_idx=None if wl.k_idx is None else wl.k_idx.to(device))


def alloc_paged(wl, page_tokens, attn_kernel=_lib.TV_ATTN_AUTO, spare_pages=None, seed=0,
                device="cuda"):
    """Page-based persistent cache ("Adapting Tree-Structured Speculative Decoding to DeepSeek-V4
    for Efficient Inference" §4.2: one logical layer, three physical layers with shared page
    pointers).  Three pools of n_pool_pages pages -- raw K/V (P rows), C4 (P/4 entries), C128
    (P/128 entries) -- and a page table [B][max_pages] mapping each request's logical page to one
    pool page used by all three layers.  The pages of the batch are a seeded random permutation
    of the pool (a fragmented pool), plus ``spare_pages`` unused ones.  Returns (shape, state); the
    raw rows of the workload are copied into their pages, compressed entries start at zero."""
    P = int(page_tokens)
    max_pages = -(-wl.raw_cap // P)
    spare = wl.B if spare_pages is None else int(spare_pages)
    n_pool = wl.B * max_pages + spare
    perm = torch.randperm(n_pool, generator=torch.Generator().manual_seed(seed))
    table = perm[: wl.B * max_pages].reshape(wl.B, max_pages).to(torch.int32)
    dt = wl.torch_dtype
    z = lambda rows: torch.zeros((n_pool, max(rows, 1), wl.d), dtype=dt, device=device)
    rawK, rawV = z(P), z(P)
    for b in range(wl.B):
        for g in range(max_pages):
            lo, hi = g * P, min((g + 1) * P, wl.raw_cap)
            if lo < hi:
                rawK[int(table[b, g]), : hi - lo] = wl.rawK[b, lo:hi].to(device)
                rawV[int(table[b, g]), : hi - lo] = wl.rawV[b, lo:hi].to(device)
    k_idx = None
    if wl.k_idx is not None:   # indexer keys stay contiguous, one row per logical C4 entry
        k_idx = torch.zeros((wl.B, max_pages * P // 4, wl.k_idx.shape[2]), dtype=wl.k_idx.dtype,
                            device=device)
        k_idx[:, : wl.k_idx.shape[1]] = wl.k_idx.to(device)
    st = DeviceState(rawK=rawK, rawV=rawV, c4K=z(P // 4), c4V=z(P // 4), c128K=z(P // 128),
                     c128V=z(P // 128), L=torch.as_tensor(wl.L, dtype=torch.int32).to(device),
                     k_idx=k_idx, page_table=table.to(device))
    shape = shape_for(wl, attn_kernel)
    shape.raw_cap, shape.c4_cap, shape.c128_cap = max_pages * P, max_pages * P // 4, max_pages * P // 128
    shape.page_tokens, shape.max_pages, shape.n_pool_pages = P, max_pages, n_pool
    shape.page_table = st.page_table.data_ptr()
    return shape, st


def alloc_pool(wl, page_tokens, n_pool_pages, attn_kernel=_lib.TV_ATTN_AUTO, stage_chain=0,
               device="cuda"):
    """Page pools whose pages tv_pages_fork, tv_pages_reserve and tv_pages_compact manage (see
    include/treeverify.h): like ``alloc_paged``, but only the pages that the committed prefixes
    cover are mapped (in order, from page 0) and ``page_refs`` counts the holders of every page;
    ``verify_round`` reserves each round's pages.  Returns (shape, state)."""
    P, n_pool = int(page_tokens), int(n_pool_pages)
    max_pages = -(-wl.raw_cap // P)
    table = torch.full((wl.B, max_pages), -1, dtype=torch.int32)
    used = 0
    for b in range(wl.B):
        n = -(-int(wl.L[b]) // P)
        table[b, :n] = torch.arange(used, used + n, dtype=torch.int32)
        used += n
    if used > n_pool:
        raise ValueError(f"the prefixes need {used} pages, the pool has {n_pool}")
    refs = torch.zeros(n_pool, dtype=torch.int32)
    refs[:used] = 1
    dt = wl.torch_dtype
    z = lambda rows: torch.zeros((n_pool, max(rows, 1), wl.d), dtype=dt, device=device)
    rawK, rawV = z(P), z(P)
    for b in range(wl.B):
        L = int(wl.L[b])
        for g in range(-(-L // P)):
            lo, hi = g * P, min((g + 1) * P, L)
            rawK[int(table[b, g]), : hi - lo] = wl.rawK[b, lo:hi].to(device)
            rawV[int(table[b, g]), : hi - lo] = wl.rawV[b, lo:hi].to(device)
    k_idx = None
    if wl.k_idx is not None:
        k_idx = torch.zeros((wl.B, max_pages * P // 4, wl.k_idx.shape[2]), dtype=wl.k_idx.dtype,
                            device=device)
        k_idx[:, : wl.k_idx.shape[1]] = wl.k_idx.to(device)
    st = DeviceState(rawK=rawK, rawV=rawV, c4K=z(P // 4), c4V=z(P // 4), c128K=z(P // 128),
                     c128V=z(P // 128), L=torch.as_tensor(wl.L, dtype=torch.int32).to(device),
                     k_idx=k_idx, page_table=table.to(device), page_refs=refs.to(device))
    shape = shape_for(wl, attn_kernel, stage_chain=stage_chain)
    shape.raw_cap, shape.c4_cap, shape.c128_cap = max_pages * P, max_pages * P // 4, max_pages * P // 128
    shape.page_tokens, shape.max_pages, shape.n_pool_pages = P, max_pages, n_pool
    shape.page_table = st.page_table.data_ptr()
    st.page_ws = torch.empty(_lib.tv_pages_workspace_size(shape), dtype=torch.uint8, device=device)
    return shape, st


def clone_pool(shape, st):
    """A copy of a managed pool that shares nothing with it: (shape, state)."""
    copy = DeviceState(**{f.name: None if getattr(st, f.name) is None else getattr(st, f.name).clone()
                          for f in fields(st)})
    new = _lib.tv_shape.from_buffer_copy(shape)
    new.page_table = copy.page_table.data_ptr()
    return new, copy


def alloc_scores(rb, shape, vocab, n_top=8, dtype=torch.bfloat16, device="cuda"):
    """Adds the buffers of a scored round to ``rb``: the logits, which the caller's model fills
    before the acceptance, and what ``score`` makes of them."""
    B, D = shape.B, shape.D
    f = lambda *s: torch.zeros(s, dtype=torch.float32, device=device)
    rb.logits = torch.zeros((B, D, vocab), dtype=dtype, device=device)
    rb.logits_lse, rb.entropy, rb.draft_logprobs = f(B, D), f(B, D), f(B, D)
    rb.top_ids = torch.zeros((B, D, n_top), dtype=torch.int32, device=device)
    rb.top_logprobs = f(B, D, n_top)


def alloc_round(wl, shape, device="cuda"):
    dt = wl.torch_dtype
    B, D, H, d = wl.B, wl.D, wl.H, wl.d
    i32 = dict(dtype=torch.int32, device=device)
    i64 = dict(dtype=torch.int64, device=device)
    ws = _lib.tv_workspace_size(shape)
    g4 = wl.g[4].to(device) if 4 in wl.g else torch.zeros(d, device=device)
    g128 = wl.g[128].to(device) if 128 in wl.g else torch.zeros(d, device=device)
    sel = torch.as_tensor(wl.sel, dtype=torch.int32).to(device) if wl.sel is not None else None
    return RoundBuffers(
        parents=torch.as_tensor(wl.parents, dtype=torch.int32).to(device),
        draft=torch.as_tensor(wl.draft, dtype=torch.int32).to(device),
        target=torch.as_tensor(wl.target, dtype=torch.int32).to(device),
        Q=wl.Q.to(device), treeK=wl.treeK.to(device), treeV=wl.treeV.to(device), sel=sel,
        g4=g4, g128=g128,
        anc=torch.zeros((B, D), **i64), depth=torch.zeros((B, D), **i32),
        raw_lo=torch.zeros((B, D), **i32), vis4=torch.zeros((B, D), **i64),
        vis128=torch.zeros((B, D), **i64),
        scrK4=torch.zeros((B, D, d), dtype=dt, device=device),
        scrV4=torch.zeros((B, D, d), dtype=dt, device=device),
        scrK128=torch.zeros((B, D, d), dtype=dt, device=device),
        scrV128=torch.zeros((B, D, d), dtype=dt, device=device),
        O=torch.zeros((B, D, H, d), dtype=dt, device=device),
        lse=torch.zeros((B, D, H), dtype=torch.float32, device=device),
        accept_len=torch.zeros(B, **i32), path=torch.zeros((B, D), **i32),
        bonus=torch.zeros(B, **i32), committed=torch.zeros((B, D), **i32),
        status=torch.zeros(1, **i32),
        workspace=torch.empty(max(ws, 256), dtype=torch.uint8, device=device),
        q_idx=None if wl.q_idx is None else wl.q_idx.to(device),
        idx_ws=None if wl.q_idx is None else torch.empty(
            max(_lib.tv_indexer_workspace_size(shape), 256), dtype=torch.uint8, device=device),
        need=torch.full((B,), D, **i32) if shape.page_tokens else None)


def prefill(shape, st, rb, stream=None):
    _lib.tv_prefill_compress(shape, st.rawK, st.rawV, st.L, rb.g4, rb.g128, st.c4K, st.c4V,
                             st.c128K, st.c128V, rb.status, stream)


def indexer(shape, st, rb, stream=None):
    """Device selection of the n_sel C4 entries per request into ``rb.sel`` (sparse path)."""
    _lib.tv_indexer_topk(shape, 64, rb.q_idx, st.k_idx, st.L, rb.sel, rb.idx_ws, rb.status, stream)


def plan(shape, st, rb, stream=None):
    _lib.tv_build_ancestor_mask(shape, rb.parents, st.L, rb.anc, rb.depth, rb.raw_lo, rb.vis4,
                                rb.vis128, rb.status, stream)


def branch_compress(shape, st, rb, stream=None):
    _lib.tv_branch_compress(shape, st.rawK, st.rawV, st.c4K, st.c4V, st.L, rb.treeK, rb.treeV,
                            rb.parents, rb.g4, rb.g128, rb.scrK4, rb.scrV4, rb.scrK128, rb.scrV128,
                            rb.status, stream)


def attention(shape, st, rb, scale=None, stream=None):
    if scale is None:
        scale = 1.0 / math.sqrt(shape.d)
    _lib.tv_tree_verify_attn(shape, rb.Q, st.c4K, st.c4V, rb.sel, st.c128K, st.c128V, st.rawK,
                             st.rawV, st.L, rb.treeK, rb.treeV, rb.anc, rb.raw_lo, rb.vis4,
                             rb.vis128, rb.scrK4, rb.scrV4, rb.scrK128, rb.scrV128, scale, rb.O,
                             rb.lse, rb.workspace, rb.status, stream)


def accept(shape, st, rb, stream=None):
    _lib.tv_accept_walk(shape, rb.parents, rb.draft, rb.target, rb.accept_len, rb.path, rb.bonus,
                        rb.status, stream)


def refresh(shape, st, rb, stream=None):
    _lib.tv_refresh_commit(shape, rb.parents, rb.accept_len, rb.path, rb.treeK, rb.treeV,
                           rb.scrK4, rb.scrV4, rb.scrK128, rb.scrV128, st.rawK, st.rawV, st.c4K,
                           st.c4V, st.c128K, st.c128V, st.L, rb.committed, rb.status, stream)


def score(shape, rb, inv_temperature=1.0, stream=None):
    """From ``rb.logits`` to the round's target tokens, the alternatives of every node, the draft
    tokens' log probabilities under their parents, and the entropies."""
    _lib.tv_token_logprobs(shape, rb.logits, rb.draft, rb.parents, inv_temperature, rb.logits_lse,
                           rb.entropy, rb.draft_logprobs, rb.top_ids, rb.top_logprobs, rb.target,
                           rb.status, stream)


def reserve(shape, st, rb, need=None, stream=None):
    """Pages for the next ``need`` positions of every request (default: ``rb.need``, the round's D
    until the caller fills in less: the depth of a request's tree plus 1 is enough, and 0 keeps an
    empty slot empty)."""
    _lib.tv_pages_reserve(shape, rb.need if need is None else need, st.L, st.page_refs, st.page_ws,
                          rb.status, stream)


def fork(shape, st, rb, source, keep=None, stream=None):
    """Releases, truncates and branches the slots of a managed pool: ``source[b]`` is b (stays), -1
    (released) or the slot that b becomes a copy of; ``keep`` truncates (see tv_pages_fork).  Rounds
    pass over a released slot once ``rb.need[b]`` is 0; else the next one starts a request on it."""
    _lib.tv_pages_fork(shape, source, keep, st.L, st.page_refs, st.rawK, st.rawV, st.c4K, st.c4V,
                       st.c128K, st.c128V, st.k_idx, st.page_ws, rb.status, stream)


def compact(shape, st, rb, remap, n_live, stream=None):
    """Moves the live pages of a managed pool into its ``n_live`` lowest pages."""
    _lib.tv_pages_compact(shape, st.L, st.page_refs, st.rawK, st.rawV, st.c4K, st.c4V, st.c128K,
                          st.c128V, remap, n_live, st.page_ws, rb.status, stream)


def append(shape, st, rb, starts, K, V, Q=None, rope_dim=0, rope_pairs=_lib.TV_ROPE_HALVES,
           inv_freq=None, Qr=None, stream=None):
    """New tokens behind the committed ones of every request: rows ``starts[b]`` to ``starts[b + 1]`` of
    ``K`` and ``V`` [n][d] (see tv_chunk_append).  Their positions need pages on a managed pool
    (``reserve``).  Rotates the queries ``Q`` [n][H][d] into ``Qr`` (default: in place)."""
    _lib.tv_chunk_append(shape, starts, K, V, Q, rope_dim, rope_pairs, inv_freq, rb.g4, rb.g128,
                         Q if Qr is None else Qr, st.rawK, st.rawV, st.c4K, st.c4V, st.c128K,
                         st.c128V, st.L, rb.status, stream)


def alloc_chunk(shape, n_new, device="cuda"):
    """Workspace of ``chunk_attention`` for up to ``n_new`` new tokens."""
    return torch.empty(max(_lib.tv_chunk_workspace_size(shape, n_new), 256), dtype=torch.uint8,
                       device=device)


def chunk_attention(shape, st, rb, starts, Q, workspace, O=None, lse=None, scale=None, stream=None):
    """Attention of the tokens that ``append`` just added, rows as there; returns (O, lse)."""
    O = torch.empty_like(Q) if O is None else O
    lse = torch.empty(Q.shape[:2], dtype=torch.float32, device=Q.device) if lse is None else lse
    _lib.tv_chunk_attn(shape, starts, Q, st.c4K, st.c4V, st.c128K, st.c128V, st.rawK, st.rawV, st.L,
                       1.0 / math.sqrt(shape.d) if scale is None else scale, O, lse, workspace,
                       rb.status, stream)
    return O, lse


@dataclass
class Beams:
    """Beam search over a managed pool: ``width`` neighbouring slots are one group.  ``scores`` starts
    as 0 in a group's first slot and -inf in the others (they become copies of it); -inf in all of a
    group's slots releases them in the next step."""
    width: int
    eos: int
    scores: torch.Tensor      # [B] fp32
    done: torch.Tensor        # [B] int32
    source: torch.Tensor      # [B] int32, what tv_pages_fork takes
    token: torch.Tensor       # [B] int32, the tokens to append next
    rank: torch.Tensor        # [B] int32
    workspace: torch.Tensor
    last_scores: torch.Tensor = None   # [B] fp32, [B] int32: scores and done in front of the last step
    last_done: torch.Tensor = None

    def __post_init__(self):
        if self.last_scores is None:
            self.last_scores, self.last_done = self.scores.clone(), self.done.clone()


def alloc_beams(shape, width, eos, device="cuda"):
    """Buffers of a search with ``width`` beams per group; ``width`` divides the shape's B."""
    size = _lib.tv_beam_workspace_size(shape, width)
    if size == 0 and shape.B > 0:
        raise ValueError(_lib.load().tv_last_error_string().decode())
    i = lambda: torch.zeros(shape.B, dtype=torch.int32, device=device)
    scores = torch.full((shape.B,), -math.inf, dtype=torch.float32, device=device)
    scores[::width] = 0.0
    ws = torch.empty(max(size, 256), dtype=torch.uint8, device=device)
    return Beams(width=width, eos=eos, scores=scores, done=i(), source=i(), token=i(), rank=i(),
                 workspace=ws)


def beam_step(shape, st, rb, beams, logits, scale=1.0, stream=None):
    """Selects the groups' best continuations from ``logits`` [B][vocab] (the rows of done and empty
    slots do not count) and reorders the pool's pages by them: slot b then holds the cache of the
    beam that ``beams.token[b]`` continues.  If the pool runs out of pages (``rb.status``:
    TV_ERR_CAPACITY), no slot changes, and ``beam_undo`` makes ``beams`` match them again."""
    _copy(((beams.last_scores, beams.scores), (beams.last_done, beams.done)), stream)
    _lib.tv_beam_select(shape, beams.width, logits, beams.scores, beams.done, beams.eos, scale,
                        beams.source, beams.token, beams.scores, beams.done, beams.rank,
                        beams.workspace, rb.status, stream)
    fork(shape, st, rb, beams.source, None, stream)


def beam_undo(beams, stream=None):
    """Takes back what the last ``beam_step`` made of ``beams.scores`` and ``beams.done``, so that it can be
    repeated with the same logits once pages are free."""
    _copy(((beams.scores, beams.last_scores), (beams.done, beams.last_done)), stream)


def _copy(pairs, stream):
    with torch.cuda.stream(stream):     # (None: the current one)
        for to, source in pairs:
            to.copy_(source)


def verify_round(shape, st, rb, scale=None, stream=None, commit=True, select=False, scored=False,
                 inv_temperature=1.0):
    """One target-verify round: plan, scratch pad, attention, acceptance, refresh; with
    ``select`` the indexer first picks the sparse path's C4 entries on the device, with ``scored``
    the target tokens come from ``rb.logits`` (else the caller has filled ``rb.target``), the log
    probabilities and entropies at ``inv_temperature``.  On a managed pool the round's pages are
    reserved first (``rb.need``)."""
    if st.page_refs is not None:
        reserve(shape, st, rb, None, stream)
    if select:
        indexer(shape, st, rb, stream)
    plan(shape, st, rb, stream)
    branch_compress(shape, st, rb, stream)
    attention(shape, st, rb, scale, stream)
    if scored:
        score(shape, rb, inv_temperature, stream)
    accept(shape, st, rb, stream)
    if commit:
        refresh(shape, st, rb, stream)


def draft_decode(shape, st, rb, scale=None, stream=None):
    """Draft-side tree attention ("Adapting Tree-Structured Speculative Decoding to DeepSeek-V4 for
    Efficient Inference" §4.1, draft decode): every candidate of the draft tree built so far
    attends to the prefix and its own ancestors, with the scratch pad isolating blocks closed
    inside the tree -- the verify round's plan, scratch-pad and attention calls on the draft
    step's tree, without acceptance or commit (nothing is accepted until the target verifies)."""
    if st.page_refs is not None:
        reserve(shape, st, rb, None, stream)
    plan(shape, st, rb, stream)
    branch_compress(shape, st, rb, stream)
    attention(shape, st, rb, scale, stream)


class RoundGraph:
    """One verify round captured as a CUDA graph on fixed buffers.

    "Adapting Tree-Structured Speculative Decoding to DeepSeek-V4 for Efficient Inference" §4.3
    replays the verification step as a CUDA graph sized for the tree configuration; here the five
    calls (and an optional ``prologue`` of stream work, e.g. refilling inputs) are captured once
    and ``replay()`` relaunches them with a single graph launch.  Construction runs one round
    without its commit (outputs and scratch pad are overwritten, the persistent state is not; the
    pages that this round takes from a managed pool, and what it reports about them, are taken back).
    The buffers in ``st`` / ``rb`` must stay allocated and at the same addresses; their contents
    may change between replays.
    """

    def __init__(self, shape, st, rb, scale=None, commit=True, prologue=None, select=False,
                 scored=False, inv_temperature=1.0):
        # one eager round first, without the commit (the persistent state is left as it was):
        # the library's once-per-device set-up happens outside the capture
        kept = [st.page_table, st.page_refs, rb.status] if st.page_refs is not None else []
        before = [t.clone() for t in kept]
        verify_round(shape, st, rb, scale, None, False, select, scored, inv_temperature)
        for t, was in zip(kept, before):
            t.copy_(was)
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            stream = torch.cuda.current_stream()
            if prologue is not None:
                prologue()
            verify_round(shape, st, rb, scale, stream, commit, select, scored, inv_temperature)

    def replay(self):
        self.graph.replay()

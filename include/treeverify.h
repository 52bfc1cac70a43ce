/*
 * treeverify.h -- C ABI of libtreeverify.so: the target-verify hot path of tree-structured
 * speculative decoding over online-compressed (C4 / C128) attention, for NVIDIA GB300 (sm_103a).
 *
 * Source of the method: "Adapting Tree-Structured Speculative Decoding to DeepSeek-V4 for
 * Efficient Inference" (arXiv 2609.24698), cited as [TSD-V4] with inferred section numbers
 * (§2.2 CSA/HCA compression, §3.1 branch-aware causality, §3.2 isolation, §4.1 three-stage
 * forward and verification plan, §4.2 scratch pad and refresh, §4.3 optimisations, §5.1 naming).
 *
 * One verify round is five calls on one stream, with no host synchronisation in between:
 *   tv_build_ancestor_mask -> tv_branch_compress -> tv_tree_verify_attn -> tv_accept_walk
 *   -> tv_refresh_commit
 * plus tv_prefill_compress, which builds the persistent compressed prefix of a fresh batch.
 *
 * Conventions shared by every call
 * --------------------------------
 * - Every pointer argument is a DEVICE pointer owned by the caller (unless stated otherwise).
 *   The library allocates nothing; scratch space for the attention is the caller's workspace.
 * - Every call is asynchronous on the cudaStream_t it is given (0 = legacy default stream) and
 *   returns TV_OK once its kernels are enqueued, or a negative TV_ERR_* code, without launching
 *   anything, when the host-side arguments are invalid (null pointer, bad shape).  The reason of
 *   the last host-side error of the calling thread is available from tv_last_error_string().
 * - Stream order holds as for ordinary launches.  Inside the library, kernels are launched as
 *   programmatic dependents of the kernel before them and start early only after one of this
 *   library's own kernels that allows it; each waits before it reads that kernel's results or
 *   writes anything, and before it completes.  A caller's kernel placed just before a call and
 *   itself allowing early starts (griddepcontrol.launch_dependents) must not write the call's
 *   inputs after that point.
 *   Two calls read ahead of the call in front on contiguous caches: tv_branch_compress (L, parents,
 *   treeK / treeV, raw rows) and tv_tree_verify_attn (L, Q, compressed entries, raw rows).  As in the
 *   round's order, tv_build_ancestor_mask must come between the former and whatever last wrote what
 *   it reads, and tv_branch_compress between the latter and the same.  With pages nothing is read
 *   ahead, and no other call reads ahead.
 * - Errors found on the device (a malformed tree, a capacity overflow, a bad selection index,
 *   a wait that ran out) are written to the caller's int32 *status word with first-error-wins
 *   semantics (the word is only ever changed from 0 to a negative code); read it after the
 *   stream has been synchronised.  The affected request's outputs are then unspecified, the
 *   other requests' outputs are valid.  Kernels never trap and every wait is bounded.
 * - Tree: node 0 is the root, the last accepted token, whose K/V and query are produced in this
 *   pass; parents[b][0] == -1 and 0 <= parents[b][v] < v (topological numbering); D counts the
 *   root ([TSD-V4] §5.1: s4_k1_d5 verifies 4 draft tokens plus the root with budget 5).
 *   Node v of request b sits at position L[b] + depth[b][v].
 * - Persistent state of request b (row-major, row length d elements, dtype of the shape):
 *     rawK/rawV  [B][raw_cap][d]   raw per-token K/V, rows 0 .. L[b]-1 committed
 *     c4K/c4V    [B][c4_cap][d]    C4 entries, rows 0 .. L[b]/4 - 1 valid
 *     c128K/V    [B][c128_cap][d]  C128 entries, rows 0 .. L[b]/128 - 1 valid
 *     L          [B] int32         committed length
 *   The number of valid compressed entries is always floor(L / m): there is no separate count.
 *   Rows beyond the valid ones are never read for their values but may be loaded; they must hold
 *   finite numbers (allocate the buffers zero-filled).
 * - Scratch pad ([TSD-V4] §4.2): scrK4/scrV4 and scrK128/scrV128 [B][D][d], one row per tree
 *   node; row v holds the compressed entry of the block that node v's token closes, or zeros.
 *   It is separate from the persistent state, which only tv_refresh_commit writes (with
 *   tv_shape.stage_chain, tv_branch_compress also stages rows past the committed length, which no
 *   call reads before tv_refresh_commit has made them part of the state).
 * - Compressor m (4 = C4, 128 = C128): block j covers positions m*j .. m*j+m-1; gate logit of
 *   token t is z_t = K_t . g_m (no scale); w = softmax(z) over the block; the entry is
 *   (sum_t w_t K_t, sum_t w_t V_t), computed in fp32 and stored in the cache dtype (round to
 *   nearest even).  [TSD-V4] §2.2 gives no formula; this gated block sum is the fixed stand-in.
 * - Visibility ([TSD-V4] §3.1, §3.2): a query at position p sees compressed entry (m, j) iff
 *   m*j+m-1 <= p-1, and raw tokens at positions raw_lo(p) .. p; a tree node sees only its own
 *   ancestors (and itself) among the tree tokens and only its proper ancestors' scratch entries.
 *   raw_lo(p) = max(0, p - W) (TV_TAIL_WINDOW) or m_min * floor(p / m_min) (TV_TAIL_REMAINDER,
 *   m_min = 4 if C4 is active, else 128).
 */
#ifndef TREEVERIFY_H
#define TREEVERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* tv_stream_t; /* the same handle type as cudaStream_t */

/* status codes */
#define TV_OK 0
#define TV_ERR_ARG (-1)        /* null pointer, unknown enum value or inconsistent argument */
#define TV_ERR_SHAPE (-2)      /* unsupported shape (D > 64, d not a multiple of 8, ...) */
#define TV_ERR_BAD_TREE (-3)   /* parents[b][0] != -1 or parents[b][v] not in [0, v) */
#define TV_ERR_CAPACITY (-4)   /* a length or entry count exceeds the buffer capacity */
#define TV_ERR_DTYPE (-5)      /* dtype not supported by the requested kernel */
#define TV_ERR_CUDA (-6)       /* a CUDA runtime call failed (launch, tensor-map encoding) */
#define TV_ERR_WORKSPACE (-7)  /* workspace too small (see tv_workspace_size) */
#define TV_ERR_TIMEOUT (-8)    /* a bounded device-side wait ran out (kernel returned early) */
#define TV_ERR_SELECTION (-9)  /* a selection index is outside the request's C4 entries */
#define TV_ERR_BOUNDS (-10)    /* bounds-checked build only: a global index failed its range
                                  check (the access was skipped; the site is printed once) */
#define TV_ERR_VALUE (-11)     /* a NaN or +inf among the logits of a row */

/* tv_shape.tail_mode */
#define TV_TAIL_WINDOW 0
#define TV_TAIL_REMAINDER 1
/* tv_shape.comp_mask bits */
#define TV_COMP_C4 1
#define TV_COMP_C128 2
/* tv_shape.dtype */
#define TV_F32 0
#define TV_BF16 1
/* tv_shape.attn_kernel */
#define TV_ATTN_AUTO 0    /* tensor-core kernel where supported, else the SIMT kernel */
#define TV_ATTN_SIMT 1    /* CUDA-core fp32 kernel: any supported shape, fp32 or bf16 */
#define TV_ATTN_TCGEN05 2 /* tcgen05 tensor-core kernels: bf16; trees d == 512, chunks d % 128 == 0 */
/* rope_pairs of tv_chunk_append */
#define TV_ROPE_HALVES 0
#define TV_ROPE_PAIRS 1

typedef struct tv_shape {
  int32_t B;           /* requests (>= 0; B == 0 turns every call into a no-op) */
  int32_t D;           /* tree nodes per request including the root, 1..64 */
  int32_t H;           /* query heads sharing the single K/V head, 1..1024 */
  int32_t d;           /* head dimension of Q, K, V and O: multiple of 8, 8..512 */
  int32_t W;           /* raw window for TV_TAIL_WINDOW, 0..1024 (ignored otherwise) */
  int32_t tail_mode;   /* TV_TAIL_WINDOW | TV_TAIL_REMAINDER */
  int32_t comp_mask;   /* non-empty subset of TV_COMP_C4 | TV_COMP_C128 */
  int32_t dtype;       /* TV_F32 | TV_BF16: storage of Q, K, V, O, raw and compressed rows */
  int32_t n_sel;       /* 0: all persistent C4 entries visible; > 0: only the n_sel listed ones */
  int32_t attn_kernel; /* TV_ATTN_* */
  int64_t raw_cap;     /* rows per request of rawK / rawV */
  int64_t c4_cap;      /* rows per request of c4K / c4V (ignored without C4) */
  int64_t c128_cap;    /* rows per request of c128K / c128V (ignored without C128) */
  /* Page-based persistent cache ([TSD-V4] §4.2: one logical layer over three physical layers
   * with shared page pointers).  page_tokens == 0: rawK/rawV, c4K/c4V, c128K/c128V are
   * contiguous [B][cap][d] arrays.  page_tokens == P > 0 (a multiple of 512): they are page pools
   * of n_pool_pages pages -- rawK [n_pool_pages][P][d], c4K [n_pool_pages][P/4][d],
   * c128K [n_pool_pages][P/128][d] (V alike) -- and logical page g of request b (tokens
   * g*P .. g*P+P-1, with their C4 and C128 entries) lives in page page_table[b][g] of all three;
   * raw_cap, c4_cap and c128_cap must then be max_pages * P, * P/4 and * P/128.  A page id outside
   * 0 .. n_pool_pages-1 that a call needs is reported as TV_ERR_ARG on the device (page 0 is read
   * instead, and nothing is written). */
  int32_t page_tokens;
  int32_t max_pages;           /* logical pages per request (columns of page_table) */
  int32_t n_pool_pages;        /* pages in each pool */
  /* Refresh skip ([TSD-V4] §4.3: the refresh can be skipped when there is a single candidate
   * chain or the accepted chain is the latest cached one) and the two refresh schedules of §4.2
   * (C4 promptly, C128 delayed until the accepted path is known).  0: off.  1: tv_branch_compress
   * writes the round's cached chain -- the root, its lowest-numbered child, that node's
   * lowest-numbered child, ... -- into the persistent raw rows L[b] + depth and the C4 entries
   * those positions close (rows and entries past the committed length: invisible to every call
   * until tv_refresh_commit advances L), and tv_refresh_commit copies only the accepted nodes off
   * that chain and the accepted C128 entries.  A single-chain tree then commits by advancing L. */
  int32_t stage_chain;
  const int32_t* page_table;   /* device [B][max_pages] int32 (page_tokens > 0 only); -1: no page.
                                  tv_pages_fork, _reserve and _compact write it, the other calls
                                  read the entries of the positions they touch */
} tv_shape;

/* Library version string (static storage). */
const char* tv_version(void);

/* Human-readable name of a TV_* status code (static storage). */
const char* tv_status_string(int code);

/* Description of the calling thread's last host-side error (thread-local storage, valid until
 * the thread's next call into the library). */
const char* tv_last_error_string(void);

/* Bytes of device workspace tv_tree_verify_attn needs for this shape (0 for B == 0).  The
 * workspace holds the split-KV partial results and the work counters; the caller allocates it
 * (any 256-byte-aligned device buffer) and may reuse it across calls on the same stream. */
size_t tv_workspace_size(const tv_shape* shape);

/* The attention kernel tv_tree_verify_attn runs for this shape on the current device:
 * TV_ATTN_SIMT or TV_ATTN_TCGEN05, or a negative TV_ERR_* code for an invalid shape. */
int tv_attn_kernel_for(const tv_shape* shape);

/*
 * Verify preprocess: the verification plan ([TSD-V4] §4.1 -- the candidate tree becomes the
 * metadata that guides attention and compression; §4.3 -- built on the device).
 *   parents  [B][D] int32   in   tree topology
 *   L        [B]    int32   in   committed lengths
 *   anc      [B][D] uint64  out  bit u of anc[b][v] set iff u is on the path root -> v
 *   depth    [B][D] int32   out  depth of v (root 0); position = L[b] + depth
 *   raw_lo   [B][D] int32   out  lowest raw position visible from v (see raw_lo(p) above)
 *   scr_vis4 [B][D] uint64  out  proper ancestors of v whose token closes a C4 block
 *                                 (nullable when C4 is inactive)
 *   scr_vis128 [B][D] uint64 out same for C128 (nullable when C128 is inactive)
 * Device errors: TV_ERR_BAD_TREE (that request's outputs are zero), TV_ERR_ARG for L < 0.
 */
int tv_build_ancestor_mask(const tv_shape* shape, const int32_t* parents, const int32_t* L,
                           uint64_t* anc, int32_t* depth, int32_t* raw_lo, uint64_t* scr_vis4,
                           uint64_t* scr_vis128, int32_t* status, tv_stream_t stream);

/*
 * Prefill compression ([TSD-V4] §2.2): writes every complete block of each request's committed
 * prefix, entries 0 .. floor(L[b]/m) - 1 of each active compressor, from the raw rows.
 *   rawK, rawV [B][raw_cap][d] in; L [B] in; g4, g128 [d] fp32 gate vectors (nullable when the
 *   compressor is inactive); c4K, c4V, c128K, c128V out.
 * Device errors: TV_ERR_CAPACITY when L > raw_cap or floor(L/m) > cap_m (request skipped).
 */
int tv_prefill_compress(const tv_shape* shape, const void* rawK, const void* rawV,
                        const int32_t* L, const float* g4, const float* g128, void* c4K,
                        void* c4V, void* c128K, void* c128V, int32_t* status,
                        tv_stream_t stream);

/*
 * Scratch-pad branch compression ([TSD-V4] §3.2, §4.1, §4.2: a chain that closes a block after
 * branching is compressed on its own, into temporary storage).  For every node v and active
 * compressor m with (L[b] + depth(v) + 1) % m == 0, row v of the m scratch pad becomes the gated
 * sum of the m positions ending at v's position, read from the sequence prefix + path(v):
 * positions < L[b] from rawK/rawV, the others from treeK/treeV of v's ancestors.  Every other
 * row is set to zero.
 * With shape->stage_chain == 1 it also stages the cached chain (see tv_shape): for every node c
 * of that chain, rawK/rawV row L[b] + depth(c) <- treeK/treeV row c, and when c closes a C4
 * block, C4 entry (L[b] + depth(c) + 1)/4 - 1 <- c's C4 scratch row; positions or entries past
 * raw_cap / c4_cap are not staged.  Nothing at or below L[b] - 1 and no C128 entry is written.
 *   rawK, rawV [B][raw_cap][d] in (and out past L[b] when staging); L [B] in; treeK, treeV
 *   [B][D][d] in (K/V of the tree tokens); parents [B][D] in; g4, g128 [d] fp32 in;
 *   scrK4, scrV4, scrK128, scrV128 [B][D][d] out (the pair of an inactive compressor is
 *   nullable); c4K, c4V [B][c4_cap][d] out past L[b]/4 when staging with C4 active (else
 *   nullable).
 * Device errors: TV_ERR_BAD_TREE, TV_ERR_CAPACITY (L > raw_cap).
 */
int tv_branch_compress(const tv_shape* shape, void* rawK, void* rawV, void* c4K, void* c4V,
                       const int32_t* L, const void* treeK, const void* treeV,
                       const int32_t* parents, const float* g4, const float* g128, void* scrK4,
                       void* scrV4, void* scrK128, void* scrV128, int32_t* status,
                       tv_stream_t stream);

/*
 * Branch-aware causal tree-verify attention ([TSD-V4] §3.1, §4.1, §4.4), split-KV.
 * Every (node v, head h) row attends, with logit scale `scale` (normally 1/sqrt(d)), to
 *   - the persistent C4 entries 0 .. L/4-1 (or, with n_sel > 0, the listed ones sel[b][i]),
 *   - the persistent C128 entries 0 .. L/128-1,
 *   - the raw rows at positions raw_lo[b][v] .. L-1,
 *   - the tree tokens u with anc bit u set and position L + depth(u) >= raw_lo[b][v],
 *   - the scratch entries of the nodes flagged in scr_vis4 / scr_vis128.
 * The compressed prefix is read once per request and shared by all D*H rows.
 *   Q    [B][D][H][d] in (dtype);  sel [B][n_sel] int32 (nullable when n_sel == 0)
 *   anc, raw_lo, scr_vis4, scr_vis128: the plan of tv_build_ancestor_mask
 *   O    [B][D][H][d] out (dtype); lse [B][D][H] fp32 out: natural-log sum of exp(logits)
 *   (Q and O 16-byte aligned)
 *   workspace: device buffer of ws_bytes >= tv_workspace_size(shape)
 * Host errors: TV_ERR_ARG (also a misaligned Q or O), TV_ERR_WORKSPACE, TV_ERR_DTYPE
 * (TV_ATTN_TCGEN05 asked for an unsupported shape).
 * Device errors: TV_ERR_SELECTION, TV_ERR_CAPACITY, TV_ERR_TIMEOUT.
 */
int tv_tree_verify_attn(const tv_shape* shape, const void* Q, const void* c4K, const void* c4V,
                        const int32_t* sel, const void* c128K, const void* c128V,
                        const void* rawK, const void* rawV, const int32_t* L,
                        const void* treeK, const void* treeV, const uint64_t* anc,
                        const int32_t* raw_lo, const uint64_t* scr_vis4,
                        const uint64_t* scr_vis128, const void* scrK4, const void* scrV4,
                        const void* scrK128, const void* scrV128, float scale, void* O,
                        float* lse, void* workspace, size_t ws_bytes, int32_t* status,
                        tv_stream_t stream);

/*
 * tv_tree_verify_attn without a workspace argument, for callers that cannot allocate device
 * memory (an engine that reserved all free memory for its own page pool, a decode loop that must
 * not pay cudaMalloc's implicit synchronisation, a plug-in host without an allocator).  The report
 * has no counterpart: this is a convenience of the library.  Same arguments, semantics and
 * outputs as tv_tree_verify_attn, minus workspace / ws_bytes.  The split-KV partial results live
 * in a 32 MiB array inside the library image, held by every GPU that loads the library's device
 * code until the process exits; a shape whose tv_workspace_size exceeds it is rejected with
 * TV_ERR_WORKSPACE.  Under CUDA's lazy module loading (the default) the device code, and with it
 * the 32 MiB, is loaded on a device at the first call there that resolves the array: call
 * tv_noalloc_prepare once per device at start-up, before reserving a memory pool and before any
 * stream capture; later calls take no device memory.  The array's address is looked up in the
 * caller's current context on every call.  All calls share the array: calls that overlap on the
 * GPU race on it (its previous contents are never read, nothing needs clearing).  Host errors name
 * tv_tree_verify_attn_noalloc.  It allocates nothing, neither on the device nor through any
 * library.
 */
int tv_tree_verify_attn_noalloc(const tv_shape* shape, const void* Q, const void* c4K,
                                const void* c4V, const int32_t* sel, const void* c128K,
                                const void* c128V, const void* rawK, const void* rawV,
                                const int32_t* L, const void* treeK, const void* treeV,
                                const uint64_t* anc, const int32_t* raw_lo,
                                const uint64_t* scr_vis4, const uint64_t* scr_vis128,
                                const void* scrK4, const void* scrV4, const void* scrK128,
                                const void* scrV128, float scale, void* O, float* lse,
                                int32_t* status, tv_stream_t stream);

/*
 * Loads the library's device code on the current device, with the built-in scratch of
 * tv_tree_verify_attn_noalloc (32 MiB), so that later calls take no device memory.  Call it once
 * per device before handing the free memory to a pool.  Returns TV_OK, or TV_ERR_CUDA if the
 * device code cannot be loaded (for instance when less than 32 MiB is free).
 */
int tv_noalloc_prepare(void);

/*
 * Accepted-path selection ([TSD-V4] §3.2, §4.1): greedy walk from the root; at each node take
 * the lowest-numbered child whose draft token equals the node's target token; stop when none.
 *   parents, draft, target [B][D] int32 in
 *   accept_len [B] out: path length including the root (>= 1)
 *   path [B][D] out: accepted node ids in order, -1 padded
 *   bonus [B] out: target token of the last accepted node
 * Device errors: TV_ERR_BAD_TREE.
 */
int tv_accept_walk(const tv_shape* shape, const int32_t* parents, const int32_t* draft,
                   const int32_t* target, int32_t* accept_len, int32_t* path, int32_t* bonus,
                   int32_t* status, tv_stream_t stream);

/*
 * Accepted-path state refresh ([TSD-V4] §3.2, §4.2: only the accepted path's token, KV and
 * compressed states reach the persistent context; rejected branches are dropped).
 * With n = accept_len[b] and path = path[b]:
 *   rawK/rawV row L+i <- treeK/treeV row path[i] (exact copy), i < n;
 *   for every active m and position e in [L, L+n-1] with (e+1) % m == 0: entry (e+1)/m - 1 <-
 *   scratch row path[e-L] of compressor m (that row is the gated sum of exactly the committed
 *   block, so the copy equals recompressing it); L[b] <- L + n;
 *   committed_pos[b][i] = old L + i for i < n, -1 otherwise.
 * The scratch pad must come from tv_branch_compress of the same round.
 * With shape->stage_chain == 1 the writes tv_branch_compress already staged are skipped: the
 * accepted nodes path[i] that are the i-th node of the cached chain (computed from parents, which
 * must then be given) keep their staged raw row and C4 entry; every other accepted raw row and C4
 * entry, and every C128 entry the accepted path closes, are copied as above.
 *   parents [B][D] in (stage_chain == 1 only, else nullable)
 * Device errors: TV_ERR_CAPACITY (L+n > raw_cap or an entry beyond cap_m; request untouched),
 * TV_ERR_ARG (accept_len outside 1..D, a path id outside 0..D-1 or, with pages, no page for a
 * committed position; request untouched).  An empty slot of a page pool is left alone without an
 * error.
 */
int tv_refresh_commit(const tv_shape* shape, const int32_t* parents, const int32_t* accept_len,
                      const int32_t* path, const void* treeK, const void* treeV, const void* scrK4,
                      const void* scrV4, const void* scrK128, const void* scrV128, void* rawK,
                      void* rawV, void* c4K, void* c4V, void* c128K, void* c128V, int32_t* L,
                      int32_t* committed_pos, int32_t* status, tv_stream_t stream);

/*
 * Indexer top-k selection of the persistent C4 entries for the sparse prefix path ([TSD-V4] §2.2:
 * CSA is compressed *sparse* attention; the report gives no selection rule, so the rule here is
 * the stand-in of the long-context workload).  For every request b with n4 = L[b]/4 C4 entries:
 *   score[j] = q_idx[b] . k_idx[b][j], j < n4, computed in fp32 as products of the bf16 inputs
 *   (exact) added in index order 0 .. d_idx-1, one round-to-nearest-even per addition, no fused
 *   multiply-add;
 *   sel[b] = the n_sel entries of largest score (equal scores: lower j first), ascending in j --
 *   the selection list tv_tree_verify_attn takes.
 * Uses shape->B, c4_cap (rows of k_idx per request), n_sel (> 0) and needs C4 in comp_mask.
 *   d_idx: indexer dimension, a multiple of 8 in 8..256
 *   q_idx [B][d_idx] bf16 in; k_idx [B][c4_cap][d_idx] bf16 in (16-byte aligned); L [B] in
 *   sel [B][n_sel] int32 out
 *   workspace: device buffer of ws_bytes >= tv_indexer_workspace_size(shape) (the fp32 scores)
 * Host errors: TV_ERR_ARG, TV_ERR_SHAPE, TV_ERR_WORKSPACE.
 * Device errors: TV_ERR_SELECTION (n4 < n_sel), TV_ERR_CAPACITY (n4 > c4_cap); that request's
 * sel row is set to -1.
 */
size_t tv_indexer_workspace_size(const tv_shape* shape);
int tv_indexer_topk(const tv_shape* shape, int d_idx, const void* q_idx, const void* k_idx,
                    const int32_t* L, int32_t* sel, void* workspace, size_t ws_bytes,
                    int32_t* status, tv_stream_t stream);

/*
 * From a round's logits to the integers and log probabilities around it: the target tokens that
 * tv_accept_walk takes, the alternatives a draft tree is grown from, the log probabilities of the
 * tokens a tree holds, and the entropy of every node's distribution.  The report leaves the step
 * from logits to target tokens to the model runtime; greedy verification takes the largest logit
 * ([TSD-V4] §3.2).  With x the logits of row (b, v) and p = softmax(scale * x) over the vocabulary:
 *   lse      [B][D] fp32: natural-log sum of exp(scale * x)
 *   entropy  [B][D] fp32: -sum p ln p, in nats
 *   target   [B][D] int32: the token of the largest logit (equal logits: the lower id)
 *   top_ids, top_logprobs [B][D][n_top]: the n_top tokens of largest logit, descending (equal
 *            logits: the lower id first), with ln p; logits of -inf are never listed, places left
 *            over hold -1 and -inf
 *   logprobs [B][n_tok] fp32: ln p(tokens[b][i]) under the distribution of node nodes[b][i]; 0
 *            where the node or the token is negative.  tokens = the draft tokens and nodes =
 *            parents (n_tok = D) scores every draft token under its parent, the root as 0.
 * Sums are kept in fp32 relative to the largest logit.  A logit of -inf is a masked token
 * (probability 0, ln p = -inf).  A row of -inf only has lse = -inf, entropy 0, target -1, no
 * alternatives and ln p = -inf.  The type's lowest finite value is an ordinary logit.  Results beyond
 * fp32's range (that value at scale > 1, say) are -inf or +inf.
 *   Uses shape->B and D (rows = B * D).  vocab 1..2^30; logits [B][D] rows of vocab elements, ld
 *   >= vocab elements apart, of type logits_dtype (TV_F32 | TV_BF16), aligned to that type only.
 *   n_tok 0..1024, tokens and nodes [B][n_tok] int32 in (nullable when n_tok == 0; nodes null:
 *   entry i is on node i, n_tok <= D); scale > 0; n_top 0..32.  lse, entropy and target are
 *   nullable (not wanted), logprobs when n_tok == 0, top_ids and top_logprobs when n_top == 0.
 * Device errors: TV_ERR_VALUE (a NaN or +inf among a row's logits: that row's floats are NaN, its
 * ids -1), TV_ERR_ARG (a node >= D or a token >= vocab: that log probability is 0).
 */
int tv_token_logprobs(const tv_shape* shape, int32_t vocab, int64_t ld, int32_t logits_dtype,
                      const void* logits, int32_t n_tok, const int32_t* tokens,
                      const int32_t* nodes, float scale, int32_t n_top, float* lse, float* entropy,
                      float* logprobs, int32_t* top_ids, float* top_logprobs, int32_t* target,
                      int32_t* status, tv_stream_t stream);

/*
 * Pages of the pools ([TSD-V4] §4.2: one logical layer over three physical layers with shared
 * page pointers; the report keeps their allocation in its serving engine).  For shapes with
 * page_tokens = P > 0.  The state is shape->page_table (entries -1 where no page is mapped), L, and
 *   page_refs [n_pool_pages] int32: holders of every page.  A table entry counts as one; a caller
 *   that holds a page of its own (a cached prefix, say) adds one itself.  0: the page is free.
 * The calls keep one rule: a page that more than one holder has holds only complete, committed
 * tokens of every request that maps it, so no round writes a shared page.  They run on the stream
 * like the others and can be captured; all three leave everything as it was when there are not
 * enough free pages (TV_ERR_CAPACITY).  Pages are taken in the order of the requests and positions
 * that need them, the lowest-numbered free page first, so results do not depend on timing.
 * An empty slot -- L[b] = 0 and no page for its first position (page_table[b][0] = -1), as
 * tv_pages_fork leaves a released one -- takes no part in a round: no call stages, selects or commits
 * anything for it (committed_pos -1) or records an error, as long as its parents are a tree and what
 * tv_token_logprobs is given for it is valid; its other outputs are unspecified.  It stays empty while
 * tv_pages_reserve is given need[b] <= 0 for it; with need[b] > 0 the round starts a request on an
 * empty prefix.
 * workspace: device buffer of ws_bytes >= tv_pages_workspace_size(shape), 256-byte aligned; calls
 * that overlap on the GPU need one each.
 */
size_t tv_pages_workspace_size(const tv_shape* shape);

/*
 * Releases, truncates and branches requests.  Per slot b, from the state before the call:
 *   source[b] == b   the slot stays; with 0 <= keep[b] < L[b] its length becomes keep[b] and the
 *                    pages behind that are released; a partial last page that others hold is
 *                    replaced by a copy
 *   source[b] == -1  the slot is released: its table row becomes -1, L[b] = 0
 *   source[b] == s   the slot's pages are released and it becomes a copy of slot s (source[s] == s
 *                    is required) at the smallest of L[s] and the non-negative ones of keep[s]
 *                    and keep[b]: the full pages are shared, the partial last page is copied
 * Only the rows of valid tokens and entries are copied; a released page is free when nobody else
 * holds it, and may be taken again by the same call.
 *   source [B] in; keep [B] in (nullable: no truncation; negative: none for that slot); L [B] and
 *   page_refs in and out; rawK .. c128V: the pools, in and out (an inactive compressor's are
 *   nullable; 16-byte aligned); k_idx: the indexer keys [B][c4_cap][d_idx] bf16 (nullable; 16-byte
 *   aligned, d_idx a multiple of 8 in 8..256): rows 0 .. L/4 - 1 of a branching slot are copied
 *   from its source's
 * Host errors: TV_ERR_ARG, TV_ERR_SHAPE, TV_ERR_WORKSPACE.
 * Device errors: TV_ERR_ARG (a source out of range, or one that is not a slot that stays, or a
 * page missing among the source's: that slot stays as it was), TV_ERR_CAPACITY (a source's length
 * outside 0 .. raw_cap: that slot stays as it was; not enough free pages: all slots do).
 */
int tv_pages_fork(const tv_shape* shape, const int32_t* source, const int32_t* keep, int32_t* L,
                  int32_t* page_refs, void* rawK, void* rawV, void* c4K, void* c4V, void* c128K,
                  void* c128V, void* k_idx, int32_t d_idx, void* workspace, size_t ws_bytes,
                  int32_t* status, tv_stream_t stream);

/*
 * Maps a page wherever one is missing for the positions L[b] .. L[b] + need[b] - 1 (a round's D
 * tokens, or a prompt to come); need[b] <= 0 leaves the slot alone.
 *   need [B] in; L [B] in; page_refs in and out
 * Device errors: TV_ERR_CAPACITY (L + need > raw_cap: that slot stays as it was; not enough free
 * pages: all slots do), TV_ERR_ARG (L < 0: that slot stays as it was; a table entry outside the
 * pool: that entry stays).
 */
int tv_pages_reserve(const tv_shape* shape, const int32_t* need, const int32_t* L,
                     int32_t* page_refs, void* workspace, size_t ws_bytes, int32_t* status,
                     tv_stream_t stream);

/*
 * Moves the live pages (those somebody holds) into the n_live lowest pages of the pool: the i-th
 * live page at or above n_live takes the i-th free page below it; the others stay.  Table and
 * counts follow; of a page that only table entries hold, the rows of valid tokens are copied, of any
 * other the whole page.
 *   L [B] in; page_refs in and out; rawK .. c128V: the pools, in and out (16-byte aligned); remap
 *   [n_pool_pages] int32 out: the new number of every page that was live, -1 for the others; n_live
 *   [1] int32 out
 * Device errors: TV_ERR_ARG (a table entry outside the pool: it stays; a page with more table
 * entries than holders: it is live all the same).
 */
int tv_pages_compact(const tv_shape* shape, const int32_t* L, int32_t* page_refs, void* rawK,
                     void* rawV, void* c4K, void* c4V, void* c128K, void* c128V, int32_t* remap,
                     int32_t* n_live, void* workspace, size_t ws_bytes, int32_t* status,
                     tv_stream_t stream);

/*
 * New tokens into the cache: a prompt, a part of one, or one token per request, in one ragged batch.
 * The report's rounds extend the cache by accepted tree tokens only ([TSD-V4] §4.2) and leave
 * prompts to the serving engine; the rules here are those of tv_prefill_compress and
 * tv_refresh_commit.  Request b's new tokens are rows starts[b] .. starts[b+1] - 1 of the batch's
 * n_new rows, in order; token i of it goes to position p = L[b] + i:
 *   rawK row p <- K row with its last rope_dim elements rotated by the position: with r = rope_dim
 *   and f = inv_freq, pair i (x, y) becomes (x cos a - y sin a, x sin a + y cos a), a = p * f[i]
 *   radians, i < r/2; the pair is elements (i, i + r/2) of the r (TV_ROPE_HALVES) or (2i, 2i + 1)
 *   (TV_ROPE_PAIRS); rotated in fp32, the angle reduced in fp64, stored in the cache dtype
 *   rawV row p <- V row;  Qr row <- Q row, every head rotated the same way
 *   every block that the new tokens complete gets its C4 / C128 entry, from the rows as they are
 *   stored: bit for bit what tv_prefill_compress writes for the same rows, however the tokens were
 *   split into calls
 *   L[b] <- L[b] + starts[b+1] - starts[b]
 * Uses shape->B, H, d, dtype, comp_mask, the capacities and the paging.
 *   n_new 0..2^30, n_new * H < 2^31; starts [B+1] int32 in, 0 <= starts[0], ascending, starts[B] <=
 *   n_new (rows of no request are left alone); K, V n_new rows of d elements in, ld_kv >= d elements
 *   apart; Q [n_new][H][d] in (nullable, with Qr), Qr [n_new][H][d] out, may be Q: then only the
 *   rotated elements are written; rope_dim even, 0..d (0: no rotation, inv_freq nullable); inv_freq
 *   [rope_dim / 2] fp32 in; g4, g128 [d] fp32 in and c4K .. c128V out (nullable when the compressor
 *   is inactive).  K, V, Q, Qr, the caches and ld_kv's bytes 16-byte aligned.
 * Device errors, each leaving that request as it was (its Qr rows are unspecified): TV_ERR_ARG
 * (starts that leave 0 .. n_new; starts that descend -- others of the batch may then be left as they were
 * too, and all Qr rows are unspecified --; L < 0; no page for a new position), TV_ERR_CAPACITY (L + n >
 * raw_cap or an entry beyond cap_m).
 */
int tv_chunk_append(const tv_shape* shape, int32_t n_new, const int32_t* starts, const void* K,
                    const void* V, int64_t ld_kv, const void* Q, int32_t rope_dim,
                    int32_t rope_pairs, const float* inv_freq, const float* g4, const float* g128,
                    void* Qr, void* rawK, void* rawV, void* c4K, void* c4V, void* c128K,
                    void* c128V, int32_t* L, int32_t* status, tv_stream_t stream);

/*
 * Attention of a chunk of new tokens over the cache that holds them ([TSD-V4] §2.2: compressed
 * attention of ordinary causal decoding; §3.1's visibility for a chain).  Request b's queries are
 * rows starts[b] .. starts[b+1] - 1; they belong to the last n = starts[b+1] - starts[b] positions
 * of its cache, p = L[b] - n + i (call it after tv_chunk_append, which advances L).  Every head of
 * the token at position p attends, with logit scale `scale`, to the C4 entries 0 .. p/4 - 1, the
 * C128 entries 0 .. p/128 - 1 and the raw rows raw_lo(p) .. p: one decode step for n = 1, the same
 * numbers as decoding token by token for any n.
 * Uses shape->B, H, d, W, tail_mode, comp_mask, dtype, attn_kernel, the capacities and the paging;
 * n_sel must be 0 (selection lists belong to rounds).
 *   n_new, starts as in tv_chunk_append; Q [n_new][H][d] in; O [n_new][H][d] out (dtype); lse
 *   [n_new][H] fp32 out: natural-log sum of exp(logits); rows of no request are left alone
 *   Q, O and the caches 16-byte aligned, O apart from Q; the chunk's rows are finite, as all rows of
 *   the caches (a NaN or infinity in a token's row also reaches the tokens in front of it that share
 *   a tile); workspace: device buffer of ws_bytes >=
 *   tv_chunk_workspace_size(shape, n_new), 256-byte aligned (what is enough for n_new tokens is for
 *   fewer); calls that overlap on the GPU need one each.
 * Host errors: TV_ERR_ARG, TV_ERR_SHAPE, TV_ERR_WORKSPACE, TV_ERR_DTYPE (TV_ATTN_TCGEN05 asked for
 * an unsupported shape).
 * Device errors, that request's rows left alone: TV_ERR_ARG (starts that leave 0 .. n_new or, with
 * all outputs unspecified, descend; L < n), TV_ERR_CAPACITY (L > raw_cap or more entries than
 * cap_m); TV_ERR_ARG for a page that is missing (page 0 is read instead); TV_ERR_TIMEOUT.
 */
size_t tv_chunk_workspace_size(const tv_shape* shape, int32_t n_new);
int tv_chunk_attn(const tv_shape* shape, int32_t n_new, const int32_t* starts, const void* Q,
                  const void* c4K, const void* c4V, const void* c128K, const void* c128V,
                  const void* rawK, const void* rawV, const int32_t* L, float scale, void* O,
                  float* lse, void* workspace, size_t ws_bytes, int32_t* status,
                  tv_stream_t stream);

/*
 * Beam search's selection over beams and vocabulary, in the slots that tv_pages_fork reorders the
 * cache by (the report keeps one sequence per request; a draft tree's levels are grown the same
 * way).  The B slots are B / width groups of `width` neighbours, each slot a beam.  With x the logits
 * of slot b and ln p as in tv_token_logprobs, slot b's candidates are its tokens t with x[t] > -inf
 * and score scores[b] + ln p(t); a beam that has ended (done[b] != 0) has one, itself: token eos at
 * score scores[b].  A score of -inf: an empty slot, no candidates.  The `width` best candidates of
 * the group go on (equal scores: the lower slot first, then the lower id; scores are formed and
 * compared in fp64, but the log of a beam's sum over the vocabulary comes from tv_token_logprobs in
 * fp32: of candidates of different beams closer than 2^-18 either may come first): a beam with
 * candidates among them keeps its best in its own slot, the others fill the group's free slots in
 * ascending order, best first.  Per slot:
 *   source [B] int32: the slot it continues (0 .. B-1), -1 if candidates ran out: what tv_pages_fork
 *          takes, which copies and releases the pages; token [B] int32 (-1 without a source);
 *          new_scores [B] fp32 (-inf without a source); new_done [B] int32: 1 if the source had
 *          ended or the token is eos, else 0; rank [B] int32: its place in the group, 0 the best
 *          (-1 without a source)
 *   Uses shape->B and comp_mask..dtype only for validation.  width 1..32 dividing B; vocab, ld,
 *   logits_dtype, logits (one row per slot) and scale as in tv_token_logprobs; scores [B] fp32 in;
 *   done [B] int32 in (nullable: none has ended; eos is then only compared with); new_scores may be
 *   scores and new_done may be done; new_done and rank are nullable.
 *   workspace: device buffer of ws_bytes >= tv_beam_workspace_size(shape, width), 256-byte aligned;
 *   calls that overlap on the GPU need one each.
 * Device errors: TV_ERR_VALUE (a NaN or +inf among the logits of a slot with a score, or such a
 * score: that slot has no candidates).
 */
size_t tv_beam_workspace_size(const tv_shape* shape, int32_t width);
int tv_beam_select(const tv_shape* shape, int32_t width, int32_t vocab, int64_t ld,
                   int32_t logits_dtype, const void* logits, const float* scores,
                   const int32_t* done, int32_t eos, float scale, int32_t* source, int32_t* token,
                   float* new_scores, int32_t* new_done, int32_t* rank, void* workspace,
                   size_t ws_bytes, int32_t* status, tv_stream_t stream);

/*
 * Testing aid for the failure path of the tensor-core attention (the report has no counterpart).
 * Sets, for every later tv_tree_verify_attn or tv_chunk_attn launch of a tcgen05 kernel in this process:
 *   timeout_ns     the bound of every device-side wait (default 2000000000 = 2 s; > 0);
 *   withhold_tile  one KV tile index (within each work item's tile range) whose K copies the
 *                  producers never issue, or -1 for none (the default).
 * With a tile withheld, the MMA issuer's wait for that tile runs out after timeout_ns; the kernel
 * then records TV_ERR_TIMEOUT in the status word, stops every CTA of the affected clusters,
 * drains the copies and MMAs it did issue and returns, leaving the context usable.  Restore
 * (2000000000, -1) afterwards.  Host errors: TV_ERR_ARG (timeout_ns <= 0 or withhold_tile < -1).
 */
int tv_debug_attn_timeout(int64_t timeout_ns, int32_t withhold_tile);

#ifdef __cplusplus
}
#endif

#endif /* TREEVERIFY_H */

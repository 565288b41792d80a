/*
 * pctree.h -- libpctree: draft-tree construction and checking for
 * speculative decoding, on AMD Instinct MI355X (gfx950).
 *
 * Pages the operations come from (cited by title and section):
 *  [PCT] qiita article on PCTree (Parent-Conditioned Drafting Tree),
 *        section "a straight draft is wasted once its first token misses"
 *        (cited below as "straight draft"): DSpark's Markov head
 *        z_d = L_d + Markov(y_{d-1}) and the chain -> tree step.
 *  [DSP] DSpark / DeepSeek-V4 explainer (xiaohu-jiedu), section "one
 *        inference, from guess to confirmation".
 *  [CAD] "Cost-Aware Diffusion Draft Trees for Speculative Decoding"
 *        (CaDDTree) summary on gist.science, section "Method".
 *
 * Conventions shared by every call
 *  - Pointers are DEVICE pointers unless marked (host).  Every call is
 *    asynchronous on `stream` (a hipStream_t passed as void*; NULL = the
 *    default stream) and never synchronises the host.
 *  - The caller owns every buffer, including the workspace, and keeps them
 *    alive until the stream has finished the work.  The library allocates
 *    nothing and keeps no pointer after a call returns.
 *  - Arrays are row-major and contiguous.  Token ids are int32 in [0, V),
 *    V < 2^18.  A parent index of -1 means the root (the anchor token); the
 *    root is not one of the N nodes.
 *  - Masks are uint64 words: bit j%64 of word j/64 of row i is set when node
 *    j is node i or one of its ancestors.
 *  - Every argument is checked on the host before anything is enqueued; a
 *    failed check returns a status and enqueues nothing.  A failed launch
 *    returns PCT_ERR_HIP.  pct_last_error() gives the reason (per thread).
 *    No exception crosses this interface and the library never aborts.
 *  - Logits must be finite.
 *  - Calls are reentrant; calls on different streams need different
 *    workspaces.
 */
#ifndef PCTREE_H
#define PCTREE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PCT_OK = 0,
  PCT_ERR_INVALID_ARG = 1,
  PCT_ERR_UNSUPPORTED = 2,
  PCT_ERR_WORKSPACE = 3,
  PCT_ERR_HIP = 4
} pct_status;

/* PCT_F16 is an element type of key-value caches only. */
typedef enum { PCT_F32 = 0, PCT_BF16 = 1, PCT_F16 = 2 } pct_dtype;

/* Shape of a parent-conditioned build.
 *  batch   independent requests
 *  B       drafted positions per block (tree depth <= B)
 *  V       vocabulary size
 *  r       rank of the Markov factors (ignored when U and W are NULL)
 *  k       children kept per parent (local top-k)
 *  beam_w  parents expanded per depth and request (per-stage pruning)
 *  N       verify budget: nodes kept per request (global top-N)
 *  uw_dtype  element type of U and W */
typedef struct {
  int32_t batch, B, V, r, k, beam_w, N;
  int32_t uw_dtype;
} pct_tree_shape;

/* Round cost of the adaptive build: C(n; l) = C_d + C_v(n; l) with
 * C_v(n; l) = c0 + c1 n + c2 n^2 + c_ell l n (convex and increasing in n
 * when c1, c2, c_ell >= 0). */
typedef struct {
  double C_d, c0, c1, c2, c_ell;
} pct_cost_model;

/* ------------------------------------------------------------------------
 * pct_markov_logits -- [PCT] "straight draft": for P parents
 * at once, z_p = L[row_p] + Markov(tok_p) with Markov(t)[v] = U[t] . W[v],
 * then the log-softmax normaliser of z_p over the vocabulary and its top-k.
 *
 *  L          [L_rows][L_row_stride] fp32 drafter logits; NULL => z = Markov
 *             (row indices outside [0, L_rows) are clamped; token ids
 *             outside [0, V) are clamped)
 *  U, W       [V][r] Markov factors (W stored vocab-major, i.e. the [r x V]
 *             factor transposed); both NULL => z = L
 *  parent_tok [P] token of each parent; parent_Lrow [P] its L row
 *  lse        [P] out: log sum_v exp(z_p[v])
 *  topk_tok   [P][k] out: tokens by (z desc, token asc)
 *  topk_logp  [P][k] out: z - lse of those tokens
 *  z_out      [P][V] out, optional (NULL in the fast path): the logit rows
 *  workspace  pct_markov_logits_workspace(P, V, k) bytes
 * Errors: PCT_ERR_INVALID_ARG for k < 1, k > V, V >= 2^18, P < 1, null
 * required pointers, or exactly one of U/W NULL; PCT_ERR_UNSUPPORTED for
 * k > 64 or P > 65535; PCT_ERR_WORKSPACE when workspace_bytes is too small.
 * bf16 factors with r in {32, 64, 128, 256} run on MFMA; other ranks and
 * fp32 factors take a plain VALU kernel. */
pct_status pct_markov_logits(const float* L, int64_t L_row_stride,
                             int32_t L_rows, const void* U, const void* W,
                             pct_dtype uw_dtype,
                             int32_t V, int32_t r, const int32_t* parent_tok,
                             const int32_t* parent_Lrow, int32_t P, int32_t k,
                             float* lse, int32_t* topk_tok, float* topk_logp,
                             float* z_out, void* workspace,
                             size_t workspace_bytes, void* stream);
size_t pct_markov_logits_workspace(int32_t P, int32_t V, int32_t k);

/* ------------------------------------------------------------------------
 * pct_build_tree -- [PCT] "straight draft": the parent-conditioned draft tree.
 * Depth d = 1..B expands every frontier parent p with
 * z_d(p) = L_d + Markov(p) (one batched call per depth), keeps each
 * parent's top-k children by log pi(v|p) = z - lse, scores a child by its
 * path log-probability s(c) = s(p) + log pi(c|p), keeps the beam_w best
 * children per request as the next frontier, and finally keeps the N best
 * of all generated children as the tree that fits the verify budget.
 * Order and ties: key (score desc, parent's pool id asc, token asc); the
 * pool id of a child is base_d + j*k + i for the i-th child of the j-th
 * frontier parent; the root's is -1.
 *
 *  L       [batch][B][V] fp32; row d-1 drives depth d
 *  U, W    [V][r] (W vocab-major) or both NULL (then z_d = L_d); both
 *          16-byte aligned
 *  anchor  [batch] root token of each request (the depth-1 parent)
 *  tok, parent, depth  [batch][N] int32 out; score [batch][N] fp32 out.
 *          Nodes come in key order, so parents precede children; parent is
 *          the output index of the parent, -1 for the root.  Entries past
 *          n_nodes hold tok -1, parent -1, depth 0, score -inf.
 *  n_nodes [batch] out: min(N, generated children)
 *  mask    [batch][N][ceil(N/64)] out, optional (NULL = not built)
 *  workspace  pct_build_tree_workspace(shape) bytes
 * Errors: as pct_markov_logits, plus PCT_ERR_INVALID_ARG for U or W not
 * 16-byte aligned, and PCT_ERR_UNSUPPORTED when the pool of generated
 * children per request exceeds 8192 or a per-depth candidate set exceeds
 * 2048. */
pct_status pct_build_tree(const pct_tree_shape* shape /*host*/,
                          const float* L, const void* U, const void* W,
                          const int32_t* anchor, int32_t* tok,
                          int32_t* parent, int32_t* depth, float* score,
                          int32_t* n_nodes, uint64_t* mask, void* workspace,
                          size_t workspace_bytes, void* stream);
size_t pct_build_tree_workspace(const pct_tree_shape* shape /*host*/);

/* ------------------------------------------------------------------------
 * pct_build_tree_adaptive -- [CAD] "Method": the greedy best-first tree
 * over a block-diffusion drafter's per-position marginals with the
 * throughput stop.  The probability of a prefix is the product of its
 * per-depth marginals, log pi_d(v) = L_d[v] - lse_d; nodes are taken in
 * best-first order, key (score desc, parent output index asc, child rank
 * asc), where a child's rank orders its row by (logit desc, token asc), so
 * equal scores fall back to the rank and equal logits to the token;
 * with P_i = exp(score_i), Phi_n = sum_{i<=n} P_i and D(n) = C(n; l), the
 * build stops at the first n whose gain
 * g(n) = P_{n+1} D(n) - (1 + Phi_n)(D(n+1) - D(n)) is not positive, i.e.
 * where (1 + Phi)/D stops increasing.  cost NULL => a fixed budget n_max.
 *
 *  L        [batch][B][V] fp32 marginal logits
 *  ctx_len  [batch] context length l of each request
 *  tok, parent, depth, score  [batch][n_max] out; the first n_star entries
 *           are the tree in best-first order, the rest are pads as above
 *  n_star   [batch] out; phi [batch] out Phi(n*); throughput [batch] out
 *           (1 + Phi)/D(n*) (1 + Phi without a cost model)
 *  mask     [batch][n_max][ceil(n_max/64)] out, optional
 * Every candidate is a child of a taken node among the min(n_max, V) best
 * tokens of its row (a node among the n best prefixes has rank < n among
 * its siblings), so the search is exact.  Each taken node opens at most
 * two candidates (its next sibling and its first child), so the open set
 * stays below 2 n_max + 2 entries.
 * Errors: PCT_ERR_INVALID_ARG for n_max < 1, B < 1, V < 1, V >= 2^18,
 * batch < 1 or null pointers; PCT_ERR_UNSUPPORTED for n_max > 1024, B > 255
 * or batch * B >= 2^22; a cost model with negative c1, c2 or c_ell, or with
 * C_d + c0 <= 0, is rejected (the stop rule is only the throughput optimum
 * for a positive, convex, increasing cost). */
pct_status pct_build_tree_adaptive(int32_t batch, int32_t B, int32_t V,
                                   int32_t n_max, const float* L,
                                   const int32_t* ctx_len,
                                   const pct_cost_model* cost /*host*/,
                                   int32_t* tok, int32_t* parent,
                                   int32_t* depth, float* score,
                                   int32_t* n_star, double* phi,
                                   double* throughput, uint64_t* mask,
                                   void* workspace, size_t workspace_bytes,
                                   void* stream);
size_t pct_build_tree_adaptive_workspace(int32_t batch, int32_t B, int32_t V,
                                         int32_t n_max);

/* ------------------------------------------------------------------------
 * pct_build_tree_adaptive_pc -- [CAD] "Method" on the parent-conditioned
 * tree of [PCT] "straight draft": the throughput stop over the key order of
 * a pct_build_tree build.  The build (shape, L, U, W, anchor as for
 * pct_build_tree, with N = n_max, the largest tree considered) yields its
 * nodes in key order, which is a best-first order: every node comes after
 * its parent.  With P_i = exp(score_i), Phi_n = sum_{i<=n} P_i and
 * D(n) = C(n; l), the tree keeps the first n* nodes, n* being the first n
 * whose gain g(n) = P_{n+1} D(n) - (1 + Phi_n)(D(n+1) - D(n)) is not
 * positive.  When k >= n* and beam_w >= n*, the kept nodes are the n* most
 * probable prefixes of the parent-conditioned drafter, i.e. the greedy
 * best-first tree (a top-n prefix has sibling rank < n and depth rank < n,
 * so the beam keeps it); with smaller k or beam_w it is the beam's
 * approximation of it.  cost NULL => n* = the number of nodes built.
 *
 *  tok, parent, depth, score  [batch][N] out: the first n_star entries are
 *           the tree, the rest pads (tok -1, parent -1, depth 0,
 *           score -inf)
 *  ctx_len  [batch] context length l of each request (needed with cost)
 *  n_star   [batch] out; phi [batch] out Phi(n*); throughput [batch] out
 *           (1 + Phi)/D(n*) (1 + Phi without a cost model)
 *  mask     [batch][N][ceil(N/64)] out, optional: the kept tree's mask
 *  workspace  pct_build_tree_adaptive_pc_workspace(shape) bytes
 * Errors: as pct_build_tree; a cost model with negative c1, c2 or c_ell, or
 * with C_d + c0 <= 0, is rejected with PCT_ERR_INVALID_ARG. */
pct_status pct_build_tree_adaptive_pc(
    const pct_tree_shape* shape /*host*/, const float* L, const void* U,
    const void* W, const int32_t* anchor, const int32_t* ctx_len,
    const pct_cost_model* cost /*host*/, int32_t* tok, int32_t* parent,
    int32_t* depth, float* score, int32_t* n_star, double* phi,
    double* throughput, uint64_t* mask, void* workspace,
    size_t workspace_bytes, void* stream);
size_t pct_build_tree_adaptive_pc_workspace(const pct_tree_shape* shape /*host*/);

/* ------------------------------------------------------------------------
 * pct_throughput_curve -- [CAD] "Method": the throughput of every prefix
 * of a best-first-ordered tree, f(n) = (1 + Phi_n) / D(n) for n = 0..N
 * (D = 1 without a cost model), as a fixed-budget (DDTree-style) build of n
 * nodes would get it; the oracle budget of a round is the n that maximises
 * it.  Budgets above a request's n_nodes repeat f(n_nodes).
 *  score    [batch][N] scores in best-first order (e.g. the output of a
 *           build without a cost model), n_nodes [batch]
 *  ctx_len  [batch] (needed with cost)
 *  f        [batch][N+1] out
 * Needs no workspace.
 * Errors: PCT_ERR_INVALID_ARG for batch < 1, N < 1, null required pointers
 * or a cost model that is not convex and increasing; PCT_ERR_UNSUPPORTED for
 * batch >= 2^26. */
pct_status pct_throughput_curve(int32_t batch, int32_t N, const float* score,
                                const int32_t* n_nodes,
                                const int32_t* ctx_len,
                                const pct_cost_model* cost /*host*/,
                                double* f, void* stream);

/* ------------------------------------------------------------------------
 * pct_tree_mask -- [PCT] "straight draft": the whole tree is verified in one
 * target forward, in which a node may see only itself and its ancestors.
 *  parent  [batch][N] (-1 = root), n_nodes [batch]
 *  mask    [batch][N][ceil(N/64)] out; rows >= n_nodes are zero
 * Errors: PCT_ERR_INVALID_ARG for batch < 1, N < 1 or null pointers. */
pct_status pct_tree_mask(int32_t batch, int32_t N, const int32_t* parent,
                         const int32_t* n_nodes, uint64_t* mask,
                         void* stream);

/* ------------------------------------------------------------------------
 * pct_verify_accept -- [DSP] "one inference, from guess to confirmation":
 * compare the draft with the target in order, accept the run of matches,
 * stop at the first mismatch where the target supplies its own token.  On
 * a tree: a node is accepted when its token equals the target's choice
 * after its parent and its parent is accepted (the root always is).
 *
 *  tok, parent, depth [batch][N] tree (parents precede children; siblings
 *          carry distinct tokens), n_nodes [batch]
 *  mask    [batch][N][ceil(N/64)] optional: the tree's packed ancestry mask
 *          (as pct_tree_mask writes it).  When given, a node is accepted
 *          exactly when every node of its mask row matches, which replaces
 *          the walk up the parent links by word operations; NULL = walk
 *  target  [batch][N+1]: target[0] is the target's token after the root,
 *          target[1+i] its token after node i
 *  tau     [batch] out: accepted tokens + 1 (the target's own token)
 *  accept_node [batch][B] out: the accepted nodes root-to-leaf, -1 padded
 *  accept_tok  [batch][B+1] out: their tokens, then the target's token,
 *          -1 padded
 * Needs no workspace.
 * Errors: PCT_ERR_INVALID_ARG for batch < 1, N < 1, B < 1, N > 8192 or
 * null required pointers; PCT_ERR_UNSUPPORTED for batch >= 2^26. */
pct_status pct_verify_accept(int32_t batch, int32_t N, int32_t B,
                             const int32_t* tok, const int32_t* parent,
                             const int32_t* depth, const int32_t* n_nodes,
                             const uint64_t* mask, const int32_t* target,
                             int32_t* tau, int32_t* accept_node,
                             int32_t* accept_tok, void* stream);

/* ------------------------------------------------------------------------
 * pct_verify_sample -- verification with temperature sampling instead of
 * greedy decoding.  The pages evaluate greedy decoding only ([PCT] "how
 * well it works, in numbers") and give no sampling rule; this call takes
 * the plainest one that keeps the target's distribution for a tree of
 * fixed (top-k) children: the target's token after each node is a sample
 * from softmax(target logits / T) rather than its argmax, and the walk of
 * pct_verify_accept runs on those samples ([DSP] "one inference, from guess
 * to confirmation": accept while the target's token is a drafted child,
 * then the target's own token).  Every emitted token is a target sample.
 * Sampling is Gumbel-max: token = argmax_v (z_v / T - log(-log(u_v))), ties
 * to the lowest token, keys in double, u_v = ((h >> 11) + 0.5) * 2^-53 with
 * h = sm(sm(sm(seed) ^ stream) ^ v), sm the SplitMix64 finaliser (Steele,
 * Lea and Flood, 2014) and stream = request * (N+1) + row.
 *
 *  tok, parent, depth, n_nodes, mask  the tree, as for pct_verify_accept
 *  target_logits  [batch][N+1][V] fp32: row 0 the target's logits after
 *          the root, row 1+i after node i (rows past n_nodes are not read)
 *  temperature    T > 0; seed  the generator's seed
 *  sampled [batch][N+1] out: the sampled target tokens (-1 past n_nodes)
 *  tau, accept_node, accept_tok  out, as for pct_verify_accept
 *  workspace  device memory of pct_verify_sample_workspace(batch, N, V)
 *          bytes: when there are few rows each row is cut into slices whose
 *          partial arg-maxes land there; may be NULL when that size is 0
 *          (enough rows to fill the GPU one workgroup per row)
 * Errors: PCT_ERR_INVALID_ARG for batch, B or V < 1, N outside [1, 8192],
 * a temperature that is not positive and finite, or null required
 * pointers; PCT_ERR_UNSUPPORTED for batch > 65535; PCT_ERR_WORKSPACE for a
 * missing or short workspace. */
size_t pct_verify_sample_workspace(int32_t batch, int32_t N, int32_t V);
pct_status pct_verify_sample(int32_t batch, int32_t N, int32_t B, int32_t V,
                             const int32_t* tok, const int32_t* parent,
                             const int32_t* depth, const int32_t* n_nodes,
                             const uint64_t* mask, const float* target_logits,
                             double temperature, uint64_t seed,
                             int32_t* sampled, int32_t* tau,
                             int32_t* accept_node, int32_t* accept_tok,
                             void* workspace, size_t workspace_bytes,
                             void* stream);

/* ------------------------------------------------------------------------
 * pct_build_tree_noalloc -- for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * allocation): pct_build_tree with the same arguments minus the workspace,
 * which is instead a fixed 32 MiB device array inside the library, one per
 * GPU, held until the process ends.  Shapes whose
 * pct_build_tree_workspace() exceeds 32 MiB return PCT_ERR_UNSUPPORTED
 * before anything is enqueued (the batch-128, N = 512 round needs about
 * 21 MB).  Allocates nothing.  All calls on one GPU share its array, so
 * calls that overlap in time on one GPU (other streams or threads) race;
 * calls ordered on one stream do not.  Errors otherwise as pct_build_tree. */
pct_status pct_build_tree_noalloc(const pct_tree_shape* shape /*host*/,
                                  const float* L, const void* U,
                                  const void* W, const int32_t* anchor,
                                  int32_t* tok, int32_t* parent,
                                  int32_t* depth, float* score,
                                  int32_t* n_nodes, uint64_t* mask,
                                  void* stream);

/* ------------------------------------------------------------------------
 * The target's side of a round ([PCT] "straight draft": the whole tree is
 * verified in one target forward) on a paged key-value cache.  The calls
 * below keep the cache's pages, write the tree's keys and values, attend
 * from the tree's rows and keep the rows that were accepted:
 *
 *   pct_build_tree (mask) -> pct_cache_plan -> per layer of the target
 *   { pct_cache_write, pct_tree_attention } -> pct_verify_accept or
 *   pct_verify_sample -> pct_cache_commit -> the next round
 *
 * With rotary positions pct_cache_write_rotary takes pct_cache_write's place.
 * Where requests share pages (pct_cache_fork), pct_cache_trim comes before the
 * plan, and pct_cache_share after it with pct_shared_attention in the layers.
 *
 * Positions of a request: its ctx_len committed tokens, then the root (the
 * last token the target supplied, not yet in the cache) at position
 * ctx_len, then node i at position ctx_len + 1 + i.  Rows: row 0 of a
 * request is its root, row 1 + i its node i, R = N + 1 rows per request, of
 * which the first n_nodes + 1 are used; n_nodes = -1 marks a padded request
 * (no row).  N = 0 is plain decoding, one new token per request.  The
 * values of ctx_len are taken as at least 0 and at most 2^30, those of
 * n_nodes as at least -1 and at most N.
 *
 * Shape of a paged cache and its rows
 *  batch      requests
 *  N          drafted nodes per request at most (0 <= N <= 8192)
 *  n_pages    pages of the cache
 *  page_size  tokens of a page, a power of two up to 1024
 *  max_pages  entries of a request's block table row;
 *             max_pages * page_size <= 2^30
 *  Hq, Hkv    query heads and key-value heads; query head h reads
 *             key-value head h / (Hq / Hkv); Hq <= 1024
 *  D          elements of a head, a multiple of 16 up to 256
 *  dtype      PCT_BF16 or PCT_F16: queries, cache and outputs
 * A cache is [n_pages][Hkv][page_size][D], keys and values apart.  The
 * block table [batch][max_pages] gives the page of each page_size
 * positions; an entry outside [0, n_pages) stands for no page: its
 * positions are not written, attended or moved, and neither are positions
 * past the table's max_pages * page_size. */
typedef struct {
  int32_t batch, N, n_pages, page_size, max_pages, Hq, Hkv, D, dtype;
} pct_cache_shape;

/* ------------------------------------------------------------------------
 * pct_cache_plan -- block tables and slots from the requests' lengths.
 * Every request is given ceil((ctx_len + n_nodes + 1) / page_size) pages
 * (at most max_pages), so a request of n_nodes = -1 keeps the pages of its
 * context and one of ctx_len = 0 and n_nodes = -1 gives all of them back.
 * Free pages are a ring: ring_state = {head, count}, the free pages are
 * ring[(head + i) % n_pages], i < count.  Pages that are needed come from
 * the head, request by request in order; from the first request that the
 * free pages of before the call do not satisfy, no request gets more.  Pages
 * past a request's need go to the tail, in the order of requests and
 * positions (they are handed out from the next call on).
 *
 *  ctx_len [batch], n_nodes [batch] (NULL = N in every request)
 *  depth   [batch][N] depth of each node (as the builds write it; needed
 *          with pos unless N = 0)
 *  block_table [batch][max_pages] in/out; entries past a request's pages
 *          that held one become -1, others there are not touched
 *  n_held  [batch] in/out: pages held (0 at first)
 *  ring    [n_pages] in/out, ring_state [2] in/out
 *  slot    [batch][R] out: page * page_size + offset of each used row; -1
 *          for unused rows and for rows whose position has no page
 *  pos     [batch][R] out, optional: the row's place in its sequence,
 *          ctx_len + its depth (the root's is 0), -1 for unused rows
 *  missing [batch] out: pages needed and not held.  A request that misses
 *          pages has rows without a slot, which are neither written nor
 *          attended: this round must not be kept (its positions would hold
 *          whatever their pages held before).  It waits for a later round.
 *  n_served [batch] out (pct_cache_plan_served): the n_nodes of the round's
 *          pct_tree_attention and pct_cache_commit, which leave out the
 *          requests that wait: n_nodes, or -1 where missing > 0.  What the
 *          acceptance walk answers for those is not used.  NULL: not written
 *  workspace  pct_cache_plan_workspace(batch) bytes
 * Only batch, N, n_pages, page_size and max_pages of the shape are read.
 * Precondition (not checked): ring and block_table hold every page once.
 * Errors: PCT_ERR_INVALID_ARG for a size outside its range, null required
 * pointers or an n_served that overlaps n_nodes or ctx_len;
 * PCT_ERR_UNSUPPORTED for batch > 65535; PCT_ERR_WORKSPACE. */
size_t pct_cache_plan_workspace(int32_t batch);
pct_status pct_cache_plan(const pct_cache_shape* shape /*host*/,
                          const int32_t* ctx_len, const int32_t* n_nodes,
                          const int32_t* depth, int32_t* block_table,
                          int32_t* n_held, int32_t* ring,
                          int32_t* ring_state, int64_t* slot, int32_t* pos,
                          int32_t* missing, void* workspace,
                          size_t workspace_bytes, void* stream);
pct_status pct_cache_plan_served(
    const pct_cache_shape* shape /*host*/, const int32_t* ctx_len,
    const int32_t* n_nodes, const int32_t* depth, int32_t* block_table,
    int32_t* n_held, int32_t* ring, int32_t* ring_state, int64_t* slot,
    int32_t* pos, int32_t* missing, int32_t* n_served, void* workspace,
    size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * pct_cache_write -- a layer's keys and values of the round's rows into
 * their slots.
 *  k, v    [batch * R] rows of [Hkv][D], k_row_stride and v_row_stride
 *          elements from row to row (views of a joint projection)
 *  slot    [batch * R]; a slot outside [0, n_pages * page_size) is left
 *          out.  The slots of one call are distinct.
 *  k_cache, v_cache  [n_pages][Hkv][page_size][D]
 * Only batch, N, n_pages, page_size, Hkv, D and dtype of the shape are read.
 * Errors: PCT_ERR_INVALID_ARG for sizes, null pointers, strides below
 * Hkv * D or not a multiple of 8, pointers that are not 16-byte aligned. */
pct_status pct_cache_write(const pct_cache_shape* shape /*host*/,
                           const void* k, int64_t k_row_stride,
                           const void* v, int64_t v_row_stride,
                           const int64_t* slot, void* k_cache, void* v_cache,
                           void* stream);

/* ------------------------------------------------------------------------
 * Rotary positions.  A rotary description says which elements of a head are
 * rotated and how fast:
 *  rot      rotated elements, the first ones of each head, even; 0: none
 *  layout   PCT_ROTARY_HALF: pair i is (i, i + rot/2),
 *           PCT_ROTARY_INTERLEAVED: (2i, 2i + 1)
 *  base     pair i turns by f_i = base^(-2i/rot) radians per position
 *  scaling, factor  for long contexts, with s = factor:
 *           PCT_ROTARY_PLAIN   f_i
 *           PCT_ROTARY_LINEAR  f_i / s
 *           PCT_ROTARY_BASE    base * s^(rot/(rot - 2)) in base's place
 *           PCT_ROTARY_RAMP    w f_i + (1 - w) f_i / s; w falls linearly with
 *                              i, from 1 at the pair (rounded down) that makes
 *                              `high` turns over `original` positions to 0 at
 *                              the pair (rounded up) that makes `low`
 *           PCT_ROTARY_BANDS   the same with w = (turns of pair i over
 *                              `original` positions - low) / (high - low)
 *           (the pairs of a ramp are kept within 0 .. rot - 1, w within 0 .. 1)
 *  amplitude  factor of the rotated elements (1: none)
 *
 * pct_rotary_table -- frequencies of a description.
 *  table  [rot/2] (host) out: turns per position in units of 2^-64 (a whole
 *         number of turns counts as none), which the caller keeps on the
 *         device for the calls below
 * Errors: PCT_ERR_INVALID_ARG for fields outside their ranges (base > 1,
 * factor > 0, original >= 1, 0 < low < high, as far as the scaling reads
 * them; rot = 2 with a scaled base). */
typedef enum { PCT_ROTARY_HALF = 0, PCT_ROTARY_INTERLEAVED = 1 }
    pct_rotary_layout;
typedef enum {
  PCT_ROTARY_PLAIN = 0,
  PCT_ROTARY_LINEAR = 1,
  PCT_ROTARY_BASE = 2,
  PCT_ROTARY_RAMP = 3,
  PCT_ROTARY_BANDS = 4
} pct_rotary_scaling;
typedef struct {
  int32_t rot, layout, scaling, original;
  double base, factor, low, high, amplitude;
} pct_rotary;
pct_status pct_rotary_table(const pct_rotary* rotary /*host*/,
                            uint64_t* table /*host*/);

/* ------------------------------------------------------------------------
 * pct_cache_write_rotary -- a layer's queries, keys and values on their way
 * to the attention: queries and keys are normalised (if weights are given)
 * and rotated to their rows' positions, queries go to q_out, keys and values
 * (as they are) into their slots:
 *   x <- x / sqrt(sum_D x^2 / D + eps) * weight     (over the whole head)
 *   (x0, x1) <- amplitude (x0 cos - x1 sin, x1 cos + x0 sin)  (its pairs)
 * in fp32, rounded once.  Angles are exact to 2^-32 turns at any position.
 *  table   [rot/2] as pct_rotary_table makes it (may be NULL if rot = 0);
 *          of the description, rot, layout and amplitude are read
 *  q_weight, k_weight  [D] fp32, NULL: no norm
 *  q       rows of [Hq][D], k and v rows of [Hkv][D], *_row_stride elements
 *          from row to row (views of a joint projection).  q (with q_out) or
 *          k and v may be NULL: these rows are then left out
 *  pos     [batch * R] position of each row; rows with a negative one are
 *          left out altogether: q_out and the cache stay as they were
 *  slot    [batch * R] as for pct_cache_write (not read without k and v)
 *  q_out   rows of [Hq][D]; may be q itself with its stride
 *  k_cache, v_cache  as for pct_cache_write
 * Only batch, N, n_pages, page_size, Hq (with q), Hkv, D and dtype of the
 * shape are read.
 * Errors: PCT_ERR_INVALID_ARG for sizes, rot > D, an eps that is negative or
 * not finite, null pointers, strides that do not hold a row or are not a
 * multiple of 8, pointers to elements that are not 16-byte aligned, a q_out
 * that overlaps q, k or v (first to last row) without being q. */
pct_status pct_cache_write_rotary(
    const pct_cache_shape* shape /*host*/, const pct_rotary* rotary /*host*/,
    const uint64_t* table, float eps, const float* q_weight,
    const float* k_weight, const void* q, int64_t q_row_stride, const void* k,
    int64_t k_row_stride, const void* v, int64_t v_row_stride,
    const int32_t* pos, const int64_t* slot, void* q_out,
    int64_t q_out_row_stride, void* k_cache, void* v_cache, void* stream);

/* ------------------------------------------------------------------------
 * pct_tree_attention -- softmax attention of the round's rows over the
 * cache.  A row sees the request's context, the root and, of the nodes,
 * those of its mask row (itself and its ancestors); without a mask node i
 * sees nodes 0..i (a straight draft, or a piece of a prompt).  With S the
 * set of seen positions that have a page,
 *   out = sum_{t in S} softmax_S(scale * q . k_t) v_t,
 *   lse = ln sum_{t in S} exp(scale * q . k_t);
 * an empty S, and one whose scores are all -inf, gives out = 0 and lse =
 * -inf.  Positions outside a row's S have
 * no influence on it, whatever the cache holds there (NaN included).
 * Scores, normalisers and sums are fp32; a probability (in fp16 2^7 times
 * it, which keeps those down to 2^-32 of the largest) is rounded to the
 * cache's type before it meets a value.
 *
 *  q       rows of [Hq][D], q_row_stride elements from row to row
 *  k_cache, v_cache, block_table, ctx_len, n_nodes (NULL = N)  as above
 *  mask    [batch][N][ceil(N/64)] as pct_tree_mask writes it, or NULL
 *  out     [batch][R][Hq][D]; lse [batch][R][Hq] optional.  Unused rows
 *          are left as they were.
 *  workspace  pct_tree_attention_workspace(shape) bytes
 * Errors: PCT_ERR_INVALID_ARG for sizes, null pointers, a scale whose
 * product with log2(e) is not finite, a stride below Hq * D or not a multiple
 * of 8, pointers that are not 16-byte aligned; PCT_ERR_UNSUPPORTED for batch > 65535;
 * PCT_ERR_WORKSPACE. */
size_t pct_tree_attention_workspace(const pct_cache_shape* shape /*host*/);
pct_status pct_tree_attention(const pct_cache_shape* shape /*host*/,
                              float scale, const void* q,
                              int64_t q_row_stride, const void* k_cache,
                              const void* v_cache,
                              const int32_t* block_table,
                              const int32_t* ctx_len, const int32_t* n_nodes,
                              const uint64_t* mask, void* out, float* lse,
                              void* workspace, size_t workspace_bytes,
                              void* stream);

/* ------------------------------------------------------------------------
 * pct_cache_commit -- after the acceptance walk: the accepted path's keys
 * and values move, in every layer, to the positions behind the root, and
 * the context grows by the root and the accepted nodes: node accept_node[j]
 * moves to position ctx_len + 1 + j, j < tau - 1, and ctx_out = ctx_len +
 * tau.  A padded request keeps its length and its cache.
 *  layers, layer_stride  caches of `layers` layers, layer_stride elements
 *          apart (at least n_pages * Hkv * page_size * D)
 *  B       entries of accept_node per request
 *  tau [batch], accept_node [batch][B]  as pct_verify_accept writes them
 *          (nodes in ascending order); the first entry outside
 *          [0, n_nodes) ends the moves
 *  ctx_len [batch]; ctx_out [batch], which may be ctx_len itself
 * Needs no workspace.
 * Errors: PCT_ERR_INVALID_ARG for sizes, null pointers, caches that are not
 * 16-byte aligned, a layer_stride that is too short or not a multiple of 8,
 * a ctx_out that overlaps ctx_len without being it, or tau, accept_node or
 * n_nodes; PCT_ERR_UNSUPPORTED for batch > 65535. */
pct_status pct_cache_commit(const pct_cache_shape* shape /*host*/,
                            int32_t layers, int64_t layer_stride, int32_t B,
                            const int32_t* tau, const int32_t* accept_node,
                            const int32_t* n_nodes,
                            const int32_t* block_table,
                            const int32_t* ctx_len, void* k_cache,
                            void* v_cache, int32_t* ctx_out, void* stream);

/* ------------------------------------------------------------------------
 * Pages that several requests hold.  The state of a cache's pages is that of
 * pct_cache_plan with a count of holders per page:
 *  ctx_len [batch], block_table [batch][max_pages], n_held [batch],
 *  ring [n_pages], ring_state [2]  as for pct_cache_plan
 *  extra   [n_pages] holders of a page beyond the first: 0 for pages that one
 *          request holds, and for free ones (all 0 at first)
 * pct_cache_plan takes pages from the ring, which leaves extra as it is, but
 * gives pages back without a look at their holders: where requests share
 * pages, pct_cache_trim comes before it and leaves it nothing to give back.
 * A shared page is in use by all of its holders: a request's context length
 * must not be lowered into its shared pages other than by pct_cache_free.
 * A request holds a page once.  Results do not depend on timing. */
typedef struct {
  int32_t *ctx_len, *block_table, *n_held, *ring, *ring_state, *extra;
} pct_page_state; /* (host) of device pointers */

/* ------------------------------------------------------------------------
 * pct_cache_free -- places become empty: ctx_len 0, n_held 0, their table
 * entries -1.  A page whose last holder lets go is free: such pages go to
 * the ring's tail in ascending order, the others' extra goes down.
 *  m, places  [m] places; entries outside [0, batch) are left out, a place
 *          may be named more than once
 *  workspace  pct_cache_free_workspace(shape) bytes
 * pct_cache_trim -- every request keeps the pages of its ctx_len + n_nodes + 1
 * positions and lets go of the rest in the same way (n_nodes NULL = N).
 * Only batch, N (trim), n_pages, page_size and max_pages are read (an N that
 * is not has to be in its range too, here and for the calls below).
 * Errors: PCT_ERR_INVALID_ARG for sizes, m < 0, null pointers, arrays or a
 * workspace that overlap; PCT_ERR_UNSUPPORTED for batch or m > 65535 or n_pages > 2^30;
 * PCT_ERR_WORKSPACE. */
size_t pct_cache_free_workspace(const pct_cache_shape* shape /*host*/);
pct_status pct_cache_free(const pct_cache_shape* shape /*host*/, int32_t m,
                          const int32_t* places,
                          const pct_page_state* state /*host*/,
                          void* workspace, size_t workspace_bytes,
                          void* stream);
pct_status pct_cache_trim(const pct_cache_shape* shape /*host*/,
                          const int32_t* n_nodes,
                          const pct_page_state* state /*host*/,
                          void* workspace, size_t workspace_bytes,
                          void* stream);

/* ------------------------------------------------------------------------
 * pct_cache_fork -- place dst[i] becomes a copy of the first length[i]
 * positions of src[i]'s context (at most ctx_len of it; length NULL: all of
 * it): it holds the same whole pages (extra goes up), and a page of its own
 * from the ring's head, in the order of the pairs, for the positions of a
 * last page in part, whose rows are copied in all layers.
 *  done    [m] out: 1, or 0 for a pair that is left out: src or dst outside
 *          [0, batch) or the same, dst holds pages or is named by an earlier
 *          pair, src does not hold the pages of its positions, or the ring
 *          has no page left (from then on no pair gets one)
 *  layers, layer_stride, k_cache, v_cache  as for pct_cache_commit
 *  workspace  pct_cache_fork_workspace(shape, m) bytes
 * All pairs see the state of before the call; a src may be named in many.
 * Only batch, n_pages, page_size, max_pages, Hkv, D and dtype are read.
 * Errors: as pct_cache_free, and as pct_cache_commit for the caches. */
size_t pct_cache_fork_workspace(const pct_cache_shape* shape /*host*/,
                                int32_t m);
pct_status pct_cache_fork(const pct_cache_shape* shape /*host*/,
                          int32_t layers, int64_t layer_stride, int32_t m,
                          const int32_t* src, const int32_t* dst,
                          const int32_t* length,
                          const pct_page_state* state /*host*/, void* k_cache,
                          void* v_cache, int32_t* done, void* workspace,
                          size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * pct_cache_compact -- the pages in use become the first ones of the cache:
 * with T pages in the tables (the first n_held entries of each row), those
 * from T on move, in ascending order, to the unused ones below T, in
 * ascending order, in all layers; the others stay where they are.
 *  state   block_table and n_held are read; ring, ring_state and extra are
 *          written from them alone (so that pages that got lost are free
 *          again): ring[i] = (T + i) mod n_pages, ring_state = {0, n_pages - T}
 *  table_out [batch][max_pages] the new table, may be block_table itself
 *  layers, layer_stride, k_cache, v_cache  as for pct_cache_commit
 *  workspace  pct_cache_compact_workspace(shape) bytes
 * Slots, share plans and tables of before the call are void.
 * Only batch, n_pages, page_size, max_pages, Hkv, D and dtype are read.
 * Errors: as pct_cache_fork. */
size_t pct_cache_compact_workspace(const pct_cache_shape* shape /*host*/);
pct_status pct_cache_compact(const pct_cache_shape* shape /*host*/,
                             int32_t layers, int64_t layer_stride,
                             const pct_page_state* state /*host*/,
                             int32_t* table_out, void* k_cache, void* v_cache,
                             void* workspace, size_t workspace_bytes,
                             void* stream);

/* ------------------------------------------------------------------------
 * pct_cache_share -- which requests of a round share a prefix, found from
 * their tables.  With full_b the whole pages of request b's context (none if
 * n_nodes = -1; its root's page is never among them) and c_j(p) the number of
 * requests with j < full_b whose entry j is page p, each request picks
 * its entry j of largest gain (j + 1) (c_j(block_table[b][j]) - 1), the first
 * such (gains from 2^33 on count as alike), or none if gain * page_size <
 * least.  Requests that picked the same page at the same j, and whose
 * tables agree in the entries 0..j with those of the lowest of them, are a
 * group, if they are two or more.
 *  least   positions that a pick must promise by its gain (>= 1).  The gain
 *          counts all requests that have the page there; a group can be fewer
 *          of them, where others pick another place or differ before it, and
 *          then saves less
 *  ctx_len, n_nodes (NULL = N), block_table  as for pct_tree_attention
 *  leader  [batch] out: lowest request of the group, b itself without one
 *  shared  [batch] out: positions that the group shares, 0 without one
 *  share   pct_cache_share_size(shape) bytes out, 16-byte aligned: the plan
 *          for pct_shared_attention, which holds the lengths too
 *  workspace  pct_cache_share_workspace(shape) bytes
 * Only batch, N, n_pages, page_size and max_pages of the shape are read.
 * Errors: PCT_ERR_INVALID_ARG for sizes, least < 1, null pointers, outputs or
 * a workspace that overlap each other or an input; PCT_ERR_UNSUPPORTED for
 * batch > 1024; PCT_ERR_WORKSPACE. */
size_t pct_cache_share_size(const pct_cache_shape* shape /*host*/);
size_t pct_cache_share_workspace(const pct_cache_shape* shape /*host*/);
pct_status pct_cache_share(const pct_cache_shape* shape /*host*/,
                           int32_t least, const int32_t* ctx_len,
                           const int32_t* n_nodes, const int32_t* block_table,
                           int32_t* leader, int32_t* shared, void* share,
                           void* workspace, size_t workspace_bytes,
                           void* stream);

/* ------------------------------------------------------------------------
 * pct_shared_attention -- pct_tree_attention that reads what a group of
 * requests shares once for all of its rows.  Arguments, results and errors
 * are those of pct_tree_attention, but
 *  share   as pct_cache_share wrote it for the same shape (precondition, not
 *          checked) from the same block_table; the lengths are the ones that
 *          it was given
 *  workspace  pct_shared_attention_workspace(shape) bytes: fp32 sums of all
 *          rows, twice (32 heads of 128: 18 MB for 8 rows, 145 MB for 16 x 65,
 *          2.4 GB for 128 x 513)
 * Every row goes through these sums, in a group or not: pct_tree_attention is
 * as fast or faster for trees of 257 rows and more, and for trees of 65 rows
 * and more that share nothing.
 *  PCT_ERR_UNSUPPORTED for batch > 1024 or batch * (N + 1) * Hq / Hkv > 2^30 */
size_t pct_shared_attention_workspace(const pct_cache_shape* shape /*host*/);
pct_status pct_shared_attention(const pct_cache_shape* shape /*host*/,
                                float scale, const void* q,
                                int64_t q_row_stride, const void* k_cache,
                                const void* v_cache,
                                const int32_t* block_table, const void* share,
                                const uint64_t* mask, void* out, float* lse,
                                void* workspace, size_t workspace_bytes,
                                void* stream);

/* ------------------------------------------------------------------------
 * Profiling (not from the pages; for measuring kernels against the
 * hardware roofline).  When enabled, every kernel launch of the calls above
 * is bracketed by two HIP events recorded on its stream, tagged with a kind
 * and its work units.  Kinds: 0 fused Markov/log-sum-exp/top-k kernel
 * (units = parents of the launch), 1 per-request expand, 2 global top-N,
 * 3 mask, 4 acceptance walk, 5 seed pre-pass (units = rows), 6 depth-1
 * init, 7 adaptive row statistics (units = rows), 8 adaptive best-first +
 * stop, 9 standalone per-parent results, 10 throughput stop / curve scan,
 * 11 sampled target tokens, 12 cache plan, 13 cache write, 14 tree
 * attention (units = rows), 15 its join, 16 cache commit, 17 rotary write,
 * 18 cache free and trim, 19 fork, 20 compaction, 21 share plan.
 * The parts of shared attention count as tree attention and its join.
 *  pct_profile_enable  turns recording on or off (the event pool, 8192
 *                      launches, is created on the first enable)
 *  pct_profile_reset   forgets recorded launches
 *  pct_profile_read    total milliseconds and number of recorded launches of
 *                      one kind (units < 0: any units); waits for the events
 * Not thread-safe against concurrent calls that launch kernels. */
pct_status pct_profile_enable(int32_t enable);
pct_status pct_profile_reset(void);
pct_status pct_profile_read(int32_t kind, int64_t units, double* total_ms,
                            int64_t* launches);

const char* pct_status_string(pct_status s);
const char* pct_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* PCTREE_H */

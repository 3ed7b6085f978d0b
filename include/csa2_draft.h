/*
 * csa2_draft.h -- C ABI of libcsa2.so's calls for drafted tokens and shared pages (GB300, sm_103a).
 *
 * A server that lets a small model draft tokens runs its large model once over all of them: a
 * request's new tokens are then a tree, whose node 0 is the last token and whose other nodes are
 * drafts.  Beside the paged cache's calls (csa2_paged.h), one step is
 *
 *   csa2p_page_plan     slots for every node (delta = nodes)
 *   csa2d_tree_plan     the nodes' positions and what each of them sees
 *   csa2p_rope, csa2p_write        as for other tokens, at those positions
 *   csa2d_tree_attn     attention of the nodes over their requests' pages
 *   csa2d_tree_verify   which path of nodes stays, and the token behind it
 *   csa2d_compact       the path's rows moved together, in every layer's cache
 *   csa2p_page_plan     the other nodes' rows given back (delta, as csa2d_compact left it)
 *
 * A request that csa2d_tree_plan leaves out has pos -1 throughout; verification and compaction take pos,
 * so that it keeps nothing and its nodes' rows all go back.
 *
 * Requests that continue one prompt in several ways share its pages:
 *
 *   csa2d_page_fork     block tables, page counts and lengths of the forked requests
 *   csa2d_page_copy     the contents of pages, in every layer's cache
 *   csa2d_page_free     requests that end, whose pages others may still hold
 *
 * The conventions are csa2_paged.h's: device pointers owned by the caller, work enqueued on
 * `stream`, no allocation, no synchronisation, errors found on the host returned before any
 * launch, errors found on the device ORed into *d_status (nullable) with every access in bounds;
 * every kernel waits for the kernel just before it on the stream before it reads any input.
 * Calls on different streams may run concurrently while what they write is disjoint from what the
 * others read or write; captured graphs that may run at the same time need workspaces of their
 * own.  Addresses of 32-bit values are multiples of 4.
 */
#ifndef CSA2_DRAFT_H
#define CSA2_DRAFT_H

#include "csa2_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further device status bit. */
#define CSA2D_DEV_NO_TOKEN 0x800u   /* a row of probabilities from which no token can be drawn     */

#define CSA2D_MAX_WORDS 32          /* words of a node's mask: trees of up to 1,024 nodes          */
#define CSA2D_MAX_VOCAB (1 << 18)
#define CSA2D_MAX_CACHES 32         /* caches of one call                                          */

/* ---------------------------------------------------------------------------------- */
/* csa2d_tree_plan -- positions and masks of trees.  Request b's nodes are the tokens          */
/* cu[b] .. cu[b+1]-1, n of them, its last n rows: row base + i, base = lens[b] - n, is node i's. */
/* parent[cu[b] + i] is the node that i follows, a lower one, or -1 (a root: it follows row       */
/* base - 1).  Of each node                                                                      */
/*   pos  = base + its depth (a root's is 0)                                                     */
/*   seen = bits of the nodes on its way up to its root, itself among them: bit k % 32 of word    */
/*          k / 32 is node k's                                                                    */
/* A parent that is not a lower node or -1 counts as -1 (CSA2_DEV_BAD_INDEX).  A request that has  */
/* more nodes than the masks have bits, fewer rows than nodes, or nodes outside 0..n_tokens is     */
/* left out (CSA2_DEV_BAD_INDEX); its tokens, and those of no request, get pos -1 and no bits.      */
/* So does every token where cu steps down within 0..n_tokens (CSA2_DEV_BAD_INDEX).                 */
/* ---------------------------------------------------------------------------------- */
typedef struct {
    int32_t batch;            /* requests, 0..CSA2P_MAX_BATCH                                    */
    int32_t n_tokens;
    int32_t words;            /* of a node's mask, 1..CSA2D_MAX_WORDS                            */
    const int32_t *parent;    /* [n_tokens]                                                      */
    const int32_t *lens;      /* [batch] rows held, the nodes' included                          */
    const int32_t *cu;        /* [batch + 1]                                                     */
    int32_t *pos;             /* [n_tokens]                                                      */
    uint32_t *seen;           /* [n_tokens, words]                                               */
} csa2d_tree_args;
CSA2_API csa2_status csa2d_tree_plan(const csa2d_tree_args *a, uint32_t *d_status, csa2_stream stream);

/* ---------------------------------------------------------------------------------- */
/* csa2d_tree_attn -- csa2p_attn for trees.  Node i of request b (cu, lens, base as above) sees   */
/* the rows                                                                                      */
/*   j < base          with j >= max(kv_start[b], pos_i + 1 - window)                             */
/*   base + k, k < n   with bit k of seen_i, and pos_k >= max(kv_start[b], pos_i + 1 - window)     */
/* (window 0: no bound from it, and node k counts as position base + k; pos may then be NULL;      */
/* kv_start NULL: 0).  seen may hold any bits: csa2d_tree_plan's, or a mask of the caller's own,    */
/* one that leaves a node nothing among them.  Products, formats, outputs, what is not finite and    */
/* the workspace are csa2p_attn's; a node without keys gets out = 0 and lse = -inf.  A request with   */
/* more rows than its table reaches sets CSA2_DEV_BAD_INDEX, as does a page id outside [0, n_pages):   */
/* such rows are no keys.  A request whose nodes are not all in 0..n_tokens, with more nodes than bits  */
/* or fewer rows than nodes is left out (CSA2_DEV_BAD_INDEX): its tokens, as those of no request, are    */
/* left as they were in out and lse.  A call in which cu steps down within 0..n_tokens sets               */
/* CSA2_DEV_BAD_INDEX and does nothing.                                                                    */
/* ---------------------------------------------------------------------------------- */
typedef struct {
    csa2p_cache cache;
    int32_t batch;            /* requests, 0..CSA2P_MAX_BATCH                                    */
    int32_t n_tokens;         /* query tokens held by q                                          */
    int32_t n_heads;          /* 1..128                                                          */
    int32_t d_v;              /* 8..512, a multiple of 8, <= d_qk; d_qk <= 576                    */
    int32_t width;            /* block table entries a request                                   */
    int32_t window;           /* >= 0; 0: no window                                              */
    int32_t words;            /* of a node's mask, 1..CSA2D_MAX_WORDS                            */
    float sm_scale;           /* above 0, at most 2.3e38                                         */
    const uint16_t *q;        /* bf16 [n_tokens, n_heads, d_qk], 16-byte aligned                 */
    const int32_t *block_table; /* [batch, width]                                                */
    const int32_t *lens;      /* [batch] rows held, the nodes' included                          */
    const int32_t *cu;        /* [batch + 1]                                                     */
    const uint32_t *seen;     /* [n_tokens, words]                                               */
    const int32_t *pos;       /* [n_tokens]; NULL only where window is 0                         */
    const int32_t *kv_start;  /* [batch] or NULL                                                 */
} csa2d_tree_attn_args;
CSA2_API size_t csa2d_tree_attn_workspace_size(const csa2d_tree_attn_args *a);    /* as csa2p_attn's */
CSA2_API csa2_status csa2d_tree_attn(const csa2d_tree_attn_args *a, uint16_t *out, float *lse, void *ws,
                                     size_t ws_bytes, uint32_t *d_status, csa2_stream stream);

/* ---------------------------------------------------------------------------------- */
/* csa2d_tree_verify -- which drafts stay.  p[t] is the target's distribution of the token that    */
/* follows node t; q[t] the one that t's children were drawn from, each for itself (q NULL: the      */
/* drafts were not drawn, they are certain).  Beginning with node 0, the kept node v's children are    */
/* tried in order; child i of token x, with the given number u[i], from 0 to 1, stays                  */
/*   with q:     where u q_v(x) m < max(p_v(x) - c q_v(x), 0);  after a rejection c += m, then          */
/*               m = sum over the vocabulary of max(p_v - c q_v, 0);  c = 0, m = 1 at first              */
/*   without q:  where u m < p_v(x);  after a rejection m = max(m - p_v(x), 0) and p_v(x) counts as 0     */
/* -- (p - c q)+ / m is what is left of p after rejections, each of which takes (p - q)+ and normalises   */
/* it anew.  The next token is then drawn, with the given r[b], from what is left of p_v (from p_v itself  */
/* where nothing is left): the lowest y with                                                              */
/*   sum_{x <= y} w(x) > floor(W M / 2^24),  W = sum w,  M = floor(r 2^24) held to 0..2^24-1               */
/* where w(x) is the weight as a whole number of 2^-40, the nearest, ties to even, held to 2^40.            */
/* So, where the rows of p and q sum to 1 and u and r are uniform, the kept tokens and the next are            */
/* distributed as the target's own, to within the numbers' steps: r counts as one of 2^24, so the chance of     */
/* each next token is less than 2^-24 off w / W (one lighter than W 2^-24 has none or 2^-24; over a flat tail    */
/* of 2^18 tokens this adds up to 1.6% at most).  Every float32 operation above is rounded once, in the order     */
/* written; sums are of whole numbers w(x) (m is their sum x 2^-40, rounded to float32): the same inputs give     */
/* the same tokens whatever the order.                                                                            */
/* Values of p and q below 0 or not finite count as 0 and set CSA2_DEV_NONFINITE where they are used.          */
/* A draft whose token is outside the vocabulary is passed over (CSA2_DEV_BAD_INDEX).                           */
/* keep[b] = nodes that stay, node 0 among them; path[b] = these nodes in order, -1 behind them;                 */
/* next_token[b] = the token drawn (-1 where p_v has no weight: CSA2D_DEV_NO_TOKEN); delta[b] = keep[b] - n.      */
/* A path of max_path nodes ends there.  A request without nodes gets keep 0, token -1, delta 0.  One with nodes   */
/* outside 0..n_tokens, with more than 32 CSA2D_MAX_WORDS of them, or, where pos is given, that csa2d_tree_plan      */
/* left out (its node 0 has a pos below 0: csa2d_tree_attn leaves its outputs as they were, so there is nothing to    */
/* verify) gets keep 0 and token -1 too (CSA2_DEV_BAD_INDEX); its delta is -n where pos is given, else 0.               */
/* ---------------------------------------------------------------------------------- */
typedef enum { CSA2D_F32 = 0, CSA2D_F16 = 1, CSA2D_BF16 = 2 } csa2d_float;
typedef struct {
    int32_t batch;            /* requests, 0..CSA2P_MAX_BATCH                                    */
    int32_t n_tokens;
    int32_t vocab;            /* 1..CSA2D_MAX_VOCAB                                              */
    int32_t type;             /* csa2d_float of p and q                                          */
    int32_t max_path;         /* >= 1                                                            */
    int64_t p_row, q_row;     /* elements between rows, >= vocab                                 */
    const void *p;            /* [n_tokens, vocab], aligned to its values                        */
    const void *q;            /* [n_tokens, vocab] or NULL                                       */
    const int32_t *token;     /* [n_tokens] (a node 0's is not read)                             */
    const int32_t *parent;    /* [n_tokens] as csa2d_tree_plan's (a node 0's is not read)        */
    const int32_t *cu;        /* [batch + 1]                                                     */
    const float *u;           /* [n_tokens] (a node 0's is not read)                             */
    const float *r;           /* [batch]                                                         */
    int32_t *keep;            /* [batch]                                                         */
    int32_t *path;            /* [batch, max_path]                                               */
    int32_t *next_token;      /* [batch]                                                         */
    int32_t *delta;           /* [batch]                                                         */
    const int32_t *pos;       /* [n_tokens] csa2d_tree_plan's, or NULL                           */
} csa2d_verify_args;
CSA2_API csa2_status csa2d_tree_verify(const csa2d_verify_args *a, uint32_t *d_status, csa2_stream stream);

/* ---------------------------------------------------------------------------------- */
/* csa2d_compact -- the kept nodes' rows moved together.  In each cache (all share the block table)   */
/* row base + path[b][i] of request b goes, as it is stored, to row base + i, i < keep[b]; other rows   */
/* stay as they are.  A path has to rise and stay below n: a request whose path does not, or whose keep   */
/* is outside 0..max_path, moves nothing; neither does one with fewer rows than nodes (CSA2_DEV_BAD_INDEX   */
/* each).  Where pos is given, neither does one whose nodes are not all in 0..n_tokens or whose node 0 has a  */
/* pos below 0: csa2d_tree_plan left it out, whatever its keep (CSA2_DEV_BAD_INDEX where that is not 0).       */
/* A row whose page is none, at either end, is not moved (CSA2_DEV_BAD_INDEX).  Caches must not share         */
/* memory, and no page may be held by two requests at rows that move.                                         */
/* delta, where it is given, is what csa2p_page_plan will add to lens (csa2d_tree_verify's): that of a request  */
/* that is left out by pos or whose path is refused is lowered to -n, so that its nodes' rows all go back;       */
/* others, and those with fewer rows than nodes, stay as they are.                                                */
/* ---------------------------------------------------------------------------------- */
typedef struct {
    int32_t batch;            /* requests, 0..CSA2P_MAX_BATCH                                    */
    int32_t width;            /* block table entries a request                                   */
    int32_t max_path;         /* entries of a path                                               */
    const int32_t *block_table; /* [batch, width]                                                */
    const int32_t *lens;      /* [batch] rows held, the nodes' included                          */
    const int32_t *cu;        /* [batch + 1]: n = cu[b+1] - cu[b] nodes                          */
    const int32_t *path;      /* [batch, max_path]                                               */
    const int32_t *keep;      /* [batch]                                                         */
    const int32_t *pos;       /* [n_tokens] csa2d_tree_plan's, or NULL                           */
    int32_t *delta;           /* [batch] in and out, or NULL                                     */
    int32_t n_tokens;         /* entries of pos                                                  */
} csa2d_compact_args;
/* caches: n of them in host memory, 0..CSA2D_MAX_CACHES, with one page size (0: nothing is done). */
CSA2_API csa2_status csa2d_compact(const csa2d_compact_args *a, const csa2p_cache *caches, int32_t n,
                                   uint32_t *d_status, csa2_stream stream);

/* ---------------------------------------------------------------------------------- */
/* csa2d_page_fork -- requests that continue others.  source[b] >= 0: request b, which holds no rows,   */
/* takes over those of request source[b], which is no such request itself.  Its full pages are shared:    */
/* their ids go into b's block table row and shares[id], the number of a page's holders beyond the first,   */
/* grows by one.  A last page that is not full is b's own: a page from the top of the free list (requests    */
/* in order), whose contents csa2d_page_copy copies: src[b], dst[b] and rows[b] say from where, to where       */
/* and how many (-1, -1, 0: none).  lens[b] = lens[source[b]].                                                 */
/* Afterwards every request appends to pages of its own alone, so csa2p_page_plan serves them as before; but    */
/* it gives pages back without looking at shares: take rows back with it only down to the length at the fork,    */
/* and end requests that share pages with csa2d_page_free.                                                        */
/* A request that is its own source, holds rows already, or whose source is out of range or forked itself, is      */
/* left as it is (CSA2_DEV_BAD_INDEX); so is one that the free list has no page for (CSA2P_DEV_NO_PAGES) or whose    */
/* source has more rows than a table row reaches (CSA2P_DEV_TABLE_FULL); dst[b] is then -2.                           */
/* Table entries below 0 are taken over as they are; one at or past n_pages too (CSA2_DEV_BAD_INDEX): neither          */
/* counts as a page, shared or copied.                                                                                  */
/* ---------------------------------------------------------------------------------- */
typedef struct {
    int32_t batch;            /* requests, 0..CSA2P_MAX_BATCH                                    */
    int32_t page;             /* rows a page, a power of two, 1..65536                           */
    int32_t width;            /* block table entries a request, >= 1                             */
    int32_t n_pages;          /* entries of shares                                               */
    int32_t free_cap;         /* entries of free_pages                                           */
    const int32_t *source;    /* [batch] (page_fork)                                             */
    const int32_t *ends;      /* [batch] (page_free)                                             */
    int32_t *lens;            /* [batch] in and out                                              */
    int32_t *block_table;     /* [batch, width] in and out                                       */
    int32_t *shares;          /* [n_pages] in and out                                            */
    int32_t *free_pages;      /* [free_cap] in and out                                           */
    int32_t *n_free;          /* [1] in and out                                                  */
    int32_t *src, *dst, *rows;/* [batch] out (page_fork)                                         */
} csa2d_share_args;
CSA2_API csa2_status csa2d_page_fork(const csa2d_share_args *a, uint32_t *d_status, csa2_stream stream);

/* csa2d_page_free: requests with ends[b] != 0 end.  Each of their pages (entries 0 .. ceil(lens[b] /  */
/* page) - 1 of their table rows that name one) loses a holder; pages that have none left go on top of   */
/* the free list, lowest ids first, with shares 0.  lens[b] = 0; table entries stay as they were.  An      */
/* entry at or past n_pages sets CSA2_DEV_BAD_INDEX; pages that the free list has no room for set            */
/* CSA2P_DEV_TABLE_FULL and are lost.  The caller keeps shares >= 0 (0 for pages that csa2p_page_plan          */
/* handed out).                                                                                               */
CSA2_API csa2_status csa2d_page_free(const csa2d_share_args *a, uint32_t *d_status, csa2_stream stream);

/* csa2d_page_copy: in each cache the first rows[i] rows (rows NULL: all) of page src[i] go, as they are   */
/* stored, to page dst[i], i < count.  Pairs with a page below 0 are skipped; one with a page at or past a   */
/* cache's n_pages is skipped there and sets CSA2_DEV_BAD_INDEX.  rows is held to 0..page.  No dst may be      */
/* another pair's src or dst; caches must not share memory.                                                    */
CSA2_API csa2_status csa2d_page_copy(const csa2p_cache *caches, int32_t n, const int32_t *src, const int32_t *dst,
                                     const int32_t *rows, int32_t count, uint32_t *d_status, csa2_stream stream);

#ifdef __cplusplus
}
#endif
#endif /* CSA2_DRAFT_H */

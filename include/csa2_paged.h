/*
 * csa2_paged.h -- C ABI of the paged-cache calls of libcsa2.so (GB300, sm_103a).
 *
 * csa2.h's calls take caches laid out [B, N, d], one run of rows per sequence.  A server that
 * holds requests of unlike and growing lengths keeps each layer's rows in fixed-size pages
 * instead and finds them through block tables.  These calls are that form of one layer's
 * latent cache (all query heads share it, V = its leading d_v dims, as in csa2_sparse_attn):
 *
 *   csa2p_page_plan  block tables, slot map and free list from the requests' lengths
 *   csa2p_rope       rotary positions with one to three axes, on queries
 *   csa2p_write      new rows rotated, quantised and stored at their slots
 *   csa2p_read       rows by slot as bf16
 *   csa2p_attn       attention of new tokens (one, or a chunk, per request) over their pages
 *
 * csa2p_attn reads every visible row (or the last `window` of them): the layers that attend a
 * sliding window only, layers whose context is no longer than Top-K, and dense baselines.
 *
 * The conventions are csa2.h's: device pointers owned by the caller, work enqueued on `stream`,
 * no allocation, no synchronisation, errors found on the host returned before any launch,
 * errors found on the device ORed into *d_status (nullable) with every access in bounds.
 * Every kernel here waits for the kernel just before it on the stream before it reads any
 * input, and lets its dependents start their set-up right after that.  Calls on different
 * streams may run concurrently while their outputs and workspaces are disjoint; two captured
 * graphs that may run at the same time need workspaces of their own.  The calls work on the
 * current device, which has to be the one that holds the pointers.  Addresses of 32-bit values
 * are multiples of 4 (else INVALID_ARG, as with the alignments given below).
 */
#ifndef CSA2_PAGED_H
#define CSA2_PAGED_H

#include "csa2.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further device status bits (csa2.h's keep their meaning). */
#define CSA2P_DEV_NO_PAGES 0x100u   /* the free list ran out: table entries and slots -1         */
#define CSA2P_DEV_TABLE_FULL 0x200u /* a request outgrew its block table, or the free list its    */
                                    /* capacity                                                  */
#define CSA2P_DEV_ROWS 0x400u       /* more new rows than the slot map holds                     */

/* Row formats of a paged cache: the codecs of csa2.h (csa2_fp4_format, csa2_swa_format). */
typedef enum {
    CSA2P_MXFP4 = 0,        /* E2M1 codes, an E8M0 scale per 32: d/2 + d/32 bytes a row            */
    CSA2P_NVFP4_E4M3_16 = 1,/* E2M1 codes, an E4M3 scale per 16: d/2 + d/16 bytes a row            */
    CSA2P_MXFP8 = 2,        /* E4M3 codes, an E8M0 scale per 32: d + d/32 bytes a row              */
    CSA2P_BF16 = 3          /* bf16 values, no scales: 2 d bytes a row                             */
} csa2p_format;

/* One layer's pages.  Row `slot` lies in page slot / page at offset slot % page; its codes are at
 * codes + (slot / page) * code_stride + (slot % page) * (code bytes a row), scales likewise.     */
typedef struct {
    int32_t fmt;            /* csa2p_format                                                       */
    int32_t d;              /* channels a row: a multiple of 32, 32..1024                         */
    int32_t page;           /* rows a page: a power of two, 1..65536                              */
    int64_t n_pages;        /* pages; n_pages * page < 2^31                                       */
    void *codes;            /* 16-byte aligned                                                    */
    void *scales;           /* NULL for BF16; NVFP4: 2-byte aligned                               */
    int64_t code_stride;    /* bytes between pages (0: dense); a multiple of 16                   */
    int64_t scale_stride;   /* bytes between pages (0: dense); NVFP4: even                        */
} csa2p_cache;

/* ---------------------------------------------------------------------------------- */
/* csa2p_page_plan -- one step's bookkeeping on the GPU.  Request b held lens[b] rows;   */
/* delta[b] > 0 appends rows, delta[b] < 0 takes the last ones back (-lens[b]: the        */
/* request ends).  With had = ceil(lens/page) and has = ceil((lens+delta)/page):          */
/*   - pages has..had-1 of each shrinking request go on top of the free list (a stack     */
/*     whose n_free valid entries come first), requests in order, pages in order;         */
/*   - growing requests then take pages had..has-1 from its top, in the same order, into  */
/*     their block table rows (entries of pages given back stay as they were);            */
/*   - cu[b] = new rows of the requests before b, cu[batch] = all of them;                */
/*   - new row r = cu[b] + i is position lens[b] + i: row_req[r] = b, row_pos[r] = that   */
/*     position, slot[r] = block_table[b][pos / page] * page + pos % page.  Rows at and   */
/*     past cu[batch] get -1 in all three.                                                */
/* A page that the free list cannot supply is -1, and so are the slots in it             */
/* (CSA2P_DEV_NO_PAGES); positions past the table's width have slot -1 and take no page   */
/* (CSA2P_DEV_TABLE_FULL); rows past n_rows are dropped (CSA2P_DEV_ROWS).  A table entry  */
/* below 0 gives slot -1, and is passed over when its request gives it back.              */
/* lens below 0 counts as 0, lens + delta is held to 0..2^31-1.  lens_out may be lens and  */
/* n_free_out may be n_free: the call is replayed in a captured graph by updating delta    */
/* alone.                                                                                 */
/* ---------------------------------------------------------------------------------- */
#define CSA2P_MAX_BATCH 16384
typedef struct {
    int32_t batch;            /* requests, 0..CSA2P_MAX_BATCH                                    */
    int32_t page;             /* rows a page, a power of two, 1..65536                           */
    int32_t width;            /* block table entries a request, >= 1                             */
    int32_t free_cap;         /* entries of free_pages                                           */
    int32_t n_rows;           /* entries of slot, row_req and row_pos                            */
    const int32_t *lens;      /* [batch]                                                         */
    const int32_t *delta;     /* [batch]                                                         */
    int32_t *lens_out;        /* [batch] lens + delta                                            */
    int32_t *block_table;     /* [batch, width] in and out                                       */
    int32_t *free_pages;      /* [free_cap] in and out                                           */
    const int32_t *n_free;    /* [1]                                                             */
    int32_t *n_free_out;      /* [1]                                                             */
    int32_t *cu;              /* [batch + 1]                                                     */
    int32_t *slot;            /* [n_rows]                                                        */
    int32_t *row_req;         /* [n_rows] or NULL                                                */
    int32_t *row_pos;         /* [n_rows] or NULL                                                */
} csa2p_plan_args;
CSA2_API csa2_status csa2p_page_plan(const csa2p_plan_args *a, uint32_t *d_status, csa2_stream stream);

/* ---------------------------------------------------------------------------------- */
/* Rotary positions with several axes (text: one; images and video: time, height, width). */
/* The last rope_dim channels are turned in adjacent pairs, as in csa2_rope_quant_fp4;     */
/* pair i < section[0] takes the angle of position axis 0, the next section[1] pairs that  */
/* of axis 1, and so on (the sections add up to rope_dim / 2).  The angle's cosine and     */
/* sine are the caller's table row of that position:                                     */
/*   c = cos_sin[p * rope_dim + i], s = cos_sin[p * rope_dim + rope_dim/2 + i],            */
/*   p = pos[axis(i) * rows + row].                                                       */
/* A position below 0 (the plan's rows past the last token) turns nothing; one at or past  */
/* n_pos sets CSA2_DEV_BAD_INDEX and turns nothing.                                        */
/* ---------------------------------------------------------------------------------- */
typedef struct {
    int32_t rope_dim;         /* even, 0..d (0: no rotation, the rest unused)                    */
    int32_t n_axes;           /* 1..3                                                            */
    int32_t section[3];       /* pairs of each axis                                              */
    const int32_t *pos;       /* [n_axes, rows]                                                  */
    const float *cos_sin;     /* [n_pos, rope_dim] rope_dim/2 cosines, then the sines            */
    int64_t n_pos;
} csa2p_rope_axes;

/* csa2p_rope: x and out bf16 [rows, heads, d] with row and head strides in elements (multiples */
/* of 8, both 16-byte aligned); out = the rotated x, each value rounded to bf16 once.  out may   */
/* be x (with x's strides: only the turned channels are then touched); otherwise they must not   */
/* overlap, and out's own vectors never.  d % 8 == 0.                                             */
CSA2_API csa2_status csa2p_rope(const uint16_t *x, int64_t x_row, int64_t x_head, uint16_t *out, int64_t out_row,
                                int64_t out_head, int32_t rows, int32_t heads, int32_t d,
                                const csa2p_rope_axes *rope, uint32_t *d_status, csa2_stream stream);

/* csa2p_write: rows of x (bf16 [rows, d], row stride ldx elements, a multiple of 8, 16-byte     */
/* aligned), rotated in float32 with one rounding per product and per sum and then quantised     */
/* exactly as csa2_rope_quant_fp4 / csa2_quant_fp8 quantise (BF16: rounded once), go to           */
/* slot[row].  Slots below 0 are skipped; a slot at or past n_pages * page sets                   */
/* CSA2_DEV_BAD_INDEX and is skipped; non-finite values set CSA2_DEV_NONFINITE (not for BF16).    */
/* The slots >= 0 of one call have to be distinct: a slot given twice ends as a mixture of rows. */
CSA2_API csa2_status csa2p_write(const csa2p_cache *cache, const uint16_t *x, int64_t ldx, int32_t rows,
                                 const int32_t *slot, const csa2p_rope_axes *rope, uint32_t *d_status,
                                 csa2_stream stream);

/* csa2p_read: out row r (bf16, row stride ldo elements, a multiple of 8, 16-byte aligned) = the  */
/* values of cache row slot[r] (exact while they stay normal in bf16, else rounded once).  Rows    */
/* whose slot is below 0 are left as they were; a slot past the cache sets CSA2_DEV_BAD_INDEX and  */
/* leaves its row too.  A slot may be given any number of times.                                   */
CSA2_API csa2_status csa2p_read(const csa2p_cache *cache, const int32_t *slot, int32_t rows, uint16_t *out,
                                int64_t ldo, uint32_t *d_status, csa2_stream stream);

/* ---------------------------------------------------------------------------------- */
/* csa2p_attn -- attention of new tokens over a paged cache.  Request b's queries are the   */
/* tokens cu[b] .. cu[b+1]-1 of q (none: nothing to do); token t of them is at position     */
/* p = pos0[b] + t (pos0 NULL: pos0[b] = lens[b] - its tokens; ratio_m must then be 1).      */
/* Its keys are the request's rows                                                         */
/*   max(0, kv_start[b], e - window) <= j < min(lens[b], e),  e = floor((p + 1) / ratio_m)   */
/* (window 0: no lower bound from it; kv_start NULL: 0).  Row j is in page                   */
/* block_table[b][j / page].  Per head h, over d_qk = cache->d dims:                        */
/*   l_j = sm_scale * q_h . k_j,  out_h = sum_j softmax(l)_j k_j[0:d_v],  lse_h = log sum e^l */
/* A token without keys gets out = 0 and lse = -inf.  Tokens of q outside every request are  */
/* left as they were in out and lse.  Rows no query of a request sees are not read; a page    */
/* id outside [0, n_pages), or a row past the table's width, sets CSA2_DEV_BAD_INDEX and its   */
/* rows are no keys.  A cache row with a value or scale that is not finite makes the outputs   */
/* of the queries that see it NaN, and of no others; scale bytes that could take a value past    */
/* float32 (MXFP4 253 and up, MXFP8 247 and up: no quantised row has them) count as such.       */
/* The codes of all pages may span up to 64 GB and their scales up to 4 GB (else UNSUPPORTED).  */
/* Products are bf16 x bf16 with float32 sums; softmax weights are rounded to bf16 for the     */
/* second product, their sum is float32.  cu has to be non-decreasing: a call in which it        */
/* steps down between 0 and n_tokens, so that requests could share rows of q, sets               */
/* CSA2_DEV_BAD_INDEX and does nothing.  Tokens outside 0..n_tokens are left out; the    */
/* request's others keep their positions.                                                       */
/* ---------------------------------------------------------------------------------- */
typedef struct {
    csa2p_cache cache;
    int32_t batch;            /* requests, 0..CSA2P_MAX_BATCH                                    */
    int32_t n_tokens;         /* query tokens held by q                                          */
    int32_t n_heads;          /* 1..128                                                          */
    int32_t d_v;              /* 8..512, a multiple of 8, <= d_qk; d_qk <= 576                    */
    int32_t width;            /* block table entries a request                                   */
    int32_t window;           /* >= 0; 0: no window                                              */
    int32_t ratio_m;          /* tokens an entry stands for, >= 1                                */
    float sm_scale;           /* above 0, at most 2.3e38                                         */
    const uint16_t *q;        /* bf16 [n_tokens, n_heads, d_qk], 16-byte aligned                 */
    const int32_t *block_table; /* [batch, width]                                                */
    const int32_t *lens;      /* [batch] rows held, the new tokens' included                     */
    const int32_t *cu;        /* [batch + 1]                                                     */
    const int32_t *pos0;      /* [batch] or NULL                                                 */
    const int32_t *kv_start;  /* [batch] or NULL                                                 */
} csa2p_attn_args;
/* Workspace: parts of rows whose keys are split over the GPU.  Its size depends on d_v and on the  */
/* current device; its contents need no preparation.  The size is 0 for a call that csa2p_attn     */
/* would refuse or that has nothing to do, pointers that are NULL or misaligned included: to size a */
/* workspace before the tensors exist, give any aligned addresses in their place (nothing is read). */
CSA2_API size_t csa2p_attn_workspace_size(const csa2p_attn_args *a);
CSA2_API csa2_status csa2p_attn(const csa2p_attn_args *a, uint16_t *out, float *lse, void *ws, size_t ws_bytes,
                                uint32_t *d_status, csa2_stream stream);

#ifdef __cplusplus
}
#endif
#endif /* CSA2_PAGED_H */

/*
 * mla_cache.h — C ABI of the operators around the paged latent cache: rotary
 * positions, the write of new rows, the cache in 8 bits and decode attention
 * over it, and the fork, free, copy and compaction of its pages.
 *
 * The cache is the one mla_decode.h describes: a pool of pages of 64 tokens,
 * a row of 576 values per token (512 latent + 64 RoPE), int32 block tables
 * [batch][max_blocks_per_seq] and lengths [batch].  A pool is held in one of
 * two forms:
 *   MLA_CACHE_BF16  bf16 [num_blocks][64][1][576] (what mla_decode_fwd reads)
 *   MLA_CACHE_E4M3  e4m3 [num_blocks][64][1][576] with kv_scales fp32
 *                   [num_blocks][1]: one scale per block of 64 tokens and KV
 *                   head (the latent cache has one head); a value is
 *                   scale * e4m3 (what mla_decode_q8_fwd reads)
 *
 * The conventions of mla_decode.h hold for every entry point: device pointers
 * owned by the caller, 16-byte aligned unless a line says otherwise; work is
 * enqueued on `stream` of the current device; nothing is allocated and nothing
 * waits for the device; arguments are checked before anything is enqueued; the
 * return value is MLA_OK or a negative MLA_ERR_* code (mla_decode_strerror
 * names it).  `status`, where a call takes one, is an optional device int32
 * (NULL or 4-byte aligned) into which the kernels OR MLA_STATUS_* bits of
 * faults in device-side data; the offending entry is skipped and nothing is
 * read or written out of range.  The caller clears it.
 */
#ifndef MLA_CACHE_H_
#define MLA_CACHE_H_

#include "mla_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MLA_CACHE_BF16 0
#define MLA_CACHE_E4M3 1

/* further device status bits */
#define MLA_STATUS_BAD_ROW 0x20        /* a row index outside the batch, a row named twice, a fork onto a row in use, or
                                          new rows that do not fit their request's length */
#define MLA_STATUS_NO_FREE_PAGE 0x40   /* the pool had too few free pages */
#define MLA_STATUS_BAD_REF_COUNT 0x80  /* a page in use had a count of 0 */

/* ------------------------------------------------------------------------
 * Rotary positions.  A rotary table holds the 32 angular frequencies of the
 * 64 RoPE columns, computed on the host in 64 bits:
 *   none    f_i = theta^(-2i/64)
 *   linear  f_i / factor
 *   yarn    f_i (1 - r_i) + f_i / factor r_i,  r_i = clamp((i - low) / (high - low), 0, 1),
 *           low / high = the dimension whose wavelength turns beta_fast / beta_slow
 *           times within original_max_position, rounded down / up
 *           (YaRN, arXiv 2309.00071, section 3.2)
 * and the amplitude the rotated values are multiplied by (1, or YaRN's
 * attention factor).  Pair i is rotated by the angle position * f_i, which is
 * reduced in 64 bits, so far positions lose nothing:
 *   interleaved layout  pair i = columns (2i, 2i + 1)
 *   half layout         pair i = columns (i, i + 32)
 *   (a, b) -> amplitude * (a cos - b sin, a sin + b cos)
 * ---------------------------------------------------------------------- */
#define MLA_ROPE_NONE 0
#define MLA_ROPE_LINEAR 1
#define MLA_ROPE_YARN 2

typedef struct mla_rope_config {
    double theta;                  /* base, > 1 */
    double factor;                 /* > 0; linear and yarn (so small that 2^31 f_i is no number: refused) */
    double beta_fast, beta_slow;   /* yarn: > 0 */
    double amplitude;              /* finite as fp32 */
    int32_t original_max_position; /* yarn: >= 1 */
    int32_t scaling;               /* MLA_ROPE_* */
    int32_t interleaved;           /* 1: pairs (2i, 2i+1); 0: pairs (i, i + 32) */
    int32_t reserved;              /* must be 0 */
} mla_rope_config;

typedef struct mla_rope_table {
    double turns[32];    /* f_i / 2 pi */
    float amplitude;
    int32_t interleaved;
} mla_rope_table;

/* Fills *table on the host; no CUDA call. */
int mla_rope_init(const mla_rope_config* config, mla_rope_table* table);

#define MLA_DTYPE_BF16 0
#define MLA_DTYPE_FP32 1

typedef struct mla_rope_dims {
    int32_t tokens;      /* T >= 0 (0: nothing to do) */
    int32_t num_heads;   /* h, 1 .. 65535 */
    int32_t width;       /* values per head row, 64 .. 2048, a multiple of 8 */
    int32_t offset;      /* first of the 64 rotary columns, a multiple of 8, offset + 64 <= width */
    int64_t x_token_stride, x_head_stride;      /* of x, in values: multiples of 8 */
    int64_t out_token_stride, out_head_stride;  /* of out, likewise */
    int32_t dtype;       /* MLA_DTYPE_* of x and out */
    int32_t transpose;   /* 1: rotate by the opposite angle, which is the transposed map: the gradient
                            of x from the gradient of out */
} mla_rope_dims;

/* out[t][h][:] = x[t][h][:] with its rotary columns rotated for positions[t]
 * (device int32 [T], 4-byte aligned, any value).  Computed in fp32 and rounded
 * once.  out may be x itself with the same strides: then only the rotary columns
 * are written.  Otherwise they must not overlap, and every column of a row is
 * written.  The rows of out must not overlap one another (MLA_ERR_INVALID_ARG
 * where the strides say they do). */
int mla_rope_apply(const mla_rope_dims* dims, const mla_rope_table* table, const void* x, const int32_t* positions,
                   void* out, void* stream);

/* ------------------------------------------------------------------------
 * The write of new rows into the cache.  Request b's new rows are rows
 * [new_offsets[b], new_offsets[b+1]) of c_kv and k_pe, and become the last
 * n_b = new_offsets[b+1] - new_offsets[b] positions of its cache_seqlens[b]
 * (the length including them): row i goes to position
 * cache_seqlens[b] - n_b + i, through block_table, as [c_kv | RoPE(k_pe)].
 *   c_kv          bf16 [tokens][512], row stride c_stride values (a multiple of 8)
 *   k_pe          bf16 [tokens][64], row stride pe_stride values (a multiple of 8)
 *   new_offsets   device int32 [batch + 1], 4-byte aligned, from 0, not falling
 *   table         rotary table for the positions, or NULL: k_pe is rotated already
 * Columns are computed in fp32 and rounded once, to bf16 or e4m3.
 *
 * MLA_CACHE_E4M3: the new rows of one page decide its scale, the least power
 * of two 2^e (2^-100 .. 2^119) with every finite |value| <= 448 * 2^e; finite values
 * above 448 * 2^119 (2.98e38) are stored as that, the largest value a page holds.  A page
 * that already holds earlier rows keeps its scale if that is larger; else
 * those rows are moved to the new scale: their exponents shift, and only
 * values that fall below 2^-6 of the new scale are rounded again.  A page's
 * scale depends on the rows it has held and not on how many calls wrote them,
 * except for that rounding.  Values that are not finite are stored as NaN.
 * Rows of the page behind the new ones are left as they were.
 *
 * Every page that is written must belong to one request alone (mla_cache_fork
 * keeps that so).  A request whose new rows do not fit (n_b < 0, n_b >
 * cache_seqlens[b], a length past max_blocks_per_seq pages, offsets past
 * tokens) is skipped whole with MLA_STATUS_BAD_ROW, rows of a page whose block-table
 * entry is outside the pool are skipped with MLA_STATUS_BAD_BLOCK_TABLE; the other
 * requests are written.
 * The kernel lets no dependent grid start before its writes are done, so a
 * decode call may follow it on the stream.
 * ---------------------------------------------------------------------- */
typedef struct mla_cache_dims {
    int32_t batch;               /* rows of the block table, >= 1 */
    int32_t max_blocks_per_seq;  /* >= 1 */
    int32_t num_blocks;          /* pages in the pool, >= 1 */
    int32_t page_size;           /* must be 64 */
    int32_t row_width;           /* must be 576 */
    int32_t dtype;               /* MLA_CACHE_* */
} mla_cache_dims;

int mla_cache_append(const mla_cache_dims* dims, int32_t tokens, const void* c_kv, int64_t c_stride, const void* k_pe,
                     int64_t pe_stride, const int32_t* new_offsets, const mla_rope_table* table,
                     const int32_t* block_table, const int32_t* cache_seqlens, void* kv_cache, float* kv_scales,
                     int32_t* status, void* stream);

/* ------------------------------------------------------------------------
 * Pages.  The pool's books are the block table, the lengths and ref_counts,
 * device int32 [num_blocks]: how many table rows hold a page (0: free).  Row b
 * holds its first ceil(cache_seqlens[b] / 64) entries.  Books and pool change
 * in place; entries behind a row's pages stay as they were.  Calls on one pool
 * have to be ordered (one stream, or events).
 * ---------------------------------------------------------------------- */

/* For i < n (1 .. 1024): row children[i], which must be empty, becomes a copy
 * of row parents[i]: it shares the parent's full pages (their counts rise), and
 * a last page that is not full is copied (with its scale) into the lowest free
 * page, in the order of i, so that both rows may be written on.  Parents are
 * taken as they are before the call: one that is a child of the same call is empty
 * then, and so is its child.  A fork that
 * cannot be made (MLA_STATUS_BAD_ROW; _NO_FREE_PAGE; _BAD_BLOCK_TABLE, or _BAD_REF_COUNT
 * where the count is not above 0, for its last page) leaves its child empty; a bad
 * entry among the full pages is copied as it is, with that word (and a page's count
 * rises).  The counts alone say which other pages are free.  parents and children are device int32 [n], 4-byte
 * aligned; workspace is mla_cache_fork_workspace_bytes(n) bytes. */
size_t mla_cache_fork_workspace_bytes(int32_t n);
int mla_cache_fork(const mla_cache_dims* dims, int32_t n, const int32_t* parents, const int32_t* children,
                   int32_t* block_table, int32_t* cache_seqlens, int32_t* ref_counts, void* kv_cache, float* kv_scales,
                   void* workspace, int32_t* status, void* stream);

/* Gives up the pages of rows[0 .. n): each page's count falls by one, the
 * rows' entries become -1 and their lengths 0.  A row that is empty, or named
 * twice, is freed once. */
int mla_cache_free(const mla_cache_dims* dims, int32_t n, const int32_t* rows, int32_t* block_table,
                   int32_t* cache_seqlens, int32_t* ref_counts, int32_t* status, void* stream);

/* kv_cache page dst[i] = page src[i] (and its scale) for i < n.  Destinations
 * must differ from one another and from every source.  An index outside the
 * pool skips its pair: a negative src without a word, others with
 * MLA_STATUS_BAD_BLOCK_TABLE. */
int mla_cache_copy_pages(const mla_cache_dims* dims, int32_t n, const int32_t* src, const int32_t* dst, void* kv_cache,
                         float* kv_scales, int32_t* status, void* stream);

/* Moves the pages in use to the front of the pool: with `live` pages in use,
 * the k-th of those at or behind `live` goes to the k-th free one before it.
 * Rewrites the rows' entries, the counts and the scales.  The table is looked through first: a page that
 * a row holds although its count is not above 0 (MLA_STATUS_BAD_REF_COUNT) is kept and
 * moved like one in use, with a count of 0; a length past the table or below 0
 * (MLA_STATUS_BAD_SEQLEN) is taken as the nearest possible one; an entry outside the pool
 * (MLA_STATUS_BAD_BLOCK_TABLE) stays as it is.  workspace is
 * mla_cache_compact_workspace_bytes(dims) bytes; its first int32 is `live`
 * afterwards. */
size_t mla_cache_compact_workspace_bytes(const mla_cache_dims* dims);
int mla_cache_compact(const mla_cache_dims* dims, int32_t* block_table, const int32_t* cache_seqlens,
                      int32_t* ref_counts, void* kv_cache, float* kv_scales, void* workspace, int32_t* status,
                      void* stream);

/* ------------------------------------------------------------------------
 * Decode attention over the 8-bit cache: the operation, the arguments, the
 * flags, the split-KV plan and the status word of mla_decode.h, with
 *   kv_cache   e4m3 [num_blocks][64][1][576]
 *   kv_scales  fp32 [num_blocks][1], positive and finite; those of one request within
 *              2^220 of each other (any that mla_cache_append writes are).  A scale that
 *              is 0, negative or NaN is read as 2^-100
 * The schedule and workspace sizes come from the two _bytes calls below, and
 * the plan from these get_schedule calls (the query groups are 16 or 32
 * columns wide).  MLA_FLAG_INLINE_PLAN builds the plan in the decode kernel up
 * to 24,528 requests (above that the call enqueues the schedule kernel).
 *
 * The cache's bytes are multiplied as they are; neither the query nor the
 * softmax weights are rounded to 8 bits: a query value is within 2^-21 of its
 * row's largest magnitude (rows whose largest is 2^-92 or more), and a weight is
 * held in 11 bits, within 2^-12 of itself, or its product with its page's scale is
 * within 2^-22 of the row's largest such product.  That holds for fp32 results too.
 * Rows past a request's length, and its last page's unused rows, may hold
 * anything.  A NaN in a row that one query token sees reaches every query token
 * of its request.
 * The pages of a row, kv_scales and the lengths must be final when the grid
 * before the call lets its dependents start (MLA_FLAG_INLINE_PLAN).
 * ---------------------------------------------------------------------- */
size_t mla_decode_q8_schedule_bytes(const mla_decode_dims* dims);
size_t mla_decode_q8_workspace_bytes(const mla_decode_dims* dims);
int mla_decode_q8_get_schedule(const mla_decode_dims* dims, const int32_t* cache_seqlens, void* schedule, void* stream);
int mla_decode_q8_get_schedule_host(const mla_decode_dims* dims, const int32_t* cache_seqlens_host, void* schedule_host);
int mla_decode_q8_fwd(const mla_decode_dims* dims, void* schedule, void* workspace, const void* q, const void* kv_cache,
                      const float* kv_scales, const int32_t* block_table, const int32_t* cache_seqlens,
                      float softmax_scale, void* out, float* lse, void* stream);
int mla_decode_q8_combine(const mla_decode_dims* dims, const void* schedule, const void* workspace, void* out, float* lse,
                          void* stream);

/* ABI version of this header. */
int mla_cache_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MLA_CACHE_H_ */

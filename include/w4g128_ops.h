/*
 * w4g128_ops -- the operators that stand around the weight stream in a decode
 * or verify step: the mixture-of-experts layer on packed int4-g128 experts,
 * rotating and appending to a paged cache of bf16 or 8 bits, attention of a few
 * new tokens over either, penalties and masks on logits, and token sampling.
 * (Token Rush README: the step is captured whole, with attention "over the
 * live length", sampling and the token fed back on the device; progress table
 * steps 4 and 13-14.)  Same conventions as w4g128.h: device pointers owned by
 * the caller, nothing allocated, calls asynchronous on `stream`, argument
 * errors returned before anything is launched, results bitwise deterministic.
 * A workspace must not be used by two calls that can run at the same time,
 * on two streams or in two captured graphs.
 */
#ifndef W4G128_OPS_H
#define W4G128_OPS_H

#include "w4g128.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Status-word code of the operators on a paged cache: a length, a row offset or a page id in
 * device memory lies outside what the arguments allow. */
#define W4G128_ERR_CACHE 9

/* ------------------------------------------------------------------------
 * SAMPLING
 *
 * One token per row from bf16 logits (the output of an lm_head product) and a
 * given random number u.  Tokens are ordered by falling logit, the lower
 * index first among equals (-0 equals +0), and weighted
 *   w_i = exp((logit_i - largest logit) / temperature).
 * Three filters each keep a prefix of that order, and at least its first
 * token: the first top_k tokens; of those, the tokens whose predecessors' sum
 * is below top_p times the sum of the top_k; the tokens with w_i >= min_p.
 * The token is the first one kept whose sum of weights, itself included,
 * exceeds u times the kept sum; its log-probability among the kept tokens is
 * log(w_i / kept sum).  Logits of -inf and NaN are never chosen.  A row
 * without any other gets token -1 and log-probability -inf.  If the largest
 * logit is +inf, the +inf tokens weigh 1 and all others 0.
 *
 * The weights are carried as 62-bit fractions of the largest and summed
 * exactly, so the token is the one that the formulas give in about 1e-13
 * relative precision, whatever the order of the sums. */
typedef struct {
  const w4g128_bf16* logits; /* row r at logits + r * row_stride; 2-byte aligned */
  long long row_stride;      /* elements, >= vocab */
  const float* temperature;  /* [rows], or NULL: 1.  Not above 0 (or NaN): the largest logit is taken (top_k = 1) */
  const int* top_k;          /* [rows], or NULL: no limit.  Not above 0: no limit */
  const float* top_p;        /* [rows], or NULL: 1.  1 and above (or NaN): no limit */
  const float* min_p;        /* [rows], or NULL: 0.  0 and below (or NaN): no limit */
  const float* u;            /* [rows], in [0, 1); taken as 0 below it (or NaN), as the last fraction below 1 above it */
  int* tokens;               /* [rows] */
  float* logprobs;           /* [rows], or NULL */
  int rows;                  /* 1 .. W4G128_MAX_SAMPLE_ROWS */
  int vocab;                 /* 1 .. W4G128_MAX_VOCAB */
} w4g128_sample_args;

#define W4G128_MAX_SAMPLE_ROWS 4096
#define W4G128_MAX_VOCAB 524160

/* Samples every row.  Needs no workspace.  The arrays named by `args` are
 * device memory and are read and written when the call runs; `args` itself is
 * host memory and is read during the call.  Returns W4G128_ERR_INVALID_ARG
 * (null logits, u or tokens; rows out of range), W4G128_ERR_SHAPE (vocab out
 * of range, row_stride below vocab), W4G128_ERR_ALIGN (logits 2 bytes, the
 * other arrays 4). */
W4G128_API int w4g128_sample(const w4g128_sample_args* args, void* stream);

/* ------------------------------------------------------------------------
 * ATTENTION OF NEW TOKENS OVER A PAGED CACHE
 *
 * For each of `count` sequences, the attention of its 0 .. max_new (at most
 * 16) newest tokens over everything the sequence has in a paged key/value
 * cache, the new tokens themselves included: a decode step (one token), or
 * the verify step of a draft.  Sequence b owns the rows row_offsets[b] ..
 * row_offsets[b + 1] - 1 of q, k_new, v_new and out, n of them; lens[b] is its
 * length with them, so its row i stands at position p = lens[b] - n + i and
 *   out[h] = sum_j softmax_j(scale q[h] . k_j[h / (q_heads / kv_heads)]) v_j
 * over the positions j <= p with p - j < window (window = 0: all) or
 * j < sinks.  Position j of sequence b is slot j % page_size of page
 * page_table[b][j / page_size].  First the new rows' k_new and v_new are
 * written to their places (k_new = v_new = NULL: they are there already); the
 * call itself reads them from k_new and v_new, not from the cache.
 *
 * A row at a negative position (more rows than the length) sees nothing: its
 * out is 0 and its key and value are not written.  So is the out of a row all of
 * whose scores are -inf.  Rows of no sequence are left as they are.  The places
 * of the new rows differ from one another and from every other position's that
 * the call sees: sequences may share the pages of a common prefix, not a page
 * that one of them extends.  Pages that no row of a sequence sees are not read, and
 * their table entries may hold anything.  Masked positions take no part in a
 * row's result whatever they hold, infinities and NaN included.
 *
 * Row m's bits depend on its own position, query and visible keys and values
 * alone, not on the other rows of the call nor on max_new, given the same
 * count, kv_heads, head_dim, max_len, window and sinks: a verify pass
 * reproduces the one-token steps (the split of a sequence into fixed chunks of
 * positions follows from those arguments).  Scores, the softmax statistics and the
 * output are held in fp32; the softmax weights enter the second product
 * rounded to bf16 and are summed as rounded, so they add up to 1. */
typedef struct {
  const w4g128_bf16* q;     /* row r, head h at r * q_row + h * head_dim */
  const w4g128_bf16* k_new; /* row r, head h at r * kv_row + h * head_dim; or NULL, with v_new */
  const w4g128_bf16* v_new;
  w4g128_bf16* k_cache;     /* page g, slot s, head h at g * page_stride + s * slot_stride + h * head_stride */
  w4g128_bf16* v_cache;     /* the same strides */
  const int* page_table;    /* sequence b at b * table_row; ceil(max_len / page_size) entries */
  const int* row_offsets;   /* [count + 1], rising, within 0 .. rows */
  const int* lens;          /* [count], 0 .. max_len */
  w4g128_bf16* out;         /* row r, head h at r * out_row + h * head_dim */
  long long q_row, kv_row, out_row;                  /* elements, as all strides */
  long long page_stride, slot_stride, head_stride;
  long long table_row;
  int rows;      /* of q, k_new, v_new and out: 1 .. 2^20 */
  int count;     /* sequences, 1 .. W4G128_MAX_SEQUENCES */
  int q_heads;   /* a multiple of kv_heads, at most 16 times as many */
  int kv_heads;  /* 1 .. 256 */
  int head_dim;  /* 64, 128 or 256 */
  int pages;     /* pages of the cache */
  int page_size; /* a multiple of 16 */
  int max_len;   /* the longest length that the table can hold, 1 .. 2^24.  Sizes the split and the workspace: far above
                    the lengths it costs time (one token at 4096, 8 heads of 128: 6.9 us at 4096, 26 us at 131072) */
  int max_new;   /* most new rows of a sequence, 1 .. 16 */
  int window;    /* 0: none */
  int sinks;     /* first positions that stay visible behind the window; 0 without a window */
  float scale;   /* finite, and so is scale log2(e): up to 2.35e38 either way */
} w4g128_attend_args;

#define W4G128_MAX_SEQUENCES 1024

/* Workspace bytes of w4g128_attend for these sizes: a status word and the
 * fp32 partial results of each chunk.  0 for arguments it would refuse. */
W4G128_API size_t w4g128_attend_workspace_bytes(const w4g128_attend_args* args);

/* The attention above.  q, k_new, v_new, the caches and out: 16-byte aligned,
 * their strides multiples of 8 elements; the int arrays 4 bytes; ws 16.  out
 * must overlap nothing else.  lens, row_offsets and the table are read on the
 * device, so a captured call follows them from replay to replay.  A sequence
 * whose length or row range lies outside the bounds above is left out, and a
 * page id outside 0 .. pages - 1 counts as a page whose cached positions no row
 * sees and takes no new rows (they are seen from k_new and v_new); both leave
 * W4G128_ERR_CACHE in the workspace's status word, until the next call on it
 * (w4g128_workspace_status).  Returns W4G128_ERR_INVALID_ARG,
 * W4G128_ERR_SHAPE, W4G128_ERR_ALIGN or W4G128_ERR_WORKSPACE for what breaks
 * the bounds above. */
W4G128_API int w4g128_attend(const w4g128_attend_args* args, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * MIXTURE OF EXPERTS
 *
 * The whole feed-forward layer of E experts for M rows (1 .. W4G128_MAX_M),
 * each expert's three projections in the packed int4-g128 format:
 *   logit[m][e] = sum_d x[m][d] router[e][d]                        (fp32)
 *   S(m)        = the top_k experts of the largest logits, the lower one
 *                 first among equals (a NaN logit ranks last)
 *   p[m][e]     = exp(logit[m][e]) / sum exp(logit[m][e']), the sum over S(m)
 *                 (renormalize = 1) or over all experts (renormalize = 0)
 *   a[m][e][f]  = r( silu(g_f) u_f ), (g, u) = x[m] . dequant(gate_up_e)
 *   y[m][n]     = bf16( residual[m][n] + sum_{e in S(m)} p[m][e] (a[m][e] . dequant(down_e))[n] )
 * with fp32 products, sums and softmax, silu(g) = g / (1 + exp(-g)); the codes
 * enter the sums with a bias of 1024, which every group's own sum undoes.  The
 * activations a are the operand of the second product and rounded for it (to
 * fp16, scaled by the largest of 16 neighbours and then of the row and expert): r
 * errs by at most 2^-11 of a and 2^-38 of the row's and expert's largest.  x
 * enters the first product exactly down to 2^-31 of its row's largest; smaller
 * values err by at most 2^-39 of that.  An infinity in a row's x or activations
 * makes the row NaN.  Only the experts that some row picks are read: once, and a
 * second time, from the L2 where it still holds them, if more than 8 rows pick
 * one.
 *
 * gate_up_e is a K = D, N = 2 F matrix (F gate columns, then F up columns),
 * down_e a K = F, N = D one, each packed as w4g128_pack writes it; the E
 * matrices follow one another without gaps, expert e at e *
 * w4g128_packed_bytes(K, N).  Row m of y depends on row m of x and residual
 * alone and is bitwise the same whatever M and the other rows are. */
typedef struct {
  const w4g128_bf16* x;        /* [M][D] */
  const w4g128_bf16* residual; /* [M][D], or NULL: 0.  May be y */
  w4g128_bf16* y;              /* [M][D]; not x */
  const w4g128_bf16* router;   /* [E][D] */
  const void* gate_up;         /* E packed matrices, K = D, N = 2 F */
  const void* down;            /* E packed matrices, K = F, N = D */
  int M;
  int D;           /* a multiple of 128, 128 .. 65536 */
  int F;           /* a multiple of 128, 128 .. 65536 */
  int E;           /* 1 .. W4G128_MAX_EXPERTS */
  int top_k;       /* 1 .. min(E, W4G128_MAX_TOP_K) */
  int renormalize; /* 0 or 1 */
} w4g128_moe_args;

#define W4G128_MAX_EXPERTS 512
#define W4G128_MAX_TOP_K 16

/* Workspace bytes of w4g128_moe for these sizes (status word, logits, the
 * experts' activations and outputs).  0 for arguments it would refuse. */
W4G128_API size_t w4g128_moe_workspace_bytes(const w4g128_moe_args* args);

/* The layer above.  All pointers and ws 16-byte aligned.  Returns
 * W4G128_ERR_INVALID_ARG (null pointers, M, top_k or renormalize out of
 * range, y = x), W4G128_ERR_SHAPE, W4G128_ERR_ALIGN, W4G128_ERR_WORKSPACE.
 * The kernels wait for one another by launch order alone; the status word
 * reads W4G128_OK after the call. */
W4G128_API int w4g128_moe(const w4g128_moe_args* args, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * ROTATED QUERIES AND KEYS, APPENDED TO A PAGED CACHE
 *
 * For each of `count` sequences its newest 0 .. max_new tokens (a decoded
 * token, a draft, or a whole prompt), in the layout of w4g128_attend: rows
 * row_offsets[b] .. row_offsets[b + 1] - 1, the last of them at position
 * lens[b] - 1.  The first rot_dim values of every head of q and k_new are
 * rotated by the row's position p: pair i, (x_i, x_(i + rot_dim / 2)) or
 * interleaved (x_2i, x_(2i + 1)), turns by the angle p freqs[i],
 *   (a, b) -> (a cos - b sin, b cos + a sin).
 * The angle is reduced in 64-bit integers of 2^-64 turns, so far positions cost
 * no precision.  The rotated queries go to q_out, the rotated keys and the
 * values to their pages: position j of sequence b to slot j % page_size of page
 * page_table[b][j / page_size].
 *
 * A cache of bf16 (block = 0) holds each value rounded once.  A cache of 8 bits
 * holds e4m3 codes, the value a code stands for is code times the scale of its
 * block and head; a block is `block` neighbouring slots of a page.  Of the keys'
 * or values' block that new rows go to, let top be their largest finite
 * magnitude.  If the block has positions before the new rows and top is at most
 * 448 times its scale, the scale stays; otherwise it becomes
 * 2^max(floor(log2 top) - 5, -100) (above every earlier one that does not fit),
 * and those earlier positions' codes are rounded to it, which is exact down to
 * 2^-6.  Codes are rounded to nearest, ties to even; what is not finite (a
 * rotated value beyond fp32's range is not) is a NaN code.  The 5 leaves new rows
 * of a block room of a factor 7 to 14 before it changes.  A key whose exact value
 * lies within 2^-21 of its pair's size of the middle between two codes may become
 * either.  With block = 1 a row's codes are its own; with larger blocks they also
 * follow the rows that share the block, and a draft row that is rejected leaves the
 * scale as it needed it.
 *
 * Rows at negative positions and of no sequence are left as they are, in q_out
 * too, and so are the slots behind a sequence's length. */
typedef struct {
  const w4g128_bf16* q;     /* row r, head h at r * q_row + h * head_dim; or NULL: no queries (then q_out is NULL) */
  w4g128_bf16* q_out;       /* row r, head h at r * q_out_row + h * head_dim; may be q, with the same stride */
  const w4g128_bf16* k_new; /* row r, head h at r * kv_row + h * head_dim */
  const w4g128_bf16* v_new;
  void* k_cache;            /* page g, slot s, head h at g * page_stride + s * slot_stride + h * head_stride */
  void* v_cache;            /* the same strides; bf16, or e4m3 codes where block > 0 */
  float* k_scale;           /* page g, head h, block i of the page at g * scale_page + h * scale_head + i; NULL where block = 0 */
  float* v_scale;           /* the same strides */
  const double* freqs;      /* [rot_dim / 2] radians a position, finite; NULL where rot_dim = 0 */
  const int* page_table;    /* sequence b at b * table_row; ceil(max_len / page_size) entries */
  const int* row_offsets;   /* [count + 1], rising, within 0 .. rows */
  const int* lens;          /* [count], 0 .. max_len, the new tokens included */
  long long q_row, q_out_row, kv_row;                /* elements, as all strides */
  long long page_stride, slot_stride, head_stride;
  long long scale_page, scale_head;
  long long table_row;
  int rows;        /* of q, q_out, k_new and v_new: 1 .. 2^20 */
  int count;       /* sequences, 1 .. W4G128_MAX_SEQUENCES */
  int q_heads;     /* 1 .. 4096; 0 without queries */
  int kv_heads;    /* 1 .. 256 */
  int head_dim;    /* 64, 128 or 256 */
  int rot_dim;     /* a multiple of 16, 0 .. head_dim */
  int interleaved; /* 0 or 1 */
  int pages;       /* pages of the cache */
  int page_size;   /* a multiple of 16 */
  int block;       /* 0, or a power of two up to 64 that divides page_size */
  int max_len;     /* the longest length that the table can hold, 1 .. 2^24 */
  int max_new;     /* most new rows of a sequence, 1 .. 2^20.  Where `rows` has room for count * max_new, the work is shared
                      out as if all had max_new; uneven batches are faster with fewer rows (a prompt of 8191 beside 63
                      single tokens: 37 us into bf16 and 48 into blocks of 16, with room for all 272 and 1352) */
} w4g128_append_args;

/* Workspace bytes of w4g128_append: a status word.  0 for arguments it would refuse. */
W4G128_API size_t w4g128_append_workspace_bytes(const w4g128_append_args* args);

/* The call above, in one launch.  q, q_out, k_new, v_new and the caches: 16-byte
 * aligned, their strides multiples of 8 elements (16 in a cache of codes);
 * freqs 8 bytes; the int arrays and scales 4; ws 16.  Nothing that is written
 * overlaps anything else, but q_out q.  The places of the new rows differ from
 * one another.  lens, row_offsets and the table are read on the device.  A
 * sequence whose length or row range lies outside the bounds above is left out,
 * new rows whose page id is outside 0 .. pages - 1 are not cached (their queries
 * are rotated); both leave W4G128_ERR_CACHE in the workspace's status word, until
 * the next call on it.  Returns W4G128_ERR_INVALID_ARG, W4G128_ERR_SHAPE,
 * W4G128_ERR_ALIGN or W4G128_ERR_WORKSPACE for what breaks the bounds above. */
W4G128_API int w4g128_append(const w4g128_append_args* args, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * ATTENTION OF NEW TOKENS OVER A PAGED CACHE OF 8 BITS
 *
 * w4g128_attend over a cache of e4m3 codes and scales as w4g128_append writes it
 * (or another program, with any normal positive scales; a value's below 2^-80
 * counts as 2^-80):
 *   out[h] = sum_j softmax_j(scale q[h] . k_j) v_j,  k_j, v_j = code * scale of the block,
 * over the same positions.  The new tokens' keys and values are in the cache
 * already.  Scores, softmax statistics and sums are held in fp32.  Codes enter
 * the products as fp16, exactly; q as fp16 scaled by its row's and head's largest
 * value, exactly down to 2^-31 of that; the softmax weights times the values'
 * scales rounded to fp16: by 2^-11 of their value, or 2^-31 of the row's largest.
 * That holds while |scale| times a row's and head's largest |q| times a visible key's
 * scale is up to 2^140; beyond, a score may pass fp32's range and the row become NaN.
 * The sum of weights is of their fp32 values, whatever the scales are; beside a
 * value's scale above 2^100 weights below 2^-28 of that sum may be left out of it.
 *
 * Row m's bits depend on its own position, query and visible codes and scales
 * alone, not on the other rows of the call nor on max_new, given the same count,
 * kv_heads, head_dim, max_len, window and sinks.  A row at a negative position, or
 * all of whose scores are -inf, has out 0.  Rows of no sequence are left as they
 * are.  Masked positions take no part whatever their codes and scales hold. */
typedef struct {
  const w4g128_bf16* q;     /* row r, head h at r * q_row + h * head_dim */
  const void* k_cache;      /* e4m3 codes: page g, slot s, head h at g * page_stride + s * slot_stride + h * head_stride */
  const void* v_cache;      /* the same strides */
  const float* k_scale;     /* page g, head h, block i of the page at g * scale_page + h * scale_head + i */
  const float* v_scale;     /* the same strides */
  const int* page_table;    /* sequence b at b * table_row; ceil(max_len / page_size) entries */
  const int* row_offsets;   /* [count + 1], rising, within 0 .. rows */
  const int* lens;          /* [count], 0 .. max_len */
  w4g128_bf16* out;         /* row r, head h at r * out_row + h * head_dim */
  long long q_row, out_row;                          /* elements, as all strides */
  long long page_stride, slot_stride, head_stride;
  long long scale_page, scale_head;
  long long table_row;
  int rows;      /* of q and out: 1 .. 2^20 */
  int count;     /* sequences, 1 .. W4G128_MAX_SEQUENCES */
  int q_heads;   /* a multiple of kv_heads, at most 16 times as many */
  int kv_heads;  /* 1 .. 256 */
  int head_dim;  /* 64, 128 or 256 */
  int pages;     /* pages of the cache */
  int page_size; /* a multiple of 16 */
  int block;     /* slots that share a scale: a power of two up to 64 that divides page_size */
  int max_len;   /* the longest length that the table can hold, 1 .. 2^24.  Sizes the split and the workspace: far above
                    the lengths it costs time (one token at 611, 8 heads of 128: 4.8 us at 624, 6.3 from 4096 on; 16
                    sequences of up to 9001, 4 heads of 64: 18.9 us at 9008, 44 at 131072) */
  int max_new;   /* most new rows of a sequence, 1 .. 16 */
  int window;    /* 0: none */
  int sinks;     /* first positions that stay visible behind the window; 0 without a window */
  float scale;   /* |scale| up to 2^14 */
} w4g128_attend8_args;

/* Workspace bytes of w4g128_attend8 for these sizes: a status word and, where several CTAs share a
 * sequence and head, their partial results in fp32.  0 for arguments it would refuse. */
W4G128_API size_t w4g128_attend8_workspace_bytes(const w4g128_attend8_args* args);

/* The attention above.  q, the caches and out: 16-byte aligned, q_row and out_row
 * multiples of 8 elements, the caches' strides of 16; the int arrays and scales 4
 * bytes; ws 16.  out must overlap nothing else.  Lengths, rows and the table are
 * read, and errors in them reported, as by w4g128_attend. */
W4G128_API int w4g128_attend8(const w4g128_attend8_args* args, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * PENALTIES, BIASES AND MASKS ON LOGITS
 *
 * What w4g128_sample's rows need before the draw.  Row r has a history of tokens,
 * history[history_start[r]] .. + history_len[r] - 1, whose first prompt_len[r]
 * are the prompt and the others its answer so far (rows of one verify step point
 * into one buffer, each with a token more).  With c_t the times that token t
 * occurs in the answer, in this order, in fp32:
 *   z = logit_t;  if t occurs in the history, z = z / repetition (z > 0) or z * repetition;
 *   z = z - frequency * c_t;  if c_t > 0, z = z - presence;
 *   z = z + bias of t, where the row's list names t (the last entry, if several do);
 *   out_t = bf16(z), or -inf where the mask forbids t.
 * Tokens outside 0 .. vocab - 1 in histories and lists are ignored.  Infinite
 * logits stay as they are under finite settings, NaN stays NaN unless masked. */
typedef struct {
  const w4g128_bf16* logits; /* row r at logits + r * row_stride; 2-byte aligned */
  w4g128_bf16* out;          /* row r at out + r * out_stride; may be logits, with the same stride */
  const int* history;        /* [history_size], or NULL: no histories */
  const long long* history_start; /* [rows], or NULL: 0 */
  const int* history_len;    /* [rows], up to 2^30; not above 0: none.  NULL with history NULL alone */
  const int* prompt_len;     /* [rows], or NULL: 0 */
  const float* repetition;   /* [rows], 2^-100 .. 2^100, or NULL: 1; divided by as multiplied by its inverse */
  const float* presence;     /* [rows], or NULL: 0 */
  const float* frequency;    /* [rows], or NULL: 0 */
  const int* bias_tokens;    /* [bias_size]: row r's entries are bias_offsets[r] .. bias_offsets[r + 1] - 1; or NULL: none */
  const float* bias_values;  /* [bias_size]; NULL with bias_tokens */
  const int* bias_offsets;   /* [rows + 1]; may be there without bias_tokens */
  const unsigned* mask;      /* row r at mask + r * mask_row: bit t % 32 of word t / 32 is 1 where t is allowed; or NULL: all */
  long long row_stride, out_stride; /* elements, >= vocab */
  long long mask_row;        /* words, >= ceil(vocab / 32) (or 0: one mask for all rows) */
  long long history_size;    /* elements; what lies outside is not read */
  int bias_size;             /* elements; what lies outside is not read, nor more than the first 65535 of a row */
  int rows;                  /* 1 .. W4G128_MAX_SAMPLE_ROWS */
  int vocab;                 /* 1 .. W4G128_MAX_VOCAB */
} w4g128_penalize_args;

/* Needs no workspace.  logits and out 2-byte aligned, history_start 8, the other
 * arrays 4.  All arrays are device memory, read when the call runs.  out overlaps
 * nothing else, but may be logits.  Returns W4G128_ERR_INVALID_ARG (null logits or
 * out; histories or lists of which only a part is there; rows, history_size or
 * bias_size out of range; out = logits with another stride), W4G128_ERR_SHAPE
 * (vocab out of range, a stride too small), W4G128_ERR_ALIGN. */
W4G128_API int w4g128_penalize(const w4g128_penalize_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W4G128_OPS_H */

/*
 * ccb_kv8.h -- a key/value cache held in 8 bits, and the operators of a
 * decoding step on it (libccb.so): append, attention, eviction by
 * accumulated attention weight, and read.
 *
 * The cache.  Pages of pageSize tokens; every page holds one block of each
 * head, and every block has one scale, so that
 *     value[page][head][slot][d] = code[page][head][slot][d] * scale[page][head]
 * with codes in int8 (largest Q = 127) or OCP e4m3 (largest Q = 448).  A page
 * table gives each sequence its pages in order: token t of sequence b is slot
 * t % pageSize of page pageTable[b][t / pageSize].  lens[b] is the number of
 * tokens that sequence b holds.  weight[b][head][t], where kept, is the
 * attention weight that token t has drawn so far.  All of it is device memory
 * of the caller's; pages may be handed out in any order.
 *
 * A decoding step: the caller adds the number of new tokens to lens[b], then
 * calls ccb_kv8_append (which fills the last tokens) and ccb_kv8_attend, and
 * now and then ccb_kv8_evict.  Every call only enqueues kernels, allocates
 * nothing and reads no device memory on the host, so all of them can be
 * captured into a HIP graph (kernel nodes only).  The conventions of ccb.h
 * hold: a ccbStatus is returned, arguments are checked before anything is
 * enqueued, and calls act on the calling thread's current device.  A call whose
 * work does not fit a launch (of the order of 2^24 blocks of a page's head, or
 * 2^23 runs of tokens with 16 rows) gets CCB_ERR_INVALID_VALUE.
 *
 * Errors found on the device.  `err` (device, one int32, may be NULL) gets
 * CCB_ERR_INVALID_VALUE stored when a call meets a page number outside 0 ..
 * numPages - 1, a length outside 0 .. maxPages * pageSize, or a count outside
 * 0 .. min(nNew, lens[b]); it is never cleared.  Nothing is read or written
 * out of range then: a sequence with a bad length or count counts as empty
 * (for ccb_kv8_append: is left alone), the tokens of a bad page count as
 * unseen (attention), as zeros (read, evict) or are dropped (append).  A bad
 * page of evict's `to` is left out, and `lens` counts its tokens all the same.
 *
 * Contents past lens[b], and pages that no sequence uses, may hold any bytes
 * (NaN codes and NaN scales among them) and reach no result.  Within a
 * sequence the scales are finite and not negative, and no e4m3 code is NaN
 * (0x7F, 0xFF): ccb_kv8_append and ccb_kv8_evict write none.
 */
#ifndef CCB_KV8_H
#define CCB_KV8_H

#include "ccb.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Code formats. */
enum { CCB_KV8_INT8 = 0, CCB_KV8_E4M3 = 1 };

/* Element types of the rows that come in and go out. */
enum { CCB_KV8_BF16 = 0, CCB_KV8_FP16 = 1, CCB_KV8_FP32 = 2 };

typedef struct ccbKv8Cache {
    void* k;                  /* codes [numPages][heads][pageSize][headDim], 16-B aligned */
    void* v;                  /* the same */
    float* kScale;            /* [numPages][heads] */
    float* vScale;            /* the same */
    const int32_t* pageTable; /* [batch][tableStride], the first maxPages of each row in use */
    int32_t* lens;            /* [batch] */
    float* weight;            /* [batch][heads][weightStride], or NULL */
    int64_t tableStride;      /* >= maxPages */
    int64_t weightStride;     /* >= maxPages * pageSize (ignored without weight) */
    int32_t format;           /* CCB_KV8_INT8 or CCB_KV8_E4M3 */
    int32_t numPages;
    int32_t heads;            /* heads of the cache */
    int32_t pageSize;         /* 16, 32, 64 or 128 */
    int32_t headDim;          /* 64, 96, 128, 192 or 256 */
    int32_t batch;
    int32_t maxPages;         /* maxPages * pageSize <= 2^30 */
    int32_t reserved;         /* 0 */
} ccbKv8Cache;

/* Rows [batch][token][head][headDim] with any strides (in elements); the
 * headDim elements of a row lie side by side.  data is 16-B aligned and every
 * stride a multiple of 8 elements. */
typedef struct ccbKv8Rows {
    void* data;
    int64_t strideBatch;
    int64_t strideToken;
    int64_t strideHead;
    int32_t type; /* CCB_KV8_BF16 or CCB_KV8_FP16; CCB_KV8_FP32 only for ccb_kv8_read */
    int32_t reserved;
} ccbKv8Rows;

/* Write new tokens.  Sequence b's c = counts[b] (counts NULL: nNew) new
 * tokens are tokens lens[b] - c .. lens[b] - 1: lens already counts them.
 * Per page and head that gets new tokens, with a the largest finite |x| among
 * them:
 *   s1 = a / Q rounded to float, at least 2^-64 when a > 0;
 *   s0 = 0 when the page's first slot is new, else the block's scale;
 *   the block's scale becomes s = max(s0, s1);
 *   a new code is x / s rounded once to the format (half to even), saturated
 *   at +-Q; NaN becomes 0 and an infinity +-Q;
 *   where s > s0 the block's older tokens become code * s0 / s, rounded once;
 *   s = 0 makes every code of the new tokens 0.
 * Older tokens' codes stay as they are where the scale does not grow, so a
 * call made twice changes nothing the second time.  weight (when kept) is set
 * to 0 for the new tokens.
 *   kNew, vNew  [batch][nNew][heads][headDim]
 *   counts      device int32 [batch], or NULL
 * Errors: NULL_POINTER, INVALID_VALUE (a cache or rows that break the rules
 * above, nNew < 0 or > maxPages * pageSize), UNSUPPORTED_DEVICE, HIP. */
CCB_API ccbStatus ccb_kv8_append(const ccbKv8Cache* cache, const ccbKv8Rows* kNew,
                                 const ccbKv8Rows* vNew, int32_t nNew, const int32_t* counts,
                                 int32_t* err, ccbStream stream);

/* Attention of nQuery queries per sequence (its last nQuery tokens) over the
 * cache.  Query head j reads cache head j / (headsQ / heads).  With n =
 * lens[b], query i sees token t when t <= n - nQuery + i and, for window > 0,
 * t > n - nQuery + i - window.  Over the tokens seen:
 *   s_t = scale * q . k_t,  m = max s_t,  l = sum exp(s_t - m),
 *   out = sum exp(s_t - m) v_t / l,  lse = m + ln l;
 * a query that sees nothing (an empty sequence, or i < nQuery - n) gets out =
 * 0 and lse = -infinity.  Products q k are exact, sums are kept in 32 bits, a
 * weight times its block's scale enters the sum of values within 2^-18 of
 * itself, and out is rounded once to its type.  accumulate != 0 adds to weight[b][head][t]
 * the sum of exp(s_t - lse) over the queries and the query heads of that head.
 * Results do not depend on timing: the same call gives the same bits.
 *   q, out  [batch][nQuery][headsQ][headDim], of one type.  out may be q itself
 *           (the same data and strides) and overlaps it in no other way; but not
 *           where accumulate needs the queries again after out is written: with
 *           R = headsQ / heads * nQuery rows for a cache head, where R > 64, or
 *           R > 16 and 4 * batch * heads * R * maxPages * pageSize > 2^25.
 *   lse     device float [batch][nQuery][headsQ], or NULL
 *   ws      device, ccb_kv8_attend_workspace_bytes(...) bytes, 128-B aligned,
 *           whatever it holds.  Calls that overlap in time need their own.
 * Errors: NULL_POINTER (also accumulate without weight), INVALID_VALUE (as
 * above; headsQ not a multiple of heads, nQuery or window < 0, more than 2^20 rows
 * (headsQ / heads * nQuery), a scale that is not finite, out over q as above, a
 * workspace too small), UNSUPPORTED_DEVICE, HIP. */
CCB_API ccbStatus ccb_kv8_attend(const ccbKv8Cache* cache, const ccbKv8Rows* q,
                                 const ccbKv8Rows* out, float* lse, int32_t headsQ, int32_t nQuery,
                                 float scale, int32_t window, int32_t accumulate, void* ws,
                                 size_t wsBytes, int32_t* err, ccbStream stream);

/* Bytes of ccb_kv8_attend's workspace, whatever the window (0 for arguments it
 * refuses).  It goes by the capacity, not by the lengths: with R as above,
 * headDim + 2 floats for R rows of each run of tokens, of which there are at most
 * max(4096, batch * heads), and with accumulate 4 * batch * heads * R * maxPages *
 * pageSize bytes for R <= 16 (and R <= 64 while that is at most 2^25): 1.1 GB for
 * 64 sequences of 131072 tokens with 8 heads and 4 rows each. */
CCB_API size_t ccb_kv8_attend_workspace_bytes(const ccbKv8Cache* cache, int32_t headsQ,
                                              int32_t nQuery, int32_t accumulate);

/* Copy the tokens worth keeping into other pages.  For every sequence and
 * head of `from`, with n = lens[b] and n' = min(n, budget): all tokens when n
 * <= budget; else the first `sinks`, the last `recent`, and of the tokens
 * between those with the largest weight until there are n' (equal weights:
 * the lower token first; a NaN ranks below every number).  In the order of
 * their tokens they become tokens 0 .. n' - 1 of sequence b in `to`, each head
 * with its own choice.  A new block's scale is the largest float(|code| * s)
 * of its tokens divided by Q and rounded to float (at least 2^-64 unless it
 * is 0), and its codes are code * s_old / s_new rounded once to the format
 * (half to even).  Writes to->lens[b] = n', to->weight (when kept: the kept
 * tokens' weights, then 0 up to budget) and kept.  `from` is only read.
 * `to` has the format, heads, headDim, pageSize and batch of `from` and room
 * for budget tokens; it may share the pools of `from`, but its pages, lens
 * and weight are not those of `from` (a page that several sequences share
 * stays whole that way).
 *   kept  device int32 [batch][heads][budget]: the kept tokens' numbers in
 *         `from`, then -1; or NULL
 *   ws    device, ccb_kv8_evict_workspace_bytes(...) bytes, 128-B aligned,
 *         whatever it holds.  Calls that overlap in time need their own.
 * Errors: NULL_POINTER (also from->weight), INVALID_VALUE (as above; budget <
 * 1, recent or sinks < 0, recent + sinks > budget, a workspace too small),
 * UNSUPPORTED_DEVICE, HIP. */
CCB_API ccbStatus ccb_kv8_evict(const ccbKv8Cache* from, const ccbKv8Cache* to, int32_t budget,
                                int32_t recent, int32_t sinks, int32_t* kept, void* ws,
                                size_t wsBytes, int32_t* err, ccbStream stream);

/* Bytes of ccb_kv8_evict's workspace (0 for arguments it refuses). */
CCB_API size_t ccb_kv8_evict_workspace_bytes(const ccbKv8Cache* from, int32_t budget);

/* The values of tokens first[b] .. first[b] + count - 1 (first NULL: from 0)
 * as dense rows: code * scale as float, rounded once to the rows' type;
 * zeros for places outside 0 .. lens[b] - 1.
 *   kOut, vOut  [batch][count][heads][headDim], either may be NULL
 *   first       device int32 [batch], or NULL
 * Errors: NULL_POINTER, INVALID_VALUE, UNSUPPORTED_DEVICE, HIP. */
CCB_API ccbStatus ccb_kv8_read(const ccbKv8Cache* cache, const ccbKv8Rows* kOut,
                               const ccbKv8Rows* vOut, int32_t count, const int32_t* first,
                               int32_t* err, ccbStream stream);

#ifdef __cplusplus
}
#endif

#endif /* CCB_KV8_H */

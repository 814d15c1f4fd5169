/*
 * ccb_kv4.h -- a key/value cache held in 4 bits, and the operators of a
 * decoding step on it (libccb.so): append by a slot map, attention, and read.
 *
 * The cache.  Pages of pageSize tokens, as in ccb_kv8.h, with codes in e2m1
 * (sign, 2 exponent bits, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two to
 * a byte, and one e8m0 scale for each 32 dimensions of a token and head (the
 * OCP microscaling format MXFP4, 4.25 bits a value):
 *     value[page][head][slot][d] = code * 2^(scale[page][head][slot][d / 32] - 127)
 * Dimension d is in byte d / 2, the even one in the low half.  Tokens share no
 * scale, so that writing one never touches another.  The page table and lens
 * are those of ccb_kv8.h; ccb_pages.h makes them, and the slot maps, on the
 * GPU.  All of it is device memory of the caller's; pages may be handed out in
 * any order.
 *
 * Every call only enqueues kernels, allocates nothing and reads no device
 * memory on the host, so all of them can be captured into a HIP graph (kernel
 * nodes only).  The conventions of ccb.h hold.  A call whose work does not fit
 * a launch (2^32 threads) gets CCB_ERR_INVALID_VALUE.
 *
 * Errors found on the device.  `err` (device, one int32, may be NULL) gets
 * CCB_ERR_INVALID_VALUE stored when a call meets a page number outside 0 ..
 * numPages - 1, a length outside 0 .. maxPages * pageSize, or a slot outside
 * -1 .. numPages * pageSize - 1; it is never cleared.  Nothing is read or
 * written out of range then: a sequence with a bad length counts as empty, the
 * tokens of a bad page count as unseen (attention) or as zeros (read), a row
 * with a bad slot is dropped.
 *
 * Contents past lens[b], and pages that no sequence uses, may hold any bytes
 * and reach no result.  Within a sequence no scale is 255 (NaN);
 * ccb_kv4_append writes 63 to 252.  Values of 2^128 and more, which only scales of
 * 253 and 254 make, are infinite: within a sequence no value is one for
 * ccb_kv4_attend (it would reach queries that do not see it, as a NaN).
 */
#ifndef CCB_KV4_H
#define CCB_KV4_H

#include "ccb_kv8.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ccbKv4Cache {
    uint8_t* k;               /* codes [numPages][heads][pageSize][headDim / 2], 16-B aligned */
    uint8_t* v;               /* the same */
    uint8_t* kScale;          /* [numPages][heads][pageSize][headDim / 32], 16-B aligned */
    uint8_t* vScale;          /* the same */
    const int32_t* pageTable; /* [batch][tableStride], the first maxPages of each row in use */
    const int32_t* lens;      /* [batch] */
    int64_t tableStride;      /* >= maxPages */
    int32_t numPages;         /* numPages * heads * pageSize < 2^32 (more than the card's memory holds) */
    int32_t heads;            /* heads of the cache, 1 .. 65536 */
    int32_t pageSize;         /* 16, 32, 64 or 128 */
    int32_t headDim;          /* 64, 96, 128, 192 or 256 */
    int32_t batch;
    int32_t maxPages;         /* maxPages * pageSize <= 2^30 */
} ccbKv4Cache;

/* Write new tokens: row i of kNew and vNew becomes the token at slots[i] (page
 * slots[i] / pageSize, slot slots[i] % pageSize); a row with slot -1 is left
 * out (and every row, where the cache's batch is 0).  For each head and each 32
 * dimensions of a row, with a the largest finite |x| among them: e is the least
 * whole number with a <= 7 * 2^e, at least -64 and at most 125; the scale is
 * e + 127; a code is x / 2^e rounded once to e2m1 (half to even), saturated at
 * +-6 (with this e nothing that is finite is off by more than half a step, but
 * for values above 7 * 2^125 and below 2^-66); NaN becomes 0 and an infinity
 * +-6.
 * Two rows of one call should not have the same slot: which of them each 8
 * dimensions and each scale are from is not defined then.
 *   kNew, vNew  [nNew][heads][headDim], bf16 or fp16 (strideBatch is not used)
 *   slots       device int64 [nNew]
 * Errors: NULL_POINTER, INVALID_VALUE (a cache or rows that break the rules
 * above, nNew < 0 or > 2^30), UNSUPPORTED_DEVICE, HIP. */
CCB_API ccbStatus ccb_kv4_append(const ccbKv4Cache* cache, const ccbKv8Rows* kNew,
                                 const ccbKv8Rows* vNew, int32_t nNew, const int64_t* slots,
                                 int32_t* err, ccbStream stream);

/* Attention of nQuery queries per sequence (its last nQuery tokens) over the
 * cache.  Query head j reads cache head j / (headsQ / heads).  With n =
 * lens[b], query i sees token t when t <= n - nQuery + i and, for window > 0,
 * t > n - nQuery + i - window.  Over the tokens seen:
 *   s_t = scale * q . k_t,  m = max s_t,  l = sum exp(s_t - m),
 *   out = sum exp(s_t - m) v_t / l,  lse = m + ln l;
 * a query that sees nothing (an empty sequence, or i < nQuery - n) gets out =
 * 0 and lse = -infinity.  Products q k are exact, sums are kept in 32 bits, a
 * weight enters the sum of values within 2^-18 of itself, and out is rounded
 * once to its type.  Weights are relative to a maximum that later scores may
 * have passed by a factor of 2^8: where that and the number of tokens take the
 * values past 2^128 (|v| >= 2^90 at the most tokens there can be) a sum may be
 * infinite.  Scores beyond the largest float are infinite: +infinity makes its
 * query's results NaN, and -infinity counts as unseen.  Results do not depend on timing: the same call gives the same bits.
 *   q, out  [batch][nQuery][headsQ][headDim], of one type.  out may be q itself
 *           (the same data and strides) and overlaps it in no other way.
 *   lse     device float [batch][nQuery][headsQ], or NULL
 *   ws      device, ccb_kv4_attend_workspace_bytes(...) bytes, 128-B aligned,
 *           whatever it holds.  Calls that overlap in time need their own.
 * Errors: NULL_POINTER, INVALID_VALUE (as above; headsQ not a multiple of heads,
 * nQuery or window < 0, more than 2^20 rows (headsQ / heads * nQuery), a scale
 * that is not finite, a workspace too small), UNSUPPORTED_DEVICE, HIP. */
CCB_API ccbStatus ccb_kv4_attend(const ccbKv4Cache* cache, const ccbKv8Rows* q,
                                 const ccbKv8Rows* out, float* lse, int32_t headsQ, int32_t nQuery,
                                 float scale, int32_t window, void* ws, size_t wsBytes,
                                 int32_t* err, ccbStream stream);

/* Bytes of ccb_kv4_attend's workspace, whatever the window (0 for arguments it
 * refuses).  It goes by the capacity, not by the lengths: headDim + 2 floats for
 * each of headsQ / heads * nQuery rows of each run of tokens, of which there are
 * at most batch * heads + 4096, and 8 bytes for every 16 of its rows. */
CCB_API size_t ccb_kv4_attend_workspace_bytes(const ccbKv4Cache* cache, int32_t headsQ,
                                              int32_t nQuery);

/* The values of tokens first[b] .. first[b] + count - 1 (first NULL: from 0)
 * as dense rows: code * 2^(scale - 127) as float, rounded once to the rows'
 * type; zeros for places outside 0 .. lens[b] - 1.
 *   kOut, vOut  [batch][count][heads][headDim], either may be NULL
 *   first       device int32 [batch], or NULL
 * Errors: NULL_POINTER, INVALID_VALUE, UNSUPPORTED_DEVICE, HIP. */
CCB_API ccbStatus ccb_kv4_read(const ccbKv4Cache* cache, const ccbKv8Rows* kOut,
                               const ccbKv8Rows* vOut, int32_t count, const int32_t* first,
                               int32_t* err, ccbStream stream);

#ifdef __cplusplus
}
#endif

#endif /* CCB_KV4_H */

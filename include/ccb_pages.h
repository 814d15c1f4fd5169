/*
 * ccb_pages.h -- the pages of a paged key/value cache, handed out and taken
 * back on the GPU (libccb.so): page tables and the slot map of a step's new
 * tokens from the sequences' lengths, with nothing read by the host.
 *
 * A pool keeps the numbers of its free pages as a stack: free[0 .. count - 1],
 * the top last.  A page table gives each sequence its pages in order: token t
 * of sequence b lies in page pages[b][t / pageSize], at slot t % pageSize; its
 * place among all slots is pages[b][t / pageSize] * pageSize + t % pageSize.
 * lens[b] is the number of tokens that sequence b holds, which are in its first
 * ceil(lens[b] / pageSize) pages; entries behind them mean nothing and stay as
 * they are.  All of it is device memory of the caller's; the tables serve
 * ccb_kv8.h and ccb_kv4.h alike.
 *
 * A step: ccb_pages_trim takes back what sequences that ended (or drafted
 * tokens that were rejected) held, ccb_pages_grow gives every sequence the
 * pages of its new tokens and says where each of them goes.  Every call only
 * enqueues one kernel, allocates nothing and reads no device memory on the
 * host, so that a whole step can be captured into a HIP graph.  Results do not
 * depend on timing.  Calls on one pool, and on one table, follow each other.
 * The conventions of ccb.h hold.
 *
 * Errors found on the device.  `err` (device, one int32, may be NULL) gets
 * CCB_ERR_INVALID_VALUE stored when a call meets a length outside 0 ..
 * maxPages * pageSize, a count of free pages outside 0 .. numPages, or what is
 * named at the calls; it is never cleared.  Nothing is read or written out of
 * range then.
 */
#ifndef CCB_PAGES_H
#define CCB_PAGES_H

#include "ccb.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Sequences that a call takes (larger tables go in several calls). */
#define CCB_PAGES_MAX_BATCH 8192

/* Bytes of a pool's state. */
#define CCB_PAGES_STATE_BYTES 2176

typedef struct ccbPagePool {
    int32_t* free;    /* [numPages], the first *count of them in use */
    int32_t* count;   /* one: free pages */
    int32_t* state;   /* CCB_PAGES_STATE_BYTES, 128-B aligned: zeros before the pool's first
                       * call, and after each */
    int32_t numPages; /* 1 .. 2^30 - 1 */
    int32_t pageSize; /* a power of two, 1 .. 32768 */
} ccbPagePool;

typedef struct ccbPageTable {
    int32_t* pages;   /* [batch][stride], the first maxPages of each row in use */
    int32_t* lens;    /* [batch] */
    int64_t stride;   /* >= maxPages */
    int32_t batch;    /* 0 .. CCB_PAGES_MAX_BATCH */
    int32_t maxPages; /* maxPages * pageSize <= 2^30 */
} ccbPageTable;

/* Where a step's new tokens go, packed: sequence after sequence. */
typedef struct ccbSlotMaps {
    int64_t* slots;     /* [tokens]: a token's slot among all, or -1 */
    int32_t* positions; /* [tokens]: its place in its sequence, or -1 */
    int32_t* sequences; /* [tokens]: its sequence, or -1 behind the last token */
    int32_t* starts;    /* [batch + 1]: the first token of each sequence, then their number */
    int32_t* granted;   /* [batch]: the tokens that the sequence got room for */
    int32_t tokens;     /* room for new tokens, 0 .. 2^30 - 1 */
    int32_t reserved;   /* 0 */
} ccbSlotMaps;          /* the first three 16-B aligned; each may be NULL */

/* Cut sequences: lens[b] becomes min(lens[b], keep[b]) (a negative keep[b]
 * leaves it), and the pages behind ceil(lens[b] / pageSize) go back onto the
 * stack: those of the last sequence first, a sequence's last page first, so that
 * a trim that undoes a grow leaves the stack as it was before.
 * A sequence with a bad length is left alone.  Where the stack would pass
 * numPages (pages given back twice) nothing is done, and err set.  A page number
 * outside 0 .. numPages - 1 goes back as -1, and err is set.
 *   keep  device int32 [batch]
 * Errors: NULL_POINTER, INVALID_VALUE (sizes outside the ranges above, bad
 * alignment), UNSUPPORTED_DEVICE, HIP. */
CCB_API ccbStatus ccb_pages_trim(const ccbPagePool* pool, const ccbPageTable* table,
                                 const int32_t* keep, int32_t* err, ccbStream stream);

/* Give sequences room: with n = lens[b] and c = counts[b], sequence b needs
 * ceil((n + c) / pageSize) - ceil(n / pageSize) pages more.  First come, first
 * served: sequence b gets them, from the top of the stack and in order, if the
 * stack holds what all sequences up to b need together (one that needs none
 * always has room); then lens[b] becomes n + c.  Else nothing of it changes,
 * granted[b] is 0 and its tokens' slots and positions are -1; that is no error.
 * The new tokens are numbered sequence after sequence, starts[b] = counts[0] +
 * .. + counts[b - 1], those that got no room too; `maps` says for each of them
 * where it goes.  Numbers that starts[batch] .. tokens - 1 stand for get -1.
 * A negative count is taken as 0.  A sequence with a bad length, a negative
 * count, n + c > maxPages * pageSize, or tokens numbered past maps->tokens
 * needs nothing, gets no room and sets err; starts stops at maps->tokens.  A
 * token in a page whose number is outside 0 .. numPages - 1 gets the slot -1,
 * and err is set.
 *   counts  device int32 [batch]
 * Errors: NULL_POINTER, INVALID_VALUE (as above; reserved), UNSUPPORTED_DEVICE,
 * HIP. */
CCB_API ccbStatus ccb_pages_grow(const ccbPagePool* pool, const ccbPageTable* table,
                                 const int32_t* counts, const ccbSlotMaps* maps, int32_t* err,
                                 ccbStream stream);

#ifdef __cplusplus
}
#endif

#endif /* CCB_PAGES_H */

// ccb_kv4_api.hip -- the C entry points of the 4-bit key/value cache
// (include/ccb_kv4.h): argument checks and launches.  Kernels live in
// ccb_kv4_cache.hip and ccb_kv4_attend.hip.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ccb_kv4_internal.h"

namespace {

using ccb::aligned;

constexpr size_t kLeastWorkspace = 128;
constexpr int64_t kMaxTokens = 1 << 30;  // of one sequence

ccbStatus check_cache(const ccbKv4Cache* c)
{
    if (c == nullptr) return CCB_ERR_NULL_POINTER;
    if (c->pageSize != 16 && c->pageSize != 32 && c->pageSize != 64 && c->pageSize != 128)
        return CCB_ERR_INVALID_VALUE;
    if (c->headDim != 64 && c->headDim != 96 && c->headDim != 128 && c->headDim != 192 &&
        c->headDim != 256)
        return CCB_ERR_INVALID_VALUE;
    if (c->numPages < 1 || c->heads < 1 || c->heads > 65536 || c->batch < 0 || c->maxPages < 1 ||
        (int64_t)c->maxPages * c->pageSize > kMaxTokens || c->tableStride < c->maxPages ||
        (int64_t)c->numPages > (int64_t)UINT32_MAX / ((int64_t)c->heads * c->pageSize))
        return CCB_ERR_INVALID_VALUE;
    if (c->batch == 0) return CCB_OK;
    if (c->k == nullptr || c->v == nullptr || c->kScale == nullptr || c->vScale == nullptr ||
        c->pageTable == nullptr || c->lens == nullptr)
        return CCB_ERR_NULL_POINTER;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->kScale, 16) || !aligned(c->vScale, 16) ||
        !aligned(c->pageTable, 4) || !aligned(c->lens, 4))
        return CCB_ERR_INVALID_VALUE;
    return CCB_OK;
}

ccbStatus check_rows(const ccbKv8Rows* r, bool allow32)
{
    if (r == nullptr || r->data == nullptr) return CCB_ERR_NULL_POINTER;
    if (r->type != CCB_KV8_BF16 && r->type != CCB_KV8_FP16 &&
        !(allow32 && r->type == CCB_KV8_FP32))
        return CCB_ERR_INVALID_VALUE;
    if (!aligned(r->data, 16) || r->strideBatch % 8 != 0 || r->strideToken % 8 != 0 ||
        r->strideHead % 8 != 0 || r->reserved != 0)
        return CCB_ERR_INVALID_VALUE;
    return CCB_OK;
}

bool attend_sizes_ok(const ccbKv4Cache* c, int32_t headsQ, int32_t nQuery)
{
    return headsQ >= 1 && headsQ % c->heads == 0 && nQuery >= 0 &&
           (int64_t)(headsQ / c->heads) * nQuery <= (1 << 20);
}

}  // namespace

extern "C" {

CCB_API ccbStatus ccb_kv4_append(const ccbKv4Cache* cache, const ccbKv8Rows* kNew,
                                 const ccbKv8Rows* vNew, int32_t nNew, const int64_t* slots,
                                 int32_t* err, ccbStream stream)
{
    ccbStatus st = check_cache(cache);
    if (st != CCB_OK) return st;
    if (nNew < 0 || nNew > kMaxTokens || !aligned(slots, 8) || !aligned(err, 4)) return CCB_ERR_INVALID_VALUE;
    if (cache->batch == 0 || nNew == 0) return CCB_OK;
    if (slots == nullptr) return CCB_ERR_NULL_POINTER;
    if ((st = check_rows(kNew, false)) != CCB_OK) return st;
    if ((st = check_rows(vNew, false)) != CCB_OK) return st;
    if (kNew->type != vNew->type || !ccb::kv4_append_fits(*cache, nNew)) return CCB_ERR_INVALID_VALUE;
    if ((st = ccb::device_ready()) != CCB_OK) return st;
    return ccb::launch_status(ccb::kv4_append(*cache, *kNew, *vNew, nNew, slots, err, (hipStream_t)stream));
}

CCB_API size_t ccb_kv4_attend_workspace_bytes(const ccbKv4Cache* cache, int32_t headsQ,
                                              int32_t nQuery)
{
    if (check_cache(cache) != CCB_OK || !attend_sizes_ok(cache, headsQ, nQuery)) return 0;
    const size_t n = ccb::kv4_attend_bytes(*cache, headsQ, nQuery);
    return n < kLeastWorkspace ? kLeastWorkspace : n;
}

CCB_API ccbStatus ccb_kv4_attend(const ccbKv4Cache* cache, const ccbKv8Rows* q,
                                 const ccbKv8Rows* out, float* lse, int32_t headsQ, int32_t nQuery,
                                 float scale, int32_t window, void* ws, size_t wsBytes,
                                 int32_t* err, ccbStream stream)
{
    ccbStatus st = check_cache(cache);
    if (st != CCB_OK) return st;
    if (!attend_sizes_ok(cache, headsQ, nQuery) || window < 0 || !isfinite(scale))
        return CCB_ERR_INVALID_VALUE;
    if (!aligned(lse, 4) || !aligned(err, 4) || !aligned(ws, CCB_LINE_BYTES))
        return CCB_ERR_INVALID_VALUE;
    if (cache->batch == 0 || nQuery == 0) return CCB_OK;
    if ((st = check_rows(q, false)) != CCB_OK) return st;
    if ((st = check_rows(out, false)) != CCB_OK) return st;
    if (q->type != out->type) return CCB_ERR_INVALID_VALUE;
    if (q->data == out->data &&  // in place: row by row
        ((cache->batch > 1 && q->strideBatch != out->strideBatch) ||
         (nQuery > 1 && q->strideToken != out->strideToken) ||
         (headsQ > 1 && q->strideHead != out->strideHead)))
        return CCB_ERR_INVALID_VALUE;
    if (ws == nullptr) return CCB_ERR_NULL_POINTER;
    if (wsBytes < kLeastWorkspace || !ccb::kv4_attend_fits(*cache, headsQ, nQuery, window, wsBytes))
        return CCB_ERR_INVALID_VALUE;
    if ((st = ccb::device_ready()) != CCB_OK) return st;
    ccb::Kv4AttendArgs a;
    a.c = *cache;
    a.q = *q;
    a.out = *out;
    a.lse = lse;
    a.headsQ = headsQ;
    a.nQuery = nQuery;
    a.window = window;
    a.scale = scale;
    a.ws = ws;
    a.err = err;
    return ccb::launch_status(ccb::kv4_attend(a, (hipStream_t)stream));
}

CCB_API ccbStatus ccb_kv4_read(const ccbKv4Cache* cache, const ccbKv8Rows* kOut,
                               const ccbKv8Rows* vOut, int32_t count, const int32_t* first,
                               int32_t* err, ccbStream stream)
{
    ccbStatus st = check_cache(cache);
    if (st != CCB_OK) return st;
    if (count < 0 || count > kMaxTokens || !aligned(first, 4) || !aligned(err, 4))
        return CCB_ERR_INVALID_VALUE;
    if (cache->batch == 0 || count == 0) return CCB_OK;
    if (kOut == nullptr && vOut == nullptr) return CCB_ERR_NULL_POINTER;
    if (kOut != nullptr && (st = check_rows(kOut, true)) != CCB_OK) return st;
    if (vOut != nullptr && (st = check_rows(vOut, true)) != CCB_OK) return st;
    if (kOut != nullptr && vOut != nullptr && kOut->type != vOut->type) return CCB_ERR_INVALID_VALUE;
    if (!ccb::kv4_read_fits(*cache, count)) return CCB_ERR_INVALID_VALUE;
    if ((st = ccb::device_ready()) != CCB_OK) return st;
    return ccb::launch_status(ccb::kv4_read(*cache, kOut, vOut, count, first, err, (hipStream_t)stream));
}

}  // extern "C"

// ccb_kv4_internal.h -- private interface between the C entry points of the 4-bit
// key/value cache (ccb_kv4_api.hip) and its kernels.  Not installed.
#ifndef CCB_KV4_INTERNAL_H
#define CCB_KV4_INTERNAL_H

#include "ccb_kv4.h"
#include "ccb_kv8_internal.h"

namespace ccb {

struct Kv4AttendArgs {
    ccbKv4Cache c;
    ccbKv8Rows q, out;
    float* lse;
    int32_t headsQ, nQuery, window;
    float scale;
    void* ws;
    int32_t* err;
};

size_t kv4_attend_bytes(const ccbKv4Cache& c, int32_t headsQ, int32_t nQuery);
// Whether a launch holds the call, and the workspace is large enough.
bool kv4_attend_fits(const ccbKv4Cache& c, int32_t headsQ, int32_t nQuery, int32_t window, size_t wsBytes);
hipError_t kv4_attend(const Kv4AttendArgs& a, hipStream_t s);

bool kv4_append_fits(const ccbKv4Cache& c, int32_t nNew);
hipError_t kv4_append(const ccbKv4Cache& c, const ccbKv8Rows& k, const ccbKv8Rows& v, int32_t nNew,
                      const int64_t* slots, int32_t* err, hipStream_t s);

bool kv4_read_fits(const ccbKv4Cache& c, int32_t count);
hipError_t kv4_read(const ccbKv4Cache& c, const ccbKv8Rows* k, const ccbKv8Rows* v, int32_t count,
                    const int32_t* first, int32_t* err, hipStream_t s);

}  // namespace ccb

#endif  // CCB_KV4_INTERNAL_H

// ccb_kv8_internal.h -- private interface between the C entry points of the 8-bit
// key/value cache (ccb_kv8_api.hip) and its kernels.  Not installed.
#ifndef CCB_KV8_INTERNAL_H
#define CCB_KV8_INTERNAL_H

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ccb_kv8.h"

namespace ccb {

// Checks that the current device is gfx950 (CCB_OK, CCB_ERR_UNSUPPORTED_DEVICE
// or CCB_ERR_HIP); in ccb_api.hip, beside the cached device properties.
ccbStatus device_ready();

// A launch holds fewer than 2^32 threads and numbers its work in 31 bits; what
// needs more is refused before anything is enqueued.
inline bool kv8_launch_fits(int64_t groups, int64_t threads)
{
    return groups <= INT32_MAX && groups * threads <= UINT32_MAX;
}
bool kv8_append_fits(const ccbKv8Cache& c, int32_t nNew);
bool kv8_read_fits(const ccbKv8Cache& c, int32_t count, int32_t sides);
bool kv8_evict_fits(const ccbKv8Cache& from, int32_t budget);
// (and whether the workspace is large enough)
bool kv8_attend_fits(const ccbKv8Cache& c, int32_t headsQ, int32_t nQuery, int32_t window,
                     int32_t accumulate, size_t wsBytes);

struct Kv8AttendArgs {
    ccbKv8Cache c;
    ccbKv8Rows q, out;
    float* lse;
    int32_t headsQ, nQuery, window, accumulate;
    float scale;
    void* ws;
    int32_t* err;
};

// Whether a call that accumulates weights keeps its scores for them; else it
// reads the queries again after the results are written.
bool kv8_attend_keeps_scores(const ccbKv8Cache& c, int32_t headsQ, int32_t nQuery);
size_t kv8_attend_bytes(const ccbKv8Cache& c, int32_t headsQ, int32_t nQuery, int32_t accumulate);
hipError_t kv8_attend(const Kv8AttendArgs& a, hipStream_t s);

size_t kv8_evict_bytes(const ccbKv8Cache& from, int32_t budget);
hipError_t kv8_evict(const ccbKv8Cache& from, const ccbKv8Cache& to, int32_t budget, int32_t recent,
                     int32_t sinks, int32_t* kept, void* ws, int32_t* err, hipStream_t s);

hipError_t kv8_append(const ccbKv8Cache& c, const ccbKv8Rows& k, const ccbKv8Rows& v, int32_t nNew,
                      const int32_t* counts, int32_t* err, hipStream_t s);

hipError_t kv8_read(const ccbKv8Cache& c, const ccbKv8Rows* k, const ccbKv8Rows* v, int32_t count,
                    const int32_t* first, int32_t* err, hipStream_t s);

}  // namespace ccb

#endif  // CCB_KV8_INTERNAL_H

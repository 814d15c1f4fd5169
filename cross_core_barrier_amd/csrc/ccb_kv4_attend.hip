// ccb_kv4_attend.hip -- attention of a decoding step over the 4-bit key/value
// cache, in one pass over the codes on the matrix cores, split over tokens.
//
// The rows of one cache head (its queries and query heads) share every key and
// value, so one workgroup takes a (sequence, cache head, run of tokens) and up
// to 16 rows.  Its eight waves take 32-token tiles in turn and never wait for
// one another in the loop; each keeps its own running maximum, sum and weighted
// values.
//
// S^T = K Q^T and O^T = V^T P^T on 16x16x32 tiles.  In that order a row of
// scores lies on one lane index (lane % 16), so the softmax needs no
// transposition: a lane's 4 + 4 scores of a tile are the 8 places of the next
// product's operand that it has to supply.  Which dimension or token stands at
// which place of a contraction is free as long as both operands agree: lane (n,
// g) takes a quarter of token n's dimensions, side by side in memory and under
// one scale (two at most), and the queries are laid out to match.  So keys go
// from memory into registers and through the conversion, which applies the
// scale, into the product; nothing of them passes LDS.  Values are converted the
// same way, written to the wave's own part of LDS as bf16, and read transposed.
//
// A code times its power of two is exact in bf16, and so is an fp16 query in two
// bf16 pieces: q k is exact up to its 32-bit sums.  The weights go into the
// second product as two bf16 pieces, together within 2^-18.  (One fp16 number,
// 2^-12, with values held relative to the largest scale, takes 8 products and 20
// instructions less a tile and was 2% faster: 24.3 us against 24.9 for 32
// sequences of 100 to 4096 tokens, too little for what it loses.)
//
// What bounds it.  A tile of 32 tokens (D = 128) costs a wave about 250
// instructions for 4352 bytes, which a workgroup of 8 waves gets through in 1.1
// us: large even calls are bound by memory (64 sequences of 16384 tokens: 1.13 GB
// in 197 us, 5.7 TB/s), a long sequence on its own workgroup by a tile's chain of
// work in two waves a SIMD (30 GB/s a CU; vector instructions take 45% of a busy
// SIMD's cycles, matrix products 19%, and the waves wait for 40% of their time), and
// short calls by the start (about 6 us: launch, length -> page -> codes, the join of
// the waves).  Taking two tiles ahead, 16
// waves a workgroup, the next tile's scores beside this one's weights, or all
// transposed reads at once changed little or cost (24.5 us against 26.2, 23.5,
// 26.6 and 25.0; 16 waves take 19.6 us against 14.6 for 200 short sequences).

#include <float.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <chrono>

#include "ccb_kv4_internal.h"
#include "ccb_kv8_device.h"

namespace {

using namespace kv8;

constexpr int kThreads = 512;  // of a workgroup that takes a run of tokens
constexpr int kWaves = kThreads / 64;
constexpr int kJoinThreads = 256;
constexpr int kRows = 16;                // of a workgroup
constexpr int kTile = 32;                // tokens of a wave's step
constexpr int kRunUnit = kWaves * kTile;
constexpr int kSegment = 32 * kRunUnit;  // tokens whose pages fit a wave's lanes
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kJoinHere = 64;   // runs that the last of them may join, at most
constexpr int kJoinRuns = 32;   // more of them are joined by a workgroup, not a wave
constexpr float kSlack = 8.0f;  // how far (in powers of two) scores may pass the running maximum

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));

struct Plan {
    ccb::Kv4AttendArgs a;
    int32_t rows;         // of a cache head
    int32_t rowBlocks;    // workgroups that share a run of tokens
    int32_t runs;         // of a head, over all sequences, at most: see place_of
    int32_t whole;        // units of a sequence that is one run
    float least;          // units of a run, at least
    float lowBy, highBy;  // about 1 / runs and 1 / (runs - sequences)
    bool joinHere;        // the run that ends last joins a sequence's, else another kernel
    float* partO;         // [head][run][row][D], of sequences with several runs
    float2* partML;       // [head][run][row]: maximum (base 2) and sum
    uint64_t* tags;       // [head][rowBlock][run]: see join_here
    uint64_t tag;         // of this call
};

__device__ __forceinline__ f4 mfma(const u4& a, const u4& b, const f4& c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
}

// Eight codes as bf16 times a power of two (the float's exponent), exactly.
__device__ __forceinline__ u4 decode8(uint32_t w, float scale)
{
    u4 u;
    u.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
    u.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
    u.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
    u.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
    return u;
}

// a and b as bf16 pieces: hi + lo is within 2^-18 of the value.
__device__ __forceinline__ void pieces(float a, float b, uint32_t& hi, uint32_t& lo)
{
    const bf2 h = {(__bf16)a, (__bf16)b};
    hi = __builtin_bit_cast(uint32_t, h);
    asm("" : "+v"(hi));  // (or the compiler rounds a once more to have it by itself)
    const bf2 l = {(__bf16)(a - of_bits(hi << 16)), (__bf16)(b - of_bits(hi & 0xffff0000u))};
    lo = __builtin_bit_cast(uint32_t, l);
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// Memory that workgroups on several XCDs share within the kernel: accesses that
// no cache of one XCD's answers.
__device__ __forceinline__ void store_shared(float* p, float a, float b)
{
    const f2 x = {a, b};
    __hip_atomic_store((uint64_t*)p, __builtin_bit_cast(uint64_t, x), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ f2 load_shared(const float* p)
{
    return __builtin_bit_cast(f2, __hip_atomic_load((const uint64_t*)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}

// What a sequence's queries may see.
struct Seen {
    int32_t len;    // 0 where the length is bad
    int32_t first;  // first token any query sees
    int32_t base;   // first, at a tile's border: where the runs start
};

__device__ __forceinline__ Seen seen_of(const ccb::Kv4AttendArgs& a, int32_t len)
{
    Seen r;
    r.len = checked_len(len, a.c.maxPages * a.c.pageSize);
    if (r.len < 0) {
        report(a.err);
        r.len = 0;
    }
    const int64_t f = a.window > 0 ? (int64_t)r.len - a.nQuery + 1 - a.window : 0;
    r.first = f > 0 ? (int32_t)f : 0;
    r.base = r.first & ~(kTile - 1);
    return r;
}

// Its length in units of kRunUnit tokens, at most 2^22.
__device__ __forceinline__ int32_t units_of(const Seen& r) { return (r.len - r.base + kRunUnit - 1) / kRunUnit; }

// A sequence's units as they count where runs are made: a short one is one run,
// and so is an empty one, whose results somebody has to write.
__device__ __forceinline__ float counted(int32_t units, int32_t whole) { return units <= whole ? 1.0f : (float)units; }

// Runs of `chunk` units in that many, whole numbers below 2^23: their quotient
// rounded up.  It comes out of the estimate at most one too small, and then the
// remainder shows it.
__device__ __forceinline__ float runs_in(float units, float chunk, float inverse)
{
    float q = floorf(units * inverse);
    const float r = fmaf(-q, chunk, units);
    q += r > 0.0f ? 1.0f : 0.0f;
    return q + (r > chunk ? 1.0f : 0.0f);
}

// x summed over the lanes up to this one (no exchange through LDS, whose latency
// six times over is a third of a microsecond).
__device__ __forceinline__ int32_t scan(int32_t x)
{
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, true);  // 1, 2, 4, 8 lanes before, in rows of 16
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // the last of a row, to the next one
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // the last of two rows, to the next two
    return x;
}

// A sequence and its runs among those of its head.
struct Place {
    int32_t b, first, n;  // n = 0: there is no such run
    int32_t chunk;        // a run's length in units
    int32_t len;          // as it stands in lens
};

// The sequence that run u belongs to, or (u < 0) sequence b itself.  A run's
// length, for all sequences, is the least with which there are no more than
// p.runs runs (of up to 64 sequences; of more, one that is enough for that), so
// that a long sequence has many workgroups and a short one few, as far as make_plan
// has left more runs than sequences.  The host knows only the capacity, which may be
// many times what a sequence holds.
__device__ __forceinline__ Place place_of(const Plan& p, int32_t u, int32_t b)
{
    const int lane = threadIdx.x & 63;
    const int32_t batch = p.a.c.batch;
    int32_t len = 0, sum = 0;
    float units = 0.0f;
    for (int32_t b0 = 0; b0 < batch; b0 += 64) {
        int32_t held = 0;
        if (b0 + lane < batch) {
            len = p.a.c.lens[b0 + lane];
            held = units_of(seen_of(p.a, len));
        }
        units = counted(held, p.whole);
        sum += __builtin_amdgcn_readlane(scan(held), 63);  // (less than 2^31: see make_plan)
    }
    // (a few parts in 2^20 above and below the quotients)
    const float high = fmaxf(ceilf((float)sum * p.highBy), p.least);
    float chunk = high;
    if (batch <= 64) {  // every lane tries another length between the bounds
        const float low = fminf(high, fmaxf(floorf((float)sum * p.lowBy), p.least));
        const float mine = lane == 63 ? high : low + floorf((high - low) * (float)lane * (1.0f / 63.0f));
        const float inverse = __builtin_amdgcn_rcpf(mine);
        float runs = 0.0f;
#pragma unroll 4
        for (int32_t i = 0; i < batch; ++i)
            runs += runs_in(of_bits(__builtin_amdgcn_readlane(bits(units), i)), mine, inverse);
        const uint64_t enough = __ballot(runs <= (float)p.runs || lane == 63);
        chunk = of_bits(__builtin_amdgcn_readlane(bits(mine), __builtin_ctzll(enough)));
    }
    const float inverse = __builtin_amdgcn_rcpf(chunk);
    int32_t before = 0;
    for (int32_t b0 = 0; b0 < batch; b0 += 64) {
        if (batch > 64 && b0 + lane < batch) {
            len = p.a.c.lens[b0 + lane];
            units = counted(units_of(seen_of(p.a, len)), p.whole);
        }
        const int32_t mine = b0 + lane < batch ? (int32_t)runs_in(units, chunk, inverse) : 0;
        const int32_t upto = scan(mine);
        const uint64_t here = __ballot(u >= 0 ? before + upto > u : b0 + lane == b);
        if (here != 0) {
            const int at = __builtin_ctzll(here);
            const int32_t n = __builtin_amdgcn_readlane(mine, at);
            return Place{b0 + at, before + __builtin_amdgcn_readlane(upto, at) - n, n, (int32_t)chunk,
                         __builtin_amdgcn_readlane(len, at)};
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    return Place{0, 0, 0, 1, 0};
}

// What query i sees, as [begin, end); empty for a row that is not there.
__device__ __forceinline__ void seen_by(const ccb::Kv4AttendArgs& a, const Seen& r, int32_t row, int32_t rows,
                                        int32_t group, int32_t& begin, int32_t& end)
{
    begin = 0, end = 0;
    if (row < rows) {
        end = r.len - a.nQuery + row / group + 1;
        begin = a.window > 0 && end > a.window ? end - a.window : 0;
    }
}

// The address of one row of queries.
__device__ __forceinline__ int64_t row_at(const ccbKv8Rows& r, int32_t b, int32_t h, int32_t row, int32_t group)
{
    return b * r.strideBatch + (row / group) * r.strideToken + (int64_t)(h * group + row % group) * r.strideHead;
}

// Writes a row's results from the sum of its weighted values: 4 of its
// dimensions from each thread that asks, lse from the one with d4 = 0.
template <int T>
__device__ __forceinline__ void write_row(const Plan& p, int32_t b, int32_t h, int32_t row, int32_t d4, const f4& o,
                                          float top, float all)
{
    const ccb::Kv4AttendArgs& a = p.a;
    const int32_t group = a.headsQ / a.c.heads;
    uint2 u = make_uint2(0, 0);
    if (all != 0.0f) {
        u.x = narrow<T>(o.x / all) | (narrow<T>(o.y / all) << 16);
        u.y = narrow<T>(o.z / all) | (narrow<T>(o.w / all) << 16);
    }
    *(uint2*)((uint16_t*)a.out.data + row_at(a.out, b, h, row, group) + d4 * 4) = u;
    if (d4 == 0 && a.lse != nullptr)
        a.lse[((int64_t)b * a.nQuery + row / group) * a.headsQ + h * group + row % group] =
            all != 0.0f ? (top + log2f(all)) * kLn2 : -INFINITY;
}

// A maximum and sum joined with another (a sum of 0 has no maximum; a NaN stays).
__device__ __forceinline__ void merge(float& top, float& all, float top2, float all2)
{
    const float t = fmaxf(top, top2);
    const float x = all == 0.0f ? 0.0f : all * exp2_(top - t);
    const float y = all2 == 0.0f ? 0.0f : all2 * exp2_(top2 - t);
    top = t;
    all = x + y;
}

// Joins a sequence's runs where there are a few: the workgroup that finds all of
// them done does it.  A run's workgroup stores its parts, waits until they are in
// memory, stores its tag, waits again, and reads the tags of all runs.  The last
// one to store its tag so finds all of them set, and so may others, which then
// write the same results; but for those that find tags cleared again, by one that
// joins already.  The tag is this call's own number, so that it does not matter
// what the workspace held, and the tags are cleared, so that a replayed call may
// use its number again.
template <int T, int D>
__device__ __forceinline__ void join_here(const Plan& p, const Place& runs, int32_t run, int32_t h, int32_t row0,
                                          uint8_t* lds)
{
    const int32_t n = runs.n;
    __shared__ int32_t all;
    const int tid = threadIdx.x;
    uint64_t* tags = p.tags + ((int64_t)h * p.rowBlocks + row0 / kRows) * p.runs + runs.first;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid < 64) {
        if (tid == 0) {
            __hip_atomic_store(tags + run, p.tag, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        bool set = true;
        for (int32_t s = tid; s < n; s += 64)
            set &= __hip_atomic_load(tags + s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == p.tag;
        set = __all(set);
        if (tid == 0) all = set;
    }
    __syncthreads();
    if (all == 0) return;
    for (int32_t s = tid; s < n; s += kThreads)
        __hip_atomic_store(tags + s, (uint64_t)0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);

    constexpr int V = D / 4, kWide = 8;  // vectors of a row; loads in flight
    f4* const sums = (f4*)lds;                   // [thread]
    float* const factor = (float*)(sums + kThreads);  // [run][kRows]
    float* const top = factor + kJoinHere * kRows;   // [kRows]
    float* const total = top + kRows;                // [kRows]
    const int32_t rows = p.rows - row0 < kRows ? p.rows - row0 : kRows, items = V * rows;
    const int32_t side = kThreads / items;  // runs side by side, where a pass has threads for them
    const int32_t sg = side > 1 ? tid / items : 0, by = side > 1 ? side : 1;
    const int64_t first = ((int64_t)h * p.runs + runs.first) * p.rows + row0;
    auto part_at = [&](int32_t s, int32_t item) {
        const float* src = p.partO + (first + (int64_t)s * p.rows + item / V) * D + item % V * 4;
        const f2 x = load_shared(src), y = load_shared(src + 2);
        return f4{x.x, x.y, y.x, y.y};
    };
    for (int32_t base = 0; base < items; base += kThreads) {
        const int32_t item = side > 1 ? tid % items : base + tid;
        const bool mine = item < items && sg < by;
        f4 v[kWide];
#pragma unroll
        for (int k = 0; k < kWide; ++k)
            if (mine && sg + k * by < n) v[k] = part_at(sg + k * by, item);
        if (base == 0) {  // a wave for every eighth row, a lane for each run
            const int lane = tid & 63;
            for (int32_t i = tid >> 6; i < rows; i += kWaves) {
                f2 x = {-INFINITY, 0.0f};
                if (lane < n) x = load_shared((const float*)(p.partML + first + (int64_t)lane * p.rows + i));
                float m = x.x;
#pragma unroll
                for (int d = 32; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
                const float f = x.y == 0.0f ? 0.0f : exp2_(x.x - m);
                float l = x.y * f;
#pragma unroll
                for (int d = 32; d >= 1; d >>= 1) l += __shfl_xor(l, d, 64);
                if (lane < n) factor[lane * kRows + i] = f;
                if (lane == 0) top[i] = m, total[i] = l;
            }
            __syncthreads();
        }
        f4 o = {0, 0, 0, 0};
        if (mine) {
            const float* f = factor + item / V;
#pragma unroll
            for (int k = 0; k < kWide; ++k)
                if (sg + k * by < n) o += v[k] * f[(sg + k * by) * kRows];
            for (int32_t s = sg + kWide * by; s < n; s += by) o += part_at(s, item) * f[s * kRows];
        }
        if (side > 1) {
            sums[tid] = o;
            __syncthreads();
            if (sg == 0)
                for (int32_t i = 1; i < side; ++i) o += sums[i * items + item];
        }
        if (mine && sg == 0) write_row<T>(p, runs.b, h, row0 + item / V, item % V, o, top[item / V], total[item / V]);
    }
}

// One half (16 tokens) of a wave's tile, keys or values: a lane's D / 4
// dimensions of token n, and the scales of the first and the last of them (no
// lane has more than two).
typedef const __attribute__((address_space(1))) uint8_t* global;

template <int D>
struct Half {
    uint32_t w[D / 32];
    uint32_t s0, s1;

    // dimensions g * D/4 + 8 j .. + 7 lie under the scale (g * D/4 + 8 j) / 32
    static __device__ __forceinline__ int group_at(int g, int j) { return (g * (D / 32) + j) >> 2; }

    // where a lane's codes and scales are within 16 rows
    static __device__ __forceinline__ uint32_t codes_at(int n, int g) { return (uint32_t)(n * (D / 2) + g * (D / 8)); }
    static __device__ __forceinline__ uint32_t scale_at(int n, int g, int j)
    {
        return (uint32_t)(n * (D / 32) + group_at(g, j));
    }

    // From the codes and scales of the half's 16 rows, the first of them `row` of
    // the cache's: scalar addresses and 32-bit offsets.
    __device__ __forceinline__ void load(const uint8_t* allCodes, const uint8_t* allScales, uint32_t row,
                                         uint32_t codesAt, uint32_t scaleAt0, uint32_t scaleAt1)
    {
        typedef const __attribute__((address_space(1))) u4* global4;
        typedef const __attribute__((address_space(1))) u2* global2;
        typedef const __attribute__((address_space(1))) uint32_t* global1;
        uint64_t at = (uint64_t)allCodes + (uint64_t)row * (D / 2), scaleAt = (uint64_t)allScales + (uint64_t)row * (D / 32);
        asm("" : "+s"(at), "+s"(scaleAt));  // (not added to the offsets in vector registers)
        const global src = (global)at + codesAt, scales = (global)scaleAt;
        if constexpr (D == 64) {
            const u2 x = *(global2)src;
            w[0] = x.x, w[1] = x.y;
        } else if constexpr (D == 96) {
            const global1 x = (global1)src;
            w[0] = x[0], w[1] = x[1], w[2] = x[2];
        } else if constexpr (D == 192) {
            const global2 x = (global2)src;
#pragma unroll
            for (int i = 0; i < 3; ++i) w[2 * i] = x[i].x, w[2 * i + 1] = x[i].y;
        } else {
            const global4 x = (global4)src;
#pragma unroll
            for (int i = 0; i < D / 128; ++i) w[4 * i] = x[i].x, w[4 * i + 1] = x[i].y, w[4 * i + 2] = x[i].z, w[4 * i + 3] = x[i].w;
        }
        s0 = scales[scaleAt0];
        s1 = D == 64 || D == 128 ? s0 : scales[scaleAt1];
    }

    // words 8 j .. 8 j + 7 as bf16
    __device__ __forceinline__ u4 values(int j, int g, float f0, float f1) const
    {
        if constexpr (D == 64 || D == 128) return decode8(w[j], f0);
        return decode8(w[j], group_at(g, j) == group_at(g, 0) ? f0 : f1);
    }
};

template <int T, int D>
// (two workgroups a CU where the registers suffice)
__global__ __launch_bounds__(kThreads, D < 96 || (D <= 128 && T == CCB_KV8_BF16) ? 4 : 2) void kv4_k_attend(Plan p)
{
    constexpr int NB = D / 16;                          // blocks of 16 dimensions
    constexpr int NJ = D / 32;                          // steps of the first product
    constexpr int NQ = T == CCB_KV8_BF16 ? 1 : 2;       // bf16 pieces of a query: exact
    // A token's values in LDS, and 32 bytes more: the 4 tokens that a quarter of a
    // wave reads 16 dimensions of fall on all the banks.  Writes meet in pairs (64
    // cycles a tile of 160 in all); to swap two pieces in every other four lanes
    // takes that away for 8 instructions more, and 25.3 us instead of 24.1.
    constexpr int S = 2 * D + 32;
    __shared__ __attribute__((aligned(16))) uint8_t vBuf[kWaves][kTile * S];
    __shared__ float sm[kWaves][kRows], sl[kWaves][kRows];

    const ccb::Kv4AttendArgs& a = p.a;
    const ccbKv4Cache& c = a.c;
    // Neighbouring workgroups, which go to different XCDs, take neighbouring
    // heads of one run: runs past the last cost every XCD alike.
    uint32_t rest = blockIdx.x;
    const int32_t h = rest % (uint32_t)c.heads;
    rest /= (uint32_t)c.heads;
    const int32_t row0 = (int32_t)(rest % (uint32_t)p.rowBlocks) * kRows;
    const int32_t number = rest / (uint32_t)p.rowBlocks;
    const int32_t P = c.pageSize, group = a.headsQ / c.heads;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;

    Place runs = {number, number, 1, 1, 0};  // as many runs as sequences: one each
    if (p.runs > c.batch) {
        runs = place_of(p, number, 0);
        if (runs.n == 0) return;
    }
    const int32_t b = runs.b, run = number - runs.first;

    // lane i's place in a segment: the wave's i-th half tile
    const int32_t shift = __builtin_ctz(P);
    const int32_t laneAt = ((lane >> 1) * kWaves + wave) * kTile + (lane & 1) * 16;
    const int32_t* table = c.pageTable + b * c.tableStride;
    // without a window a single run's place does not depend on the length: the
    // first page numbers are fetched beside it (they may be of pages past the end)
    int32_t entry = -1;
    const bool early = a.window == 0 && run == 0;
    if (early && laneAt < c.maxPages * P) entry = table[laneAt >> shift];

    Seen r = seen_of(a, p.runs > c.batch ? runs.len : c.lens[b]);
    // (alike in all lanes: what follows from it stays in scalar registers)
    r.len = __builtin_amdgcn_readfirstlane(r.len);
    r.first = __builtin_amdgcn_readfirstlane(r.first);
    r.base = __builtin_amdgcn_readfirstlane(r.base);
    const int32_t tokens = runs.chunk * kRunUnit, lo = r.base + (runs.n > 1 ? run * tokens : 0);
    const int32_t hi = runs.n > 1 && r.len - lo > tokens ? lo + tokens : r.len;

    // Queries, 8 values of a row per lane and step (a row that is not there
    // computes row0's again, for nothing).  Scores are scaled by |scale|, a
    // negative one turns the queries' signs.
    const float scale2 = fabsf(a.scale) * kLog2e;
    u4 q[NJ][NQ];
    int32_t begin, end;
    const int32_t mine = row0 + n;
    seen_by(a, r, mine, p.rows, group, begin, end);
    const uint16_t* src = (const uint16_t*)a.q.data + row_at(a.q, b, h, mine < p.rows ? mine : row0, group) + g * (D / 4);
    const uint32_t turn = a.scale < 0 ? 0x80008000u : 0u;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        u4 x = *(const u4*)(src + 8 * j);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] ^= turn;
        if constexpr (NQ == 1) {
            q[j][0] = x;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t hi, low;
                pieces(widen<T>(x[e] & 0xffffu), widen<T>(x[e] >> 16), hi, low);
                q[j][0][e] = hi, q[j][NQ - 1][e] = low;
            }
        }
    }
    // tokens in [allBegin, allEnd) are seen by every row of the workgroup
    int32_t allBegin, allEnd, unused;
    {
        const int32_t last = row0 + kRows < p.rows ? row0 + kRows - 1 : p.rows - 1;
        seen_by(a, r, last, p.rows, group, allBegin, unused);
        seen_by(a, r, row0, p.rows, group, unused, allEnd);
        allBegin = __builtin_amdgcn_readfirstlane(allBegin), allEnd = __builtin_amdgcn_readfirstlane(allEnd);
    }

    f4 o[NB];
    // What weights are relative to, a maximum that scores may pass by kSlack; the
    // lowest float for a row that has seen nothing (less it, every score grows).
    float ref = -FLT_MAX, l = 0.0f;
#pragma unroll
    for (int d = 0; d < NB; ++d) o[d] = f4{0, 0, 0, 0};

    // Whether a maximum has passed 2^20: what the product's rounding adds to the
    // maximum, 2^-24 of it, would no longer be small as an exponent.
    bool loud = false;
    const uint32_t laneCodes = Half<D>::codes_at(n, g);
    const uint32_t laneScale0 = Half<D>::scale_at(n, g, 0), laneScale1 = Half<D>::scale_at(n, g, D / 32 - 1);
    // where this lane reads values: 4 lanes for a token's 16 dimensions
    const int vTok = 4 * g + (n >> 2);
    uint8_t* const buf = vBuf[wave];
    const uint8_t* const vFrom = buf + vTok * S + (n & 3) * 8;
    uint8_t* const vTo = buf + n * S + g * (D / 2);

    for (int32_t seg = lo; seg < hi; seg += kSegment) {
        const int32_t segEnd = hi - seg < kSegment ? hi : seg + kSegment;
        // Lane i holds the first row of the wave's i-th half tile, among all of the
        // cache's (less than 2^32).  Bit i of `held` is clear where that page is
        // unseen: page 0 is loaded in its place, and not used.
        uint32_t rows = 0;
        bool seen = false;
        {
            const int32_t t = seg + laneAt;
            if (t < segEnd && t + 16 > r.first) {
                const int32_t page = checked_page(early && seg == lo ? entry : table[t >> shift], c.numPages);
                seen = page >= 0;
                if (!seen) report(a.err);
                else rows = ((((uint32_t)page * (uint32_t)c.heads) + (uint32_t)h) << shift) + ((uint32_t)t & (uint32_t)(P - 1));
            }
        }
        const uint64_t held = __ballot(seen);
        const int32_t nTiles = ((segEnd - seg + kTile - 1) / kTile - wave + kWaves - 1) / kWaves;

        auto load = [&](int32_t i, const uint8_t* codes, const uint8_t* scales, Half<D>(&x)[2]) {
            // (the compiler has to see here that these are 32 bits)
            uint32_t codesAt = laneCodes, scaleAt0 = laneScale0, scaleAt1 = laneScale1;
            asm("" : "+v"(codesAt), "+v"(scaleAt0), "+v"(scaleAt1));
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint32_t row = (uint32_t)__builtin_amdgcn_readlane((int32_t)rows, 2 * i + half);
                x[half].load(codes, scales, row, codesAt, scaleAt0, scaleAt1);
            }
        };

        Half<D> key[2], val[2];
        auto step = [&](int32_t i) {
            const int32_t t0 = seg + (i * kWaves + wave) * kTile;
            const uint32_t pair = (uint32_t)(held >> (2 * i)) & 3u;
            const bool whole = t0 >= allBegin && t0 + kTile <= allEnd && pair == 3u;
            // scores
            f4 s[2];
            {
                float f[2][2];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    f[half][0] = of_bits(key[half].s0 << 23), f[half][1] = of_bits(key[half].s1 << 23);
                    s[half] = f4{0, 0, 0, 0};
                }
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const u4 k8 = key[half].values(j, g, f[half][0], f[half][1]);
#pragma unroll
                        for (int k = 0; k < NQ; ++k) s[half] = mfma(k8, q[j][k], s[half]);
                    }
            }
            // the next tile's keys (behind the last one's: the same again, so that the
            // number of loads in flight is the same in every step)
            const int32_t next = i + 1 < nTiles ? i + 1 : i;
            load(next, c.k, c.kScale, key);
            // Scores are multiplied by `by` where the maximum is subtracted, in one
            // rounding; or before.
            float by = scale2;
            bool grows = false;
            if (!whole || loud) {
                asm volatile("");  // a branch: its instructions would be a third of the step's
                by = 1.0f;
                const bool there0 = (pair & 1u) != 0, there1 = (pair & 2u) != 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int32_t t = t0 + 4 * g + e;
                    s[0][e] = t >= begin && t < end && there0 ? s[0][e] * scale2 : -INFINITY;
                    s[1][e] = t + 16 >= begin && t + 16 < end && there1 ? s[1][e] * scale2 : -INFINITY;
                }
                // values that are not there: any scale, but a number
                if (!(there0 && t0 + n < r.len)) val[0].s0 = val[0].s1 = 127;
                if (!(there1 && t0 + 16 + n < r.len)) val[1].s0 = val[1].s1 = 127;
            }
            // values into LDS, as bf16
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float f0 = of_bits(val[half].s0 << 23), f1 = of_bits(val[half].s1 << 23);
#pragma unroll
                for (int j = 0; j < NJ; ++j) *(u4*)(vTo + 16 * half * S + 16 * j) = val[half].values(j, g, f0, f1);
            }
            load(next, c.v, c.vScale, val);
            // Transposed, the first blocks of 16 dimensions are asked for before the
            // weights are computed.  (A wave's LDS accesses keep the program's order.)
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            constexpr int NR = NB % 4 == 0 ? 4 : 3;
            u4 value[NR];
            auto transposed = [&](int d) {
                typedef __attribute__((address_space(3))) s4 lds4;
                const u2 y0 = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(vFrom + 32 * d)));
                const u2 y1 = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(vFrom + 16 * S + 32 * d)));
                return u4{y0.x, y0.y, y1.x, y1.y};
            };
#pragma unroll
            for (int d = 0; d < NR; ++d) value[d] = transposed(d);
            __builtin_amdgcn_sched_barrier(0);
            f4 y[2];  // exponents, then weights
            auto exponents = [&]() {
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[half][e] = fmaf(s[half][e], by, -ref);
            };
            exponents();
            const float x = fmaxf(fmaxf(y[0].x, y[0].y), fmaxf(y[0].z, y[0].w));
            grows |= fmaxf(x, fmaxf(fmaxf(y[1].x, y[1].y), fmaxf(y[1].z, y[1].w))) > kSlack;
            if (__any(grows)) {  // a new maximum, for the row's four lanes alike
                float top = fmaxf(fmaxf(s[0].x, s[0].y), fmaxf(s[0].z, s[0].w));
                top = fmaxf(top, fmaxf(fmaxf(s[1].x, s[1].y), fmaxf(s[1].z, s[1].w))) * by;
                top = fmaxf(top, __shfl_xor(top, 16, 64));
                top = fmaxf(ref, fmaxf(top, __shfl_xor(top, 32, 64)));
                const float f = exp2_(ref - top);
                ref = top;
                l *= f;
#pragma unroll
                for (int d = 0; d < NB; ++d) o[d] *= f;
                loud |= __ballot(fabsf(top) > 0x1p20f && top != -FLT_MAX) != 0;
                if (loud) {
                    s[0] *= by, s[1] *= by;
                    by = 1.0f;
                }
                exponents();
            }
            u4 ph, pl;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                f4 p;
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = exp2_(y[half][e]);
                l += (p.x + p.y) + (p.z + p.w);
                uint32_t h0, l0, h1, l1;
                pieces(p.x, p.y, h0, l0);
                pieces(p.z, p.w, h1, l1);
                ph[2 * half] = h0, ph[2 * half + 1] = h1;
                pl[2 * half] = l0, pl[2 * half + 1] = l1;
            }
#pragma unroll
            for (int d0 = 0; d0 < NB; d0 += NR) {
                if (d0 > 0) {
#pragma unroll
                    for (int d = 0; d < NR; ++d) value[d] = transposed(d0 + d);
                }
#pragma unroll
                for (int d = 0; d < NR; ++d) o[d0 + d] = mfma(value[d], ph, o[d0 + d]);
#pragma unroll
                for (int d = 0; d < NR; ++d) o[d0 + d] = mfma(value[d], pl, o[d0 + d]);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        };

        if (nTiles > 0) {
            load(0, c.k, c.kScale, key);
            load(0, c.v, c.vScale, val);
            for (int32_t i = 0; i < nTiles; ++i) step(i);
        }
    }

    // join the waves
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    if (l == 0.0f) ref = -INFINITY;
    if (g == 0) sm[wave][n] = ref, sl[wave][n] = l;
    __syncthreads();
    const int64_t part = ((int64_t)h * p.runs + number) * p.rows;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, sm[w][n]);
    const float f = l == 0.0f ? 0.0f : exp2_(ref - top);  // (a NaN stays)
    // chunks of 4 dimensions are swapped so that rows fall on different banks
    float* dst = (float*)vBuf[wave] + n * D;
#pragma unroll
    for (int d = 0; d < NB; ++d) *(f4*)(dst + (((4 * d + g) ^ (n & 7)) * 4)) = o[d] * f;
    __syncthreads();
    for (int32_t at = threadIdx.x; at < 4 * D; at += kThreads) {
        const int32_t i = at / (D / 4), d4 = at % (D / 4), row = row0 + i;
        if (row >= p.rows) continue;
        f4 sum = {0, 0, 0, 0};
        float mm = -INFINITY, ll = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            sum += *(const f4*)((const float*)vBuf[w] + i * D + ((d4 ^ (i & 7)) * 4));
            mm = fmaxf(mm, sm[w][i]);
        }
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            ll += sl[w][i] == 0.0f ? 0.0f : sl[w][i] * exp2_(sm[w][i] - mm);
        if (runs.n == 1) {
            write_row<T>(p, b, h, row, d4, sum, mm, ll);
        } else if (p.joinHere) {
            float* dst = p.partO + (part + row) * D + d4 * 4;
            store_shared(dst, sum.x, sum.y);
            store_shared(dst + 2, sum.z, sum.w);
            if (d4 == 0) store_shared((float*)(p.partML + part + row), mm, ll);
        } else {
            *(f4*)(p.partO + (part + row) * D + d4 * 4) = sum;
            if (d4 == 0) p.partML[part + row] = make_float2(mm, ll);
        }
    }
    __syncthreads();
    if (runs.n > 1 && p.joinHere) join_here<T, D>(p, runs, run, h, row0, vBuf[0]);
}

// Joins the runs of a row: four rows to a workgroup, or one where there are
// many runs.
template <int T>
__global__ __launch_bounds__(kJoinThreads) void kv4_k_join(Plan p, int32_t D)
{
    constexpr int kJoinWaves = kJoinThreads / 64;
    __shared__ f4 sum[kJoinThreads];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t V = D / 4;  // vectors of a row
    const int64_t step = (int64_t)p.rows * D;
    const bool many = p.runs - p.a.c.batch >= kJoinRuns;
    const int64_t at = many ? blockIdx.x : (int64_t)blockIdx.x * kJoinWaves + wave;
    const int32_t pair = (int32_t)(at / p.rows), row = (int32_t)(at % p.rows);
    if (pair >= p.a.c.batch * p.a.c.heads) return;  // (not where the workgroup works together)
    const int32_t h = pair % p.a.c.heads, b = pair / p.a.c.heads;
    const Place runs = place_of(p, -1, b);
    const int32_t n = runs.n;
    if (n <= 1) return;  // written by the run itself (the same in a workgroup that works together)
    const int64_t first = ((int64_t)h * p.runs + runs.first) * p.rows + row;
    const float2* ml = p.partML + first;
    float top = -INFINITY, all = 0.0f;
    for (int32_t s = lane; s < n; s += 64) {
        const float2 x = ml[(int64_t)s * p.rows];
        merge(top, all, x.x, x.y);
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) merge(top, all, __shfl_xor(top, d, 64), __shfl_xor(all, d, 64));
    // threads of a row: V for the vectors, and runs side by side
    const int32_t me = many ? tid : lane, groups = (many ? kJoinThreads : 64) / V;
    const int32_t d4 = me % V, sg = me / V;
    const float* src = p.partO + first * D + d4 * 4;
    f4 o = {0, 0, 0, 0};
    if (sg < groups) {
        int32_t s = sg;
        for (; s + 7 * groups < n; s += 8 * groups) {  // 8 loads in flight
            f4 v[8];
            float2 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = *(const f4*)(src + (s + i * groups) * step);
                x[i] = ml[(int64_t)(s + i * groups) * p.rows];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) o += v[i] * (x[i].y == 0.0f ? 0.0f : exp2_(x[i].x - top));
        }
        for (; s < n; s += groups) {
            const float2 x = ml[(int64_t)s * p.rows];
            o += *(const f4*)(src + s * step) * (x.y == 0.0f ? 0.0f : exp2_(x.x - top));
        }
    }
    sum[tid] = o;
    if (many) {
        __syncthreads();
    } else {  // a row's lanes are one wave's, whose LDS accesses keep the program's order
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    if (me < V) {
        for (int32_t i = 1; i < groups; ++i) o += sum[(tid - me) + i * V + d4];
        write_row<T>(p, b, h, row, d4, o, top, all);
    }
}

// How a call is split, and where its workspace's parts lie; returns its bytes,
// which do not depend on the window.  There is a sequence and a query.
size_t make_plan(Plan& p, const ccbKv4Cache& c, int32_t headsQ, int32_t nQuery, int32_t window, void* ws)
{
    const int64_t rows = (int64_t)nQuery * (headsQ / c.heads), batch = c.batch;
    auto up = [](int64_t x, int64_t by) { return (x + by - 1) / by; };
    p.rows = (int32_t)rows;
    p.rowBlocks = (int32_t)up(rows, kRows);
    const int64_t groups = (int64_t)c.heads * p.rowBlocks;  // workgroups that take a run
    // tokens that a sequence's queries may see, from a tile's border
    const int64_t room = (int64_t)c.maxPages * c.pageSize;
    int64_t span = room;
    if (window > 0 && (int64_t)window + nQuery - 1 + kTile < span)
        span = (int64_t)window + nQuery - 1 + kTile;
    // One workgroup of 8 waves for each CU: the second one that it has room for
    // brings no bandwidth, pays its start once more and makes more to join (16
    // sequences of 4096 tokens 20.4 us, with 384 or 512 workgroups 23.7 and 21.5;
    // 8 of 1500 to 16384, D = 256, 26.3 and 41).  More where a run could pass 2 MB
    // of codes: many short sequences do not wait for a long one's end.  Measured on
    // lengths that spread evenly, and right for those.  One long sequence among as many
    // short ones as there are CUs for stays whole, whatever the lengths are: of 8 heads, D
    // = 128, one sequence of 16384 tokens among 200 each, 28 take 24.2 us, 31 45.4 and
    // 32 72 (32 of 2098 each, three times the tokens, 15.4).
    constexpr int64_t target = 256, limit = 16 * target;
    const int64_t longest = (1 << 21) / c.headDim;
    // A sequence of so many units stays whole: a join costs 3 us, a unit 1.1 at D =
    // 128 and 2.2 at 256 (6 sequences with a window of 1000: 9.8 us, cut 12.2).
    p.whole = c.headDim <= 128 ? 5 : 2;
    // runs of a head for sequences of up to `tokens`, and their least length
    auto runs = [&](int64_t tokens, float& least) {
        int64_t n = target / groups;
        least = 1.0f;
        if (tokens <= p.whole * kRunUnit || batch * up(tokens, kRunUnit) > INT32_MAX) return batch;
        if (n <= batch) {  // enough workgroups, unless a sequence is long
            if (tokens <= longest) return batch;
            least = (float)up(longest, kRunUnit);
            const int64_t more = up(batch * tokens, longest);
            n = batch + (more < limit / groups ? more : limit / groups);
        }
        const int64_t most = batch * up(tokens, kRunUnit);
        return n < most ? n : most;
    };
    float unused;
    const int64_t roomy = runs(room, unused);  // over every window: the workspace holds so many
    const int64_t asked = runs(span, p.least);
    p.runs = (int32_t)(asked < roomy ? asked : roomy);
    p.lowBy = (1.0f - 0x1p-20f) / (float)p.runs;
    p.highBy = p.runs > batch ? (1.0f + 0x1p-20f) / (float)(p.runs - batch) : 0.0f;
    const int64_t most = roomy > batch ? roomy : 0;
    size_t bytes = 0;
    auto take = [&](int64_t n, size_t each) {
        char* here = (char*)ws + bytes;
        bytes += ((size_t)n * each + 127) / 128 * 128;
        return here;
    };
    p.partO = (float*)take(c.heads * most * rows * c.headDim, sizeof(float));
    p.partML = (float2*)take(c.heads * most * rows, sizeof(float2));
    p.tags = (uint64_t*)take(groups * most, sizeof(uint64_t));
    // Runs that one sequence may have, and may be taken to have.  The last of them
    // joins a few (8 sequences of 1500 to 16384 tokens: 26.4 us, with a kernel of its
    // own 28.5); where a head's parts pass 64 KB one workgroup is too slow for them
    // (32 runs of 8 rows, D = 128: 60.4 us against 59.5).
    const int64_t extra = p.runs - batch + 1, byLength = up(up(span, kRunUnit), (int64_t)p.least);
    const int64_t here = extra < byLength ? extra : byLength, few = up(2 * p.runs, batch);
    p.joinHere = here <= kJoinHere &&
                 (here < few ? here : few) * (rows < kRows ? rows : kRows) * c.headDim * 4 <= (64 << 10);
    return bytes;
}

// A number that no other call of this process has, nor one of another whose
// memory this one may have got (up to 2^-64); not 0.
uint64_t new_tag()
{
    static std::atomic<uint64_t> next{
        (uint64_t)std::chrono::system_clock::now().time_since_epoch().count() * 0x9E3779B97F4A7C15u ^ (uint64_t)&next};
    const uint64_t n = next.fetch_add(1, std::memory_order_relaxed);
    return n != 0 ? n : next.fetch_add(1, std::memory_order_relaxed);
}

// Whether a kernel of its own joins what is cut.
bool joins_apart(const Plan& p) { return p.runs > p.a.c.batch && !p.joinHere; }

int64_t join_groups(const Plan& p)
{
    const int64_t rows = (int64_t)p.rows * p.a.c.batch * p.a.c.heads;
    return p.runs - p.a.c.batch >= kJoinRuns ? rows : (rows + 3) / 4;
}

template <int T, int D>
hipError_t launch(const Plan& p, hipStream_t s)
{
    const int64_t groups = (int64_t)p.a.c.heads * p.rowBlocks * p.runs;
    hipError_t e = enqueue(kv4_k_attend<T, D>, groups, kThreads, s, p);
    if (e == hipSuccess && joins_apart(p)) e = enqueue(kv4_k_join<T>, join_groups(p), kJoinThreads, s, p, D);
    return e;
}

}  // namespace

namespace ccb {

size_t kv4_attend_bytes(const ccbKv4Cache& c, int32_t headsQ, int32_t nQuery)
{
    if (c.batch == 0 || nQuery == 0 || (int64_t)c.batch * c.heads > INT32_MAX) return 0;
    Plan p;
    return make_plan(p, c, headsQ, nQuery, 0, nullptr);
}

bool kv4_attend_fits(const ccbKv4Cache& c, int32_t headsQ, int32_t nQuery, int32_t window, size_t wsBytes)
{
    const int64_t pairs = (int64_t)c.batch * c.heads, rows = (int64_t)nQuery * (headsQ / c.heads);
    if (pairs > INT32_MAX || pairs * rows > INT32_MAX) return false;
    Plan p;
    p.a.c = c;
    return make_plan(p, c, headsQ, nQuery, window, nullptr) <= wsBytes &&
           kv8_launch_fits((int64_t)c.heads * p.rowBlocks * p.runs, kThreads) &&
           (!joins_apart(p) || kv8_launch_fits(join_groups(p), kJoinThreads));
}

hipError_t kv4_attend(const Kv4AttendArgs& a, hipStream_t s)
{
    Plan p;
    p.a = a;
    make_plan(p, a.c, a.headsQ, a.nQuery, a.window, a.ws);
    p.tag = new_tag();
#define KV4_ATTEND_DIM(T) \
    switch (a.c.headDim) { \
    case 64: return launch<T, 64>(p, s); \
    case 96: return launch<T, 96>(p, s); \
    case 128: return launch<T, 128>(p, s); \
    case 192: return launch<T, 192>(p, s); \
    default: return launch<T, 256>(p, s); \
    }
    if (a.q.type == CCB_KV8_BF16) KV4_ATTEND_DIM(CCB_KV8_BF16)
    KV4_ATTEND_DIM(CCB_KV8_FP16)
}

}  // namespace ccb

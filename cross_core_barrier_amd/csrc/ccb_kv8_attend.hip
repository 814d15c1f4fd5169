// ccb_kv8_attend.hip -- attention of a decoding step over the 8-bit
// key/value cache, in one pass over the codes on the matrix cores, split over
// tokens.
//
// The rows of one cache head (its queries and query heads) share every key
// and value, so one workgroup takes a (sequence, cache head, run of tokens)
// and up to 16 * NT rows.  Its eight waves take 32-token tiles in turn and
// never wait for one another in the loop: a wave streams its own tiles into
// its own part of LDS (16 bytes per lane, straight from memory; the next
// tile's keys are on their way as soon as this one's are read, and its values
// likewise) and keeps its own running maximum, sum and weighted values.
//
// S^T = K Q^T and O^T = V^T P^T on 16x16x32 tiles.  In that order a row of
// scores lies on one lane index (lane % 16), so the softmax needs no
// transposition: a lane's 4 + 4 scores of a tile are the 8 places of the next
// product's operand that it has to supply.  Which token or dimension stands at
// which place of a contraction is free as long as both operands agree; keys
// are read 16 dimensions at a time, values through the transposing LDS read.
//
// Codes become 16-bit values exactly (int8 and e4m3 both fit bf16 and fp16),
// so q k is exact up to its 32-bit sums.  The weights p (times the block's
// scale) go into the second product as two bf16 pieces, together within 2^-18
// of p; one piece would cost 2^-9.
//
// A tile of 32 tokens costs a wave about 350 instructions for 64 * D bytes, so
// large calls are bound by memory (64 sequences of 8192 tokens, D = 128: 1.06
// GB in 183 us, 5.8 TB/s; one of 131071 with its scores kept: 65 us, 4.6 TB/s)
// and short ones by the start of a kernel: about 4 us until all XCDs run it, 3
// until the first tile is there (length -> page -> codes; scales and queries
// are asked for meanwhile), 2 for the join of the waves.  A second tile in
// flight for each wave changed nothing (22.3 us against 22.2 for 16 sequences
// of up to 4096 tokens, before the reads of LDS stopped waiting for it).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ccb_kv8_internal.h"
#include "ccb_kv8_device.h"

// Scores are kept for the weights of up to 16 rows: writing and reading them (8
// bytes a row and token) costs less than a kernel more that reads, converts and
// multiplies every key again.  In us, kept and again, 8 cache heads:
//                               rows    D = 64      D = 128     D = 256
//   16 sequences of 4096 tokens    4    23   39     33   61     65  109
//                                 16    29   39     46   66     78  119
//   64 of 8192 (D = 256: 32)       4   154  239    270  437    243  406
//                                 16   263  242    373  448    287  431
// Only D = 64 with 16 rows in a cache of 2^19 tokens goes the other way.  17 to
// 64 rows keep theirs where all of them stay in the caches (8 sequences of 500 tokens, D = 128, 32 rows: 14.6 and 19.5).
// Beyond that it depends on the head size (64 rows of 16 x 4096: 79 and 70 at
// D = 64, 176 and 220 at 256), and the scores would take more memory than the
// gain is worth (64 x 8192, 64 rows: 1.1 GB).
bool ccb::kv8_attend_keeps_scores(const ccbKv8Cache& c, int32_t headsQ, int32_t nQuery)
{
    const int64_t pairs = (int64_t)c.batch * c.heads, rows = (int64_t)nQuery * (headsQ / c.heads);
    return rows <= 16 || (rows <= 64 && pairs * rows * c.maxPages * c.pageSize * 4 <= (32 << 20));
}

namespace {

using namespace kv8;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kRunThreads = 512;  // of a workgroup that takes a run of tokens
constexpr int kRunWaves = kRunThreads / 64;
constexpr int kTile = 32;                        // tokens of a wave's step
constexpr int kRunUnit = kRunWaves * kTile;
constexpr int kSegment = 32 * kRunWaves * kTile;  // tokens whose pages fit a wave's lanes
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kJoinRuns = 32;  // more of them are joined by a workgroup, not a wave
constexpr float kSlack = 8.0f;  // how far (in powers of two) scores may pass the running maximum

typedef float f4 __attribute__((ext_vector_type(4)));
typedef int i2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

struct Plan {
    ccb::Kv8AttendArgs a;
    int32_t pairs;      // (sequence, cache head)
    int32_t rows;       // of a cache head
    int32_t tilesN;     // NT
    int32_t rowBlocks;  // workgroups that share a run of tokens
    int32_t splits;     // runs of a sequence, see range_of
    int32_t tiles;      // a sequence may have
    bool direct;        // one run: its workgroup writes the results
    int32_t joinRows;   // workgroups of the join for the rows
    int64_t joinBlocks; // all of the join's, those for the tokens among them,
    int32_t joinSpan;   // so many each
    float* partO;   // [pair][split][row][D]
    float2* partML; // [pair][split][row]: maximum (base 2) and sum
    float* scores;  // [pair][tile][row][kTile] (base 2), or null: see score_at
    float* lse2;    // [pair][row], +infinity for a row that sees nothing; or null
};

// Four codes (lowest byte first) as two words of two 16-bit values.
template <int F, int T>
__device__ __forceinline__ void codes16(uint32_t w, uint32_t& a, uint32_t& b)
{
    if constexpr (F == kE4m3 && T == CCB_KV8_BF16) {
        a = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
        b = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true));
    } else if constexpr (F == kE4m3) {
        a = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
        b = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true));
    } else if constexpr (T == CCB_KV8_BF16) {
        // a whole number below 2^8 is exact in the upper half of its float
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = (float)(int8_t)(w >> (8 * i));
        a = __builtin_amdgcn_perm(bits(f[1]), bits(f[0]), 0x07060302u);
        b = __builtin_amdgcn_perm(bits(f[3]), bits(f[2]), 0x07060302u);
    } else {
        // 0x6400 | u is 1024 + u in fp16; u = code + 128
        const uint32_t u = w ^ 0x80808080u;
        const h2 m = {(_Float16)-1152.0f, (_Float16)-1152.0f};
        const h2 x = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, u, 0x07010700u)) + m;
        const h2 y = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, u, 0x07030702u)) + m;
        a = __builtin_bit_cast(uint32_t, x);
        b = __builtin_bit_cast(uint32_t, y);
    }
}

template <int F, int T>
__device__ __forceinline__ u4 codes16x8(uint32_t lo, uint32_t hi)
{
    uint32_t a, b, c, d;
    codes16<F, T>(lo, a, b);
    codes16<F, T>(hi, c, d);
    return u4{a, b, c, d};
}

template <int T>
__device__ __forceinline__ f4 mfma(const u4& a, const u4& b, const f4& c)
{
    if constexpr (T == CCB_KV8_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a),
                                                       __builtin_bit_cast(bf8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a),
                                                      __builtin_bit_cast(h8, b), c, 0, 0, 0);
}

// a and b as bf16 pieces: hi + lo is within 2^-18 of the value.
__device__ __forceinline__ void pieces(float a, float b, uint32_t& hi, uint32_t& lo)
{
    const bf2 h = {(__bf16)a, (__bf16)b};
    hi = __builtin_bit_cast(uint32_t, h);
    const bf2 l = {(__bf16)(a - of_bits(hi << 16)), (__bf16)(b - of_bits(hi & 0xffff0000u))};
    lo = __builtin_bit_cast(uint32_t, l);
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// The score of a pair's row and token (counted from base).  A tile's rows lie
// side by side, so that what a wave stores is one piece of memory.
__device__ __forceinline__ float* score_at(const Plan& p, int32_t pair, int32_t row, int32_t t)
{
    const int64_t tile = (int64_t)pair * p.tiles + t / kTile;
    return p.scores + (tile * p.rows + row) * kTile + t % kTile;
}

// What a sequence's queries may see, and its runs.  Every sequence has
// p.splits of them, as long as its own length asks: the capacity, which is all
// that the host knows, may be many times what a sequence holds.
struct Range {
    int32_t len;    // 0 where the length is bad
    int32_t first;  // first token any query sees
    int32_t base;   // first, at a tile's border: where the runs start
    int32_t chunk;  // tokens of a run, a multiple of kRunUnit
    int32_t runs;   // that hold tokens
};

__device__ __forceinline__ Range range_of(const Plan& p, int32_t b)
{
    const ccb::Kv8AttendArgs& a = p.a;
    Range r;
    r.len = checked_len(a.c.lens[b], a.c.maxPages * a.c.pageSize);
    if (r.len < 0) {
        if (threadIdx.x == 0) report(a.err);
        r.len = 0;
    }
    const int64_t f = a.window > 0 ? (int64_t)r.len - a.nQuery + 1 - a.window : 0;
    r.first = f > 0 ? (int32_t)f : 0;
    r.base = r.first & ~(kTile - 1);
    const uint32_t held = (uint32_t)(r.len - r.base), splits = (uint32_t)p.splits;
    r.chunk = (int32_t)(((held + splits * kRunUnit - 1) / (splits * kRunUnit)) * kRunUnit);
    r.runs = r.chunk > 0 ? (int32_t)((held + (uint32_t)r.chunk - 1) / (uint32_t)r.chunk) : 0;
    return r;
}

// What query i sees, as [begin, end); empty for a row that is not there.
__device__ __forceinline__ void seen_by(const ccb::Kv8AttendArgs& a, const Range& r, int32_t row,
                                        int32_t rows, int32_t group, int32_t& begin, int32_t& end)
{
    begin = 0, end = 0;
    if (row < rows) {
        end = r.len - a.nQuery + row / group + 1;
        begin = a.window > 0 && end > a.window ? end - a.window : 0;
    }
}

// How the chunks of 16 codes of a token are swapped in LDS, so that 16 tokens
// read at one chunk fall on all the banks.  Depends on the token modulo 16.
template <int D>
__device__ __forceinline__ int swap_of(int r)
{
    constexpr int C = D / 16;
    return C == 8 ? (r >> 1) & 7 : C == 16 ? r & 15 : C == 6 ? (r >> 3) & 1 : (r >> 2) & 3;
}

// Bytes straight from memory into LDS: lane i's 16 bytes land at dst + 16 i.
__device__ __forceinline__ void load_lds(const uint8_t* src, uint8_t* dst)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                     (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

template <int N>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// The address of one row of queries.
__device__ __forceinline__ int64_t row_at(const ccbKv8Rows& r, int32_t b, int32_t h, int32_t row,
                                          int32_t group)
{
    return b * r.strideBatch + (row / group) * r.strideToken +
           (int64_t)(h * group + row % group) * r.strideHead;
}

// The 8 query values of a row that stand opposite the key's 8 codes in step j.
template <int D>
__device__ __forceinline__ int dim_at(int j, int g)
{
    return (D % 64 != 0 && j == D / 32 - 1) ? 32 * j + 8 * g : 64 * (j >> 1) + 16 * g + 8 * (j & 1);
}

// Writes a row's results from the sum of its weighted values: 4 of its
// dimensions from each thread that asks, lse from the one with d4 = 0.
template <int T>
__device__ __forceinline__ void write_row(const Plan& p, int32_t b, int32_t h, int32_t pair, int32_t row,
                                          int32_t d4, const f4& o, float top, float all)
{
    const ccb::Kv8AttendArgs& a = p.a;
    const int32_t group = a.headsQ / a.c.heads;
    uint2 u = make_uint2(0, 0);
    if (all != 0.0f) {
        u.x = narrow<T>(o.x / all) | (narrow<T>(o.y / all) << 16);
        u.y = narrow<T>(o.z / all) | (narrow<T>(o.w / all) << 16);
    }
    *(uint2*)((uint16_t*)a.out.data + row_at(a.out, b, h, row, group) + d4 * 4) = u;
    if (d4 == 0) {
        const float lse = all != 0.0f ? top + log2f(all) : INFINITY;
        if (p.lse2 != nullptr) p.lse2[(int64_t)pair * p.rows + row] = lse;
        if (a.lse != nullptr)
            a.lse[((int64_t)b * a.nQuery + row / group) * a.headsQ + h * group + row % group] =
                all != 0.0f ? lse * kLn2 : -INFINITY;
    }
}

__device__ __forceinline__ uint32_t lds_at(const uint8_t* p)
{
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)p;
}

// A lane's keys of a tile: 16 codes for two steps of the first product, 8 for a
// last odd one, of token n and token 16 + n.  In one block with the wait for
// them: behind reads that it knows as such the compiler waits for every load
// into LDS that is in flight, the values' too (64 sequences of 8192 tokens: 188
// us instead of 183; 32 rows a head, 16 of 4096: 34.7 instead of 31).
template <int D>
__device__ __forceinline__ void read_keys(const uint8_t* buf, int at, int swap, int g, 
                                          u4 (&key)[2][(D / 32 + 1) / 2])
{
    const uint32_t row = lds_at(buf) + (uint32_t)at;
    const uint32_t a0 = row + ((g ^ swap) * 16), a1 = row + (((4 + g) ^ swap) * 16);
    if constexpr (D == 64) {
        asm volatile(
            "ds_read_b128 %0, %2\n\t"
            "ds_read_b128 %1, %2 offset:1024\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(key[0][0]), "=&v"(key[1][0]) : "v"(a0) : "memory");
    } else if constexpr (D == 96) {
        typedef uint32_t u2 __attribute__((ext_vector_type(2)));
        const uint32_t t = row + (((4 + (g >> 1)) ^ swap) * 16 + 8 * (g & 1));
        u2 x, y;
        asm volatile(
            "ds_read_b128 %0, %4\n\t"
            "ds_read_b128 %1, %4 offset:1536\n\t"
            "ds_read_b64 %2, %5\n\t"
            "ds_read_b64 %3, %5 offset:1536\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(key[0][0]), "=&v"(key[1][0]), "=&v"(x), "=&v"(y) : "v"(a0), "v"(t) : "memory");
        key[0][1] = u4{x.x, x.y, 0, 0};
        key[1][1] = u4{y.x, y.y, 0, 0};
    } else if constexpr (D == 128) {
        asm volatile(
            "ds_read_b128 %0, %4\n\t"
            "ds_read_b128 %1, %5\n\t"
            "ds_read_b128 %2, %4 offset:2048\n\t"
            "ds_read_b128 %3, %5 offset:2048\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(key[0][0]), "=&v"(key[0][1]), "=&v"(key[1][0]), "=&v"(key[1][1])
            : "v"(a0), "v"(a1) : "memory");
    } else {
        const uint32_t a2 = row + (((8 + g) ^ swap) * 16);
        if constexpr (D == 192) {
            asm volatile(
                "ds_read_b128 %0, %6\n\t"
                "ds_read_b128 %1, %7\n\t"
                "ds_read_b128 %2, %8\n\t"
                "ds_read_b128 %3, %6 offset:3072\n\t"
                "ds_read_b128 %4, %7 offset:3072\n\t"
                "ds_read_b128 %5, %8 offset:3072\n\t"
                "s_waitcnt lgkmcnt(0)"
                : "=&v"(key[0][0]), "=&v"(key[0][1]), "=&v"(key[0][2]), "=&v"(key[1][0]), "=&v"(key[1][1]),
                  "=&v"(key[1][2])
                : "v"(a0), "v"(a1), "v"(a2) : "memory");
        } else {
            const uint32_t a3 = row + (((12 + g) ^ swap) * 16);
            asm volatile(
                "ds_read_b128 %0, %8\n\t"
                "ds_read_b128 %1, %9\n\t"
                "ds_read_b128 %2, %10\n\t"
                "ds_read_b128 %3, %11\n\t"
                "ds_read_b128 %4, %8 offset:4096\n\t"
                "ds_read_b128 %5, %9 offset:4096\n\t"
                "ds_read_b128 %6, %10 offset:4096\n\t"
                "ds_read_b128 %7, %11 offset:4096\n\t"
                "s_waitcnt lgkmcnt(0)"
                : "=&v"(key[0][0]), "=&v"(key[0][1]), "=&v"(key[0][2]), "=&v"(key[0][3]), "=&v"(key[1][0]),
                  "=&v"(key[1][1]), "=&v"(key[1][2]), "=&v"(key[1][3])
                : "v"(a0), "v"(a1), "v"(a2), "v"(a3) : "memory");
        }
    }
}

// Transposed reads of 16 dimensions of a lane's 8 tokens, N blocks of them; as
// above in one block with the wait.
template <int N>
__device__ __forceinline__ void read_values(const uint32_t* at, i2* w)
{
    static_assert(N == 4 || N == 6 || N == 8, "blocks of 16 dimensions at once");
    if constexpr (N == 4)
        asm volatile("ds_read_b64_tr_b8 %0, %4\n\t"
                     "ds_read_b64_tr_b8 %1, %5\n\t"
                     "ds_read_b64_tr_b8 %2, %6\n\t"
                     "ds_read_b64_tr_b8 %3, %7\n\t"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(w[0]), "=&v"(w[1]), "=&v"(w[2]), "=&v"(w[3])
                     : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3])
                     : "memory");
    else if constexpr (N == 6)
        asm volatile("ds_read_b64_tr_b8 %0, %6\n\t"
                     "ds_read_b64_tr_b8 %1, %7\n\t"
                     "ds_read_b64_tr_b8 %2, %8\n\t"
                     "ds_read_b64_tr_b8 %3, %9\n\t"
                     "ds_read_b64_tr_b8 %4, %10\n\t"
                     "ds_read_b64_tr_b8 %5, %11\n\t"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(w[0]), "=&v"(w[1]), "=&v"(w[2]), "=&v"(w[3]), "=&v"(w[4]), "=&v"(w[5])
                     : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "v"(at[4]), "v"(at[5])
                     : "memory");
    else
        asm volatile("ds_read_b64_tr_b8 %0, %8\n\t"
                     "ds_read_b64_tr_b8 %1, %9\n\t"
                     "ds_read_b64_tr_b8 %2, %10\n\t"
                     "ds_read_b64_tr_b8 %3, %11\n\t"
                     "ds_read_b64_tr_b8 %4, %12\n\t"
                     "ds_read_b64_tr_b8 %5, %13\n\t"
                     "ds_read_b64_tr_b8 %6, %14\n\t"
                     "ds_read_b64_tr_b8 %7, %15\n\t"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(w[0]), "=&v"(w[1]), "=&v"(w[2]), "=&v"(w[3]), "=&v"(w[4]), "=&v"(w[5]),
                       "=&v"(w[6]), "=&v"(w[7])
                     : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "v"(at[4]), "v"(at[5]),
                       "v"(at[6]), "v"(at[7])
                     : "memory");
}

template <int F, int T, int D, int NT>
__global__ __launch_bounds__(kRunThreads, D <= 128 && NT == 1 ? 4 : 2) void kv8_k_attend(Plan p)
{
    constexpr int C = D / 16;             // chunks of 16 codes in a token
    constexpr int NI = kTile * C / 64;    // loads of a wave for a tile of keys
    constexpr int NB = D / 16;            // blocks of 16 dimensions
    constexpr int NJ = D / 32;            // steps of the first product
    __shared__ __attribute__((aligned(16))) uint8_t kBuf[kRunWaves][kTile * D];
    __shared__ __attribute__((aligned(16))) uint8_t vBuf[kRunWaves][kTile * D];
    __shared__ float sm[kRunWaves][16 * NT], sl[kRunWaves][16 * NT], slse[16 * NT];

    const ccb::Kv8AttendArgs& a = p.a;
    const ccbKv8Cache& c = a.c;
    // Neighbouring workgroups, which go to different XCDs, take neighbouring
    // heads of one run: runs past short sequences' ends cost every XCD alike.
    uint32_t rest = blockIdx.x;
    const int32_t pair = rest % (uint32_t)p.pairs;
    rest /= (uint32_t)p.pairs;
    const int32_t row0 = (int32_t)(rest % (uint32_t)p.rowBlocks) * (16 * NT);
    const int32_t split = rest / (uint32_t)p.rowBlocks;
    const int32_t h = pair % c.heads, b = pair / c.heads;
    const int32_t P = c.pageSize, group = a.headsQ / c.heads;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;

    // lane i's place in a segment: the wave's i-th half tile
    const int32_t shift = __builtin_ctz(P);
    const int32_t laneAt = ((lane >> 1) * kRunWaves + wave) * kTile + (lane & 1) * 16;
    // without a window a single run's place does not depend on the length: the
    // first page numbers are fetched beside it (they may be of pages past the end)
    int32_t entry = -1;
    const bool early = a.window == 0 && p.splits == 1;
    const int32_t* table = c.pageTable + b * c.tableStride;
    if (early && laneAt < c.maxPages * P) entry = table[laneAt >> shift];

    const Range r = range_of(p, b);
    if (split > 0 && split >= r.runs) return;  // the join knows
    const int32_t lo = r.base + split * r.chunk;
    const int32_t hi = r.len - lo < r.chunk ? r.len : lo + r.chunk;

    // queries, 8 values of a row per lane and step (a row that is not there
    // computes row0's again, for nothing)
    u4 q[NT][NJ];
    int32_t begin[NT], end[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int32_t row = row0 + nt * 16 + n;
        seen_by(a, r, row, p.rows, group, begin[nt], end[nt]);
        const uint16_t* src = (const uint16_t*)a.q.data + row_at(a.q, b, h, row < p.rows ? row : row0, group);
#pragma unroll
        for (int j = 0; j < NJ; ++j) q[nt][j] = *(const u4*)(src + dim_at<D>(j, g));
    }
    // tokens in [allBegin, allEnd) are seen by every row of the workgroup
    int32_t allBegin, allEnd, unused;
    {
        const int32_t last = row0 + 16 * NT < p.rows ? row0 + 16 * NT - 1 : p.rows - 1;
        seen_by(a, r, last, p.rows, group, allBegin, unused);
        seen_by(a, r, row0, p.rows, group, unused, allEnd);
    }

    const float scale2 = a.scale * kLog2e;  // scores in powers of two
    const bool stored = p.scores != nullptr;
    f4 o[NT][NB];
    float m[NT], ref[NT], l[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt] = -INFINITY, ref[nt] = 0.0f, l[nt] = 0.0f;
#pragma unroll
        for (int d = 0; d < NB; ++d) o[nt][d] = f4{0, 0, 0, 0};
    }

    // where this lane's chunks of a tile come from (in bytes, within 16 tokens)
    int32_t from[NI];
#pragma unroll
    for (int it = 0; it < NI; ++it) {
        const int at = it * 64 + lane, tok = at / C;
        from[it] = ((tok & 15) * C + ((at % C) ^ swap_of<D>(tok & 15))) * 16;
    }
    // where this lane reads keys (its token n) and values (two lanes for a token)
    const int kAt = n * C * 16, kSwap = swap_of<D>(n);
    const int vSlot = n >> 1;
    const int vTok = 4 * g + (vSlot & 3) + (vSlot < 4 ? 0 : 16);
    const int vAt = vTok * C * 16 + 8 * (lane & 1), vSwap = swap_of<D>(vTok & 15);

    for (int32_t seg = lo; seg < hi; seg += kSegment) {
        const int32_t segEnd = hi - seg < kSegment ? hi : seg + kSegment;
        // lane i holds page and scales of the wave's i-th half tile
        int32_t page = -1;
        float kScale = 0.0f, vScale = 0.0f;
        {
            const int32_t t = seg + laneAt;
            const bool seen = t < segEnd && t + 16 > r.first;
            if (seen) page = checked_page(early && seg == lo ? entry : table[t >> shift], c.numPages);
            // The compiler has to know before the loop that the queries and the
            // scales are there: left to the loop, the wait for them is one for every
            // load, in every step.  The queries were asked for before the pages.
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int jj = 0; jj < NJ; ++jj) asm volatile("" : "+v"(q[nt][jj]));
            if (page >= 0) {
                const int64_t block = (int64_t)page * c.heads + h;
                kScale = c.kScale[block];
                vScale = c.vScale[block];
            } else if (seen) {
                report(a.err);
            }
        }
        const int32_t nTiles = ((segEnd - seg + kTile - 1) / kTile - wave + kRunWaves - 1) / kRunWaves;

        auto issue = [&](const void* codes, int32_t i, uint8_t* buf) {
            const int32_t t = seg + (i * kRunWaves + wave) * kTile;
            const uint8_t* src[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                int32_t pg = __builtin_amdgcn_readlane(page, 2 * i + half);
                pg = pg < 0 ? 0 : pg;  // an unseen page's place: page 0 is loaded and not used
                src[half] = (const uint8_t*)codes +
                            (((int64_t)pg * c.heads + h) * P + ((t + 16 * half) & (P - 1))) * D;
            }
#pragma unroll
            for (int it = 0; it < NI; ++it) {
                const uint8_t* s = (it * 64 + 63) / C < 16 ? src[0] : it * 64 / C >= 16 ? src[1]
                                   : (it * 64 + lane) / C < 16 ? src[0] : src[1];
                load_lds(s + from[it], buf + it * 1024);
            }
        };

        auto step = [&](int32_t i, uint8_t* kb, uint8_t* vb) {
            const int32_t t0 = seg + (i * kRunWaves + wave) * kTile;
            const bool more = i + 1 < nTiles;
            // Scores.  Behind this tile's keys: its values, and between them the last
            // step's stores of scores, two at least where they are kept (a wait that
            // does not count them waits for the stores, and below for the next keys).
            if (stored && i > 0) wait_loads<NI + 2>(); else wait_loads<NI>();
            u4 key[2][(NJ + 1) / 2];
            read_keys<D>(kb, kAt, kSwap, g, key);
            if (more) {
                issue(c.k, i + 1, kb);
                asm volatile("" ::: "memory");  // the stores come after these loads
            }
            f4 s[NT][2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) s[nt][half] = f4{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < NJ; j += 2) {
                    const u4 w = key[half][j / 2];
                    const u4 x = codes16x8<F, T>(w.x, w.y);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) s[nt][half] = mfma<T>(x, q[nt][j], s[nt][half]);
                    if (j + 1 < NJ) {
                        const u4 y = codes16x8<F, T>(w.z, w.w);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) s[nt][half] = mfma<T>(y, q[nt][j + 1], s[nt][half]);
                    }
                }
            }
            const int32_t pg0 = __builtin_amdgcn_readlane(page, 2 * i);
            const int32_t pg1 = __builtin_amdgcn_readlane(page, 2 * i + 1);
            const float kf0 = of_bits(__builtin_amdgcn_readlane(bits(kScale), 2 * i)) * scale2;
            const float kf1 = of_bits(__builtin_amdgcn_readlane(bits(kScale), 2 * i + 1)) * scale2;
            const float vf0 = of_bits(__builtin_amdgcn_readlane(bits(vScale), 2 * i));
            const float vf1 = of_bits(__builtin_amdgcn_readlane(bits(vScale), 2 * i + 1));
            const bool whole = t0 >= allBegin && t0 + kTile <= allEnd && (pg0 | pg1) >= 0;
            bool grows = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                s[nt][0] *= kf0, s[nt][1] *= kf1;
                if (!whole) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int32_t t = t0 + 4 * g + e;
                        if (!(t >= begin[nt] && t < end[nt] && pg0 >= 0)) s[nt][0][e] = -INFINITY;
                        if (!(t + 16 >= begin[nt] && t + 16 < end[nt] && pg1 >= 0))
                            s[nt][1][e] = -INFINITY;
                    }
                }
                if (stored && row0 + nt * 16 + n < p.rows) {
                    float* dst = score_at(p, pair, row0 + nt * 16 + n, t0 - r.base) + 4 * g;
                    *(f4*)dst = s[nt][0];
                    *(f4*)(dst + 16) = s[nt][1];
                }
                float mx = fmaxf(fmaxf(s[nt][0].x, s[nt][0].y), fmaxf(s[nt][0].z, s[nt][0].w));
                mx = fmaxf(mx, fmaxf(fmaxf(s[nt][1].x, s[nt][1].y), fmaxf(s[nt][1].z, s[nt][1].w)));
                grows |= mx > m[nt] + kSlack;
            }
            if (__any(grows)) {  // a new maximum, for the row's four lanes alike
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float mx = fmaxf(fmaxf(s[nt][0].x, s[nt][0].y), fmaxf(s[nt][0].z, s[nt][0].w));
                    mx = fmaxf(mx, fmaxf(fmaxf(s[nt][1].x, s[nt][1].y), fmaxf(s[nt][1].z, s[nt][1].w)));
                    mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
                    mx = fmaxf(m[nt], fmaxf(mx, __shfl_xor(mx, 32, 64)));
                    ref[nt] = mx == -INFINITY ? 0.0f : mx;
                    const float f = exp2_(m[nt] - ref[nt]);
                    m[nt] = mx;
                    l[nt] *= f;
#pragma unroll
                    for (int d = 0; d < NB; ++d) o[nt][d] *= f;
                }
            }
            u4 ph[NT], pl[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    f4 x;
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = exp2_(s[nt][half][e] - ref[nt]);
                    l[nt] += (x.x + x.y) + (x.z + x.w);
                    x *= half ? vf1 : vf0;
                    uint32_t h0, l0, h1, l1;
                    pieces(x.x, x.y, h0, l0);
                    pieces(x.z, x.w, h1, l1);
                    ph[nt][2 * half] = h0, ph[nt][2 * half + 1] = h1;
                    pl[nt][2 * half] = l0, pl[nt][2 * half + 1] = l1;
                }
            }
            // values
            if (stored) {
                if (more) wait_loads<NI + 2>(); else wait_loads<2>();
            } else {
                if (more) wait_loads<NI>(); else wait_loads<0>();
            }
            uint32_t keep0 = ~0u, keep1 = ~0u;  // e4m3: NaN codes where nothing is held
            if (F == kE4m3 && !whole) {
                keep0 = keep1 = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    keep0 |= (pg0 >= 0 && t0 + 4 * g + e < r.len) ? 0xffu << (8 * e) : 0u;
                    keep1 |= (pg1 >= 0 && t0 + 16 + 4 * g + e < r.len) ? 0xffu << (8 * e) : 0u;
                }
            }
            constexpr int NR = NB <= 8 ? NB : NB / 2;  // blocks read at once
#pragma unroll
            for (int d0 = 0; d0 < NB; d0 += NR) {
                uint32_t at[NR];
                i2 w[NR];
#pragma unroll
                for (int d = 0; d < NR; ++d) at[d] = lds_at(vb) + (uint32_t)(vAt + (((d0 + d) ^ vSwap) * 16));
                read_values<NR>(at, w);
                if (more && d0 + NR == NB) issue(c.v, i + 1, vb);
#pragma unroll
                for (int d = 0; d < NR; ++d) {
                    if (F == kE4m3 && !whole) w[d].x &= keep0, w[d].y &= keep1;
                    const u4 x = codes16x8<F, CCB_KV8_BF16>(w[d].x, w[d].y);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        o[nt][d0 + d] = mfma<CCB_KV8_BF16>(x, ph[nt], o[nt][d0 + d]);
                        o[nt][d0 + d] = mfma<CCB_KV8_BF16>(x, pl[nt], o[nt][d0 + d]);
                    }
                }
            }
        };

        if (nTiles > 0) {
            issue(c.k, 0, kBuf[wave]);
            issue(c.v, 0, vBuf[wave]);
            asm volatile("" : "+v"(kScale), "+v"(vScale));
            for (int32_t i = 0; i < nTiles; ++i) step(i, kBuf[wave], vBuf[wave]);
        }
    }

    // join the waves
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        l[nt] += __shfl_xor(l[nt], 16, 64);
        l[nt] += __shfl_xor(l[nt], 32, 64);
        if (g == 0) sm[wave][nt * 16 + n] = m[nt], sl[wave][nt * 16 + n] = l[nt];
    }
    __syncthreads();
    const int64_t part = ((int64_t)pair * p.splits + split) * p.rows;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kRunWaves; ++w) top = fmaxf(top, sm[w][nt * 16 + n]);
        const float f = l[nt] == 0.0f ? 0.0f : exp2_(m[nt] - top);  // (a NaN stays)
        // chunks of 4 dimensions are swapped so that rows fall on different banks
        float* dst = (float*)(wave < kRunWaves / 2 ? kBuf[0] : vBuf[0]) + (wave % (kRunWaves / 2) * 16 + n) * D;
#pragma unroll
        for (int d = 0; d < NB; ++d) *(f4*)(dst + (((4 * d + g) ^ (n & 7)) * 4)) = o[nt][d] * f;
        __syncthreads();
        for (int32_t at = threadIdx.x; at < 4 * D; at += kRunThreads) {
            const int32_t i = at / (D / 4), d4 = at % (D / 4), row = row0 + nt * 16 + i;
            if (row >= p.rows) continue;
            f4 sum = {0, 0, 0, 0};
            float mm = -INFINITY, ll = 0.0f;
#pragma unroll
            for (int w = 0; w < kRunWaves; ++w) {
                const float* src = (const float*)(w < kRunWaves / 2 ? kBuf[0] : vBuf[0]);
                sum += *(const f4*)(src + (w % (kRunWaves / 2) * 16 + i) * D + ((d4 ^ (i & 7)) * 4));
                mm = fmaxf(mm, sm[w][nt * 16 + i]);
            }
#pragma unroll
            for (int w = 0; w < kRunWaves; ++w)
                ll += sl[w][nt * 16 + i] == 0.0f ? 0.0f : sl[w][nt * 16 + i] * exp2_(sm[w][nt * 16 + i] - mm);
            if (p.direct) {
                write_row<T>(p, b, h, pair, row, d4, sum, mm, ll);
                if (d4 == 0) slse[nt * 16 + i] = ll != 0.0f ? mm + log2f(ll) : INFINITY;
            } else {
                *(f4*)(p.partO + (part + row) * D + d4 * 4) = sum;
                if (d4 == 0) p.partML[part + row] = make_float2(mm, ll);
            }
        }
        __syncthreads();
    }
    if (p.direct && p.scores != nullptr) {
        // this workgroup has all scores of its head: add the weights at once
        float* w = c.weight + (int64_t)pair * c.weightStride;
        for (int32_t t0 = r.first + (int32_t)threadIdx.x; t0 < r.len; t0 += 4 * kRunThreads) {
            float old[4], x[4];  // four tokens' loads in flight
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int32_t t = t0 + k * kRunThreads;
                old[k] = t < r.len ? w[t] : 0.0f;
                x[k] = 0.0f;
            }
            for (int32_t i = 0; i < p.rows; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int32_t t = t0 + k * kRunThreads;
                    if (t < r.len) x[k] += exp2_(score_at(p, pair, i, t - r.base)[0] - slse[i]);
                }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int32_t t = t0 + k * kRunThreads;
                if (t < r.len) w[t] = old[k] + x[k];
            }
        }
    }
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

// Join the runs of a sequence's tokens: rows (out and lse), four to a
// workgroup, or one where there are many runs; and tokens (weights, from the
// stored scores).  A workgroup a row took 10 us for 2048 rows of 2 runs, a
// wave a row takes 5.
template <int T>
__global__ __launch_bounds__(kThreads) void kv8_k_join(Plan p, int32_t D)
{
    __shared__ f4 sum[kThreads];
    __shared__ float factor[kThreads];
    const ccb::Kv8AttendArgs& a = p.a;
    const ccbKv8Cache& c = a.c;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t V = D / 4;  // vectors of a row
    const int64_t step = (int64_t)p.rows * D;

    if (blockIdx.x < (uint32_t)p.joinRows) {
        const bool many = p.splits > kJoinRuns;
        const int64_t at = many ? blockIdx.x : (int64_t)blockIdx.x * kWaves + wave;
        const int32_t pair = (int32_t)(at / p.rows), row = (int32_t)(at % p.rows);
        if (pair >= p.pairs) return;  // (not where the workgroup works together)
        const int32_t h = pair % c.heads, b = pair / c.heads;
        const Range r = range_of(p, b);
        const int32_t n = r.runs;
        const float2* ml = p.partML + (int64_t)pair * p.splits * p.rows + row;
        float top = -INFINITY, all = 0.0f;
        for (int32_t s = lane; s < n; s += 64) {
            const float2 x = ml[(int64_t)s * p.rows];
            merge(top, all, x.x, x.y);
        }
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) merge(top, all, __shfl_xor(top, d, 64), __shfl_xor(all, d, 64));
        // threads of a row: V for the vectors, and runs side by side
        const int32_t me = many ? tid : lane, groups = (many ? kThreads : 64) / V;
        const int32_t d4 = me % V, sg = me / V;
        const float* src = p.partO + ((int64_t)pair * p.splits * p.rows + row) * D + d4 * 4;
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
            write_row<T>(p, b, h, pair, row, d4, o, top, all);
        }
        return;
    }
    const int32_t pair = (blockIdx.x - p.joinRows) % (uint32_t)p.pairs;
    const int32_t from = (int32_t)((blockIdx.x - p.joinRows) / (uint32_t)p.pairs) * p.joinSpan;  // from base
    const Range r = range_of(p, pair / c.heads);
    if (r.base + (int64_t)from >= r.len) return;
    const int32_t n = r.runs;
    const float2* ml = p.partML + (int64_t)pair * p.splits * p.rows;
    // every row's lse: 16 threads each, or one for many rows of few runs
    const int32_t team = n <= 16 && p.rows > 16 ? 1 : 16;
    for (int32_t row = tid / team; row < p.rows; row += kThreads / team) {
        float top = -INFINITY, all = 0.0f;
#pragma unroll 8
        for (int32_t s = tid % team; s < n; s += team) {
            const float2 x = ml[(int64_t)s * p.rows + row];
            merge(top, all, x.x, x.y);
        }
        for (int d = team >> 1; d >= 1; d >>= 1)
            merge(top, all, __shfl_xor(top, d, 64), __shfl_xor(all, d, 64));
        if (tid % team == 0) factor[row] = all != 0.0f ? top + log2f(all) : INFINITY;
    }
    __syncthreads();
    // A lane takes four tokens.  Few rows: every thread its own tokens and all
    // rows; many: a wave takes every fourth row of the same 256 tokens, so that
    // the loads of a row do not queue up behind each other.
    const bool shared = p.joinSpan == 4 * 64;
    const int32_t at = from + 4 * (shared ? lane : tid), by = shared ? kWaves : 1;
    const float* sc = score_at(p, pair, 0, at);
    float* w = c.weight + (int64_t)pair * c.weightStride;
    f4 x = {0, 0, 0, 0};
    if (r.base + (int64_t)at < r.len) {
#pragma unroll 4
        for (int32_t i = shared ? wave : 0; i < p.rows; i += by) {
            const f4 s = *(const f4*)(sc + i * kTile);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] += exp2_(s[e] - factor[i]);
        }
    }
    if (shared) {
        sum[tid] = x;
        __syncthreads();
        const int32_t t = r.base + from + tid;  // now a thread to a token
        const float* one = (const float*)sum;
        if (t >= r.first && t < r.len)
            w[t] += (one[tid] + one[256 + tid]) + (one[512 + tid] + one[768 + tid]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int32_t t = r.base + at + e;
            if (t >= r.first && t < r.len) w[t] += x[e];
        }
    }
}

// Weights of many rows: the scores again, S = Q K^T so that a token's rows lie
// on one lane index.  One wave takes 32 tokens and goes over all rows.
template <int F, int T, int D>
__global__ __launch_bounds__(kThreads) void kv8_k_weights(Plan p, int32_t blocks)
{
    constexpr int NJ = D / 32;
    const ccb::Kv8AttendArgs& a = p.a;
    const ccbKv8Cache& c = a.c;
    const int32_t pair = blockIdx.x % (uint32_t)p.pairs, part = blockIdx.x / (uint32_t)p.pairs;
    const int32_t h = pair % c.heads, b = pair / c.heads;
    const int32_t P = c.pageSize, group = a.headsQ / c.heads;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = lane & 15, g = lane >> 4;
    const Range r = range_of(p, b);
    for (int64_t from = (int64_t)r.base + ((int64_t)part * kWaves + wave) * kTile;
         from < r.len; from += (int64_t)blocks * kWaves * kTile) {
        u4 k[2][NJ];
        float kf[2];
        bool held[2];
        int32_t tok[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int32_t t = tok[half] = (int32_t)from + 16 * half + n;
            const int32_t page = t < r.len && t >= r.first
                                     ? checked_page(c.pageTable[b * c.tableStride + t / P], c.numPages)
                                     : -1;
            held[half] = page >= 0;
            const int64_t block = (int64_t)(page < 0 ? 0 : page) * c.heads + h;
            kf[half] = held[half] ? c.kScale[block] * (a.scale * kLog2e) : 0.0f;
            const uint8_t* src = (const uint8_t*)c.k + (block * P + (t & (P - 1))) * D;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const uint2 w = *(const uint2*)(src + 32 * j + 8 * g);
                k[half][j] = codes16x8<F, T>(w.x, w.y);
            }
        }
        float sum[2] = {0.0f, 0.0f};
        for (int32_t row0 = 0; row0 < p.rows; row0 += 16) {
            const int32_t row = row0 + n;
            const uint16_t* src =
                (const uint16_t*)a.q.data + row_at(a.q, b, h, row < p.rows ? row : row0, group);
            f4 s[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const u4 q = *(const u4*)(src + 32 * j + 8 * g);
                s[0] = mfma<T>(q, k[0][j], s[0]);
                s[1] = mfma<T>(q, k[1][j], s[1]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                int32_t begin, end;
                seen_by(a, r, row0 + 4 * g + e, p.rows, group, begin, end);
                const float lse = end > begin ? p.lse2[(int64_t)pair * p.rows + row0 + 4 * g + e] : INFINITY;
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    if (held[half] && tok[half] >= begin && tok[half] < end)
                        sum[half] += exp2_(s[half][e] * kf[half] - lse);
            }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            sum[half] += __shfl_xor(sum[half], 16, 64);
            sum[half] += __shfl_xor(sum[half], 32, 64);
            if (g == 0 && held[half])
                c.weight[(int64_t)pair * c.weightStride + tok[half]] += sum[half];
        }
    }
}

// How a call is split, and where its workspace's parts lie; returns its bytes,
// which do not depend on the window.  There is a sequence and a query.
size_t make_plan(Plan& p, const ccbKv8Cache& c, int32_t headsQ, int32_t nQuery, int32_t window,
                 int32_t accumulate, void* ws)
{
    const int64_t pairs = (int64_t)c.batch * c.heads;
    const int64_t rows = (int64_t)nQuery * (headsQ / c.heads);
    p.pairs = (int32_t)pairs;
    p.rows = (int32_t)rows;
    // tokens that a sequence's queries may see, from a tile's border
    const int64_t room = (int64_t)c.maxPages * c.pageSize;
    int64_t span = room;
    if (window > 0 && (int64_t)window + nQuery - 1 + kTile < span)
        span = (int64_t)window + nQuery - 1 + kTile;
    // One workgroup of 8 waves for each CU: a second one pays its first loads'
    // latency once more and brings no bandwidth.  Against two (of 8 waves, or
    // four of 4) a CU, 16 sequences of 4096 tokens take 28.5 us instead of 31.1;
    // where lengths spread from 500 to 4096 it is 27.3 instead of 25.2.  More,
    // up to 16 a CU, where a run could pass 2 MB of codes: many short sequences
    // do not wait for a long one's end.
    constexpr int64_t target = 256, limit = 16 * target;
    auto up = [](int64_t x, int64_t by) { return (x + by - 1) / by; };
    auto runs = [&](int64_t tokens, int64_t groups) {
        const int64_t byLength = up(tokens, (1 << 20) / c.headDim), mostHere = limit / groups;
        int64_t n = byLength < mostHere ? byLength : mostHere;
        n = n > target / groups ? n : target / groups;
        n = n < up(tokens, kRunUnit) ? n : up(tokens, kRunUnit);
        return n > 1 && tokens > 256 ? n : 1;
    };
    // Two tiles of rows share a key's conversion, which pays (10% for 64 rows)
    // where their accumulators leave room for enough waves, and where a
    // workgroup more for the other rows would have to wait for its place.
    const int64_t tilesOfRows = up(rows, 16);
    p.tilesN = rows > 16 && c.headDim <= 96 && pairs * up(span, kRunUnit) * tilesOfRows > target ? 2 : 1;
    p.rowBlocks = (int32_t)up(rows, 16 * p.tilesN);
    p.splits = (int32_t)runs(span, pairs * p.rowBlocks);
    p.tiles = (int32_t)up(span, kTile);
    const int64_t mostSplits = runs(room, pairs);  // over every window
    size_t bytes = 0;
    auto take = [&](int64_t n, size_t each) {
        char* here = (char*)ws + bytes;
        bytes += ((size_t)n * each + 127) / 128 * 128;
        return here;
    };
    const bool stored = accumulate && ccb::kv8_attend_keeps_scores(c, headsQ, nQuery);
    p.direct = p.splits == 1 && (p.rowBlocks == 1 || !stored);
    const int64_t parts = mostSplits > 1 || rows > 16 ? pairs * mostSplits * rows : 0;
    p.partO = (float*)take(parts * c.headDim, sizeof(float));
    p.partML = (float2*)take(parts, sizeof(float2));
    p.scores = nullptr, p.lse2 = nullptr;
    if (stored)
        p.scores = (float*)take(pairs * rows * up(room, kTile), kTile * sizeof(float));
    else if (accumulate)
        p.lse2 = (float*)take(pairs * rows, sizeof(float));
    p.joinRows = (int32_t)(p.splits > kJoinRuns ? pairs * rows : up(pairs * rows, kWaves));
    p.joinSpan = rows <= 16 ? 4 * kThreads : 4 * 64;
    p.joinBlocks = p.joinRows + (p.scores != nullptr ? pairs * up(span, p.joinSpan) : 0);
    return bytes;
}

// Workgroups that share a pair's tokens when the weights are computed again.
int64_t weight_blocks(const Plan& p, int64_t pairs)
{
    const int64_t each = ((int64_t)p.tiles + kWaves - 1) / kWaves;
    const int64_t most = pairs < 4096 ? 8192 / pairs : 2;
    return each < most ? each : most;
}

template <int F, int T, int D>
hipError_t launch(const Plan& p, int64_t blocks, hipStream_t s)
{
    hipError_t e = hipSuccess;
    if (p.tilesN == 1)
        e = enqueue(kv8_k_attend<F, T, D, 1>, blocks, kRunThreads, s, p);
    else if constexpr (D <= 96)
        e = enqueue(kv8_k_attend<F, T, D, 2>, blocks, kRunThreads, s, p);
    if (e == hipSuccess && !p.direct) e = enqueue(kv8_k_join<T>, p.joinBlocks, kThreads, s, p, D);
    if (e == hipSuccess && p.lse2 != nullptr) {
        const int64_t each = weight_blocks(p, p.pairs);
        e = enqueue(kv8_k_weights<F, T, D>, p.pairs * each, kThreads, s, p, (int32_t)each);
    }
    return e;
}

}  // namespace

namespace ccb {

size_t kv8_attend_bytes(const ccbKv8Cache& c, int32_t headsQ, int32_t nQuery, int32_t accumulate)
{
    if (c.batch == 0 || nQuery == 0) return 0;
    Plan p;
    return make_plan(p, c, headsQ, nQuery, 0, accumulate, nullptr);
}

bool kv8_attend_fits(const ccbKv8Cache& c, int32_t headsQ, int32_t nQuery, int32_t window, int32_t accumulate,
                     size_t wsBytes)
{
    const int64_t pairs = (int64_t)c.batch * c.heads;
    if (pairs > INT32_MAX) return false;
    Plan p;
    return make_plan(p, c, headsQ, nQuery, window, accumulate, nullptr) <= wsBytes &&
           kv8_launch_fits(pairs * p.rowBlocks * p.splits, kRunThreads) && pairs * p.rows <= INT32_MAX &&
           (p.direct || kv8_launch_fits(p.joinBlocks, kThreads)) &&
           (!accumulate || kv8_attend_keeps_scores(c, headsQ, nQuery) ||
            kv8_launch_fits(pairs * weight_blocks(p, pairs), kThreads));
}

hipError_t kv8_attend(const Kv8AttendArgs& a, hipStream_t s)
{
    const ccbKv8Cache& c = a.c;
    Plan p;
    p.a = a;
    make_plan(p, c, a.headsQ, a.nQuery, a.window, a.accumulate, a.ws);
    const int64_t blocks = (int64_t)p.pairs * p.rowBlocks * p.splits;
#define KV8_ATTEND_DIM(F, T) \
    switch (c.headDim) { \
    case 64: return launch<F, T, 64>(p, blocks, s); \
    case 96: return launch<F, T, 96>(p, blocks, s); \
    case 128: return launch<F, T, 128>(p, blocks, s); \
    case 192: return launch<F, T, 192>(p, blocks, s); \
    default: return launch<F, T, 256>(p, blocks, s); \
    }
    if (c.format == CCB_KV8_INT8) {
        if (a.q.type == CCB_KV8_BF16) KV8_ATTEND_DIM(kInt8, CCB_KV8_BF16)
        KV8_ATTEND_DIM(kInt8, CCB_KV8_FP16)
    }
    if (a.q.type == CCB_KV8_BF16) KV8_ATTEND_DIM(kE4m3, CCB_KV8_BF16)
    KV8_ATTEND_DIM(kE4m3, CCB_KV8_FP16)
}

}  // namespace ccb

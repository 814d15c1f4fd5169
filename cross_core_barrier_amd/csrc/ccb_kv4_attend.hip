// ccb_kv4_attend.hip -- attention of a decoding step over the 4-bit key/value
// cache, in one pass over the codes on the matrix cores, split over tokens.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ccb_kv4_internal.h"
#include "ccb_kv8_device.h"

namespace {

using namespace kv8;

constexpr int kThreads = 512;  // of a workgroup that takes a run of tokens
constexpr int kWaves = kThreads / 64;
constexpr int kJoinThreads = 256;
constexpr int kTile = 32;                     // tokens of a wave's step
constexpr int kRunUnit = kWaves * kTile;
constexpr int kSegment = 32 * kWaves * kTile;  // tokens whose pages fit a wave's lanes
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
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
    int32_t pairs;      // (sequence, cache head)
    int32_t rows;       // of a cache head
    int32_t tilesN;     // NT
    int32_t rowBlocks;  // workgroups that share a run of tokens
    int32_t splits;     // runs of a sequence, see range_of
    float* partO;       // [pair][split][row][D], unused for one run
    float2* partML;     // [pair][split][row]: maximum (base 2) and sum
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
    const bf2 l = {(__bf16)(a - of_bits(hi << 16)), (__bf16)(b - of_bits(hi & 0xffff0000u))};
    lo = __builtin_bit_cast(uint32_t, l);
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

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
    const ccb::Kv4AttendArgs& a = p.a;
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
__device__ __forceinline__ void seen_by(const ccb::Kv4AttendArgs& a, const Range& r, int32_t row, int32_t rows,
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

// How the chunks of 16 dimensions (32 bytes) of a token's values are swapped in
// LDS, so that the 8 tokens that half a wave reads at one chunk fall on all the banks.
template <int D>
__device__ __forceinline__ int swap_of(int t)
{
    return D == 64 || D == 192 ? (t >> 1) & 3 : D == 96 ? (t >> 2) & 1 : t & 7;
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

// One half (16 tokens) of a wave's tile, keys or values: a lane's D / 4
// dimensions of token n, and the scales of the first and the last of them (no
// lane has more than two).
template <int D>
struct Half {
    uint32_t w[D / 32];
    uint32_t s0, s1;

    // dimensions g * D/4 + 8 j .. + 7 lie under the scale (g * D/4 + 8 j) / 32
    static __device__ __forceinline__ int group_at(int g, int j) { return (g * (D / 32) + j) >> 2; }

    // from the codes and scales of the half's 16 rows
    __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, int n, int g)
    {
        const uint8_t* src = codes + (n * (D / 2) + g * (D / 8));
        if constexpr (D == 64) {
            const u2 x = *(const u2*)src;
            w[0] = x.x, w[1] = x.y;
        } else if constexpr (D == 96) {
            const uint32_t* x = (const uint32_t*)src;
            w[0] = x[0], w[1] = x[1], w[2] = x[2];
        } else if constexpr (D == 192) {
            const u2* x = (const u2*)src;
#pragma unroll
            for (int i = 0; i < 3; ++i) w[2 * i] = x[i].x, w[2 * i + 1] = x[i].y;
        } else {
            const u4* x = (const u4*)src;
#pragma unroll
            for (int i = 0; i < D / 128; ++i) w[4 * i] = x[i].x, w[4 * i + 1] = x[i].y, w[4 * i + 2] = x[i].z, w[4 * i + 3] = x[i].w;
        }
        const uint8_t* s = scales + n * (D / 32);
        s0 = s[group_at(g, 0)];
        s1 = D <= 128 && D != 96 ? s0 : s[group_at(g, D / 32 - 1)];
    }

    // words 8 j .. 8 j + 7 as bf16
    __device__ __forceinline__ u4 values(int j, int g, float f0, float f1) const
    {
        if constexpr (D == 64 || D == 128) return decode8(w[j], f0);
        return decode8(w[j], group_at(g, j) == group_at(g, 0) ? f0 : f1);
    }
};

template <int D>
struct Tile {
    Half<D> k[2], v[2];
};

template <int T, int D, int NT>
__global__ __launch_bounds__(kThreads, 2) void kv4_k_attend(Plan p)
{
    constexpr int NB = D / 16;                          // blocks of 16 dimensions
    constexpr int NJ = D / 32;                          // steps of the first product
    constexpr int NQ = T == CCB_KV8_BF16 ? 1 : 2;       // bf16 pieces of a query: exact
    __shared__ __attribute__((aligned(16))) uint8_t vBuf[kWaves][kTile * D * 2];
    __shared__ float sm[kWaves][16 * NT], sl[kWaves][16 * NT];

    const ccb::Kv4AttendArgs& a = p.a;
    const ccbKv4Cache& c = a.c;
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
    const int32_t laneAt = ((lane >> 1) * kWaves + wave) * kTile + (lane & 1) * 16;
    const int32_t* table = c.pageTable + b * c.tableStride;

    const Range r = range_of(p, b);
    if (split > 0 && split >= r.runs) return;  // the join knows
    const int32_t lo = r.base + split * r.chunk;
    const int32_t hi = r.len - lo < r.chunk ? r.len : lo + r.chunk;

    // Queries, 8 values of a row per lane and step (a row that is not there
    // computes row0's again, for nothing).  Scores are scaled by |scale|, a
    // negative one turns the queries' signs.
    const float scale2 = fabsf(a.scale) * kLog2e;
    u4 q[NT][NJ][NQ];
    int32_t begin[NT], end[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int32_t row = row0 + nt * 16 + n;
        seen_by(a, r, row, p.rows, group, begin[nt], end[nt]);
        const uint16_t* src = (const uint16_t*)a.q.data + row_at(a.q, b, h, row < p.rows ? row : row0, group) + g * (D / 4);
        const uint32_t turn = a.scale < 0 ? 0x80008000u : 0u;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            u4 x = *(const u4*)(src + 8 * j);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] ^= turn;
            if constexpr (NQ == 1) {
                q[nt][j][0] = x;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t hi, low;
                    pieces(widen<T>(x[e] & 0xffffu), widen<T>(x[e] >> 16), hi, low);
                    q[nt][j][0][e] = hi, q[nt][j][NQ - 1][e] = low;
                }
            }
        }
    }
    // tokens in [allBegin, allEnd) are seen by every row of the workgroup
    int32_t allBegin, allEnd, unused;
    {
        const int32_t last = row0 + 16 * NT < p.rows ? row0 + 16 * NT - 1 : p.rows - 1;
        seen_by(a, r, last, p.rows, group, allBegin, unused);
        seen_by(a, r, row0, p.rows, group, unused, allEnd);
    }

    f4 o[NT][NB];
    float m[NT], ref[NT], l[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt] = -INFINITY, ref[nt] = 0.0f, l[nt] = 0.0f;
#pragma unroll
        for (int d = 0; d < NB; ++d) o[nt][d] = f4{0, 0, 0, 0};
    }

    // where this lane reads values: 4 lanes for a token's 16 dimensions
    const int vTok = 4 * g + (n >> 2);
    uint8_t* const buf = vBuf[wave];
    const uint8_t* const vFrom[2] = {buf + vTok * (2 * D) + (n & 3) * 8, buf + (16 + vTok) * (2 * D) + (n & 3) * 8};
    const int vSwap = swap_of<D>(vTok), wSwap = swap_of<D>(n);  // alike for token 16 + x

    for (int32_t seg = lo; seg < hi; seg += kSegment) {
        const int32_t segEnd = hi - seg < kSegment ? hi : seg + kSegment;
        // lane i holds the page of the wave's i-th half tile
        int32_t page = -1;
        {
            const int32_t t = seg + laneAt;
            if (t < segEnd && t + 16 > r.first) {
                page = checked_page(table[t >> shift], c.numPages);
                if (page < 0) report(a.err);
            }
        }
        const int32_t nTiles = ((segEnd - seg + kTile - 1) / kTile - wave + kWaves - 1) / kWaves;

        auto load = [&](int32_t i, Tile<D>& x) {
            const int32_t t = seg + (i * kWaves + wave) * kTile;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                int32_t pg = __builtin_amdgcn_readlane(page, 2 * i + half);
                pg = pg < 0 ? 0 : pg;  // an unseen page's place: page 0 is loaded and not used
                const int64_t row = ((int64_t)pg * c.heads + h) * P + ((t + 16 * half) & (P - 1));
                x.k[half].load(c.k + row * (D / 2), c.kScale + row * (D / 32), n, g);
                x.v[half].load(c.v + row * (D / 2), c.vScale + row * (D / 32), n, g);
            }
        };

        auto step = [&](int32_t i, Tile<D>& x) {
            const int32_t t0 = seg + (i * kWaves + wave) * kTile;
            const int32_t pg0 = __builtin_amdgcn_readlane(page, 2 * i);
            const int32_t pg1 = __builtin_amdgcn_readlane(page, 2 * i + 1);
            const bool whole = t0 >= allBegin && t0 + kTile <= allEnd && (pg0 | pg1) >= 0;
            // scores
            f4 s[NT][2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float f0 = of_bits(x.k[half].s0 << 23), f1 = of_bits(x.k[half].s1 << 23);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) s[nt][half] = f4{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const u4 key = x.k[half].values(j, g, f0, f1);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < NQ; ++k) s[nt][half] = mfma(key, q[nt][j][k], s[nt][half]);
                }
            }
            float by = scale2;
            bool grows = false;
            if (!whole) {
                by = 1.0f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int32_t t = t0 + 4 * g + e;
                        s[nt][0][e] = t >= begin[nt] && t < end[nt] && pg0 >= 0 ? s[nt][0][e] * scale2 : -INFINITY;
                        s[nt][1][e] = t + 16 >= begin[nt] && t + 16 < end[nt] && pg1 >= 0 ? s[nt][1][e] * scale2 : -INFINITY;
                    }
                // values that are not there: any scale, but a number
                if (!(pg0 >= 0 && t0 + n < r.len)) x.v[0].s0 = x.v[0].s1 = 127;
                if (!(pg1 >= 0 && t0 + 16 + n < r.len)) x.v[1].s0 = x.v[1].s1 = 127;
            }
            // values into LDS, as bf16
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float f0 = of_bits(x.v[half].s0 << 23), f1 = of_bits(x.v[half].s1 << 23);
                uint8_t* dst = buf + (16 * half + n) * (2 * D);
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const int at = g * NJ + j;  // of 8 dimensions
                    *(u4*)(dst + ((((at >> 1) ^ wSwap) << 5) | ((at & 1) << 4))) = x.v[half].values(j, g, f0, f1);
                }
            }
            float mx[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mx[nt] = fmaxf(fmaxf(s[nt][0].x, s[nt][0].y), fmaxf(s[nt][0].z, s[nt][0].w));
                mx[nt] = fmaxf(mx[nt], fmaxf(fmaxf(s[nt][1].x, s[nt][1].y), fmaxf(s[nt][1].z, s[nt][1].w))) * by;
                grows |= mx[nt] > m[nt] + kSlack;
            }
            if (__any(grows)) {  // a new maximum, for the row's four lanes alike
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float top = fmaxf(mx[nt], __shfl_xor(mx[nt], 16, 64));
                    top = fmaxf(m[nt], fmaxf(top, __shfl_xor(top, 32, 64)));
                    ref[nt] = top == -INFINITY ? 0.0f : top;
                    const float f = exp2_(m[nt] - ref[nt]);
                    m[nt] = top;
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
                    f4 y;
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = exp2_(fmaf(s[nt][half][e], by, -ref[nt]));
                    l[nt] += (y.x + y.y) + (y.z + y.w);
                    uint32_t h0, l0, h1, l1;
                    pieces(y.x, y.y, h0, l0);
                    pieces(y.z, y.w, h1, l1);
                    ph[nt][2 * half] = h0, ph[nt][2 * half + 1] = h1;
                    pl[nt][2 * half] = l0, pl[nt][2 * half + 1] = l1;
                }
            }
            // a wave's LDS accesses keep the program's order
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int d = 0; d < NB; ++d) {
                typedef __attribute__((address_space(3))) s4 lds4;
                const s4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(vFrom[0] + ((d ^ vSwap) << 5)));
                const s4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(vFrom[1] + ((d ^ vSwap) << 5)));
                const u2 y0 = __builtin_bit_cast(u2, v0), y1 = __builtin_bit_cast(u2, v1);
                const u4 y = {y0.x, y0.y, y1.x, y1.y};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    o[nt][d] = mfma(y, ph[nt], o[nt][d]);
                    o[nt][d] = mfma(y, pl[nt], o[nt][d]);
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        };

        // One tile ahead; the last is asked for again, so that the number of
        // loads in flight is the same in every step.
        if (nTiles > 0) {
            Tile<D> x, y;
            load(0, x);
            for (int32_t i = 0; i < nTiles; i += 2) {
                load(i + 1 < nTiles ? i + 1 : i, y);
                step(i, x);
                if (i + 1 >= nTiles) break;
                load(i + 2 < nTiles ? i + 2 : i + 1, x);
                step(i + 1, y);
            }
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
        for (int w = 0; w < kWaves; ++w) top = fmaxf(top, sm[w][nt * 16 + n]);
        const float f = l[nt] == 0.0f ? 0.0f : exp2_(m[nt] - top);  // (a NaN stays)
        // chunks of 4 dimensions are swapped so that rows fall on different banks
        float* dst = (float*)vBuf[wave] + n * D;
#pragma unroll
        for (int d = 0; d < NB; ++d) *(f4*)(dst + (((4 * d + g) ^ (n & 7)) * 4)) = o[nt][d] * f;
        __syncthreads();
        for (int32_t at = threadIdx.x; at < 4 * D; at += kThreads) {
            const int32_t i = at / (D / 4), d4 = at % (D / 4), row = row0 + nt * 16 + i;
            if (row >= p.rows) continue;
            f4 sum = {0, 0, 0, 0};
            float mm = -INFINITY, ll = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                sum += *(const f4*)((const float*)vBuf[w] + i * D + ((d4 ^ (i & 7)) * 4));
                mm = fmaxf(mm, sm[w][nt * 16 + i]);
            }
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                ll += sl[w][nt * 16 + i] == 0.0f ? 0.0f : sl[w][nt * 16 + i] * exp2_(sm[w][nt * 16 + i] - mm);
            if (p.splits == 1) {
                write_row<T>(p, b, h, row, d4, sum, mm, ll);
            } else {
                *(f4*)(p.partO + (part + row) * D + d4 * 4) = sum;
                if (d4 == 0) p.partML[part + row] = make_float2(mm, ll);
            }
        }
        __syncthreads();
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
    const bool many = p.splits > kJoinRuns;
    const int64_t at = many ? blockIdx.x : (int64_t)blockIdx.x * kJoinWaves + wave;
    const int32_t pair = (int32_t)(at / p.rows), row = (int32_t)(at % p.rows);
    if (pair >= p.pairs) return;  // (not where the workgroup works together)
    const int32_t h = pair % p.a.c.heads, b = pair / p.a.c.heads;
    const int32_t n = range_of(p, b).runs;
    const float2* ml = p.partML + (int64_t)pair * p.splits * p.rows + row;
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
        write_row<T>(p, b, h, row, d4, o, top, all);
    }
}

// How a call is split, and where its workspace's parts lie; returns its bytes,
// which do not depend on the window.  There is a sequence and a query.
size_t make_plan(Plan& p, const ccbKv4Cache& c, int32_t headsQ, int32_t nQuery, int32_t window, void* ws)
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
    constexpr int64_t target = 256, limit = 16 * target;
    auto up = [](int64_t x, int64_t by) { return (x + by - 1) / by; };
    auto runs = [&](int64_t tokens, int64_t groups) {
        const int64_t byLength = up(tokens, (1 << 21) / c.headDim), mostHere = limit / groups;
        int64_t n = byLength < mostHere ? byLength : mostHere;
        n = n > target / groups ? n : target / groups;
        n = n < up(tokens, kRunUnit) ? n : up(tokens, kRunUnit);
        return n > 1 && tokens > 256 ? n : 1;
    };
    p.tilesN = 1;
    p.rowBlocks = (int32_t)up(rows, 16 * p.tilesN);
    p.splits = (int32_t)runs(span, pairs * p.rowBlocks);
    const int64_t mostSplits = runs(room, pairs);  // over every window
    size_t bytes = 0;
    auto take = [&](int64_t n, size_t each) {
        char* here = (char*)ws + bytes;
        bytes += ((size_t)n * each + 127) / 128 * 128;
        return here;
    };
    const int64_t parts = mostSplits > 1 || rows > 16 ? pairs * mostSplits * rows : 0;
    p.partO = (float*)take(parts * c.headDim, sizeof(float));
    p.partML = (float2*)take(parts, sizeof(float2));
    return bytes;
}

int64_t join_groups(const Plan& p)
{
    const int64_t rows = (int64_t)p.pairs * p.rows;
    return p.splits > kJoinRuns ? rows : (rows + 3) / 4;
}

template <int T, int D>
hipError_t launch(const Plan& p, hipStream_t s)
{
    const int64_t groups = (int64_t)p.pairs * p.rowBlocks * p.splits;
    hipError_t e = enqueue(kv4_k_attend<T, D, 1>, groups, kThreads, s, p);
    if (e == hipSuccess && p.splits > 1) e = enqueue(kv4_k_join<T>, join_groups(p), kJoinThreads, s, p, D);
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
    const int64_t pairs = (int64_t)c.batch * c.heads;
    if (pairs > INT32_MAX) return false;
    Plan p;
    return make_plan(p, c, headsQ, nQuery, window, nullptr) <= wsBytes && pairs * p.rows <= INT32_MAX &&
           kv8_launch_fits(pairs * p.rowBlocks * p.splits, kThreads) && kv8_launch_fits(join_groups(p), kJoinThreads);
}

hipError_t kv4_attend(const Kv4AttendArgs& a, hipStream_t s)
{
    Plan p;
    p.a = a;
    make_plan(p, a.c, a.headsQ, a.nQuery, a.window, a.ws);
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

// What the kernels of attention over the paged 4-bit cache share: a call's work as
// one line of steps, cut into equal stretches for the workgroups, and the joins of the parts
// that stretches leave of a row.
#pragma once

#include "cache4.hpp"
#include "common.hpp"

namespace dq {

namespace {

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ uint32_t u32_of(f16x2_t v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ f16x2_t f16x2_of(uint32_t v) { return __builtin_bit_cast(f16x2_t, v); }

// Reductions over the four lanes of a row (l, l ^ 16, l ^ 32, l ^ 48): a swap
// of 32-lane halves, then of odd and even 16-lane rows, each leaving the pair's
// two values in every lane of the pair.
__device__ __forceinline__ void row_pair(float v, bool half, float& x, float& y)
{
    typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
    const uint32_t u = __float_as_uint(v);
    const u32x2_t r = half ? __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(u, u, false, false))
                           : __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane16_swap(u, u, false, false));
    x = __uint_as_float(r.x);
    y = __uint_as_float(r.y);
}
__device__ __forceinline__ float row_max(float v)
{
    float x, y;
    row_pair(v, true, x, y);
    row_pair(fmaxf(x, y), false, x, y);
    return fmaxf(x, y);
}
__device__ __forceinline__ float row_sum(float v)
{
    float x, y;
    row_pair(v, true, x, y);
    row_pair(x + y, false, x, y);
    return x + y;
}
// max within 16 lanes (row_ror 8, 4, 2, 1), and over the wave of values that are
// not negative, NaN counting as 0; the same in every lane
template <int kRor>
__device__ __forceinline__ uint32_t ror_max(uint32_t u)
{
    const uint32_t t = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x120 + kRor, 0xf, 0xf, false);
    return max(u, t);
}
__device__ __forceinline__ uint32_t row16_max(uint32_t u)
{
    return ror_max<1>(ror_max<2>(ror_max<4>(ror_max<8>(u))));
}
// Keeps v computed here, in a register: a value that is used behind a branch
// would else be computed there, its operands kept alive until then.
template <class T>
__device__ __forceinline__ void pin(T& v)
{
    asm volatile("" : "+v"(v));
}

// 2^n for n clamped to fp32's normal range
__device__ __forceinline__ float pow2(int n)
{
    n = n < -126 ? -126 : (n > 127 ? 127 : n);
    return __uint_as_float((uint32_t)(n + 127) << 23);
}
// floor(log2 v) of a normal v (-127 for zero and subnormals, 128 for inf / NaN)
__device__ __forceinline__ int exponent(float v)
{
    return (int)((__float_as_uint(v) >> 23) & 0xff) - 127;
}

struct AttnArgs {
    Cache4 c;
    Cache4Batch bt;
    const uint16_t* q;
    int64_t q_stride;
    uint16_t* out;
    int64_t tokens;
    int32_t q_heads;
    float scale_log2;
    float* part;      // unfinished tiles: normalised outputs [workgroup, 2, 16, D]
    float2* part_ml;  // and their maxima and sums [workgroup, 2, 16]
    int32_t groups;   // workgroups of the attention kernel
    int32_t step_shift;  // log2 of a step's positions; 31: a unit is one step
};

// The scale that the quantizer stores for a group whose codes are all 0: fl32(1 / 7).
constexpr uint32_t kZeroScale = 0x3e124925u;

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;
constexpr int kStep = 32;                // positions per wave and step
constexpr int kStride = kWaves * kStep;  // positions per workgroup and step

// a / b of values that are not negative: the 64-bit division is some hundred
// instructions, and these nearly always fit 32 bits.
__device__ __forceinline__ int64_t udiv(int64_t a, int64_t b)
{
    if ((((uint64_t)a | (uint64_t)b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
    return a / b;
}

// Longest sequence: positions a few steps past its end are still below 2^31.
constexpr int kMaxLen = 0x7fff0000;

// What a workgroup knows of its sequence.  Token rows and positions are below 2^31.
struct Rows {
    int first, nq, len;  // first token row, new tokens, cached tokens
    int held;            // of them inside the table; rows that see more are NaN
    bool bad;            // longer than kMaxLen
    int per;             // query heads of a kv head
    __device__ __forceinline__ int64_t rows() const { return (int64_t)nq * per; }
    // positions seen by row r (a new token's head)
    __device__ __forceinline__ int seen(int64_t r) const { return len - nq + (int)udiv(r, per) + 1; }
};

__device__ __forceinline__ Rows rows_of(const AttnArgs& a, int64_t b)
{
    Rows r;
    int64_t first, nq;
    cache4_rows(a.bt, b, a.tokens, first, nq);
    r.first = (int)first;
    r.nq = (int)nq;
    r.len = a.bt.lens[b];
    r.bad = r.len > kMaxLen;
    if (r.len < 0 || r.bad) r.len = 0;
    const int64_t table = a.bt.width << a.c.page_shift;
    r.held = r.len < table ? r.len : (int)table;
    r.per = a.q_heads / a.c.heads;
    return r;
}

// The work of a call as one line of steps: sequence by sequence, in it unit by
// unit (a kv head's tile of rows, tiles of a head next to each other), in that
// the sequence's steps of positions (at least one, which writes rows that see
// nothing).  Workgroup w takes an equal stretch of the line, so lengths do not
// have to be equal, nor known to the host, for the CUs to be.  Cut: rows of a
// tile, threads of the workgroup that lays the line out.
template <int kTileRows, int kGroupThreads>
struct Cut {
    static constexpr int kRows = kTileRows, kThreads = kGroupThreads;
};
using SmallCut = Cut<16, kThreads>;
struct Line {
    int64_t total;   // steps of the call
    int64_t q, r;    // a workgroup's steps: q + 1 for the first r, else q
    int64_t before;  // steps before the found sequence
    int b;           // the found sequence (-1: none)
    Rows rw;         // its rows
    __device__ __forceinline__ int64_t first(int64_t w) const { return w * q + (w < r ? w : r); }
    // the workgroup that has step x
    __device__ __forceinline__ int64_t group_of(int64_t x) const
    {
        const int64_t big = r * (q + 1);
        return x < big ? udiv(x, q + 1) : r + udiv(x - big, q);
    }
};

__device__ __forceinline__ int steps_of(const AttnArgs& a, const Rows& rw)
{
    return rw.held > 0 ? ((rw.held - 1) >> a.step_shift) + 1 : 1;
}
template <class C>
__device__ __forceinline__ int64_t tiles_of(const Rows& rw)
{
    return (rw.rows() + C::kRows - 1) / C::kRows;
}
template <class C>
__device__ __forceinline__ int64_t line_steps(const AttnArgs& a, const Rows& rw)
{
    return tiles_of<C>(rw) * a.c.heads * steps_of(a, rw);
}

__device__ __forceinline__ int64_t lane64(int64_t v, int lane)
{
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(v >> 32), lane);
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Lays the line out and finds the sequence of workgroup w's first step (b < 0:
// it has none), or, given a sequence, the steps before it.  Every thread of
// the workgroup takes part.  Up to 64 sequences: a lane each, every wave for
// itself, one round of loads and no barrier (a launch's workgroups all start
// here, so nothing else hides it).  More: each thread adds up a run of
// sequences, and a scan over the workgroup joins the runs.
template <class C, bool kFind>
__device__ __forceinline__ Line lay_line_short(const AttnArgs& a, int64_t w, int b)
{
    Line ln;
    const int lane = threadIdx.x & (kWave - 1);
    const bool in = lane < a.bt.count;
    const Rows mine = rows_of(a, in ? lane : 0);
    const int64_t n = in ? line_steps<C>(a, mine) : 0;
    int64_t upto = n;
    for (int o = 1; o < a.bt.count; o <<= 1) {
        const int64_t t = __shfl_up(upto, o, kWave);
        if (lane >= o) upto += t;
    }
    ln.total = lane64(upto, (int)a.bt.count - 1);
    ln.q = udiv(ln.total, a.groups);
    ln.r = ln.total - ln.q * a.groups;
    if (kFind) {
        const int64_t x = ln.first(w);
        const uint64_t at = __ballot(x >= upto - n && x < upto);
        ln.b = at ? (int)__builtin_ctzll(at) : -1;
    } else {
        ln.b = b;
    }
    const int from = ln.b < 0 ? 0 : ln.b;
    ln.before = lane64(upto - n, from);
    ln.rw.first = __builtin_amdgcn_readlane(mine.first, from);
    ln.rw.nq = __builtin_amdgcn_readlane(mine.nq, from);
    ln.rw.len = __builtin_amdgcn_readlane(mine.len, from);
    ln.rw.held = __builtin_amdgcn_readlane(mine.held, from);
    ln.rw.bad = __builtin_amdgcn_readlane((int)mine.bad, from) != 0;
    ln.rw.per = mine.per;
    return ln;
}

template <class C, bool kFind>
__device__ __forceinline__ Line lay_line_long(const AttnArgs& a, int64_t w, int b)
{
    constexpr int kGroupWaves = C::kThreads / kWave;
    __shared__ int64_t wave_sum[kGroupWaves];
    __shared__ int64_t found[2];
    Line ln;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int64_t count = a.bt.count;
    const int64_t run = (count + C::kThreads - 1) / C::kThreads;
    const int64_t lo = run * tid < count ? run * tid : count;
    const int64_t hi = lo + run < count ? lo + run : count;
    int64_t mine = 0, to_b = 0;
    for (int64_t i = lo; i < hi; ++i) {
        if (!kFind && i == b) to_b = mine;
        mine += line_steps<C>(a, rows_of(a, i));
    }
    int64_t upto = mine;  // inclusive scan over the wave
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const int64_t t = __shfl_up(upto, o, kWave);
        if (lane >= o) upto += t;
    }
    if (lane == kWave - 1) wave_sum[wave] = upto;
    if (tid == 0) found[0] = -1;
    __syncthreads();
    int64_t base = 0;
    ln.total = 0;
#pragma unroll
    for (int i = 0; i < kGroupWaves; ++i) {
        if (i < wave) base += wave_sum[i];
        ln.total += wave_sum[i];
    }
    ln.q = udiv(ln.total, a.groups);
    ln.r = ln.total - ln.q * a.groups;
    int64_t before = base + upto - mine;
    if (kFind) {
        const int64_t x = ln.first(w);
        if (x >= before && x < before + mine) {
            for (int64_t i = lo; i < hi; ++i) {
                const int64_t n = line_steps<C>(a, rows_of(a, i));
                if (x < before + n) {
                    found[0] = i;
                    found[1] = before;
                    break;
                }
                before += n;
            }
        }
    } else if (b >= lo && b < hi) {
        found[0] = b;
        found[1] = before + to_b;
    }
    __syncthreads();
    ln.b = __builtin_amdgcn_readfirstlane((int)found[0]);
    ln.before = found[1];
    ln.rw = rows_of(a, ln.b < 0 ? 0 : ln.b);
    return ln;
}

template <class C, bool kFind>
__device__ __forceinline__ Line lay_line(const AttnArgs& a, int64_t w, int b)
{
    return a.bt.count <= kWave ? lay_line_short<C, kFind>(a, w, b) : lay_line_long<C, kFind>(a, w, b);
}

__device__ __forceinline__ int64_t uniform64(int64_t v)
{
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ uint32_t bf16x2(float a, float b)
{
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)a) |
           ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)b) << 16);
}

template <int kPieces>
__device__ __forceinline__ int swizzle(int row)
{
    return kPieces == 8 ? (row >> 1) & 7 : row & 15;
}
typedef float f32x16_t __attribute__((ext_vector_type(16)));


// every wave's LDS operations done, then the barrier (loads stay in flight)
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A piece by its LDS address.
typedef __attribute__((address_space(3))) const void lds_void;
__device__ __forceinline__ uint32_t lds_address(const uint4* p)
{
    return (uint32_t)(uintptr_t)(lds_void*)p;
}
__device__ __forceinline__ f16x8_t lds_piece(uint32_t address)
{
    return *(__attribute__((address_space(3))) const f16x8_t*)(uintptr_t)address;
}

// Joins the parts of a unit's rows: out = sum_s w_s o_s / sum_s w_s, w_s = l_s
// 2^(m_s - max m), s over the workgroups that share it.  Two forms:
// cache4_join_kernel, one workgroup per row (of a sequence's new tokens and a kv
// head's query heads), kv head and sequence, for few units of many parts; and
// cache4_join_edges_kernel, one per neighbouring pair of stretches, for so many
// units that each has only a part or two.
template <int D, class C>
__global__ __launch_bounds__(kThreads) void cache4_join_kernel(AttnArgs a)
{
    constexpr int kPer = D / 4;            // threads of a part: four dimensions each
    constexpr int kPar = kThreads / kPer;  // parts in flight
    __shared__ float2 ml_of[kPar];
    __shared__ __attribute__((aligned(16))) f32x4_t sums[kThreads];
    const int tid = threadIdx.x;
    const int b = blockIdx.z;
    const int kvh = blockIdx.y;
    const Line ln = lay_line<Cut<C::kRows, kThreads>, false>(a, 0, b);
    const Rows rw = ln.rw;
    if ((int64_t)blockIdx.x >= rw.rows()) return;
    const int steps = steps_of(a, rw);
    const int64_t tiles = tiles_of<C>(rw);
    const int d4 = tid % kPer;

    for (int64_t row = blockIdx.x; row < rw.rows(); row += gridDim.x) {
        const int r = (int)(row % C::kRows);
        const int64_t x = ln.before + (kvh * tiles + row / C::kRows) * steps;
        const int64_t g0 = ln.group_of(x), g1 = ln.group_of(x + steps - 1);
        if (g0 == g1) continue;  // written by the attention kernel
        const int64_t n = g1 - g0 + 1;
        // a workgroup whose stretch begins in the unit has it in its slot 0
        const auto slot_of = [&](int64_t s) { return ((g0 + s) * 2 + (s == 0 && ln.first(g0) != x)) * C::kRows + r; };
        // a thread's parts, all loads of eight in flight, against their own maximum
        float mx = -INFINITY, tot = 0.0f;
        f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
        for (int64_t s0 = tid / kPer; s0 < n; s0 += 8 * kPar) {
            float2 ml[8];
            f32x4_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t s = s0 + i * kPar < n ? s0 + i * kPar : s0;
                ml[i] = a.part_ml[slot_of(s)];
                v[i] = *reinterpret_cast<const f32x4_t*>(a.part + slot_of(s) * D + 4 * d4);
                if (s0 + i * kPar >= n) ml[i] = make_float2(-INFINITY, 0.0f);
            }
            float m8 = mx;
#pragma unroll
            for (int i = 0; i < 8; ++i) m8 = fmaxf(m8, ml[i].x);
            const float base = m8 == -INFINITY ? 0.0f : m8;
            const float old = tot * __builtin_amdgcn_exp2f(mx - base);
            tot = old;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // nothing seen: no weight (and a NaN sum keeps its)
                ml[i].y = ml[i].y == 0.0f ? 0.0f : ml[i].y * __builtin_amdgcn_exp2f(ml[i].x - base);
                tot += ml[i].y;
            }
            // a weighted mean all along: sums of weights * values could pass fp32
            const float inv = tot == 0.0f ? 0.0f : 1.0f / tot;
            acc *= old * inv;
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] = fmaf(ml[i].y * inv, v[i][e], acc[e]);
            mx = m8;
        }
        sums[tid] = acc;
        if (d4 == 0) ml_of[tid / kPer] = make_float2(mx, tot);
        __syncthreads();
        if (tid < kPer) {
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < kPar; ++i) top = fmaxf(top, ml_of[i].x);
            const float base = top == -INFINITY ? 0.0f : top;
            float w[kPar];
            tot = 0.0f;
#pragma unroll
            for (int i = 0; i < kPar; ++i) {
                w[i] = ml_of[i].y * __builtin_amdgcn_exp2f(ml_of[i].x - base);
                tot += w[i];
            }
            const float inv = tot == 0.0f ? 0.0f : 1.0f / tot;
            acc = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kPar; ++i) {
                const f32x4_t v = sums[i * kPer + tid];
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] = fmaf(v[e], w[i] * inv, acc[e]);
            }
            const int qi = (int)udiv(row, rw.per);
            const int head = kvh * rw.per + (int)(row - (int64_t)qi * rw.per);
            uint16_t* op = a.out + ((int64_t)(rw.first + qi) * a.q_heads + head) * D + 4 * d4;
            *reinterpret_cast<uint2*>(op) =
                make_uint2(bf16x2(acc[0], acc[1]), bf16x2(acc[2], acc[3]));
        }
        __syncthreads();
    }
}

template <int D, class C>
__global__ __launch_bounds__(kThreads) void cache4_join_edges_kernel(AttnArgs a)
{
    constexpr int N = D / 16;  // dimensions of a thread
    const int64_t w = (int64_t)blockIdx.x + 1;
    const Line ln = lay_line<Cut<C::kRows, kThreads>, true>(a, w, 0);
    if (ln.b < 0) return;
    const int64_t x = ln.first(w);
    const Rows rw = ln.rw;
    const int steps = steps_of(a, rw);
    const int64_t unit = udiv(x - ln.before, steps);
    const int64_t start = ln.before + unit * steps;
    // the unit's second stretch joins it
    if (x == start || x >= ln.total || ln.group_of(start) != w - 1) return;
    const int64_t n = ln.group_of(start + steps - 1) - w + 2;
    const int64_t tiles = tiles_of<C>(rw);
    const int kvh = (int)udiv(unit, tiles);
    const int r = (int)blockIdx.y * 16 + (threadIdx.x >> 4);  // of the tile
    const int64_t row = (unit - kvh * tiles) * C::kRows + r;
    if (row >= rw.rows()) return;
    const int d = (threadIdx.x & 15) * N;
    const auto slot_of = [&](int64_t s) {
        return ((w - 1 + s) * 2 + (s == 0 && ln.first(w - 1) != start)) * C::kRows + r;
    };
    float mx = -INFINITY;
    for (int64_t s = 0; s < n; ++s) mx = fmaxf(mx, a.part_ml[slot_of(s)].x);
    const float base = mx == -INFINITY ? 0.0f : mx;
    const auto weight = [&](int64_t s) {
        const float2 ml = a.part_ml[slot_of(s)];
        return ml.y == 0.0f ? 0.0f : ml.y * __builtin_amdgcn_exp2f(ml.x - base);
    };
    float tot = 0.0f;
    for (int64_t s = 0; s < n; ++s) tot += weight(s);
    const float inv = tot == 0.0f ? 0.0f : 1.0f / tot;
    float acc[N];
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.0f;
    for (int64_t s = 0; s < n; ++s) {
        const float ws = weight(s) * inv;  // (sums of weights * values could pass fp32)
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const f32x4_t v = *reinterpret_cast<const f32x4_t*>(a.part + slot_of(s) * D + d + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i + e] = fmaf(ws, v[e], acc[i + e]);
        }
    }
    const int qi = (int)udiv(row, rw.per);
    const int head = kvh * rw.per + (int)(row - (int64_t)qi * rw.per);
    uint16_t* op = a.out + ((int64_t)(rw.first + qi) * a.q_heads + head) * D + d;
#pragma unroll
    for (int i = 0; i < N; i += 4)
        *reinterpret_cast<uint2*>(op + i) = make_uint2(bf16x2(acc[i], acc[i + 1]), bf16x2(acc[i + 2], acc[i + 3]));
}

}  // namespace

}  // namespace dq

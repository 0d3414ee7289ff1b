// Filling and reading the paged 4-bit key/value cache (geometry: cache4.hpp).
// A head's vector is quantized as a row of the group-wise quantizer at b = 4
// ("量化" tutorial, aiknowledge.cn, exercise 1 of its exercises): per group of g
// dimensions s = fl32(max / 7) (1.0 replaces a zero max), q = clip(rint(fl32(
// v / s)), -8, 7), code u = q + 8; a group with a NaN or an infinity gets a NaN
// scale and q = 0.
//
// Both kernels are bound by memory and by the chain of loads that finds a token's
// place (its sequence, the sequence's length, the page).  A workgroup has one kv
// head of 2048 / D consecutive tokens (a page has their codes and scales next to
// each other, so each wave writes and reads whole lines); a thread has 8 dimensions
// of the key and of the value, D/8 neighbouring threads a vector, g/8 of them a
// group, whose maximum is a butterfly over those lanes.  6207 tokens of 8 heads of
// 128 in bf16, g = 64: append (25 MB in, 7 MB out) 14.1 us, 2.3 TB/s, read (the
// reverse) 10.0 us, 3.2 TB/s; 32 tokens 4.8 and 3.5 us.  (A workgroup per two tokens, all
// heads: 15.8 and 11.6 us, for a page's lines are then written two tokens at a
// time; 32 tokens 4.1 and 3.7.)  About half of the append's time is vector work.
// (The read of heads of 256 takes a code out of 64 bits.  A word picked by a lane's bit became
// an array in LDS, for whose address a kernel reads its dispatch packet, in host memory: 2 x 700 tokens
// appended and read 20.3 us, now 8.9.)
#include "cache4.hpp"
#include "common.hpp"
#include "launch_serving.hpp"
#include "quant_rule.hpp"

namespace dq {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kFillGroups = 1024;

// The place of token row t: -2 for one of no sequence, -1 for one that the cache
// does not hold.  All threads of the wave take part, kParts neighbours with the same
// t, the tokens of a wave being consecutive: with up to 64 sequences each lane looks
// at the start of one, so the search is one load (the 32 tokens of a decode step,
// searched by halving: 5.4 us instead of 4.8).
template <int kParts>
__device__ __forceinline__ int64_t find_slot(const Cache4& c, const Cache4Batch& bt, int64_t t, int64_t tokens,
                                             int64_t* position = nullptr)
{
    int64_t b = 0;
    if (bt.count <= kWave) {
        const int lane = threadIdx.x % kWave;
        const int32_t start = bt.starts[lane < bt.count ? lane : bt.count - 1];
        const int64_t t0 = t - lane / kParts;
#pragma unroll
        for (int i = 0; i < kWave / kParts; ++i) {
            const int before = __popcll(__ballot(lane < bt.count && start <= t0 + i));
            if (lane / kParts == i) b = before > 0 ? before - 1 : 0;
        }
    } else {
        b = cache4_sequence(bt, t);
    }
    int64_t first, n;
    cache4_rows(bt, b, tokens, first, n);
    if (t < first || t >= first + n) return -2;
    const int64_t pos = (int64_t)bt.lens[b] - n + (t - first);
    if (position) *position = pos;
    return cache4_slot(c, bt, b, pos);
}

// Where the parts of (page, head, token) begin: its code row, and the scale of its
// first group (the next group's is P floats on).
struct Place {
    int64_t row, scale;
};
template <int D>
__device__ __forceinline__ Place place_of(const Cache4& c, int64_t slot, int head, int group_shift)
{
    const int64_t block = (slot >> c.page_shift) * c.heads + head;
    const int64_t off = slot & ((1LL << c.page_shift) - 1);
    return {((block << c.page_shift) + off) * (D / 8),
            (((block * D) >> group_shift) << c.page_shift) + off};
}

// 8 elements as they lie in memory.
template <bool BF16>
struct Raw {
    uint4 d[BF16 ? 1 : 2];
    __device__ __forceinline__ void floats(float (&x)[8]) const
    {
        const uint32_t u[4] = {d[0].x, d[0].y, d[0].z, d[0].w};
        if constexpr (BF16) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[2 * e] = __uint_as_float(u[e] << 16);
                x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
            }
        } else {
            const uint32_t w[4] = {d[1].x, d[1].y, d[1].z, d[1].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = __uint_as_float(u[e]);
                x[4 + e] = __uint_as_float(w[e]);
            }
        }
    }
};
template <bool BF16>
__device__ __forceinline__ Raw<BF16> load8(const void* p, int64_t off)
{
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + off * (BF16 ? 2 : 4));
    Raw<BF16> r;
    r.d[0] = src[0];
    if constexpr (!BF16) r.d[1] = src[1];
    return r;
}

// The 8 codes of a thread (LSB first) and its group's scale.
__device__ __forceinline__ uint32_t quantize8(const float (&x)[8], int group_threads, float* scale)
{
    float q[8];
    uint32_t amax = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = max(amax, __float_as_uint(x[e]) & 0x7fffffffu);
    for (int o = group_threads >> 1; o > 0; o >>= 1)
        amax = max(amax, (uint32_t)__shfl_xor((int)amax, o, kWave));
    float s;
    bool zero = false;
    if (amax >= 0x7f800000u) {
        s = __uint_as_float(0x7fc00000u);
        zero = true;
    } else {
        const float a = __uint_as_float(amax);
        s = (a == 0.0f ? 1.0f : a) / 7.0f;
        if (a == 0.0f || s == 0.0f) {
            s = 1.0f / 7.0f;
            zero = true;
        }
    }
    *scale = s;
    clipped_quotients(x, s, __builtin_amdgcn_rcpf(s), quotient_margin(8.0f), 7.0f, q);
    // four codes at a time as the exact fp32 sum of 16^e (q + 8)
    float lo = 34952.0f, hi = 34952.0f;  // 0x8888
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        lo = fmaf(q[e], (float)(1 << (4 * e)), lo);
        hi = fmaf(q[4 + e], (float)(1 << (4 * e)), hi);
    }
    return zero ? 0x88888888u : (uint32_t)hi << 16 | (uint32_t)lo;
}
template <bool BF16>
__device__ __forceinline__ uint32_t quantize8(const Raw<BF16>& raw, int group_threads, float* scale)
{
    float x[8];
    raw.floats(x);
    return quantize8(x, group_threads, scale);
}

// The value codes of a thread (8 dimensions of a vector, LSB first) turned into
// the word that it stores, by way of LDS (mine: the vector's D/8 words).
template <int D>
__device__ __forceinline__ uint32_t turn_values(uint32_t wv, int part, uint32_t* mine)
{
    constexpr int kPer = D / 16;               // value codes of a c (cache4.hpp)
    constexpr int kRun = kPer < 8 ? kPer : 8;  // of them in a word
    // dimension 8 part + e is 16 j + c with j = part / 2, c = 8 (part & 1) + e, and
    // word w holds codes 8 w + n = c (D/16) + j: the words of one half of the c's lie
    // next to each other (a vector is within a wave, whose LDS accesses are in order)
    mine[(part & 1) * kPer + (part >> 1)] = wv;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int c0 = part * 8 / kPer;
    const uint4* from = reinterpret_cast<const uint4*>(mine + (c0 >> 3) * kPer + part * 8 % kPer);
    uint32_t x8[kRun];
#pragma unroll
    for (int e = 0; e < kRun; e += 4) {
        const uint4 d = from[e / 4];
        x8[e] = d.x, x8[e + 1] = d.y, x8[e + 2] = d.z, x8[e + 3] = d.w;
    }
    uint32_t w = 0;
#pragma unroll
    for (int n = 0; n < 8; ++n) w |= ((x8[n % kRun] >> (4 * ((c0 + n / kRun) & 7))) & 15u) << (4 * n);
    return w;
}

template <int D, bool BF16>
__global__ __launch_bounds__(kThreads) void cache4_append_kernel(
    Cache4 c, Cache4Batch bt, const void* __restrict__ k, const void* __restrict__ v,
    int64_t tokens, int64_t from_token, int64_t k_stride, int64_t v_stride)
{
    constexpr int kParts = D / 8;
    __shared__ __attribute__((aligned(16))) uint32_t turn[kThreads];
    const int64_t t = from_token + (int64_t)blockIdx.x * (kThreads / kParts) + threadIdx.x / kParts;
    const int part = threadIdx.x % kParts;
    const int head = blockIdx.y;
    const int64_t at = (int64_t)head * D + part * 8;
    const int64_t row = t < tokens ? t : tokens - 1;
    const Raw<BF16> rk = load8<BF16>(k, row * k_stride + at), rv = load8<BF16>(v, row * v_stride + at);
    const int64_t slot = find_slot<kParts>(c, bt, t, tokens);

    const int group_shift = 31 - __builtin_clz(c.group);
    const int group_threads = c.group >> 3;
    float sk, sv;
    const uint32_t wk = quantize8<BF16>(rk, group_threads, &sk);
    const uint32_t wv = quantize8<BF16>(rv, group_threads, &sv);

    const uint32_t w = turn_values<D>(wv, part, turn + (threadIdx.x - part));

    if (slot < 0) return;
    const Place p = place_of<D>(c, slot, head, group_shift);
    // (keys: dimensions 8 part .. = 32 i + 8 r are word r (D/32) + i)
    c.k_codes[p.row + (part & 3) * (D / 32) + (part >> 2)] = wk;
    c.v_codes[p.row + part] = w;
    if ((part & (group_threads - 1)) == 0) {
        const int64_t o = p.scale + ((int64_t)((part * 8) >> group_shift) << c.page_shift);
        c.k_scales[o] = sk;
        c.v_scales[o] = sv;
    }
}

// The same with the keys rotated (rope.hpp) on the way.  Angles, sines, cosines and
// products are fp64 and the rotated key is rounded once, to fp32: next to a border
// between codes fp32 angles would decide by their own error.
//
// A workgroup keeps the 1024 or fewer cosines and sines of its tokens in LDS (16 KB) and
// walks its heads with those of a thread's 8 dimensions in registers, so that they
// are worked out once for all heads; the next head's vectors are asked for a head ahead.  The
// partner of a dimension is in the same thread (interleaved) or comes from the thread dims / 16
// away, by a shuffle.  Bound by vector work (the fp64 rotation, the group rule) and memory together:
// 6207 tokens of 8 heads of 128 in bf16, g = 64 18.7 us (without rotation 14.1), 32 tokens 6.0.
template <int D, bool BF16>
__global__ __launch_bounds__(kThreads) void cache4_append_rope_kernel(
    Cache4 c, Cache4Batch bt, const void* __restrict__ k, const void* __restrict__ v,
    int64_t tokens, int64_t from_token, int64_t k_stride, int64_t v_stride, Rope rope,
    const int32_t* __restrict__ positions)
{
    constexpr int kParts = D / 8;
    constexpr int kTokens = kThreads / kParts;
    constexpr int kPairs = D / 2;
    __shared__ __attribute__((aligned(16))) uint32_t turn[kThreads];
    __shared__ __attribute__((aligned(16))) double2 turns[kTokens * kPairs];
    __shared__ int32_t at_position[kTokens];
    const int64_t t = from_token + (int64_t)blockIdx.x * kTokens + threadIdx.x / kParts;
    const int part = threadIdx.x % kParts;
    const int per = (c.heads + (int)gridDim.y - 1) / (int)gridDim.y;
    const int head0 = (int)blockIdx.y * per;
    const int head1 = head0 + per < c.heads ? head0 + per : c.heads;
    const int64_t row = t < tokens ? t : tokens - 1;
    const int d0 = part * 8;
    // (a head's vectors are asked for a head ahead)
    const auto load_k = [&](int head) { return load8<BF16>(k, row * k_stride + (int64_t)head * D + d0); };
    const auto load_v = [&](int head) { return load8<BF16>(v, row * v_stride + (int64_t)head * D + d0); };
    Raw<BF16> rk = load_k(head0 < head1 ? head0 : 0), rv = load_v(head0 < head1 ? head0 : 0);
    // (a thread works out one pair's angles, of every so many tokens)
    const int pairs = rope.dims / 2, pair = threadIdx.x % kPairs;
    const double pair_turn = rope.turns[pair < pairs ? pair : 0];
    int64_t pos = 0;
    const int64_t slot = find_slot<kParts>(c, bt, t, tokens, &pos);
    if (part == 0) at_position[threadIdx.x / kParts] = positions ? positions[row] : (int32_t)pos;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTokens * kPairs / kThreads; ++i) {
        const int at = i * kThreads + threadIdx.x;
        if (pair < pairs) {
            double s, co;
            sincos_turn(turn_fraction(at_position[at / kPairs], pair_turn), s, co);
            turns[at] = make_double2(co * rope.factor, s * rope.factor);
        }
    }
    __syncthreads();
    const bool inter = rope.interleaved;
    const bool turned = d0 < rope.dims;
    const bool upper = !inter && d0 >= pairs;   // the second of a pair
    const int shift = pairs / 8;                // threads to the partner
    const int partner = (int)(threadIdx.x & (kWave - 1)) + (turned && !inter ? (upper ? -shift : shift) : 0);
    double2 cs[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int pair = inter ? (d0 + e) / 2 : (upper ? d0 + e - pairs : d0 + e);
        cs[e] = turned ? turns[(threadIdx.x / kParts) * kPairs + pair] : make_double2(1.0, 0.0);
        if (!inter && !upper) cs[e].y = -cs[e].y;
    }

    const int group_shift = 31 - __builtin_clz(c.group);
    const int group_threads = c.group >> 3;
    for (int head = head0; head < head1; ++head) {
        const int ahead = head + 1 < head1 ? head + 1 : head;
        const Raw<BF16> next_k = load_k(ahead), next_v = load_v(ahead);
        Raw<BF16> other = rk;
        if (!inter) {
#pragma unroll
            for (int i = 0; i < (BF16 ? 1 : 2); ++i) {
                other.d[i].x = (uint32_t)__shfl((int)rk.d[i].x, partner, kWave);
                other.d[i].y = (uint32_t)__shfl((int)rk.d[i].y, partner, kWave);
                other.d[i].z = (uint32_t)__shfl((int)rk.d[i].z, partner, kWave);
                other.d[i].w = (uint32_t)__shfl((int)rk.d[i].w, partner, kWave);
            }
        }
        float x[8], y[8], z[8];
        rk.floats(x);
        other.floats(y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const double partner_of = inter ? (e & 1 ? (double)x[e ^ 1] : -(double)x[e ^ 1]) : (double)y[e];
            z[e] = turned ? (float)fma(partner_of, cs[e].y, (double)x[e] * cs[e].x) : x[e];
        }
        float sk, sv;
        const uint32_t wk = quantize8(z, group_threads, &sk);
        const uint32_t wv = quantize8<BF16>(rv, group_threads, &sv);
        const uint32_t w = turn_values<D>(wv, part, turn + (threadIdx.x - part));
        rk = next_k;
        rv = next_v;
        if (slot < 0) continue;
        const Place p = place_of<D>(c, slot, head, group_shift);
        c.k_codes[p.row + (part & 3) * (D / 32) + (part >> 2)] = wk;
        c.v_codes[p.row + part] = w;
        if ((part & (group_threads - 1)) == 0) {
            const int64_t o = p.scale + ((int64_t)((part * 8) >> group_shift) << c.page_shift);
            c.k_scales[o] = sk;
            c.v_scales[o] = sv;
        }
    }
}

// Moves the entries of accepted tokens to the front of a call's tokens: row path[j] of
// a sequence's new ones goes to row j.  A workgroup has one kv head of a sequence; a thread
// 16 bytes of the codes or a scale of one token, as many tokens side by side as fit.  All
// of them are read before any is written, and with path[j] >= j what is written is never a
// later one's source.  Bound by the chain of loads to a token's place and its data: 64 sequences of
// 64 tokens, 8 heads of 128 4.2 us, one of 16 3.7.  (One of 16 and its
// read: tokens one after another 9.4 us, side by side 6.9.)
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
constexpr int kKeepThreads = 512;
template <int D>
__global__ __launch_bounds__(kKeepThreads) void cache4_keep_kernel(Cache4 c, Cache4Batch bt,
                                                               const int32_t* __restrict__ path,
                                                               const int32_t* __restrict__ accepted,
                                                               int64_t tokens)
{
    constexpr int kPieces = D / 32;  // of a code row
    const int64_t b = blockIdx.y;
    const int head = blockIdx.x;
    const int groups = D / c.group;
    const int columns = 2 * kPieces + 2 * groups;
    const int side = kKeepThreads / columns;  // tokens side by side
    const int mine = (int)threadIdx.x / columns, column = (int)threadIdx.x - mine * columns;
    int64_t first, n;
    cache4_rows(bt, b, tokens, first, n);
    const int64_t base = (int64_t)bt.lens[b] - n;
    int64_t count = accepted[b];
    count = count < n ? count : n;
    const int group_shift = 31 - __builtin_clz(c.group);
    const bool code = column < 2 * kPieces;
    const bool key = code ? column < kPieces : column < 2 * kPieces + groups;
    const int at = code ? (key ? column : column - kPieces) : column - 2 * kPieces - (key ? 0 : groups);
    uint32_t* const codes = key ? c.k_codes : c.v_codes;
    float* const scales = key ? c.k_scales : c.v_scales;
    const auto place = [&](int64_t slot) {
        const Place p = place_of<D>(c, slot, head, group_shift);
        return code ? p.row + 4 * at : p.scale + ((int64_t)at << c.page_shift);
    };
    for (int64_t j0 = 0; j0 < count; j0 += side) {
        const int64_t j = j0 + mine;
        const int64_t r = mine < side && j < count ? path[first + j] : -1;
        const bool moves = r > j && r < n;
        const int64_t from = moves ? cache4_slot(c, bt, b, base + r) : -1;
        const int64_t to = moves ? cache4_slot(c, bt, b, base + j) : -1;
        // (a vector type: the compiler would keep a struct that is set in two ways in LDS)
        u32x4_t v = {0, 0, 0, 0};
        if (from >= 0 && to >= 0)
            v = code ? *reinterpret_cast<const u32x4_t*>(codes + place(from))
                     : (u32x4_t){__float_as_uint(scales[place(from)]), 0, 0, 0};
        __syncthreads();
        if (from >= 0 && to >= 0) {
            if (code)
                *reinterpret_cast<u32x4_t*>(codes + place(to)) = v;
            else
                scales[place(to)] = __uint_as_float(v.x);
        }
        __syncthreads();
    }
}

// Elements of an output vector.
template <bool BF16>
__device__ __forceinline__ void store8(void* dst, int64_t o, const float (&x)[8])
{
    if constexpr (BF16) {
        uint32_t p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            p[e] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * e]) |
                   ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * e + 1]) << 16);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + o) = make_uint4(p[0], p[1], p[2], p[3]);
    } else {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(dst) + o);
        p[0] = make_float4(x[0], x[1], x[2], x[3]);
        p[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

template <int D, bool BF16>
__global__ __launch_bounds__(kThreads) void cache4_read_kernel(Cache4 c, Cache4Batch bt,
                                                               void* __restrict__ k,
                                                               void* __restrict__ v, int64_t tokens,
                                                               int64_t from_token)
{
    constexpr int kParts = D / 8;
    constexpr int kWords = D / 64 * 4;  // of the 8 c's of a thread's value dimensions
    const int64_t t = from_token + (int64_t)blockIdx.x * (kThreads / kParts) + threadIdx.x / kParts;
    const int part = threadIdx.x % kParts;
    const int head = blockIdx.y;
    const int64_t slot = find_slot<kParts>(c, bt, t, tokens);
    if (slot == -2) return;
    const int64_t o = (t * c.heads + head) * D + part * 8;
    float x[8], y[8];
    if (slot < 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = y[e] = __uint_as_float(0x7fc00000u);
    } else {
        const int group_shift = 31 - __builtin_clz(c.group);
        const Place p = place_of<D>(c, slot, head, group_shift);
        const uint32_t wk = c.k_codes[p.row + (part & 3) * (D / 32) + (part >> 2)];
        const uint4* src = reinterpret_cast<const uint4*>(c.v_codes + p.row + (part & 1) * kWords);
        uint32_t w[kWords];
#pragma unroll
        for (int e = 0; e < kWords; e += 4) {
            const uint4 d = src[e / 4];
            w[e] = d.x, w[e + 1] = d.y, w[e + 2] = d.z, w[e + 3] = d.w;
        }
        const int64_t so = p.scale + ((int64_t)((part * 8) >> group_shift) << c.page_shift);
        const float sk = c.k_scales[so], sv = c.v_scales[so];
        const int j = part >> 1;  // the code of each c
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint32_t u;
            if constexpr (D == 64)
                u = w[e / 2] >> (16 * (e & 1) + 4 * j);
            else if constexpr (D == 128)
                u = w[e] >> (4 * j);
            else
                u = (uint32_t)(((uint64_t)w[2 * e + 1] << 32 | w[2 * e]) >> (4 * j));
            x[e] = (float)((int32_t)((wk >> (4 * e)) & 15u) - 8) * sk;
            y[e] = (float)((int32_t)(u & 15u) - 8) * sv;
        }
    }
    store8<BF16>(k, o, x);
    store8<BF16>(v, o, y);
}

// Launches for the tokens from, from + kLaunchTokens, ... (a launch has at most
// 2^32 - 1 threads a dimension).
constexpr int64_t kLaunchTokens = 1LL << 26;
template <class F>
hipError_t by_tokens(const Cache4& c, int64_t tokens, F launch)
{
    for (int64_t from = 0; from < tokens; from += kLaunchTokens) {
        const int64_t n = tokens - from < kLaunchTokens ? tokens - from : kLaunchTokens;
        launch(dim3((unsigned)ceil_div(n, kThreads / (c.dim / 8)), (unsigned)c.heads), from);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_cache4_append(const Cache4& c, const Cache4Batch& bt, const void* k,
                                const void* v, bool bf16, int64_t tokens, int64_t k_stride,
                                int64_t v_stride, hipStream_t stream)
{
#define CALL(D) \
    (bf16 ? cache4_append_kernel<D, true> : cache4_append_kernel<D, false>)
    const auto kernel = c.dim == 64 ? CALL(64) : (c.dim == 128 ? CALL(128) : CALL(256));
    return by_tokens(c, tokens, [&](dim3 grid, int64_t from) {
        kernel<<<grid, kThreads, 0, stream>>>(c, bt, k, v, tokens, from, k_stride, v_stride);
    });
#undef CALL
}

hipError_t launch_cache4_append_rope(const Cache4& c, const Cache4Batch& bt, const void* k, const void* v,
                                     bool bf16, int64_t tokens, int64_t k_stride, int64_t v_stride,
                                     const Rope& rope, const int32_t* positions, hipStream_t stream)
{
#define CALL(D) \
    (bf16 ? cache4_append_rope_kernel<D, true> : cache4_append_rope_kernel<D, false>)
    const auto kernel = c.dim == 64 ? CALL(64) : (c.dim == 128 ? CALL(128) : CALL(256));
    return by_tokens(c, tokens, [&](dim3 grid, int64_t from) {
        // Heads of a workgroup: all, unless that leaves fewer than kFillGroups workgroups (7500 tokens, append
        // and read 34.0 us; up to 256 workgroups 36.8, one head each 38.7).
        const int64_t split = kFillGroups / grid.x;
        grid.y = (unsigned)(split < 1 ? 1 : (split > c.heads ? c.heads : split));
        kernel<<<grid, kThreads, 0, stream>>>(c, bt, k, v, tokens, from, k_stride, v_stride, rope, positions);
    });
#undef CALL
}

hipError_t launch_cache4_keep(const Cache4& c, const Cache4Batch& bt, const int32_t* path,
                              const int32_t* accepted, int64_t tokens, hipStream_t stream)
{
    const auto kernel = c.dim == 64 ? cache4_keep_kernel<64>
                                    : (c.dim == 128 ? cache4_keep_kernel<128> : cache4_keep_kernel<256>);
    kernel<<<dim3((unsigned)c.heads, (unsigned)bt.count), kKeepThreads, 0, stream>>>(c, bt, path, accepted, tokens);
    return hipGetLastError();
}

hipError_t launch_cache4_read(const Cache4& c, const Cache4Batch& bt, void* k, void* v, bool bf16,
                              int64_t tokens, hipStream_t stream)
{
#define CALL(D) \
    (bf16 ? cache4_read_kernel<D, true> : cache4_read_kernel<D, false>)
    const auto kernel = c.dim == 64 ? CALL(64) : (c.dim == 128 ? CALL(128) : CALL(256));
    return by_tokens(c, tokens, [&](dim3 grid, int64_t from) {
        kernel<<<grid, kThreads, 0, stream>>>(c, bt, k, v, tokens, from);
    });
#undef CALL
}

}  // namespace dq

// Causal attention of new queries over the paged 4-bit cache (cache4.hpp):
//   o[i,h] = sum_t p_t vhat[t] / sum_t p_t,  p_t = exp(scale q[i,h] . khat[t] - max),
// over the cached positions t up to query i's own, khat / vhat = q4 * group scale.
//
// One wave takes 16 rows (query, head of one kv head's group) and walks the
// positions 32 at a time with the running maximum and sum of a softmax.  Both
// products run on v_mfma_f32_16x16x32_f16 in transposed form, S^T = K Q^T and
// O^T = V^T P^T, so that a lane holds one row (lane & 15) throughout: the
// softmax is in-lane but for two steps across the four lanes of a row, and S^T
// comes out in the lane and order in which P^T goes in.
//   * The codes are exact in fp16 (u | 0x6400 is 1024 + u; the offset comes off
//     exactly).  Each row of q is multiplied by a power of two that puts its
//     largest element in [2^14, 2^15): exact for every element above 2^-28 of
//     it.  A group's partial dot products are scaled in fp32.
//   * p * (value scale) is rounded once, to fp16, after multiplication by a
//     power of two that puts the largest scale of the group seen so far in [2^14,
//     2^15): relative error 2^-11 down to 2^-29 of the largest.  Groups whose codes
//     are all 0 (their stored scale says nothing) do not count for that, nor do
//     positions that a row does not see: where the causal mask crosses a step with
//     larger scales, every row takes a power of two of its own (finish_step).
// This form (cache4_attention_kernel) is for few new tokens: bound by the cache's
// bytes, and below them by the vector work of expanding the codes.  One token over
// 65000 (8 kv heads of 128, 32 query heads, g = 32; 83 MB of cache) 29 us, of which
// 15 are launch, first bytes and the join; 40 sequences of 3250 to 6000 (8 kv, 40
// query heads; 240 MB) 60 us, 4.0 TB/s; 8 x 5 tokens over up to 1100 13 us.  Waves
// of one workgroup take neighbouring steps and join through LDS; workgroups take
// equal stretches of all sequences' steps (below) and join through the workspace: one
// workgroup per sequence, head and 16 rows left the first case's long axis to 8 of
// them, 4.7 ms.  For many new tokens see cache4_prompt_kernel.
#include "cache4.hpp"
#include "cache4_line.hpp"
#include "common.hpp"
#include "gemm_tiles.hpp"
#include "launch_serving.hpp"

namespace dq {

namespace {

// (v & mask) | bits in one instruction: one constant in a scalar register, the
// other in a vector register (the compiler's own choice is two instructions
// with a literal each).
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits)
{
    uint32_t r;
    asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(r) : "v"(v), "s"(mask), "v"(bits));
    return r;
}

// The codes in bits 0..3 and 16..19 of v as fp16 (u - 8), exact.
__device__ __forceinline__ uint32_t low_codes(uint32_t v)
{
    const f16x2_t h = f16x2_of(and_or(v, 0x000f000fu, 0x64006400u));  // 1024 + u
    return u32_of(h - (f16x2_t){(_Float16)1032.0f, (_Float16)1032.0f});
}
// The codes in bits 4..7 and 20..23.
__device__ __forceinline__ uint32_t high_codes(uint32_t v)
{
    const f16x2_t h = f16x2_of(and_or(v, 0x00f000f0u, 0x64006400u));  // 1024 + 16 u
    const _Float16 s = (_Float16)0.0625f, o = (_Float16)-72.0f;
    return u32_of(__builtin_elementwise_fma(h, (f16x2_t){s, s}, (f16x2_t){o, o}));
}

// The 8 codes of a word as an fp16 operand, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ f16x8_t word_codes(uint32_t w)
{
    const uint32_t x = w >> 8;
    return __builtin_bit_cast(f16x8_t, (u32x4_t){low_codes(w), high_codes(w), low_codes(x), high_codes(x)});
}

__device__ __forceinline__ float wave_max_abs(float v)
{
    uint32_t u = row16_max(v >= 0.0f ? __float_as_uint(v) : 0u);
    float x, y;
    row_pair(__uint_as_float(u), true, x, y);
    u = max(__float_as_uint(x), __float_as_uint(y));
    row_pair(__uint_as_float(u), false, x, y);
    return __uint_as_float(max(__float_as_uint(x), __float_as_uint(y)));
}

// n consecutive words at byte offset off of a buffer.
template <int N>
__device__ __forceinline__ void load_n(__amdgpu_buffer_rsrc_t rs, uint32_t off, uint32_t (&w)[N])
{
    if constexpr (N == 2) {
        const u32x2v_t v = __builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, 0);
        w[0] = v.x;
        w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const u32x4v_t v = __builtin_amdgcn_raw_buffer_load_b128(rs, off + 4 * i, 0, 0);
            w[i] = v.x;
            w[i + 1] = v.y;
            w[i + 2] = v.z;
            w[i + 3] = v.w;
        }
    }
}

// A workgroup of four waves walks its stretch of the line: in each unit wave w
// takes 32 of a step's 128 positions, and the four partial results are
// joined through LDS in a fixed order.  A unit that the workgroup has whole is
// written out here; the (at most two) that it shares with its neighbours go to
// the workspace and are joined by cache4_join_kernel, in order.
//
// A step's loads are issued a step ahead, as soon as the registers that they
// fill are free, its page numbers two steps ahead (scalar loads).  Codes come
// straight into the registers that expand them; a step's scales come one float
// per lane and are handed round through wave-private LDS (each lane needs the
// scales of 8 positions and every group).  A tile of 16 positions lies in one
// page, so its four arrays are buffers with scalar bases, and a lane's place
// in them is the same in every step.
template <int D, int G>
__global__ __launch_bounds__(kThreads, D == 64 ? 4 : (D == 128 ? 3 : 2)) void cache4_attention_kernel(AttnArgs a)
{
    constexpr int NC = D / 32;  // 32-dimension steps of a dot product
    constexpr int NG = D / G;   // groups of a head
    constexpr int GC = G / 32;  // steps of a group
    constexpr int NT = D / 16;  // 16-dimension tiles of the output
    constexpr int VW = D / 128 > 0 ? D / 128 : 1;  // value words a lane reads of a token
    constexpr int NL = (NG + 3) / 4;               // scale loads per 16 positions
    constexpr int SC = 4 * NL * 16;                // floats of 16 positions' scales in LDS
    __shared__ __attribute__((aligned(16))) float scales[kWaves][2][2 * SC];  // keys, values
    __shared__ __attribute__((aligned(16))) float join[kWaves / 2][(NT * 4 + 2) * kWave];

    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r16 = lane & 15;
    const int kg = lane >> 4;
    const int shift = a.c.page_shift;

    // byte offsets of this lane's data in 16 positions of one head
    const uint32_t k_lane = r16 * (D / 2) + kg * NC * 4;
    const uint32_t v_lane = 4 * kg * (D / 2) + r16 * (D / 32);
    uint32_t s_lane[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int g = 4 * i + kg < NG ? 4 * i + kg : NG - 1;
        s_lane[i] = (((uint32_t)g << shift) + r16) * 4;
    }

    // consecutive stretches (which may read the same keys) on one XCD
    const int group = (a.groups & 7) == 0 ? (int)(blockIdx.x & 7) * (a.groups >> 3) + (int)(blockIdx.x >> 3)
                                          : (int)blockIdx.x;
    const Line ln = lay_line<SmallCut, true>(a, group, 0);
    const int64_t x0 = uniform64(ln.first(group)), x1 = uniform64(ln.first(group + 1));
    int b = ln.b;
    int64_t before = uniform64(ln.before);
    if (b < 0) return;

    Rows rw = ln.rw;
    for (int64_t x = x0; x < x1;) {
        const int steps = steps_of(a, rw);
        const int64_t tiles = tiles_of<SmallCut>(rw);
        if (x >= before + tiles * a.c.heads * steps) {
            before += tiles * a.c.heads * steps;
            ++b;
            rw = rows_of(a, b);
            continue;
        }
        const int64_t unit = udiv(x - before, steps);
        const int step0 = (int)(x - before - unit * steps);
        const int take = (int)(x1 - x < steps - step0 ? x1 - x : steps - step0);
        const bool whole = take == steps;
        const int slot = x == x0 ? 0 : 1;
        // (readfirstlane: known to be the same in all lanes, so that page numbers and
        // buffer bases stay in scalar registers)
        const int kvh = __builtin_amdgcn_readfirstlane((int)udiv(unit, tiles));
        const int64_t tile = unit - kvh * tiles;
        const int64_t r0 = tile * 16;
        const int64_t rows = rw.rows();
        const bool live = r0 + r16 < rows;
        const int64_t row = live ? r0 + r16 : 0;
        const int qi = (int)udiv(row, rw.per);
        const int head = kvh * rw.per + (int)(row - (int64_t)qi * rw.per);
        const int seen = live ? rw.len - rw.nq + qi + 1 : 0;  // positions that the row sees
        // positions that every live row of the tile sees, and the last one (in the table)
        const int all_see = __builtin_amdgcn_readfirstlane(seen);
        const int end = min(__builtin_amdgcn_readlane(seen, rows - r0 < 16 ? (int)(rows - r0) - 1 : 15),
                            __builtin_amdgcn_readfirstlane(rw.held));
        const int begin = __builtin_amdgcn_readfirstlane(step0) * kStride;
        int stop = end;  // (a unit that is one step may have any length)
        if (take < steps - step0 && begin + take * kStride < end)
            stop = begin + __builtin_amdgcn_readfirstlane(take) * kStride;
        stop = __builtin_amdgcn_readfirstlane(stop);
        x += take;
        // constant address space: scalar loads, which leave the count of vector
        // loads in flight alone
        const __attribute__((address_space(4))) int32_t* table =
            (const __attribute__((address_space(4))) int32_t*)(
                a.bt.table + __builtin_amdgcn_readfirstlane(b) * a.bt.width);

        f16x8_t qf[NC];
        float logit = 1.0f;
        float m = -INFINITY, l = 0.0f;
        // The scales of a group are measured in units of 2^(ve - 14), and so is o; lane
        // (r16, kg) has ve for the groups 4 i + kg, as vtop = 65504 2^(ve - 14), what fp16
        // holds of them.  It is raised to the exponent of a scale that passes vtop, so
        // scales that grow by less than two or four times leave it (and o) as it is.
        constexpr uint32_t kTopBits = 0x7fe000u;  // mantissa of 65504
        uint32_t vtop[NL];
#pragma unroll
        for (int i = 0; i < NL; ++i) vtop[i] = (16u << 23) + kTopBits;  // ve = -112
        bool finished = false;  // o and l are what the wave hands on (finish_step)
        f32x4_t o[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) o[j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};

        // A step's two tiles of 16 positions (the last ones again past the
        // end): page, then (page, head) block and offset in it
        uint32_t kw[2][NC], vw[8][VW];
        float ksl[2][NL], vsl[2][NL];
        uint32_t bad[2];  // a NaN's bits where the page is outside the cache
        int pg[2];
        int64_t block[2];
        auto tile_at = [&](int tt) { return tt < stop ? tt : (stop - 1) & ~15; };
        auto load_pages = [&](int t0) __attribute__((always_inline)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) pg[h] = table[tile_at(t0 + 16 * h) >> shift];
        };
        auto load_k = [&](int t0) __attribute__((always_inline)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int off = tile_at(t0 + 16 * h) & ((1 << shift) - 1);
                const bool ok = (unsigned)pg[h] < (unsigned)a.c.pages;
                bad[h] = ok ? 0u : 0x7fc00000u;
                block[h] = (int64_t)(ok ? pg[h] : 0) * a.c.heads + kvh;
                const uint32_t* kc = a.c.k_codes + ((block[h] << shift) + off) * (D / 8);
                load_n<NC>(make_rsrc(kc, 16 * (D / 2)), k_lane, kw[h]);
                const int64_t sb = ((block[h] * NG) << shift) + off;
                const uint32_t bytes = (((NG - 1) << shift) + 16) * 4;
                const __amdgpu_buffer_rsrc_t ks = make_rsrc(a.c.k_scales + sb, bytes);
                const __amdgpu_buffer_rsrc_t vs = make_rsrc(a.c.v_scales + sb, bytes);
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    ksl[h][i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(ks, s_lane[i], 0, 0));
                    vsl[h][i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(vs, s_lane[i], 0, 0));
                }
            }
        };
        auto load_v = [&](int t0) __attribute__((always_inline)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int off = tile_at(t0 + 16 * h) & ((1 << shift) - 1);
                const uint32_t* vc = a.c.v_codes + ((block[h] << shift) + off) * (D / 8);
                const __amdgpu_buffer_rsrc_t rs = make_rsrc(vc, 16 * (D / 2));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (D == 64)
                        vw[4 * h + e][0] = __builtin_amdgcn_raw_buffer_load_b16(rs, v_lane + e * (D / 2), 0, 0);
                    else if constexpr (D == 128)
                        vw[4 * h + e][0] = __builtin_amdgcn_raw_buffer_load_b32(rs, v_lane + e * (D / 2), 0, 0);
                    else
                        load_n<VW>(rs, v_lane + e * (D / 2), vw[4 * h + e]);
                }
            }
        };
        float* const lk = &scales[wave][0][0];
        float* const lv = &scales[wave][1][0];
        // 2^(ve - 14) of group g
        const auto group_unit = [&](int g) {
            return pow2((int)(__builtin_amdgcn_readlane(vtop[g / 4], 16 * (g % 4)) >> 23) - 142);
        };
        // Scales of groups whose codes are all 0 become 0.  Lanes (c, kg) hold the codes of
        // the tokens 4 kg + e of both tiles, a group's in some of their bits.
        auto drop_zero_groups = [&]() __attribute__((always_inline)) {
            uint32_t zero[NG == 8 ? 2 : 1] = {};  // bit e * NG + g (of the 8 tokens, two words where NG is 8)
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    constexpr int n = G / 16;  // codes of the group in a lane
                    const uint32_t mask = (n == 8 ? ~0u : (1u << (4 * (n & 7))) - 1u) << (4 * (g * n % 8));
                    const uint64_t lanes = __ballot(((vw[e][g * n / 8] ^ 0x88888888u) & mask) == 0);
                    if (((lanes >> (16 * kg)) & 0xffffu) == 0xffffu)
                        zero[NG == 8 ? e / 4 : 0] |= 1u << ((e * NG + g) & 31);
                }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t z = (uint32_t)__shfl((int)zero[NG == 8 ? h : 0], (r16 & 12) << 2, kWave);
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    const int g = 4 * i + kg < NG ? 4 * i + kg : NG - 1;
                    const bool none = (z >> (((4 * h + (r16 & 3)) * NG + g) & 31)) & 1;
                    if (none) vsl[h][i] = 0.0f;
                }
            }
        };
        // A value scale that is not finite: NaN in its dimensions, in the rows that see it
        // (whatever their weight), and 0 from here on.
        auto mark_nan = [&](int t0) __attribute__((always_inline)) {
            uint64_t lanes[2][NL];  // of a tile: bits 16 n + position, n + 4 i the group
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    const bool nan = !(fabsf(vsl[h][i]) < INFINITY);
                    lanes[h][i] = __ballot(nan);
                    if (nan) vsl[h][i] = 0.0f;
                }
            const int see = seen - t0;
            const uint32_t mine = see >= 32 ? ~0u : (see <= 0 ? 0u : (1u << see) - 1u);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const uint32_t at = (uint32_t)(lanes[0][g / 4] >> (16 * (g % 4)) & 0xffffu) |
                                    (uint32_t)(lanes[1][g / 4] >> (16 * (g % 4)) & 0xffffu) << 16;
                if ((at & mine) != 0) {
#pragma unroll
                    for (int j = g * G / 16; j < (g + 1) * G / 16; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[j][e] = __uint_as_float(0x7fc00000u);
                }
            }
        };
        // The reference of each group follows the step's largest scales.
        auto raise = [&](bool first) __attribute__((always_inline)) {
            int down[NL];
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                uint32_t top = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h) top = max(top, __float_as_uint(vsl[h][i]) & 0x7fffffffu);
                const uint32_t was = vtop[i] >> 23;
                top = row16_max(top);
                const uint32_t now = top >= vtop[i] ? (top >> 23) + 1 : was;
                vtop[i] = (now << 23) + kTopBits;
                down[i] = (int)was - (int)now;
            }
            if (first) return;  // o is 0 (or NaN)
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const float f = pow2(__builtin_amdgcn_readlane(down[g / 4], 16 * (g % 4)));
#pragma unroll
                for (int j = g * G / 16; j < (g + 1) * G / 16; ++j) o[j] *= f;
            }
        };
        // The products of a step that the causal mask crosses (the wave's last of the unit,
        // for the rows of a tile are at most 15 positions apart), with a power of two per row
        // and group that puts the row's own largest weight * scale in [2^14, 2^15): p the
        // weights (0 where hidden), the scales in LDS as they are.  Leaves o and l as the
        // wave hands them on.
        auto finish_step = [&](const float (&p)[8]) __attribute__((always_inline)) {
            l = row_sum(l);
            const float inv = l > 0.0f ? 1.0f / l : l;  // (0 and NaN stay)
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                __builtin_amdgcn_sched_barrier(0);  // a group at a time
                float t[8];
                float top = 0.0f;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const f32x4_t vs = *reinterpret_cast<const f32x4_t*>(lv + h * SC + g * 16 + 4 * kg);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        t[4 * h + e] = p[4 * h + e] * vs[e];
                        top = fmaxf(top, fabsf(t[4 * h + e]));
                    }
                }
                const int up = 14 - max(exponent(row_max(top)), -112);
                const float f = pow2(up), unit = group_unit(g), back = pow2(-up) * inv;
                f16x8_t pf;
#pragma unroll
                for (int e = 0; e < 8; ++e) pf[e] = (_Float16)(t[e] * f);
#pragma unroll
                for (int w = g * G / 32; w < (g + 1) * G / 32; ++w) {
                    __builtin_amdgcn_sched_barrier(0);
                    const uint32_t sel = 0x0c000c00u | ((uint32_t)(4 + w % 4) << 16) | (uint32_t)(w % 4);
                    uint32_t lo[4], hi[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t v = __builtin_amdgcn_perm(vw[2 * e + 1][w / 4], vw[2 * e][w / 4], sel);
                        lo[e] = low_codes(v);
                        hi[e] = high_codes(v);
                    }
                    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
                    const f32x4_t x = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                        __builtin_bit_cast(f16x8_t, (u32x4_t){lo[0], lo[1], lo[2], lo[3]}), pf, zero, 0, 0, 0);
                    const f32x4_t y = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                        __builtin_bit_cast(f16x8_t, (u32x4_t){hi[0], hi[1], hi[2], hi[3]}), pf, zero, 0, 0, 0);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        o[2 * w][e] = fmaf(x[e], back, o[2 * w][e] * inv * unit);
                        o[2 * w + 1][e] = fmaf(y[e], back, o[2 * w + 1][e] * inv * unit);
                    }
                }
            }
        };
        auto step = [&](auto Finish, int t0) __attribute__((always_inline)) {
            constexpr bool kFinish = decltype(Finish)::value;
            // value scales: none past the end, those of a group measured by a common power of two
            bool larger = false;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    if (t0 + 16 * h + r16 >= end) vsl[h][i] = 0.0f;
                    larger |= !(fabsf(vsl[h][i]) < __uint_as_float(vtop[i]));
                }
            if (kFinish || __builtin_expect(__any(larger), 0)) {
                bool unsure = false, nan = false;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < NL; ++i) {
                        unsure |= __float_as_uint(vsl[h][i]) == kZeroScale;
                        nan |= !(fabsf(vsl[h][i]) < INFINITY);
                    }
                if (__builtin_expect(__any(nan), 0)) mark_nan(t0);
                if (__builtin_expect(__any(unsure), 0)) drop_zero_groups();
                if (!kFinish) raise(t0 == begin + wave * kStep);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    // times 2^(14 - ve), or as they are
                    const float f = kFinish ? 1.0f : __uint_as_float((269u << 23) + kTopBits - vtop[i]);
                    lk[h * SC + i * 64 + lane] = __uint_as_float(__float_as_uint(ksl[h][i]) | bad[h]);
                    lv[h * SC + i * 64 + lane] = vsl[h][i] * f;
                }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");  // other lanes read them
            __builtin_amdgcn_wave_barrier();
            // S^T = K Q^T, a group at a time; positions past the row's own at -inf
            const int left = seen - t0 - 4 * kg;
            f32x4_t ks[2][NG];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    ks[h][g] = *reinterpret_cast<const f32x4_t*>(lk + h * SC + g * 16 + 4 * kg);
            __builtin_amdgcn_sched_barrier(0);  // all LDS reads in flight behind the expansion
            float s[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    f32x4_t part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < GC; ++i)
                        part = __builtin_amdgcn_mfma_f32_16x16x32_f16(word_codes(kw[h][g * GC + i]),
                                                                      qf[g * GC + i], part, 0, 0, 0);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[e] = fmaf(ks[h][g][e], part[e], acc[e]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[4 * h + e] = 16 * h + e < left ? acc[e] : -INFINITY;
                }
            }
            __builtin_amdgcn_sched_barrier(0);  // the loads here, not where registers would be free
            f32x4_t vs[2][NG];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    vs[h][g] = *reinterpret_cast<const f32x4_t*>(lv + h * SC + g * 16 + 4 * kg);
            if (!kFinish) load_k(t0 + kStride);
            __builtin_amdgcn_sched_barrier(0);
            // running maximum (of logits) and sum
            float mx = s[0];
#pragma unroll
            for (int e = 1; e < 8; ++e) mx = fmaxf(mx, s[e]);
            mx = row_max(mx);
            const float mn = fmaxf(m, mx * logit);
            const float base = mn == -INFINITY ? 0.0f : mn;
            const float alpha = __builtin_amdgcn_exp2f(m - base);
            m = mn;
            float p[8];
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                p[e] = __builtin_amdgcn_exp2f(fmaf(s[e], logit, -base));
                sum += p[e];
            }
            l = fmaf(l, alpha, sum);
#pragma unroll
            for (int e = 0; e < 8; ++e) pin(p[e]);
            if (__any(alpha != 1.0f)) {
#pragma unroll
                for (int j = 0; j < NT; ++j) o[j] *= alpha;
            }
            if constexpr (kFinish) {
                finish_step(p);
                return;
            }
            f16x8_t pf[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) pf[g][4 * h + e] = (_Float16)(p[4 * h + e] * vs[h][g][e]);
                }
            }
            // page numbers after the step's last LDS read: a wait for one waits for both
            load_pages(t0 + 2 * kStride);
            __builtin_amdgcn_sched_barrier(0);  // else the expansions of all tiles are hoisted and spill
            // O^T = V^T P^T; tile j: nibble j of the lane's codes of 8 positions, in pairs
#pragma unroll
            for (int i = 0; i < VW; ++i) {
#pragma unroll
                for (int n = 0; n < (D == 64 ? 2 : 4); ++n) {
                    const uint32_t sel = 0x0c000c00u | ((uint32_t)(4 + n) << 16) | (uint32_t)n;
                    uint32_t lo[4], hi[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t v = __builtin_amdgcn_perm(vw[2 * e + 1][i], vw[2 * e][i], sel);
                        lo[e] = low_codes(v);
                        hi[e] = high_codes(v);
                    }
                    const int j = 8 * i + 2 * n;
                    const f16x8_t vl = __builtin_bit_cast(f16x8_t, (u32x4_t){lo[0], lo[1], lo[2], lo[3]});
                    const f16x8_t vh = __builtin_bit_cast(f16x8_t, (u32x4_t){hi[0], hi[1], hi[2], hi[3]});
                    o[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vl, pf[16 * j / G], o[j], 0, 0, 0);
                    o[j + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vh, pf[16 * (j + 1) / G], o[j + 1], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            load_v(t0 + kStride);
        };

        // the first step's loads go out before q is touched
        int t0 = begin + wave * kStep;
        if (t0 < stop) {
            load_pages(t0);
            load_k(t0);
            load_v(t0);
            load_pages(t0 + kStride);
        }
        __builtin_amdgcn_sched_barrier(0);
        // q row -> fp16 operands, scaled by a power of two (and by the sign of
        // the softmax's scale, so that larger is always larger)
        {
            const uint16_t* qp = a.q + (int64_t)(rw.first + qi) * a.q_stride + (int64_t)head * D + 8 * kg;
            uint4 qr[NC];
            uint32_t qmax = 0;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                qr[i] = *reinterpret_cast<const uint4*>(qp + 32 * i);
                const uint32_t u[4] = {qr[i].x, qr[i].y, qr[i].z, qr[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e)  // as integers: a NaN is the largest
                    qmax = max(qmax, max((u[e] << 16) & 0x7fffffffu, u[e] & 0x7fff0000u));
            }
            qmax = max(qmax, (uint32_t)__shfl_xor((int)qmax, 16, kWave));
            qmax = max(qmax, (uint32_t)__shfl_xor((int)qmax, 32, kWave));
            const int ue = min(14 - exponent(__uint_as_float(qmax)), 126);
            float up = a.scale_log2 < 0.0f ? -pow2(ue) : pow2(ue);
            logit = fabsf(a.scale_log2) * pow2(-ue);
            if (logit == 0.0f) {  // logits of 0 (and no 0 * -inf where positions are hidden)
                up = 0.0f;
                logit = 1.0f;
            }
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const uint32_t u[4] = {qr[i].x, qr[i].y, qr[i].z, qr[i].w};
                float f[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[2 * e] = __uint_as_float(u[e] << 16) * up;
                    f[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u) * up;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {  // the order of word_codes
                    qf[i][2 * e] = (_Float16)f[e];
                    qf[i][2 * e + 1] = (_Float16)f[e + 4];
                }
            }
        }
        if (t0 < stop) {
            for (; min(t0 + kStep, stop) <= all_see && t0 < stop; t0 += kStride) step(std::false_type{}, t0);
            if (t0 < stop) {
                step(std::true_type{}, t0);
                finished = true;
            }
        }

        int lane_e = (int)threadIdx.x & (kWave - 1);
        pin(lane_e);  // what follows from it is worked out here, not kept over the steps
        const int lane = lane_e, r16 = lane & 15, kg = lane >> 4;
        // the wave's own result: sum p v / sum p, its maximum and its sum of weights
        if (!finished) {
            l = row_sum(l);
            const float inv = l > 0.0f ? 1.0f / l : l;  // (0 and NaN stay)
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const float unit = group_unit(g);
#pragma unroll
                for (int j = g * G / 16; j < (g + 1) * G / 16; ++j) o[j] = o[j] * inv * unit;
            }
        }
        // join the waves: the upper half into the lower, and so on (the join buffers
        // are free again after the last barrier)
        auto put = [&](float* dst) {
#pragma unroll
            for (int j = 0; j < NT; ++j) *reinterpret_cast<f32x4_t*>(dst + (j * kWave + lane) * 4) = o[j];
            dst[NT * 4 * kWave + lane] = m;
            dst[(NT * 4 + 1) * kWave + lane] = l;
        };
        auto add = [&](const float* src) {
            const float m2 = src[NT * 4 * kWave + lane];
            const float l2 = src[(NT * 4 + 1) * kWave + lane];
            const float mn = fmaxf(m, m2);
            const float base = mn == -INFINITY ? 0.0f : mn;
            const float w1 = l * __builtin_amdgcn_exp2f(m - base), w2 = l2 * __builtin_amdgcn_exp2f(m2 - base);
            l = w1 + w2;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const float f1 = w1 * inv, f2 = w2 * inv;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const f32x4_t x = *reinterpret_cast<const f32x4_t*>(src + (j * kWave + lane) * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[j][e] = fmaf(x[e], f2, o[j][e] * f1);
            }
            m = mn;
        };
#pragma unroll
        for (int n = kWaves / 2; n > 0; n >>= 1) {
            if (wave >= n && wave < 2 * n) put(join[wave - n]);
            __syncthreads();
            if (wave < n) add(join[wave]);
            __syncthreads();
        }
        if (wave == 0) {
            if (rw.bad || seen > rw.held) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[j][e] = __uint_as_float(0x7fc00000u);
            }
            if (whole) {
                if (live) {
                    uint16_t* op = a.out + ((int64_t)(rw.first + qi) * a.q_heads + head) * D + 4 * kg;
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        *reinterpret_cast<uint2*>(op + 16 * j) =
                            make_uint2(bf16x2(o[j][0], o[j][1]), bf16x2(o[j][2], o[j][3]));
                }
            } else if (live) {
                const int64_t at = ((int64_t)group * 2 + slot) * 16 + r16;
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    *reinterpret_cast<f32x4_t*>(a.part + at * D + 16 * j + 4 * kg) = o[j];
                if (kg == 0) a.part_ml[at] = make_float2(m, l);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Many new tokens (a prompt, or a piece of one): bound by the matrix cores and
// the vector units, so each code is expanded once for many rows.  NW waves of 32
// rows each share steps of 16 NW positions.  Half of the waves expand a step's
// keys, half its values, 32 positions each, to fp16 in LDS (code * scale, two
// buffers, one barrier per step; a step's words are loaded two steps ahead);
// then every wave multiplies with v_mfma_f32_32x32x16_f16, transposed as above
// (lane & 31 is a row throughout, P^T goes in as S^T comes out).
//
// Here keys and values are rounded: a scale to fp16 (2^-11, after a power of
// two common to 32 positions), its product with the code again (2^-11).  The
// alternative, exact codes and a scale per group after the product, is 128 more
// vector operations per 64 positions, a third of the step.  A value scale that is
// NaN is taken as 0 and marked: its dimensions become NaN in the rows that see it.
// The common power of two counts no group whose codes are all 0.  Where the causal
// mask crosses the 32 and their scales lie far apart, each position takes a power of
// two of its own instead, and a wave whose rows see less than its exponents stand
// for scales its weights row by row and adds the products in fp32.
//
// LDS: 16-byte pieces.  Keys: word w of position t is piece w of row t; values,
// transposed: the 8 positions that a lane's operand holds are a piece of
// dimension d's row.  Piece p of a row lies at p ^ swizzle(row), which spreads the
// rows of a pass over the banks (of rows of 8 pieces, two share all banks).
//
// 1000 new tokens over 6000 and 569 over 4083 (8 kv heads of 128, 32 query heads,
// g = 32) 215 us: 126 GFLOP, 0.59 PFLOP/s.  The join is 14 us of it.  A step of 128
// positions takes 6.2 us, about the sum of what its parts take alone (counted
// instructions): vector work 2.4 (softmax, expansion), LDS reads 2.2, matrix
// instructions 1.5; two waves per SIMD, which the registers of 32 rows by 128
// dimensions allow, overlap little of it.  The registers do not suffice either: heads
// of 128 spill 71 to 110 of them (260 bytes of scratch a lane at g = 32), nearly all
// outside the steps; a dozen scratch accesses are in the loop.  Tiles of 128 rows
// (half as many codes shared) were slower, 294 against 254 us before the stretches;
// whole units (200 for 256 CUs, 32 to 47 steps) 268 us.

constexpr int kValueShift = 24;  // keeps a weight (up to 2^14) times a value's power of two in fp32
template <int D, int G, int NW>
struct PromptTile {
    static constexpr int kRows = 32 * NW;
    static constexpr int kTiles = NW / 2;      // of 32 positions per step
    static constexpr int kPos = 32 * kTiles;
    static constexpr int kThreads = 64 * NW;
    static constexpr int kOcc = D == 256 ? 1 : 2;  // waves per SIMD
};

template <int D, int G, int NW>
__global__ __launch_bounds__(64 * NW, (PromptTile<D, G, NW>::kOcc)) void cache4_prompt_kernel(AttnArgs a, int32_t grid_tiles)
{
    using Tl = PromptTile<D, G, NW>;
    constexpr int NC = D / 32, NG = D / G, NT = D / 32;
    constexpr int TT = Tl::kTiles, kPos = Tl::kPos;
    constexpr int KW = D / 16;                     // key words of a lane: half a row
    constexpr int VW = D / 128 > 0 ? D / 128 : 1;  // value words of a lane and position
    constexpr int NS = (NG + 1) / 2;               // scales of a lane
    __shared__ __attribute__((aligned(16))) uint4 Kt[2][kPos * (D / 8)];
    __shared__ __attribute__((aligned(16))) uint4 Vt[2][D * (kPos / 8)];
    __shared__ __attribute__((aligned(16))) _Float16 sc[NW][32 * NG];
    __shared__ int kexp[2][TT], vexp[2][TT];  // twice the exponent; odd: one per position
    __shared__ __attribute__((aligned(16))) float kpow[2][TT][32], vpow[2][TT][32];
    __shared__ uint32_t vnan[2][TT][NG];

    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r32 = lane & 31;
    const int h = lane >> 5;
    const int shift = a.c.page_shift;

    // units (sequence, kv head, tile), a contiguous range of them per XCD, so that
    // the tiles of a kv head share an L2; a head's last tiles, the longest, first
    // Or, with grid_tiles = 0, an equal stretch of the line of steps, and the parts
    // of a unit are joined by cache4_join_edges_kernel.
    const bool split = grid_tiles == 0;
    int b, kvh = 0, group = 0;
    int64_t tile = 0, x = 0, x1 = 0, before = 0;
    Rows rw;
    if (split) {
        group = (a.groups & 7) == 0 ? (int)(blockIdx.x & 7) * (a.groups >> 3) + (int)(blockIdx.x >> 3)
                                    : (int)blockIdx.x;
        const Line ln = lay_line<Tl, true>(a, group, 0);
        if (ln.b < 0) return;
        b = ln.b;
        x = uniform64(ln.first(group));
        x1 = uniform64(ln.first(group + 1));
        before = uniform64(ln.before);
        rw = ln.rw;
    } else {
        const int64_t units = (int64_t)a.bt.count * a.c.heads * grid_tiles;
        const int64_t u = (int64_t)(blockIdx.x & 7) * ((units + 7) >> 3) + (blockIdx.x >> 3);
        if (u >= units) return;
        const int64_t head_unit = uniform64(udiv(u, grid_tiles));
        tile = grid_tiles - 1 - (int)(u - head_unit * grid_tiles);
        b = __builtin_amdgcn_readfirstlane((int)udiv(head_unit, a.c.heads));
        kvh = (int)(head_unit - (int64_t)b * a.c.heads);
        rw = rows_of(a, b);
    }
    const int64_t x0 = x;

    for (;; tile += grid_tiles) {
        const int64_t rows = rw.rows();
        const int steps = steps_of(a, rw);
        int step0 = 0, take = steps, slot = 0;
        if (split) {
            if (x >= x1) break;
            const int64_t tiles = tiles_of<Tl>(rw);
            if (x >= before + tiles * a.c.heads * steps) {
                before += tiles * a.c.heads * steps;
                ++b;
                rw = rows_of(a, b);
                continue;
            }
            const int64_t unit = uniform64(udiv(x - before, steps));
            step0 = (int)(x - before - unit * steps);
            take = (int)(x1 - x < steps - step0 ? x1 - x : steps - step0);
            slot = x == x0 ? 0 : 1;
            kvh = __builtin_amdgcn_readfirstlane((int)udiv(unit, tiles));
            tile = unit - kvh * tiles;
            x += take;
        } else if (tile * Tl::kRows >= rows) {
            break;
        }
        const __attribute__((address_space(4))) int32_t* table =
            (const __attribute__((address_space(4))) int32_t*)(a.bt.table + b * a.bt.width);
        const int64_t r0 = tile * Tl::kRows;
        const int64_t w0 = r0 + wave * 32;  // the wave's first row
        const bool live = w0 + r32 < rows;
        const int64_t row = live ? w0 + r32 : 0;
        const int qi = (int)udiv(row, rw.per);
        const int head = kvh * rw.per + (int)(row - (int64_t)qi * rw.per);
        const int seen = live ? rw.seen(row) : 0;
        const auto seen_at = [&](int64_t r) { return __builtin_amdgcn_readfirstlane(rw.seen(r < rows ? r : rows - 1)); };
        const int end = min(seen_at(r0 + Tl::kRows - 1), rw.held);   // of the workgroup's rows
        const int wave_end = w0 < rows ? min(seen_at(w0 + 31), rw.held) : 0;  // of the wave's
        const int begin = step0 * kPos;
        const int stop = end < begin + take * kPos ? end : begin + take * kPos;
        const int all_see = w0 < rows ? seen_at(w0) : 0;             // by every live row of it
        const int tile_see = seen_at(r0);                            // and of the workgroup

        // q rows: operand kk = 2 i + p holds dimensions 32 i + 8 (2 p + h) + (0 4 1 5 2 6 3 7)
        f16x8_t qf[2 * NC];
        float logit;
        {
            const uint16_t* qp = a.q + (int64_t)(rw.first + qi) * a.q_stride + (int64_t)head * D + 8 * h;
            uint4 qr[2 * NC];
            uint32_t qmax = 0;
#pragma unroll
            for (int k = 0; k < 2 * NC; ++k) {
                qr[k] = *reinterpret_cast<const uint4*>(qp + 16 * k);
                const uint32_t v[4] = {qr[k].x, qr[k].y, qr[k].z, qr[k].w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    qmax = max(qmax, max((v[e] << 16) & 0x7fffffffu, v[e] & 0x7fff0000u));
            }
            qmax = max(qmax, (uint32_t)__shfl_xor((int)qmax, 32, kWave));
            const int ue = min(14 - exponent(__uint_as_float(qmax)), 126);
            float up = a.scale_log2 < 0.0f ? -pow2(ue) : pow2(ue);
            logit = fabsf(a.scale_log2) * pow2(-ue);
            if (logit == 0.0f) {
                up = 0.0f;
                logit = 1.0f;
            }
#pragma unroll
            for (int k = 0; k < 2 * NC; ++k) {
                const uint32_t v[4] = {qr[k].x, qr[k].y, qr[k].z, qr[k].w};
                float f[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[2 * e] = __uint_as_float(v[e] << 16) * up;
                    f[2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u) * up;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    qf[k][2 * e] = (_Float16)f[e];
                    qf[k][2 * e + 1] = (_Float16)f[e + 4];
                }
            }
        }

        int vrun = -1000;  // the largest exponent of the values that this wave expanded
        // ---- a step's words: wave w < TT has the keys of 32 positions, w >= TT values
        const bool keys = wave < TT;
        const int part = keys ? wave : wave - TT;  // which 32 positions of the step
        uint32_t raw[KW > 8 * VW ? KW : 8 * VW];  // key words, or value words [position][word]
        float sl[NS];
        uint32_t bad = 0;  // a NaN's bits where the page is outside the cache
        auto load = [&](int pos0) __attribute__((always_inline)) {
            const int t0 = pos0 + 32 * part;
            int pg[2], tt[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                tt[i] = t0 + 16 * i < end ? t0 + 16 * i : (end - 1) & ~15;
                pg[i] = table[tt[i] >> shift];
            }
            // this lane's 16 positions: the lower or the upper half of the wave
            const int t16 = h ? tt[1] : tt[0];
            const int page = h ? pg[1] : pg[0];
            const bool ok = (unsigned)page < (unsigned)a.c.pages;
            bad = ok ? 0u : 0x7fc00000u;
            const int64_t block = (int64_t)(ok ? page : 0) * a.c.heads + kvh;
            const int off = t16 & ((1 << shift) - 1);
            const int64_t code_row = (block << shift) + off;
            if (keys) {
                const uint32_t* kp = a.c.k_codes + (code_row + ((lane >> 1) & 15)) * (D / 8) + (lane & 1) * KW;
#pragma unroll
                for (int i = 0; i < KW; i += 4) {
                    const uint4 v = *reinterpret_cast<const uint4*>(kp + i);
                    raw[i] = v.x, raw[i + 1] = v.y, raw[i + 2] = v.z, raw[i + 3] = v.w;
                }
            } else {
                // positions 4 h' + e and 8 + 4 h' + e of the 16, h' = bit 4 of the lane
                const int first = ((lane >> 4) & 1) * 4;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t* vp = a.c.v_codes + (code_row + first + (e & 3) + (e & 4) * 2) * (D / 8);
                    if constexpr (D == 64) {
                        raw[e] = reinterpret_cast<const uint16_t*>(vp)[lane & 15];
                    } else {
#pragma unroll
                        for (int i = 0; i < VW; ++i) raw[e * VW + i] = vp[(lane & 15) * VW + i];
                    }
                }
            }
            // scales of position lane & 15 of the 16, groups of the parity of bit 4
            const float* sp = (keys ? a.c.k_scales : a.c.v_scales) + ((block * NG) << shift) + off + (lane & 15);
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const int g = 2 * i + ((lane >> 4) & 1) < NG ? 2 * i + ((lane >> 4) & 1) : NG - 1;
                sl[i] = sp[(int64_t)g << shift];
            }
        };
        // Scales of groups whose codes are all 0 become 0 (a NaN stays NaN).
        auto drop_zero_groups = [&](int lane) __attribute__((always_inline)) {
            const int t = lane & 15, gpar = (lane >> 4) & 1;
            uint32_t zero[2] = {0, 0};
            if (keys) {
                // two lanes have the words of a position, which say whether a group has others
                uint32_t some = 0;
#pragma unroll
                for (int k = 0; k < KW; ++k)
                    if (raw[k] != 0x88888888u) some |= 1u << (k % NC * 32 / G);
                some |= (uint32_t)__shfl_xor((int)some, 1, kWave);
                zero[0] = ~(uint32_t)__shfl((int)some, (lane & 32) + 2 * t, kWave);
            } else {
                // 16 lanes have those of 8 positions; bit e * NG + g, two words where NG is 8
                uint32_t none[2] = {0, 0};
#pragma unroll
                for (int e = 0; e < 8; ++e)
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        constexpr int n = G / 16;  // codes of the group in a lane
                        const uint32_t mask = (n == 8 ? ~0u : (1u << (4 * (n & 7))) - 1u) << (4 * (g * n % 8));
                        const uint64_t lanes = __ballot(((raw[e * VW + g * n / 8] ^ 0x88888888u) & mask) == 0);
                        if (((lanes >> (lane & 48)) & 0xffffu) == 0xffffu)
                            none[NG == 8 ? e / 4 : 0] |= 1u << ((e * NG + g) & 31);
                    }
                const int from = (lane & 32) + 4 * (t & 4);
                zero[0] = (uint32_t)__shfl((int)none[0], from, kWave);
                zero[1] = NG == 8 ? (uint32_t)__shfl((int)none[1], from, kWave) : 0u;
                if (NG == 8 && t >= 8) zero[0] = zero[1];
                zero[0] >>= ((t & 3) + (NG == 8 ? 0 : t >> 3 << 2)) * NG & 31;
            }
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const int g = 2 * i + gpar < NG ? 2 * i + gpar : NG - 1;
                if ((zero[0] >> g & 1) && sl[i] == sl[i]) sl[i] = 0.0f;
            }
        };
        // the loaded words -> fp16 pieces of buffer nb
        auto expand = [&](int pos0, int nb) __attribute__((always_inline)) {
            int lane = (int)threadIdx.x & (kWave - 1);
            pin(lane);  // what follows from it is worked out here, not kept
            const int h = lane >> 5;
            const bool past = pos0 + 32 * part + 16 * h + (lane & 15) >= end;
            const int gpar = (lane >> 4) & 1;
            uint64_t nan_at[NS];
            bool unsure = false;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                if (past) sl[i] = 0.0f;
                nan_at[i] = 0;
                if (!keys) {
                    const bool nan = !(fabsf(sl[i]) < INFINITY);
                    nan_at[i] = __ballot(nan);
                    if (nan) sl[i] = 0.0f;
                }
                unsure |= __float_as_uint(sl[i]) == kZeroScale;
            }
            // the exponent of the largest scale of the 32 positions
            const auto top_exponent = [&]() __attribute__((always_inline)) {
                float top = 0.0f;
#pragma unroll
                for (int i = 0; i < NS; ++i) top = fmaxf(top, fabsf(sl[i]));
                const int ex = exponent(__uint_as_float(
                    __builtin_amdgcn_readfirstlane(__float_as_uint(wave_max_abs(top)))));
                return ex < -104 ? -104 : ex;
            };
            int ex = top_exponent();
            // Groups whose codes are all 0 must not raise it, nor positions that some row
            // does not see those of the rows that do not: where the causal mask crosses the
            // 32 and scales lie far apart, each position has an exponent of its own.
            const bool crossed = pos0 + 32 * part + 32 > tile_see;
            bool apart = false;
            if (__builtin_expect(crossed || (keys ? __any(unsure) != 0 : ex > vrun), 0)) {
                if (__any(unsure)) {
                    drop_zero_groups(lane);
                    ex = top_exponent();
                }
                uint32_t low = 0;  // of the smallest scale but 0, turned round
#pragma unroll
                for (int i = 0; i < NS; ++i)
                    if (sl[i] != 0.0f) low = max(low, 0x7f800000u - (__float_as_uint(fabsf(sl[i])) & 0x7f800000u));
                low = __float_as_uint(wave_max_abs(__uint_as_float(low)));
                const int least = 128 - (int)(__builtin_amdgcn_readfirstlane(low) >> 23);
                apart = ex - least > (keys ? 20 : 8) && (keys || crossed);
                if (!crossed && ex > vrun) vrun = ex;
            }
            // values: in steps of 8, so that the running exponent seldom moves
            if (!keys) ex |= 7;
            int own = ex;
            if (__builtin_expect(apart, 0)) {
                float top = 0.0f;
#pragma unroll
                for (int i = 0; i < NS; ++i) top = fmaxf(top, fabsf(sl[i]));
                top = fmaxf(top, __shfl_xor(top, 16, kWave));
                own = max(exponent(top), -104);  // (a position without codes: the least)
                float* const table = keys ? kpow[nb][part] : vpow[nb][part];
                table[16 * h + (lane & 15)] = pow2(own - (keys ? 10 : kValueShift));
            }
            const float fac = pow2(10 - own);
            _Float16* const s16 = sc[wave];
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const int g = 2 * i + gpar;
                if (g < NG) {
                    const float x = sl[i] * fac;
                    if (keys) {
                        // NaN stays, and a page outside the cache is one
                        s16[(16 * h + (lane & 15)) * NG + g] =
                            (_Float16)__uint_as_float(__float_as_uint(x) | bad);
                    } else {
                        const int t = lane & 15;
                        s16[g * 32 + (2 * h + ((t >> 2) & 1)) * 8 + (t & 3) + 4 * (t >> 3)] = (_Float16)x;
                    }
                }
            }
            if (lane == 0) {
                if (keys) {
                    kexp[nb][part] = 2 * ex + (apart ? 1 : 0);
                } else {
                    vexp[nb][part] = 2 * ex + (apart ? 1 : 0);
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        // lanes 32 s + 16 (g & 1) + t: position 16 s + t
                        const uint64_t m = nan_at[g >> 1] >> (16 * (g & 1));
                        vnan[nb][part][g] = (uint32_t)(m & 0xffffu) | ((uint32_t)(m >> 32) << 16);
                    }
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (keys) {
                const int t = lane >> 1;
                uint4* const dst = &Kt[nb][(32 * part + t) * (D / 8)];
                f16x2_t s2[NG];
#pragma unroll
                for (int g = 0; g < NG; ++g) s2[g] = (f16x2_t){s16[t * NG + g], s16[t * NG + g]};
#pragma unroll
                for (int k = 0; k < KW; ++k) {
                    const f16x2_t s = s2[(k % NC) * 32 / G];
                    const uint32_t x = raw[k] >> 8;
                    const uint4 v = make_uint4(u32_of(f16x2_of(low_codes(raw[k])) * s), u32_of(f16x2_of(high_codes(raw[k])) * s),
                                               u32_of(f16x2_of(low_codes(x)) * s), u32_of(f16x2_of(high_codes(x)) * s));
                    dst[((lane & 1) * KW + k) ^ swizzle<D / 8>(t)] = v;
                }
            } else {
                const int tg = lane >> 4;
                uint32_t s4[NG][4];
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const uint4 v = *reinterpret_cast<const uint4*>(s16 + g * 32 + tg * 8);
                    s4[g][0] = v.x, s4[g][1] = v.y, s4[g][2] = v.z, s4[g][3] = v.w;
                }
#pragma unroll
                for (int i = 0; i < VW; ++i) {
#pragma unroll
                    for (int n = 0; n < (D == 64 ? 2 : 4); ++n) {
                        const uint32_t sel = 0x0c000c00u | ((uint32_t)(4 + n) << 16) | (uint32_t)n;
                        const int j = 8 * i + 2 * n;
                        uint32_t lo[4], hi[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t v = __builtin_amdgcn_perm(raw[(2 * e + 1) * VW + i], raw[2 * e * VW + i], sel);
                            lo[e] = u32_of(f16x2_of(low_codes(v)) * f16x2_of(s4[16 * j / G][e]));
                            hi[e] = u32_of(f16x2_of(high_codes(v)) * f16x2_of(s4[16 * (j + 1) / G][e]));
                        }
                        const int d = 16 * j + (lane & 15);
                        const int q = (4 * part + tg) ^ swizzle<kPos / 8>(d);
                        Vt[nb][d * (kPos / 8) + q] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        Vt[nb][(d + 16) * (kPos / 8) + q] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    }
                }
            }
        };

        float m = -INFINITY, l = 0.0f;
        int ve = -97;  // exponent of the row's values in o
        f32x16_t o[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[j][e] = 0.0f;

        // LDS addresses of this lane's operand pieces in the buffer to multiply next.
        // Held as they are (pin): left to itself the compiler keeps far more derived
        // ones over the loop than there are registers, and spills them.
        uint32_t ka[2 * NC], va[2 * TT];
#pragma unroll
        for (int k = 0; k < 2 * NC; ++k)
            ka[k] = lds_address(&Kt[0][r32 * (D / 8) + (((2 * (k & 1) + h) * NC + (k >> 1)) ^ swizzle<D / 8>(r32))]);
#pragma unroll
        for (int k = 0; k < 2 * TT; ++k)
            va[k] = lds_address(&Vt[0][r32 * (kPos / 8) + ((2 * k + h) ^ swizzle<kPos / 8>(r32))]);
        constexpr int kHop = sizeof(Kt[0]), vHop = sizeof(Vt[0]);  // to the other buffer

        // 64 positions of buffer cb, the tiles 2 hp and 2 hp + 1
        auto compute = [&](int pos, int cb, int hp) __attribute__((always_inline)) {
            f32x16_t s[2];
            float f[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int e = 0; e < 16; ++e) s[t][e] = 0.0f;
#pragma unroll
                for (int k = 0; k < 2 * NC; ++k)
                    s[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                        lds_piece(ka[k] + 32 * (2 * hp + t) * (2 * D)), qf[k], s[t], 0, 0, 0);
                const int kx = __builtin_amdgcn_readfirstlane(kexp[cb][2 * hp + t]);
                // (not 0, which a hidden position's -inf would make NaN)
                f[t] = fmaxf(logit * pow2((kx >> 1) - 10), 0x1p-126f);
                if (__builtin_expect(kx & 1, 0)) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x4_t w = *reinterpret_cast<const f32x4_t*>(&kpow[cb][2 * hp + t][8 * q + 4 * h]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[t][4 * q + e] *= logit * w[e];
                    }
                    f[t] = 1.0f;
                }
            }
            if (pos + 64 > all_see) {
                const int left = seen - pos - 4 * h;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (32 * t + 8 * (e >> 2) + (e & 3) >= left) s[t][e] = -INFINITY;
            }
            float mx[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                mx[t] = s[t][0];
#pragma unroll
                for (int e = 1; e < 16; ++e) mx[t] = fmaxf(mx[t], s[t][e]);
            }
            float x0 = fmaxf(mx[0] * f[0], mx[1] * f[1]), x1;
            row_pair(x0, true, x0, x1);
            const float top = fmaxf(x0, x1);
            // the reference only moves by more than 2^8 (weights stay below it), and
            // the values' exponent with the largest seen
            const int x0v = __builtin_amdgcn_readfirstlane(vexp[cb][2 * hp]);
            const int x1v = __builtin_amdgcn_readfirstlane(vexp[cb][2 * hp + 1]);
            const int v0 = x0v >> 1, v1 = x1v >> 1;
            // a row may see less than the tiles' exponents stand for: a scale for each row
            const bool alone = ((x0v | x1v) & 1) != 0 || (pos + 64 > all_see && __any(max(v0, v1) > ve));
            const int vn = alone ? ve : max(ve, max(v0, v1));
            if (__any(top > m + 8.0f || vn != ve)) {
                const float mn = top > m + 8.0f ? top : m;
                const float alpha = mn == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
                const float os = alpha * pow2(ve - vn);
                m = mn;
                ve = vn;
                l *= alpha;
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[j][e] *= os;
            }
            // weights up to 2^14: fp16's normal range then reaches 2^-20 of the largest
            const float base = m == -INFINITY ? 0.0f : m - 6.0f;
            f16x8_t p[2][2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float sum = 0.0f;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    s[t][e] = __builtin_amdgcn_exp2f(fmaf(s[t][e], f[t], -base));
                    sum += s[t][e];
                }
                l += sum;
            }
            if (__builtin_expect(alone, 0)) {
                // The weights times a power of two of each position's values, and of each row
                // that puts the largest of it in [2^14, 2^15); the products are added to o
                // in fp32, in units that follow what the row sees.
                float top2 = 0.0f;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float all = pow2((t ? v1 : v0) - kValueShift);
                        f32x4_t w = {all, all, all, all};
                        if ((t ? x1v : x0v) & 1)
                            w = *reinterpret_cast<const f32x4_t*>(&vpow[cb][2 * hp + t][8 * q + 4 * h]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            s[t][4 * q + e] *= w[e];
                            top2 = fmaxf(top2, s[t][4 * q + e]);
                        }
                    }
                float y0, y1;
                row_pair(top2, true, y0, y1);
                const int tx = max(exponent(fmaxf(y0, y1)), -112);
                const int vm = max(ve, tx + kValueShift - 14);
                const float os = pow2(ve - vm), up = pow2(14 - tx), back = pow2(tx - 14 + kValueShift - vm);
                ve = vm;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 16; ++e) p[t][e >> 3][e & 7] = (_Float16)(s[t][e] * up);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    f32x16_t x;
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = 0.0f;
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            x = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                                lds_piece(va[2 * (2 * hp + t) + k] + 32 * j * (2 * kPos)), p[t][k], x, 0, 0, 0);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[j][e] = fmaf(x[e], back, o[j][e] * os);
                    __builtin_amdgcn_sched_barrier(0);
                }
            } else {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int de = (t ? v1 : v0) - ve;
                    if (__any(de != 0)) {  // values of another exponent
                        const float down = pow2(de);
#pragma unroll
                        for (int e = 0; e < 16; ++e) s[t][e] *= down;
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) p[t][e >> 3][e & 7] = (_Float16)s[t][e];
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) {
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            o[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                                lds_piece(va[2 * (2 * hp + t) + k] + 32 * j * (2 * kPos)), p[t][k], o[j], 0, 0, 0);
                }
            }
            // a NaN value scale: NaN in its dimensions, in the rows that see it
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint32_t n0 = vnan[cb][2 * hp][32 * j / G], n1 = vnan[cb][2 * hp + 1][32 * j / G];
                if ((n0 | n1) != 0) {
                    const int see = seen - pos;  // positions of these 64
                    const uint64_t mask = (uint64_t)n0 | ((uint64_t)n1 << 32);
                    const uint64_t mine = see >= 64 ? mask : (see <= 0 ? 0 : mask & ((1ull << see) - 1));
                    if (mine) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[j][e] = __uint_as_float(0x7fc00000u);
                    }
                }
            }
        };

        if (begin < stop) {
            load(begin);
            expand(begin, 0);
            if (begin + kPos < stop) load(begin + kPos);
            for (int pos = begin, cb = 0; pos < stop; pos += kPos, cb ^= 1) {
                lds_barrier();  // buffer cb is whole, the other is read by no wave any more
                // the waves of the keys expand before they multiply, those of the
                // values after: a SIMD has one of each, and so both kinds of work
                auto refill = [&]() __attribute__((always_inline)) {
                    if (pos + kPos < stop) {
                        expand(pos + kPos, cb ^ 1);
                        if (pos + 2 * kPos < stop) load(pos + 2 * kPos);
                    }
                };
                if (keys) refill();
#pragma unroll
                for (int hp = 0; hp < TT / 2; ++hp)
                    if (pos + 64 * hp < wave_end) compute(pos + 64 * hp, cb, hp);
                if (!keys) refill();
#pragma unroll
                for (int k = 0; k < 2 * NC; ++k) {
                    ka[k] += cb ? -kHop : kHop;
                    pin(ka[k]);
                }
#pragma unroll
                for (int k = 0; k < 2 * TT; ++k) {
                    va[k] += cb ? -vHop : vHop;
                    pin(va[k]);
                }
            }
        }

        int lane_e = (int)threadIdx.x & (kWave - 1);
        pin(lane_e);  // what follows from it is worked out here, not kept over the steps
        const int r32 = lane_e & 31, h = lane_e >> 5;
        float l0, l1;
        row_pair(l, true, l0, l1);
        l = l0 + l1;
        float inv = l > 0.0f ? pow2(ve - 10) / l : (l == 0.0f ? 0.0f : l);  // NaN stays
        if (rw.bad || seen > rw.held) inv = __uint_as_float(0x7fc00000u);
        if (live && take < steps) {
            const int64_t at = ((int64_t)group * 2 + slot) * Tl::kRows + wave * 32 + r32;
            float* pp = a.part + at * D + 4 * h;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *reinterpret_cast<f32x4_t*>(pp + 32 * j + 8 * e) =
                        (f32x4_t){o[j][4 * e], o[j][4 * e + 1], o[j][4 * e + 2], o[j][4 * e + 3]} * inv;
            if (h == 0) a.part_ml[at] = make_float2(m, l);
        } else if (live) {
            uint16_t* op = a.out + ((int64_t)(rw.first + qi) * a.q_heads + head) * D + 4 * h;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *reinterpret_cast<uint2*>(op + 32 * j + 8 * e) =
                        make_uint2(bf16x2(o[j][4 * e] * inv, o[j][4 * e + 1] * inv),
                                   bf16x2(o[j][4 * e + 2] * inv, o[j][4 * e + 3] * inv));
        }
        lds_barrier();  // the buffers are free for the next tile
    }
}

// The launch's shape.  Few new tokens: kFill stretches of the line, fewer where
// there are not that many steps (half of it for heads of 256, whose LDS lets fewer
// workgroups onto a CU); units are steps as they are, and nothing is joined, while
// they are short or fill the CUs.  Decode with 8 kv heads of 128, whole / cut: 8
// sequences of 400 10.3 / 11.2 us, of 800 14.0 / 12.8; 24 (192 units) of up to 1600
// 22.5 / 23.2, of 2400 29.7 / 26.4; 64 (512) of 4000 63.7 / 64.7, of 7000 107 / 102;
// 32 of 600 12.9 / 19.8.  Beyond 4096 one long sequence would outlast all others.
// Many: cache4_prompt_kernel from kPromptUnits units (sequence, kv head, tile of
// rows) on, or kPromptRows rows per kv head and kPromptSteps steps for each of its
// workgroups.  It splits units into stretches below kSplitUnits units for each
// workgroup, if the steps that the causal mask takes from a stretch are
// few (len >= kSplitLen new).  Both limits are rough: a stretch counts a unit's steps
// as if its rows saw the whole sequence, so first prompts stay whole though few
// units leave CUs idle (1 x 1000 over 1000, 128 units, 54 us; 1 x 2000 over 2000 99
// us), and the last but one line below has 1128 units and takes the slower form.
// Measured with 32 query and 8 kv heads of 128, one sequence's new tokens over its
// length:
//   100 over 20000 (400 rows, 12 steps): 110 us, cache4_attention_kernel 129 us;
//    64 over 20000 (256 rows,  5 steps):  97 us, cache4_attention_kernel  91 us;
//   2 x 100 over 6000 (400 rows, 6 steps): 76 us, cache4_attention_kernel 69 us;
//   512 over 8000: split 144 us, whole units of 128 rows 338 us;
//   3 x 3000 over 12000: split 1842 us, whole 2100 us;
//   4 x 2000 over 2000: split 337 us, whole 242 us.
constexpr int64_t kFill = 512;
constexpr int64_t kWholeFill = 2048;
constexpr int64_t kPromptUnits = 96;
constexpr int64_t kPromptRows = 320;
constexpr int64_t kPromptSteps = 8;
constexpr int64_t kSplitUnits = 4;
constexpr int64_t kSplitLen = 2;

struct Plan {
    int64_t rows, units, groups;
    int step_shift;
    int prompt_waves;      // 0: cache4_attention_kernel, else waves of cache4_prompt_kernel
    int64_t prompt_tiles;  // its row tiles per (sequence, kv head)
    size_t part_bytes, ml_bytes;
};

// heads * tiles, or kMaxUnits, which as a product with any length fits 64 bits
constexpr int64_t kMaxUnits = 1LL << 23;
int64_t units_of(int64_t heads, int64_t tiles)
{
    return tiles > kMaxUnits / heads ? kMaxUnits : heads * tiles;
}

Plan plan_of(const Cache4& c, int64_t count, int64_t tokens, int q_heads, int64_t max_q, int64_t max_len)
{
    Plan p{};
    if (max_q > tokens) max_q = tokens;
    if (max_len > 0x7fffffffLL) max_len = 0x7fffffffLL;
    p.rows = max_q * (q_heads / c.heads);
    for (int waves = 8; waves >= 4; waves /= 2) {
        if (waves == 8 && c.dim == 256) continue;  // the buffers would not fit in LDS
        const int64_t tiles = ceil_div(p.rows, 32 * waves);
        const int64_t units = units_of(count * c.heads, tiles);
        const int64_t fill = c.dim != 256 && waves == 4 ? 512 : 256;
        const bool many = units >= kPromptUnits;
        const bool deep = fill == 256 && p.rows >= kPromptRows &&
                          units * ceil_div(max_len, 16 * waves) >= kPromptSteps * fill;
        // (a launch has at most 2^32 - 1 threads)
        if (p.rows < 16 * waves || !(many || deep) || units > kMaxUnits / 2) continue;
        p.prompt_waves = waves;
        p.step_shift = waves == 8 ? 7 : 6;
        p.prompt_tiles = tiles;
        if (!many || (units < kSplitUnits * fill && max_len >= kSplitLen * max_q)) {
            p.groups = fill;
            p.part_bytes = (size_t)fill * 2 * 32 * waves * c.dim * sizeof(float);
            p.ml_bytes = (size_t)fill * 2 * 32 * waves * sizeof(float2);
        }
        return p;
    }
    p.units = units_of(count * c.heads, ceil_div(p.rows, 16));
    const int64_t fill = c.dim == 256 ? kFill / 2 : kFill;
    if (max_len <= 512 || (p.units >= 192 && max_len <= (p.units < 512 ? 8 * p.units : 4096))) {
        p.groups = p.units < kWholeFill ? p.units : kWholeFill;
        p.step_shift = 31;
        return p;
    }
    p.step_shift = 7;
    p.groups = p.units > fill ? fill : p.units * ceil_div(max_len, kStride);
    if (p.groups > fill) p.groups = fill;
    p.part_bytes = (size_t)p.groups * 2 * 16 * c.dim * sizeof(float);
    p.ml_bytes = (size_t)p.groups * 2 * 16 * sizeof(float2);
    return p;
}

template <int D, int G, int NW>
void launch_prompt(const AttnArgs& a, const Plan& p, hipStream_t stream)
{
    if (p.groups) {
        cache4_prompt_kernel<D, G, NW><<<(unsigned)p.groups, 64 * NW, 0, stream>>>(a, 0);
        cache4_join_edges_kernel<D, PromptTile<D, G, NW>>
            <<<dim3((unsigned)p.groups - 1, 2 * NW), kThreads, 0, stream>>>(a);
    } else {
        const int64_t units = a.bt.count * a.c.heads * p.prompt_tiles;
        cache4_prompt_kernel<D, G, NW><<<(unsigned)((units + 7) & ~7LL), 64 * NW, 0, stream>>>(a, (int32_t)p.prompt_tiles);
    }
}

template <int D, int G>
hipError_t launch_dg(const AttnArgs& a, const Plan& p, hipStream_t stream)
{
    if (p.prompt_waves == 8) {
        if constexpr (D != 256) launch_prompt<D, G, 8>(a, p, stream);
    } else if (p.prompt_waves == 4) {
        launch_prompt<D, G, 4>(a, p, stream);
    } else {
        cache4_attention_kernel<D, G><<<(unsigned)a.groups, kThreads, 0, stream>>>(a);
        if (a.groups > 1 && a.step_shift < 31) {
            if (p.units * 2 > a.groups) {
                cache4_join_edges_kernel<D, SmallCut><<<(unsigned)a.groups - 1, kThreads, 0, stream>>>(a);
            } else {
                const dim3 jgrid((unsigned)p.rows, (unsigned)a.c.heads, (unsigned)a.bt.count);
                cache4_join_kernel<D, SmallCut><<<jgrid, kThreads, 0, stream>>>(a);
            }
        }
    }
    return hipGetLastError();
}

}  // namespace

size_t cache4_attention_workspace(const Cache4& c, int64_t count, int64_t tokens,
                                  int q_heads, int64_t max_q, int64_t max_len)
{
    const Plan p = plan_of(c, count, tokens, q_heads, max_q, max_len);
    return p.part_bytes + p.ml_bytes;
}

hipError_t launch_cache4_attention(const Cache4& c, const Cache4Batch& bt, const uint16_t* q,
                                   int64_t tokens, int64_t q_stride, int q_heads, float scale,
                                   int64_t max_q, int64_t max_len, uint16_t* out, void* workspace,
                                   hipStream_t stream)
{
    const Plan p = plan_of(c, bt.count, tokens, q_heads, max_q, max_len);
    const AttnArgs a{c, bt, q, q_stride, out, tokens, q_heads, scale * kLog2e,
                     static_cast<float*>(workspace),
                     reinterpret_cast<float2*>(static_cast<char*>(workspace) + p.part_bytes),
                     (int32_t)p.groups, p.step_shift};
    switch (c.dim * 1000 + c.group) {
    case 64032: return launch_dg<64, 32>(a, p, stream);
    case 64064: return launch_dg<64, 64>(a, p, stream);
    case 128032: return launch_dg<128, 32>(a, p, stream);
    case 128064: return launch_dg<128, 64>(a, p, stream);
    case 128128: return launch_dg<128, 128>(a, p, stream);
    case 256032: return launch_dg<256, 32>(a, p, stream);
    case 256064: return launch_dg<256, 64>(a, p, stream);
    case 256128: return launch_dg<256, 128>(a, p, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace dq

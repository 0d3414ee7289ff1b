// Attention of drafted tokens over the paged 4-bit cache (cache4.hpp): every token sees the
// cached context, and of the call's own tokens those whose bits its mask has.
//   o[i,h] = sum_t p_t vhat[t] / sum_t p_t,  p_t = exp(scale q[i,h] . khat[t] - max).
//
// A tree has 8 to 64 tokens, so a kv head has some 32 to 500 rows (token, query head),
// between the one tile of 16 that cache4_attention_kernel is made for and the
// thousands of a prompt.  Here a wave expands the codes of 32 positions in registers for a
// tile of 32 rows (32 by 128 of output are 64 registers), and the four waves of a workgroup take neighbouring positions, each with a
// softmax of its own; they meet only at the end of a unit.  Both products run on
// v_mfma_f32_32x32x16_f16 in transposed form, S^T = K Q^T and O^T = V^T P^T: lane & 31 is a
// row throughout, and S^T comes out in the lane and order in which P^T goes in.  Rows of q
// lie in LDS as operands (registers for them would halve the waves of a SIMD).  Codes and scales
// come by buffer loads straight into a wave's ring of two steps in LDS: no register holds
// a load in flight (registers instead of the ring: 245 us for the first case below, the ring 146).
//
// Bound by vector work and matrix work in turn.  A step of 32 positions and 32 rows of 128 is 16
// matrix instructions (512 cycles) and, counted over a call, 380 vector ones, of which 181
// expand codes and 100 are the softmax: 151 k cycles of vector and 47 k of matrix instructions in
// the 218 k that a wave lives (second case below), so two waves hardly overlap; a third (168
// registers, 3 x 52 KB of LDS) changed nothing.  Two tiles of rows a wave, which halve the expansion,
// spill 56 registers: 132 us for the first case, but wrong results where a workgroup has several
// units, so they are not built.  With 8 kv heads of 128, g = 32: 64 tokens of 32 heads over 65000
// positions 144 us with their join (68 GFLOP, 0.47 PFLOP/s), 24 sequences of 24 tokens of 40 heads over
// up to 6000 116 us and 7 (42 GFLOP, 0.34 PFLOP/s; 1.2 TB/s of cache), 8 of 6 tokens over 1100 (16 / 4
// heads of 64) 8.3 us and 5.
//
// Expansion.  A code u in bits 0..3 (or 4..7) of a half is the fp16 subnormal u 2^-24 (u
// 2^-20), so (u - 8) * scale is one packed fma, u 2^-24 * S - 8 2^-24 * S, with S the scale
// times a power of two that puts it below 65504.  Two roundings to 11 bits: of S and of
// the result.
//   * Keys: the power of two is each position's own, by the largest of its groups (not
//     those whose codes are all 0: their stored scale says nothing), and comes back as a
//     factor of the position's logits; where the exponents of 32 positions lie within 2^6 they
//     share the largest.  An element below fp16's normal range is off by up to 2^-25, where
//     the largest of the position (of the 32) is 7 2^-9 or more: by 2^-18 of that.
//   * Values: the power of two is a group's, common to the positions that all rows see, and
//     follows the largest scale so far.  An element far below it is off by 2^-20 of that.
// Steps of 32 positions that touch the call's own tokens (the last ones) are different:
// masked weights, codes expanded exactly, the weight times the value's scale rounded after
// a power of two of each row and group, and sums as weighted means, so that what a row does not
// see has no part in its rounding either.
//
// Weights are fp16 up to 2^14 (a row's reference moves only when passed by 2^8): 11 bits
// down to 2^-20 of the largest, then to 2^-31 of it.
#include "cache4.hpp"
#include "cache4_line.hpp"
#include "common.hpp"
#include "gemm_tiles.hpp"
#include "launch_serving.hpp"

namespace dq {

namespace {

struct TreeArgs {
    AttnArgs a;
    const int32_t* mask;  // [tokens, words]
    int64_t words;
};

constexpr int kTiles = 1;  // tiles of 32 rows of a wave
using TreeCut = Cut<32 * kTiles, kThreads>;
constexpr uint32_t kTopBits = 0x7fe000u;  // mantissa of 65504, fp16's largest

__device__ __forceinline__ f16x2_t twice(float v)
{
    const _Float16 h = (_Float16)v;
    return (f16x2_t){h, h};
}
__device__ __forceinline__ f16x8_t operand(const uint32_t (&w)[4])
{
    return __builtin_bit_cast(f16x8_t, (u32x4_t){w[0], w[1], w[2], w[3]});
}
__device__ __forceinline__ uint32_t scaled(uint32_t codes, f16x2_t s, f16x2_t b)
{
    return u32_of(__builtin_elementwise_fma(f16x2_of(codes), s, b));
}

// max over the 32 lanes of a half of the wave
__device__ __forceinline__ uint32_t half_max(uint32_t u)
{
    float x, y;
    row_pair(__uint_as_float(row16_max(u)), false, x, y);
    return max(__float_as_uint(x), __float_as_uint(y));
}

// The 32 mask bits of positions from (bit `at` of the row's words) on; bits before 0 are 1.
__device__ __forceinline__ uint32_t mask_window(const int32_t* row, int64_t words, int at)
{
    if (at < 0) return (uint32_t)row[0] << -at | ((1u << -at) - 1);
    const int w = at >> 5, s = at & 31;
    uint32_t v = w < words ? (uint32_t)row[w] >> s : 0u;
    if (s != 0 && w + 1 < words) v |= (uint32_t)row[w + 1] << (32 - s);
    return v;
}

// A wave's ring of steps in LDS: the codes and scales of 32 positions, copied straight from memory
// (buffer loads to LDS), two tiles of 16 positions each.  Tiles of codes are rows of D / 16
// 16-byte pieces; piece j of row r lies at j ^ turn(r), which spreads what a pass of lanes reads over
// the banks (the copy's lanes pick their pieces accordingly).  Scales lie four groups of a position next
// to each other, keys' in order, values' the even ones first.
template <int D, int G>
struct Ring {
    static constexpr int kPieces = D / 32;               // of a row of codes (D / 2 bytes)
    static constexpr int kCodes = 16 * kPieces * 16;     // bytes of a tile's codes
    static constexpr int kCopies = (kCodes + 1023) / 1024;
    static constexpr int kQuads = (D / G + 3) / 4;       // groups by four
    static constexpr int kKeys = 0, kValues = 2 * kCodes, kKeyScales = 4 * kCodes;
    static constexpr int kValueScales = kKeyScales + 2 * kQuads * 256;
    static constexpr int kBytes = kValueScales + 2 * kQuads * 256;
    static constexpr int kLoads = 4 * kCopies + 4 * kQuads;  // of a step
    static __device__ __forceinline__ int turn(int r)
    {
        return D == 64 ? (r >> 2) & 1 : (D == 128 ? (r >> 1) & 3 : r & 7);
    }
};

// Waits until at most N of the wave's loads are in flight (and for no LDS operation).
template <int N>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
    asm volatile("" ::: "memory");
}

// Reads of the ring, by LDS address, each block with its own wait: reads that the compiler knew of
// would wait for every copy in flight, those of later steps among them.
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
template <int D, int kQuads>
__device__ __forceinline__ void read_keys(uint32_t k0, uint32_t k1, uint32_t ks, uint32_t vs, u32x4_t (&kw)[D == 256 ? 4 : 2],
                                          u32x4_t (&kscale)[kQuads], u32x2_t (&vscale)[kQuads])
{
    if constexpr (D == 64) {
        u32x2_t a, b;
        asm volatile(
            "ds_read_b64 %0, %4\n\tds_read_b64 %1, %5\n\tds_read_b128 %2, %6\n\tds_read_b64 %3, %7\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(a), "=&v"(b), "=&v"(kscale[0]), "=&v"(vscale[0])
            : "v"(k0), "v"(k1), "v"(ks), "v"(vs)
            : "memory");
        kw[0] = (u32x4_t){a.x, a.y, 0u, 0u};
        kw[1] = (u32x4_t){b.x, b.y, 0u, 0u};
    } else if constexpr (D == 128) {
        asm volatile(
            "ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\tds_read_b128 %2, %6\n\tds_read_b64 %3, %7\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(kw[0]), "=&v"(kw[1]), "=&v"(kscale[0]), "=&v"(vscale[0])
            : "v"(k0), "v"(k1), "v"(ks), "v"(vs)
            : "memory");
    } else {
        // pieces 2 h, 2 h + 1, 4 + 2 h, 5 + 2 h: a lane's are an exclusive or of 16 or 64 bytes away
        asm volatile(
            "ds_read_b128 %0, %6\n\tds_read_b128 %1, %7\n\tds_read_b128 %2, %8\n\tds_read_b128 %3, %9\n\t"
            "ds_read_b128 %4, %10\n\tds_read_b64 %5, %11\n\ts_waitcnt lgkmcnt(0)"
            : "=&v"(kw[0]), "=&v"(kw[1]), "=&v"(kw[2]), "=&v"(kw[3]), "=&v"(kscale[0]), "=&v"(vscale[0])
            : "v"(k0), "v"(k0 ^ 16u), "v"(k1), "v"(k1 ^ 16u), "v"(ks), "v"(vs)
            : "memory");
        if constexpr (kQuads == 2)
            asm volatile("ds_read_b128 %0, %2 offset:512\n\tds_read_b64 %1, %3 offset:512\n\ts_waitcnt lgkmcnt(0)"
                         : "=&v"(kscale[1]), "=&v"(vscale[1])
                         : "v"(ks), "v"(vs)
                         : "memory");
    }
}

// The value words of 16 positions: register 8 i + 4 q + j is row 8 q + 4 h + j of tile i; v[j] the address of
// row 4 h + j of tile 0.
template <int D>
__device__ __forceinline__ void read_values(const uint32_t (&v)[4], uint32_t (&w)[16][D == 256 ? 2 : 1])
{
    constexpr int kTile = Ring<D, D == 64 ? 64 : 128>::kCodes, kHalf = kTile / 2;
#define READ16(OP, W)                                                                                        \
    asm volatile(OP " %0, %16\n\t" OP " %1, %17\n\t" OP " %2, %18\n\t" OP " %3, %19\n\t" OP                   \
                    " %4, %16 offset:%20\n\t" OP " %5, %17 offset:%20\n\t" OP " %6, %18 offset:%20\n\t" OP   \
                    " %7, %19 offset:%20\n\t" OP " %8, %16 offset:%21\n\t" OP " %9, %17 offset:%21\n\t" OP   \
                    " %10, %18 offset:%21\n\t" OP " %11, %19 offset:%21\n\t" OP " %12, %16 offset:%22\n\t" OP \
                    " %13, %17 offset:%22\n\t" OP " %14, %18 offset:%22\n\t" OP " %15, %19 offset:%22\n\t"   \
                    "s_waitcnt lgkmcnt(0)"                                                                   \
                 : "=&v"(W[0]), "=&v"(W[1]), "=&v"(W[2]), "=&v"(W[3]), "=&v"(W[4]), "=&v"(W[5]),             \
                   "=&v"(W[6]), "=&v"(W[7]), "=&v"(W[8]), "=&v"(W[9]), "=&v"(W[10]), "=&v"(W[11]),           \
                   "=&v"(W[12]), "=&v"(W[13]), "=&v"(W[14]), "=&v"(W[15])                                    \
                 : "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3]), "n"(kHalf), "n"(kTile), "n"(kTile + kHalf)    \
                 : "memory")
    if constexpr (D == 256) {
        u32x2_t t[16];
        READ16("ds_read_b64", t);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            w[e][0] = t[e].x;
            w[e][1] = t[e].y;
        }
    } else {
        uint32_t t[16];
        if constexpr (D == 64)
            READ16("ds_read_u16", t);
        else
            READ16("ds_read_b32", t);
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e][0] = t[e];
    }
#undef READ16
}

template <int D, int G>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void cache4_tree_kernel(TreeArgs args)
{
    constexpr int T = kTiles;
    using C = TreeCut;
    using R = Ring<D, G>;
    constexpr int S = 2;  // steps of the ring
    constexpr int NC = D / 32;    // 32-dimension steps of a dot product, and tiles of the output
    constexpr int NG = D / G;     // groups of a head
    constexpr int NL = (NG + 1) / 2;               // value scales of a lane
    constexpr int VW = D / 128 > 0 ? D / 128 : 1;  // value words of a lane and position
    constexpr int kPieces = D / 8;                 // of a row of q in LDS
    constexpr int kCols = D == 64 ? 1 : 2;  // tiles of the output that the waves join at a time (in the ring)
    static_assert(kWaves * S * R::kBytes >= kWaves * kCols * 4096, "the ring holds them");
    __shared__ __attribute__((aligned(16))) char shared[C::kRows * D * 2];  // the rows of q
    __shared__ float logits[C::kRows];
    __shared__ __attribute__((aligned(16))) float kpow[kWaves][32];
    __shared__ __attribute__((aligned(16))) float vscale[kWaves][NG][32];  // (masked), or halves: scales, biases
    __shared__ float2 sums[kWaves][T][32];
    __shared__ __attribute__((aligned(128))) char ring[kWaves][S][R::kBytes];
    uint4* const qs = reinterpret_cast<uint4*>(shared);

    const AttnArgs& a = args.a;
    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r32 = lane & 31;
    const int h = lane >> 5;
    const int shift = a.c.page_shift;
    const int nibble = (lane >> 4) & 1 ? 0 : 4;  // shift that puts a lane's value codes in bits 4..7

    // byte offsets of a lane's piece in a tile of codes (the copy's lane i fills piece i, that of rows of
    // the next copy lie 1024 bytes on), and of its scale in those of a tile
    uint32_t code_lane, ks_lane[R::kQuads], vs_lane[R::kQuads];
    {
        const int r = lane / R::kPieces % 16, j = lane % R::kPieces;
        code_lane = r * (D / 2) + (j ^ R::turn(r)) * 16;
#pragma unroll
        for (int n = 0; n < R::kQuads; ++n) {
            const int i = lane & 3, kg = 4 * n + i, vg = 4 * n + (i & 1) * 2 + (i >> 1);
            ks_lane[n] = (uint32_t)(((kg < NG ? kg : NG - 1) << shift) + (lane >> 2)) * 4;
            vs_lane[n] = (uint32_t)(((vg < NG ? vg : NG - 1) << shift) + (lane >> 2)) * 4;
        }
    }
    // where a lane reads in a step of the ring
    uint32_t k_read[2], v_read[4], s_read;
    {
        const int t = lane & 15, tile = (lane >> 4) & 1;  // position r32: row t of a tile
        const uint32_t at = lds_address(reinterpret_cast<const uint4*>(ring[wave][0]));
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // words (2 i + h) NC on
            const int byte = (2 * i + h) * NC * 4;
            k_read[i] = at + R::kKeys + tile * R::kCodes + t * (D / 2) + ((byte >> 4) ^ R::turn(t)) * 16 + (byte & 15);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // the codes of the dimensions that are t modulo 16, of row 4 h + j
            const int r = 4 * h + j, byte = t * (D / 32);
            v_read[j] = at + R::kValues + r * (D / 2) + ((byte >> 4) ^ R::turn(r)) * 16 + (byte & 15);
        }
        s_read = at + R::kKeyScales + tile * 256 + t * 16;
    }

    // consecutive stretches (which may read the same keys) on one XCD
    const int group = (a.groups & 7) == 0 ? (int)(blockIdx.x & 7) * (a.groups >> 3) + (int)(blockIdx.x >> 3)
                                          : (int)blockIdx.x;
    const Line ln = lay_line<C, true>(a, group, 0);
    const int64_t x0 = uniform64(ln.first(group)), x1 = uniform64(ln.first(group + 1));
    int b = ln.b;
    int64_t before = uniform64(ln.before);
    if (b < 0) return;

    Rows rw = ln.rw;
    for (int64_t x = x0; x < x1;) {
        const int steps = steps_of(a, rw);
        const int64_t tiles = tiles_of<C>(rw);
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
        const int kvh = __builtin_amdgcn_readfirstlane((int)udiv(unit, tiles));
        const int64_t tile = unit - kvh * tiles;
        const int64_t r0 = tile * C::kRows;
        const int64_t rows = rw.rows();
        const int len = __builtin_amdgcn_readfirstlane(rw.held);
        const int context = __builtin_amdgcn_readfirstlane(rw.len - rw.nq);
        const bool nothing = rw.bad || rw.len > rw.held;  // all rows NaN
        const int begin = __builtin_amdgcn_readfirstlane(step0) * kStride;
        int stop = len;  // (a unit that is one step may have any length)
        if (take < steps - step0 && begin + take * kStride < len)
            stop = begin + __builtin_amdgcn_readfirstlane(take) * kStride;
        stop = __builtin_amdgcn_readfirstlane(stop);
        x += take;
        const int32_t* table = a.bt.table + __builtin_amdgcn_readfirstlane(b) * a.bt.width;
        // token row and query head of row r of the unit (of the first where there is none)
        const auto row_at = [&](int r, int64_t& token, int& head) {
            const int64_t row = r0 + r < rows ? r0 + r : 0;
            const int qi = (int)udiv(row, rw.per);
            token = rw.first + qi;
            head = kvh * rw.per + (int)(row - (int64_t)qi * rw.per);
        };

        // ---- a step's copies into the ring
        uint32_t bad_tiles = 0;  // two bits for each step in flight: a tile whose page is outside the cache
        // Page numbers of 32 of the wave's steps, a tile's in each lane (scalar loads would count with the LDS
        // operations, and a wait for those would wait for memory in every step).
        int pages = 0, pages_from = 0;
        const auto tile_at = [&](int t) { return t < stop ? t : (stop - 1) & ~15; };
        const auto load_pages = [&](int t0) __attribute__((always_inline)) {
            pages = table[tile_at(t0 + (lane >> 1) * kStride + (lane & 1) * 16) >> shift];
            pages_from = t0;
        };
        int t0 = begin + wave * kStep;
        if (t0 < stop) load_pages(t0);
        // the rows of q that the unit's threads have, asked for before the copies: loads come back in order
        constexpr int kPer = kThreads / C::kRows;  // threads of a row
        constexpr int kMine = kPieces / kPer;      // pieces of a thread
        uint4 qr[kMine];
        {
            int64_t token;
            int head;
            row_at(tid / kPer, token, head);
            const uint16_t* qp = a.q + token * a.q_stride + (int64_t)head * D + tid % kPer * kMine * 8;
#pragma unroll
            for (int i = 0; i < kMine; ++i) qr[i] = reinterpret_cast<const uint4*>(qp)[i];
        }
        const auto copy = [&](int t0, char* to, int ahead) __attribute__((always_inline)) {
            if (t0 - pages_from >= 32 * kStride) load_pages(t0);
            const int at = (t0 - pages_from) / kStride * 2;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int page = __builtin_amdgcn_readlane(pages, at + i);
                const bool ok = (unsigned)page < (unsigned)a.c.pages;
                bad_tiles |= (ok ? 0u : 1u) << (2 * ahead + i);
                const int64_t block = (int64_t)(ok ? page : 0) * a.c.heads + kvh;
                const int off = tile_at(t0 + 16 * i) & ((1 << shift) - 1);
                const BufRef kb{a.c.k_codes + ((block << shift) + off) * (D / 8), R::kCodes};
                const BufRef vb{a.c.v_codes + ((block << shift) + off) * (D / 8), R::kCodes};
                const int64_t sb = ((block * NG) << shift) + off;
                const uint32_t bytes = (((NG - 1) << shift) + 16) * 4;
                const BufRef ks{a.c.k_scales + sb, bytes}, vs{a.c.v_scales + sb, bytes};
                if (D != 64 || lane < 32) {  // (heads of 64: a tile is 32 pieces)
#pragma unroll
                    for (int n = 0; n < R::kCopies; ++n) {
                        buf_load_lds16(kb, to + R::kKeys + i * R::kCodes + n * 1024, code_lane, n * 1024);
                        buf_load_lds16(vb, to + R::kValues + i * R::kCodes + n * 1024, code_lane, n * 1024);
                    }
                }
#pragma unroll
                for (int n = 0; n < R::kQuads; ++n) {
                    buf_load_lds4(ks, to + R::kKeyScales + n * 512 + i * 256, ks_lane[n], 0);
                    buf_load_lds4(vs, to + R::kValueScales + n * 512 + i * 256, vs_lane[n], 0);
                }
            }
        };
        char* const mine = ring[wave][0];
        if (t0 < stop) {
            copy(t0, mine, 0);
            if (S > 2 && t0 + kStride < stop) copy(t0 + kStride, mine + R::kBytes, 1);
        }
        // what the step at hand has in registers
        u32x4_t kw[D == 256 ? 4 : 2];  // words (h NC + i), then ((2 + h) NC + i)
        uint32_t vw[16][VW];
        float ksl[NG], vsl[NL];
        constexpr int kHalf = D == 256 ? 2 : 1;  // of them
        int stage = 0;  // of the step at hand

        // ---- rows of q -> fp16 operands in LDS, each times a power of two (and the sign of the softmax's
        // scale, so that larger is always larger)
        {
            const int r = tid / kPer, sub = tid % kPer;
            uint32_t qmax = 0;
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const uint32_t u[4] = {qr[i].x, qr[i].y, qr[i].z, qr[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e)  // as integers: a NaN is the largest
                    qmax = max(qmax, max((u[e] << 16) & 0x7fffffffu, u[e] & 0x7fff0000u));
            }
#pragma unroll
            for (int o = 1; o < kPer; o <<= 1) qmax = max(qmax, (uint32_t)__shfl_xor((int)qmax, o, kWave));
            const int ue = min(14 - exponent(__uint_as_float(qmax)), 126);
            float up = a.scale_log2 < 0.0f ? -pow2(ue) : pow2(ue);
            float logit = fabsf(a.scale_log2) * pow2(-ue);
            if (logit == 0.0f) {  // logits of 0 (and no 0 * -inf where positions are hidden)
                up = 0.0f;
                logit = 1.0f;
            }
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const uint32_t u[4] = {qr[i].x, qr[i].y, qr[i].z, qr[i].w};
                float f[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[2 * e] = __uint_as_float(u[e] << 16) * up;
                    f[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u) * up;
                }
                uint32_t w[4];  // the order in which a word's codes come: 0 4 1 5 2 6 3 7
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = u32_of((f16x2_t){(_Float16)f[e], (_Float16)f[e + 4]});
                qs[r * kPieces + ((sub * kMine + i) ^ swizzle<kPieces>(r))] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            // (a key is its codes times 2^(9 + the position's exponent) less than it is)
            if (sub == 0) logits[r] = logit * 512.0f;
        }
        lds_barrier();

        // this lane's first operand: piece h of row r32 (its row is a multiple of 2 kPieces pieces
        // from the start, so piece 2 k + h is an exclusive or away)
        const uint32_t q_lane = (uint32_t)(r32 * kPieces + (h ^ swizzle<kPieces>(r32))) * 16;
        float logit[T], m[T], l[T];
        f32x16_t o[T][NC];
#pragma unroll
        for (int n = 0; n < T; ++n) {
            logit[n] = logits[32 * n + r32];
            m[n] = -INFINITY;
            l[n] = 0.0f;
#pragma unroll
            for (int j = 0; j < NC; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[n][j][e] = 0.0f;
        }
        // The scales of a group are measured in units of 2^(ve - 15) (and o in as many of 2^(5 + ve));
        // lanes of half h have ve for the groups 2 i + h, as vtop = 65504 2^(ve - 15), what fp16
        // then holds of them.  It is raised past the exponent of a scale that passes vtop.
        uint32_t vtop[NL];
#pragma unroll
        for (int i = 0; i < NL; ++i) vtop[i] = (16u << 23) + kTopBits;  // ve = -111
        const auto group_unit = [&](int g) {
            return pow2((int)(__builtin_amdgcn_readlane(vtop[g / 2], 32 * (g & 1)) >> 23) - 127);
        };

        const auto read_words = [&](uint32_t here) __attribute__((always_inline)) {
            const uint32_t at[4] = {v_read[0] + here, v_read[1] + here, v_read[2] + here, v_read[3] + here};
            read_values<D>(at, vw);
        };
        // Key scales of groups whose codes are all 0 become 0 (the words of a position lie in two lanes).
        const auto drop_zero_keys = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                uint32_t some = 0;
#pragma unroll
                for (int i = g * G / 32; i < (g + 1) * G / 32; ++i)
                    some |= (kw[i / 4][i % 4] ^ 0x88888888u) | (kw[kHalf + i / 4][i % 4] ^ 0x88888888u);
                some |= (uint32_t)__shfl_xor((int)some, 32, kWave);
                if (some == 0 && ksl[g] == ksl[g]) ksl[g] = 0.0f;
            }
        };
        // The same of values: 16 lanes have the codes of 16 positions (register r of half i: position
        // 16 (r >> 3) + 8 (r >> 2 & 1) + 4 i + (r & 3)).
        const auto drop_zero_values = [&](uint32_t here) __attribute__((always_inline)) {
            read_words(here);
            const int r = (r32 >> 4) * 8 + ((r32 >> 3) & 1) * 4 + (r32 & 3);  // where position r32 is
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                uint32_t none = 0;
                constexpr int n = G / 16;  // codes of the group in a lane
                const uint32_t mask = (n == 8 ? ~0u : (1u << (4 * (n & 7))) - 1u) << (4 * (g * n % 8));
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const uint64_t lanes = __ballot(((vw[e][g * n / 8] ^ 0x88888888u) & mask) == 0);
                    if (((lanes >> (32 * h)) & 0xffffu) == 0xffffu) none |= 1u << e;
                }
                const uint32_t z0 = __builtin_amdgcn_readlane(none, 0), z1 = __builtin_amdgcn_readlane(none, 32);
                const bool zero = (((r32 >> 2) & 1 ? z1 : z0) >> r & 1) != 0;
                if ((g & 1) == h && zero) vsl[g / 2] = 0.0f;
                if (NG == 1 && zero) vsl[0] = 0.0f;
            }
        };
        // A value scale that is not finite: NaN in its dimensions, in the rows that see it (vis[n]: the
        // positions that a lane's row of tile n sees), whatever their weight, and 0 from here on.
        const auto mark_nan = [&](const uint32_t (&vis)[T]) __attribute__((always_inline)) {
            uint64_t lanes[NL];  // bits 32 h + position: group 2 i + h
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const bool nan = !(fabsf(vsl[i]) < INFINITY);
                lanes[i] = __ballot(nan);
                if (nan) vsl[i] = 0.0f;
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const uint32_t at = (uint32_t)(lanes[g / 2] >> (32 * (g & 1)));
#pragma unroll
                for (int n = 0; n < T; ++n)
                    if ((at & vis[n]) != 0) {
#pragma unroll
                        for (int j = g * G / 32; j < (g + 1) * G / 32; ++j)
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[n][j][e] = __uint_as_float(0x7fc00000u);
                    }
            }
        };
        // The reference of each group follows the step's largest scales.
        const auto raise = [&]() __attribute__((always_inline)) {
            int down[NL];
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const uint32_t top = half_max(__float_as_uint(vsl[i]) & 0x7fffffffu), was = vtop[i] >> 23;
                const uint32_t now = top >= vtop[i] ? (top >> 23) + 1 : was;
                vtop[i] = (now << 23) + kTopBits;
                down[i] = (int)was - (int)now;
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const float f = pow2(__builtin_amdgcn_readlane(down[g / 2], 32 * (g & 1)));
#pragma unroll
                for (int n = 0; n < T; ++n)
#pragma unroll
                    for (int j = g * G / 32; j < (g + 1) * G / 32; ++j) o[n][j] *= f;
            }
        };
        // Value codes of tile j, positions of half i: an operand, times 2^-20 S + B.
        const auto value_operand = [&](int i, int j, const f16x2_t (&s)[4], const f16x2_t (&bias)[4])
                                       __attribute__((always_inline)) {
            constexpr uint32_t kBytes = 0x0c000c00u;
            const uint32_t sel = kBytes | (uint32_t)(4 + j % 4) << 16 | (uint32_t)(j % 4);
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[e] = scaled(__builtin_amdgcn_perm(vw[8 * i + 2 * e + 1][j / 4], vw[8 * i + 2 * e][j / 4], sel), s[e],
                              bias[e]);
            return operand(w);
        };

        const auto step = [&](auto Masked, int t0) __attribute__((always_inline)) {
            constexpr bool kMasked = decltype(Masked)::value;
            // the copies of a step to come go out, then those of this one are waited for
            const int free = stage == 0 ? S - 1 : stage - 1;
            if (t0 + (S - 1) * kStride < stop) {
                copy(t0 + (S - 1) * kStride, mine + free * R::kBytes, S - 1);
                wait_loads<(S - 1) * R::kLoads>();
            } else if (S > 2 && t0 + kStride < stop) {
                wait_loads<R::kLoads>();
            } else {
                wait_loads<0>();
            }
            const uint32_t here = stage * R::kBytes;
            stage = stage == S - 1 ? 0 : stage + 1;
            {
                u32x4_t ks[R::kQuads];
                u32x2_t vs[R::kQuads];
                read_keys<D, R::kQuads>(k_read[0] + here, k_read[1] + here, s_read + here,
                                        s_read + here + (R::kValueScales - R::kKeyScales) + 8 * h, kw, ks, vs);
                const uint32_t bad = (bad_tiles >> ((lane >> 4) & 1) & 1) ? 0x7fc00000u : 0u;
                bad_tiles >>= 2;
#pragma unroll
                for (int g = 0; g < NG; ++g) ksl[g] = __uint_as_float(ks[g / 4][g % 4] | bad);
#pragma unroll
                for (int i = 0; i < NL; ++i) vsl[i] = __uint_as_float(vs[i / 2][i % 2]);
            }
            uint32_t q_at = q_lane;
            pin(q_at);  // (its pieces' addresses are worked out as they are needed, not kept)
            uint32_t vis[T];
#pragma unroll
            for (int n = 0; n < T; ++n) {
                vis[n] = ~0u;
                if (kMasked) {
                    int64_t token;
                    int head;
                    row_at(32 * n + r32, token, head);
                    vis[n] = mask_window(args.mask + token * args.words, args.words, t0 - context);
                    if (len - t0 < 32) vis[n] &= (1u << (len - t0)) - 1;
                }
            }
            // scales
            bool unsure = false, larger = false;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                unsure |= __float_as_uint(ksl[g]) == kZeroScale;
            }
            if (__builtin_expect(__any(unsure), 0)) drop_zero_keys();
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                if (kMasked && t0 + r32 >= len) vsl[i] = 0.0f;
                larger |= !(fabsf(vsl[i]) < __uint_as_float(vtop[i]));
            }
            if (kMasked || __builtin_expect(__any(larger), 0)) {
                bool zero = false, nan = false;
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    zero |= __float_as_uint(vsl[i]) == kZeroScale;
                    nan |= !(fabsf(vsl[i]) < INFINITY);
                }
                if (__builtin_expect(__any(nan), 0)) mark_nan(vis);
                if (__builtin_expect(__any(zero), 0)) drop_zero_values(here);
                if (!kMasked) raise();
            }
            float top = 0.0f;
#pragma unroll
            for (int g = 0; g < NG; ++g) top = fmaxf(top, fabsf(ksl[g]));
            // the exponent that leaves the largest at most 65504 2^-15
            int ex = (int)((__float_as_uint(top) + 0x1fffu) >> 23) - 127;
            ex = ex < -104 ? -104 : (ex > 127 ? 127 : ex);
            // In steps that all rows see whole the 32 positions share the largest, if all are within 2^6 of it:
            // one factor of the logits in place of one each.
            bool each = true;
            float unit = 1.0f;
            if (!kMasked) {
                const int most = (int)__builtin_amdgcn_readfirstlane(half_max((uint32_t)(ex + 104))) - 104;
                each = __any(ex < most - 6);
                if (!each) {
                    ex = most;
                    unit = pow2(most);
                }
            }
            const float down = pow2(15 - ex);
            kpow[wave][r32] = pow2(ex);
            f16x2_t ks[NG], kh[NG], kb[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                ks[g] = twice(ksl[g] * down);
                kh[g] = ks[g] * (f16x2_t){(_Float16)0.0625f, (_Float16)0.0625f};
                kb[g] = ks[g] * (f16x2_t){(_Float16)-0x1p-21f, (_Float16)-0x1p-21f};
            }
            // (where position r32 is in the order of value_operand's halves)
            const int at = (r32 & 16) + ((r32 >> 2) & 1) * 8 + ((r32 >> 3) & 1) * 4 + (r32 & 3);
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int g = 2 * i + h;
                if (g < NG) {
                    if (kMasked) {
                        vscale[wave][g][r32] = vsl[i];
                    } else {  // times 2^(15 - ve)
                        _Float16* const to = reinterpret_cast<_Float16*>(vscale[wave][g]) + at;
                        const _Float16 v = (_Float16)(vsl[i] * __uint_as_float((269u << 23) + kTopBits - vtop[i]));
                        to[0] = v;
                        to[32] = v * (_Float16)-0x1p-17f;
                    }
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");  // other lanes read them
            __builtin_amdgcn_wave_barrier();

            // S^T = K Q^T
            f32x16_t s[T];
#pragma unroll
            for (int n = 0; n < T; ++n)
#pragma unroll
                for (int e = 0; e < 16; ++e) s[n][e] = 0.0f;
            // (a step's first operands of q are read ahead, each pair's next ones before its matrix
            // instructions: their latency is not waited for)
            f16x8_t qf[2][T];
            const auto read_q = [&](int k) __attribute__((always_inline)) {
#pragma unroll
                for (int n = 0; n < T; ++n)
                    qf[k & 1][n] =
                        *reinterpret_cast<const f16x8_t*>(shared + (q_at ^ (32 * k)) + 32 * n * kPieces * 16);
            };
            read_q(0);
            // (a wave at its matrix instructions comes first: the other wave of the SIMD has vector work to put
            // beside them.  24 x 24 tokens over 6000: 127 -> 123 us)
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int k = 0; k < 2 * NC; ++k) {
                const int i = k >> 1, g = 32 * i / G;
                if (k + 1 < 2 * NC) read_q(k + 1);
                __builtin_amdgcn_sched_barrier(0);
                // (pins: else all keys are expanded ahead of the matrix instructions, and spill)
                uint32_t w = kw[(k & 1) * kHalf + i / 4][i % 4];
                pin(w);
                const uint32_t y = w >> 8;
                const uint32_t c[4] = {scaled(w & 0x000f000fu, ks[g], kb[g]), scaled(w & 0x00f000f0u, kh[g], kb[g]),
                                       scaled(y & 0x000f000fu, ks[g], kb[g]), scaled(y & 0x00f000f0u, kh[g], kb[g])};
                const f16x8_t key = operand(c);
#pragma unroll
                for (int n = 0; n < T; ++n) {
                    s[n] = __builtin_amdgcn_mfma_f32_32x32x16_f16(key, qf[k & 1][n], s[n], 0, 0, 0);
                    pin(s[n]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_setprio(0);
            read_words(here);  // (their latency runs beside the matrix instructions')

            // weights
            f16x8_t p[T][2];
            float carry[T], inv[T];  // masked steps: what is left of the mean so far, 1 / the new sum
#pragma unroll
            for (int n = 0; n < T; ++n) {
                float mx = -INFINITY;
                if (each) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f32x4_t kf = *reinterpret_cast<const f32x4_t*>(&kpow[wave][8 * i + 4 * h]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[n][4 * i + e] *= kf[e];
                    }
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    if (kMasked && !(vis[n] >> (8 * (e >> 2) + 4 * h + (e & 3)) & 1)) s[n][e] = -INFINITY;
                    mx = fmaxf(mx, s[n][e]);
                }
                float y0, y1;
                row_pair(mx, true, y0, y1);
                mx = fmaxf(y0, y1) * (logit[n] * unit);
                float alpha = 1.0f;
                if (__any(mx > m[n] + 8.0f)) {
                    const float mn = mx > m[n] + 8.0f ? mx : m[n];
                    alpha = mn == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m[n] - mn);
                    m[n] = mn;
                    if (!kMasked) {
                        l[n] *= alpha;
#pragma unroll
                        for (int j = 0; j < NC; ++j) o[n][j] *= alpha;
                    }
                }
                // weights up to 2^14: fp16's normal range then reaches 2^-20 of the largest
                // (masked steps, whose weights meet fp32 scales first, 2^-14 of that)
                const float base = m[n] == -INFINITY ? 0.0f : m[n] - (kMasked ? -8.0f : 6.0f);
#pragma unroll
                for (int e = 0; e < 16; ++e) s[n][e] = __builtin_amdgcn_exp2f(fmaf(s[n][e], logit[n] * unit, -base));
                if constexpr (kMasked) {
                    float sum = 0.0f;
#pragma unroll
                    for (int e = 0; e < 16; ++e) sum += s[n][e];
                    row_pair(sum, true, y0, y1);
                    const float old = l[n] * alpha;
                    l[n] = fmaf(y0 + y1, 0x1p14f, old);
                    inv[n] = l[n] > 0.0f ? 1.0f / l[n] : l[n];  // (0 and NaN stay)
                    carry[n] = l[n] == 0.0f ? 1.0f : old * inv[n];
                } else {
                    // (the sum of the weights as they are rounded, two at a time)
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const f16x2_t w = {(_Float16)s[n][e], (_Float16)s[n][e + 1]};
                        l[n] = __builtin_amdgcn_fdot2(w, (f16x2_t){(_Float16)1.0f, (_Float16)1.0f}, l[n], false);
                        p[n][e >> 3][e & 7] = w.x;
                        p[n][e >> 3][(e & 7) + 1] = w.y;
                    }
                }
            }
            // O^T = V^T P^T
#pragma unroll
            for (int e = 0; e < 16; ++e)
#pragma unroll
                for (int w = 0; w < VW; ++w) vw[e][w] = (vw[e][w] << nibble) & 0xf0f0f0f0u;
            if constexpr (!kMasked) {
                // scales and biases of half i of group g, read a pair ahead
                uint4 sv[2], bv[2];
                const auto read_scales = [&](int k) __attribute__((always_inline)) {
                    const float* at = &vscale[wave][k >> 1][8 * (k & 1) + 4 * h];
                    sv[k & 1] = *reinterpret_cast<const uint4*>(at);
                    bv[k & 1] = *reinterpret_cast<const uint4*>(at + 16);
                };
                read_scales(0);
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int k = 0; k < 2 * NG; ++k) {
                    const int g = k >> 1, i = k & 1;
                    if (k + 1 < 2 * NG) read_scales(k + 1);
                    __builtin_amdgcn_sched_barrier(0);
                    const f16x2_t sc[4] = {f16x2_of(sv[i].x), f16x2_of(sv[i].y), f16x2_of(sv[i].z), f16x2_of(sv[i].w)};
                    const f16x2_t bias[4] = {f16x2_of(bv[i].x), f16x2_of(bv[i].y), f16x2_of(bv[i].z),
                                             f16x2_of(bv[i].w)};
#pragma unroll
                    for (int j = g * G / 32; j < (g + 1) * G / 32; ++j) {
                        const f16x8_t v = value_operand(i, j, sc, bias);
#pragma unroll
                        for (int n = 0; n < T; ++n)
                            o[n][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, p[n][i], o[n][j], 0, 0, 0);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
                __builtin_amdgcn_s_setprio(0);
            } else {
                const f16x2_t one = twice(0x1p15f), eight = twice(-0x1p-2f);  // (u - 8) 2^-5
                const f16x2_t sc[4] = {one, one, one, one}, bias[4] = {eight, eight, eight, eight};
#pragma unroll
                for (int n = 0; n < T; ++n) {
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        __builtin_amdgcn_sched_barrier(0);  // a group at a time, its codes expanded again for
#pragma unroll                                              // each tile of rows
                        for (int e = 0; e < 16; ++e)
#pragma unroll
                            for (int w = 0; w < VW; ++w) pin(vw[e][w]);
                        float t[16], high = 0.0f;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const f32x4_t v = *reinterpret_cast<const f32x4_t*>(&vscale[wave][g][8 * i + 4 * h]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                t[4 * i + e] = s[n][4 * i + e] * v[e];
                                high = fmaxf(high, fabsf(t[4 * i + e]));
                            }
                        }
                        float y0, y1;
                        row_pair(high, true, y0, y1);
                        const int tx = max(exponent(fmaxf(y0, y1)), -112);
                        const float up = pow2(14 - tx), back = pow2(tx) * (inv[n] * 32.0f);
                        f16x8_t pf[2];
#pragma unroll
                        for (int e = 0; e < 16; ++e) pf[e >> 3][e & 7] = (_Float16)(t[e] * up);
#pragma unroll
                        for (int j = g * G / 32; j < (g + 1) * G / 32; ++j) {
                            f32x16_t z;
#pragma unroll
                            for (int e = 0; e < 16; ++e) z[e] = 0.0f;
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                z = __builtin_amdgcn_mfma_f32_32x32x16_f16(value_operand(i, j, sc, bias), pf[i], z, 0,
                                                                           0, 0);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[n][j][e] = fmaf(z[e], back, o[n][j][e] * carry[n]);
                        }
                    }
                }
            }
        };
        // from sums of weights and values in units of the groups to means
        const auto to_means = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int n = 0; n < T; ++n) {
                float y0, y1;
                row_pair(l[n], true, y0, y1);
                l[n] = y0 + y1;
                const float inv = l[n] > 0.0f ? 1.0f / l[n] : l[n];  // (0 and NaN stay)
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float unit = group_unit(g);
#pragma unroll
                    for (int j = g * G / 32; j < (g + 1) * G / 32; ++j) o[n][j] = o[n][j] * (inv * 32.0f) * unit;
                }
            }
        };

        if (t0 < stop && t0 + kStep <= context) {
            do {
                step(std::false_type{}, t0);
                t0 += kStride;
            } while (t0 < stop && t0 + kStep <= context);
            to_means();
        }
        for (; t0 < stop; t0 += kStride) step(std::true_type{}, t0);

        // Join the waves, kCols tiles of the output at a time: each wave takes the rows of four dimensions in
        // 16 from all of them.
        f32x4_t* const join = reinterpret_cast<f32x4_t*>(ring[0][0]);
        if (h == 0) {
#pragma unroll
            for (int n = 0; n < T; ++n) sums[wave][n][r32] = make_float2(m[n], l[n]);
        }
        lds_barrier();  // q and the ring are read no more
#pragma unroll
        for (int n = 0; n < T; ++n) {
            float top = -INFINITY, tot = 0.0f, f[kWaves];
#pragma unroll
            for (int w = 0; w < kWaves; ++w) top = fmaxf(top, sums[w][n][r32].x);
            const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float2 ml = sums[w][n][r32];
                f[w] = ml.y * __builtin_amdgcn_exp2f(ml.x - base);
                tot += f[w];
            }
            const float inv = nothing ? __uint_as_float(0x7fc00000u) : (tot == 0.0f ? 0.0f : 1.0f / tot);
#pragma unroll
            for (int w = 0; w < kWaves; ++w) f[w] *= inv;
            int64_t token;
            int head;
            row_at(32 * n + r32, token, head);
            const bool live = r0 + 32 * n + r32 < rows;
            const int64_t at = ((int64_t)group * 2 + slot) * C::kRows + 32 * n + r32;
            if (!whole && live && wave == 0 && h == 0) a.part_ml[at] = make_float2(top, tot);
            const int64_t place = (whole ? token * a.q_heads + head : at) * D + 8 * wave + 4 * h;
#pragma unroll
            for (int j0 = 0; j0 < NC; j0 += kCols) {
#pragma unroll
                for (int j = 0; j < kCols; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        join[((wave * kCols + j) * 4 + e) * kWave + lane] =
                            (f32x4_t){o[n][j0 + j][4 * e], o[n][j0 + j][4 * e + 1], o[n][j0 + j][4 * e + 2],
                                      o[n][j0 + j][4 * e + 3]};
                lds_barrier();
#pragma unroll
                for (int j = 0; j < kCols; ++j) {
                    f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int w = 0; w < kWaves; ++w) {
                        const f32x4_t x = join[((w * kCols + j) * 4 + wave) * kWave + lane];
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = fmaf(x[e], f[w], v[e]);
                    }
                    if (!live) continue;
                    if (whole)
                        *reinterpret_cast<uint2*>(a.out + place + 32 * (j0 + j)) =
                            make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
                    else
                        *reinterpret_cast<f32x4_t*>(a.part + place + 32 * (j0 + j)) = v;
                }
                lds_barrier();
            }
        }
    }
}

// The launch's shape; a step is 128 positions, a stretch what one workgroup takes of the line.
struct TreePlan {
    int64_t rows, units, groups;
    int step_shift;  // 31: a unit is one step, and nothing is joined
    size_t part_bytes, ml_bytes;
};
constexpr int64_t kMaxUnits = 1LL << 23;
// The choices, in us, 32 query / 8 kv heads of 128, g = 32, sequences x tokens over positions:
//
// Units that are cut into stretches need a second launch, and memory for the parts; whole ones leave CUs idle
// at the end.
//     whole, 512 stretches:  16 x 16 over 1000 20, 46;  64 x 8 over 1500 35, 52;  4 x 32 over 2000 30, 35;
//                            1 x 64 over 2000 29, 26 (256: 23);  8 x 64 over 3000 59, 55;
//                            8 x 8 over 4000 50, 31;  32 x 8 over 4000 56, 67;  32 x 8 over 8000 101, 92;
//                            12 x 60 over 2500 (40 heads) 90, 71;  24 x 24 over 6000 (40 heads) 145, 125
// so whole up to 16 steps if there are more units than run at a time, up to 4 always, and between them where a
// quarter of the workgroups have a unit and stretches would save no more than 16 steps.
constexpr int64_t kWholeSteps = 16;

TreePlan plan_of(const Cache4& c, int64_t count, int64_t tokens, int q_heads, int64_t max_q, int64_t max_len)
{
    const int64_t fill = c.dim == 256 ? 256 : 512;  // workgroups that run at a time (registers: 512 a lane, or 256)
    TreePlan p{};
    if (max_q > tokens) max_q = tokens;
    if (max_len > 0x7fffffffLL) max_len = 0x7fffffffLL;
    p.rows = max_q * (q_heads / c.heads);
    const int64_t heads = count * c.heads, steps = ceil_div(max_len, kStride);
    const int64_t tiles = ceil_div(p.rows, TreeCut::kRows);
    p.units = tiles > kMaxUnits / heads ? kMaxUnits : heads * tiles;
    const int64_t total = p.units * steps;  // (below 2^48)
    const bool whole = p.units > fill ? steps <= kWholeSteps
                                      : steps <= 4 || (4 * p.units >= fill && steps - total / fill <= kWholeSteps);
    if (whole) {
        p.groups = p.units < 4 * fill ? p.units : 4 * fill;
        p.step_shift = 31;
        return p;
    }
    p.step_shift = 7;
    p.groups = total / 4 < fill ? total / 4 : fill;  // (a stretch of fewer than 4 steps is mostly its ends)
    if (p.groups < 256) p.groups = total < 256 ? total : 256;
    p.part_bytes = (size_t)p.groups * 2 * TreeCut::kRows * c.dim * sizeof(float);
    p.ml_bytes = (size_t)p.groups * 2 * TreeCut::kRows * sizeof(float2);
    return p;
}

template <int D, int G>
hipError_t launch_dg(const TreeArgs& t, const TreePlan& p, hipStream_t stream)
{
    const AttnArgs& a = t.a;
    cache4_tree_kernel<D, G><<<(unsigned)a.groups, kThreads, 0, stream>>>(t);
    if (a.groups > 1 && a.step_shift < 31) {
        if (p.units * 2 > a.groups) {
            cache4_join_edges_kernel<D, TreeCut>
                <<<dim3((unsigned)a.groups - 1, TreeCut::kRows / 16), kThreads, 0, stream>>>(a);
        } else {
            const dim3 grid((unsigned)p.rows, (unsigned)a.c.heads, (unsigned)a.bt.count);
            cache4_join_kernel<D, TreeCut><<<grid, kThreads, 0, stream>>>(a);
        }
    }
    return hipGetLastError();
}

}  // namespace

size_t cache4_tree_workspace(const Cache4& c, int64_t count, int64_t tokens, int q_heads, int64_t max_q,
                             int64_t max_len)
{
    const TreePlan p = plan_of(c, count, tokens, q_heads, max_q, max_len);
    return p.part_bytes + p.ml_bytes;
}

hipError_t launch_cache4_tree(const Cache4& c, const Cache4Batch& bt, const uint16_t* q, int64_t tokens,
                              int64_t q_stride, int q_heads, const int32_t* mask, int64_t words,
                              float scale, int64_t max_q, int64_t max_len, uint16_t* out,
                              void* workspace, hipStream_t stream)
{
    const TreePlan p = plan_of(c, bt.count, tokens, q_heads, max_q, max_len);
    const TreeArgs t{{c, bt, q, q_stride, out, tokens, q_heads, scale * kLog2e,
                      static_cast<float*>(workspace),
                      reinterpret_cast<float2*>(static_cast<char*>(workspace) + p.part_bytes),
                      (int32_t)p.groups, p.step_shift},
                     mask, words};
    switch (c.dim * 1000 + c.group) {
    case 64032: return launch_dg<64, 32>(t, p, stream);
    case 64064: return launch_dg<64, 64>(t, p, stream);
    case 128032: return launch_dg<128, 32>(t, p, stream);
    case 128064: return launch_dg<128, 64>(t, p, stream);
    case 128128: return launch_dg<128, 128>(t, p, stream);
    case 256032: return launch_dg<256, 32>(t, p, stream);
    case 256064: return launch_dg<256, 64>(t, p, stream);
    case 256128: return launch_dg<256, 128>(t, p, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace dq

// Integer products of int8 activations (tokens.hip) and packed b-bit weights,
// 2 <= b <= 8:
//   y[m,n] = sx[m] * sw[n] * sum_k xq[m,k] (u[n,k] - z[n]),
// u the stored codes, z = 2^(b-1) (symmetric) or the row's zero point.  The sum
// is exact: with c = 128 for b = 8 (u xor 0x80 is u - 128 as a signed byte) and
// c = 0 below (u < 128 is a signed byte as it is), the matrix cores add
// xq * (u - c) in int32, and (z - c) * sum_k xq comes off in the epilogue.
// |xq| <= 128, |u - z| <= 255 and K <= 65536 keep every sum inside int32.
// Three roundings follow: the sum to fp32, times sx, times sw (and one more to
// bf16 when y is bf16).
//
// Every token row of codes is padded with zeros to a multiple of 128 bytes, so K
// needs no tail: whatever a weight load past a row's codes brings (the next
// row's, or the buffer's zeros past the last) meets a zero.
#include "common.hpp"
#include "gemm_tiles.hpp"
#include "i8_tiles.hpp"
#include "launch_serving.hpp"

namespace dq {

namespace {

struct I8Args {
    const int8_t* x;  // [M, pitch]
    const float* x_scales;
    const int32_t* x_sums;
    int64_t M;
    int64_t pitch;
    const uint32_t* packed;
    const float* scales;
    const int32_t* zeros;
    int64_t N;
    int64_t row_words;
    void* y;
    bool bf16;
};

// ---------------------------------------------------------------------------
// Few tokens (M <= 64): bound by the packed weights.  A workgroup of four waves
// has 16 R weight rows, all tokens (16 T, the last ones again past M) and all
// of K: wave w takes the steps w, w + 4, ... of 256 codes, and the four sums
// are added through LDS.  v_mfma_i32_16x16x64_i8 with the weights as its rows:
// lane (r, g) holds, of weight row r, the chunks 2 g and 2 g + 1 of the step,
// 2 B consecutive words, so codes go from memory to registers to the matrix
// cores, a row's 256 codes with four lanes' neighbouring loads.  The tokens'
// bytes of the same codes come from L1 / L2 likewise.  A step's loads are in
// flight while the step before is multiplied.
//
// Rows per workgroup: the more, the less often the tokens' bytes are read and
// the fewer rows are open at once, as long as every CU has a workgroup.  16 x
// 28672 x 8192 at b = 6: 112 rows (256 workgroups) 39.5 us (4.5 TB/s of
// weights), 64 rows 45.8, 32 rows 53.9, 16 rows 56; 1 x 4096 x 4096 at b = 4:
// 16 rows (256 workgroups) 4.1 us, 32 rows 5.3, 64 rows 7.7.
constexpr int kFewThreads = 256;
constexpr int kFewWaves = kFewThreads / kWave;

template <int B, int R, int T>
__global__ __launch_bounds__(kFewThreads, R >= 7 || T == 4 ? 1 : (R == 1 ? 4 : 2)) void few_i8_kernel(I8Args a)
{
    __shared__ __attribute__((aligned(16))) int32_t part[kFewWaves][R * T * 4 * kWave];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane & 15;
    const int g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * R);
    const int64_t nrows = a.N - n0 < 16 * R ? a.N - n0 : 16 * R;
    const int steps = (int)((a.pitch + 255) >> 8);

    const uint32_t row_bytes = (uint32_t)a.row_words * 4;
    const BufRef wbuf = uniform_buf(a.packed + n0 * a.row_words, (uint32_t)nrows * row_bytes);
    const uint32_t xbytes = (uint32_t)(a.M * a.pitch);
    const BufRef xbuf = uniform_buf(a.x, xbytes);
    uint32_t woff[R], xoff[T];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int row = 16 * i + r < nrows ? 16 * i + r : (int)nrows - 1;
        woff[i] = row * row_bytes + g * (8 * B);
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const int64_t m = 16 * t + r < a.M ? 16 * t + r : a.M - 1;
        xoff[t] = (uint32_t)(m * a.pitch) + g * 64;
    }

    i32x4_t acc[R][T];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int t = 0; t < T; ++t) acc[i][t] = (i32x4_t){0, 0, 0, 0};

    uint32_t w[R][2 * B];
    u32x4v_t x[2][T][4];
    auto load_w = [&](int i, int s) __attribute__((always_inline)) {
        // a step past the last is past the buffer: nothing is fetched
        buf_load_words<2 * B>(wbuf, s < steps ? woff[i] + (uint32_t)s * (32 * B) : 0xfffff000u, 0, w[i]);
    };
    auto load_x = [&](auto S, int s) __attribute__((always_inline)) {
        constexpr int st = decltype(S)::value;
        // likewise, and the second half of a last half step; such bytes read as 0
        const bool in = 256 * s + 64 * g < a.pitch;
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const uint32_t off = in ? xoff[t] + 256 * (uint32_t)s : 0xffffff00u;
#pragma unroll
            for (int q = 0; q < 4; ++q) x[st][t][q] = buf_load_b128(xbuf, off + 16 * q, 0);
        }
    };
    // the tokens' bytes of a wave's next step are loaded at the top, a row tile's
    // codes as soon as its words are expanded
    auto step = [&](auto S, int s) __attribute__((always_inline)) {
        constexpr int st = decltype(S)::value;
        load_x(std::integral_constant<int, st ^ 1>{}, s + kFewWaves);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            i32x4_t codes[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                codes[q] = expand16<B>(reinterpret_cast<const uint32_t(&)[B]>(w[i][(q >> 1) * B]), q & 1);
            load_w(i, s + kFewWaves);
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int t = 0; t < T; ++t)
                    acc[i][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                        codes[q], __builtin_bit_cast(i32x4_t, x[st][t][q]), acc[i][t], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    load_x(std::integral_constant<int, 0>{}, wave);
#pragma unroll
    for (int i = 0; i < R; ++i) load_w(i, wave);
    for (int s = wave; s < steps; s += 2 * kFewWaves) {
        step(std::integral_constant<int, 0>{}, s);
        step(std::integral_constant<int, 1>{}, s + kFewWaves);
    }

    // lane (m = lane & 15, g) holds rows 4 g + e of tile i for token 16 t + m
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int t = 0; t < T; ++t)
            *reinterpret_cast<i32x4_t*>(&part[wave][((i * T + t) * kWave + lane) * 4]) = acc[i][t];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < R * T; ++j) {
        const int o = j * kFewThreads + threadIdx.x;
        int32_t sum = part[0][o];
#pragma unroll
        for (int v = 1; v < kFewWaves; ++v) sum += part[v][o];
        const int tl = o / (4 * kWave), l = (o >> 2) & (kWave - 1);
        const int64_t m = 16 * (tl % T) + (l & 15);
        const int64_t n = n0 + 16 * (tl / T) + 4 * (l >> 4) + (o & 3);
        if (m < a.M && n < a.N) {
            const float v = finish_i8(sum, code_shift<B>(a.zeros, n), a.x_sums[m], a.x_scales[m], a.scales[n]);
            if (a.bf16)
                store_y<true>(a.y, m * a.N + n, v);
            else
                store_y<false>(a.y, m * a.N + n, v);
        }
    }
}

template <int B, int R, int T>
hipError_t launch_few(const I8Args& a, hipStream_t stream)
{
    few_i8_kernel<B, R, T><<<dim3((unsigned)ceil_div(a.N, 16 * R)), kFewThreads, 0, stream>>>(a);
    return hipGetLastError();
}

// The most rows per workgroup that leave 224 workgroups or more for the 256 CUs.
template <int B, int T>
hipError_t launch_few_rows(const I8Args& a, hipStream_t stream)
{
    constexpr int64_t kFill = 224;
    if (a.N >= 16 * 7 * kFill) return launch_few<B, 7, T>(a, stream);
    if (a.N >= 16 * 4 * kFill) return launch_few<B, 4, T>(a, stream);
    if (a.N >= 16 * 2 * kFill) return launch_few<B, 2, T>(a, stream);
    return launch_few<B, 1, T>(a, stream);
}

// ---------------------------------------------------------------------------
// Many tokens: bound by the matrix cores.  Four waves side by side along N;
// wave w owns all 32 MT token rows and columns [32 NT w, 32 NT (w + 1)) of the
// workgroup's tile, as MT x NT tiles of v_mfma_i32_32x32x32_i8.  No two waves
// expand the same codes.
//
// A step is 128 codes: substep t (0 .. 3) multiplies, for lane half h, the bytes
// 64 h + 16 t .. + 15 of it, so a lane takes its weight operands from the chunks
// 2 h and 2 h + 1 of its row (2 B consecutive words), straight from memory
// into registers, and its token operands from 16-byte piece 4 h + t of its row
// in LDS.  Tokens go from memory to LDS directly, in three stages of a step,
// piece p of row r at slot p ^ ((r >> 1) & 7), which spreads a read over the
// banks; codes have three register stages.  Each substep's MFMAs run beside the
// expansion and the LDS reads of the next.  Per step a wave waits for its own
// copies of the next step's tokens (an exact count of later loads may remain in
// flight), and one barrier makes that stage visible.
template <int MT, int NT>
struct ManyTile {
    static constexpr int BM = 32 * MT;
    static constexpr int BN = 128 * NT;
    static constexpr int kStages = 3;
    static constexpr int kCopies = BM / 32;  // 16-byte pieces per thread and step
};

__device__ __forceinline__ int piece_slot(int row) { return (row >> 1) & 7; }

template <int B, int MT, int NT, int kOcc>
__global__ __launch_bounds__(256, kOcc) void many_i8_kernel(I8Args a)
{
    using Tl = ManyTile<MT, NT>;
    constexpr int kStages = Tl::kStages, kCopies = Tl::kCopies;
    __shared__ __attribute__((aligned(16))) uint4 As[kStages][Tl::BM * 8];

    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int c = lane & 31;
    const int h = lane >> 5;

    // consecutive workgroups go round robin to the 8 XCDs; each XCD gets a
    // contiguous range of tiles, groups of 4 row tiles by all column tiles
    const int64_t ntm = ceil_div(a.M, Tl::BM);
    const int64_t ntn = ceil_div(a.N, Tl::BN);
    const int64_t tiles = ntm * ntn;
    int64_t L = blockIdx.x;
    if ((tiles & 7) == 0) L = (L & 7) * (tiles >> 3) + (L >> 3);
    const int64_t gm = (ntm & 3) == 0 ? 4 : ntm;
    const int64_t grp = L / (gm * ntn), rem = L % (gm * ntn);
    const int64_t m0 = (grp * gm + rem % gm) * Tl::BM;
    const int64_t n0 = (rem / gm) * Tl::BN;
    const int nk = (int)(a.pitch >> 7);

    const int64_t mrows = a.M - m0 < Tl::BM ? a.M - m0 : Tl::BM;
    const BufRef xbuf = uniform_buf(a.x + m0 * a.pitch, (uint32_t)(mrows * a.pitch));
    uint32_t xoff[kCopies];
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
        const int slot = (wave * kCopies + i) * 64 + lane;
        const int row = slot >> 3;
        const int p = (slot & 7) ^ piece_slot(row);
        xoff[i] = (uint32_t)((row < mrows ? row : mrows - 1) * a.pitch + 16 * p);
    }
    const int64_t nrows = a.N - n0 < Tl::BN ? a.N - n0 : Tl::BN;
    const BufRef wbuf = uniform_buf(a.packed + n0 * a.row_words, (uint32_t)(nrows * a.row_words * 4));
    uint32_t woff[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int64_t nl = wave * 32 * NT + j * 32 + c;
        woff[j] = (uint32_t)((nl < nrows ? nl : nrows - 1) * a.row_words * 4 + h * (8 * B));
    }
    int abase[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) abase[t] = c * 8 + ((4 * h + t) ^ piece_slot(c));

    i32x16_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

    uint32_t w[kStages][NT][2 * B];
    i32x4_t bq[NT];     // weight operands of the current substep
    i32x4_t aq[2][MT];  // token operands of the current and the next substep
    auto load_x = [&](auto S, int ks) __attribute__((always_inline)) {
        constexpr int st = decltype(S)::value;
#pragma unroll
        for (int i = 0; i < kCopies; ++i)
            buf_load_lds16(xbuf, &As[st][(wave * kCopies + i) * 64], xoff[i], (uint32_t)ks * 128);
    };
    auto load_w = [&](auto S, int ks) __attribute__((always_inline)) {
        constexpr int st = decltype(S)::value;
#pragma unroll
        for (int j = 0; j < NT; ++j) buf_load_words<2 * B>(wbuf, woff[j], (uint32_t)ks * (16 * B), w[st][j]);
    };
    auto codes = [&](auto S, int j, int t) __attribute__((always_inline)) {
        constexpr int st = decltype(S)::value;
        return expand16<B>(reinterpret_cast<const uint32_t(&)[B]>(w[st][j][(t >> 1) * B]), t & 1);
    };
    auto read_a = [&](auto S, int t, i32x4_t (&dst)[MT]) __attribute__((always_inline)) {
        constexpr int st = decltype(S)::value;
#pragma unroll
        for (int i = 0; i < MT; ++i) dst[i] = __builtin_bit_cast(i32x4_t, As[st][abase[t] + 256 * i]);
    };
    // vector-memory operations issued after the copy of step ks + 1 when step ks
    // waits for it: the codes of step ks + 2
    constexpr int kWLoads = NT * ((2 * B) / 4 + ((2 * B) % 4 != 0 ? 1 : 0));
    constexpr int kWaitX = (kWLoads & 15) | ((kWLoads >> 4) << 14) | (7 << 4) | (15 << 8);
    constexpr int kPro = kCopies + 2 * kWLoads;  // after the copy of step 0 in the prologue
    constexpr int kWaitPro = (kPro & 15) | ((kPro >> 4) << 14) | (7 << 4) | (15 << 8);
    static_assert(kPro < 64, "vmcnt holds at most 63");

    auto step = [&](auto S, int ks) __attribute__((always_inline)) {
        constexpr int st = decltype(S)::value;
        constexpr int s1 = (st + 1) % kStages, s2 = (st + 2) % kStages;
        const int k2 = ks + 2 < nk ? ks + 2 : nk - 1;  // past the end: in bounds, never used
        load_w(std::integral_constant<int, s2>{}, k2);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            i32x4_t nb[NT];
            if (t < 3)
                read_a(S, t + 1, aq[(t + 1) & 1]);
            else
                read_a(std::integral_constant<int, s1>{}, 0, aq[0]);
#pragma unroll
            for (int j = 0; j < NT; ++j)
                nb[j] = t < 3 ? codes(S, j, t + 1) : codes(std::integral_constant<int, s1>{}, j, 0);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(aq[t & 1][i], bq[j], acc[i][j], 0, 0, 0);
#pragma unroll
            for (int j = 0; j < NT; ++j) bq[j] = nb[j];
            // an MFMA covers a share of the next substep's reads and expansion
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
#pragma unroll
                for (int j = 1; j < NT; ++j) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            if (t == 2) {
                __builtin_amdgcn_s_waitcnt(kWaitX);
                __syncthreads();  // stage ks + 1 is whole; stage ks + 2 is read by no wave any more
                load_x(std::integral_constant<int, s2>{}, k2);
            }
        }
    };

    load_x(std::integral_constant<int, 0>{}, 0);
    load_x(std::integral_constant<int, 1>{}, nk > 1 ? 1 : 0);
    load_w(std::integral_constant<int, 0>{}, 0);
    load_w(std::integral_constant<int, 1>{}, nk > 1 ? 1 : 0);
    __builtin_amdgcn_s_waitcnt(kWaitPro);
    __syncthreads();
    read_a(std::integral_constant<int, 0>{}, 0, aq[0]);
#pragma unroll
    for (int j = 0; j < NT; ++j) bq[j] = codes(std::integral_constant<int, 0>{}, j, 0);
    int ks = 0;
    for (; ks + kStages <= nk; ks += kStages) {
        step(std::integral_constant<int, 0>{}, ks);
        step(std::integral_constant<int, 1>{}, ks + 1);
        step(std::integral_constant<int, 2>{}, ks + 2);
    }
    if (ks < nk) step(std::integral_constant<int, 0>{}, ks);
    if (ks + 1 < nk) step(std::integral_constant<int, 1>{}, ks + 1);

    // the last copies into LDS have landed in every wave before the stages
    // serve for the tokens' scales and sums
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    float* const sx = reinterpret_cast<float*>(&As[0][0]);
    int32_t* const ssum = reinterpret_cast<int32_t*>(sx + Tl::BM);
    if (tid < Tl::BM) {
        const int64_t m = m0 + tid < a.M ? m0 + tid : a.M - 1;
        sx[tid] = a.x_scales[m];
        ssum[tid] = a.x_sums[m];
    }
    __syncthreads();

    // lane (c, h) holds column c of each tile, rows 8 (e / 4) + 4 h + e % 4
    const int64_t y_row = a.N * (a.bf16 ? 2 : 4);
    const bool fits = Tl::BM * y_row <= 0xffffffffLL;
    const BufRef yb = uniform_buf(static_cast<char*>(a.y) + m0 * y_row, (uint32_t)(fits ? mrows * y_row : 0));
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int64_t n = n0 + wave * 32 * NT + j * 32 + c;
        const bool in = n < a.N;
        const float sw = in ? a.scales[n] : 0.0f;
        const int32_t z = in ? code_shift<B>(a.zeros, n) : 0;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = i * 32 + 8 * q + 4 * h;
                const float4 s4 = *reinterpret_cast<const float4*>(sx + row);
                const int4 t4 = *reinterpret_cast<const int4*>(ssum + row);
                const float s[4] = {s4.x, s4.y, s4.z, s4.w};
                const int32_t t[4] = {t4.x, t4.y, t4.z, t4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v = finish_i8(acc[i][j][4 * q + e], z, t[e], s[e], sw);
                    if (fits) {
                        // rows past M lie past the buffer; columns past N are sent there
                        const uint32_t voff = in ? (uint32_t)(4 * h * y_row + n * (a.bf16 ? 2 : 4)) : 0xfffffff0u;
                        const uint32_t soff = (uint32_t)((i * 32 + 8 * q + e) * y_row);
                        if (a.bf16)
                            __builtin_amdgcn_raw_buffer_store_b16(bf16_round(v), make_rsrc(yb.base, yb.bytes), voff, soff, 2);
                        else
                            buf_store_f32_nt(yb, v, voff, soff);
                    } else if (in && row + e < mrows) {
                        if (a.bf16)
                            store_y<true>(a.y, (m0 + row + e) * a.N + n, v);
                        else
                            store_y<false>(a.y, (m0 + row + e) * a.N + n, v);
                    }
                }
            }
        }
    }
}

template <int B, int MT, int NT, int kOcc>
hipError_t launch_many(const I8Args& a, hipStream_t stream)
{
    using Tl = ManyTile<MT, NT>;
    const int64_t tiles = ceil_div(a.M, Tl::BM) * ceil_div(a.N, Tl::BN);
    if (tiles > 0x7fffffffLL) return hipErrorInvalidConfiguration;
    many_i8_kernel<B, MT, NT, kOcc><<<dim3((unsigned)tiles), dim3(256), 0, stream>>>(a);
    return hipGetLastError();
}

template <int B>
hipError_t launch_b(const I8Args& a, hipStream_t stream)
{
    if (a.M <= 64) {
        if (a.M <= 16) return launch_few_rows<B, 1>(a, stream);
        if (a.M <= 32) return launch_few_rows<B, 2>(a, stream);
        return launch_few_rows<B, 4>(a, stream);
    }
    // 256 x 256 tiles when they fill the 256 CUs in whole rounds (at least 80 %
    // of the last round busy)
    const int64_t wide = ceil_div(a.M, 256) * ceil_div(a.N, 256);
    if (a.M >= 256 && wide >= 256 && wide * 5 >= ceil_div(wide, 256) * 256 * 4)
        return launch_many<B, 8, 2, 1>(a, stream);
    if (ceil_div(a.M, 128) * ceil_div(a.N, 256) >= 400) return launch_many<B, 4, 2, 2>(a, stream);
    return launch_many<B, 4, 1, 2>(a, stream);
}

}  // namespace

hipError_t launch_gemm_i8(const int8_t* x, const float* x_scales, const int32_t* x_sums, int64_t M,
                          const uint32_t* packed, const float* scales, const int32_t* zeros,
                          int64_t N, int64_t K, int bits, void* y, bool bf16, hipStream_t stream)
{
    const I8Args a{x,      x_scales, x_sums, M, token_row_bytes(K), packed, scales, zeros,
                   N,      packed_row_words(K, bits), y, bf16};
#define CALL(B) launch_b<B>(a, stream)
    DQ_I8_BITS_SWITCH(bits, CALL)
#undef CALL
}

}  // namespace dq

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
#include "product_plan.hpp"

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
// Few tokens: bound by the packed weights.  A workgroup of W = 4 waves has 16 R
// weight rows, all tokens (M <= 64: 16 T, the last ones again past M) and all of
// K: wave w takes the steps w, w + W, ... of 256 codes, and the waves' sums are
// added through LDS.  (W = 8 with 16 T of more tokens: few tiles, see product_plan.hpp.)
// v_mfma_i32_16x16x64_i8 with the weights as its rows: lane (r, g) holds, of
// weight row r, the chunks 2 g and 2 g + 1 of the step, 2 B consecutive words, so
// codes go from memory to registers to the matrix cores, a row's 256 codes with
// four lanes' neighbouring loads.  The tokens' bytes of the same codes come from L1
// / L2 likewise.  A step's loads are in flight while the step before is multiplied.
//
// Rows per workgroup: the more, the less often the tokens' bytes are read and
// the fewer rows are open at once, as long as every CU has a workgroup.  16 x
// 28672 x 8192 at b = 6: 112 rows (256 workgroups) 39.5 us (4.5 TB/s of
// weights), 64 rows 45.8, 32 rows 53.9, 16 rows 56; 1 x 4096 x 4096 at b = 4:
// 16 rows (256 workgroups) 4.1 us, 32 rows 5.3, 64 rows 7.7.
template <int B, int R, int T, int W>
__global__ __launch_bounds__(W * kWave, W == 8 ? 2 : (R >= 7 || T == 4 ? 1 : (R == 1 ? 4 : 2))) void few_i8_kernel(I8Args a)
{
    constexpr int kFewWaves = W, kFewThreads = W * kWave;
    __shared__ __attribute__((aligned(16))) int32_t part[kFewWaves][R * T * 4 * kWave];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane & 15;
    const int g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * R);
    const int64_t m0 = (int64_t)blockIdx.y * (16 * T);
    const int64_t mrows = a.M - m0 < 16 * T ? a.M - m0 : 16 * T;
    const int64_t nrows = a.N - n0 < 16 * R ? a.N - n0 : 16 * R;
    const int steps = (int)((a.pitch + 255) >> 8);

    const uint32_t row_bytes = (uint32_t)a.row_words * 4;
    const BufRef wbuf = uniform_buf(a.packed + n0 * a.row_words, (uint32_t)nrows * row_bytes);
    const BufRef xbuf = uniform_buf(a.x + m0 * a.pitch, (uint32_t)(mrows * a.pitch));
    uint32_t woff[R], xoff[T];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int row = 16 * i + r < nrows ? 16 * i + r : (int)nrows - 1;
        woff[i] = row * row_bytes + g * (8 * B);
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const int64_t m = 16 * t + r < mrows ? 16 * t + r : mrows - 1;
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
    for (int j = 0; j < R * T * 4 / W; ++j) {
        const int o = j * kFewThreads + threadIdx.x;
        int32_t sum = part[0][o];
#pragma unroll
        for (int v = 1; v < kFewWaves; ++v) sum += part[v][o];
        const int tl = o / (4 * kWave), l = (o >> 2) & (kWave - 1);
        const int64_t m = m0 + 16 * (tl % T) + (l & 15);
        const int64_t n = n0 + 16 * (tl / T) + 4 * (l >> 4) + (o & 3);
        if (m < a.M && n < a.N) {
            const float v = finish_i8(sum, code_shift<B>(a.zeros, n), a.x_sums[m], token_scale(a.x_scales[m]), a.scales[n]);
            if (a.bf16)
                store_y<true>(a.y, m * a.N + n, v);
            else
                store_y<false>(a.y, m * a.N + n, v);
        }
    }
}

template <int B, int R, int T, int W = 4>
hipError_t launch_few(const I8Args& a, hipStream_t stream)
{
    few_i8_kernel<B, R, T, W>
        <<<dim3((unsigned)ceil_div(a.N, 16 * R), (unsigned)ceil_div(a.M, 16 * T)), W * kWave, 0, stream>>>(a);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Many tokens: bound by the matrix cores.  4 WM waves: four side by side along
// N, WM along M; a wave owns 32 MT token rows and 32 NT columns of the
// workgroup's tile, as MT x NT tiles of v_mfma_i32_32x32x32_i8.
//
// A step is 128 codes.  Tokens and packed codes both go from memory to LDS
// directly, as whole 128-byte lines of a row, in two or four stages of a step.  (Codes
// straight into the registers of their lanes touch 64 lines per load, eight
// loads per line, and L1 looks up a line a cycle: 2048 x 8192 x 8192 at b = 8 took
// 137 us so.)  Substep t (0 .. 3) multiplies, for lane half h, the bytes 64 h + 16 t ..
// + 15 of the step: token operands are 16-byte piece 4 h + t of a row, weight
// operands half t & 1 of chunk 2 h + (t >> 1), whose words a lane reads from LDS once
// per step and expands a substep ahead.  Piece p of a row lies at slot p ^ f(row),
// with f such that the rows of one LDS pass spread over all banks.  Each
// substep's MFMAs run beside the expansion and the LDS reads of the next; after
// the third, the step's stage has been read by every wave, and behind one
// barrier the copies of the step after next go out into it.
template <int MT, int NT, int WM>
struct ManyTile {
    static constexpr int BM = 32 * MT * WM;
    static constexpr int kThreads = 256 * WM;
    static constexpr int BN = 128 * NT;
    static constexpr int kCopies = MT;  // 16-byte pieces of tokens per thread and step
};

// Slot of 16-byte piece p of a row of tokens (8 pieces).
__device__ __forceinline__ int x_slot(int row, int p) { return p ^ ((row >> 1) & 7); }
// Slot of piece p of a row's codes (B pieces): rows of 6 and 2 pieces, and of an
// odd number, read in 8-byte parts, spread over the banks as they are.
template <int B>
__device__ __forceinline__ int w_slot(int row, int p)
{
    if constexpr (B == 8) return p ^ ((row >> 1) & 7);
    if constexpr (B == 4) return p ^ ((row >> 2) & 3);
    return p;
}

// The 2 B words of half h of a row's codes in LDS.
template <int B>
__device__ __forceinline__ void read_words(const uint4* rows, int row, int h, uint32_t (&w)[2 * B])
{
    if constexpr (B % 2 == 0) {
#pragma unroll
        for (int i = 0; i < B / 2; ++i) {
            const uint4 v = rows[row * B + w_slot<B>(row, h * (B / 2) + i)];
            w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
    } else {
        const uint2* p = reinterpret_cast<const uint2*>(rows + row * B) + h * B;
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const uint2 v = p[i];
            w[2 * i] = v.x, w[2 * i + 1] = v.y;
        }
    }
}

// Waits until at most n of the wave's vector-memory operations and none of its
// LDS operations are in flight, then for the other waves (__syncthreads would
// wait for every copy).
template <int n>
__device__ __forceinline__ void join_waves()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (7 << 4));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}

template <int B, int MT, int NT, int WM, int kOcc, int S>
__global__ __launch_bounds__(256 * WM, kOcc) void many_i8_kernel(I8Args a)
{
    using Tl = ManyTile<MT, NT, WM>;
    static_assert(S == 2 || S == 4, "stages");
    constexpr int kCopies = Tl::kCopies;
    constexpr int kWCopies = NT * B / (2 * WM);  // whole pieces of codes per thread and step
    constexpr bool kWHalf = (NT * B) % (2 * WM) != 0;  // and one more for half of the threads
    // an array per stage: a read of one stage is then known not to depend on the
    // copies in flight into another (one array for all: every read waited for
    // every copy, a whole memory latency per step)
    __shared__ __attribute__((aligned(16))) uint4 As0[Tl::BM * 8], As1[Tl::BM * 8];
    __shared__ __attribute__((aligned(16))) uint4 Ws0[Tl::BN * B], Ws1[Tl::BN * B];
    __shared__ __attribute__((aligned(16))) uint4 As2[S > 2 ? Tl::BM * 8 : 1], As3[S > 2 ? Tl::BM * 8 : 1];
    __shared__ __attribute__((aligned(16))) uint4 Ws2[S > 2 ? Tl::BN * B : 1], Ws3[S > 2 ? Tl::BN * B : 1];
    auto as = [&](auto St) __attribute__((always_inline)) -> uint4* {
        if constexpr (decltype(St)::value == 0) return As0;
        else if constexpr (decltype(St)::value == 1) return As1;
        else if constexpr (decltype(St)::value == 2) return As2;
        else return As3;
    };
    auto ws = [&](auto St) __attribute__((always_inline)) -> uint4* {
        if constexpr (decltype(St)::value == 0) return Ws0;
        else if constexpr (decltype(St)::value == 1) return Ws1;
        else if constexpr (decltype(St)::value == 2) return Ws2;
        else return Ws3;
    };

    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wn = wave & 3;
    const int wm = wave >> 2;
    const int c = lane & 31;
    const int h = lane >> 5;

    // consecutive workgroups go round robin to the 8 XCDs; each XCD gets a
    // contiguous range of tiles, groups of 4 row tiles by all column tiles
    const int64_t ntm = ceil_div(a.M, Tl::BM);
    const int64_t ntn = ceil_div(a.N, Tl::BN);
    const int64_t tiles = ntm * ntn;
    const int64_t L = (int64_t)(blockIdx.x & 7) * ((tiles + 7) >> 3) + (blockIdx.x >> 3);
    if (L >= tiles) return;
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
        const int p = x_slot(row, slot & 7);
        xoff[i] = (uint32_t)((row < mrows ? row : mrows - 1) * a.pitch + 16 * p);
    }
    const int64_t nrows = a.N - n0 < Tl::BN ? a.N - n0 : Tl::BN;
    const uint32_t row_bytes = (uint32_t)a.row_words * 4;
    const BufRef wbuf = uniform_buf(a.packed + n0 * a.row_words, (uint32_t)nrows * row_bytes);
    // 128 NT rows of B pieces, 64 pieces per wave and copy
    constexpr int kWAll = kWCopies + (kWHalf ? 1 : 0);
    constexpr int kStepCopies = kCopies + kWCopies;  // of the waves that copy the least
    uint32_t woff[kWAll];
#pragma unroll
    for (int i = 0; i < kWAll; ++i) {
        const int slot = (i * 4 * WM + wave) * 64 + lane;
        const int row = slot / B;
        const int p = w_slot<B>(row, slot % B);
        woff[i] = (uint32_t)(row < nrows ? row : nrows - 1) * row_bytes + 16 * p;
    }
    int abase[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) abase[t] = wm * (256 * MT) + c * 8 + x_slot(c, 4 * h + t);

    i32x16_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

    uint32_t w[NT][2 * B];
    i32x4_t bq[NT];     // weight operands of the current substep
    i32x4_t aq[2][MT];  // token operands of the current and the next substep
    auto copy = [&](auto St, int ks) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kCopies; ++i)
            buf_load_lds16(xbuf, as(St) + (wave * kCopies + i) * 64, xoff[i], (uint32_t)ks * 128);
#pragma unroll
        for (int i = 0; i < kWAll; ++i)
            if (i < kWCopies || wave < 2 * WM)
                buf_load_lds16(wbuf, ws(St) + (i * 4 * WM + wave) * 64, woff[i] + (uint32_t)ks * (16 * B), 0);
    };
    auto read_w = [&](auto St) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NT; ++j) read_words<B>(ws(St), (wn * NT + j) * 32 + c, h, w[j]);
    };
    auto codes = [&](int j, int t) __attribute__((always_inline)) {
        return expand16<B>(reinterpret_cast<const uint32_t(&)[B]>(w[j][(t >> 1) * B]), t & 1);
    };
    auto read_a = [&](auto St, int t, i32x4_t (&dst)[MT]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < MT; ++i) dst[i] = __builtin_bit_cast(i32x4_t, as(St)[abase[t] + 256 * i]);
    };

    auto step = [&](auto St, int ks) __attribute__((always_inline)) {
        constexpr int st = decltype(St)::value;
        using Other = std::integral_constant<int, (st + 1) % S>;
        const int k2 = ks + S < nk ? ks + S : nk - 1;  // past the end: in bounds, never used
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            i32x4_t nb[NT];
            if (t < 3) {
                read_a(St, t + 1, aq[(t + 1) & 1]);
            } else {
                read_w(Other{});
                read_a(Other{}, 0, aq[0]);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) nb[j] = codes(j, (t + 1) & 3);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(aq[t & 1][i], bq[j], acc[i][j], 0, 0, 0);
#pragma unroll
            for (int j = 0; j < NT; ++j) bq[j] = nb[j];
            __builtin_amdgcn_sched_barrier(0);
            if (t == 2) {
                // stage ks + 1 is whole; stage ks is read by no wave any more
                join_waves<(S - 2) * kStepCopies>();
                copy(St, k2);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };

    using First = std::integral_constant<int, 0>;
    static_for<S>([&](auto St) {
        copy(St, (int)St.value < nk ? (int)St.value : nk - 1);
        __builtin_amdgcn_sched_barrier(0);
    });
    join_waves<(S - 1) * kStepCopies>();
    read_w(First{});
    read_a(First{}, 0, aq[0]);
#pragma unroll
    for (int j = 0; j < NT; ++j) bq[j] = codes(j, 0);
    int ks = 0;
    for (; ks + S <= nk; ks += S) static_for<S>([&](auto St) { step(St, ks + (int)St.value); });
    static_for<S - 1>([&](auto St) {
        if (ks + (int)St.value < nk) step(St, ks + (int)St.value);
    });

    // the last copies into LDS have landed in every wave before the stages
    // serve for the tokens' scales and sums
    join_waves<0>();
    float* const sx = reinterpret_cast<float*>(As0);
    float* const sup = sx + Tl::BM;
    int32_t* const ssum = reinterpret_cast<int32_t*>(sup + Tl::BM);
    if (tid < Tl::BM) {
        const int64_t m = m0 + tid < a.M ? m0 + tid : a.M - 1;
        const TokenScale ts = token_scale(a.x_scales[m]);
        sx[tid] = ts.s;
        sup[tid] = ts.up;
        ssum[tid] = a.x_sums[m];
    }
    __syncthreads();

    // lane (c, h) holds column c of each tile, rows 8 (e / 4) + 4 h + e % 4
    const int64_t y_row = a.N * (a.bf16 ? 2 : 4);
    // whole tiles store without checks, at scalar row offsets (the tile's rows of y
    // must span less than 4 GiB)
    const bool inside = Tl::BM * y_row <= 0xffffffffLL && m0 + Tl::BM <= a.M && n0 + Tl::BN <= a.N;
    const BufRef yb = uniform_buf(static_cast<char*>(a.y) + m0 * y_row, (uint32_t)(inside ? Tl::BM * y_row : 0));
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int64_t n = n0 + wn * 32 * NT + j * 32 + c;
        const bool in = n < a.N;
        const float sw = in ? a.scales[n] : 0.0f;
        const int32_t z = in ? code_shift<B>(a.zeros, n) : 0;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = (wm * MT + i) * 32 + 8 * q + 4 * h;
                const float4 s4 = *reinterpret_cast<const float4*>(sx + row);
                const float4 u4 = *reinterpret_cast<const float4*>(sup + row);
                const int4 t4 = *reinterpret_cast<const int4*>(ssum + row);
                const TokenScale s[4] = {{s4.x, u4.x}, {s4.y, u4.y}, {s4.z, u4.z}, {s4.w, u4.w}};
                const int32_t t[4] = {t4.x, t4.y, t4.z, t4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v = finish_i8(acc[i][j][4 * q + e], z, t[e], s[e], sw);
                    if (inside) {
                        const uint32_t voff = (uint32_t)(4 * h * y_row + n * (a.bf16 ? 2 : 4));
                        const uint32_t soff = (uint32_t)(((wm * MT + i) * 32 + 8 * q + e) * y_row);
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

template <int B, int MT, int NT, int WM, int kOcc, int S = 2>
hipError_t launch_many(const I8Args& a, hipStream_t stream)
{
    using Tl = ManyTile<MT, NT, WM>;
    const int64_t tiles = ceil_div(a.M, Tl::BM) * ceil_div(a.N, Tl::BN);
    if (tiles > 0x7ffffff0LL) return hipErrorInvalidConfiguration;
    many_i8_kernel<B, MT, NT, WM, kOcc, S><<<dim3((unsigned)((tiles + 7) & ~7LL)), dim3(Tl::kThreads), 0, stream>>>(a);
    return hipGetLastError();
}

template <int B>
hipError_t launch_b(const I8Args& a, hipStream_t stream)
{
    switch (i8_kernel(a.M, a.N)) {
    case I8Kernel::few_1_1: return launch_few<B, 1, 1>(a, stream);
    case I8Kernel::few_2_1: return launch_few<B, 2, 1>(a, stream);
    case I8Kernel::few_4_1: return launch_few<B, 4, 1>(a, stream);
    case I8Kernel::few_7_1: return launch_few<B, 7, 1>(a, stream);
    case I8Kernel::few_1_2: return launch_few<B, 1, 2>(a, stream);
    case I8Kernel::few_2_2: return launch_few<B, 2, 2>(a, stream);
    case I8Kernel::few_4_2: return launch_few<B, 4, 2>(a, stream);
    case I8Kernel::few_7_2: return launch_few<B, 7, 2>(a, stream);
    case I8Kernel::few_2_4: return launch_few<B, 2, 4>(a, stream);
    case I8Kernel::few_4_4: return launch_few<B, 4, 4>(a, stream);
    case I8Kernel::few_7_4: return launch_few<B, 7, 4>(a, stream);
    case I8Kernel::split_2: return launch_few<B, 2, 2, 8>(a, stream);
    case I8Kernel::split_4: return launch_few<B, 2, 4, 8>(a, stream);
    case I8Kernel::tiles_256x256: return launch_many<B, 4, 2, 2, 2>(a, stream);
    case I8Kernel::tiles_128x128: return launch_many<B, 4, 1, 1, B <= 5 ? 3 : 2>(a, stream);
    case I8Kernel::tiles_64x128_deep: return launch_many<B, 2, 1, 1, 1, 4>(a, stream);
    case I8Kernel::tiles_64x128: return launch_many<B, 2, 1, 1, 3>(a, stream);
    default: return hipErrorInvalidValue;
    }
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

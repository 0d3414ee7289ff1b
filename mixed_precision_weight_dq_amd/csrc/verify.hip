// Drafted tokens: the masks of a tree of them, and their verification against the
// target's probabilities from given random numbers.
//
// A sequence's rows of a call are a tree: row 0 is its root, row i's parent an earlier
// row (else no path reaches it).  p[r] is the target's distribution of the token after
// row r, tok[i] and u[i] row i's token and random number.  From cur = 0 on, cur's
// children are tried in order of their rows:
//   without draft probabilities child c is taken if u[c] * rest < p[cur][tok[c]], rest
//     being 1 less the probabilities of the children tried before (a token twice counts
//     once), and cur = c; else its token's probability becomes 0.  So a child is taken with
//     its probability given that the ones before it were not: for any candidates the
//     token that comes out is distributed as p;
//   with draft probabilities q, from which the first child's token was drawn, it is taken if
//     u[c] * q[cur][tok[c]] < p[cur][tok[c]]; else p becomes max(p - q, 0) and no other
//     child is tried.
// The next token is then drawn from what p[cur] has become: the first x whose running sum
// passes u[0] times the whole sum.
//
// Sums of a vocabulary, and what is compared, are fp64: fp32 sums of 10^5 terms would move
// the borders between tokens by 10^-6, and some draw in a batch would go the other way.
//
// Bound by one row of p (and of q) per sequence, and where those are few by the trips to memory that
// wait for each other (starts, parents and ids, probabilities, the row; the sums, the stretch).
// Children have larger rows than their parents, so a walk is one pass over a sequence's rows, 64 of
// them in a wave's lanes.  verify_sums_kernel: every wave walks for itself (no barrier, and the
// loads of all waves of a sequence are the same) and sums one stretch of kStretch tokens;
// verify_draw_kernel: a workgroup per sequence finds the stretch, and the token in it.  6 rows of 32000
// with draft probabilities 4.8 + 3.5 us, 16 trees of 32 rows of 50001 5.7 + 4.7, 48 x 7 of 128000 with draft
// probabilities (49 MB) 12 + 5, the sums at 4.0 TB/s.
#include "common.hpp"
#include "launch_serving.hpp"

namespace dq {

namespace {

constexpr int kThreads = 256;
// Tokens of a stretch: 1 x 6 x 32000 7.6 us, 48 x 7 x 128000 16.7 (2048: 9.2, 18.4; 512: 7.1, 18.2).
constexpr int kStretch = 1024;
constexpr int kEach = kStretch / kWave;

// Rows of sequence b, within the call's.
__device__ __forceinline__ void rows_of(const int32_t* starts, int64_t b, int64_t tokens, int64_t& first, int64_t& n)
{
    int64_t s = starts[b], e = starts[b + 1];
    s = s < 0 ? 0 : (s > tokens ? tokens : s);
    e = e < s ? s : (e > tokens ? tokens : e);
    first = s;
    n = e - s;
}

__device__ __forceinline__ int read_lane(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ float read_lane(float v, int lane)
{
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}

// 64 rows of a sequence, one in each lane.
struct Lanes {
    int64_t base;
    int parent, token;  // parent -2 where there is no row
};

__device__ __forceinline__ Lanes load_lanes(const VerifyArgs& a, int64_t first, int64_t n, int64_t base)
{
    Lanes r{base, -2, 0};
    const int64_t i = base + (threadIdx.x & (kWave - 1));
    if (i > 0 && i < n) {
        r.parent = a.parents[first + i];
        r.token = a.ids[first + i];
    }
    return r;
}

// Lanes whose rows are children of cur, and rows behind it.
__device__ __forceinline__ uint64_t children(const Lanes& r, int64_t cur)
{
    const int64_t i = r.base + (threadIdx.x & (kWave - 1));
    return __ballot(i > cur && r.parent == cur);
}

// f(token) of every child of cur before row end (all were tried).
template <class F>
__device__ __forceinline__ void each_child(const VerifyArgs& a, int64_t first, int64_t cur, int64_t end, F f)
{
    if (end > kMaxDrafts) end = kMaxDrafts;
    for (int64_t base = cur & ~(int64_t)(kWave - 1); base < end; base += kWave) {
        const Lanes r = load_lanes(a, first, end, base);
        for (uint64_t left = children(r, cur); left; left &= left - 1) f(read_lane(r.token, __builtin_ctzll(left)));
    }
}

// The walk of sequence b: the last row taken, whether its child's draft probabilities come off,
// and, where write is set, the path.
struct Walked {
    int64_t cur;
    bool less;
};
template <bool kDraft>
__device__ __forceinline__ Walked walk(const VerifyArgs& a, int64_t b, int64_t first, int64_t n, bool write)
{
    const int lane = threadIdx.x & (kWave - 1);
    Walked w{0, false};
    int64_t at = 1;
    double rest = 1.0;
    const int64_t drafts = n < kMaxDrafts ? n : kMaxDrafts;
    if (write && lane == 0) a.path[first] = 0;
    for (int64_t base = 0; base < drafts && !w.less; base += kWave) {
        const Lanes r = load_lanes(a, first, drafts, base);
        const int64_t i = base + lane;
        // what each row would be tried with
        float u = 0.0f, p = 0.0f, q = 0.0f;
        if (r.parent >= 0 && r.parent < i) {
            u = a.uniforms[first + i];
            if (r.token >= 0 && r.token < a.vocab) {
                p = a.probs[(first + r.parent) * a.probs_stride + r.token];
                if (kDraft) q = a.draft[(first + r.parent) * a.draft_stride + r.token];
            }
        }
        uint64_t left = children(r, w.cur);
        while (left) {
            const int l = __builtin_ctzll(left);
            left &= left - 1;
            const double ul = read_lane(u, l);
            double pl = read_lane(p, l);
            bool take;
            if (kDraft) {
                take = ul * (double)read_lane(q, l) < pl;
                w.less = !take;
                if (!take) break;
            } else {
                const int token = read_lane(r.token, l);
                // a token that was tried before
                bool again = (children(r, w.cur) & __ballot(r.token == token) & ((1ull << l) - 1)) != 0;
                if (base > w.cur)
                    each_child(a, first, w.cur, base, [&](int other) { again |= other == token; });
                if (again) pl = 0.0;
                take = ul * rest < pl;
                rest -= pl;
            }
            if (take) {
                w.cur = base + l;
                rest = 1.0;
                if (write && lane == 0) a.path[first + at] = (int32_t)w.cur;
                ++at;
                left = children(r, w.cur);
            }
        }
    }
    if (write) {
        for (int64_t j = at + lane; j < n; j += kWave) a.path[first + j] = -1;
        if (lane == 0) a.accepted[b] = (int32_t)at;
    }
    return w;
}

__device__ __forceinline__ float positive(float v) { return v > 0.0f ? v : 0.0f; }

// What is left of p at x, given both probabilities.
__device__ __forceinline__ double left_of(double p, double q)
{
    const double v = p - q;
    return v > 0.0 ? v : 0.0;
}

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
    return v;
}

template <bool kDraft>
__global__ __launch_bounds__(kThreads) void verify_sums_kernel(VerifyArgs a)
{
    const int64_t wave = (int64_t)blockIdx.x * (kThreads / kWave) + threadIdx.x / kWave;
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t b = blockIdx.y;
    if (wave >= a.chunks) return;
    int64_t first, n;
    rows_of(a.starts, b, a.tokens, first, n);
    if (n == 0) {
        if (wave == 0 && lane == 0) {
            a.accepted[b] = 0;
            a.next[b] = -1;
        }
        return;
    }
    const Walked w = walk<kDraft>(a, b, first, n, wave == 0);
    if (wave == 0 && lane == 0) {
        a.state[2 * b] = (int32_t)w.cur;
        a.state[2 * b + 1] = w.less;
    }
    const int64_t x0 = wave * kStretch;
    const float* p = a.probs + (first + w.cur) * a.probs_stride;
    // (past the vocabulary: the last token again, which counts as 0)
    float v[kEach];
    const auto place = [&](int e) {
        const int64_t x = x0 + e * kWave + lane;
        return x < a.vocab ? x : a.vocab - 1;
    };
#pragma unroll
    for (int e = 0; e < kEach; ++e) v[e] = p[place(e)];
    double sum = 0.0;
    if (kDraft && w.less) {
        const float* q = a.draft + (first + w.cur) * a.draft_stride;
        float d[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) d[e] = q[place(e)];
        __builtin_amdgcn_sched_barrier(0);  // both rows in flight
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            sum += x0 + e * kWave + lane < a.vocab ? left_of(positive(v[e]), d[e]) : 0.0;
    } else {
        if (!kDraft)
            each_child(a, first, w.cur, n, [&](int token) {
                const int64_t at = token - x0;
                if (at < 0 || at >= kStretch) return;
#pragma unroll
                for (int e = 0; e < kEach; ++e)
                    if (at == e * kWave + lane) v[e] = 0.0f;
            });
#pragma unroll
        for (int e = 0; e < kEach; ++e) sum += x0 + e * kWave + lane < a.vocab ? positive(v[e]) : 0.0f;
    }
    sum = wave_sum(sum);
    if (lane == 0) a.sums[b * a.chunks + wave] = sum;
}

__device__ __forceinline__ double wave_scan(double v)
{
    const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const double t = __shfl_up(v, o, kWave);
        if (lane >= o) v += t;
    }
    return v;
}

// The first stretch (of sums that sum_of gives) whose running sum passes u times the whole,
// or the last with any probability, or -1; before: the running sum before it.  A wave's work.
template <class F>
__device__ __forceinline__ int64_t find_stretch(int64_t chunks, float u, F sum_of, double& before, double& target)
{
    const int lane = threadIdx.x & (kWave - 1);
    const double own = lane < chunks ? sum_of(lane) : 0.0;  // of the first 64
    double total = own;
    for (int64_t c = kWave + lane; c < chunks; c += kWave) total += sum_of(c);
    total = wave_sum(total);
    target = (double)u * total;
    before = 0.0;
    int64_t last = -1;
    for (int64_t c0 = 0; c0 < chunks; c0 += kWave) {
        const double mine = c0 == 0 ? own : (c0 + lane < chunks ? sum_of(c0 + lane) : 0.0);
        const double upto = wave_scan(mine);
        const uint64_t passes = __ballot(mine > 0.0 && before + upto > target), some = __ballot(mine > 0.0);
        if (passes) {
            const int l = __builtin_ctzll(passes);
            before += __shfl(upto - mine, l, kWave);
            return c0 + l;
        }
        if (some) last = c0 + 63 - __builtin_clzll(some);
        before += __shfl(upto, kWave - 1, kWave);
    }
    target = __builtin_huge_val();  // (a random number of 1 or more, a sum that is not finite)
    return last;
}

// Four waves per sequence: each finds the stretch for itself, a thread has 4 of its tokens.
template <bool kDraft>
__global__ __launch_bounds__(kThreads) void verify_draw_kernel(VerifyArgs a)
{
    constexpr int kMine = kStretch / kThreads;
    __shared__ double wave_total[kThreads / kWave];
    __shared__ int wave_pass[kThreads / kWave], wave_last[kThreads / kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t b = blockIdx.x;
    const double* sums = a.sums + b * a.chunks;
    const int64_t cur = a.state[2 * b];
    const bool less = a.state[2 * b + 1] != 0;
    int64_t first, n;
    rows_of(a.starts, b, a.tokens, first, n);
    if (n == 0) return;
    const float u = a.uniforms[first];
    const float* p = a.probs + (first + cur) * a.probs_stride;
    double before, target;
    int64_t c = find_stretch(a.chunks, u, [&](int64_t i) { return sums[i]; }, before, target);
    // nothing left, as where p and q are the same: of p as it is
    const bool plain = c < 0;
    if (plain)
        c = find_stretch(
            a.chunks, u,
            [&](int64_t i) {
                double sum = 0.0;
                for (int64_t x = i * kStretch; x < (i + 1) * kStretch && x < a.vocab; ++x) sum += positive(p[x]);
                return sum;
            },
            before, target);
    if (c < 0) {
        if (threadIdx.x == 0) a.next[b] = -1;
        return;
    }
    const int64_t x0 = c * kStretch + threadIdx.x * kMine;
    const auto place = [&](int e) { return x0 + e < a.vocab ? x0 + e : a.vocab - 1; };
    double v[kMine];
#pragma unroll
    for (int e = 0; e < kMine; ++e) v[e] = positive(p[place(e)]);
    if (!plain) {
        if (kDraft && less) {
            const float* q = a.draft + (first + cur) * a.draft_stride;
#pragma unroll
            for (int e = 0; e < kMine; ++e) v[e] = left_of(v[e], q[place(e)]);
        } else if (!kDraft) {
            each_child(a, first, cur, n, [&](int token) {
#pragma unroll
                for (int e = 0; e < kMine; ++e)
                    if (token == x0 + e) v[e] = 0.0;
            });
        }
    }
    double mine = 0.0;
#pragma unroll
    for (int e = 0; e < kMine; ++e) {
        if (x0 + e >= a.vocab) v[e] = 0.0;
        mine += v[e];
    }
    const double upto = wave_scan(mine);
    if (lane == kWave - 1) wave_total[wave] = upto;
    __syncthreads();
    double run = before + (upto - mine);
    for (int w = 0; w < wave; ++w) run += wave_total[w];
    // the thread's own first token that passes, or its last with any probability
    int pass = -1, last = -1;
#pragma unroll
    for (int e = 0; e < kMine; ++e) {
        run += v[e];
        if (v[e] > 0.0) {
            last = (int)(x0 + e);
            if (pass < 0 && run > target) pass = (int)(x0 + e);
        }
    }
    const uint64_t passes = __ballot(pass >= 0), some = __ballot(last >= 0);
    if (lane == 0) {
        wave_pass[wave] = -1;
        wave_last[wave] = -1;
    }
    if (passes && lane == (int)__builtin_ctzll(passes)) wave_pass[wave] = pass;
    if (some && lane == 63 - (int)__builtin_clzll(some)) wave_last[wave] = last;
    __syncthreads();
    if (threadIdx.x == 0) {
        int token = -1;
        for (int w = kThreads / kWave - 1; w >= 0; --w)
            if (token < 0) token = wave_last[w];
        for (int w = kThreads / kWave - 1; w >= 0; --w)
            if (wave_pass[w] >= 0) token = wave_pass[w];
        a.next[b] = token;
    }
}

// Mask and position of every drafted row, a thread each (latency: a tree's depth of parents): the bits of itself and its ancestors, and the cached
// tokens before the call's own plus its depth.  A row that is no tree's (its parent is no earlier
// row, or it lies past kMaxDrafts) is a root.
__global__ __launch_bounds__(kThreads) void draft_tree_kernel(const int32_t* __restrict__ parents,
                                                              const int32_t* __restrict__ starts,
                                                              const int32_t* __restrict__ lens, int64_t tokens,
                                                              int64_t words, int32_t* __restrict__ mask,
                                                              int32_t* __restrict__ positions)
{
    const int64_t b = blockIdx.y;
    int64_t first, n;
    rows_of(starts, b, tokens, first, n);
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        // from the row up to its root, the words from the last to the first
        int32_t* const row = mask + (first + i) * words;
        int64_t word = words - 1, at = i;
        uint32_t bits = 0;
        int32_t depth = 0;
        while (true) {
            const int64_t to = at >> 5;
            for (; word > to; --word) {
                row[word] = (int32_t)bits;
                bits = 0;
            }
            if (to < words) bits |= 1u << (at & 31);
            const int64_t up = at < kMaxDrafts ? parents[first + at] : -1;
            if (up < 0 || up >= at) break;
            at = up;
            ++depth;
        }
        for (; word >= 0; --word) {
            row[word] = (int32_t)bits;
            bits = 0;
        }
        if (positions) positions[first + i] = (int32_t)(lens[b] - n + depth);
    }
}

}  // namespace

size_t verify_workspace(int64_t count, int64_t vocab)
{
    return (size_t)count * (ceil_div(vocab, kStretch) * sizeof(double) + 2 * sizeof(int32_t));
}

hipError_t launch_verify(VerifyArgs a, void* workspace, hipStream_t stream)
{
    a.chunks = ceil_div(a.vocab, kStretch);
    a.sums = static_cast<double*>(workspace);
    a.state = reinterpret_cast<int32_t*>(a.sums + a.count * a.chunks);
    const dim3 grid((unsigned)ceil_div(a.chunks, kThreads / kWave), (unsigned)a.count);
    (a.draft ? verify_sums_kernel<true> : verify_sums_kernel<false>)<<<grid, kThreads, 0, stream>>>(a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    (a.draft ? verify_draw_kernel<true> : verify_draw_kernel<false>)<<<(unsigned)a.count, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_draft_tree(const int32_t* parents, const int32_t* starts, const int32_t* lens, int64_t count,
                             int64_t tokens, int64_t words, int32_t* mask, int32_t* positions, hipStream_t stream)
{
    const int64_t each = ceil_div(ceil_div(tokens, count), kThreads);
    draft_tree_kernel<<<dim3((unsigned)(each < 64 ? each : 64), (unsigned)count), kThreads, 0, stream>>>(
        parents, starts, lens, tokens, words, mask, positions);
    return hipGetLastError();
}

}  // namespace dq

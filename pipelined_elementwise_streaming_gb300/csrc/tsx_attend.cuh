// How the attention kernels share out their work, and how parts are joined.
//
// The queries of a sequence that read one head are rows, `group` to a token, cut
// into tiles of M rows; a tile goes over the keys that its last row sees, TK at a
// time.  One such step is a unit, and as many more before a tile's first step, COST,
// stand for its start and end.  All units of a call stand in a row (by sequence, head,
// tile, step), and each of a fixed number of CTAs takes an equal run of them: lengths
// of sequences need not be known to the host, none of them leaves CTAs without work,
// and single long ones are split.  A CTA whose run starts or ends
// within a tile writes a part of that tile's result (the unnormalised sum, the
// maximum and the sum of weights) to the scratch, and a second kernel joins the
// parts in order.
#pragma once

#include "attention.h"
#include "tsx_norm.cuh"

namespace tsx {
namespace dev {

// Which of a sequence's pages holds a position.
__device__ __forceinline__ int page_of(const PagedArgs& p, int position)
{
    return p.page_shift >= 0 ? position >> p.page_shift : position / p.page_size;
}

// A sequence with new tokens.
struct Seq {
    int first;     // its first row of tokens
    int fresh;     // new tokens
    int length;    // keys, new ones among them
    int prior;     // keys before the first new token (negative: a length shorter than that)
};

__device__ __forceinline__ Seq seq_of(const AttendArgs& a, int b)
{
    const int tokens = static_cast<int>(a.tokens);
    Seq s;
    s.first = min(max(a.paged.starts[b], 0), tokens);
    s.fresh = min(max(a.paged.starts[b + 1], s.first), tokens) - s.first;
    const int64_t most = min(static_cast<int64_t>(a.paged.most_pages) * a.paged.page_size, static_cast<int64_t>(kMostKeys));
    s.length = static_cast<int>(min(static_cast<int64_t>(max(a.paged.lengths[b], 0)), most));
    s.prior = s.length - s.fresh;
    return s;
}

// Keys that a row sees: those before this one.
__device__ __forceinline__ int row_limit(const AttendArgs& a, const Seq& s, int row)
{
    return max(s.prior + row / a.group + 1, 0);
}

// a / by; in 32 bits, at a fifth of the instructions, where that is enough.  What
// runs once in a kernel waits for its instructions rather than for its arithmetic, so
// the long ways are there once (a tile's results took 5 us in place of 2.5 in longer
// code).
static __device__ __noinline__ uint64_t long_quotient(uint64_t a, uint64_t by) { return a / by; }
__device__ __forceinline__ uint64_t quotient(uint64_t a, uint64_t by)
{
    return (a | by) >> 32 ? long_quotient(a, by) : static_cast<uint32_t>(a) / static_cast<uint32_t>(by);
}

// Sum of floor((step i + from) / by) over 0 <= i < n: the whole parts, and the same
// sum mirrored.
static __device__ __noinline__ uint64_t long_floor_sum(uint64_t n, uint64_t by, uint64_t step, uint64_t from)
{
    uint64_t sum = 0;
    while (n) {
        const uint64_t p = step / by, q = from / by;
        sum += n * (n - 1) / 2 * p + n * q;
        step -= p * by;
        const uint64_t top = step * n + (from - q * by);
        n = top / by;
        from = top - n * by;
        const uint64_t t = by;
        by = step;
        step = t;
    }
    return sum;
}
__device__ __forceinline__ uint64_t floor_sum(uint64_t n, uint64_t by, uint64_t step, uint64_t from)
{
    // n < 2^31: the largest number met in 32 bits is step n + from
    if ((by | (step * n + from)) >> 32)
        return long_floor_sum(n, by, step, from);
    uint32_t n32 = static_cast<uint32_t>(n), by32 = static_cast<uint32_t>(by), step32 = static_cast<uint32_t>(step),
             from32 = static_cast<uint32_t>(from);
    uint64_t sum = 0;
#pragma unroll 1
    while (n32) {
        const uint32_t p = step32 / by32, q = from32 / by32;
        sum += (static_cast<uint64_t>(n32) * (n32 - 1) >> 1) * p + static_cast<uint64_t>(n32) * q;
        step32 -= p * by32;
        const uint32_t top = step32 * n32 + (from32 - q * by32);
        n32 = top / by32;
        from32 = top - n32 * by32;
        const uint32_t t = by32;
        by32 = step32;
        step32 = t;
    }
    return sum;
}

template <int M>
__device__ __forceinline__ int tiles_of(const AttendArgs& a, const Seq& s)
{
    return (s.fresh * a.group + M - 1) / M;   // tokens * heads < 2^31
}

// Steps of a tile, at least one.
template <int M, int TK>
__device__ __forceinline__ int steps_of(const AttendArgs& a, const Seq& s, int tile)
{
    if (s.prior < 0)
        return max((s.length + TK - 1) / TK, 1);
    const int last = min(s.fresh * a.group - tile * M, M) + tile * M - 1;
    return (row_limit(a, s, last) + TK - 1) / TK;
}

// Steps of the first n tiles.
template <int M, int TK>
__device__ __forceinline__ int64_t steps_before(const AttendArgs& a, const Seq& s, int n)
{
    if (s.prior < 0)
        return static_cast<int64_t>(n) * max((s.length + TK - 1) / TK, 1);
    // ceil((prior + 1 + floor(last row / group)) / TK) with the divisions in one
    return static_cast<int64_t>(floor_sum(static_cast<uint64_t>(n), static_cast<uint64_t>(a.group) * TK, M,
                                          M - 1 + static_cast<uint64_t>(a.group) * (s.prior + TK)));
}

// Units of the first n tiles, and of a head.
template <int M, int TK, int COST>
__device__ __forceinline__ int64_t units_before(const AttendArgs& a, const Seq& s, int n)
{
    return steps_before<M, TK>(a, s, n) + static_cast<int64_t>(n) * COST;
}

template <int M, int TK, int COST>
__device__ __forceinline__ int64_t units_of_head(const AttendArgs& a, const Seq& s)
{
    const int tiles = tiles_of<M>(a, s);
    if (tiles == 0)
        return 0;
    return COST + steps_of<M, TK>(a, s, tiles - 1) + (tiles > 1 ? units_before<M, TK, COST>(a, s, tiles - 1) : 0);
}

// A CTA's run of units, and where it starts.
struct Run {
    int64_t from, to, per;   // units; per: of a CTA
    int b, head, tile;
    int64_t off;             // units of the tile before `from`
};

__device__ __forceinline__ void share_out(Run& r, int64_t total, int64_t least)
{
    r.per = max(static_cast<int64_t>(quotient(total + gridDim.x - 1, gridDim.x)), least);
    r.from = min(static_cast<int64_t>(blockIdx.x) * r.per, total);
    r.to = min(r.from + r.per, total);
}

__device__ __forceinline__ int64_t sum_upto(int64_t v, int lane)
{
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
        const int64_t o = __shfl_up_sync(0xffffffffu, v, m);
        v += lane >= m ? o : 0;
    }
    return v;
}

// The tile of unit `rest` of a head.
template <int M, int TK, int COST>
__device__ __forceinline__ void find_tile(const AttendArgs& a, const Seq& s, int64_t rest, Run& r)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = tiles_of<M>(a, s);   // units_before(lo) <= rest < units_before(hi)
    int64_t before = 0;
#pragma unroll 1
    while (hi - lo > 1) {   // 32 places looked at at once
        const int apart = (hi - lo + 32) / 33;
        const int64_t at = lo + static_cast<int64_t>(lane + 1) * apart;
        const int64_t units = at < hi ? units_before<M, TK, COST>(a, s, static_cast<int>(at)) : rest + 1;
        const int under = __popc(__ballot_sync(0xffffffffu, units <= rest));
        if (under)
            before = __shfl_sync(0xffffffffu, units, under - 1);
        lo += under * apart;
        hi = min(hi, lo + apart);
    }
    r.tile = lo;
    r.off = rest - before;
}

// Every thread of the CTA takes part; `sums` holds a word to each warp and three
// more.  Up to 32 sequences are a lane's each, in every warp alike; more of them are
// shared out among all threads.
template <int M, int TK, int COST, int THREADS>
__device__ __forceinline__ Run run_of(const AttendArgs& a, int64_t least, int64_t* sums)
{
    constexpr int kWarps = THREADS / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    Run r{};
    int64_t rest, head;   // units before mine in the sequence, and of a head
    if (a.paged.seqs <= 32) {
        Seq s{};
        head = 0;
        if (lane < a.paged.seqs) {
            s = seq_of(a, lane);
            head = units_of_head<M, TK, COST>(a, s);
        }
        const int64_t mine = head * a.heads, upto = sum_upto(mine, lane);
        share_out(r, __shfl_sync(0xffffffffu, upto, 31), least);
        if (r.from >= r.to)
            return r;
        r.b = __ffs(__ballot_sync(0xffffffffu, upto - mine <= r.from && r.from < upto)) - 1;
        rest = __shfl_sync(0xffffffffu, r.from - (upto - mine), r.b);
        head = __shfl_sync(0xffffffffu, head, r.b);
    } else {
        int64_t total = 0;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {   // the sum of all, then who has the first of mine
            int64_t before = 0;
#pragma unroll 1
            for (int base = 0; base < a.paged.seqs; base += THREADS) {
                const int b = base + threadIdx.x;
                head = b < a.paged.seqs ? units_of_head<M, TK, COST>(a, seq_of(a, b)) : 0;
                const int64_t mine = head * a.heads;
                int64_t upto = sum_upto(mine, lane), all = 0;
                if (lane == 31)
                    sums[warp] = upto;
                __syncthreads();
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    upto += w < warp ? sums[w] : 0;
                    all += sums[w];
                }
                upto += before;
                before += all;
                if (pass == 0 && base + THREADS >= a.paged.seqs) {
                    total = before;
                    share_out(r, total, least);
                }
                // one block of sequences: its sums are at hand
                if ((pass == 1 || a.paged.seqs <= THREADS) && r.from < r.to && upto - mine <= r.from && r.from < upto) {
                    sums[kWarps] = b;
                    sums[kWarps + 1] = r.from - (upto - mine);
                    sums[kWarps + 2] = head;
                }
                __syncthreads();
            }
            if (a.paged.seqs <= THREADS || r.from >= r.to)
                break;
        }
        if (r.from >= r.to)
            return r;
        r.b = static_cast<int>(sums[kWarps]);
        rest = sums[kWarps + 1];
        head = sums[kWarps + 2];
    }
    r.head = static_cast<int>(quotient(rest, head));
    find_tile<M, TK, COST>(a, seq_of(a, r.b), rest - r.head * head, r);
    return r;
}

// A part of a run within one tile: steps `step` .. end - 1 of `steps`; none where the
// run ends before the tile's first.
struct Piece {
    Seq seq;
    int b, head, tile, step, end, steps, rows;
    int64_t units;
    __device__ __forceinline__ bool whole() const { return step == 0 && end == steps; }
    __device__ __forceinline__ bool empty() const { return end <= step; }
};

template <int M, int TK, int COST>
__device__ __forceinline__ Piece piece_of(const AttendArgs& a, const Run& r)
{
    Piece p;
    p.seq = seq_of(a, r.b);
    p.b = r.b;
    p.head = r.head;
    p.tile = r.tile;
    p.steps = steps_of<M, TK>(a, p.seq, r.tile);
    p.units = min(p.steps + COST - r.off, r.to - r.from);
    p.step = static_cast<int>(max(r.off - COST, static_cast<int64_t>(0)));
    p.end = static_cast<int>(max(r.off + p.units - COST, static_cast<int64_t>(0)));
    p.rows = min(p.seq.fresh * a.group - r.tile * M, M);
    return p;
}

template <int M>
__device__ __forceinline__ void advance(const AttendArgs& a, Run& r, const Piece& p)
{
    r.from += p.units;
    r.off = 0;
    if (r.from >= r.to)
        return;
    if (++r.tile < tiles_of<M>(a, p.seq))
        return;
    r.tile = 0;
    if (++r.head < a.heads)
        return;
    r.head = 0;
    do
        ++r.b;
    while (seq_of(a, r.b).fresh == 0);   // units are left, so some sequence has tokens
}

// The scratch: parts of a CTA's first and last tile, and what its last one is.
struct Tail {
    int64_t last, per;   // the tile's last unit, and the units of a CTA; per 0: nothing to join
    int token, row0, rows, head;
    // CTAs after `cta` that go on with the tile
    __device__ __forceinline__ int follow(int cta) const { return per ? static_cast<int>(last / per) - cta : 0; }
};

// Where the CTA's part of this piece goes, and what is to be joined.
__device__ __forceinline__ int part_slot(const Piece& p) { return 2 * blockIdx.x + (p.step == 0 ? 1 : 0); }

template <int M, int COST>
__device__ __forceinline__ Tail tail_of(const Run& r, const Piece& p)
{
    Tail t{};
    if (p.step == 0 && p.end < p.steps) {
        t.last = r.from - r.off + COST + p.steps - 1;
        t.per = r.per;
        t.token = p.seq.first;
        t.row0 = p.tile * M;
        t.rows = p.rows;
        t.head = p.head;
    }
    return t;
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Weights are exp2(score - reference), the reference 2^kLift under the maximum that is
// in use: fp16 has no normal numbers under 2^-14, and of a row whose first key leads
// all others by 2^25 nothing but that key would be left in the product with v (a lead of
// 2^24.5 over 16384 keys took a fifth of the result).  MOST: weights are 2^MOST at most
// relative to the maximum, and 2^15 in all.  bf16 has the exponents of fp32.
template <int DT, int MOST>
TSX_HD constexpr float lift() { return DT == TSX_F16 ? 15 - MOST : 0; }
// Rounded up, so that no weight is larger.
__device__ __forceinline__ float reference(float top, float under) { return __fsub_ru(top, under); }

// The tensor cores add with truncation: N products one after the other lose some N
// 2^-23.5 of their sum (0.6 % of 1M keys alike in weight, 2.3 % of 4M).  So after every
// kFold products of a piece a thread adds its sums to others that it keeps in the scratch,
// where fp32 rounds to nearest: its row there has `fours` fours of sums, then a sum of
// weights and its reference, for each of the thread's rows.  What is lost is 2^-13.5 of a
// result whatever the length.
constexpr int kFold = 1024;

template <int THREADS, int FOURS>
__device__ __forceinline__ float4* folded_at(const AttendArgs& a)
{
    return a.folded + static_cast<int64_t>(blockIdx.x) * THREADS * (FOURS + 1) + threadIdx.x;
}

// By which sums of the reference `top` are scaled to the reference `now`.
__device__ __forceinline__ float refer(float top, float now) { return top == -INFINITY ? 0.f : exp2_fast(top - now); }

// Row `row` of a sequence's rows of a head: element of q or out.
__device__ __forceinline__ int64_t row_at(const AttendArgs& a, int first, int head, int row, int64_t pitch,
                                          int64_t head_pitch)
{
    const int t = row / a.group;
    return (first + t) * pitch + (head * a.group + row - t * a.group) * head_pitch;
}

__device__ __forceinline__ void store_lse(const AttendArgs& a, int first, int head, int row, float top, float sum)
{
    const int t = row / a.group;
    if (a.lse)
        a.lse[static_cast<int64_t>(first + t) * a.heads * a.group + head * a.group + row - t * a.group] =
            sum > 0.f || sum != sum ? top * 0.69314718055994531f + logf(sum) : -INFINITY;
}

// Two fp32 values into one word of the element type.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    if constexpr (DT == TSX_BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    } else {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}

// Whether a word of two elements holds an infinity or a NaN.
template <int DT>
__device__ __forceinline__ bool not_finite(uint32_t w)
{
    const uint32_t e = DT == TSX_BF16 ? 0x7f80u : 0x7c00u;
    return (w & e) == e || (w >> 16 & e) == e;
}

}  // namespace dev

// What a part's statistics add: its factor relative to the maximum `m`, and its
// share of the sum of weights.  A part that has seen nothing has no weight, and
// zeros for sums; a sum of weights that is NaN stays it.
__device__ __forceinline__ float part_factor(float2 s, float m, float* add)
{
    const bool none = s.x == -INFINITY && s.y == s.y;
    const float f = none ? 0.f : s.x == -INFINITY ? s.y : dev::exp2_fast(s.x - m);
    *add = none ? 0.f : s.y * f;
    return f;
}

// Joins the parts of the tile that CTA blockIdx.x has begun and not ended, of few
// rows and many parts: WARPS warps to ROWS rows, which they share evenly, so that a
// row's parts are one warp's or those of several warps that take them in turn.
// Statistics are read a lane to a part, so that the sums of values do not wait for
// one another: one sequence of 100003 keys and two heads, 152 parts to a head, 13 us
// in place of 72 part after part.
template <int DT, int D, int M, int ROWS, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) attend_join_kernel(const __grid_constant__ AttendArgs a)
{
    using namespace dev;
    constexpr int kEach = D / 32, kAtOnce = 32 / kEach;   // channels to a lane, parts in flight
    __shared__ float sums[WARPS][D];
    __shared__ float2 tops[WARPS];
    wait_for_last();
    const Tail t = a.tails[blockIdx.x];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, row0 = blockIdx.y * ROWS;
    const int rows = min(ROWS, t.rows - row0);
    const int follow = t.follow(blockIdx.x);
    if (!follow || rows <= 0)
        return;
    int share = 1;   // warps to a row
    while (2 * share * rows <= WARPS)
        share *= 2;
    const int row = row0 + warp / share, parts = follow + 1;
    const bool live = row < row0 + rows;
    const int first = 2 * blockIdx.x + 1;   // then the first slots of the CTAs that follow
    // running maximum and sums over 32 of the warp's parts at a time
    float m = -INFINITY, l = 0.f, v[kEach] = {};
    for (int i0 = warp % share; live && i0 < parts; i0 += 32 * share) {
        const int mine = i0 + lane * share;
        const int64_t slot = mine ? first - 1 + 2 * static_cast<int64_t>(mine) : first;
        float2 s = make_float2(-INFINITY, 0.f);
        if (mine < parts)
            s = a.stats[slot * M + row];
        float most = s.x;
#pragma unroll
        for (int k = 16; k > 0; k /= 2)
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, k));
        const float now = fmaxf(m, most);
        const float old = m == -INFINITY ? 1.f : exp2_fast(m - now);
        float add;
        const float f = part_factor(s, now, &add);
#pragma unroll
        for (int k = 16; k > 0; k /= 2)
            add += __shfl_xor_sync(0xffffffffu, add, k);
        l = l * old + add;
        m = now;
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            v[e] *= old;
        const int n = min(32, (parts - i0 + share - 1) / share);
        for (int k0 = 0; k0 < n; k0 += kAtOnce) {
            float2 o[kAtOnce][kEach / 2];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                if (k0 + k >= n)
                    continue;
                const int part = i0 + (k0 + k) * share;
                const int64_t at = part ? first - 1 + 2 * static_cast<int64_t>(part) : first;
                const float* p = a.parts + (at * M + row) * D + lane * kEach;
#pragma unroll
                for (int e = 0; e < kEach / 2; ++e)
                    o[k][e] = *reinterpret_cast<const float2*>(p + 2 * e);
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const float g = __shfl_sync(0xffffffffu, f, (k0 + k) & 31);
                if (k0 + k < n)
#pragma unroll
                    for (int e = 0; e < kEach / 2; ++e) {
                        v[2 * e] += o[k][e].x * g;
                        v[2 * e + 1] += o[k][e].y * g;
                    }
            }
        }
    }
    if (share > 1) {
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            sums[warp][lane * kEach + e] = v[e];
        if (lane == 0)
            tops[warp] = make_float2(m, l);
        __syncthreads();
        if (!live || warp % share)
            return;
        const float2 own = make_float2(m, l);
        for (int w = 1; w < share; ++w)
            m = fmaxf(m, tops[warp + w].x);
        const float f = part_factor(own, m, &l);
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            v[e] *= f;
        for (int w = 1; w < share; ++w) {
            float add;
            const float g = part_factor(tops[warp + w], m, &add);
            l += add;
#pragma unroll
            for (int e = 0; e < kEach; ++e)
                v[e] += sums[warp + w][lane * kEach + e] * g;
        }
    }
    if (!live)
        return;
    const float f = l > 0.f || l != l ? 1.f / l : 0.f;
    char* to = a.out + (row_at(a, t.token, t.head, t.row0 + row, a.out_pitch, a.out_head) + lane * kEach) * 2;
#pragma unroll
    for (int e = 0; e < kEach; e += 2)
        if (lane * kEach + e < a.dim)
            *reinterpret_cast<uint32_t*>(to + e * 2) = pack2<DT>(v[e] * f, v[e + 1] * f);
    if (lane == 0)
        store_lse(a, t.token, t.head, t.row0 + row, m, l);
}

// The same of many rows and, as a rule, two or three parts: a warp to four rows, 32
// rows to a CTA.
constexpr int kJoinMany = 32;

template <int DT, int D, int M>
__global__ void __launch_bounds__(256) attend_join_many_kernel(const __grid_constant__ AttendArgs a)
{
    using namespace dev;
    constexpr int kEach = D / 32, kRowsAtOnce = 4;
    wait_for_last();
    const Tail t = a.tails[blockIdx.x];
    const int lane = threadIdx.x % 32, row0 = blockIdx.y * kJoinMany + threadIdx.x / 32 * kRowsAtOnce;
    const int follow = t.follow(blockIdx.x);
    if (!follow || row0 >= t.rows)
        return;
    float m[kRowsAtOnce], l[kRowsAtOnce], v[kRowsAtOnce][kEach] = {};
#pragma unroll
    for (int r = 0; r < kRowsAtOnce; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
    }
#pragma unroll 2
    for (int i = 0; i <= follow; ++i) {
        const int64_t at = (2 * static_cast<int64_t>(blockIdx.x) + (i ? 2 * i : 1)) * M + row0;
        float2 s[kRowsAtOnce], o[kRowsAtOnce][kEach / 2];
#pragma unroll
        for (int r = 0; r < kRowsAtOnce; ++r) {   // all rows of a slot are there to be read
            s[r] = a.stats[at + r];
#pragma unroll
            for (int e = 0; e < kEach / 2; ++e)
                o[r][e] = *reinterpret_cast<const float2*>(a.parts + (at + r) * D + lane * kEach + 2 * e);
        }
#pragma unroll
        for (int r = 0; r < kRowsAtOnce; ++r) {
            if (row0 + r >= t.rows)   // what was never written
                continue;
            const float now = fmaxf(m[r], s[r].x), old = m[r] == -INFINITY ? 1.f : exp2_fast(m[r] - now);
            float add;
            const float f = part_factor(s[r], now, &add);
            l[r] = l[r] * old + add;
            m[r] = now;
#pragma unroll
            for (int e = 0; e < kEach / 2; ++e) {
                v[r][2 * e] = v[r][2 * e] * old + o[r][e].x * f;
                v[r][2 * e + 1] = v[r][2 * e + 1] * old + o[r][e].y * f;
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRowsAtOnce; ++r) {
        if (row0 + r >= t.rows)
            continue;
        const float f = l[r] > 0.f || l[r] != l[r] ? 1.f / l[r] : 0.f;
        char* to = a.out + (row_at(a, t.token, t.head, t.row0 + row0 + r, a.out_pitch, a.out_head) + lane * kEach) * 2;
#pragma unroll
        for (int e = 0; e < kEach; e += 2)
            if (lane * kEach + e < a.dim)
                *reinterpret_cast<uint32_t*>(to + e * 2) = pack2<DT>(v[r][e] * f, v[r][e + 1] * f);
        if (lane == 0)
            store_lse(a, t.token, t.head, t.row0 + row0 + r, m[r], l[r]);
    }
}

}  // namespace tsx

// Attention over a paged cache for many rows to a head, on the tensor cores.
//
// A CTA goes over two tiles of 128 rows at once, 128 keys to a step.  Per step and
// tile: S = q k^T (both operands in shared memory), weights P = exp2(S scale - m),
// O += P v with P as an operand in tensor memory, in the place of S.  The products
// of one tile run while the other's weights are computed, so that neither the
// tensor cores nor the exponentials wait for the other: 2 x 128^3 multiply-adds a
// step and tile are 1024 cycles at 4096 a cycle, 128^2 exponentials 512 at 32.
//
//   warps 0-3, 4-7   a tile each, a thread to a row: scores, maxima, weights, sums,
//                    results (nothing between threads)
//   warp 8           brings keys and values, by TMA: boxes of the pages, one to a
//                    lane; and tells which of the step's keys exist
//   warps 9, 10      bring queries, and look through values that not every row sees
//   warp 11          issues the products
//
// Pages that are no power of two of at least 8 slots do not fit the swizzle's eight
// rows: then warps 8 and 9 bring everything by cp.async.
//
// The running maximum is not followed closely: O and the sum are scaled only when
// a row's maximum has grown by more than 2^8 over the one in use, which is rare
// after the first steps; weights are then up to 2^8 (2^15 in fp16, where they are
// taken 2^7 larger), with the same relative error.
// Weights are rounded into the element type for the product with v, by up to 2^-8 (bf16)
// or 2^-11 of each, their sum is not: relative to the result's norm the error is 2.3e-3
// where fp32 weights have 1.66e-3 (bf16; fp16 2.6e-4 and 2.1e-4).  What rounding leaves
// in a product of its own would be half as many products again, in a kernel that they
// bound.
//
// Every wait gives up after kPatience; then the CTA's remaining rows become NaN.  Waits
// that may be for a whole piece (of the queries' warps) or several (of a second tile's,
// for a piece that has one) go on for as long as steps are brought.
//
// Measured on GB300 as in the kernel for few rows; in parentheses the time of the
// products at the 1897 TFLOP/s of cuBLAS.  bf16, chunks of 1024 tokens of two prompts of
// 16384 and 13000, 32 heads over 8 of 128, pages of 32: 241 us (192), 1.51 PFLOP/s; the
// products alone would take 150 of them at the tensor cores' 4096 multiply-adds a
// cycle.  With heads of 64 channels 198 (96): the exponentials are as many; of 72, 80 and
// 96 233, 234 and 237 (108, 120, 144): products are those of 128.  A ragged batch of 12 (1
// to 300 new tokens, up to 3000 keys, f16, 10 heads over 2 of 64): 27, most of it the start
// and end of pieces of five steps and their joins.
// Steps that led here, for the first of them: mma.m16n8k16 2316 us; tcgen05 from one
// thread, cp.async loads 489; an elected lane 464; loads with few shuffles 371; four
// threads to a row and boxes of pages 337; one thread to a row 287; short code for what
// runs once 257; a tile's start and end counted as work 247; the weights of half a step
// handed over while the others are computed 240.  What bounds a step now (2600 cycles
// for two tiles): a tile's chain of scores, weights and products, 1260 + 1024 cycles
// and the hand-overs between them.
// Waits that poll without a pause, and weights taken before their maximum is known,
// were slower.

#include "tsx_attend.cuh"
#include "tsx_tcgen05.cuh"

namespace tsx {
namespace {

using namespace dev;

constexpr int kHalf = 128, kRows = 2 * kHalf, kKeys = 128;
constexpr int kWeighers = 256, kLoaders = 64, kThreads = 384;
// What a tile costs beside its steps, in steps, and units to a CTA at least.  The
// ragged batch above takes 33.6 us with a cost of 0, 29.2 with 2, 26.8 with 3, 27.7 with 4;
// the large one 250, 247, 243, 245.
constexpr int kCost = 3;
constexpr int64_t kLeast = 4;
constexpr int kMasks = 8;            // steps whose keys are remembered
constexpr int kBlock = kKeys * 128;  // bytes of a block: 128 rows of 64 channels
constexpr int kLag = 2;              // groups of loads in flight behind the last
constexpr int kFoldSteps = kFold / (kKeys / 16);
constexpr float kGrowth = 8.f;
// Scores (times 1 / ln 2) from which on half a step of fp32, 2^-4, is too much between a
// rounded score, which the reference is, and the exact one of an fma.
constexpr float kFar = 0x1p20f;
constexpr uint64_t kPatience = 4000000000ull;   // ns
constexpr int kLoadWarp = kWeighers / 32, kIssueWarp = kLoadWarp + 3;

// Keys or values of a step take a stage.  One CTA to an SM, which is what the
// tensor memory is for: the stages of D = 64 are as many as keep a second one out.
template <int D>
TSX_HD constexpr int stages() { return D == 128 ? 4 : 8; }

template <int D>
struct Shared {
    static constexpr int kTile = D / 64 * kBlock;   // bytes of 128 rows
    static constexpr int kQ = 0, kRing = 2 * kTile, kStore = kRing + stages<D>() * kTile,
                         kEnd = kStore + kWeighers / 32 * 4096;   // kStore: results on their way out
    // barriers
    static constexpr int kFull = kEnd, kEmpty = kFull + 8 * stages<D>(), kQFull = kEmpty + 8 * stages<D>(),
                         kQEmpty = kQFull + 8, kS = kQEmpty + 8, kP = kS + 16, kO = kP + 32,
                         kReset = kO + 16, kDrain = kReset + 8, kRaw = kDrain + 8;
    static constexpr int kMask = (kRaw + 8 * stages<D>() + 15) / 16 * 16;                 // [kMasks][4] words
    static constexpr int kOdd = kMask + kMasks * 16;      // [3][D] first keys with a NaN, +inf, -inf
    static constexpr int kSums = kOdd + 3 * D * 4;        // words of run_of
    static constexpr int kWords = kSums + (kThreads / 32 + 3) * 8;   // tensor memory, first tiles done, odd values met, second tiles done
    static constexpr int kBrought = kWords + 16;          // steps of which loads have been issued
    static constexpr int kBytes = kBrought + 16;
};

// False once nothing has been brought since the last time that this was asked.
template <int D>
__device__ __forceinline__ bool goes_on(uint32_t mem, uint32_t& seen)
{
    const uint32_t before = seen;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(seen) : "r"(mem + Shared<D>::kBrought) : "memory");
    return seen != before;
}
template <int D>
__device__ __forceinline__ void brought(uint32_t mem, uint32_t steps)
{
    asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(mem + Shared<D>::kBrought), "r"(steps) : "memory");
}

__device__ __forceinline__ bool wait(uint32_t bar, uint32_t phase) { return mbar_wait(bar, phase & 1, kPatience); }
// The same answer for all threads of the warp.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t phase)
{
    return __all_sync(0xffffffffu, wait(bar, phase));
}
// Where the wait may be for more than the ring's steps: for as long as steps are brought.
// Two forms of it, the first where a step's time shows (the large chunk above takes 240.7
// us, 239.5 with no such wait, 242.6 with the first form in both places, 247 and 259 with
// either in every wait).
template <int D>
__device__ __forceinline__ bool wait_on(uint32_t mem, int bar, uint32_t phase)
{
    bool done = true;
    if (!mbar_try_wait(mem + bar, phase & 1)) {
        uint64_t since = globaltimer_ns();
        uint32_t seen = ~0u;
#pragma unroll 1
        while (done && !mbar_try_wait(mem + bar, phase & 1))
            if (globaltimer_ns() - since > kPatience) {
                done = goes_on<D>(mem, seen);
                since = globaltimer_ns();
            }
    }
    return __all_sync(0xffffffffu, done);
}
template <int D>
__device__ __forceinline__ bool wait_long(uint32_t mem, int bar, uint32_t phase)
{
    uint32_t seen = ~0u;
    while (!wait_warp(mem + bar, phase))
        if (!__all_sync(0xffffffffu, goes_on<D>(mem, seen)))
            return false;
    return true;
}

// w's two values times 0, and sum.
template <int DT>
__device__ __forceinline__ uint32_t times_zero(uint32_t w, uint32_t sum)
{
    if constexpr (DT == TSX_BF16)
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(w) : "r"(w), "r"(0), "r"(sum));
    else
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(w) : "r"(w), "r"(0), "r"(sum));
    return w;
}

// ------------------------------------------------------------------ loads

// A place in the ring of stages.
template <int D>
struct Place {
    int stage = 0;
    uint32_t turn = 0;   // how often the ring has been gone round
    __device__ __forceinline__ void next()
    {
        if (++stage == stages<D>()) {
            stage = 0;
            ++turn;
        }
    }
};

// What a group of loads announces when it has landed: a barrier, and for values
// that some rows do not see, where they lie.
struct Landing {
    uint32_t bar;
    int stage;   // bytes from the shared memory's start
    int base;    // position of the step's first key
    bool check;
};

// Values of keys that not every row sees: 0 times an infinity or a NaN would reach
// the rows that do not.  Such values are taken out, and the first key of each kind
// is kept for each channel; the rows from that key on get it added at the end.
// tile: the values' tile; base: the position of its first key.
template <int DT, int D>
__device__ __noinline__ void take_out(unsigned char* memory, unsigned char* tile, int row, int chunk, int base)
{
    int* odd = reinterpret_cast<int*>(memory + Shared<D>::kOdd);
    uint16_t* at =
        reinterpret_cast<uint16_t*>(tile + chunk / 8 * kBlock + row * 128 + ((chunk & 7) ^ (row & 7)) * 16);
    for (int e = 0; e < 8; ++e) {
        const uint32_t w = at[e];
        if (!not_finite<DT>(w))
            continue;
        const bool nan = w & (DT == TSX_BF16 ? 0x7fu : 0x3ffu);
        atomicMin(odd + (nan ? 0 : w >> 15 ? 2 : 1) * D + chunk * 8 + e, base + row);
        at[e] = 0;
        reinterpret_cast<int*>(memory + Shared<D>::kWords)[2] = 1;
    }
}

// Chunk i of a thread's chunks of a tile is that of `row(i)` and `chunk(i)`; `keys`
// of the tile's rows are keys, the others become zeros.  0 times a value is 0 or NaN,
// which a sum keeps: eight values are looked at in four instructions.
template <int DT, int D, int N, class Row, class Chunk>
__device__ __forceinline__ void look_through(unsigned char* memory, unsigned char* tile, int base, int keys, Row row,
                                             Chunk chunk)
{
    const auto place = [&](int i) {
        return reinterpret_cast<uint4*>(tile + chunk(i) / 8 * kBlock + row(i) * 128 + ((chunk(i) & 7) ^ (row(i) & 7)) * 16);
    };
    uint32_t sum = 0;
    for (int i0 = 0; i0 < N; i0 += 8) {
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (row(i0 + i) < keys)
                v[i] = *place(i0 + i);
            else
                *place(i0 + i) = v[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum = times_zero<DT>(v[i].w, times_zero<DT>(v[i].z, times_zero<DT>(v[i].y, times_zero<DT>(v[i].x, sum))));
    }
    if (sum & 0x7fff7fffu)   // not 0 or -0
        for (int i = 0; i < N; ++i)
            if (row(i) < keys)
                take_out<DT, D>(memory, tile, row(i), chunk(i), base);
}

// Before the first such values of a piece: nothing has been taken out.  False if
// the last piece's rows have not used what was: every piece before has a first
// tile, `seconds` of them a second one, and the warps of a tile count for themselves
// (those of a second tile that is not there run ahead, and must not stand in for
// the first's).
template <int D>
__device__ __forceinline__ bool forget(unsigned char* memory, uint32_t piece, uint32_t seconds, uint32_t resets,
                                       int mine)
{
    using S = Shared<D>;
    constexpr int kTileWarps = kHalf / 32;
    const volatile int* words = reinterpret_cast<const int*>(memory + S::kWords);
    int* odd = reinterpret_cast<int*>(memory + S::kOdd);
    if (piece) {
        const uint64_t since = globaltimer_ns();
        while (!__all_sync(0xffffffffu, words[1] >= static_cast<int>(kTileWarps * piece) &&
                                            words[3] >= static_cast<int>(kTileWarps * seconds)))
            if (__any_sync(0xffffffffu, globaltimer_ns() - since > kPatience))
                return false;
        __threadfence_block();
    }
    for (int i = mine; i < 3 * D; i += kLoaders)
        odd[i] = 0x7fffffff;
    if (mine == 0)
        reinterpret_cast<int*>(memory + S::kWords)[2] = 0;
    mbar_arrive(smem_addr(memory) + S::kReset);
    return wait_warp(smem_addr(memory) + S::kReset, resets);
}

template <int DT, int D>
__device__ __forceinline__ void land(unsigned char* memory, const Landing& l)
{
    if (l.check) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x / 32 & 1;   // the chunks that this thread has copied
        look_through<DT, D, D / 4>(
            memory, memory + l.stage, l.base, kKeys, [=](int i) { return warp * 64 + i % 16 * 4 + lane / 8; },
            [=](int i) { return i / 16 * 8 + lane % 8; });
    }
    fence_proxy_async_smem();
    mbar_arrive(l.bar);
}

// 32 rows, whose elements start at `at` (bytes; < 0: zeros) of lane's row, into a
// tile from its row `row0` on.  Eight lanes copy 128 bytes of a row, so that a row's
// place is asked for once for both of its halves.
template <int D>
__device__ __forceinline__ void load_rows(const char* base, int64_t at, int dim, uint32_t tile, int row0)
{
    const int lane = threadIdx.x & 31, chunk = lane & 7, first = lane >> 3;
    const uint32_t to[2] = {tile + (row0 + first) * 128 + ((chunk ^ first) * 16),
                            tile + (row0 + first) * 128 + ((chunk ^ (4 + first)) * 16)};
    base += chunk * 16;
    if (dim == D && __all_sync(0xffffffffu, at >= 0)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const char* from = base + __shfl_sync(0xffffffffu, at, 4 * j + first);
#pragma unroll
            for (int half = 0; half < D / 64; ++half)
                cp_async_whole(to[j & 1] + half * kBlock + j * 512, from + half * 128);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t from = __shfl_sync(0xffffffffu, at, 4 * j + first);
#pragma unroll
        for (int half = 0; half < D / 64; ++half) {
            const uint32_t bytes = from >= 0 && half * 64 + chunk * 8 < dim ? 16 : 0;
            cp_async(to[j & 1] + half * kBlock + j * 512, base + (bytes ? from + half * 128 : 0), 16, bytes);
        }
    }
}

// Half of the queries of both tiles.
template <int D>
__device__ __forceinline__ void load_queries(const AttendArgs& a, const Piece& p, uint32_t mem, int which)
{
    using S = Shared<D>;
    for (int t = 0; t < (p.rows > kHalf ? 2 : 1); ++t)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int in_tile = which * 64 + g * 32, row = t * kHalf + in_tile + static_cast<int>(threadIdx.x & 31);
            const int64_t at =
                row < p.rows ? row_at(a, p.seq.first, p.head, p.tile * kRows + row, a.q_pitch, a.q_head) * 2 : -1;
            load_rows<D>(a.q, at, a.dim, mem + S::kQ + t * S::kTile, in_tile);
        }
}

// Keys and values in boxes of the pages.  A barrier of its own (kRaw) for values
// that helper() looks through before it announces them.  Copies in flight where this
// gives up have been for all of kPatience.
template <int D>
__device__ __forceinline__ void boxes(const AttendArgs& a, Run run, unsigned char* memory, const CUtensorMap* keys,
                                      const CUtensorMap* values)
{
    using S = Shared<D>;
    const uint32_t mem = smem_addr(memory);
    const int lane = threadIdx.x & 31, rows = min(a.paged.page_size, kKeys), n = kKeys / rows;
    const int mine = lane % n, half = lane / n;   // the page and the channels of the lane's box
    const bool active = half < D / 64;
    const uint32_t to = mem + S::kRing + half * kBlock + mine * rows * 128;
    Place<D> place;
    uint32_t count = 0;   // steps of all pieces
    while (run.from < run.to) {
        const Piece p = piece_of<kRows, kKeys, kCost>(a, run);
        if (p.empty())
            break;   // the run's last units, before a tile's first step
        const int first_limit = row_limit(a, p.seq, p.tile * kRows);
        const int limit = min(row_limit(a, p.seq, p.tile * kRows + p.rows - 1), p.seq.length);
        const int32_t* pages = a.paged.pages + p.b * a.paged.pages_pitch;
        int position = p.step * kKeys + mine * rows;
        int page = position < limit ? pages[page_of(a.paged, position)] : -1;
        for (int step = p.step; step < p.end; ++step, ++count) {
            const int base = step * kKeys, slot = position & (a.paged.page_size - 1);
            const bool there = page >= 0 && page < a.paged.cache_pages;
            const uint32_t exist = __ballot_sync(0xffffffffu, there);
            const int box = there ? page : static_cast<int>(a.paged.cache_pages);   // beyond the tensor: zeros
            uint4 seen = make_uint4(~0u, ~0u, ~0u, ~0u);
            if (exist != ~0u || base + kKeys > limit) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = i * 32 + lane;
                    w[i] = __ballot_sync(0xffffffffu, (exist >> (key / rows) & 1) && base + key < limit);
                }
                seen = make_uint4(w[0], w[1], w[2], w[3]);
            }
            if (lane == 0) {   // the step that had this place is long over: its values' stage has been used again
                *reinterpret_cast<uint4*>(memory + S::kMask + count % kMasks * 16) = seen;
                brought<D>(mem, count);
            }
            position += kKeys;
            page = position < limit ? pages[page_of(a.paged, position)] : -1;   // a step ahead
#pragma unroll
            for (int kv = 0; kv < 2; ++kv, place.next()) {
                if (place.turn && !wait_warp(mem + S::kEmpty + 8 * place.stage, place.turn - 1))
                    return;
                const bool look = kv == 1 && base + kKeys > first_limit;
                const uint32_t bar = mem + 8 * place.stage + (look ? S::kRaw : S::kFull);
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, S::kTile);
                    if (!look)   // as the helper's two warps
                        mbar_arrive(bar);
                }
                __syncwarp();
                if (active)
                    tma_load_4d(to + place.stage * S::kTile, kv ? values : keys, half * 64, slot, p.head, box, bar);
            }
        }
        advance<kRows>(a, run, p);
    }
}

// Queries; and values that not every row sees: those that no row sees become zeros,
// for the rest see take_out.
template <int DT, int D>
__device__ __forceinline__ void helper(const AttendArgs& a, Run run, unsigned char* memory)
{
    using S = Shared<D>;
    const uint32_t mem = smem_addr(memory);
    const int mine = threadIdx.x - (kLoadWarp + 1) * 32;
    uint32_t piece = 0, seconds = 0, resets = 0, tile = 0, raw = 0;   // raw: a bit to each stage, the phase to wait for
    while (run.from < run.to) {
        const Piece p = piece_of<kRows, kKeys, kCost>(a, run);
        if (p.empty())
            break;   // the run's last units, before a tile's first step
        if (piece && !wait_long<D>(mem, S::kQEmpty, piece - 1))
            return;
        load_queries<D>(a, p, mem, mine / 32);
        cp_async_commit();
        cp_async_wait(0);
        fence_proxy_async_smem();
        mbar_arrive(mem + S::kQFull);
        const int first_limit = row_limit(a, p.seq, p.tile * kRows);
        const int limit = min(row_limit(a, p.seq, p.tile * kRows + p.rows - 1), p.seq.length);
        bool fresh = true;
        for (int step = max(p.step, first_limit / kKeys); step < p.end; ++step) {   // base + kKeys > first_limit
            if (fresh && !forget<D>(memory, piece, seconds, resets++, mine))
                return;
            fresh = false;
            const int stage = (tile + 2 * (step - p.step) + 1) % stages<D>(), base = step * kKeys;
            if (!wait_long<D>(mem, S::kRaw + 8 * stage, raw >> stage))
                return;
            raw ^= 1u << stage;
            unsigned char* values = memory + S::kRing + stage * S::kTile;
            constexpr int kChunks = D / 8;
            look_through<DT, D, kKeys * kChunks / kLoaders>(
                memory, values, base, limit - base, [=](int i) { return i * (kLoaders / kChunks) + mine / kChunks; },
                [=](int) { return mine % kChunks; });
            fence_proxy_async_smem();
            __syncwarp();
            if (mine % 32 == 0)
                mbar_arrive(mem + S::kFull + 8 * stage);
        }
        tile += 2 * (p.end - p.step);
        ++piece;
        seconds += p.rows > kHalf;
        advance<kRows>(a, run, p);
    }
}

// Everything by cp.async.
template <int DT, int D>
__device__ __forceinline__ void loader(const AttendArgs& a, Run run, unsigned char* memory)
{
    using S = Shared<D>;
    const uint32_t mem = smem_addr(memory);
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32 & 1, mine = threadIdx.x % kLoaders;
    uint32_t piece = 0, seconds = 0, resets = 0, count = 0;   // count: steps of all pieces
    Place<D> place;
    Landing pending[kLag];
    int waiting = 0;   // of `pending`
    const auto put = [&](const Landing& l) {
        cp_async_commit();
        if (waiting == kLag) {
            cp_async_wait(kLag);
            land<DT, D>(memory, pending[0]);
#pragma unroll
            for (int i = 0; i + 1 < kLag; ++i)
                pending[i] = pending[i + 1];
            pending[kLag - 1] = l;
        } else {
#pragma unroll
            for (int i = 0; i < kLag; ++i)
                if (i == waiting)
                    pending[i] = l;
            ++waiting;
        }
    };
    const auto flush = [&] {
        cp_async_wait(0);
#pragma unroll
        for (int i = 0; i < kLag; ++i)
            if (i < waiting)
                land<DT, D>(memory, pending[i]);
        waiting = 0;
    };
    while (run.from < run.to) {
        const Piece p = piece_of<kRows, kKeys, kCost>(a, run);
        if (p.empty())
            break;   // the run's last units, before a tile's first step
        if (piece && !wait_warp(mem + S::kQEmpty, piece - 1))
            return;
        load_queries<D>(a, p, mem, warp);
        put(Landing{mem + S::kQFull, 0, 0, false});
        const int first_limit = row_limit(a, p.seq, p.tile * kRows);
        const int limit = min(row_limit(a, p.seq, p.tile * kRows + p.rows - 1), p.seq.length);
        const int32_t* pages = a.paged.pages + p.b * a.paged.pages_pitch;
        int position = p.step * kKeys + warp * 64 + lane;   // and 32 further on
        int page[2];
#pragma unroll
        for (int g = 0; g < 2; ++g)
            page[g] = position + 32 * g < limit ? pages[page_of(a.paged, position + 32 * g)] : -1;
        bool fresh = true;   // no value of the piece has been looked at
        for (int step = p.step; step < p.end; ++step, ++count) {
            int64_t at[2];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const bool there = page[g] >= 0 && page[g] < a.paged.cache_pages;
                const int here = position + 32 * g, slot = here - page_of(a.paged, here) * a.paged.page_size;
                at[g] = there ? (page[g] * a.paged.page_pitch + slot * a.slot_pitch + p.head * a.head_pitch) * 2 : -1;
                const uint32_t seen = __ballot_sync(0xffffffffu, there);
                if (lane == 0)   // the step that had this place is long over: its values' stage has been used again
                    reinterpret_cast<uint32_t*>(memory + S::kMask)[count % kMasks * 4 + warp * 2 + g] = seen;
                page[g] = here + kKeys < limit ? pages[page_of(a.paged, here + kKeys)] : -1;   // a step ahead
            }
            position += kKeys;
            if (mine == 0)
                brought<D>(mem, count);
            const int base = step * kKeys;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv, place.next()) {
                if (place.turn && !wait_warp(mem + S::kEmpty + 8 * place.stage, place.turn - 1))
                    return;
                const bool check = kv == 1 && base + kKeys > first_limit;
                if (check && fresh) {   // the last piece's have been used
                    fresh = false;
                    if (!forget<D>(memory, piece, seconds, resets++, mine))
                        return;
                }
                const int stage = S::kRing + place.stage * S::kTile;
#pragma unroll
                for (int g = 0; g < 2; ++g)
                    load_rows<D>(kv ? a.v : a.k, at[g], a.dim, mem + stage, warp * 64 + g * 32);
                put(Landing{mem + S::kFull + 8 * place.stage, stage, base, check});
            }
        }
        flush();
        ++piece;
        seconds += p.rows > kHalf;
        advance<kRows>(a, run, p);
    }
}

// --------------------------------------------------------------- products

template <int DT, int D, bool FOLD>
__device__ __forceinline__ void issuer(const AttendArgs& a, Run run, unsigned char* memory, uint32_t tmem)
{
    using S = Shared<D>;
    const uint32_t mem = smem_addr(memory);
    const uint32_t scores = product(DT == TSX_BF16, 128, kKeys, false, a.negated);
    const uint32_t values = product(DT == TSX_BF16, 128, D, true, false);
    uint32_t piece = 0, weights[2] = {0, 0};
    Place<D> place;
    const auto full = [&](const Place<D>& at) { return wait_warp(mem + S::kFull + 8 * at.stage, at.turn); };
    const auto release = [&](const Place<D>& at) { mma_commit(mem + S::kEmpty + 8 * at.stage); };
    const auto score = [&](int t, const Place<D>& at) {
        const uint32_t q = mem + S::kQ + t * S::kTile, k = mem + S::kRing + at.stage * S::kTile;
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
            mma_smem64(tmem + t * kHalf, operand(q + i * kBlock, 16), operand(k + i * kBlock, 16), scores, i > 0);
        mma_commit(mem + S::kS + 8 * t);
    };
    while (run.from < run.to) {
        const Piece p = piece_of<kRows, kKeys, kCost>(a, run);
        if (p.empty())
            break;   // the run's last units, before a tile's first step
        const int tiles = p.rows > kHalf ? 2 : 1, steps = p.end - p.step;
        if (!wait_warp(mem + S::kQFull, piece) || !full(place))
            return;
        tcgen05_after();
        for (int t = 0; t < tiles; ++t)
            score(t, place);
        release(place);
        if (steps == 1)
            mma_commit(mem + S::kQEmpty);
        for (int i = 0; i < steps; ++i) {
            place.next();
            const Place<D> values_at = place;
            if (!full(values_at))
                return;
            const bool more = i + 1 < steps;
            place.next();
            for (int t = 0; t < tiles; ++t) {
                const uint32_t v = mem + S::kRing + values_at.stage * S::kTile;
#pragma unroll
                for (int k = 0; k < kKeys / 64; ++k) {   // as the weights come, 64 keys at a time
                    if (!wait_warp(mem + S::kP + 16 * t + 8 * k, weights[t]))
                        return;
                    tcgen05_after();
                    mma_tmem64(tmem + kRows + t * kHalf, tmem + t * kHalf + k * 32, operand(v + k * 8192, kBlock), values,
                               (FOLD ? i % kFoldSteps : i) > 0 || k > 0);
                }
                ++weights[t];
                if (t == tiles - 1)
                    release(values_at);
                if (!more) {
                    mma_commit(mem + S::kO + 8 * t);
                } else {
                    if (t == 0 && !full(place))
                        return;
                    score(t, place);
                }
            }
            if (more) {
                release(place);
                if (i + 2 == steps)
                    mma_commit(mem + S::kQEmpty);
            }
        }
        ++piece;
        advance<kRows>(a, run, p);
    }
}

// ---------------------------------------------------------------- weights

__device__ __forceinline__ float4 add_scaled(float4 a, float4 b, float f)
{
    return make_float4(a.x + b.x * f, a.y + b.y * f, a.z + b.z * f, a.w + b.w * f);
}

// NaN is passed over, as by fmaxf.
__device__ __forceinline__ float max3(float a, uint32_t b, uint32_t c)
{
    float m;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
    return m;
}

// Results go out through shared memory, 128 bytes of a row at a time: rows lie far
// apart, and stores of 16 bytes to each of 32 rows took 5 to 20 us for a tile.
// N words of the thread's row, from its 16-byte chunk `first` of 8 on; chunk c of
// row r at place c ^ (r & 7).  place: of the warp's 4096 bytes.
template <int N>
__device__ __forceinline__ void stage_words(uint4* place, const uint32_t* w, int first)
{
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
        place[lane * 8 + ((first + i) ^ (lane & 7))] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

// Rows of the warp, at `to` of each lane's row, from their byte `from` on; `width`
// bytes of a row exist.
__device__ __forceinline__ void send_rows(const uint4* place, char* to, uint32_t alive, int from, int width)
{
    const int lane = threadIdx.x % 32, chunk = lane % 8;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = i * 4 + lane / 8;
        char* at = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), row));
        const uint4 v = place[row * 8 + (chunk ^ (row & 7))];
        if ((alive >> row & 1) && from + chunk * 16 < width)
            *reinterpret_cast<uint4*>(at + from + chunk * 16) = v;
    }
    __syncwarp();
}

template <int DT, int D, bool FOLD>
__device__ __forceinline__ void weigher(const AttendArgs& a, Run run, unsigned char* memory, uint32_t tmem, Tail* tail)
{
    using S = Shared<D>;
    const uint32_t mem = smem_addr(memory);
    const int t = threadIdx.x / kHalf, row = threadIdx.x % kHalf;   // of the tile
    const uint32_t lanes = static_cast<uint32_t>(row / 32 * 32) << 16;
    const uint32_t s_at = tmem + t * kHalf + lanes, o_at = tmem + kRows + t * kHalf + lanes;
    constexpr float kLift = lift<DT, int(kGrowth)>();
    constexpr int kFours = fold_fours(true, D);
    static_assert(kWeighers == fold_threads(true), "a row of folded sums to each thread");
    const int* odd = reinterpret_cast<const int*>(memory + S::kOdd);
    int* words = reinterpret_cast<int*>(memory + S::kWords);
    uint32_t scored = 0, ended = 0, count = 0;   // count: steps of all pieces
    bool ok = true;
    while (run.from < run.to) {
        const Piece p = piece_of<kRows, kKeys, kCost>(a, run);
        if (p.empty())
            break;   // the run's last units, before a tile's first step
        const int first = p.tile * kRows + t * kHalf;   // of the tile's rows
        const int all = row_limit(a, p.seq, first);     // keys that every row of the tile sees
        const bool live = t * kHalf + row < p.rows, busy = p.rows > t * kHalf;
        const int limit = live ? row_limit(a, p.seq, first + row) : 0;
        float top = -INFINITY, sum = 0.f;   // the weights' reference, and their sum
        bool far = false;                   // the reference is beyond kFar
        for (int step = p.step; busy && ok && step < p.end; ++step) {
            ok = wait_on<D>(mem, S::kS + 8 * t, scored);
            if (!ok)
                break;
            ++scored;
            tcgen05_after();
            if (FOLD && step > p.step && (step - p.step) % kFoldSteps == 0) {   // O is at rest, and begins anew
                asm volatile("" ::: "memory");   // a branch in earnest
                float4* const folded = folded_at<kWeighers, kFours>(a);
                float4 held = make_float4(0.f, -INFINITY, 0.f, 0.f);
                const bool none = step - p.step == kFoldSteps;
                if (!none)
                    held = folded[kFours * kWeighers];
                const float f = refer(held.y, top);
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    uint32_t o[16];
                    tmem_load16(o_at + c, o);
                    tmem_wait16(o);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float4* at = folded + (c / 4 + i) * kWeighers;
                        float4 g = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                               __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
                        if (!none)
                            g = add_scaled(g, *at, f);
                        *at = g;
                    }
                }
                folded[kFours * kWeighers] = make_float4(sum + held.x * f, top, 0.f, 0.f);
                sum = 0.f;
            }
            uint32_t s[kKeys];
#pragma unroll
            for (int c = 0; c < kKeys; c += 32)
                tmem_load32(s_at + c, s + c);
            const int base = step * kKeys;
            const uint4 there = *reinterpret_cast<const uint4*>(memory + S::kMask + (count + (step - p.step)) % kMasks * 16);
#pragma unroll
            for (int c = 0; c < kKeys; c += 32)
                tmem_wait32(s + c);
            if (__any_sync(0xffffffffu, base + kKeys > all || (there.x & there.y & there.z & there.w) != ~0u)) {
                asm volatile("" ::: "memory");   // a branch in earnest: as selections they would be made in every step
                const uint32_t w[4] = {there.x, there.y, there.z, there.w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int left = limit - base - 32 * c;   // keys of these that the row may see
                    const uint32_t sees = w[c] & (left >= 32 ? ~0u : left <= 0 ? 0u : (1u << left) - 1);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (!(sees >> i & 1))
                            s[32 * c + i] = 0xff800000u;
                }
            }
            float m[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                m[j] = __uint_as_float(s[j]);
#pragma unroll
            for (int i = 4; i + 7 < kKeys; i += 8)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    m[j] = max3(m[j], s[i + j], s[i + 4 + j]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                m[j] = fmaxf(m[j], __uint_as_float(s[kKeys - 4 + j]));
            const float now = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * a.scale_log2;
            const bool grows = now - top > kGrowth + kLift;   // not where both are infinite
            float scale = a.scale_log2;
            if (__any_sync(0xffffffffu, grows || far)) {
                const float next = reference(now, kLift), f = grows && top != -INFINITY ? exp2_fast(top - next) : 1.f;
                top = grows ? next : top;
                far = fabsf(top) > kFar && top != -INFINITY;
                sum *= f;
                if (step > p.step && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {   // O is at rest: the scores came after its last product
                        uint32_t o[16];
                        tmem_load16(o_at + c, o);
                        tmem_wait16(o);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_store16(o_at + c, o);
                    }
                }
                if (__any_sync(0xffffffffu, far)) {   // rounded as the maximum is, that their differences are exact
                    asm volatile("" ::: "memory");
#pragma unroll
                    for (int i = 0; i < kKeys; ++i)
                        s[i] = __float_as_uint(__uint_as_float(s[i]) * scale);
                    scale = 1.f;
                }
            }
            const float2 by = pair_of(scale), less = pair_of(top == -INFINITY ? 0.f : -top);
            float2 total[2] = {pair_of(0.f), pair_of(0.f)};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t w[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float2 v = make_float2(__uint_as_float(s[64 * c + 2 * i]), __uint_as_float(s[64 * c + 2 * i + 1]));
                    v = __ffma2_rn(v, by, less);
                    v.x = exp2_fast(v.x);
                    v.y = exp2_fast(v.y);
                    total[i & 1] = __fadd2_rn(total[i & 1], v);
                    w[i] = pack2<DT>(v.x, v.y);
                }
                tmem_store32(s_at + 32 * c, w);
                tmem_wait_stores();
                tcgen05_before();
                mbar_arrive(mem + S::kP + 16 * t + 8 * c);
            }
            const float2 both = __fadd2_rn(total[0], total[1]);
            sum += both.x + both.y;
        }
        if (busy) {
            ok = ok && wait_warp(mem + S::kO + 8 * t, ended++);
            tcgen05_after();
            const bool whole = p.whole();
            const bool strange = ok && p.end * kKeys > row_limit(a, p.seq, p.tile * kRows) && words[2];
            const int64_t slot = part_slot(p);
            const bool more = FOLD && p.end - p.step > kFoldSteps;   // sums have been folded
            const float4* const folded = folded_at<kWeighers, kFours>(a);
            float g = 0.f;
            if (more) {
                const float4 held = folded[kFours * kWeighers];
                g = refer(held.y, top);
                sum += held.x * g;
            }
            sum = ok ? sum : NAN;
            const float f = !whole && ok ? 1.f : sum > 0.f || sum != sum ? 1.f / sum : 0.f;
            char* to = live && whole ? a.out + row_at(a, p.seq.first, p.head, first + row, a.out_pitch, a.out_head) * 2
                                     : reinterpret_cast<char*>(a.parts + (slot * kRows + t * kHalf + row) * D);
            if (live && whole)
                store_lse(a, p.seq.first, p.head, first + row, top, sum);
            if (live && !whole)
                a.stats[slot * kRows + t * kHalf + row] = make_float2(top, sum);
            uint4* place = reinterpret_cast<uint4*>(memory + S::kStore + threadIdx.x / 32 * 4096);
            const int width = whole ? a.dim * 2 : D * 4;   // bytes of a row
            const uint32_t alive = __ballot_sync(0xffffffffu, live);
#pragma unroll 1   // short code: it runs once in a while, and waits for its instructions
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                if (ok)
                    tmem_load32(o_at + c, o);
                tmem_wait32(o);
                if (more)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 v = add_scaled(make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                                __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3])),
                                                    folded[(c / 4 + i) * kWeighers], g);
                        o[4 * i] = __float_as_uint(v.x);
                        o[4 * i + 1] = __float_as_uint(v.y);
                        o[4 * i + 2] = __float_as_uint(v.z);
                        o[4 * i + 3] = __float_as_uint(v.w);
                    }
                if (strange)
#pragma unroll 1
                    for (int k = 0; k < 3; ++k) {
                        const float add = k == 0 ? NAN : k == 1 ? INFINITY : -INFINITY;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) + (odd[k * D + c + i] < limit ? add : 0.f));
                    }
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    o[i] = __float_as_uint(ok ? __uint_as_float(o[i]) * f : NAN);
                if (whole) {   // 64 channels make 128 bytes
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        o[i] = pack2<DT>(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
                    stage_words<16>(place, o, c / 32 % 2 * 4);
                    if (c / 32 % 2)
                        send_rows(place, to, alive, (c - 32) * 2, width);
                } else {
                    stage_words<32>(place, o, 0);
                    send_rows(place, to, alive, c * 4, width);
                }
            }
            tcgen05_before();
        }
        __syncwarp();
        if (busy && threadIdx.x % 32 == 0) {   // what has been taken out is used
            __threadfence_block();
            atomicAdd(words + 1 + 2 * t, 1);
        }
        count += p.end - p.step;
        const Tail now = tail_of<kRows, kCost>(run, p);
        if (now.per)
            *tail = now;
        advance<kRows>(a, run, p);
    }
}

// FOLD: tiles may go over more than kFoldSteps steps.
template <int DT, int D, bool BOXES, bool FOLD>
__global__ void __launch_bounds__(kThreads, 1)
    attend_tiles_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap keys,
                        const __grid_constant__ CUtensorMap values)
{
    extern __shared__ __align__(1024) unsigned char memory[];
    using S = Shared<D>;
    const uint32_t mem = smem_addr(memory);
    const int warp = threadIdx.x / 32;
    int* words = reinterpret_cast<int*>(memory + S::kWords);
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages<D>(); ++i) {
            mbar_init(mem + S::kFull + 8 * i, BOXES ? 2 : kLoaders);
            mbar_init(mem + S::kEmpty + 8 * i, 1);
            mbar_init(mem + S::kRaw + 8 * i, 1);
        }
        mbar_init(mem + S::kQFull, kLoaders);
        mbar_init(mem + S::kQEmpty, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(mem + S::kS + 8 * t, 1);
            mbar_init(mem + S::kP + 16 * t, kWeighers / 2);
            mbar_init(mem + S::kP + 16 * t + 8, kWeighers / 2);
            mbar_init(mem + S::kO + 8 * t, 1);
        }
        mbar_init(mem + S::kReset, kLoaders);
        mbar_init(mem + S::kDrain, 1);
        words[1] = words[2] = words[3] = 0;
        brought<D>(mem, 0);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    let_next_start();
    if (warp == kIssueWarp)
        tmem_alloc(mem + S::kWords, 512);
    tcgen05_before();
    // also the barrier after the initialisation
    const Run run = run_of<kRows, kKeys, kCost, kThreads>(a, kLeast, reinterpret_cast<int64_t*>(memory + S::kSums));
    __syncthreads();
    tcgen05_after();
    const uint32_t tmem = static_cast<uint32_t>(words[0]);
    // 168 registers a thread at the launch: 256 x 208 and 128 x 88 are as many.  The weighers' 128
    // scores and what stands beside them spill some 430 bytes: 0.4 % of the instructions that run
    if (warp < kLoadWarp) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        Tail tail{};
        weigher<DT, D, FOLD>(a, run, memory, tmem, &tail);
        if (threadIdx.x == 0)
            a.tails[blockIdx.x] = tail;
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (BOXES && warp == kLoadWarp) {
            boxes<D>(a, run, memory, &keys, &values);
        } else if (warp < kLoadWarp + (BOXES ? 3 : 2)) {
            if constexpr (BOXES)
                helper<DT, D>(a, run, memory);
            else
                loader<DT, D>(a, run, memory);
            cp_async_wait(0);
        } else if (warp == kIssueWarp) {
            issuer<DT, D, FOLD>(a, run, memory, tmem);
            mma_commit(mem + S::kDrain);   // where it gave up, products may be under way
            (void)wait(mem + S::kDrain, 0);
        }
        __syncwarp();
    }
    tcgen05_before();
    __syncthreads();
    tcgen05_after();
    if (warp == kIssueWarp)
        tmem_free(tmem, 512);
}

template <int DT, int D, bool BOXES, bool FOLD>
cudaError_t launch_form(const AttendArgs& a, const CUtensorMap& keys, const CUtensorMap& values, cudaStream_t st)
{
    const cudaError_t e = launch_grid<attend_tiles_kernel<DT, D, BOXES, FOLD>>(
        dim3(unsigned(a.ctas)), kThreads, Shared<D>::kBytes, 1, false, st, a, keys, values);
    if (e != cudaSuccess)
        return e;
    return launch_grid<attend_join_many_kernel<DT, D, kRows>>(dim3(unsigned(a.ctas), kRows / kJoinMany), 256, 0, 1, true,
                                                              st, a);
}

// Where page lists hold no more keys than a tile goes over without folding its sums, the
// form that cannot: chunks of 1024 tokens over 16384 keys take 240.7 us in it and 245 in
// the other.
template <int DT, int D, bool BOXES>
cudaError_t launch_many(const AttendArgs& a, const CUtensorMap& keys, const CUtensorMap& values, cudaStream_t st)
{
    if (static_cast<int64_t>(a.paged.most_pages) * a.paged.page_size > static_cast<int64_t>(kFoldSteps) * kKeys)
        return launch_form<DT, D, BOXES, true>(a, keys, values, st);
    return launch_form<DT, D, BOXES, false>(a, keys, values, st);
}

template <int DT, int D>
cudaError_t launch_pages(const AttendArgs& a, const CUtensorMap* maps, cudaStream_t st)
{
    return maps ? launch_many<DT, D, true>(a, maps[0], maps[1], st)
                : launch_many<DT, D, false>(a, CUtensorMap{}, CUtensorMap{}, st);
}

}  // namespace

int attend_many_rows() { return kRows; }

cudaError_t launch_attend_many(int dtype, const AttendArgs& a, const CUtensorMap* maps, cudaStream_t st)
{
    if (dtype == TSX_BF16)
        return a.dim <= 64 ? launch_pages<TSX_BF16, 64>(a, maps, st) : launch_pages<TSX_BF16, 128>(a, maps, st);
    return a.dim <= 64 ? launch_pages<TSX_F16, 64>(a, maps, st) : launch_pages<TSX_F16, 128>(a, maps, st);
}

}  // namespace tsx

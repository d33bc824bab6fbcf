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
//                    results (no reduction between threads)
//   warps 8-11       loads: queries, keys and values by cp.async, since a page may
//                    lie anywhere; which of the step's keys exist
//   warp 12          one thread issues the products
//
// The running maximum is not followed closely: O and the sum are scaled only when
// a row's maximum has grown by more than 2^8 over the one in use, which is rare
// after the first steps; weights are then up to 2^8, with the same relative error.
//
// Every wait gives up after kPatience; then the CTA's remaining rows become NaN.

#include "tsx_attend.cuh"
#include "tsx_tcgen05.cuh"

namespace tsx {
namespace {

using namespace dev;

constexpr int kHalf = 128, kRows = 2 * kHalf, kKeys = 128, kThreads = 512;
constexpr int kLoaders = 128;
constexpr int64_t kLeast = 2;        // steps to a CTA at least
constexpr int kMasks = 8;            // steps whose keys are remembered
constexpr int kBlock = kKeys * 128;  // bytes of a block: 128 rows of 64 channels
constexpr int kLag = 2;              // groups of loads in flight behind the last
constexpr float kGrowth = 8.f;
constexpr uint64_t kPatience = 4000000000ull;   // ns

// Keys or values of a step take a stage.  One CTA to an SM, which is what the
// tensor memory is for: the stages of D = 64 are as many as keep a second one out.
template <int D>
TSX_HD constexpr int stages() { return D == 128 ? 5 : 8; }

template <int D>
struct Shared {
    static constexpr int kTile = D / 64 * kBlock;   // bytes of 128 rows
    static constexpr int kQ = 0, kRing = 2 * kTile, kEnd = kRing + stages<D>() * kTile;
    // barriers
    static constexpr int kFull = kEnd, kEmpty = kFull + 8 * stages<D>(), kQFull = kEmpty + 8 * stages<D>(),
                         kQEmpty = kQFull + 8, kS = kQEmpty + 8, kP = kS + 16, kO = kP + 16,
                         kReset = kO + 16, kDrain = kReset + 8;
    static constexpr int kMask = kDrain + 8;                 // [kMasks][4] words
    static constexpr int kOdd = kMask + kMasks * 16;      // [3][D] first keys with a NaN, +inf, -inf
    static constexpr int kSums = kOdd + 3 * D * 4;        // words of run_of
    static constexpr int kWords = kSums + (kThreads / 32 + 3) * 8;   // tensor memory, pieces done, odd values met
    static constexpr int kBytes = kWords + 16;
};

__device__ __forceinline__ bool wait(uint32_t bar, uint32_t phase) { return mbar_wait(bar, phase & 1, kPatience); }
// The same answer for all threads of the warp.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t phase)
{
    return __all_sync(0xffffffffu, wait(bar, phase));
}

// ------------------------------------------------------------------ loads

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
template <int DT, int D>
__device__ void take_out(unsigned char* memory, const Landing& l)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32 & 3;
    int* odd = reinterpret_cast<int*>(memory + Shared<D>::kOdd);
    int* met = reinterpret_cast<int*>(memory + Shared<D>::kWords) + 2;
    constexpr int kChunks = D / 8;
    for (int i = 0; i < kChunks; ++i) {   // the chunks that this thread has copied
        const int id = i * 32 + lane, row = warp * 32 + id / kChunks, chunk = id % kChunks;
        uint32_t* at = reinterpret_cast<uint32_t*>(memory + l.stage + chunk / 8 * kBlock + row * 128 +
                                                   ((chunk & 7) ^ (row & 7)) * 16);
        for (int w = 0; w < 4; ++w) {
            uint32_t v = at[w];
            if (!not_finite<DT>(v))
                continue;
            for (int e = 0; e < 2; ++e) {
                const uint32_t half = v >> (16 * e) & 0xffffu;
                if (!not_finite<DT>(half))
                    continue;
                const bool nan = half & (DT == TSX_BF16 ? 0x7fu : 0x3ffu);
                atomicMin(odd + (nan ? 0 : half >> 15 ? 2 : 1) * D + chunk * 8 + w * 2 + e, l.base + row);
                v &= e ? 0x0000ffffu : 0xffff0000u;
                *met = 1;
            }
            at[w] = v;
        }
    }
}

template <int DT, int D>
__device__ __forceinline__ void land(unsigned char* memory, const Landing& l)
{
    if (l.check)
        take_out<DT, D>(memory, l);
    fence_proxy_async_smem();
    mbar_arrive(l.bar);
}

// 32 rows of a warp, whose elements start at `at` (bytes; < 0: zeros), into a tile.
template <int D>
__device__ __forceinline__ void load_rows(const char* base, int64_t at, int dim, uint32_t tile)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32 & 3;
    constexpr int kChunks = D / 8;
#pragma unroll 4
    for (int i = 0; i < kChunks; ++i) {
        const int id = i * 32 + lane, in_warp = id / kChunks, chunk = id % kChunks, row = warp * 32 + in_warp;
        const int64_t from = __shfl_sync(0xffffffffu, at, in_warp);
        const uint32_t bytes = from >= 0 && chunk * 8 < dim ? 16 : 0;
        cp_async(tile + chunk / 8 * kBlock + row * 128 + ((chunk & 7) ^ (row & 7)) * 16,
                 bytes ? base + from + chunk * 16 : base, 16, bytes);
    }
}

template <int DT, int D>
__device__ __forceinline__ void loader(const AttendArgs& a, Run run, unsigned char* memory)
{
    using S = Shared<D>;
    const uint32_t mem = smem_addr(memory);
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32 & 3;
    volatile int* done = reinterpret_cast<int*>(memory + S::kWords) + 1;
    int* odd = reinterpret_cast<int*>(memory + S::kOdd);
    uint32_t tile = 0, piece = 0, resets = 0;
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
        const Piece p = piece_of<kRows, kKeys>(a, run);
        if (piece && !wait_warp(mem + S::kQEmpty, piece - 1))
            return;
        for (int t = 0; t < (p.rows > kHalf ? 2 : 1); ++t) {
            const int row = t * kHalf + warp * 32 + lane;
            const int64_t at = row < p.rows
                                   ? row_at(a, p.seq.first, p.head, p.tile * kRows + row, a.q_pitch, a.q_head) * 2
                                   : -1;
            load_rows<D>(a.q, at, a.dim, mem + S::kQ + t * S::kTile);
        }
        put(Landing{mem + S::kQFull, 0, 0, false});
        const int first_limit = row_limit(a, p.seq, p.tile * kRows);
        const int limit = min(row_limit(a, p.seq, p.tile * kRows + p.rows - 1), p.seq.length);
        const int32_t* pages = a.paged.pages + p.b * a.paged.pages_pitch;
        int position = p.step * kKeys + warp * 32 + lane;
        int page = position < limit ? pages[position / a.paged.page_size] : -1;
        bool fresh = true;   // no value of the piece has been looked at
        for (int step = p.step; step < p.end; ++step) {
            const bool there = page >= 0 && page < a.paged.cache_pages;
            const int slot = position % a.paged.page_size;
            const int64_t at =
                there ? (page * a.paged.page_pitch + slot * a.slot_pitch + p.head * a.head_pitch) * 2 : -1;
            const uint32_t seen = __ballot_sync(0xffffffffu, there);
            position += kKeys;
            page = position < limit ? pages[position / a.paged.page_size] : -1;   // a step ahead
            const int base = step * kKeys;
            for (int kv = 0; kv < 2; ++kv, ++tile) {
                const int stage = tile % stages<D>();
                const uint32_t turn = tile / stages<D>();
                if (turn && !wait_warp(mem + S::kEmpty + 8 * stage, turn - 1))
                    return;
                if (kv == 0 && lane == 0)
                    reinterpret_cast<uint32_t*>(memory + S::kMask)[step % kMasks * 4 + warp] = seen;
                const bool check = kv == 1 && base + kKeys > first_limit;
                if (check && fresh) {   // the last piece's have been used
                    fresh = false;
                    if (piece) {
                        const uint64_t since = globaltimer_ns();
                        while (!__all_sync(0xffffffffu, *done >= static_cast<int>(8 * piece)))
                            if (__any_sync(0xffffffffu, globaltimer_ns() - since > kPatience))
                                return;
                        __threadfence_block();
                    }
                    for (int i = threadIdx.x % kLoaders; i < 3 * D; i += kLoaders)
                        odd[i] = 0x7fffffff;
                    if (threadIdx.x % kLoaders == 0)
                        reinterpret_cast<int*>(memory + S::kWords)[2] = 0;
                    mbar_arrive(mem + S::kReset);
                    if (!wait_warp(mem + S::kReset, resets++))
                        return;
                }
                load_rows<D>(kv ? a.v : a.k, at, a.dim, mem + S::kRing + stage * S::kTile);
                put(Landing{mem + S::kFull + 8 * stage, S::kRing + stage * S::kTile, base, check});
            }
        }
        flush();
        ++piece;
        advance<kRows>(a, run, p);
    }
}

// --------------------------------------------------------------- products

template <int DT, int D>
__device__ __forceinline__ void issuer(const AttendArgs& a, Run run, unsigned char* memory, uint32_t tmem)
{
    using S = Shared<D>;
    const uint32_t mem = smem_addr(memory);
    const uint32_t scores = product(DT == TSX_BF16, 128, kKeys, false, a.negated);
    const uint32_t values = product(DT == TSX_BF16, 128, D, true, false);
    uint32_t tile = 0, piece = 0, weights[2] = {0, 0};
    const auto full = [&](uint32_t n) { return wait(mem + S::kFull + 8 * (n % stages<D>()), n / stages<D>()); };
    const auto release = [&](uint32_t n) { mma_commit(mem + S::kEmpty + 8 * (n % stages<D>())); };
    const auto score = [&](int t, uint32_t n) {
        const uint32_t q = mem + S::kQ + t * S::kTile, k = mem + S::kRing + n % stages<D>() * S::kTile;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const uint32_t at = i / 4 * kBlock + i % 4 * 32;
            mma_smem(tmem + t * kHalf, operand(q + at, 16), operand(k + at, 16), scores, i > 0);
        }
        mma_commit(mem + S::kS + 8 * t);
    };
    while (run.from < run.to) {
        const Piece p = piece_of<kRows, kKeys>(a, run);
        const int tiles = p.rows > kHalf ? 2 : 1, steps = p.end - p.step;
        if (!wait(mem + S::kQFull, piece) || !full(tile))
            return;
        tcgen05_after();
        for (int t = 0; t < tiles; ++t)
            score(t, tile);
        release(tile);
        if (steps == 1)
            mma_commit(mem + S::kQEmpty);
        for (int i = 0; i < steps; ++i, tile += 2) {
            if (!full(tile + 1))
                return;
            const bool more = i + 1 < steps;
            for (int t = 0; t < tiles; ++t) {
                if (!wait(mem + S::kP + 8 * t, weights[t]++))
                    return;
                tcgen05_after();
                const uint32_t v = mem + S::kRing + (tile + 1) % stages<D>() * S::kTile;
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                    mma_tmem(tmem + kRows + t * kHalf, tmem + t * kHalf + k * 8, operand(v + k * 2048, kBlock), values,
                             i > 0 || k > 0);
                if (t == tiles - 1)
                    release(tile + 1);
                if (!more) {
                    mma_commit(mem + S::kO + 8 * t);
                } else {
                    if (t == 0 && !full(tile + 2))
                        return;
                    score(t, tile + 2);
                }
            }
            if (more) {
                release(tile + 2);
                if (i + 2 == steps)
                    mma_commit(mem + S::kQEmpty);
            }
        }
        ++piece;
        advance<kRows>(a, run, p);
    }
}

// ---------------------------------------------------------------- weights

template <int DT>
__device__ __forceinline__ void store_row(const AttendArgs& a, const Piece& p, int row, int first, const float* v, int n)
{
    char* to = a.out + (row_at(a, p.seq.first, p.head, p.tile * kRows + row, a.out_pitch, a.out_head) + first) * 2;
#pragma unroll
    for (int c = 0; c < n; c += 8)
        if (first + c < a.dim)
            *reinterpret_cast<uint4*>(to + c * 2) = make_uint4(pack2<DT>(v[c], v[c + 1]), pack2<DT>(v[c + 2], v[c + 3]),
                                                               pack2<DT>(v[c + 4], v[c + 5]),
                                                               pack2<DT>(v[c + 6], v[c + 7]));
}

template <int DT, int D>
__device__ __forceinline__ void weigher(const AttendArgs& a, Run run, unsigned char* memory, uint32_t tmem, Tail* tail)
{
    using S = Shared<D>;
    const uint32_t mem = smem_addr(memory);
    const int t = threadIdx.x / kHalf, mine = threadIdx.x % kHalf, row = t * kHalf + mine;
    const uint32_t lanes = static_cast<uint32_t>(mine / 32 * 32) << 16;
    const uint32_t s_at = tmem + t * kHalf + lanes, o_at = tmem + kRows + t * kHalf + lanes;
    const int* odd = reinterpret_cast<const int*>(memory + S::kOdd);
    int* words = reinterpret_cast<int*>(memory + S::kWords);
    uint32_t scored = 0, ended = 0;
    bool ok = true;
    while (run.from < run.to) {
        const Piece p = piece_of<kRows, kKeys>(a, run);
        const int all = row_limit(a, p.seq, p.tile * kRows + t * kHalf);   // keys that every row of the tile sees
        const int limit = row < p.rows ? row_limit(a, p.seq, p.tile * kRows + row) : 0;
        const bool busy = p.rows > t * kHalf;
        float top = -INFINITY, sum = 0.f;
        for (int step = p.step; busy && ok && step < p.end; ++step) {
            ok = wait_warp(mem + S::kS + 8 * t, scored);
            if (!ok)
                break;
            ++scored;
            tcgen05_after();
            uint32_t s[kKeys];
#pragma unroll
            for (int i = 0; i < kKeys; i += 32)
                tmem_load32(s_at + i, s + i);
            tmem_wait_loads();
            const int base = step * kKeys;
            const uint4 seen = *reinterpret_cast<const uint4*>(memory + S::kMask + step % kMasks * 16);
            if (base + kKeys > all || (seen.x & seen.y & seen.z & seen.w) != 0xffffffffu) {
                const uint32_t words4[4] = {seen.x, seen.y, seen.z, seen.w};
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int left = limit - base - 32 * w;
                    const uint32_t sees = words4[w] & (left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (!(sees >> i & 1))
                            s[32 * w + i] = 0xff800000u;
                }
            }
            float most[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                most[i] = __uint_as_float(s[i]);
#pragma unroll
            for (int i = 4; i < kKeys; i += 8)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (i + 4 < kKeys)
                        most[j] = fmaxf(most[j], fmaxf(__uint_as_float(s[i + j]), __uint_as_float(s[i + 4 + j])));
                    else
                        most[j] = fmaxf(most[j], __uint_as_float(s[i + j]));
            const float now = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3])) * a.scale_log2;
            const bool grows = now > top + kGrowth || (top == -INFINITY && now > top);
            if (__any_sync(0xffffffffu, grows)) {
                const float f = grows && top != -INFINITY ? exp2_fast(top - now) : 1.f;
                top = grows ? now : top;
                sum *= f;
                if (step > p.step && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll
                    for (int c = 0; c < D; c += 16) {   // O is at rest: the scores came after its last product
                        uint32_t o[16];
                        tmem_load16(o_at + c, o);
                        tmem_wait_loads();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_store16(o_at + c, o);
                    }
                }
            }
            const float2 less = pair_of(top == -INFINITY ? 0.f : -top), by = pair_of(a.scale_log2);
            float2 total[2] = {pair_of(0.f), pair_of(0.f)};
#pragma unroll
            for (int c = 0; c < kKeys; c += 64) {
                uint32_t w[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float2 v = make_float2(__uint_as_float(s[c + 2 * i]), __uint_as_float(s[c + 2 * i + 1]));
                    v = __ffma2_rn(v, by, less);
                    v.x = exp2_fast(v.x);
                    v.y = exp2_fast(v.y);
                    total[i & 1] = __fadd2_rn(total[i & 1], v);
                    w[i] = pack2<DT>(v.x, v.y);
                }
                tmem_store32(s_at + c / 2, w);
            }
            tmem_wait_stores();
            tcgen05_before();
            mbar_arrive(mem + S::kP + 8 * t);
            const float2 both = __fadd2_rn(total[0], total[1]);
            sum += both.x + both.y;
        }
        if (busy) {
            ok = ok && wait_warp(mem + S::kO + 8 * t, ended++);
            tcgen05_after();
            const bool whole = p.whole(), live = row < p.rows;
            const int slot = part_slot(p);
            const bool strange = ok && p.end * kKeys > row_limit(a, p.seq, p.tile * kRows) && words[2];
            const float f = !ok ? NAN : !whole ? 1.f : sum > 0.f || sum != sum ? 1.f / sum : 0.f;
#pragma unroll
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                float v[32];
                if (ok) {
                    tmem_load32(o_at + c, o);
                    tmem_wait_loads();
                }
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    v[i] = ok ? __uint_as_float(o[i]) : 0.f;
                if (strange)
                    for (int k = 0; k < 3; ++k)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (odd[k * D + c + i] < limit)
                                v[i] += k == 0 ? NAN : k == 1 ? INFINITY : -INFINITY;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    v[i] *= f;
                if (!live)
                    continue;
                if (whole) {
                    store_row<DT>(a, p, row, c, v, 32);
                } else {
                    float4* to = reinterpret_cast<float4*>(a.parts + (static_cast<int64_t>(slot) * kRows + row) * D + c);
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        to[i / 4] = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                }
            }
            if (live && whole)
                store_lse(a, p.seq.first, p.head, p.tile * kRows + row, top, ok ? sum : NAN);
            if (live && !whole)
                a.stats[slot * kRows + row] = make_float2(top, ok ? sum : NAN);
            tcgen05_before();
        }
        __syncwarp();
        if (threadIdx.x % 32 == 0) {
            __threadfence_block();
            atomicAdd(words + 1, 1);
        }
        const Tail now = tail_of<kRows>(run, p);
        if (now.follow)
            *tail = now;
        advance<kRows>(a, run, p);
    }
}

template <int DT, int D>
__global__ void __launch_bounds__(kThreads, 1) attend_tiles_kernel(const __grid_constant__ AttendArgs a)
{
    extern __shared__ __align__(1024) unsigned char memory[];
    using S = Shared<D>;
    const uint32_t mem = smem_addr(memory);
    const int warp = threadIdx.x / 32;
    int* words = reinterpret_cast<int*>(memory + S::kWords);
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages<D>(); ++i) {
            mbar_init(mem + S::kFull + 8 * i, kLoaders);
            mbar_init(mem + S::kEmpty + 8 * i, 1);
        }
        mbar_init(mem + S::kQFull, kLoaders);
        mbar_init(mem + S::kQEmpty, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(mem + S::kS + 8 * t, 1);
            mbar_init(mem + S::kP + 8 * t, kHalf);
            mbar_init(mem + S::kO + 8 * t, 1);
        }
        mbar_init(mem + S::kReset, kLoaders);
        mbar_init(mem + S::kDrain, 1);
        words[1] = words[2] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    let_next_start();
    if (warp == 12)
        tmem_alloc(mem + S::kWords, 512);
    tcgen05_before();
    // also the barrier after the initialisation
    const Run run = run_of<kRows, kKeys, kThreads>(a, kLeast, reinterpret_cast<int64_t*>(memory + S::kSums));
    __syncthreads();
    tcgen05_after();
    const uint32_t tmem = static_cast<uint32_t>(words[0]);
    // 128 registers a thread at the launch: 256 x 200 and 256 x 56 are as many
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        Tail tail{};
        weigher<DT, D>(a, run, memory, tmem, &tail);
        if (threadIdx.x == 0)
            a.tails[blockIdx.x] = tail;
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp < 12) {
            loader<DT, D>(a, run, memory);
            cp_async_wait(0);
        } else if (threadIdx.x == 12 * 32) {
            issuer<DT, D>(a, run, memory, tmem);
            mma_commit(mem + S::kDrain);   // where it gave up, products may be under way
            (void)wait(mem + S::kDrain, 0);
        }
        __syncwarp();
    }
    tcgen05_before();
    __syncthreads();
    tcgen05_after();
    if (warp == 12)
        tmem_free(tmem, 512);
}

template <int DT, int D>
cudaError_t launch_many(const AttendArgs& a, cudaStream_t st)
{
    const cudaError_t e =
        launch_grid<attend_tiles_kernel<DT, D>>(dim3(unsigned(a.ctas)), kThreads, Shared<D>::kBytes, 1, false, st, a);
    if (e != cudaSuccess)
        return e;
    return launch_grid<attend_join_kernel<DT, D, kRows>>(dim3(unsigned(a.ctas), kRows / 4), 128, 0, 1, true, st, a);
}

}  // namespace

int attend_many_rows() { return kRows; }

cudaError_t launch_attend_many(int dtype, const AttendArgs& a, cudaStream_t st)
{
    if (dtype == TSX_BF16)
        return a.dim <= 64 ? launch_many<TSX_BF16, 64>(a, st) : launch_many<TSX_BF16, 128>(a, st);
    return a.dim <= 64 ? launch_many<TSX_F16, 64>(a, st) : launch_many<TSX_F16, 128>(a, st);
}

}  // namespace tsx

// The C ABI of the layer operators (include/tsx_layers.h): argument checks,
// how rows are laid over threads, launches.

#include "layers.h"

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <numeric>

#include "plan.h"

namespace tsx {

namespace {

int round_up(int64_t v, int to) { return int((v + to - 1) / to * to); }

// Neighbouring threads that share a checkpoint block, or (vec false) read
// neighbouring elements; no more than the octs need.
int team_of(int64_t cols, int block, bool vec)
{
    const int64_t octs = (cols + kOct - 1) / kOct;
    int team = block ? block / kOct : vec ? 1 : 16;
    while (team > 1 && team / 2 >= octs)
        team /= 2;
    return team;
}

}  // namespace

RowLayout row_layout(int64_t rows, int64_t cols, int block, bool vec, int want)
{
    RowLayout lay{};
    lay.rows = rows;
    lay.cols = int(cols);
    lay.vec = vec;
    const int64_t octs = (cols + kOct - 1) / kOct;
    lay.team = team_of(cols, block, vec);
    const int64_t chunks = (octs + want - 1) / want;
    const int64_t v = round_up((octs + chunks - 1) / chunks, lay.team);
    lay.V = int(v);
    lay.per_v = lane_factor(lay.V);
    lay.chunk_cols = lay.V * kOct;
    lay.chunks = int((cols + lay.chunk_cols - 1) / lay.chunk_cols);
    int64_t p = want / v;
    p = p < 1 ? 1 : p > rows ? rows : p;
    lay.P = int(p);
    lay.threads = (lay.P * lay.V + 31) / 32 * 32;
    return lay;
}

namespace {

// Threads of the elementwise layer kernels' CTAs.
constexpr int kElementwiseThreads = kLayerThreads;
constexpr int64_t kMaxExtent = 0x7fffffff;
constexpr int kMaxChunks = 65535;   // grid.y

int fail(int rc, const char* call, const char* msg)
{
    char buf[256];
    std::snprintf(buf, sizeof buf, "%s: %s", call, msg);
    set_last_error(buf);
    return rc;
}

int launched(cudaError_t e, const char* call)
{
    if (e != cudaSuccess) {
        (void)cudaGetLastError();   // reported here, so no later call's
        return fail(TSX_ERR_CUDA, call, cudaGetErrorString(e));
    }
    set_last_error("");
    return TSX_OK;
}

bool known_dtype(int dtype) { return dtype == TSX_F16 || dtype == TSX_BF16 || dtype == TSX_F32; }
bool known_act(int act) { return act == TSX_ACT_NONE || act == TSX_ACT_SILU || act == TSX_ACT_GELU; }

bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// Shape, form and block of a call; TSX_OK also for an empty tensor.
int check_shape(const char* call, int dtype, int64_t rows, int64_t cols, int form, int block)
{
    if (!known_dtype(dtype))
        return fail(TSX_ERR_INVALID, call, "unknown dtype");
    if (rows < 0 || cols < 0 || rows >= kMaxExtent || cols >= kMaxExtent)
        return fail(TSX_ERR_INVALID, call, "rows and cols must be 0 .. 2^31 - 2");
    if (form != TSX_INT8 && form != TSX_E4M3)
        return fail(TSX_ERR_INVALID, call, "unknown 8-bit form");
    if (block != 32 && block != 64 && block != 128)
        return fail(TSX_ERR_INVALID, call, "block must be 32, 64 or 128");
    return TSX_OK;
}

// Whether rows of `cols` elements at this pitch from `p` move as vectors.
bool vectors(const void* p, int64_t cols, int64_t pitch, int es)
{
    return !p || (cols % kOct == 0 && pitch * es % 16 == 0 && aligned(p, 16));
}
// The same of the dense bytes of a checkpoint.
bool held_vectors(const void* q, int64_t cols) { return !q || (cols % kOct == 0 && aligned(q, 8)); }

int check_layout(const char* call, const RowLayout& lay)
{
    if (lay.chunks > kMaxChunks)
        return fail(TSX_ERR_UNSUPPORTED, call, "rows are too long");
    return TSX_OK;
}

int pack_args(const char* call, int dtype, int64_t rows, int64_t cols, int64_t pitch, int form, int block,
              const void* x, const void* q, const float* scale, PackArgs* a)
{
    if (!x || !q || !scale)
        return fail(TSX_ERR_INVALID, call, "x, q and scale are required");
    const int es = elem_size(dtype);
    if (!aligned(x, es) || !aligned(scale, 4))
        return fail(TSX_ERR_ALIGN, call, "a base pointer is not aligned to its elements");
    a->lay = row_layout(rows, cols, block, vectors(x, cols, pitch, es) && held_vectors(q, cols), kElementwiseThreads);
    a->pitch = pitch;
    a->form = form;
    a->block = block;
    a->blocks = (cols + block - 1) / block;
    return check_layout(call, a->lay);
}

}  // namespace
}  // namespace tsx

using namespace tsx;

extern "C" int tsx_pack(tsx_dtype dtype, int64_t rows, int64_t cols, int64_t pitch, tsx_form form, int block,
                        const void* x, void* q, float* scale, tsx_stream_t stream)
{
    const char* call = "tsx_pack";
    int rc = check_shape(call, dtype, rows, cols, form, block);
    if (rc != TSX_OK)
        return rc;
    if (pitch < cols)
        return fail(TSX_ERR_INVALID, call, "the pitch is shorter than a row");
    if (rows == 0 || cols == 0)
        return launched(cudaSuccess, call);
    PackArgs a{};
    rc = pack_args(call, dtype, rows, cols, pitch, form, block, x, q, scale, &a);
    if (rc != TSX_OK)
        return rc;
    return launched(launch_pack(dtype, a, x, HeldOut{q, scale}, reinterpret_cast<cudaStream_t>(stream)), call);
}

extern "C" int tsx_unpack(tsx_dtype dtype, int64_t rows, int64_t cols, int64_t pitch, tsx_form form, int block,
                          const void* q, const float* scale, void* x, tsx_stream_t stream)
{
    const char* call = "tsx_unpack";
    int rc = check_shape(call, dtype, rows, cols, form, block);
    if (rc != TSX_OK)
        return rc;
    if (pitch < cols)
        return fail(TSX_ERR_INVALID, call, "the pitch is shorter than a row");
    if (rows == 0 || cols == 0)
        return launched(cudaSuccess, call);
    PackArgs a{};
    rc = pack_args(call, dtype, rows, cols, pitch, form, block, x, q, scale, &a);
    if (rc != TSX_OK)
        return rc;
    return launched(launch_unpack(dtype, a, q, scale, x, reinterpret_cast<cudaStream_t>(stream)), call);
}

namespace {

// What forward and backward check alike.  held: the call reads or writes
// checkpoints (all four pointers), which alone decide about `block`.
int gated_args(const char* call, int dtype, int64_t rows, int64_t cols, int64_t in_pitch, int64_t out_pitch, int act,
               int form, int block, GatedArgs* a)
{
    const int rc = check_shape(call, dtype, rows, cols, form, block);
    if (rc != TSX_OK)
        return rc;
    if (!known_act(act))
        return fail(TSX_ERR_INVALID, call, "unknown activation");
    if (in_pitch < cols || out_pitch < cols)
        return fail(TSX_ERR_INVALID, call, "a pitch is shorter than a row");
    a->in_pitch = in_pitch;
    a->out_pitch = out_pitch;
    a->act = act;
    a->form = form;
    a->block = block;
    a->blocks = (cols + block - 1) / block;
    return TSX_OK;
}

}  // namespace

extern "C" int tsx_gated_act(tsx_dtype dtype, int64_t rows, int64_t cols, int64_t in_pitch, int64_t out_pitch,
                             tsx_act act, tsx_form form, int block, const void* gate, const void* up, void* h,
                             void* q_gate, float* scale_gate, void* q_up, float* scale_up, tsx_stream_t stream)
{
    const char* call = "tsx_gated_act";
    GatedArgs a{};
    int rc = gated_args(call, dtype, rows, cols, in_pitch, out_pitch, act, form, block, &a);
    if (rc != TSX_OK)
        return rc;
    const int held = !!q_gate + !!scale_gate + !!q_up + !!scale_up;
    if (held != 0 && held != 4)
        return fail(TSX_ERR_INVALID, call, "both checkpoints, or neither");
    if (rows == 0 || cols == 0)
        return launched(cudaSuccess, call);
    if (!gate || !up || !h)
        return fail(TSX_ERR_INVALID, call, "gate, up and h are required");
    const int es = elem_size(dtype);
    if (!aligned(gate, es) || !aligned(up, es) || !aligned(h, es) || !aligned(scale_gate, 4) || !aligned(scale_up, 4))
        return fail(TSX_ERR_ALIGN, call, "a base pointer is not aligned to its elements");
    const bool vec = vectors(gate, cols, in_pitch, es) && vectors(up, cols, in_pitch, es) &&
                     vectors(h, cols, out_pitch, es) && held_vectors(q_gate, cols) && held_vectors(q_up, cols);
    a.lay = row_layout(rows, cols, held ? block : 0, vec, kElementwiseThreads);
    rc = check_layout(call, a.lay);
    if (rc != TSX_OK)
        return rc;
    return launched(launch_gated(dtype, a, gate, up, h, HeldOut{q_gate, scale_gate}, HeldOut{q_up, scale_up},
                                 reinterpret_cast<cudaStream_t>(stream)),
                    call);
}

extern "C" int tsx_gated_act_backward(tsx_dtype dtype, int64_t rows, int64_t cols, int64_t in_pitch,
                                      int64_t out_pitch, tsx_act act, tsx_form form, int block, const void* dh,
                                      const void* gate, const void* up, const void* q_gate, const float* scale_gate,
                                      const void* q_up, const float* scale_up, void* dgate, void* dup, void* h,
                                      tsx_stream_t stream)
{
    const char* call = "tsx_gated_act_backward";
    GatedArgs a{};
    int rc = gated_args(call, dtype, rows, cols, in_pitch, out_pitch, act, form, block, &a);
    if (rc != TSX_OK)
        return rc;
    if (rows == 0 || cols == 0)
        return launched(cudaSuccess, call);
    const int held = !!q_gate + !!scale_gate + !!q_up + !!scale_up, full = !!gate + !!up;
    if (!((held == 4 && full == 0) || (held == 0 && full == 2)))
        return fail(TSX_ERR_INVALID, call, "gate and up are either two tensors or two checkpoints");
    if (!dh || !dgate || !dup)
        return fail(TSX_ERR_INVALID, call, "dh, dgate and dup are required");
    const int es = elem_size(dtype);
    if (!aligned(dh, es) || !aligned(gate, es) || !aligned(up, es) || !aligned(dgate, es) || !aligned(dup, es) ||
        !aligned(h, es) || !aligned(scale_gate, 4) || !aligned(scale_up, 4))
        return fail(TSX_ERR_ALIGN, call, "a base pointer is not aligned to its elements");
    const bool vec = vectors(dh, cols, out_pitch, es) && vectors(h, cols, out_pitch, es) &&
                     vectors(gate, cols, in_pitch, es) && vectors(up, cols, in_pitch, es) &&
                     vectors(dgate, cols, in_pitch, es) && vectors(dup, cols, in_pitch, es) &&
                     held_vectors(q_gate, cols) && held_vectors(q_up, cols);
    a.lay = row_layout(rows, cols, held ? block : 0, vec, kElementwiseThreads);
    rc = check_layout(call, a.lay);
    if (rc != TSX_OK)
        return rc;
    return launched(launch_gated_backward(dtype, a, dh, Saved{gate, q_gate, scale_gate}, Saved{up, q_up, scale_up},
                                          dgate, dup, h, reinterpret_cast<cudaStream_t>(stream)),
                    call);
}

// ---------------------------------------------------------- group norm
// The times in the comments below are GPU times of calls in a CUDA graph that
// repeats them on the same tensors.

namespace {

// Channels of a CTA's run at most (its shared memory holds a pair of floats
// for each channel and row lane, and for each group), and its threads.
constexpr int kNormRun = 2048;
constexpr int kTokenRun = 2048;
// CTAs of the token kernels: what the SMs hold at once, two each backward and
// where a checkpoint is written, else three (a second wave half full: bf16
// [8192, 4096] with its checkpoint 39.2 us in 456 CTAs, 33.2 in 304).
constexpr int64_t kTokenThrees = 3 * 152, kTokenPairs = 2 * 152;
constexpr int64_t kNormRanks = 8;      // CTAs of a cluster at most
constexpr int64_t kNormSamples = 64;   // samples side by side at most
constexpr int64_t kHeldCtas = 2 * 152;    // CTAs to keep before samples are put side by side
constexpr int64_t kHeldFew = 16384;       // elements to a CTA where there are fewer CTAs than half the SMs
constexpr int64_t kHeldRows = 64;         // rows to a lane at most
constexpr int64_t kHeldWave = 256;        // CTAs of clusters of eight that the SMs hold at once, two each
// Ranges are cut so that at most this many CTAs share the work: as many as the
// 152 SMs hold at once, two each backward and for fp32, else three.  A constant
// of the chip, not read from it, so that results depend on the shape alone.
constexpr int64_t kNormThrees = 3 * 152, kNormPairs = 2 * 152;
constexpr int64_t kNormWide = 640, kNormGroups = 128;
constexpr int64_t kNormParts = 160;   // parts of a sample that the second kernel's CTAs join by themselves
constexpr int kNormRowsAtOnce = 4;

// Threads of a CTA that a run of channels puts to work.
int64_t filled(int64_t cols, int team)
{
    const int64_t v = round_up((cols + kOct - 1) / kOct, team);
    return v > kNormThreads ? 0 : kNormThreads / v * ((cols + kOct - 1) / kOct);
}

// Slices for dweight and dbias where `all` CTAs of a run would write one each:
// as many, unless they would take more than 16 MB.  Then each CTA adds up what it
// has of eight samples or more (tiles of them), and the CTAs of all runs are as
// many whole waves, of `wave`, as the 16 MB allow.  8192 tokens of 4096 channels
// in one group would otherwise have 268 MB of them, four times the bf16 tensor,
// and take 671 us in place of 536; heads of 80 channels, [8192, 2560], 289 in
// place of 239.  Under 16 MB the sums to and fro cost as much as the slices
// ([2000, 64, 256] 63 us in place of 68, but [1200, 16, 512] 24.9 for 24.3, [7088,
// 3, 363] 94 for 83); above, single elements lose up to 10 % ([70000, 3, 363]
// 900 us for 877, from a checkpoint 1018 for 948).  In waves that are not whole
// the last takes as long as the others: [8192, 2560] 265 us in 4.04 of them.
int64_t shared_slices(const tsx_norm_desc& d, int64_t all, int64_t wave, int64_t runs)
{
    constexpr int64_t kSliceBytes = 16 << 20, kEach = 8;
    const int64_t most = kSliceBytes / (8 * d.c);
    if (all <= most)
        return all;
    const int64_t waves = std::min(most, all / kEach) * runs / wave;
    return std::min(all, std::max<int64_t>(std::max<int64_t>(waves, 1) * wave / runs, 1));
}

// The streaming layout for rows of c channels; block: channels to a scale
// where the call writes checkpoints, else 0.  False if this alignment (vec,
// block) cannot be had with these groups.
bool stream_layout(const tsx_norm_desc& d, bool vec, int block, bool backward, NormLayout* out)
{
    const int64_t per = d.c / d.groups;
    NormLayout lay{};
    lay.kind = kNormStream;
    lay.vec = vec;
    lay.oct_in_group = vec && per % kOct == 0;
    // runs start on whole octs / blocks
    const int64_t align = block ? block : vec ? kOct : 1;
    if (per > kNormRun) {
        if (per % align != 0)
            return false;
        lay.run_groups = 1;
        const int64_t pieces = (per + kNormRun - 1) / kNormRun;
        const int64_t to = 128;   // whole teams of any size
        lay.run_cols = int(((per + pieces - 1) / pieces + to - 1) / to * to);
        lay.pieces = int((per + lay.run_cols - 1) / lay.run_cols);
        lay.runs = int(d.groups) * lay.pieces;
    } else {
        // the widest run of at most kNormWide channels and kNormGroups groups
        // that fills a CTA with rows side by side, or the one that comes
        // nearest; one of whole 128 bytes if any
        const int64_t unit = align / std::gcd(per, align);
        int64_t groups = 0, best = 0;
        if (d.c <= kNormWide && d.groups <= kNormGroups) {
            groups = d.groups;
        } else {
            const int64_t all = d.c <= kNormRun ? d.groups : 0;   // where runs cannot start on whole octs or blocks
            for (int64_t g = kNormRun / per / unit * unit; g > 0; g -= unit) {
                const int64_t cols = g * per;
                if (g >= d.groups || ((cols > kNormWide || g > kNormGroups) && g > unit))
                    continue;
                if (cols * elem_size(d.dtype) < 128 && groups > 0)
                    break;
                const int64_t full = filled(cols, team_of(cols, block, vec));
                if (full > best) {
                    best = full;
                    groups = g;
                }
            }
            if (groups == 0)
                groups = all;
        }
        if (groups == 0)
            return false;
        lay.run_groups = int(groups);
        lay.run_cols = int(groups * per);
        lay.pieces = 1;
        lay.runs = int((d.groups + groups - 1) / groups);
    }
    lay.team = team_of(lay.run_cols, block, vec);
    lay.V = round_up((lay.run_cols + kOct - 1) / kOct, lay.team);
    lay.per_v = lane_factor(lay.V);
    int64_t p = kNormThreads / lay.V;
    p = p < 1 ? 1 : p > d.l ? d.l : p;
    lay.P = int(p);
    lay.threads = round_up(lay.P * lay.V, 32);
    const int64_t ctas = (backward || d.dtype == TSX_F32 ? kNormPairs : kNormThrees) / (d.n * lay.runs);
    const int64_t most = (d.l + p * kNormRowsAtOnce - 1) / (p * kNormRowsAtOnce);
    int64_t splits = ctas < 1 ? 1 : ctas < most ? ctas : most;
    // many ranges: clusters join eight each, so that few parts are left.  The SMs hold fewer CTAs in clusters of eight (408 of 456, 288 of
    // 304), and a second wave for the last costs more than the room
    lay.ranks = splits > kNormParts ? 8 : 1;
    if (lay.ranks == 8 && splits > ctas * 5 / 6)
        splits = ctas * 5 / 6;
    splits = splits / lay.ranks * lay.ranks;
    lay.range = (d.l + splits - 1) / splits;   // the last ranges may be short, or empty
    lay.splits = splits;
    // samples that are cut into ranges make one wave as they are
    lay.slices = splits > 1 ? d.n * splits : shared_slices(d, d.n, kNormPairs, lay.runs);
    lay.samples = 1;
    lay.lanes = lay.P;
    *out = lay;
    return true;
}

// Tokens: groups of a power of two of octs, at most a warp's.
bool token_layout(const tsx_norm_desc& d, bool vec, int block, bool backward, NormLayout* out)
{
    const int64_t per = d.c / d.groups;
    if (d.l != 1 || !vec || per % kOct != 0 || per > 32 * kOct || (per & (per - 1)) != 0)
        return false;
    NormLayout lay{};
    lay.kind = kNormToken;
    lay.vec = lay.oct_in_group = true;
    const int64_t align = block > per ? block : per;   // powers of two
    const int64_t cols = d.c < kTokenRun ? d.c : kTokenRun / align * align;
    lay.run_cols = int(cols);
    lay.run_groups = int(cols / per);
    lay.pieces = 1;
    lay.runs = int((d.c + cols - 1) / cols);
    lay.team = team_of(lay.run_cols, block, true);
    const int own = int(per / kOct);
    lay.V = round_up(lay.run_cols / kOct, own > lay.team ? own : lay.team);
    lay.per_v = lane_factor(lay.V);
    int64_t p = kTokenThreads / lay.V;
    p = p < 1 ? 1 : p > d.n ? d.n : p;
    lay.P = int(p);
    lay.threads = round_up(lay.P * lay.V, 32);
    lay.ranks = lay.samples = lay.lanes = 1;
    const int64_t at_once = p * (backward ? 2 : 4);
    const int64_t most = (d.n + at_once - 1) / at_once;
    const int64_t want = (backward || block ? kTokenPairs : kTokenThrees) / lay.runs;
    lay.splits = most < want ? most : want < 1 ? 1 : want;
    lay.range = (d.n + lay.splits - 1) / lay.splits;   // rows to a CTA
    lay.splits = (d.n + lay.range - 1) / lay.range;
    lay.slices = lay.splits;
    *out = lay;
    return true;
}

// Samples on chip.  Two CTAs share an SM, or four of half the threads.  A sample of several CTAs (a cluster)
// is held only if all samples fit on the chip at once: the chain from the loads
// over the cluster's barrier to the stores is then gone through once, in less
// time than the streaming kernels' two launches, and beyond that it is not
// (measured: see k_norm_held.cu).  Samples of one CTA are held however many
// there are.
bool held_layout(const tsx_norm_desc& d, bool vec, int block, bool backward, bool held, NormLayout* out)
{
    const int64_t per = d.c / d.groups;
    if (per > kNormRun)
        return false;
    const int es = elem_size(d.dtype);
    const int64_t align = block ? block : vec ? kOct : 1;
    const int64_t unit = align / std::gcd(per, align);
    int64_t best = 0;   // CTAs of the layout found
    // Samples for several waves of CTAs: four CTAs of half the threads to an SM
    // rather than two, where a quarter of its memory holds a sample's run (bf16
    // [2000, 64, 256] 29.3 us, in two 36.8, and its gradient 68.4, 71.4; [1000,
    // 33, 512] 15.5, 20.3 and 41.2, 43.4).
    for (int small = d.n >= 2 * kHeldCtas ? 1 : 0; small >= 0; --small)
    for (int64_t groups = d.c <= kNormRun ? d.groups : kNormRun / per / unit * unit; groups > 0;) {
        const int64_t threads = small ? kNormThreads / 2 : kNormThreads, wave = small ? 2 * kHeldCtas : kHeldCtas;
        for (int ranks = 1; ranks <= (small ? 1 : kNormRanks); ranks *= 2) {
            NormLayout lay{};
            lay.kind = kNormHeld;
            lay.vec = vec;
            lay.oct_in_group = vec && per % kOct == 0;
            lay.run_groups = int(groups);
            lay.run_cols = int(groups * per);
            lay.pieces = 1;
            lay.runs = int((d.groups + groups - 1) / groups);
            lay.team = team_of(lay.run_cols, block, vec);
            lay.V = round_up((lay.run_cols + kOct - 1) / kOct, lay.team);
            lay.per_v = lane_factor(lay.V);
            const int64_t lanes = threads / lay.V;
            if (lanes == 0)
                continue;
            lay.ranks = ranks;
            lay.range = (d.l + ranks - 1) / ranks;   // the last ranks may have no rows
            lay.splits = 1;
            // row lanes: as many as there are rows, or fewer, of eight rows
            // each, with several samples side by side while there are
            // CTAs enough
            int64_t own = lay.range < lanes ? lay.range : lanes, samples = 1;
            if (ranks == 1) {
                const int64_t few = (lay.range + 7) / 8, most = d.n * lay.runs / wave;
                samples = lanes / few < most ? lanes / few : most;
                samples = samples < 1 ? 1 : samples > kNormSamples ? kNormSamples : samples;
                own = lanes / samples < own ? lanes / samples : own;
            }
            lay.samples = int(samples);
            lay.lanes = int(own);
            lay.P = int(samples * own);
            lay.threads = round_up(lay.P * lay.V, 32);
            const int64_t lane_rows = (lay.range + own - 1) / own;
            if (lane_rows > kHeldRows)
                continue;
            lay.lane_rows = int(lane_rows);
            if (int64_t(held_bytes(lay, es, backward, held)) > kSmemPerSm / (small ? 4 : 2) - kSmemPerCtaReserved)
                continue;
            const int64_t tiles = (d.n + samples - 1) / samples, ctas = tiles * lay.runs * ranks;
            lay.slices = ranks > 1 ? tiles * ranks : shared_slices(d, tiles, wave, lay.runs);
            if (ranks > 1 && ctas > kHeldWave)
                continue;
            // Backward, two operands and their sums leave room for narrow runs
            // only, and the CTAs past the first wave pay for their parameters
            // and sums again.  Short samples gain all the same (bf16 [2000,
            // 64, 256] 68.0 us against 109.7 streaming, [700, 100, 128] 23.7
            // against 31.6), longer ones do not ([128, 128, 512] 21.4 against
            // 18.1, [64, 256, 512] 20.2 against 18.0, [256, 256, 512] 66.5
            // against 57.9).
            if (backward && d.l >= 128 && ctas > kHeldCtas)
                continue;
            // Nor do clusters whose loads go element by element, and so wait
            // (fp32 [3, 1009, 198] 13.7 against 11.8, from int8 17.0, 14.8).
            if (backward && !vec && ranks > 1)
                continue;
            // the most CTAs, and of those the widest runs and fewest ranks
            if (ctas > best) {
                best = ctas;
                *out = lay;
            }
            if (ranks == 1 && ctas >= wave)
                return true;
        }
        const int64_t next = (groups / 2 + unit - 1) / unit * unit;
        if (next >= groups || next * per * es < 128)
            break;
        groups = next;
    }
    // a few CTAs with much to do: the streaming kernels spread it further
    const int64_t elements = d.n * d.l * d.c;
    return best >= 76 || (best > 0 && elements <= best * kHeldFew);
}

// How a call runs; held: backward from a checkpoint.  The search takes
// microseconds, as long as a launch, so a thread remembers the layouts of its
// last shapes.
bool find_layout(const tsx_norm_desc& d, bool vec, int block, bool backward, bool held, NormLayout* out)
{
    if (token_layout(d, vec, block, backward, out))
        return true;
    if (!held_layout(d, vec, block, backward, held, out) && !stream_layout(d, vec, block, backward, out))
        return false;
    // The forward kernels' sums over row lanes: as many threads to a column as
    // there are, while an item's columns and shares are a warp's work.
    const int per = int((out->pieces > 1 ? out->run_cols : d.c / d.groups) / (out->oct_in_group ? kOct : 1));
    const int columns = out->samples * out->run_groups * per;
    int shares = std::min({out->threads / columns, 64 / per, out->lanes});
    shares = std::max(shares, 1);
    out->share_lanes = (out->lanes + shares - 1) / shares;
    out->shares = (out->lanes + out->share_lanes - 1) / out->share_lanes;
    return true;
}

struct LayoutKey {
    int64_t n, l, c;
    int32_t dtype, groups, block, flags;
};

bool norm_layout(const tsx_norm_desc& d, bool vec, int block, bool backward, bool held, NormLayout* out)
{
    struct Entry {
        LayoutKey key;
        bool used, found;
        NormLayout lay;
    };
    constexpr int kEntries = 16;
    thread_local Entry entries[kEntries];
    thread_local int next;
    LayoutKey key;
    std::memset(&key, 0, sizeof key);
    key.n = d.n;
    key.l = d.l;
    key.c = d.c;
    key.dtype = d.dtype;
    key.groups = d.groups;
    key.block = block;
    key.flags = vec | backward << 1 | held << 2;
    for (const Entry& e : entries)
        if (e.used && std::memcmp(&e.key, &key, sizeof key) == 0) {
            *out = e.lay;
            return e.found;
        }
    Entry& e = entries[next];
    next = (next + 1) % kEntries;
    e.key = key;
    e.lay = NormLayout{};
    e.found = find_layout(d, vec, block, backward, held, &e.lay);
    e.used = true;
    *out = e.lay;
    return e.found;
}

size_t part_bytes(const tsx_norm_desc& d, const NormLayout& lay)
{
    if (lay.kind != kNormStream)
        return 0;
    const size_t b = size_t(d.n) * size_t(lay.splits) * size_t(lay.pieces) * size_t(d.groups) * sizeof(float2);
    return (b + 15) / 16 * 16;
}
size_t chan_bytes(const tsx_norm_desc& d, const NormLayout& lay)
{
    return size_t(lay.slices) * 2 * size_t(d.c) * sizeof(float);
}

int check_norm(const char* call, const tsx_norm_desc* d)
{
    if (!d)
        return fail(TSX_ERR_INVALID, call, "no descriptor");
    if (d->n < 0 || d->l < 0 || (d->n > 0 && d->l > (kMaxExtent - 1) / d->n))
        return fail(TSX_ERR_INVALID, call, "n and l must be >= 0 and n * l under 2^31 - 1");
    const int rc = check_shape(call, d->dtype, d->n * d->l, d->c, d->form, d->block);
    if (rc != TSX_OK)
        return rc;
    if (d->param_dtype != TSX_F32 && d->param_dtype != d->dtype)
        return fail(TSX_ERR_INVALID, call, "weight and bias are fp32 or of the element type");
    if (!known_act(d->act))
        return fail(TSX_ERR_INVALID, call, "unknown activation");
    if (d->groups < 1 || d->c % d->groups != 0)
        return fail(TSX_ERR_INVALID, call, "c must be a multiple of groups >= 1");
    if (d->x_pitch < d->c || d->y_pitch < d->c)
        return fail(TSX_ERR_INVALID, call, "a pitch is shorter than a row");
    if (!(d->eps >= 0.f) || std::isinf(d->eps))
        return fail(TSX_ERR_INVALID, call, "eps must be finite and >= 0");
    return TSX_OK;
}

// The layout that a call takes: with vectors where its rows allow them and its
// groups' runs can start on them.
bool call_layout(const tsx_norm_desc& d, bool vec, int block, bool backward, bool held, NormLayout* out)
{
    return norm_layout(d, vec, block, backward, held, out) ||
           (vec && norm_layout(d, false, block, backward, held, out));
}

// Scratch that covers every layout the call may take.
size_t norm_workspace(const tsx_norm_desc& d, bool backward, bool aligned)
{
    size_t most = 0;
    if (d.n == 0 || d.l == 0 || d.c == 0)
        return 0;
    // rows of whole vectors: then an aligned call takes no other layout
    const int64_t es = elem_size(d.dtype);
    const bool whole = d.c % kOct == 0 && d.x_pitch * es % 16 == 0 && d.y_pitch * es % 16 == 0;
    for (int vec = aligned && whole ? 1 : 0; vec < (whole ? 2 : 1); ++vec)
        for (int held = 0; held < 2; ++held) {   // with a checkpoint, written or read
            NormLayout lay;
            if (!call_layout(d, vec != 0, held && !backward ? d.block : 0, backward, held != 0, &lay))
                continue;
            const size_t b = part_bytes(d, lay) + (backward ? chan_bytes(d, lay) : 0);
            most = b > most ? b : most;
        }
    return most;
}

int norm_args(const char* call, const tsx_norm_desc& d, bool vec, int block, bool backward, bool held, const void* weight,
              const void* bias, NormArgs* a)
{
    if (!call_layout(d, vec, block, backward, held, &a->lay))
        return fail(TSX_ERR_UNSUPPORTED, call, "no layout");
    if (a->lay.runs > kMaxChunks)
        return fail(TSX_ERR_UNSUPPORTED, call, "rows are too long");
    a->n = d.n;
    a->l = d.l;
    a->c = int(d.c);
    a->groups = d.groups;
    a->per_group = int(d.c / d.groups);
    a->x_pitch = d.x_pitch;
    a->y_pitch = d.y_pitch;
    a->eps = d.eps;
    a->act = d.act;
    a->form = d.form;
    a->block = d.block;
    a->blocks = (d.c + d.block - 1) / d.block;
    a->wide_params = d.param_dtype == TSX_F32;
    a->packed_params = aligned(weight, 16) && aligned(bias, 16);
    return TSX_OK;
}

int check_scratch(const char* call, size_t need, const void* workspace, size_t bytes)
{
    if (need == 0)
        return TSX_OK;
    if (bytes < need || !workspace)
        return fail(TSX_ERR_INVALID, call, "the workspace is smaller than tsx_group_norm_workspace says");
    if (!aligned(workspace, 16))
        return fail(TSX_ERR_ALIGN, call, "the workspace must be 16-byte aligned");
    return TSX_OK;
}

}  // namespace

extern "C" int tsx_group_norm_workspace(const tsx_norm_desc* desc, int backward, int aligned, size_t* bytes)
{
    const char* call = "tsx_group_norm_workspace";
    const int rc = check_norm(call, desc);
    if (rc != TSX_OK)
        return rc;
    if (!bytes)
        return fail(TSX_ERR_INVALID, call, "bytes is required");
    *bytes = norm_workspace(*desc, backward != 0, aligned != 0);
    set_last_error("");
    return TSX_OK;
}

extern "C" int tsx_group_norm(const tsx_norm_desc* desc, const void* x, const void* weight, const void* bias, void* y,
                              float* mean, float* rstd, void* q, float* scale, void* workspace,
                              size_t workspace_bytes, tsx_stream_t stream)
{
    const char* call = "tsx_group_norm";
    int rc = check_norm(call, desc);
    if (rc != TSX_OK)
        return rc;
    const tsx_norm_desc& d = *desc;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!q != !scale)
        return fail(TSX_ERR_INVALID, call, "q and scale come together");
    if (d.n == 0 || (d.c == 0 && !mean && !rstd))
        return launched(cudaSuccess, call);
    if (!mean || !rstd)
        return fail(TSX_ERR_INVALID, call, "mean and rstd are required");
    if (!aligned(mean, 4) || !aligned(rstd, 4))
        return fail(TSX_ERR_ALIGN, call, "a base pointer is not aligned to its elements");
    if (d.l == 0 || d.c == 0)
        return launched(launch_norm_empty(mean, rstd, d.n * d.groups, d.eps, st), call);
    if (!x || !weight || !bias || !y)
        return fail(TSX_ERR_INVALID, call, "x, weight, bias and y are required");
    const int es = elem_size(d.dtype), ps = elem_size(d.param_dtype);
    if (!aligned(x, es) || !aligned(y, es) || !aligned(weight, ps) || !aligned(bias, ps) || !aligned(scale, 4))
        return fail(TSX_ERR_ALIGN, call, "a base pointer is not aligned to its elements");
    const bool vec = vectors(x, d.c, d.x_pitch, es) && vectors(y, d.c, d.y_pitch, es) && held_vectors(q, d.c);
    // the checkpoint rides along where runs can start on its blocks
    NormLayout lay;
    const bool ride = q && call_layout(d, vec, d.block, false, true, &lay);
    NormArgs a{};
    rc = norm_args(call, d, vec, ride ? d.block : 0, false, ride, weight, bias, &a);
    if (rc == TSX_OK)
        rc = check_scratch(call, part_bytes(d, a.lay), workspace, workspace_bytes);
    if (rc != TSX_OK)
        return rc;
    if (q && !ride) {
        // before y is written: y may be x
        PackArgs p{};
        rc = pack_args(call, d.dtype, d.n * d.l, d.c, d.x_pitch, d.form, d.block, x, q, scale, &p);
        if (rc != TSX_OK)
            return rc;
        const cudaError_t e = launch_pack(d.dtype, p, x, HeldOut{q, scale}, st);
        if (e != cudaSuccess)
            return launched(e, call);
    }
    const NormScratch scratch{static_cast<float2*>(workspace), nullptr};
    const HeldOut held = ride ? HeldOut{q, scale} : HeldOut{nullptr, nullptr};
    cudaError_t e;
    if (a.lay.kind == kNormToken)
        e = launch_norm_token(d.dtype, a, x, weight, bias, y, mean, rstd, held, st);
    else if (a.lay.kind == kNormHeld)
        e = launch_norm_held(d.dtype, a, x, weight, bias, y, mean, rstd, held, st);
    else
        e = launch_norm(d.dtype, a, x, weight, bias, y, mean, rstd, held, scratch, st);
    return launched(e, call);
}

extern "C" int tsx_group_norm_backward(const tsx_norm_desc* desc, const void* dy, const void* x, const void* q,
                                       const float* scale, const void* weight, const void* bias, const float* mean,
                                       const float* rstd, void* dx, float* dweight, float* dbias, void* workspace,
                                       size_t workspace_bytes, tsx_stream_t stream)
{
    const char* call = "tsx_group_norm_backward";
    int rc = check_norm(call, desc);
    if (rc != TSX_OK)
        return rc;
    const tsx_norm_desc& d = *desc;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (d.c == 0)
        return launched(cudaSuccess, call);
    if (!dweight || !dbias)
        return fail(TSX_ERR_INVALID, call, "dweight and dbias are required");
    if (!aligned(dweight, 4) || !aligned(dbias, 4))
        return fail(TSX_ERR_ALIGN, call, "a base pointer is not aligned to its elements");
    if (d.n == 0 || d.l == 0) {
        cudaError_t e = cudaMemsetAsync(dweight, 0, size_t(d.c) * sizeof(float), st);
        if (e == cudaSuccess)
            e = cudaMemsetAsync(dbias, 0, size_t(d.c) * sizeof(float), st);
        return launched(e, call);
    }
    if (!q != !scale || !x == !q)
        return fail(TSX_ERR_INVALID, call, "either x, or its checkpoint q and scale");
    if (!dy || !weight || !bias || !mean || !rstd || !dx)
        return fail(TSX_ERR_INVALID, call, "dy, weight, bias, mean, rstd and dx are required");
    const int es = elem_size(d.dtype), ps = elem_size(d.param_dtype);
    if (!aligned(dy, es) || !aligned(x, es) || !aligned(dx, es) || !aligned(weight, ps) || !aligned(bias, ps) ||
        !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(scale, 4))
        return fail(TSX_ERR_ALIGN, call, "a base pointer is not aligned to its elements");
    const bool vec = vectors(dy, d.c, d.y_pitch, es) && vectors(x, d.c, d.x_pitch, es) &&
                     vectors(dx, d.c, d.x_pitch, es) && held_vectors(q, d.c);
    NormArgs a{};
    rc = norm_args(call, d, vec, 0, true, q != nullptr, weight, bias, &a);
    if (rc == TSX_OK)
        rc = check_scratch(call, part_bytes(d, a.lay) + chan_bytes(d, a.lay), workspace, workspace_bytes);
    if (rc != TSX_OK)
        return rc;
    NormScratch scratch;
    scratch.part = static_cast<float2*>(workspace);
    scratch.chan = reinterpret_cast<float*>(static_cast<char*>(workspace) + part_bytes(d, a.lay));
    const Saved saved{x, q, scale};
    const auto run = a.lay.kind == kNormToken  ? launch_norm_token_backward
                     : a.lay.kind == kNormHeld ? launch_norm_held_backward
                                               : launch_norm_backward;
    return launched(run(d.dtype, a, dy, saved, weight, bias, mean, rstd, dx, dweight, dbias, scratch, st), call);
}

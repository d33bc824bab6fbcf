// The C ABI of the operators around attention (include/tsx_attention.h):
// argument checks, frequencies, how heads are laid over threads, launches.

#include "attention.h"

#include <algorithm>
#include <cmath>
#include <cstdio>

#include "plan.h"

namespace tsx {
namespace {

constexpr int64_t kMostItems = 0x7fffffff - (1 << 20);   // tokens * heads
constexpr int64_t kMostPitch = int64_t(1) << 37;         // elements: strides of tensor maps are under 2^40 bytes

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
bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }
// Whether a pitch, or a pointer, is a multiple of 16 bytes; pitches of a dimension of one element are not used.
bool even(int64_t pitch, int64_t extent, int es) { return extent <= 1 || pitch * es % 16 == 0; }

int check_desc(const char* call, const tsx_rotary_desc* d)
{
    if (!d)
        return fail(TSX_ERR_INVALID, call, "the description is NULL");
    if (!known_dtype(d->dtype))
        return fail(TSX_ERR_INVALID, call, "unknown dtype");
    if (d->param_dtype != TSX_F32 && d->param_dtype != d->dtype)
        return fail(TSX_ERR_INVALID, call, "param_dtype must be fp32 or dtype");
    if (d->q_heads < 0 || d->k_heads < 0)
        return fail(TSX_ERR_INVALID, call, "q_heads and k_heads must not be negative");
    if (d->dim < 1 || d->dim > kRotaryDim)
        return fail(TSX_ERR_INVALID, call, "dim must be 1 .. 256");
    if (d->rot < 0 || d->rot > d->dim || d->rot % 2)
        return fail(TSX_ERR_INVALID, call, "rot must be even, 0 .. dim");
    if (d->layout != TSX_ROPE_HALF && d->layout != TSX_ROPE_INTERLEAVED)
        return fail(TSX_ERR_INVALID, call, "unknown rotary layout");
    if (d->norm != 0 && d->norm != 1)
        return fail(TSX_ERR_INVALID, call, "unknown norm");
    if (!(d->eps >= 0) || !std::isfinite(d->eps))
        return fail(TSX_ERR_INVALID, call, "eps must be finite and not negative");
    if (!std::isfinite(d->amplitude))
        return fail(TSX_ERR_INVALID, call, "the amplitude must be finite");
    return TSX_OK;
}

int check_tokens(const char* call, int64_t tokens, int64_t heads)
{
    if (tokens < 0 || tokens > kMostItems || tokens * std::max<int64_t>(heads, 1) > kMostItems)
        return fail(TSX_ERR_INVALID, call, "tokens, and tokens times heads, must be 0 .. 2^31 - 2^20");
    return TSX_OK;
}

int check_position_bytes(const char* call, int position_bytes)
{
    if (position_bytes != 4 && position_bytes != 8)
        return fail(TSX_ERR_INVALID, call, "positions have 4 or 8 bytes");
    return TSX_OK;
}

// A tensor [tokens, heads, dim] that the call needs: there, and no two of its elements in one place.
int check_heads(const char* call, const char* name, const tsx_heads* t, int64_t tokens, int64_t heads, int64_t dim, int es)
{
    char buf[128];
    if (!t || !t->data) {
        std::snprintf(buf, sizeof buf, "%s is required", name);
        return fail(TSX_ERR_INVALID, call, buf);
    }
    const int64_t pitch = t->pitch, head = t->head_pitch;
    bool ok = (tokens == 1 || (pitch >= 0 && pitch <= kMostPitch)) && (heads == 1 || (head >= 0 && head <= kMostPitch));
    if (ok && heads > 1 && tokens > 1)
        ok = (head >= dim && head <= pitch / heads) || (pitch >= dim && pitch <= head / tokens);
    else if (ok && heads > 1)
        ok = head >= dim;
    else if (ok && tokens > 1)
        ok = pitch >= dim;
    if (!ok) {
        std::snprintf(buf, sizeof buf, "the pitches of %s put heads or tokens over one another", name);
        return fail(TSX_ERR_INVALID, call, buf);
    }
    if (!aligned(t->data, size_t(es))) {
        std::snprintf(buf, sizeof buf, "%s is not aligned to its elements", name);
        return fail(TSX_ERR_ALIGN, call, buf);
    }
    return TSX_OK;
}

bool vectors(const tsx_heads* t, int64_t tokens, int64_t heads, int es)
{
    return aligned(t->data, 16) && even(t->pitch, tokens, es) && even(t->head_pitch, heads, es);
}

// Whether heads can be cut into eights of whole pairs.
bool eights(const tsx_rotary_desc& d)
{
    return d.dim % 8 == 0 && d.rot % 8 == 0;
}

void rotary_args(const tsx_rotary_desc& d, int64_t tokens, RotaryArgs* a)
{
    *a = RotaryArgs{};
    a->tokens = tokens;
    a->dim = d.dim;
    a->rot = d.rot;
    a->layout = d.layout;
    a->norm = d.norm;
    a->wide_params = d.param_dtype == TSX_F32;
    a->eps = d.eps;
    a->amplitude = d.amplitude;
    a->by_dim = 1.f / float(d.dim);
    a->team = 1;
    while (a->team * 8 < d.dim)
        a->team *= 2;
    std::copy(d.turns, d.turns + TSX_ROPE_PAIRS, a->turns);
}

RotaryRole role(int which, const tsx_heads* x, const tsx_heads* out, int heads, const void* weight)
{
    RotaryRole r{};
    r.which = which;
    r.x = static_cast<const char*>(x->data);
    r.x_pitch = x->pitch;
    r.x_head = x->head_pitch;
    if (out) {
        r.out = static_cast<char*>(out->data);
        r.out_pitch = out->pitch;
        r.out_head = out->head_pitch;
    }
    r.heads = heads;
    r.weight = weight;
    r.packed_weight = aligned(weight, 16);
    r.turn = which < 2;
    return r;
}

constexpr int64_t kSms = 152;   // a constant of the chip, not read from it: the order of sums depends on the shape alone
// Heads that a thread goes over with one set of sines, cosines and weights: forward
// bf16 [8192, 32 + 8, 128] with a norm 29.8 us in place of 33.3 with eight (27.2 and
// 27.9 without); the gradient through a norm 56.2 with eight and 70 with sixteen.
constexpr int kForwardHeads = 16, kBackwardHeads = 8;

// How a call's heads are shared out: teams of threads that take several heads of a
// token each, as many as leave two CTAs of work to each SM (one that stays), down to
// one.  Element by
// element a team is a warp.  wave: CTAs at most, each tensor's by its heads, which
// stay for all their tokens; 0: as many as there is work.
int lay_out(RotaryArgs* a, bool vec, int each, int64_t wave)
{
    const int64_t teams = kRotaryThreads / (vec ? a->team : 32);
    int64_t heads = 0;
    for (int i = 0; i < a->roles; ++i)
        heads += a->role[i].heads;
    each = int(std::max<int64_t>(std::min<int64_t>(each, a->tokens * heads / (teams * (wave ? 1 : 2) * kSms)), 1));
    int first = 0;
    for (int i = 0; i < a->roles; ++i) {
        RotaryRole& r = a->role[i];
        r.parts = (r.heads + each - 1) / each;
        r.first = first;
        const int64_t all = (a->tokens * r.parts + teams - 1) / teams;
        r.ctas = int(wave ? std::min(all, std::max<int64_t>(wave * r.heads / heads, 1)) : all);
        first += r.ctas;
    }
    return first;
}

int64_t slice_bytes(const RotaryArgs& a, int i) { return int64_t(a.role[i].ctas) * a.dim * 4; }

}  // namespace
}  // namespace tsx

using namespace tsx;

extern "C" int tsx_rotary_frequencies(int rot, double base, tsx_rope_scaling scaling, double factor, double length,
                                      double fast, double slow, double* frequencies, float* amplitude)
{
    const char* call = "tsx_rotary_frequencies";
    const double kPi = 3.14159265358979323846;
    if (rot < 0 || rot > kRotaryDim || rot % 2)
        return fail(TSX_ERR_INVALID, call, "rot must be even, 0 .. 256");
    if (!frequencies || !amplitude)
        return fail(TSX_ERR_INVALID, call, "frequencies and amplitude are required");
    if (!(base > 1) || !std::isfinite(base))
        return fail(TSX_ERR_INVALID, call, "base must be above 1");
    if (scaling < TSX_ROPE_PLAIN || scaling > TSX_ROPE_YARN)
        return fail(TSX_ERR_INVALID, call, "unknown scaling");
    if (scaling != TSX_ROPE_PLAIN && (!(factor >= 1) || !std::isfinite(factor)))
        return fail(TSX_ERR_INVALID, call, "factor must be at least 1");
    if (scaling == TSX_ROPE_YARN && (!(length > 0) || !(fast > 0) || !(slow > 0) || !std::isfinite(length) ||
                                     !std::isfinite(fast) || !std::isfinite(slow) || fast < slow))
        return fail(TSX_ERR_INVALID, call, "length and slow must be above 0, and fast at least slow");
    double first = 0, last = 0;
    if (scaling == TSX_ROPE_NTK && rot > 2)
        base *= std::pow(factor, double(rot) / (rot - 2));
    if (scaling == TSX_ROPE_YARN) {
        first = std::max(std::floor(rot * std::log(length / (2 * kPi * fast)) / (2 * std::log(base))), 0.0);
        last = std::min(std::ceil(rot * std::log(length / (2 * kPi * slow)) / (2 * std::log(base))), double(rot - 1));
    }
    for (int i = 0; i < rot / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot);
        if (scaling == TSX_ROPE_LINEAR)
            f /= factor;
        if (scaling == TSX_ROPE_YARN) {
            const double ramp = std::min(std::max((i - first) / std::max(last - first, 1e-3), 0.0), 1.0);
            f = std::fma(f / factor, ramp, f * (1 - ramp));
        }
        frequencies[i] = f;
    }
    *amplitude = scaling == TSX_ROPE_YARN ? float(1 + 0.1 * std::log(factor)) : 1.f;
    set_last_error("");
    return TSX_OK;
}

extern "C" int tsx_rotary_turns(int pairs, const double* frequencies, uint64_t* turns)
{
    const char* call = "tsx_rotary_turns";
    if (pairs < 0 || pairs > TSX_ROPE_PAIRS)
        return fail(TSX_ERR_INVALID, call, "0 .. 128 pairs");
    if (pairs && (!frequencies || !turns))
        return fail(TSX_ERR_INVALID, call, "frequencies and turns are required");
    // 2 pi as the sum of two doubles; the quotient f / (2 pi) as well, so that the
    // 64 bits of its fraction are good to a unit or two
    const double hi = 6.283185307179586, lo = 2.4492935982947064e-16;
    for (int i = 0; i < pairs; ++i) {
        const double f = std::fabs(frequencies[i]);
        if (!(f <= 0x1p30))
            return fail(TSX_ERR_INVALID, call, "frequencies must be finite, 2^30 at most");
        const double q = f / hi;
        const double rest = std::fma(-q, lo, std::fma(-q, hi, f));
        const double whole = std::floor(q);
        // q - whole is exact; both parts in units of 2^-64, where 2^64 itself is 0 again
        const double big = std::ldexp(q - whole, 64), small = std::ldexp(rest / hi, 64);
        const uint64_t b = big >= 0x1p64 ? 0 : uint64_t(big);
        const uint64_t t = b + uint64_t(int64_t(std::nearbyint(small + (big >= 0x1p64 ? 0 : big - double(b)))));
        turns[i] = frequencies[i] < 0 ? 0 - t : t;
    }
    set_last_error("");
    return TSX_OK;
}

namespace {

int check_outputs(const char* call, const tsx_rotary_desc& d, int64_t tokens, const tsx_heads* q, const tsx_heads* k,
                  const tsx_heads* q_out, const tsx_heads* k_out, const char* const (&names)[4])
{
    const int es = elem_size(d.dtype);
    int rc = TSX_OK;
    if (d.q_heads) {
        rc = check_heads(call, names[0], q, tokens, d.q_heads, d.dim, es);
        if (rc == TSX_OK)
            rc = check_heads(call, names[2], q_out, tokens, d.q_heads, d.dim, es);
    }
    if (rc == TSX_OK && d.k_heads) {
        rc = check_heads(call, names[1], k, tokens, d.k_heads, d.dim, es);
        if (rc == TSX_OK)
            rc = check_heads(call, names[3], k_out, tokens, d.k_heads, d.dim, es);
    }
    return rc;
}

int check_weights(const char* call, const tsx_rotary_desc& d, const void* q_weight, const void* k_weight)
{
    if (!d.norm && (q_weight || k_weight))
        return fail(TSX_ERR_INVALID, call, "weights belong to a norm");
    const size_t es = size_t(elem_size(d.param_dtype));
    if (!aligned(q_weight, es) || !aligned(k_weight, es))
        return fail(TSX_ERR_ALIGN, call, "a weight is not aligned to its elements");
    return TSX_OK;
}

int check_positions(const char* call, const void* positions, int position_bytes)
{
    if (!positions)
        return fail(TSX_ERR_INVALID, call, "positions are required");
    if (!aligned(positions, size_t(position_bytes)))
        return fail(TSX_ERR_ALIGN, call, "positions are not aligned to their elements");
    return TSX_OK;
}

}  // namespace

extern "C" int tsx_rotary(const tsx_rotary_desc* desc, int64_t tokens, const void* positions, int position_bytes,
                          const tsx_heads* q, const tsx_heads* k, const void* q_weight, const void* k_weight,
                          const tsx_heads* q_out, const tsx_heads* k_out, tsx_stream_t stream)
{
    const char* call = "tsx_rotary";
    int rc = check_desc(call, desc);
    if (rc == TSX_OK)
        rc = check_tokens(call, tokens, std::max(desc->q_heads, desc->k_heads));
    if (rc == TSX_OK)
        rc = check_position_bytes(call, position_bytes);
    if (rc == TSX_OK)
        rc = check_weights(call, *desc, q_weight, k_weight);
    if (rc != TSX_OK)
        return rc;
    const tsx_rotary_desc& d = *desc;
    if (tokens == 0 || (d.q_heads == 0 && d.k_heads == 0))
        return launched(cudaSuccess, call);
    rc = check_positions(call, positions, position_bytes);
    if (rc == TSX_OK)
        rc = check_outputs(call, d, tokens, q, k, q_out, k_out, {"q", "k", "q_out", "k_out"});
    if (rc != TSX_OK)
        return rc;
    RotaryArgs a;
    rotary_args(d, tokens, &a);
    a.positions = positions;
    a.wide_positions = position_bytes == 8;
    const int es = elem_size(d.dtype);
    bool vec = eights(d);
    if (d.q_heads) {
        vec = vec && vectors(q, tokens, d.q_heads, es) && vectors(q_out, tokens, d.q_heads, es);
        a.role[a.roles++] = role(0, q, q_out, d.q_heads, q_weight);
    }
    if (d.k_heads) {
        vec = vec && vectors(k, tokens, d.k_heads, es) && vectors(k_out, tokens, d.k_heads, es);
        a.role[a.roles++] = role(1, k, k_out, d.k_heads, k_weight);
    }
    const int ctas = lay_out(&a, vec, kForwardHeads, 0);
    return launched(launch_rotary(d.dtype, a, vec, ctas, reinterpret_cast<cudaStream_t>(stream)), call);
}

extern "C" int tsx_rotary_workspace(const tsx_rotary_desc* desc, int64_t tokens, size_t* bytes)
{
    const char* call = "tsx_rotary_workspace";
    int rc = check_desc(call, desc);
    if (rc == TSX_OK)
        rc = check_tokens(call, tokens, std::max(desc->q_heads, desc->k_heads));
    if (rc != TSX_OK)
        return rc;
    if (!bytes)
        return fail(TSX_ERR_INVALID, call, "bytes is NULL");
    // a slice to each CTA: a wave's at most, whatever the layout
    *bytes = desc->norm && tokens ? size_t(backward_ctas(desc->dtype) * kSms + 2) * desc->dim * 4 : 0;
    set_last_error("");
    return TSX_OK;
}

extern "C" int tsx_rotary_backward(const tsx_rotary_desc* desc, int64_t tokens, const void* positions,
                                   int position_bytes, const tsx_heads* dq, const tsx_heads* dk, const tsx_heads* q,
                                   const tsx_heads* k, const void* q_weight, const void* k_weight,
                                   const tsx_heads* dq_out, const tsx_heads* dk_out, float* dq_weight,
                                   float* dk_weight, void* workspace, size_t workspace_bytes, tsx_stream_t stream)
{
    const char* call = "tsx_rotary_backward";
    int rc = check_desc(call, desc);
    if (rc == TSX_OK)
        rc = check_tokens(call, tokens, std::max(desc->q_heads, desc->k_heads));
    if (rc == TSX_OK)
        rc = check_position_bytes(call, position_bytes);
    if (rc == TSX_OK)
        rc = check_weights(call, *desc, q_weight, k_weight);
    if (rc != TSX_OK)
        return rc;
    const tsx_rotary_desc& d = *desc;
    if (!!q_weight != !!dq_weight || !!k_weight != !!dk_weight)
        return fail(TSX_ERR_INVALID, call, "a weight and its gradient are given together");
    if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4))
        return fail(TSX_ERR_ALIGN, call, "a weight's gradient is not aligned to its elements");
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (tokens == 0 || (d.q_heads == 0 && d.k_heads == 0)) {
        cudaError_t e = cudaSuccess;
        for (float* w : {dq_weight, dk_weight})
            if (w && e == cudaSuccess)
                e = cudaMemsetAsync(w, 0, size_t(d.dim) * 4, st);
        return launched(e, call);
    }
    rc = check_positions(call, positions, position_bytes);
    if (rc == TSX_OK)
        rc = check_outputs(call, d, tokens, dq, dk, dq_out, dk_out, {"dq", "dk", "dq_out", "dk_out"});
    if (rc != TSX_OK)
        return rc;
    const int es = elem_size(d.dtype);
    if (!d.norm && (q || k))
        return fail(TSX_ERR_INVALID, call, "q and k belong to the gradient of a norm");
    if (d.norm && d.q_heads)
        rc = check_heads(call, "q", q, tokens, d.q_heads, d.dim, es);
    if (rc == TSX_OK && d.norm && d.k_heads)
        rc = check_heads(call, "k", k, tokens, d.k_heads, d.dim, es);
    if (rc != TSX_OK)
        return rc;
    RotaryArgs a;
    rotary_args(d, tokens, &a);
    a.positions = positions;
    a.wide_positions = position_bytes == 8;
    bool vec = eights(d);
    const tsx_heads* in[2] = {dq, dk};
    const tsx_heads* saved[2] = {q, k};
    const tsx_heads* out[2] = {dq_out, dk_out};
    const int heads[2] = {d.q_heads, d.k_heads};
    const void* weight[2] = {q_weight, k_weight};
    for (int i = 0; i < 2; ++i) {
        if (!heads[i])
            continue;
        RotaryRole r = role(i, in[i], out[i], heads[i], weight[i]);
        vec = vec && vectors(in[i], tokens, heads[i], es) && vectors(out[i], tokens, heads[i], es);
        if (d.norm) {
            vec = vec && vectors(saved[i], tokens, heads[i], es);
            r.saved = static_cast<const char*>(saved[i]->data);
            r.saved_pitch = saved[i]->pitch;
            r.saved_head = saved[i]->head_pitch;
        }
        a.role[a.roles++] = r;
    }
    if (!d.norm) {   // turned by the opposite angles
        for (uint64_t& t : a.turns)
            t = 0 - t;
        const int ctas = lay_out(&a, vec, kForwardHeads, 0);
        return launched(launch_rotary(d.dtype, a, vec, ctas, st), call);
    }
    const int ctas = lay_out(&a, vec, kBackwardHeads, backward_ctas(d.dtype) * kSms);
    const bool sums = dq_weight || dk_weight;
    if (sums) {
        int64_t need = 0;
        for (int i = 0; i < a.roles; ++i) {
            if (a.role[i].weight)
                a.role[i].slices = reinterpret_cast<float*>(static_cast<char*>(workspace) + need);
            need += slice_bytes(a, i);
        }
        if (!workspace || workspace_bytes < size_t(need))
            return fail(TSX_ERR_INVALID, call, "the workspace is smaller than tsx_rotary_workspace says");
        if (!aligned(workspace, 16))
            return fail(TSX_ERR_ALIGN, call, "the workspace is not aligned to 16 bytes");
    }
    cudaError_t e = launch_rotary_norm_backward(d.dtype, a, vec, ctas, st);
    if (e == cudaSuccess && sums)
        e = launch_rotary_weights(a, dq_weight, dk_weight, st);
    return launched(e, call);
}

namespace {

int check_cache(const char* call, const tsx_cache* c)
{
    if (!c)
        return fail(TSX_ERR_INVALID, call, "the cache is NULL");
    if (!known_dtype(c->dtype))
        return fail(TSX_ERR_INVALID, call, "unknown dtype");
    if (c->heads < 1 || c->heads > 65535 || c->dim < 1 || c->dim > kRotaryDim)
        return fail(TSX_ERR_INVALID, call, "the cache has 1 .. 65535 heads of 1 .. 256 channels");
    if (c->page_size < 1 || c->page_size > (1 << 20) || c->pages < 0 || c->pages > 0x7fffffff)
        return fail(TSX_ERR_INVALID, call, "the cache has up to 2^31 - 1 pages of 1 .. 2^20 slots");
    const int64_t slot = c->slot_pitch, head = c->head_pitch, page = c->page_pitch;
    if (slot < 0 || head < 0 || page < 0 || slot > kMostPitch || head > kMostPitch || page > kMostPitch)
        return fail(TSX_ERR_INVALID, call, "a pitch of the cache is negative or too large");
    const int64_t slots = c->page_size, heads = c->heads, dim = c->dim;
    // the furthest element of a page, with either of slots and heads outside
    bool ok = true;
    if (slots > 1 && heads > 1)
        ok = (head >= dim && head <= slot / heads) || (slot >= dim && slot <= head / slots);
    else if (heads > 1)
        ok = head >= dim;
    else if (slots > 1)
        ok = slot >= dim;
    const int64_t extent = (slots - 1) * slot * (slots > 1) + (heads - 1) * head * (heads > 1) + dim;
    if (!ok || (c->pages > 1 && page < extent))
        return fail(TSX_ERR_INVALID, call, "the pitches of the cache put slots, heads or pages over one another");
    if (c->pages && (!c->k || !c->v))
        return fail(TSX_ERR_INVALID, call, "the cache's k and v are required");
    const size_t es = size_t(elem_size(c->dtype));
    if (!aligned(c->k, es) || !aligned(c->v, es))
        return fail(TSX_ERR_ALIGN, call, "the cache is not aligned to its elements");
    return TSX_OK;
}

int check_batch(const char* call, const tsx_batch* b)
{
    if (!b)
        return fail(TSX_ERR_INVALID, call, "the batch is NULL");
    if (b->seqs < 0 || b->seqs > (1 << 24) || b->most_pages < 0)
        return fail(TSX_ERR_INVALID, call, "seqs must be 0 .. 2^24 and most_pages not negative");
    if (b->seqs > 1 && (b->pages_pitch < b->most_pages || b->pages_pitch > kMostPitch))
        return fail(TSX_ERR_INVALID, call, "pages_pitch is shorter than a page list");
    if (b->seqs && (!b->starts || !b->lengths || (b->most_pages && !b->pages)))
        return fail(TSX_ERR_INVALID, call, "starts, lengths and pages are required");
    if (!aligned(b->starts, 4) || !aligned(b->lengths, 4) || !aligned(b->pages, 4))
        return fail(TSX_ERR_ALIGN, call, "starts, lengths or pages are not aligned to their elements");
    return TSX_OK;
}

PagedArgs paged_args(const tsx_cache& c, const tsx_batch& b)
{
    PagedArgs p{};
    p.starts = b.starts;
    p.lengths = b.lengths;
    p.pages = b.pages;
    p.pages_pitch = b.pages_pitch;
    p.cache_pages = c.pages;
    p.page_pitch = c.page_pitch;
    p.seqs = b.seqs;
    p.most_pages = b.most_pages;
    p.page_size = c.page_size;
    p.page_shift = -1;
    if ((c.page_size & (c.page_size - 1)) == 0)
        for (p.page_shift = 0; 1 << p.page_shift < c.page_size; ++p.page_shift) {
        }
    return p;
}

bool cache_vectors(const tsx_cache& c)
{
    const int es = elem_size(c.dtype);
    return aligned(c.k, 16) && aligned(c.v, 16) && even(c.page_pitch, c.pages, es) &&
           even(c.slot_pitch, c.page_size, es) && even(c.head_pitch, c.heads, es);
}

}  // namespace

extern "C" int tsx_cache_append(const tsx_rotary_desc* desc, const tsx_cache* cache, const tsx_batch* batch,
                                int64_t tokens, const tsx_heads* q, const tsx_heads* k, const tsx_heads* v,
                                const void* q_weight, const void* k_weight, const tsx_heads* q_out,
                                tsx_stream_t stream)
{
    const char* call = "tsx_cache_append";
    int rc = check_desc(call, desc);
    if (rc == TSX_OK)
        rc = check_cache(call, cache);
    if (rc == TSX_OK)
        rc = check_batch(call, batch);
    if (rc == TSX_OK)
        rc = check_tokens(call, tokens, std::max(desc->q_heads, desc->k_heads));
    if (rc == TSX_OK)
        rc = check_weights(call, *desc, q_weight, k_weight);
    if (rc != TSX_OK)
        return rc;
    const tsx_rotary_desc& d = *desc;
    if (d.dtype != cache->dtype || d.k_heads != cache->heads || d.dim != cache->dim)
        return fail(TSX_ERR_INVALID, call, "dtype, k_heads and dim must be the cache's");
    if (tokens == 0 || batch->seqs == 0)
        return launched(cudaSuccess, call);
    const int es = elem_size(d.dtype);
    rc = check_heads(call, "k", k, tokens, d.k_heads, d.dim, es);
    if (rc == TSX_OK)
        rc = check_heads(call, "v", v, tokens, d.k_heads, d.dim, es);
    if (rc == TSX_OK && d.q_heads)
        rc = check_heads(call, "q", q, tokens, d.q_heads, d.dim, es);
    if (rc == TSX_OK && d.q_heads)
        rc = check_heads(call, "q_out", q_out, tokens, d.q_heads, d.dim, es);
    if (rc != TSX_OK)
        return rc;
    RotaryArgs a;
    rotary_args(d, tokens, &a);
    a.paged = paged_args(*cache, *batch);
    bool vec = eights(d) && cache_vectors(*cache) && vectors(k, tokens, d.k_heads, es) && vectors(v, tokens, d.k_heads, es);
    if (d.q_heads) {
        vec = vec && vectors(q, tokens, d.q_heads, es) && vectors(q_out, tokens, d.q_heads, es);
        a.role[a.roles++] = role(0, q, q_out, d.q_heads, q_weight);
    }
    const tsx_heads slots[2] = {{cache->k, cache->slot_pitch, cache->head_pitch},
                                {cache->v, cache->slot_pitch, cache->head_pitch}};
    a.role[a.roles++] = role(1, k, &slots[0], d.k_heads, k_weight);
    a.role[a.roles++] = role(2, v, &slots[1], d.k_heads, nullptr);
    for (int i = 0; i < a.roles; ++i)
        a.role[i].paged = a.role[i].which > 0;
    const int ctas = lay_out(&a, vec, kForwardHeads, 0);
    return launched(launch_rotary(d.dtype, a, vec, ctas, reinterpret_cast<cudaStream_t>(stream)), call);
}

namespace {

// Whether a step's 128 keys are whole pages, or part of one, that start on the
// eight rows of the swizzle: then boxes of the pages can be copied.
bool box_pages(const tsx_cache& c)
{
    return c.pages > 0 && c.page_size >= 8 && (c.page_size & (c.page_size - 1)) == 0;
}

int cache_maps(const tsx_cache& c, CUtensorMap (&maps)[2])
{
    const uint64_t es = uint64_t(elem_size(c.dtype)), one = 16;   // a stride that is not used
    const uint64_t dims[4] = {uint64_t(c.dim), uint64_t(c.page_size), uint64_t(c.heads), uint64_t(c.pages)};
    const uint64_t strides[3] = {c.page_size > 1 ? uint64_t(c.slot_pitch) * es : one,
                                 c.heads > 1 ? uint64_t(c.head_pitch) * es : one,
                                 c.pages > 1 ? uint64_t(c.page_pitch) * es : one};
    const uint32_t box[4] = {64, uint32_t(std::min(c.page_size, 128)), 1, 1};
    const int rc = encode_pages_map(c.dtype, c.k, dims, strides, box, &maps[0]);
    return rc != TSX_OK ? rc : encode_pages_map(c.dtype, c.v, dims, strides, box, &maps[1]);
}

// Bytes of the parts of an attention call: their sums, statistics and tails, and the
// sums that threads fold.
struct Parts {
    int rows, ctas, padded;
    bool many() const { return rows == attend_many_rows(); }
    size_t sums() const { return size_t(2) * ctas * rows * padded * 4; }
    size_t stats() const { return size_t(2) * ctas * rows * 8; }
    size_t tails() const { return size_t(ctas) * 32; }
    size_t folded() const { return size_t(ctas) * fold_threads(many()) * (fold_fours(many(), padded) + 1) * 16; }
    size_t bytes() const { return sums() + stats() + tails() + folded(); }
};

// By rows to a head: tiles of 8 or 16 for as many, and of many for more in heads of up to
// 128 channels.
Parts parts_of(int dim, int64_t most_new, int group)
{
    const int padded = dim <= 64 ? 64 : dim <= 128 ? 128 : 256;
    if (dim <= 128 && most_new * group > 16)
        return Parts{attend_many_rows(), 152, padded};
    return Parts{most_new * group > 8 ? 16 : 8, attend_few_ctas(dim), padded};
}

int check_attention(const char* call, const tsx_cache* cache, int64_t tokens, int q_heads, int64_t most_new)
{
    int rc = check_cache(call, cache);
    if (rc != TSX_OK)
        return rc;
    if (q_heads < 1 || q_heads % cache->heads)
        return fail(TSX_ERR_INVALID, call, "q_heads must be a multiple of the cache's heads");
    if (most_new < 0 || most_new > kMostItems)
        return fail(TSX_ERR_INVALID, call, "most_new must be 0 .. 2^31 - 2^20");
    return check_tokens(call, tokens, q_heads);
}

}  // namespace

extern "C" int tsx_paged_attention_workspace(const tsx_cache* cache, int64_t tokens, int q_heads, int64_t most_new,
                                             size_t* bytes)
{
    const char* call = "tsx_paged_attention_workspace";
    const int rc = check_attention(call, cache, tokens, q_heads, most_new);
    if (rc != TSX_OK)
        return rc;
    if (!bytes)
        return fail(TSX_ERR_INVALID, call, "bytes is NULL");
    *bytes = parts_of(cache->dim, most_new, q_heads / cache->heads).bytes();
    set_last_error("");
    return TSX_OK;
}

extern "C" int tsx_paged_attention(const tsx_cache* cache, const tsx_batch* batch, int64_t tokens, int q_heads,
                                   int64_t most_new, float scale, const tsx_heads* q, const tsx_heads* out, float* lse,
                                   void* workspace, size_t workspace_bytes, tsx_stream_t stream)
{
    const char* call = "tsx_paged_attention";
    int rc = check_attention(call, cache, tokens, q_heads, most_new);
    if (rc == TSX_OK)
        rc = check_batch(call, batch);
    if (rc != TSX_OK)
        return rc;
    if (!(std::fabs(scale) <= 0x1p127f))   // scale / ln 2 is an fp32 number too
        return fail(TSX_ERR_INVALID, call, "scale must be finite, 2^127 at most");
    if (cache->dtype == TSX_F32)
        return fail(TSX_ERR_UNSUPPORTED, call, "fp32 is not supported: fp16 and bf16 are");
    if (cache->dim % 8)
        return fail(TSX_ERR_UNSUPPORTED, call, "dim must be a multiple of 8");
    if (tokens == 0 || batch->seqs == 0)
        return launched(cudaSuccess, call);
    rc = check_heads(call, "q", q, tokens, q_heads, cache->dim, 2);
    if (rc == TSX_OK)
        rc = check_heads(call, "out", out, tokens, q_heads, cache->dim, 2);
    if (rc != TSX_OK)
        return rc;
    if (!cache_vectors(*cache) || !vectors(q, tokens, q_heads, 2) || !vectors(out, tokens, q_heads, 2) ||
        !aligned(lse, 4) || !aligned(workspace, 16))
        return fail(TSX_ERR_ALIGN, call, "pitches must be multiples of 8 elements and pointers of 16 bytes");
    const Parts parts = parts_of(cache->dim, most_new, q_heads / cache->heads);
    if (!workspace || workspace_bytes < parts.bytes())
        return fail(TSX_ERR_INVALID, call, "the workspace is smaller than tsx_paged_attention_workspace says");
    AttendArgs a{};
    a.paged = paged_args(*cache, *batch);
    // without pages nothing is read, but copies of no bytes name an address
    a.k = static_cast<const char*>(cache->pages ? cache->k : q->data);
    a.v = static_cast<const char*>(cache->pages ? cache->v : q->data);
    a.q = static_cast<const char*>(q->data);
    a.out = static_cast<char*>(out->data);
    a.lse = lse;
    a.slot_pitch = cache->slot_pitch;
    a.head_pitch = cache->head_pitch;
    a.q_pitch = q->pitch;
    a.q_head = q->head_pitch;
    a.out_pitch = out->pitch;
    a.out_head = out->head_pitch;
    a.tokens = tokens;
    a.heads = cache->heads;
    a.group = q_heads / cache->heads;
    a.dim = cache->dim;
    a.scale_log2 = float(double(scale) * 1.44269504088896340736);
    a.ctas = parts.ctas;
    char* scratch = static_cast<char*>(workspace);
    a.parts = reinterpret_cast<float*>(scratch);
    a.stats = reinterpret_cast<float2*>(scratch + parts.sums());
    a.tails = reinterpret_cast<dev::Tail*>(scratch + parts.sums() + parts.stats());
    a.folded = reinterpret_cast<float4*>(scratch + parts.sums() + parts.stats() + parts.tails());
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!parts.many())
        return launched(launch_attend_few(cache->dtype, a, parts.rows, st), call);
    // a positive scale, so that the largest score is the largest product; not 0, which -infinity must not meet: with
    // the least number above it the largest product's score is 2^-21
    a.negated = a.scale_log2 < 0;
    a.scale_log2 = std::max(std::fabs(a.scale_log2), 0x1p-149f);
    CUtensorMap maps[2];
    const bool boxes = box_pages(*cache);
    if (boxes) {
        rc = cache_maps(*cache, maps);
        if (rc != TSX_OK)
            return rc;
    }
    return launched(launch_attend_many(cache->dtype, a, boxes ? maps : nullptr, st), call);
}

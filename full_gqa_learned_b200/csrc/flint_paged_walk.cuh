// How the step kernel (flint_paged_step.cu) shares its work out, in code that
// also runs on the host: the tiles of a sequence, the place where a CTA's share
// begins, and the walk over the share's pairs.
#pragma once
#include <algorithm>

#include "flint_paged.cuh"

namespace flint {

#ifndef __CUDA_ARCH__
using std::max;
using std::min;
#endif

// A walk over a share of the step's work: the pairs (row group, KV head),
// sequence by sequence, group by group, head by head.
struct StepWalk {
    int b, a, n, len;            // the sequence, its first packed row, new tokens, cached positions
    int z1, len1;                // the next sequence's end and cached positions, on their way
    int row0, head, off, left;   // next pair: first row, head, tile it is entered at; tiles left in the share
    bool ill;                    // the plan found ill-formed entries
};
struct StepSeg {
    int b, head, p0, row, nrows, tiles, t0, t1;
    bool whole;
};
// Tiles start at a multiple of the box: min(page, tile).
__host__ __device__ __forceinline__ int step_base(const PagedAttnParams& p, int lo, int tile) {
    return lo & ~(min(1 << p.c.ps_log2, tile) - 1);
}
__host__ __device__ __forceinline__ int step_tiles(const PagedAttnParams& p, int p0, int nrows, int tile) {
    const int lo = p.window > 0 ? max(0, p0 - p.window + 1) : 0;
    return (p0 + nrows - step_base(p, lo, tile) + tile - 1) / tile;
}
// Enters sequence b (rows [a, z), cached positions len), or the next one with
// new tokens; the whole warp calls it.  Runs of empty sequences are skipped by
// one search: their boundaries are all z.  That holds for non-decreasing
// boundaries only (a search over falling ones may jump over sequences that the
// plan counted), so a call with ill-formed entries goes from sequence to
// sequence, as the plan does.  n <= 0 afterwards: there is none.
__host__ __device__ __forceinline__ void step_enter(const PagedAttnParams& p, StepWalk& w, int b, int a, int z, int len) {
    const PagedCache& c = p.c;
    for (;;) {
        const int n = paged_new(c, p.max_new, a, z, len);
        w.b = b;
        w.a = a;
        w.n = n;
        w.len = len;
        const bool more = b + 1 < c.B;
        w.z1 = more ? paged_ld(c.cu + b + 2) : 0;
        w.len1 = more ? paged_ld(c.len + b + 1) : 0;
        if (n > 0 || !more) return;
        a = z;
        ++b;
        if (w.ill || w.z1 > a) {
            z = w.z1;
            len = w.len1;
        } else {
            b += warp_last_leq(c.cu + b, c.B - b, a);
            a = paged_ld(c.cu + b);
            z = paged_ld(c.cu + b + 1);
            len = paged_ld(c.len + b);
        }
    }
}
template <int NT>
__host__ __device__ __forceinline__ bool step_next(const PagedAttnParams& p, StepWalk& w, StepSeg& s, int tile) {
    if (w.left <= 0) return false;
    s.b = w.b;
    s.head = w.head;
    s.p0 = w.len + w.row0;
    s.row = w.a + w.row0;
    s.nrows = min(NT, w.n - w.row0);
    s.tiles = step_tiles(p, s.p0, s.nrows, tile);
    s.t0 = w.off;
    s.t1 = min(s.tiles, w.off + w.left);
    s.whole = s.t0 == 0 && s.t1 == s.tiles;
    w.left -= s.t1 - s.t0;
    w.off = 0;
    if (++w.head == p.c.ng) {
        w.head = 0;
        w.row0 += NT;
        if (w.row0 >= w.n) {
            w.row0 = 0;
            // the last sequence ends the walk, whatever is left of the share
            if (w.b + 1 >= p.c.B) w.left = 0;
            if (w.left > 0) {
                step_enter(p, w, w.b + 1, paged_ld(p.c.cu + w.b + 1), w.z1, w.len1);
                if (w.n <= 0) w.left = 0;
            }
        }
    }
    return true;
}

// Tiles (of one head) of the sequence with rows [a, z) at positions len ..;
// *ill where its entries are ill-formed (it has none then).
template <int NT>
__host__ __device__ __forceinline__ long long step_seq_tiles(const PagedAttnParams& p, int a, int z, int len, int tile, bool* ill) {
    const int n = paged_new(p.c, p.max_new, a, z, len);
    if (n < 0) *ill = true;
    long long sum = 0;
    for (int r = 0; r < n; r += NT) sum += step_tiles(p, len + r, min(NT, n - r), tile);
    return sum;
}
// Where tile `in` of the pairs of sequences [b0, b1) lies: at = the sequence,
// its group's first row, the head, the tile of that pair.
template <int NT>
__host__ __device__ __forceinline__ void step_place(const PagedAttnParams& p, int b0, int b1, long long in, int tile, int* at) {
    const PagedCache& c = p.c;
    for (int b = b0; b < b1; ++b) {
        const int len = paged_ld(c.len + b), a = paged_ld(c.cu + b), z = paged_ld(c.cu + b + 1);
        const int n = paged_new(c, p.max_new, a, z, len);
        for (int r = 0; r < n; r += NT) {
            const long long tl = step_tiles(p, len + r, min(NT, n - r), tile);
            if (in < tl * c.ng) {
                at[0] = b;
                at[1] = r;
                at[2] = (int)(in / tl);
                at[3] = (int)(in % tl);
                return;
            }
            in -= tl * c.ng;
        }
    }
}
// Begins the walk over a share of `left` tiles at that place.
__host__ __device__ __forceinline__ void step_begin(const PagedAttnParams& p, StepWalk& w, const int* at, int left, bool ill) {
    const int b = at[0];
    w.ill = ill;
    step_enter(p, w, b, paged_ld(p.c.cu + b), paged_ld(p.c.cu + b + 1), paged_ld(p.c.len + b));
    w.row0 = at[1];
    w.head = at[2];
    w.off = at[3];
    w.left = left;
}
}  // namespace flint

// Host-and-device arithmetic of attention's plan (attn.cu): the line of tiles
// that the requests' own keys form, and its cut into one part per CTA.  Kept
// free of device intrinsics so that a host compiler can build it for the
// plan's tests.
//
// A head's line holds its segments one after the other, each with the cost of
// its start and of its tiles; the heads' lines follow each other.  A position
// on the line is a cost, and a CTA has the tiles whose positions lie in its
// part.
#pragma once

#ifndef __CUDACC__
#ifndef __host__
#define __host__
#define __device__
#endif
#endif

namespace attnline {

constexpr int OV = 2;   // cost of an item's start, in tiles
constexpr int OVP = 3;  // the same with the partial result of a prefix item

// A plan may hold 2^23 segments of 2^24 tiles: one causal prompt of 741000
// tokens at 128 query heads a key/value head already costs more than 2^31.
typedef long long cost_t;

__host__ __device__ inline cost_t segment_cost(int ntile) { return (cost_t)ntile + OV; }

// largest i in [0, n) with a(i) <= x (a ascending, a(0) <= x)
template <class F>
__host__ __device__ inline int upper(int n, long long x, F a) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((long long)a(mid) <= x) lo = mid; else hi = mid;
    }
    return lo;
}

struct Line {
    cost_t cost;    // of one head
    cost_t S;       // of all heads
    int n_seg;      // segments of a head
    int k0, n1;     // prefix items of a CTA, and how many CTAs (the first ones) have one more
    long long q0, q1;  // line cost of a CTA, and of one with one prefix item more

    // n_items prefix items of c tiles are dealt out to the CTAs beside the line
    __host__ __device__ Line(cost_t cost_, int Hkv, int n_seg_, int n_cta, int n_items, int c)
        : cost(cost_), S(cost_ * Hkv), n_seg(n_seg_), k0(n_items / n_cta), n1(n_items % n_cta), q1(0) {
        const int n0 = n_cta - n1;
        const long long p0 = (long long)k0 * (c + OVP), p1 = p0 + (n1 ? c + OVP : 0);
        const long long W = (S + n1 * p1 + n0 * p0 + n_cta - 1) / n_cta;
        if (n1 && W <= p1) {
            q0 = (S + n0 - 1) / n0;
        } else {
            q1 = n1 ? W - p1 : 0;
            q0 = W - p0;
        }
        if (q0 < 1) q0 = 1;
    }
    // the part of CTA i is [start_of(i), start_of(i + 1))
    __host__ __device__ long long start_of(int i) const {
        const long long x = i < n1 ? i * q1 : n1 * q1 + (i - n1) * q0;
        return x < S ? x : S;
    }
    __host__ __device__ int cta_of(long long x) const {
        return x < n1 * q1 ? (int)(x / q1) : n1 + (int)((x - n1 * q1) / q0);
    }
    // head * n_seg + segment that holds position x; cum(i): cost of a head's segments before segment i
    template <class F>
    __host__ __device__ int at(long long x, F cum) const {
        const int h = (int)(x / cost);
        return h * n_seg + upper(n_seg, x - h * cost, cum);
    }
    template <class F>
    __host__ __device__ long long begin_of(int l, F cum) const {
        return (l / n_seg) * cost + cum(l % n_seg);
    }
    // tiles [t0, t1) of a segment that begins at b and has ntile tiles, in the part [x0, x1)
    __host__ __device__ static void tiles(long long b, int ntile, long long x0, long long x1, int& t0, int& t1) {
        const long long a = x0 - b - OV, e = x1 - b - OV;
        t0 = (int)(a > 0 ? a : 0);
        t1 = (int)(e < 0 ? 0 : e < ntile ? e : ntile);
    }
    // items of the part [x0, x1), which is not empty and goes from segment l0 to l1, which begins at b1: where only
    // the start cost of the last one lies in it, its tiles are the next CTA's
    __host__ __device__ static int items(int l0, int l1, long long b1, long long x1) {
        return l1 - l0 + 1 - (x1 - b1 <= OV ? 1 : 0);
    }
    // the CTAs that have the first and the last of its tiles
    __host__ __device__ void holders(long long b, int ntile, int& c0, int& c1) const {
        c0 = cta_of(b + OV);
        c1 = cta_of(b + OV + ntile - 1);
    }
};

}  // namespace attnline

// ft_beam_select: the N best of K*V continuations of each request.
//
//   score(k, v) = s_k + x_kv - lse_k,   lse_k = log(sum over u of exp x_ku)
//
// Bound: HBM for large batches (the logits are read once), latency for small
// ones.  One kernel.  A CTA takes a chunk of one row into registers, sums the
// exponentials and finds the chunk's N largest logits; the CTA of a request
// that finishes last joins the chunks' sums to lse_k and takes the N best of the
// K * chunks * N that are left.
//
// N largest without a sort: the N-th largest of the maxima of 64 groups of a
// chunk is at most the N-th largest value of the chunk, and few values reach it.
// Those are collected and ranked by counting, on keys that no two values share
// (value, then place), so the order does not depend on timing.  Within a row
// logits are compared as they are; scores of different rows are compared in 64
// bits.
#include "ft_kv.cuh"
#include "../../include/ft_gen.h"

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <new>

struct ft_beam {
    int V, dtype, R_max, N_max;
    int device, num_sms;
    cudaStream_t stream;
    void* arena;
    unsigned* err;
    unsigned* arrived;     // [R_max] CTAs of a request that have finished; 0 at rest
    struct BeamSum* sums;  // [lists]
    uint64_t* keys;        // [lists][N_max]
    long long lists;       // chunks of all rows
};

// Sum over a chunk: l * e^m.
struct BeamSum {
    double m;
    float l;
    int pad;
};

namespace {

constexpr int CT = 256;     // threads of a CTA
constexpr int GROUPS = 64;  // quads of lanes
constexpr int CAP = 1024;   // candidates that are ranked at once
constexpr int MAX_N = 64, MAX_K = 64;
constexpr float LOG2E = 1.44269504088896340736f;  // rounded to fp32; used in both directions, so its error cancels

struct SelParams {
    const void* logits;
    long long ld;
    const float* scores;
    const int* rows;
    const int* done;
    float* out_scores;
    int *out_parents, *out_tokens, *out_done;
    int V, K, N, C, eos;
    BeamSum* sums;
    uint64_t* keys;
    unsigned* arrived;
    unsigned* err;
};

// Order of floats as unsigned integers, and back.
__device__ __forceinline__ uint32_t ord(float f) {
    const uint32_t u = __float_as_uint(f);
    return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unord(uint32_t o) {
    return __uint_as_float(o ^ (o >> 31 ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Values of a 16-byte vector.
template <int TYPE>
__device__ __forceinline__ void unpack(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (TYPE == FT_T_F32) {
            f[i] = __uint_as_float(w[i]);
        } else if (TYPE == FT_T_BF16) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        }
    }
}

// The vector of values i..i+VEC-1 of a row of V, of which some are outside it: those are -inf.
template <int TYPE>
__device__ uint4 load_edge(const void* row, long long i, int V) {
    constexpr int VEC = TYPE == FT_T_F32 ? 4 : 8;
    uint4 v;
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
    if (TYPE == FT_T_F32) {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            w[j] = i + j >= 0 && i + j < V ? static_cast<const uint32_t*>(row)[i + j] : 0xff800000u;
    } else {
        const uint32_t none = TYPE == FT_T_BF16 ? 0xff80u : 0xfc00u;
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
            const uint32_t a = i + j >= 0 && i + j < V ? static_cast<const uint16_t*>(row)[i + j] : none;
            const uint32_t b = i + j + 1 >= 0 && i + j + 1 < V ? static_cast<const uint16_t*>(row)[i + j + 1] : none;
            w[j / 2] = a | b << 16;
        }
    }
    return v;
}

struct ScanSmem {
    float group[GROUPS];
    double wm[CT / 32];
    float wl[CT / 32];
    float bar;
    int n;
    uint64_t list[CAP];
};
struct JoinSmem {
    // score = base + (x - top) with lse = top + log l, base = s - log l, so that logits of any size keep their
    // differences; of an ended beam s and 0; base -inf: no candidates
    double base[MAX_K], top[MAX_K];
    bool ended[MAX_K];
    float group[GROUPS];
    float bar;
    int n;
    double score[CAP];
    uint64_t at[CAP];    // beam << 32 | token
};

// The N-th largest of the groups' maxima (N <= GROUPS), by counting; call by whole warps 0 and 1.
__device__ __forceinline__ void nth_of_groups(const float* group, int N, float* bar) {
    const int g = threadIdx.x;
    const float mine = group[g];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < GROUPS; ++j) {
        const float o = group[j];
        rank += o > mine || (o == mine && j < g);
    }
    if (rank == N - 1) *bar = mine;
}

// The chunk's sum and its N largest values to the workspace.
template <int TYPE, int NJ>
__device__ void scan_chunk(const SelParams& p, const void* row, int chunk, long long list, ScanSmem& s) {
    constexpr int VEC = TYPE == FT_T_F32 ? 4 : 8, SIZE = TYPE == FT_T_F32 ? 4 : 2;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    // vectors are aligned in memory: the first of a row may start before it
    const int shift = (int)((uintptr_t)row % 16) / SIZE;
    const long long i0 = (long long)chunk * (CT * VEC * NJ) + threadIdx.x * VEC - shift;
    uint4 v[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const long long i = i0 + (long long)j * (CT * VEC);
        if (i >= 0 && i + VEC <= p.V) v[j] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + i * SIZE));
        else v[j] = load_edge<TYPE>(row, i, p.V);
    }
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        float f[VEC];
        unpack<TYPE>(v[j], f);
#pragma unroll
        for (int k = 0; k < VEC; ++k) m = fmaxf(m, f[k]);
    }
    float g = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 2));
    if ((lane & 3) == 0) s.group[threadIdx.x >> 2] = g;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
    if (threadIdx.x == 0) s.n = 0;
    // Sum of exponentials on the warp's reference: 2^(x log2(e) - c) with c a whole number near the largest exponent, so
    // that each exponent is rounded once.  The reference in x is c / log2(e) with the same constant.  Values whose
    // exponents an fp32 cannot hold to a fraction are taken by differences from the largest.
    double ref = 0.;
    float l = 0.f;
    if (fabsf(g) <= 1048576.f || g == -INFINITY) {
        const float c = g == -INFINITY ? 0.f : rintf(g * LOG2E);
        float l1 = 0.f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            float f[VEC];
            unpack<TYPE>(v[j], f);
#pragma unroll
            for (int k = 0; k < VEC; k += 2) {
                l += ex2(fmaf(f[k], LOG2E, -c));
                l1 += ex2(fmaf(f[k + 1], LOG2E, -c));
            }
        }
        l += l1;
        ref = (double)c / (double)LOG2E;
    } else {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            float f[VEC];
            unpack<TYPE>(v[j], f);
#pragma unroll
            for (int k = 0; k < VEC; ++k) l += ex2((f[k] - g) * LOG2E);  // (+inf gives a NaN)
        }
        ref = g;
    }
    l = ft::warp_sum(l);
    if (lane == 0) {
        s.wm[wid] = ref;
        s.wl[wid] = l;
    }
    __syncthreads();
    if (wid < GROUPS / 32) nth_of_groups(s.group, p.N, &s.bar);
    if (wid == 7) {
        double r = s.wm[lane & 7];
        const float lw = s.wl[lane & 7];
        // a warp without a value has its reference at 0 and must not set the others'
        double top = lw == 0.f ? -INFINITY : r;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
        float t = lw == 0.f ? 0.f : lw * expf((float)(r - top));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        if (lane == 0) p.sums[list] = BeamSum{top, t, 0};
    }
    __syncthreads();
    const float bar = s.bar;
    auto key = [&](float f, long long i) { return (uint64_t)ord(f) << 32 | (uint32_t)(0xffffffffu - (uint32_t)i); };
    if (m >= bar && m > -INFINITY) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            float f[VEC];
            unpack<TYPE>(v[j], f);
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                if (f[k] >= bar && f[k] > -INFINITY) {
                    const int at = atomicAdd(&s.n, 1);
                    if (at < CAP) s.list[at] = key(f[k], i0 + (long long)j * (CT * VEC) + k);
                }
        }
    }
    __syncthreads();
    int n = s.n;
    if (n > CAP) {
        // Many equal values.  Keys are all different, so some bar between the lowest of these and the largest lets
        // N to CAP of them pass: halve the range until one does.
        uint64_t lo = (uint64_t)max(ord(bar), ord(-INFINITY) + 1) << 32, hi = ~0ull;
        for (int it = 0; it < 64; ++it) {
            const uint64_t mid = lo + (hi - lo) / 2;
            int mine = 0;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                float f[VEC];
                unpack<TYPE>(v[j], f);
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    mine += f[k] > -INFINITY && key(f[k], i0 + (long long)j * (CT * VEC) + k) >= mid;
            }
            __syncthreads();
            if (threadIdx.x == 0) s.n = 0;
            __syncthreads();
            if (mine) atomicAdd(&s.n, mine);
            __syncthreads();
            n = s.n;
            if (n > CAP) lo = mid;
            else if (n < p.N) hi = mid;
            else { lo = mid; break; }
        }
        __syncthreads();
        if (threadIdx.x == 0) s.n = 0;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            float f[VEC];
            unpack<TYPE>(v[j], f);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const uint64_t q = key(f[k], i0 + (long long)j * (CT * VEC) + k);
                if (f[k] > -INFINITY && q >= lo) {
                    const int at = atomicAdd(&s.n, 1);
                    if (at < CAP) s.list[at] = q;
                }
            }
        }
        __syncthreads();
        n = min(s.n, CAP);
    }
    uint64_t* out = p.keys + list * p.N;
    for (int i = threadIdx.x; i < n; i += CT) {
        const uint64_t mine = s.list[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += s.list[j] > mine;
        if (rank < p.N) out[rank] = mine;
    }
    for (int i = n + threadIdx.x; i < p.N; i += CT) out[i] = 0;
}

// (score, beam, token) a before b.
__device__ __forceinline__ bool before(double sa, uint64_t a, double sb, uint64_t b) {
    return sa > sb || (sa == sb && a < b);
}

// The N best of what the chunks of request b left.
__device__ void join_request(const SelParams& p, int b, JoinSmem& s) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int per = p.C * p.N, E = p.K * per;
    for (int k = wid; k < p.K; k += CT / 32) {
        const int row = b * p.K + k;
        const float sc = p.scores[row];
        const bool live = sc > -INFINITY && sc < INFINITY;
        const bool ended = p.done && p.done[row];
        double base = sc, top = 0.;
        if (!live) {
            base = -INFINITY;
            if (lane == 0 && !(sc == -INFINITY)) atomicOr(p.err, FT_DEVERR_ARG);
        } else if (!ended) {
            top = -INFINITY;
            for (int c = lane; c < p.C; c += 32) {
                const BeamSum* q = p.sums + (long long)row * p.C + c;
                if (__ldcg(&q->l) != 0.f) top = fmax(top, __ldcg(&q->m));
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
            float l = 0.f;
            for (int c = lane; c < p.C; c += 32) {
                const BeamSum* q = p.sums + (long long)row * p.C + c;
                const float lc = __ldcg(&q->l);
                if (lc != 0.f) l += lc * expf((float)(__ldcg(&q->m) - top));
            }
            l = ft::warp_sum(l);
            if (!(l > 0.f && l < INFINITY)) {
                base = -INFINITY;
                if (lane == 0 && l != 0.f) atomicOr(p.err, FT_DEVERR_ARG);  // a NaN or an infinity in the row
            } else {
                // log l = e log 2 + log f with f in [1/sqrt 2, sqrt 2), so that the fp32 logarithm is of a small number
                int e;
                float f = frexpf(l, &e);
                if (f < 0.70710678f) {
                    f *= 2.f;
                    --e;
                }
                base -= e * 0.693147180559945309 + (double)logf(f);
            }
        }
        if (lane == 0) {
            s.base[k] = base;
            s.top[k] = top;
            s.ended[k] = ended;
        }
    }
    if (threadIdx.x == 0) s.n = 0;
    __syncthreads();
    // entry e of the beams' lists, then one entry for each beam that has ended
    auto entry = [&](int e, double& sc, uint64_t& at) {
        int k;
        if (e < E) {
            k = e / per;
            const double base = s.base[k];
            if (base == -INFINITY || s.ended[k]) return false;
            const long long row = (long long)b * p.K + k;
            const uint64_t q = __ldcg(reinterpret_cast<const unsigned long long*>(p.keys) + row * per + (e - k * per));
            if (q == 0) return false;
            sc = base + ((double)unord((uint32_t)(q >> 32)) - s.top[k]);
            at = (uint64_t)k << 32 | (0xffffffffu - (uint32_t)q);
            return true;
        }
        k = e - E;
        if (k >= p.K || !s.ended[k] || s.base[k] == -INFINITY) return false;
        sc = s.base[k];
        at = (uint64_t)k << 32 | (uint32_t)p.eos;
        return true;
    };
    const int all = E + (p.done ? p.K : 0);
    float m = -INFINITY;
    for (int e = threadIdx.x; e < all; e += CT) {
        double sc;
        uint64_t at;
        if (entry(e, sc, at)) m = fmaxf(m, (float)sc);
    }
    float g = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 2));
    if ((lane & 3) == 0) s.group[threadIdx.x >> 2] = g;
    __syncthreads();
    if (wid < GROUPS / 32) nth_of_groups(s.group, p.N, &s.bar);
    __syncthreads();
    const float bar = s.bar;
    // Ranks of the list's entries; those below N move to the front (keep) or are the result.
    auto rank_list = [&](bool keep) {
        const int n = s.n;
        double sc[CAP / CT];
        uint64_t at[CAP / CT];
        int rank[CAP / CT];
#pragma unroll
        for (int u = 0; u < CAP / CT; ++u) {
            const int i = u * CT + threadIdx.x;
            rank[u] = MAX_N;
            if (i >= n) continue;
            sc[u] = s.score[i];
            at[u] = s.at[i];
            rank[u] = 0;
            for (int j = 0; j < n; ++j) rank[u] += before(s.score[j], s.at[j], sc[u], at[u]);
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < CAP / CT; ++u) {
            if (rank[u] >= p.N) continue;
            if (keep) {
                s.score[rank[u]] = sc[u];
                s.at[rank[u]] = at[u];
                continue;
            }
            const int k = (int)(at[u] >> 32), v = (int)(uint32_t)at[u], row = b * p.K + k;
            const long long o = (long long)b * p.N + rank[u];
            p.out_scores[o] = (float)sc[u];
            p.out_parents[o] = p.rows ? p.rows[row] : row;
            p.out_tokens[o] = v;
            if (p.out_done) p.out_done[o] = v == p.eos;  // (an ended beam's only candidate)
        }
        if (!keep)
            for (int i = n + threadIdx.x; i < p.N; i += CT) {
                const long long o = (long long)b * p.N + i;
                p.out_scores[o] = -INFINITY;
                p.out_parents[o] = p.out_tokens[o] = -1;
                if (p.out_done) p.out_done[o] = 0;
            }
        if (keep) {
            if (threadIdx.x == 0) s.n = min(n, p.N);
            __syncthreads();
        }
    };
    for (int e0 = 0; e0 < all; e0 += CT) {
        double sc;
        uint64_t at;
        if (e0 + (int)threadIdx.x < all && entry(e0 + threadIdx.x, sc, at) && (float)sc >= bar) {
            const int i = atomicAdd(&s.n, 1);
            s.score[i] = sc;
            s.at[i] = at;
        }
        if (all > CAP) {  // the list may fill up
            __syncthreads();
            if (s.n > CAP - CT) rank_list(true);
            else __syncthreads();
        }
    }
    __syncthreads();
    rank_list(false);
}

template <int TYPE, int NJ>
__global__ void __launch_bounds__(CT) beam_select_kernel(const SelParams p) {
    __shared__ union {
        ScanSmem scan;
        JoinSmem join;
    } s;
    __shared__ bool last;
    ft::grid_dep_launch();
    ft::grid_dep_wait();
    const long long list = blockIdx.x;
    const int row = (int)(list / p.C), chunk = (int)(list % p.C), b = row / p.K;
    const float sc = p.scores[row];
    if (sc > -INFINITY && !(p.done && p.done[row])) {
        constexpr int SIZE = TYPE == FT_T_F32 ? 4 : 2;
        scan_chunk<TYPE, NJ>(p, static_cast<const uint8_t*>(p.logits) + row * p.ld * SIZE, chunk, list, s.scan);
    }
    // every thread's stores, then the count: the last CTA of the request sees them all
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        unsigned c;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(c) : "l"(p.arrived + b) : "memory");
        last = c == (unsigned)(p.K * p.C - 1);
        if (last) p.arrived[b] = 0;
        __threadfence();
    }
    __syncthreads();
    if (last) join_request(p, b, s.join);
}

constexpr int NJ_OF(int type, bool wide) { return wide ? (type == FT_T_F32 ? 8 : 4) : (type == FT_T_F32 ? 2 : 1); }
constexpr int WIDE = 8192, NARROW = 2048;  // values of a chunk

template <int TYPE>
const void* kernel_of(bool wide) {
    return wide ? (const void*)beam_select_kernel<TYPE, NJ_OF(TYPE, true)> : (const void*)beam_select_kernel<TYPE, NJ_OF(TYPE, false)>;
}

int chunks_of(int V, int dtype, int size) {
    const int vec = dtype == FT_T_F32 ? 4 : 8;
    return (V + vec - 1 + size - 1) / size;  // a row may start vec-1 values into its first vector
}

bool sizes_ok(int V, int dtype, int R_max, int N_max) {
    return V >= 1 && V <= 1 << 24 && dtype >= FT_T_BF16 && dtype <= FT_T_F32 && R_max >= 1 && R_max <= 65536 && N_max >= 1 &&
           N_max <= MAX_N && (long long)R_max * chunks_of(V, dtype, WIDE) * N_max < (1ll << 31);
}

struct Layout {
    long long lists;
    size_t err, arrived, sums, keys, total;
};
Layout layout(int V, int dtype, int R_max, int N_max, int sms) {
    Layout l;
    l.lists = (long long)R_max * chunks_of(V, dtype, WIDE);
    if (l.lists < 4ll * sms) l.lists = 4ll * sms;
    size_t off = 0;
    auto carve = [&](size_t bytes) {
        const size_t o = off;
        off = (off + bytes + 255) / 256 * 256;
        return o;
    };
    l.err = carve(4);
    l.arrived = carve((size_t)R_max * 4);
    l.sums = carve((size_t)l.lists * sizeof(BeamSum));
    l.keys = carve((size_t)l.lists * N_max * 8);
    l.total = off;
    return l;
}

// [p, p + n) of bytes.
struct Bytes {
    uintptr_t p;
    size_t n;
};
bool overlap(const Bytes& a, const Bytes& b) { return a.p && b.p && a.p < b.p + b.n && b.p < a.p + a.n; }

}  // namespace

extern "C" {

size_t ft_beam_scratch_bytes(int32_t V, int32_t dtype, int32_t R_max, int32_t N_max) {
    if (!sizes_ok(V, dtype, R_max, N_max)) return 0;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return layout(V, dtype, R_max, N_max, sms).total;
}

ft_status ft_beam_init(ft_beam** out, int32_t V, int32_t dtype, int32_t R_max, int32_t N_max, void* stream) {
    if (!out) return FT_ERR_ARG;
    *out = nullptr;
    if (!sizes_ok(V, dtype, R_max, N_max)) return FT_ERR_ARG;
    ft_beam* bm = new (std::nothrow) ft_beam();
    if (!bm) return FT_ERR_OOM;
    bm->V = V; bm->dtype = dtype; bm->R_max = R_max; bm->N_max = N_max;
    bm->stream = (cudaStream_t)stream;
    auto fail = [&](ft_status s) {
        cudaGetLastError();
        cudaFree(bm->arena);
        delete bm;
        return s;
    };
    if (cudaGetDevice(&bm->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&bm->num_sms, cudaDevAttrMultiProcessorCount, bm->device) != cudaSuccess)
        return fail(FT_ERR_CUDA);
    const Layout l = layout(V, dtype, R_max, N_max, bm->num_sms);
    const cudaError_t e = cudaMalloc(&bm->arena, l.total);
    if (e != cudaSuccess) return fail(e == cudaErrorMemoryAllocation ? FT_ERR_OOM : FT_ERR_CUDA);
    // lists are written before they are read; the rest starts at 0
    if (cudaMemset(bm->arena, 0, l.sums) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) return fail(FT_ERR_CUDA);
    uint8_t* a = (uint8_t*)bm->arena;
    bm->err = (unsigned*)(a + l.err);
    bm->arrived = (unsigned*)(a + l.arrived);
    bm->sums = (BeamSum*)(a + l.sums);
    bm->keys = (uint64_t*)(a + l.keys);
    bm->lists = l.lists;
    *out = bm;
    return FT_OK;
}

ft_status ft_beam_select(ft_beam* bm, int32_t B, int32_t K, int32_t N, const void* logits, int64_t ld,
                         const float* scores, const int32_t* rows, const int32_t* done, int32_t eos, float* out_scores,
                         int32_t* out_parents, int32_t* out_tokens, int32_t* out_done) {
    if (!bm || B < 0 || K < 1 || K > MAX_K || N < 1 || N > bm->N_max || (long long)B * K > bm->R_max || eos < -1 || eos >= bm->V ||
        (done && eos < 0))
        return FT_ERR_ARG;
    if (B == 0) return FT_OK;
    const int size = bm->dtype == FT_T_F32 ? 4 : 2;
    if (!logits || !scores || !out_scores || !out_parents || !out_tokens || ld < bm->V || ld > (1ll << 40) || (uintptr_t)logits % size)
        return FT_ERR_ARG;
    for (const void* q : {(const void*)scores, (const void*)rows, (const void*)done, (const void*)out_scores,
                          (const void*)out_parents, (const void*)out_tokens, (const void*)out_done})
        if ((uintptr_t)q % 4) return FT_ERR_ARG;
    const size_t R = (size_t)B * K, M = (size_t)B * N;
    const Bytes in[] = {{(uintptr_t)logits, (size_t)((R - 1) * ld + bm->V) * size}, {(uintptr_t)scores, R * 4},
                        {(uintptr_t)rows, R * 4}, {(uintptr_t)done, R * 4}};
    const Bytes outs[] = {{(uintptr_t)out_scores, M * 4}, {(uintptr_t)out_parents, M * 4}, {(uintptr_t)out_tokens, M * 4},
                          {(uintptr_t)out_done, M * 4}};
    for (int o = 0; o < 4; ++o) {
        for (int i = 0; i < 4; ++i) {
            const bool in_place = N == K && outs[o].p == in[i].p && ((o == 0 && i == 1) || (o == 3 && i == 3));
            if (overlap(outs[o], in[i]) && !in_place) return FT_ERR_ARG;
        }
        for (int q = o + 1; q < 4; ++q)
            if (overlap(outs[o], outs[q])) return FT_ERR_ARG;
    }
    SelParams p{};
    p.logits = logits; p.ld = ld; p.scores = scores; p.rows = rows; p.done = done; p.eos = eos;
    p.out_scores = out_scores; p.out_parents = out_parents; p.out_tokens = out_tokens; p.out_done = out_done;
    p.V = bm->V; p.K = K; p.N = N;
    p.sums = bm->sums; p.keys = bm->keys; p.arrived = bm->arrived; p.err = bm->err;
    // narrow chunks while all of them run at once
    const long long narrow = (long long)R * chunks_of(bm->V, bm->dtype, NARROW);
    const bool wide = narrow > 4ll * bm->num_sms;
    p.C = chunks_of(bm->V, bm->dtype, wide ? WIDE : NARROW);
    const void* k = bm->dtype == FT_T_BF16 ? kernel_of<FT_T_BF16>(wide) : bm->dtype == FT_T_F16 ? kernel_of<FT_T_F16>(wide)
                                                                                                : kernel_of<FT_T_F32>(wide);
    void* args[] = {&p};
    const cudaError_t e = launch_dependent(k, (int)(R * p.C), CT, 0, bm->stream, args);
    if (e == cudaSuccess) return FT_OK;
    if (getenv("FT_DEBUG")) fprintf(stderr, "libft: launch -> %s\n", cudaGetErrorString(e));
    return FT_ERR_CUDA;
}

ft_status ft_beam_status(ft_beam* bm) {
    if (!bm) return FT_ERR_ARG;
    if (cudaStreamSynchronize(bm->stream) != cudaSuccess) return FT_ERR_CUDA;
    unsigned e = 0;
    if (cudaMemcpy(&e, bm->err, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return FT_ERR_CUDA;
    if (e && cudaMemset(bm->err, 0, 4) != cudaSuccess) return FT_ERR_CUDA;
    if (e && cudaDeviceSynchronize() != cudaSuccess) return FT_ERR_CUDA;
    return e ? FT_ERR_DEVICE : FT_OK;
}

void ft_beam_destroy(ft_beam* bm) {
    if (!bm) return;
    cudaStreamSynchronize(bm->stream);
    cudaFree(bm->arena);
    delete bm;
}

}  // extern "C"

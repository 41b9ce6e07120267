// Page operations of the key/value cache: one control kernel per call (one
// CTA: it validates the whole list before it changes anything) and, where
// pages move, a copy kernel over all layers.
//
// The control kernels are bound by the latency of dependent reads (lists,
// lengths, table entries), about 0.7 us each: what does not depend on the list
// (the first 4096 reference counts) is read beside it, rows are marked in
// shared memory, and a table entry that was checked is read again from L1.
// Measured: a fork of one row of 1000 tokens into three with its copy 8.5 us; a
// step of beam search over 64 rows of up to 2000 tokens (free 32, fork 32,
// extend 64, 23 MB copied) 20.7 us for its four kernels.  The layout of a step of
// 64 requests 4.6 us, of 1024 requests' drafts 12.1; a reordering of 4 rows of
// 1000 tokens with its copy 7.3, of 256 rows 14.7.
#include "ft_kv.cuh"

namespace {

constexpr int CT = 1024;  // threads of the control kernels

struct KvCtl {
    int *table, *lens, *refs;
    int n_pages, n_rows, row_pages, page, page_log;
    int *info, *n_copy, *free_list, *remap, *rank;
    KvCopy* copies;
    unsigned* err;
};

KvCtl ctl_of(const ft_kv* kv) {
    return KvCtl{kv->table, kv->lens, kv->refs, kv->n_pages, kv->n_rows, kv->row_pages, kv->page, __builtin_ctz(kv->page),
                 kv->info, kv->n_copy, kv->free_list, kv->remap, kv->rank, kv->copies, kv->err};
}

// The scans for free pages look at 4 pages a thread first (which are read ahead), then at 16.  A warp's pages are PER * 32
// in a row, 32 at a time.
constexpr int FREE_FIRST = 4, FREE_MORE = 16;
template <int PER>
__device__ __forceinline__ int scan_page(int base, int j) {
    return base + ((threadIdx.x >> 5) * PER + j) * 32 + (threadIdx.x & 31);
}

// Which of this thread's pages of the step at `base` are free, one bit each.  CG: past L1, for counts that other CTAs
// changed in this kernel.
template <int PER, bool CG>
__device__ __forceinline__ unsigned free_bits(const KvCtl& c, int base) {
    int v[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int p = scan_page<PER>(base, j);
        v[j] = p >= c.n_pages ? 1 : CG ? __ldcg(c.refs + p) : c.refs[p];
    }
    unsigned f = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) f |= v[j] == 0 ? 1u << j : 0;
    return f;
}

// A step of the scan: its free pages go to list from place `have` on, as far as `want`; returns how many it has.
template <int PER>
__device__ __forceinline__ int list_free(int base, unsigned f, int have, int want, int (&ws)[32], int* list) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    unsigned m[PER];
    int cnt = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        m[j] = __ballot_sync(0xffffffffu, f >> j & 1u);
        cnt += __popc(m[j]);
    }
    __syncthreads();  // the reads of ws before this are over
    if (lane == 0) ws[wid] = cnt;
    __syncthreads();
    int total = ws[lane], at = lane < wid ? total : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        at += __shfl_xor_sync(0xffffffffu, at, o);
        total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    at += have;
    if (cnt && at < want) {  // (the same in all lanes)
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int mine = at + __popc(m[j] & ((1u << lane) - 1));
            if ((f >> j & 1u) && mine < want) list[mine] = scan_page<PER>(base, j);
            at += __popc(m[j]);
        }
    }
    return total;
}

// The lowest `want` free pages, ascending, to list; returns how many there are
// (at most a few more than `want` are counted).  first: free_bits<FREE_FIRST>(c, 0).
template <bool CG>
__device__ int take_free(const KvCtl& c, int want, int (&ws)[32], unsigned first, int* list) {
    int have = 0;
    if (want > 0) have = list_free<FREE_FIRST>(0, first, 0, want, ws, list);
    for (int base = FREE_FIRST * CT; base < c.n_pages && have < want; base += FREE_MORE * CT)
        have += list_free<FREE_MORE>(base, free_bits<FREE_MORE, CG>(c, base), have, want, ws, list);
    __syncthreads();
    return have;
}

// Bits of the rows that a list names.
struct RowMarks {
    unsigned w[KV_MAX_ROWS / 32];
};
__device__ __forceinline__ void clear(RowMarks& m, int n_rows) {
    for (int i = threadIdx.x; i < (n_rows + 31) / 32; i += CT) m.w[i] = 0;
    __syncthreads();
}
// Marks row r; false if it is out of range or marked already.
__device__ __forceinline__ bool mark(RowMarks& m, int r, int n_rows) {
    if (r < 0 || r >= n_rows) return false;
    return !(atomicOr(&m.w[r >> 5], 1u << (r & 31)) >> (r & 31) & 1u);
}

__device__ void set_info(const KvCtl& c, int allocated, int copied, int live) {
    if (threadIdx.x == 0) {
        c.info[KV_ALLOCATED] = allocated;
        c.info[KV_COPIED] = copied;
        c.info[KV_LIVE] = live;
        *c.n_copy = copied;
    }
}

__device__ void refuse(const KvCtl& c, unsigned bit) {
    if (threadIdx.x == 0) atomicOr(c.err, bit);
    set_info(c, 0, 0, -1);
}

__global__ void __launch_bounds__(CT) kv_extend_kernel(KvCtl c, int n, const int* __restrict__ rows,
                                                       const int* __restrict__ add) {
    __shared__ int ws[32];
    __shared__ RowMarks marks;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    clear(marks, c.n_rows);
    ft::grid_dep_launch();
    ft::grid_dep_wait();
    const unsigned first = free_bits<FREE_FIRST, false>(c, 0);
    int want = 0;
    bool ok = true;
    for (int base = 0; base < n; base += CT) {
        const int i = base + threadIdx.x;
        int need = 0;
        if (i < n) {
            const int r = rows[i], a = add[i];
            if (mark(marks, r, c.n_rows)) {
                const long long len = c.lens[r], to = len + a;
                if (len < 0 || a < 0 || to > (long long)c.row_pages * c.page)
                    ok = false;
                else
                    need = (int)((to + c.page - 1) / c.page - (len + c.page - 1) / c.page);
            } else {
                ok = false;
            }
        }
        int total;
        const int at = want + ft::block_scan(need, ws, total);
        if (i < n) c.rank[i] = at;
        want += total;
    }
    if (!__syncthreads_and(ok)) return refuse(c, FT_DEVERR_ARG);
    if (take_free<false>(c, want, ws, first, c.free_list) < want) return refuse(c, FT_DEVERR_CAPACITY);
    for (int i = wid; i < n; i += CT / 32) {
        const int r = rows[i], len = c.lens[r], to = len + add[i], at = c.rank[i];
        const int have = (len + c.page - 1) / c.page, end = (to + c.page - 1) / c.page;
        for (int j = have + lane; j < end; j += 32) {
            const int p = c.free_list[at + j - have];
            c.table[(size_t)r * c.row_pages + j] = p;
            c.refs[p] = 1;
        }
        __syncwarp();
        if (lane == 0) c.lens[r] = to;
    }
    set_info(c, want, 0, -1);
}

__global__ void __launch_bounds__(CT) kv_fork_kernel(KvCtl c, int n, const int* __restrict__ parents,
                                                     const int* __restrict__ children) {
    __shared__ int ws[32];
    __shared__ RowMarks marks;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    clear(marks, c.n_rows);
    ft::grid_dep_launch();
    ft::grid_dep_wait();
    const unsigned first = free_bits<FREE_FIRST, false>(c, 0);
    int want = 0;
    bool ok = true;
    for (int base = 0; base < n; base += CT) {
        const int i = base + threadIdx.x;
        int need = 0;
        if (i < n) {
            const int p = parents[i], ch = children[i];
            if (mark(marks, ch, c.n_rows) && p >= 0 && p < c.n_rows) {
                const int len = c.lens[p];
                if (c.lens[ch] != 0 || len < 0 || len > (long long)c.row_pages * c.page) ok = false;
                need = ok && len % c.page ? 1 : 0;
            } else {
                ok = false;
            }
        }
        int total;
        const int at = want + ft::block_scan(need, ws, total);
        if (i < n) c.rank[i] = at;
        want += total;
    }
    if (!__syncthreads_and(ok)) return refuse(c, FT_DEVERR_ARG);
    // no parent is a child; their pages are in range
    for (int i = wid; i < n; i += CT / 32) {
        const int p = parents[i];
        if (marks.w[p >> 5] >> (p & 31) & 1u) ok = false;
        const int* row = c.table + (size_t)p * c.row_pages;
        const int np = (c.lens[p] + c.page - 1) / c.page;
        for (int j = lane; j < np; j += 32)
            if (row[j] < 0 || row[j] >= c.n_pages) ok = false;
    }
    if (!__syncthreads_and(ok)) return refuse(c, FT_DEVERR_ARG);
    if (take_free<false>(c, want, ws, first, c.free_list) < want) return refuse(c, FT_DEVERR_CAPACITY);
    for (int i = wid; i < n; i += CT / 32) {
        const int p = parents[i], len = c.lens[p], full = len / c.page, tok = len % c.page;
        const int* src = c.table + (size_t)p * c.row_pages;
        int* dst = c.table + (size_t)children[i] * c.row_pages;
        for (int j = lane; j < c.row_pages; j += 32) {
            int v = -1;
            if (j < full) {
                v = src[j];
                atomicAdd(&c.refs[v], 1);
            } else if (j == full && tok) {
                v = c.free_list[c.rank[i]];
                c.refs[v] = 1;
                c.copies[c.rank[i]] = KvCopy{src[j], v, tok};
            }
            dst[j] = v;
        }
        if (lane == 0) c.lens[children[i]] = len;
    }
    set_info(c, want, want, -1);
}

__global__ void __launch_bounds__(CT) kv_free_kernel(KvCtl c, int n, const int* __restrict__ rows) {
    __shared__ RowMarks marks;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    clear(marks, c.n_rows);
    ft::grid_dep_launch();
    ft::grid_dep_wait();
    bool ok = true;
    for (int i = wid; i < n; i += CT / 32) {
        const int r = rows[i];
        bool mine = true;
        if (lane == 0) mine = mark(marks, r, c.n_rows);
        if (!__all_sync(0xffffffffu, mine)) {
            ok = false;
            continue;
        }
        const long long len = c.lens[r];
        if (len < 0 || len > (long long)c.row_pages * c.page) {
            ok = false;
            continue;
        }
        const int np = (int)((len + c.page - 1) / c.page);
        for (int j = lane; j < np; j += 32) {
            const int p = c.table[(size_t)r * c.row_pages + j];
            if (p < 0 || p >= c.n_pages) ok = false;
        }
    }
    if (!__syncthreads_and(ok)) return refuse(c, FT_DEVERR_ARG);
    for (int i = wid; i < n; i += CT / 32) {
        const int r = rows[i];
        const int np = (c.lens[r] + c.page - 1) / c.page;
        for (int j = lane; j < np; j += 32) {
            int* e = c.table + (size_t)r * c.row_pages + j;
            const int p = *e;
            *e = -1;
            if (atomicSub(&c.refs[p], 1) <= 0) {
                atomicAdd(&c.refs[p], 1);
                ok = false;
            }
        }
        __syncwarp();
        if (lane == 0) c.lens[r] = 0;
    }
    if (!ok) atomicOr(c.err, FT_DEVERR_ARG);
    set_info(c, 0, 0, -1);
}

// ---- layout of a step

// Largest i in [0, n) with start[i] <= x (start ascending from 0, x >= 0).
__device__ __forceinline__ int owner_of(const int* start, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

struct BatchOut {
    int *cu_q, *row_of, *pos;
    long long* slots;
    int T;
};

// Lists the tokens t0, t0 + step, ... of the requests whose first tokens are start[0..B).  A request's length before the
// call is held[b], or where held is null that of its row, less add[b] where add is given.
__device__ __forceinline__ void list_tokens(const KvCtl& c, const BatchOut& o, int B, const int* rows, const int* held,
                                            const int* add, const int* start, int total, int t0, int step) {
    for (long long t = t0; t < o.T; t += step) {
        int r = -1, p = 0;
        long long slot = -1;
        if (t < total) {
            // (one token each: no search)
            const bool single = t < B && start[t] == t && (t + 1 < B ? start[t + 1] : total) == t + 1;
            const int b = single ? (int)t : owner_of(start, B, (int)t);
            r = rows ? rows[b] : b;
            p = (held ? held[b] : c.lens[r] - (add ? add[b] : 0)) + ((int)t - start[b]);
            if (o.slots) slot = (long long)c.table[(size_t)r * c.row_pages + (p >> c.page_log)] * c.page + (p & (c.page - 1));
        }
        o.row_of[t] = r;
        o.pos[t] = p;
        if (o.slots) o.slots[t] = slot;
    }
}

// Tokens that the first kernel lists itself: 2000 tokens of 500 requests 7.6 us with one kernel, 8.8 with two; 3300 of 1024
// requests 13.2 and 12.0.
constexpr int LIST_HERE = 2048;
constexpr int BATCH_SMEM = 2048;  // requests that are kept in shared memory

struct TokPage {
    long long tok;
    int page;
};
// Exclusive prefix sums of both over the CTA, in one pass; total gets the sums.
__device__ __forceinline__ TokPage block_scan2(TokPage v, TokPage (&ws)[32], TokPage& total) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    TokPage x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, x.tok, o);
        const int g = __shfl_up_sync(0xffffffffu, x.page, o);
        if (lane >= o) {
            x.tok += t;
            x.page += g;
        }
    }
    __syncthreads();  // the previous call's reads of ws are over
    if (lane == 31) ws[wid] = x;
    __syncthreads();
    // every warp joins the 32 sums for itself
    TokPage s = ws[lane];
    TokPage before{lane < wid ? s.tok : 0, lane < wid ? s.page : 0};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        before.tok += __shfl_xor_sync(0xffffffffu, before.tok, o);
        before.page += __shfl_xor_sync(0xffffffffu, before.page, o);
        s.tok += __shfl_xor_sync(0xffffffffu, s.tok, o);
        s.page += __shfl_xor_sync(0xffffffffu, s.page, o);
    }
    total = s;
    return TokPage{x.tok - v.tok + before.tok, x.page - v.page + before.page};
}

// Rows grow as in kv_extend_kernel; then, with list_here, one thread a token lists them.  Bound by dependent reads: list,
// length, counts of the pages, and what a token needs; rows, lengths and both prefix sums stay in shared memory.
__global__ void __launch_bounds__(CT) kv_batch_kernel(KvCtl c, int B, const int* __restrict__ rows,
                                                      const int* __restrict__ add, BatchOut o, int list_here) {
    __shared__ int ws[32];
    __shared__ TokPage wl[32];
    __shared__ RowMarks marks;
    __shared__ int s_tok[BATCH_SMEM], s_page[BATCH_SMEM], s_row[BATCH_SMEM], s_len[BATCH_SMEM];
    clear(marks, c.n_rows);
    ft::grid_dep_launch();
    ft::grid_dep_wait();
    const unsigned first = free_bits<FREE_FIRST, false>(c, 0);
    const bool small = B <= BATCH_SMEM;
    int* tok = small ? s_tok : o.cu_q;
    int* pg = small ? s_page : c.rank;
    TokPage sum{0, 0};
    bool ok = true;
    for (int base = 0; base < B; base += CT) {
        const int i = base + threadIdx.x;
        TokPage need{0, 0};
        if (i < B) {
            const int r = rows ? rows[i] : i, a = add[i];
            int len = 0;
            if (mark(marks, r, c.n_rows)) {
                len = c.lens[r];
                const long long to = (long long)len + a;
                if (len < 0 || a < 0 || to > (long long)c.row_pages * c.page)
                    ok = false;
                else
                    need = TokPage{a, (int)(((to + c.page - 1) >> c.page_log) - (((long long)len + c.page - 1) >> c.page_log))};
            } else {
                ok = false;
            }
            if (small) {
                s_row[i] = r;
                s_len[i] = len;
            }
        }
        TokPage total;
        const TokPage at = block_scan2(need, wl, total);
        if (i < B) {
            tok[i] = (int)min(sum.tok + at.tok, (long long)o.T);
            pg[i] = sum.page + at.page;
        }
        sum.tok += total.tok;
        sum.page += total.page;
        if (sum.tok > o.T) {  // (the same in all threads; the sum of pages stays in its range)
            ok = false;
            break;
        }
    }
    int tokens = (int)min(sum.tok, (long long)o.T);
    const int want = sum.page;
    unsigned bad = 0;
    if (!__syncthreads_and(ok)) bad = FT_DEVERR_ARG;
    else if (take_free<false>(c, want, ws, first, c.free_list) < want) bad = FT_DEVERR_CAPACITY;
    if (bad) {
        refuse(c, bad);
        tokens = 0;
        for (int i = threadIdx.x; i <= B; i += CT) o.cu_q[i] = 0;
    } else {
        for (int w = threadIdx.x; w < want; w += CT) {
            const int i = owner_of(pg, B, w);
            const int r = small ? s_row[i] : rows ? rows[i] : i, len = small ? s_len[i] : c.lens[r], p = c.free_list[w];
            c.table[(size_t)r * c.row_pages + ((len + c.page - 1) >> c.page_log) + (w - pg[i])] = p;
            c.refs[p] = 1;
        }
        if (small)
            for (int i = threadIdx.x; i < B; i += CT) o.cu_q[i] = tok[i];
        if (threadIdx.x == 0) o.cu_q[B] = tokens;
        set_info(c, want, 0, -1);
        if (list_here) __syncthreads();
    }
    if (list_here) {
        if (small) list_tokens(c, o, B, s_row, s_len, nullptr, tok, tokens, threadIdx.x, CT);
        else list_tokens(c, o, B, rows, nullptr, nullptr, tok, tokens, threadIdx.x, CT);
    }
    if (bad) return;
    __syncthreads();
    for (int i = threadIdx.x; i < B; i += CT) {
        const int r = small ? s_row[i] : rows ? rows[i] : i;
        c.lens[r] = (small ? s_len[i] : c.lens[r]) + add[i];
    }
}

// The lists of a long step, a thread a token; the requests' first tokens are searched in shared memory where they fit.
__global__ void __launch_bounds__(256) kv_list_kernel(KvCtl c, int B, const int* __restrict__ rows,
                                                      const int* __restrict__ add, BatchOut o) {
    __shared__ int s_tok[BATCH_SMEM];
    ft::grid_dep_launch();
    ft::grid_dep_wait();
    const bool small = B <= BATCH_SMEM;
    const int total = o.cu_q[B];
    if (small) {
        for (int i = threadIdx.x; i < B; i += 256) s_tok[i] = o.cu_q[i];
        __syncthreads();
    }
    list_tokens(c, o, B, rows, nullptr, add, small ? s_tok : o.cu_q, total, blockIdx.x * blockDim.x + threadIdx.x,
                gridDim.x * blockDim.x);
}

// ---- reordering
//
// Table entries are the work: for each row that changes, the pages that it gets and those that it held are checked,
// counted and written.  Units of RO_COLS columns of one row are spread over the warps of a cluster of CTAs, which share the
// short control part (each does it for itself) and meet at cluster barriers: about 10 us for 256 rows of 63 pages, 44 in one
// CTA.

constexpr int RO_MAX = 1024;      // rows of a call, one thread each
constexpr int RO_COLS = 128;      // columns of a unit, four a lane
constexpr int RO_SLOTS = 320;     // units that a CTA stages at a time (160 KB)
constexpr int RO_CTAS = 8;        // CTAs of a cluster
// Rows and table entries up to which one CTA does it all: 64 rows of 17 pages 13.2 us, with their copy, and 14.0 by a
// cluster; 128 rows 15.5 and 12.1; 4 rows of 2000 pages 17.9 and 15.7.
constexpr int RO_ALONE = 64, RO_ALONE_ENTRIES = 4096;
// a column block of all rows is staged at once
static_assert(RO_SLOTS >= RO_ALONE && RO_SLOTS * RO_CTAS >= RO_MAX, "rows of a call");

struct ReorderSmem {
    union {
        int stage[RO_SLOTS][RO_COLS];
        uint16_t item_of[KV_MAX_ROWS];  // of a row in the list: its place there
    };
    RowMarks marks;
    int ws[32];
    // of each item: row, parent, tokens it gets, pages it held, complete pages it gets, its last page (0: none, 1: kept,
    // 2 + rank: new), who keeps its own row's last page
    int row[RO_MAX], par[RO_MAX], len[RO_MAX], old[RO_MAX], full[RO_MAX], last[RO_MAX], keep[RO_MAX];
    int free[RO_MAX];
    int cols;
    unsigned flag[2];
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// All threads of a cluster of `ctas` CTAs (one alone needs no more than its own barrier: 0.1 instead of 0.8 us).
__device__ __forceinline__ void cluster_sync(int ctas) {
    __syncthreads();
    if (ctas > 1) {
        cluster_arrive();
        cluster_wait();
    }
}
__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ unsigned cluster_size() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// Whether ok holds in all threads of the cluster; flag: a word of its own for each call.
__device__ __forceinline__ bool cluster_all(bool ok, unsigned* flag, int ctas) {
    const bool mine = __syncthreads_and(ok);
    if (ctas == 1) return mine;
    if (threadIdx.x == 0) *flag = mine;
    cluster_sync(ctas);
    unsigned v = 1;
    if (threadIdx.x < ctas) {
        uint32_t a;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ft::smem_addr(flag)), "r"(threadIdx.x));
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    }
    return __syncthreads_and(v);
}

__global__ void __launch_bounds__(CT, 1) kv_reorder_kernel(KvCtl c, int n, const int* __restrict__ rows,
                                                           const int* __restrict__ parents) {
    extern __shared__ __align__(16) uint8_t smem[];
    ReorderSmem& s = *reinterpret_cast<ReorderSmem*>(smem);
    const int lane = threadIdx.x & 31, rank = cluster_rank(), ctas = (int)cluster_size();
    const int wid = rank * (CT / 32) + (threadIdx.x >> 5), warps = ctas * (CT / 32);
    if (threadIdx.x == 0) s.cols = 0;
    clear(s.marks, c.n_rows);
    ft::grid_dep_launch();
    ft::grid_dep_wait();
    const int i = threadIdx.x;
    int r = -1, p = -1, len = 0;
    bool ok = true;
    if (i < n) {
        r = rows ? rows[i] : i;
        p = parents[i];
        if (!mark(s.marks, r, c.n_rows) || p < -1 || p >= c.n_rows) {
            ok = false;
        } else {
            const int old = c.lens[r];
            len = p < 0 ? 0 : c.lens[p];
            const long long most = (long long)c.row_pages * c.page;
            if (old < 0 || old > most || len < 0 || len > most) {
                ok = false;
            } else {
                s.row[i] = r;
                s.par[i] = p;
                s.len[i] = len;
                s.old[i] = (old + c.page - 1) >> c.page_log;
                s.full[i] = len >> c.page_log;
                s.keep[i] = 0x7fffffff;
                if (p != r) atomicMax(&s.cols, max(s.old[i], (len + c.page - 1) >> c.page_log));
                s.item_of[r] = (uint16_t)i;
            }
        }
    }
    auto leave = [&](unsigned bit) {
        if (bit && rank == 0) refuse(c, bit);
        cluster_sync(ctas);  // no CTA ends while another may read its flags
    };
    // (every CTA finds the same)
    if (!__syncthreads_and(ok)) return leave(FT_DEVERR_ARG);
    // the child that keeps the last page of a parent whose own row is in the list
    int j = -1;
    if (i < n && p >= 0 && (s.marks.w[p >> 5] >> (p & 31) & 1u)) {
        j = s.item_of[p];
        atomicMin(&s.keep[j], p == r ? -1 : i);
    }
    __syncthreads();
    const bool part = i < n && (len & (c.page - 1)) != 0;
    const bool keeps = j >= 0 && s.keep[j] == (p == r ? -1 : i);
    int want;
    const int at = ft::block_scan(part && !keeps ? 1 : 0, s.ws, want);
    if (i < n) s.last[i] = !part ? 0 : keeps ? 1 : 2 + at;
    __syncthreads();
    // Units: columns cb * RO_COLS .. of item k; a row that stays as it is has no work.
    const int blocks = (s.cols + RO_COLS - 1) / RO_COLS, units = blocks * n;
    struct Unit {
        const int *from, *mine;  // the parent's entries and the row's own
        int got, held;           // how many of them from here on (got: with a last page that is new)
        int k;
    };
    auto unit = [&](int u) {
        const int cb = u / n, k = u - cb * n, c0 = cb * RO_COLS;
        Unit x;
        x.k = k;
        x.from = c.table + (size_t)max(s.par[k], 0) * c.row_pages + c0;
        x.mine = c.table + (size_t)s.row[k] * c.row_pages + c0;
        const bool same = s.row[k] == s.par[k];
        x.got = same ? 0 : min(max(s.full[k] + (s.last[k] != 0) - c0, 0), RO_COLS);
        x.held = same ? 0 : min(max(s.old[k] - c0, 0), RO_COLS);
        return x;
    };
    // counts of the pages: those that the rows get, less those that they held (a new last page is not one of them)
    auto count = [&](int sign) {
        for (int u = wid; u < units; u += warps) {
            const Unit x = unit(u);
            const int c0 = (u / n) * RO_COLS;
            const int got = min(x.got, max(s.full[x.k] + (s.last[x.k] == 1) - c0, 0));
#pragma unroll
            for (int h = 0; h < RO_COLS / 32; ++h) {
                const int q = 32 * h + lane;
                const int to = q < got ? x.from[q] : -1, was = q < x.held ? x.mine[q] : -1;
                if (to == was) continue;  // (a page that the row keeps: beams of a request share many)
                if (to >= 0) atomicAdd(&c.refs[to], sign);
                if (was >= 0) atomicAdd(&c.refs[was], -sign);
            }
        }
    };
    // The rows' new entries are staged as they are read; where not all of them fit, again below, some columns at a time.
    const int most = n ? RO_SLOTS * ctas / n * n : 1;  // (n or more)
    const bool single = units <= most;
    for (int u = wid, slot = threadIdx.x >> 5; u < units; u += warps, slot += CT / 32) {
        const Unit x = unit(u);
        int a[RO_COLS / 32], b[RO_COLS / 32];
#pragma unroll
        for (int h = 0; h < RO_COLS / 32; ++h) {
            const int q = 32 * h + lane;
            a[h] = q < x.got ? x.from[q] : -1;
            b[h] = q < x.held ? x.mine[q] : 0;
        }
#pragma unroll
        for (int h = 0; h < RO_COLS / 32; ++h) {
            if ((32 * h + lane < x.got && (unsigned)a[h] >= (unsigned)c.n_pages) || (unsigned)b[h] >= (unsigned)c.n_pages) ok = false;
            if (single) s.stage[slot][32 * h + lane] = a[h];
        }
    }
    if (!cluster_all(ok, &s.flag[0], ctas)) return leave(FT_DEVERR_ARG);
    count(1);
    cluster_sync(ctas);
    const unsigned first = want ? free_bits<FREE_FIRST, true>(c, 0) : 0;
    // a page that a row held without being counted
    for (int u = wid; u < units; u += warps) {
        const Unit x = unit(u);
        int b[RO_COLS / 32];
#pragma unroll
        for (int h = 0; h < RO_COLS / 32; ++h) b[h] = 32 * h + lane < x.held ? __ldcg(&c.refs[x.mine[32 * h + lane]]) : 0;
#pragma unroll
        for (int h = 0; h < RO_COLS / 32; ++h)
            if (b[h] < 0) ok = false;
    }
    const int have = take_free<true>(c, want, s.ws, first, s.free);  // (in every CTA)
    const bool sound = cluster_all(ok, &s.flag[1], ctas);
    if (!sound || have < want) {
        count(-1);
        return leave(sound ? FT_DEVERR_CAPACITY : FT_DEVERR_ARG);
    }
    auto write = [&](int u, int slot) {
        const Unit x = unit(u);
        const int full = s.full[x.k] - (u / n) * RO_COLS, last = s.last[x.k];
#pragma unroll
        for (int h = 0; h < RO_COLS / 32; ++h) {
            const int q = 32 * h + lane;
            if (q >= max(x.got, x.held)) continue;
            int v = s.stage[slot][q];
            if (q == full && last >= 2) {
                const int src = v;
                v = s.free[last - 2];
                c.refs[v] = 1;
                c.copies[last - 2] = KvCopy{src, v, s.len[x.k] & (c.page - 1)};
            }
            const_cast<int*>(x.mine)[q] = v;
        }
    };
    // all rows have been read before one is written
    if (single) {
        if (ctas > 1) cluster_arrive();  // (this CTA has read the others' flags)
        for (int u = wid, slot = threadIdx.x >> 5; u < units; u += warps, slot += CT / 32) write(u, slot);
    } else {
        for (int u0 = 0; u0 < units; u0 += most) {
            const int end = min(units, u0 + most);
            for (int u = u0 + wid, slot = threadIdx.x >> 5; u < end; u += warps, slot += CT / 32) {
                const Unit x = unit(u);
                int a[RO_COLS / 32];
#pragma unroll
                for (int h = 0; h < RO_COLS / 32; ++h) a[h] = 32 * h + lane < x.got ? x.from[32 * h + lane] : -1;
#pragma unroll
                for (int h = 0; h < RO_COLS / 32; ++h) s.stage[slot][32 * h + lane] = a[h];
            }
            cluster_sync(ctas);
            for (int u = u0 + wid, slot = threadIdx.x >> 5; u < end; u += warps, slot += CT / 32) write(u, slot);
            cluster_sync(ctas);
        }
    }
    if (rank == 0) {
        if (i < n) c.lens[r] = len;
        set_info(c, want, want, -1);
    }
    if (single && ctas > 1) cluster_wait();
}

// live = pages in use; the k-th page in use at index >= live pairs with the
// k-th free page below it (there are equally many).  The two lists fill the
// copy list's ends independently, so both scans are one pass over refs.
__global__ void __launch_bounds__(CT) kv_compact_kernel(KvCtl c) {
    ft::grid_dep_launch();
    ft::grid_dep_wait();
    __shared__ int ws[32];
    int live = 0;
    for (int p = threadIdx.x; p < c.n_pages; p += CT) live += c.refs[p] > 0;
    ft::block_scan(live, ws, live);
    int holes = 0, movers = 0;
    for (int base = 0; base < c.n_pages; base += CT) {
        const int p = base + threadIdx.x;
        const bool in = p < c.n_pages, used = in && c.refs[p] > 0;
        const bool hole = in && p < live && !used, mover = used && p >= live;
        // at most 2^10 of each kind in a step: both counts in one word
        int total;
        const int at = ft::block_scan((hole ? 1 : 0) | (mover ? 1 << 16 : 0), ws, total);
        if (hole) c.copies[holes + (at & 0xffff)].dst = p;
        if (mover) c.copies[movers + (at >> 16)].src = p;
        holes += total & 0xffff;
        movers += total >> 16;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < movers; i += CT) {
        KvCopy& k = c.copies[i];
        k.tok = c.page;
        c.remap[k.src] = k.dst;
        c.refs[k.dst] = c.refs[k.src];
        c.refs[k.src] = 0;
    }
    set_info(c, 0, movers, live);
}

// The copies of the list.  A unit is 4 KiB of one bank of one page (a warp
// moves 512 bytes an instruction, eight loads in flight); banks of a page that
// is copied in part have their first tok*D values copied.  With `live` set,
// the table's entries past the live pages are replaced too.  HBM bound: 601
// pages of 1 MB moved by a compaction take 201 us with its control pass, 6.26
// TB/s, 92% of the copy rate.  Reads and writes bypass L1 and leave L2 first: a
// compaction reads no page twice (forks of one parent read its last page once a
// child, a few KB of it).
__global__ void __launch_bounds__(256) kv_copy_kernel(const int* n_copy, const KvCopy* __restrict__ copies, uint8_t* pool,
                                                      int banks, int bank_bytes, int tok_bytes, int* table,
                                                      long long entries, const int* __restrict__ remap,
                                                      const int* live, int n_pages) {
    ft::grid_dep_launch();
    ft::grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const long long wid = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const long long nw = (long long)gridDim.x * (blockDim.x >> 5);
    const int n = *n_copy;
    const int subs = (bank_bytes + 4095) / 4096;
    const long long units = (long long)n * banks * subs;
    for (long long u = wid; u < units; u += nw) {
        const int sub = (int)(u % subs);
        const long long pb = u / subs;
        const int b = (int)(pb % banks);
        const KvCopy k = copies[pb / banks];
        const int bytes = k.tok * tok_bytes - sub * 4096;
        const size_t off = (size_t)b * bank_bytes + (size_t)sub * 4096 + lane * 16;
        const uint8_t* s = pool + (size_t)k.src * banks * bank_bytes + off;
        uint8_t* d = pool + (size_t)k.dst * banks * bank_bytes + off;
        uint4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j * 512 + lane * 16 < bytes) v[j] = __ldcs(reinterpret_cast<const uint4*>(s + j * 512));
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j * 512 + lane * 16 < bytes) __stcs(reinterpret_cast<uint4*>(d + j * 512), v[j]);
    }
    if (live) {
        const int lv = *live;
        const long long step = (long long)gridDim.x * blockDim.x;
        for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < entries; i += step) {
            const int p = table[i];
            if (p >= lv && p < n_pages) table[i] = remap[p];
        }
    }
}

// at most `most` pages are copied
cudaError_t launch_copy(ft_kv* kv, bool compact, long long most) {
    int banks = kv->L * 2 * kv->Hkv, bank_bytes = kv->page * kv->D * 2, tok_bytes = kv->D * 2;
    long long entries = compact ? (long long)kv->n_rows * kv->row_pages : 0;
    const int* live = compact ? kv->info + KV_LIVE : nullptr;
    void* args[] = {&kv->n_copy, &kv->copies, &kv->pool, &banks, &bank_bytes, &tok_bytes,
                    &kv->table, &entries, &kv->remap, &live, &kv->n_pages};
    const long long ctas = (most * banks * ((bank_bytes + 4095) / 4096) + 7) / 8;  // a unit a warp
    const int grid = (int)(ctas < kv->num_sms * 8 ? ctas : kv->num_sms * 8);
    return launch_dependent((const void*)kv_copy_kernel, grid, 256, 0, kv->stream, args);
}

}  // namespace

cudaError_t launch_kv_extend(ft_kv* kv, int n, const int* rows, const int* add) {
    KvCtl c = ctl_of(kv);
    void* args[] = {&c, &n, &rows, &add};
    return launch_dependent((const void*)kv_extend_kernel, 1, CT, 0, kv->stream, args);
}

cudaError_t launch_kv_fork(ft_kv* kv, int n, const int* parents, const int* children) {
    KvCtl c = ctl_of(kv);
    void* args[] = {&c, &n, &parents, &children};
    const cudaError_t e = launch_dependent((const void*)kv_fork_kernel, 1, CT, 0, kv->stream, args);
    return e == cudaSuccess && n > 0 ? launch_copy(kv, false, n) : e;
}

cudaError_t launch_kv_free(ft_kv* kv, int n, const int* rows) {
    KvCtl c = ctl_of(kv);
    void* args[] = {&c, &n, &rows};
    return launch_dependent((const void*)kv_free_kernel, 1, CT, 0, kv->stream, args);
}

cudaError_t launch_kv_batch(ft_kv* kv, int B, const int* rows, const int* add, int T, int* cu_q, int* row_of, int* pos,
                            long long* slots) {
    KvCtl c = ctl_of(kv);
    BatchOut o{cu_q, row_of, pos, slots, T};
    int here = T <= LIST_HERE;
    void* args[] = {&c, &B, &rows, &add, &o, &here};
    const cudaError_t e = launch_dependent((const void*)kv_batch_kernel, 1, CT, 0, kv->stream, args);
    if (e != cudaSuccess || here) return e;
    void* list[] = {&c, &B, &rows, &add, &o};
    const long long ctas = ((long long)T + 255) / 256;
    return launch_dependent((const void*)kv_list_kernel, (int)(ctas < kv->num_sms * 8 ? ctas : kv->num_sms * 8), 256, 0,
                            kv->stream, list);
}

cudaError_t launch_kv_reorder(ft_kv* kv, int n, const int* rows, const int* parents) {
    KvCtl c = ctl_of(kv);
    cudaLaunchConfig_t cfg = {};
    const int ctas = n <= RO_ALONE && (long long)n * kv->row_pages <= RO_ALONE_ENTRIES ? 1 : RO_CTAS;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(CT);
    cfg.dynamicSmemBytes = sizeof(ReorderSmem);
    cfg.stream = kv->stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim = {(unsigned)ctas, 1, 1};
    cfg.attrs = at;
    cfg.numAttrs = 2;
    void* args[] = {&c, &n, &rows, &parents};
    const cudaError_t e = cudaLaunchKernelExC(&cfg, (const void*)kv_reorder_kernel, args);
    return e == cudaSuccess && n > 0 ? launch_copy(kv, false, n) : e;
}

cudaError_t kv_pages_setup() {
    return cudaFuncSetAttribute((const void*)kv_reorder_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(ReorderSmem));
}

cudaError_t launch_kv_compact(ft_kv* kv) {
    KvCtl c = ctl_of(kv);
    void* args[] = {&c};
    const cudaError_t e = launch_dependent((const void*)kv_compact_kernel, 1, CT, 0, kv->stream, args);
    return e == cudaSuccess ? launch_copy(kv, true, kv->n_pages) : e;
}

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
// extend 64, 23 MB copied) 20.7 us for its four kernels.
#include "ft_kv.cuh"

namespace {

constexpr int CT = 1024;  // threads of the control kernels

struct KvCtl {
    int *table, *lens, *refs;
    int n_pages, n_rows, row_pages, page;
    int *info, *n_copy, *free_list, *remap, *rank;
    KvCopy* copies;
    unsigned* err;
};

KvCtl ctl_of(const ft_kv* kv) {
    return KvCtl{kv->table, kv->lens, kv->refs, kv->n_pages, kv->n_rows, kv->row_pages, kv->page,
                 kv->info, kv->n_copy, kv->free_list, kv->remap, kv->rank, kv->copies, kv->err};
}

// Which of the four pages from base + 4 * thread on are free, one bit each.
__device__ __forceinline__ unsigned free_bits(const KvCtl& c, int base) {
    const int p = base + 4 * threadIdx.x;
    unsigned f = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (p + j < c.n_pages && c.refs[p + j] == 0) f |= 1u << j;
    return f;
}

// The lowest `want` free pages, ascending, to list; returns how many there are
// (at most a few more than `want` are counted).  first: free_bits(c, 0).
__device__ int take_free(const KvCtl& c, int want, int (&ws)[32], unsigned first) {
    int have = 0;
    for (int base = 0; base < c.n_pages && have < want; base += 4 * CT) {
        const unsigned f = base ? free_bits(c, base) : first;
        int total;
        int at = have + ft::block_scan(__popc(f), ws, total);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (f >> j & 1u) {
                if (at < want) c.free_list[at] = base + 4 * threadIdx.x + j;
                ++at;
            }
        have += total;
    }
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
    const unsigned first = free_bits(c, 0);
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
    if (take_free(c, want, ws, first) < want) return refuse(c, FT_DEVERR_CAPACITY);
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
    const unsigned first = free_bits(c, 0);
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
    if (take_free(c, want, ws, first) < want) return refuse(c, FT_DEVERR_CAPACITY);
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

cudaError_t launch_kv_compact(ft_kv* kv) {
    KvCtl c = ctl_of(kv);
    void* args[] = {&c};
    const cudaError_t e = launch_dependent((const void*)kv_compact_kernel, 1, CT, 0, kv->stream, args);
    return e == cudaSuccess ? launch_copy(kv, true, kv->n_pages) : e;
}

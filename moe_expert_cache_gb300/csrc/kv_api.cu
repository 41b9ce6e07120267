// Host side of the paged key/value cache: the C ABI declared in
// include/ft_kv.h.  Owns the handle's scratch, checks arguments and enqueues
// the kernels on the cache's stream; no call of a step synchronises or
// allocates.
#include "ft_kv.cuh"

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <new>

namespace {

bool sizes_ok(int Hq, int Hkv, int D, int n_pages, int n_rows, int T_max, int B_max) {
    if (!(Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0 && Hq / Hkv <= ATTN_BM && (D == 64 || D == 128 || D == 256) &&
          n_pages >= 1 && n_rows >= 1 && n_rows <= KV_MAX_ROWS && T_max >= 1 && B_max >= 1 && B_max <= ATTN_MAX_B &&
          (long long)T_max * Hq < (1ll << 30)))
        return false;
    // the plan numbers rows of partial results in 32 bits (attn_plan_sizes; at least 256 bytes a row, so more of them
    // would not fit the card either).  2^23 are kept for the CTAs' own: five items of 128 rows each for 13107 CTAs
    const long long tiles = ((long long)T_max * (Hq / Hkv) + ATTN_BM - 1) / ATTN_BM;
    return Hkv * (tiles + B_max) * ATTN_BM + (long long)T_max * Hq < (1ll << 31) - (1ll << 23);
}

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

// Offsets of the arrays in the scratch allocation.
struct Layout {
    size_t err, info, n_copy, copies, free_list, remap, rank, hdr, ctas, works, merges, seg, part_o, part_ml,
        total;
};

Layout layout(const AttnPlan& p, int D, int n_pages, int n_rows) {
    Layout l;
    size_t off = 0;
    auto carve = [&](size_t bytes) {
        const size_t o = off;
        off = align_up(off + bytes);
        return o;
    };
    l.err = carve(4);
    l.info = carve(KV_INFO_WORDS * 4);
    l.n_copy = carve(4);
    l.copies = carve((size_t)n_pages * sizeof(KvCopy));
    l.free_list = carve((size_t)n_pages * 4);
    l.remap = carve((size_t)n_pages * 4);
    l.rank = carve((size_t)n_rows * 4);
    l.hdr = carve(sizeof(AttnHdr));
    l.ctas = carve((size_t)p.n_cta * sizeof(AttnCta));
    l.works = carve((size_t)p.cap_works * sizeof(AttnWork));
    l.merges = carve((size_t)p.cap_merges * sizeof(AttnMerge));
    l.seg = carve(attn_seg_bytes(p));
    l.part_ml = carve((size_t)p.part_rows * sizeof(float2));
    l.part_o = carve((size_t)p.part_rows * D * 4);
    l.total = off;
    return l;
}

ft_status launched(cudaError_t e) {
    if (e == cudaSuccess) return FT_OK;
    if (getenv("FT_DEBUG")) fprintf(stderr, "libft: launch -> %s\n", cudaGetErrorString(e));
    return FT_ERR_CUDA;
}

bool misaligned(const void* p, size_t a) { return (uintptr_t)p % a != 0; }

// Whether rows [n] of w values of 2 bytes at a, ld values apart, and of v values at b, ld_b apart, may touch: their spans
// overlap, and they are not different columns of the rows of one buffer.
bool may_touch(const void* a, int64_t ld, int64_t w, const void* b, int64_t ld_b, int64_t v, int64_t n) {
    const uintptr_t a0 = (uintptr_t)a, a1 = a0 + ((size_t)(n - 1) * ld + w) * 2;
    const uintptr_t b0 = (uintptr_t)b, b1 = b0 + ((size_t)(n - 1) * ld_b + v) * 2;
    if (!(a0 < b1 && b0 < a1)) return false;
    if (ld != ld_b) return true;
    const uintptr_t row = (uintptr_t)ld * 2, off = b0 >= a0 ? (b0 - a0) % row : (row - (a0 - b0) % row) % row;
    return off < (uintptr_t)w * 2 || off + (uintptr_t)v * 2 > row;
}

}  // namespace

extern "C" {

size_t ft_kv_page_bytes(int32_t L, int32_t Hkv, int32_t D, int32_t page) {
    if (L < 1 || Hkv < 1 || (long long)L * 2 * Hkv >= (1ll << 31) - 1 || (D != 64 && D != 128 && D != 256) ||
        (page != 16 && page != 32 && page != 64 && page != 128))
        return 0;
    return (size_t)L * 2 * Hkv * page * D * 2;
}

size_t ft_kv_scratch_bytes(int32_t Hq, int32_t Hkv, int32_t D, int32_t n_pages, int32_t n_rows, int32_t T_max,
                           int32_t B_max) {
    if (!sizes_ok(Hq, Hkv, D, n_pages, n_rows, T_max, B_max)) return 0;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    AttnPlan p{};
    attn_plan_sizes(Hq, Hkv, D, T_max, B_max, sms, p);
    return layout(p, D, n_pages, n_rows).total;
}

ft_status ft_kv_init(ft_kv** out, int32_t L, int32_t Hq, int32_t Hkv, int32_t D, int32_t page, int32_t n_pages,
                     int32_t n_rows, int32_t row_pages, int32_t dtype, int32_t T_max, int32_t B_max, void* pool,
                     int32_t* table, int32_t* lens, int32_t* refs, void* stream) {
    if (!out) return FT_ERR_ARG;
    *out = nullptr;
    if (!ft_kv_page_bytes(L, Hkv, D, page) || !sizes_ok(Hq, Hkv, D, n_pages, n_rows, T_max, B_max) ||
        row_pages < 1 || (long long)row_pages * page >= (1ll << 31) - 1024 ||
        (long long)n_pages * L * 2 * Hkv >= (1ll << 31) - 1 || (long long)n_rows * row_pages >= (1ll << 31) - 1 ||
        (dtype != FT_KV_BF16 && dtype != FT_KV_F16) || !pool || !table || !lens || !refs || misaligned(pool, 128) ||
        misaligned(table, 4) || misaligned(lens, 4) || misaligned(refs, 4))
        return FT_ERR_ARG;
    ft_kv* kv = new (std::nothrow) ft_kv();
    if (!kv) return FT_ERR_OOM;
    kv->L = L; kv->Hq = Hq; kv->Hkv = Hkv; kv->D = D; kv->page = page;
    kv->n_pages = n_pages; kv->n_rows = n_rows; kv->row_pages = row_pages; kv->dtype = dtype;
    kv->T_max = T_max; kv->B_max = B_max;
    kv->pool = (uint8_t*)pool;
    kv->table = table; kv->lens = lens; kv->refs = refs;
    kv->stream = (cudaStream_t)stream;
    auto fail = [&](ft_status s) {
        cudaGetLastError();
        cudaFree(kv->arena);
        delete kv;
        return s;
    };
    if (cudaGetDevice(&kv->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&kv->num_sms, cudaDevAttrMultiProcessorCount, kv->device) != cudaSuccess)
        return fail(FT_ERR_CUDA);
    attn_plan_sizes(Hq, Hkv, D, T_max, B_max, kv->num_sms, kv->plan);
    const Layout l = layout(kv->plan, D, n_pages, n_rows);
    cudaError_t e = cudaMalloc(&kv->arena, l.total);
    if (e != cudaSuccess) return fail(e == cudaErrorMemoryAllocation ? FT_ERR_OOM : FT_ERR_CUDA);
    // the partial results are written before they are read; the rest starts at 0
    if (cudaMemset(kv->arena, 0, l.part_ml) != cudaSuccess) return fail(FT_ERR_CUDA);
    if (cudaDeviceSynchronize() != cudaSuccess) return fail(FT_ERR_CUDA);
    uint8_t* a = (uint8_t*)kv->arena;
    kv->err = (unsigned*)(a + l.err);
    kv->info = (int*)(a + l.info);
    kv->n_copy = (int*)(a + l.n_copy);
    kv->copies = (KvCopy*)(a + l.copies);
    kv->free_list = (int*)(a + l.free_list);
    kv->remap = (int*)(a + l.remap);
    kv->rank = (int*)(a + l.rank);
    kv->plan.hdr = (AttnHdr*)(a + l.hdr);
    kv->plan.ctas = (AttnCta*)(a + l.ctas);
    kv->plan.works = (AttnWork*)(a + l.works);
    kv->plan.merges = (AttnMerge*)(a + l.merges);
    kv->plan.seg = (int*)(a + l.seg);
    kv->part_o = (float*)(a + l.part_o);
    kv->part_ml = (float2*)(a + l.part_ml);
    if (!attn_encode_map(kv) || attn_setup(kv) != cudaSuccess) return fail(FT_ERR_CUDA);
    *out = kv;
    return FT_OK;
}

ft_status ft_kv_extend(ft_kv* kv, int32_t n, const int32_t* rows, const int32_t* add) {
    if (!kv || n < 0 || n > kv->n_rows || (n > 0 && (!rows || !add))) return FT_ERR_ARG;
    return launched(launch_kv_extend(kv, n, rows, add));
}

ft_status ft_kv_fork(ft_kv* kv, int32_t n, const int32_t* parents, const int32_t* children) {
    if (!kv || n < 0 || n > kv->n_rows || (n > 0 && (!parents || !children))) return FT_ERR_ARG;
    return launched(launch_kv_fork(kv, n, parents, children));
}

ft_status ft_kv_free(ft_kv* kv, int32_t n, const int32_t* rows) {
    if (!kv || n < 0 || n > kv->n_rows || (n > 0 && !rows)) return FT_ERR_ARG;
    return launched(launch_kv_free(kv, n, rows));
}

ft_status ft_kv_compact(ft_kv* kv) {
    if (!kv) return FT_ERR_ARG;
    return launched(launch_kv_compact(kv));
}

ft_status ft_qk_rope_store(ft_kv* kv, int32_t layer, int32_t T, const void* qkv, int64_t ld, const int32_t* row_of,
                           const int32_t* pos, void* q_out, int64_t ld_q, const void* q_norm, const void* k_norm,
                           float eps, const float* cos_sin, int32_t max_pos, int32_t rot, int32_t pair) {
    if (!kv || layer < 0 || layer >= kv->L || T < 0 || rot < 0 || rot > kv->D || rot % 16 || (pair != 0 && pair != 1) ||
        !(eps >= 0.f) || !std::isfinite(eps))
        return FT_ERR_ARG;
    if (T == 0) return FT_OK;
    const int64_t w = ((int64_t)kv->Hq + 2 * (int64_t)kv->Hkv) * kv->D, wq = (int64_t)kv->Hq * kv->D;
    if (!qkv || !row_of || !pos || !q_out || ld < w || ld % 8 || ld_q < wq || ld_q % 8 || misaligned(qkv, 16) || misaligned(q_out, 16) ||
        misaligned(q_norm, 16) || misaligned(k_norm, 16) || (rot && (!cos_sin || max_pos < 1 || misaligned(cos_sin, 16))) ||
        (q_out == qkv ? ld != ld_q : may_touch(qkv, ld, w, q_out, ld_q, wq, T)))
        return FT_ERR_ARG;
    RopeArgs a{qkv, ld, row_of, pos, q_out, ld_q, q_norm, k_norm, eps, cos_sin, rot ? max_pos : 0x7fffffff, rot, pair,
               layer, T};
    return launched(launch_qk_rope_store(kv, a));
}

ft_status ft_attn_plan(ft_kv* kv, int32_t B, int32_t T, const int32_t* cu_q, const int32_t* rows, int32_t n_groups,
                       const int32_t* group_start, const int32_t* group_tokens) {
    if (!kv || B < 0 || B > kv->B_max || T < 0 || T > kv->T_max || n_groups < 0 || n_groups > B || (B > 0 && !cu_q) ||
        (n_groups > 0 && (!group_start || !group_tokens)))
        return FT_ERR_ARG;
    kv->have_plan = false;
    const ft_status st = launched(launch_attn_plan(kv, B, T, cu_q, rows, n_groups, group_start, group_tokens));
    if (st == FT_OK) {
        kv->have_plan = true;
        kv->plan_T = T;
    }
    return st;
}

ft_status ft_attn_forward(ft_kv* kv, int32_t layer, const void* q, int64_t ld_q, void* out, int64_t ld_o, float scale) {
    if (!kv || layer < 0 || layer >= kv->L || !(scale > 0.f) || !std::isfinite(scale)) return FT_ERR_ARG;
    if (!kv->have_plan) return FT_ERR_STATE;
    if (kv->plan_T == 0) return FT_OK;
    const int64_t w = (int64_t)kv->Hq * kv->D;
    if (!q || !out || ld_q < w || ld_o < w || ld_q % 8 || ld_o % 8 || misaligned(q, 16) || misaligned(out, 16))
        return FT_ERR_ARG;
    // out may lie between the rows of q only if no row of it touches one of q: refuse any overlap of the two spans
    const uintptr_t q0 = (uintptr_t)q, q1 = q0 + ((size_t)(kv->plan_T - 1) * ld_q + w) * 2;
    const uintptr_t o0 = (uintptr_t)out, o1 = o0 + ((size_t)(kv->plan_T - 1) * ld_o + w) * 2;
    if (q0 < o1 && o0 < q1) return FT_ERR_ARG;
    return launched(launch_attn_forward(kv, layer, q, ld_q, out, ld_o, scale));
}

ft_status ft_kv_last(ft_kv* kv, ft_kv_info* out) {
    if (!kv || !out) return FT_ERR_ARG;
    int w[KV_INFO_WORDS];
    if (cudaStreamSynchronize(kv->stream) != cudaSuccess) return FT_ERR_CUDA;
    if (cudaMemcpy(w, kv->info, sizeof w, cudaMemcpyDeviceToHost) != cudaSuccess) return FT_ERR_CUDA;
    out->allocated = w[KV_ALLOCATED];
    out->copied = w[KV_COPIED];
    out->live = w[KV_LIVE];
    return FT_OK;
}

ft_status ft_kv_status(ft_kv* kv) {
    if (!kv) return FT_ERR_ARG;
    if (cudaStreamSynchronize(kv->stream) != cudaSuccess) return FT_ERR_CUDA;
    unsigned e = 0;
    if (cudaMemcpy(&e, kv->err, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return FT_ERR_CUDA;
    if (e && cudaMemset(kv->err, 0, 4) != cudaSuccess) return FT_ERR_CUDA;
    if (e && cudaDeviceSynchronize() != cudaSuccess) return FT_ERR_CUDA;
    if (e & FT_DEVERR_TIMEOUT) return FT_ERR_TIMEOUT;
    if (e & FT_DEVERR_ARG) return FT_ERR_DEVICE;
    if (e & FT_DEVERR_CAPACITY) return FT_ERR_CAPACITY;
    return FT_OK;
}

void ft_kv_destroy(ft_kv* kv) {
    if (!kv) return;
    cudaStreamSynchronize(kv->stream);
    cudaFree(kv->arena);
    delete kv;
}

}  // extern "C"

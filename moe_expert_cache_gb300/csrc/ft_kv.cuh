// The paged key/value cache's handle, its plan records and the launchers of
// its kernels.  Internal to libft (the ABI is include/ft_kv.h).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/ft_kv.h"
#include "ft_common.cuh"

#define FT_DEVERR_CAPACITY 4u  // too few free pages

constexpr int KV_MAX_ROWS = 65536;  // rows of a table (a bit each in shared memory)

// Words of the page operations' summary.
enum { KV_ALLOCATED = 0, KV_COPIED, KV_LIVE, KV_INFO_WORDS };

// One page to copy: the first `tok` tokens of every bank of record src to dst.
struct KvCopy {
    int src, dst, tok;
};

// ------------------------------------------------------------ attention plan
//
// A segment is up to 128 query rows of one key/value head that run over one
// range of keys.  Row r of an owner (a request, or the requests of a group
// taken together) is query token tok0 + r / G, query head h*G + r % G, with
// G = Hq / Hkv: token-major, so that the rows of consecutive requests are
// consecutive.  A work item is a segment of one head, or the part of one that
// a CTA got.

constexpr int ATTN_BM = 128;        // rows of a work item (TMEM lanes)
constexpr int ATTN_BN = 128;        // keys of a tile
constexpr int ATTN_MAX_B = 1024;    // requests of a plan (one thread each)
constexpr int ATTN_NOMASK = 0x7fffffff;

struct __align__(16) AttnWork {
    int head;     // key/value head
    int trow;     // table row whose pages hold the keys
    int pos0;     // position of the first key of the first tile
    int ntile;    // tiles of 128 keys
    int kend;     // keys at positions >= kend are not there
    int vis0;     // token i of the owner sees positions < vis0 + i
    int tok0;     // first query token of the owner
    int r0;       // row of the owner that is row 0 here
    int nrows;    // 1..128
    int prow;     // first row of the partial result, or -1: write the output
    int pad[2];   // 48 bytes: records are fetched by bulk copies of 16-byte multiples
};

// What a CTA finds first: its items and a copy of the first of them.
struct __align__(16) AttnCta {
    int w0, w1, pad[2];
    AttnWork first;
};

// Rows to join, at most 8 / wpr of them.
struct AttnMerge {
    int head, tok0, r0, nrows;  // as in AttnWork
    int brow;                   // partial row of the first row's piece that starts its segment
    int c0, nc;                 // CTAs c0 .. c0+nc-1 hold further pieces
    int ptok0;                  // first token of the group whose shared prefix these rows ran over, or -1
    int pitem, pnrt, pnch;      // its first item of this head, row tiles and chunks
    int wpr;                    // warps of a row: 1, 2, 4 or 8
};

struct AttnHdr {
    int n_merge;
    int n_works;
};

struct AttnPlan {
    AttnHdr* hdr;
    AttnCta* ctas;      // [n_cta]
    AttnWork* works;    // [cap_works]
    AttnMerge* merges;  // [cap_merges]
    int* seg;           // scratch of the plan kernel
    int n_cta;
    int cap_segs, cap_works, cap_merges;
    int cap_items;      // prefix items (region A of the partials)
    long long b_row;    // first row of region B (a segment's first piece)
    long long c_row;    // first row of region C (one piece per CTA)
    long long part_rows;
};

struct ft_kv {
    int L, Hq, Hkv, D, page, n_pages, n_rows, row_pages, dtype, T_max, B_max;
    int device, num_sms;
    uint8_t* pool;
    int *table, *lens, *refs;
    cudaStream_t stream;
    void* arena;
    unsigned* err;
    int* info;         // [KV_INFO_WORDS]
    int* n_copy;       // pages of the copy list
    KvCopy* copies;    // [n_pages]
    int* free_list;    // [n_pages]
    int* remap;        // [n_pages]
    int* rank;         // [n_rows]
    AttnPlan plan;
    float* part_o;     // [part_rows, D] unnormalised partial outputs
    float2* part_ml;   // [part_rows] running maximum (log2 units) and sum
    bool have_plan;
    bool few_rows;     // the plan's requests have few rows each on average and share nothing
    int plan_T;
    CUtensorMap map;   // [n_pages*L*2*Hkv][page][D] of the pool
};

cudaError_t launch_kv_extend(ft_kv* kv, int n, const int* rows, const int* add);
cudaError_t launch_kv_fork(ft_kv* kv, int n, const int* parents, const int* children);
cudaError_t launch_kv_free(ft_kv* kv, int n, const int* rows);
cudaError_t launch_kv_compact(ft_kv* kv);

struct RopeArgs {
    const void* qkv;
    long long ld;
    const int* row_of;
    const int* pos;
    void* q_out;
    long long ld_q;
    const void* q_norm;
    const void* k_norm;
    float eps;
    const float* cos_sin;
    int max_pos, rot, pair, layer, T;
};
cudaError_t launch_qk_rope_store(ft_kv* kv, const RopeArgs& a);

// sizes of a plan's arrays and of the partial results
void attn_plan_sizes(int Hq, int Hkv, int D, int T_max, int B_max, int num_sms, AttnPlan& p);
size_t attn_seg_bytes(const AttnPlan& p);
bool attn_encode_map(ft_kv* kv);
cudaError_t attn_setup(ft_kv* kv);  // the kernels' shared-memory limits, once per handle
cudaError_t launch_attn_plan(ft_kv* kv, int B, int T, const int* cu_q, const int* rows, int n_groups,
                             const int* group_start, const int* group_tokens);
cudaError_t launch_attn_forward(ft_kv* kv, int layer, const void* q, long long ld_q, void* out, long long ld_o,
                                float scale);

// Launch on s as a programmatic dependent of the kernel before it: the CTAs may
// start while that one drains, set themselves up, and wait for its end (and its
// writes) by grid_dep_wait() before they touch any global memory.
inline cudaError_t launch_dependent(const void* k, int grid, int block, size_t smem, cudaStream_t s, void** args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, k, args);
}

namespace ft {
__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Exclusive prefix sum over a CTA of 1024 threads; total gets the sum.
template <class V>
__device__ __forceinline__ V block_scan(V v, V (&ws)[32], V& total) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    V x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const V y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // the previous call's reads of ws are over
    if (lane == 31) ws[wid] = x;
    __syncthreads();
    if (wid == 0) {
        V s = ws[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const V y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        ws[lane] = s;
    }
    __syncthreads();
    total = ws[31];
    return x - v + (wid ? ws[wid - 1] : 0);
}
}  // namespace ft

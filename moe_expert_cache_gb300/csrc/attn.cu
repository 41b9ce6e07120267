// ft_attn_plan, ft_attn_forward: attention over the page table, with the
// prefix that the requests of a group share multiplied once for all of them.
//
//   S = Q K^T, P = exp2(scale*log2(e)*(S - m)), O = P V, l = sum P
//
// with the running maximum m of a row over the tiles seen so far; pieces of
// the key axis that different CTAs computed join by
//   out = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k,   M = max m_k.
//
// A work item is up to 128 query rows of one key/value head (the G query heads
// of a token are G rows) over a range of 128-key tiles.  Where a group shares a
// prefix, the rows of all its requests form the tiles that run over it, so each
// key is read once for 128 rows; the requests' own keys follow as items of
// their own rows.  Work is laid out by the plan kernel: the shared ranges in
// equal chunks, round robin, so that the CTAs that work on one chunk with
// different rows do so at the same time and share it in L2; everything else as
// one line of tiles cut into equal parts, one per CTA, whatever request or head
// a cut falls into.
//
// One CTA: 4 softmax warps (a thread per row), a TMA warp each for keys and
// values, an MMA warp; K and V tiles in rings of shared memory with 128-byte
// swizzle; S and O in TMEM; P goes back to TMEM over its S and is the A operand
// of P V.  Two CTAs an SM at head sizes 64 and 128: while one's softmax works,
// the tensor core has the other's products.  At 256, where O takes half of
// TMEM, one CTA with two score buffers.
//
// Requests with few rows that share nothing (up to 16 rows each on average, head
// sizes 128 and 256) run a kernel that takes such items transposed,
//   S^T = K Q^T, O^T = V^T P^T,
// so that a softmax thread has a key and its few queries instead of a row and
// 128 keys: 64 requests of 512 keys 14.8 -> 12.5 us, 76 of 640 17.8 -> 15.1
// (13.1 -> 12.7 and 15.6 -> 14.8 at 256).  Beside a shared prefix it loses: 64
// requests behind 8192 keys at equal time, 256 with 64 keys of their own 54 ->
// 61 us, 6 behind 131072 keys 57 -> 58.5, and a kernel that only has both forms
// costs the other 2-3%; head size 64, whose products have N = 64 already, 19 ->
// 24 us.  Hence the rule on what the plan call says.
//
// The running maximum is a reference that may fall behind: past an item's first
// tile the weights are taken on the present one, and only where a tile's weights
// sum to more than 4096 (f16: 254) is the tile done again on its own maximum and O
// rescaled.  The weights stay as exact (they are floating-point numbers on any
// scale), no maxima are taken, and almost no tile touches O.
//
// What bounds it: few rows, HBM (8 rows over 262144 keys: 537 MB in 85 us with
// the join, 93% of the copy rate); many rows, the chain scores -> weights ->
// product of a CTA beside the other CTA's (a prompt of 4096 tokens behind 8192
// at head size 128: 490 us, 1400 TFLOP/s, 73% of cuBLAS; 387 us at head size
// 256); short items, the latency of their start (about 3 us).
//
// The weights are rounded to the cache's type, as the tensor core takes both
// operands in one: against 64 bits 2.3e-3 in bf16 and 2.8e-4 in f16, where the
// rounding of the output alone gives 1.7e-3 and 2.1e-4.
// Tried at head size 128 and left: tiles of 64 keys (the products of 128 x 64
// wait for Q's reads; 4% slower), one CTA with two streams of 128 rows over
// shared tiles (prompts 4% faster, short items 1.6 times slower) or over
// alternate tiles (the ring could not keep up), rings of half tiles (3% slower),
// the weights of half a tile handed over before the other half's (14% slower),
// a cooperative launch with the join at its end (launch +2 us).
#include <climits>
#include <type_traits>

#include "attn_line.cuh"
#include "ft_kv.cuh"
#include "ft_tc.cuh"

namespace {

constexpr int G_THREADS = 256;        // 4 softmax warps, two TMA warps, an MMA warp, an idle one
// with two CTAs an SM: 128 registers a thread at launch; 128 x 208 + 128 x 48 = 256 x 128
constexpr int REGS_SOFTMAX = 208, REGS_OTHER = 48;
constexpr float LOG2E = 1.4426950408889634f;
// f16 weights are taken on a reference 2^8 below the row's own: 2^-24, the smallest f16 number, is then 2^-32 of the
// largest weight, and a strong first key does not drown a long context (4096 keys of 2^-26 to 2^-30 of its weight each
// lost all of their 2^-15 of the result).  bf16 has the range without.  MAX_SUM is the most that a tile's weights may
// sum to on a reference that has fallen behind, 254 and 4096 of the reference's own weight (f16 holds 65504; a tile's
// 128 weights sum to 128 of it at most while the reference is the largest score).
template <bool BF>
constexpr float SHIFT = BF ? 0.f : 8.f;
template <bool BF>
constexpr float MAX_SUM = BF ? 4096.f : 65024.f;
// pieces that a warp of the join has in flight, and the join's CTAs on an SM.  More pieces need registers that the
// loads' addresses want (64 requests behind 8192 keys at head size 128: 6 pieces 28.6 us, 12 30.1, 16 31.3; with 3 CTAs
// an SM 30.5; 130 behind 16384 at 256, 2 CTAs: 4 pieces 58.7 us, 6 58.1, 8 58.9, 4 with 3 CTAs 61.8)
constexpr int MERGE_NB(int D) { return D == 64 ? 8 : 6; }
constexpr int MERGE_CTAS(int D) { return D == 64 ? 3 : 2; }
constexpr int NQ = 16;               // items of up to this many rows take the transposed form
constexpr int NWORK = 16;            // work items of a CTA that are kept in shared memory
using attnline::OVP;
using attnline::upper;

template <int D>
struct Cfg {
    static constexpr int CTAS = D != 256 ? 2 : 1;             // per SM
    static constexpr uint32_t TCOLS = CTAS == 1 ? 512 : 256; // O: D columns, S: NS x 128
    static constexpr int NS = CTAS == 1 ? 2 : 1;
    static constexpr uint32_t QBYTES = ATTN_BM * D * 2;
    // K and V have a ring each.  At head size 256 their tiles come in halves (K by values, V by keys), so that a stage
    // is free again, and the next load under way, while the other half is still in use (prompts 441 -> 413 us); with two
    // CTAs an SM the other CTA covers that, and the doubled number of copies cost 3%
    static constexpr int HALVES = D == 256 ? 2 : 1;
    static constexpr uint32_t STAGE = ATTN_BN * D * 2 / HALVES;
    static constexpr int NK = D == 256 ? 2 : D == 128 ? 1 : 3, NV = D == 128 ? 1 : 3;      // stages
    static constexpr size_t SMEM = QBYTES + (size_t)(NK + NV) * STAGE;
};

struct AttnArgs {
    const AttnHdr* hdr;
    const AttnWork* works;
    const AttnCta* ctas;
    const AttnMerge* merges;
    long long c_row;
    const uint16_t* q;
    long long ld_q;
    uint16_t* out;
    long long ld_o;
    const int* table;
    int row_pages, page, page_log, n_pages, L, Hkv, G, layer;
    float c;        // scale * log2(e)
    float* part_o;
    float2* part_ml;
    unsigned* err;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 operations in one instruction, on the halves of a 64-bit register.
__device__ __forceinline__ uint64_t f2(float a, float b) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ float2 unf2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

template <bool BF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if (BF) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Shared-memory descriptors, split into the low word (start >> 4, and at bit 16
// the leading byte offset >> 4) and a constant high word (stride 1024 bytes,
// version 1, 128-byte swizzle).  K-major (Q, K): rows of 64 values, 8-row groups
// 1024 bytes apart; the leading offset is not used.  V lies transposed: atoms of
// 64 values by 8 keys, 1024 bytes from one group of 8 keys to the next, `lead`
// bytes from one block of 64 values to the next.
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(const void* tile) { return (ft::smem_addr(tile) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_v(const void* tile, uint32_t lead) {
    return (ft::smem_addr(tile) >> 4) | ((lead >> 4) << 16);
}

// kind::f16 with bf16 (1) or f16 (0) operands, fp32 accumulator; bits 15 and
// 16: A is given with M, B with N contiguous.
constexpr uint32_t idesc_of(bool bf, int N, bool a_mn, bool b_mn) {
    return (1u << 4) | ((bf ? 1u : 0u) << 7) | ((bf ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
           ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(ATTN_BM >> 4) << 24);
}

// The MMA warp runs converged and elects the issuing thread inside each
// instruction: its operands then stay in uniform registers.  Beside two busy
// softmax warps on its scheduler a 128 x 128 x 16 product measured 81 cycles an
// instruction this way (64 is its own time), 220 issued by one diverged thread,
// which moves every operand from its own registers.

// D[tmem] (+)= A[smem] * B[smem]^T
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\t.reg .b32 t;\n\t"
        "mov.b64 da, {%1, %5};\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "elect.sync t|q, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(DESC_HI)
        : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\t.reg .b32 t;\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "elect.sync t|q, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(DESC_HI)
        : "memory");
}
// Arrive once on `bar` when all that the elected thread has issued so far is done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t.reg .b32 t;\n\t"
        "elect.sync t|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(ft::smem_addr(bar))
        : "memory");
}
// S (+)= Q K^T over NB blocks of 64 values: steps of 16 values.
template <int NB>
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t q, uint32_t k, uint32_t idesc, uint32_t accumulate) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            mma_ss(d, q + b * (ATTN_BM * 128 / 16) + 2 * i, k + b * (ATTN_BN * 128 / 16) + 2 * i, idesc,
                   (b | i) ? 1u : accumulate);
}
// O (+)= P V over 64 keys: steps of 16 keys, 8 columns of P and 2048 bytes of V.
__device__ __forceinline__ void mma_values(uint32_t o, uint32_t pt, uint32_t v, uint32_t idesc, uint32_t accumulate) {
#pragma unroll
    for (int i = 0; i < 4; ++i) mma_ts(o, pt + 8 * i, v + 128 * i, idesc, i ? 1u : accumulate);
}

// O^T (+)= V^T P^T over 64 keys, 128 values: both operands in shared memory.
__device__ __forceinline__ void mma_values_t(uint32_t o, uint32_t v, uint32_t pt, uint32_t idesc, uint32_t accumulate) {
#pragma unroll
    for (int i = 0; i < 4; ++i) mma_ss(o, v + 128 * i, pt + 2 * i, idesc, i ? 1u : accumulate);
}

// A place in the ring and the parity of its phase.
struct Slot {
    int st = 0;
    uint32_t ph = 0;
};
template <int NST>
__device__ __forceinline__ void advance(Slot& s) {
    if (++s.st == NST) {
        s.st = 0;
        s.ph ^= 1u;
    }
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
// 32 lanes x 16 columns: one row a thread.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// x[j] of all lanes by op, for 16 j: each step hands half of the values to the partner.  Lane i gets j = i / 2; x is
// used up.
template <class Op>
__device__ __forceinline__ float warp_columns(float* x, int lane, Op op) {
#pragma unroll
    for (int o = 16; o > 1; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int j = 0; j < o / 2; ++j) {
            const float send = up ? x[j] : x[j + o / 2], keep = up ? x[j + o / 2] : x[j];
            x[j] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
    }
    return op(x[0], __shfl_xor_sync(0xffffffffu, x[0], 1));
}
// Whether a predicate holds in any of the four softmax warps, and a barrier for them.
__device__ __forceinline__ bool any_of_128(bool x) {
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((int)x)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"((uint16_t)v) : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 TMEM lanes x 32 columns.  A quad of threads holds 8 columns of a block of 8 values: r[4*b + e] is column
// 8*b + 2*(lane % 4) + e of row lane / 4, r[4*b + 2 + e] of row lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_quads(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// Partial results keep the values of a row's 32-column group in the order in which that load has them in a quad:
// the 8 values of a thread, 32 bytes, lie together, and a store of a warp fills whole lines of 8 rows instead of a
// sector of each of 32.  Column of place x, and place of column x:
__device__ __forceinline__ int part_column(int x) { return (x & ~30) | (x & 6) << 2 | (x >> 2 & 6); }

// 32 bytes to global memory in one store (a whole sector of one row).
__device__ __forceinline__ void st_global32(void* d, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(d), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Joins the pieces of the rows that have more than one: a CTA per record, D/32
// columns a lane.  The order of the pieces is fixed by the plan, so is the
// order of the sums.  Rows with many pieces (a long sequence has one per CTA
// that worked on it) have several warps, which share the pieces.
template <int D, bool BF>
__global__ void __launch_bounds__(256, MERGE_CTAS(D)) attn_merge_kernel(const AttnArgs p) {
    constexpr int V = D / 32, NB = MERGE_NB(D);
    __shared__ float s_acc[8 * D];
    __shared__ float2 s_md[8];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    ft::grid_dep_launch();
    ft::grid_dep_wait();
    // the first record is read beside the count (there is room for as many records as CTAs)
    AttnMerge k = p.merges[blockIdx.x];
    const int n = p.hdr->n_merge;
    for (int u = blockIdx.x; u < n; u += gridDim.x) {
        if (u != (int)blockIdx.x) k = p.merges[u];
        const int na = k.ptok0 >= 0 ? k.pnch : 0, np = na + 1 + k.nc, wpr = k.wpr;
        const int share = wid % wpr, r = wid / wpr;  // a record has at most 8 / wpr rows
        const bool on = r < k.nrows;
        const int R = k.r0 + r, tok = k.tok0 + R / p.G, gh = R % p.G;
        float M = -INFINITY, den = 0.f, acc[V];
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = 0.f;
        if (on) {
            long long abase = 0;
            if (na) {
                const int PR = (tok - k.ptok0) * p.G + gh;
                abase = (long long)(k.pitem + PR / ATTN_BM) * ATTN_BM + PR % ATTN_BM;
            }
            // this warp's pieces are share, share + wpr, ...; 32 of them at a time, one a lane
            for (int b = share; b < np; b += 32 * wpr) {
                const int i = b + lane * wpr;
                const long long pr = i < na    ? abase + (long long)i * k.pnrt * ATTN_BM
                                     : i == na ? (long long)k.brow + r
                                               : p.c_row + (long long)(k.c0 + i - na - 1) * ATTN_BM + R % ATTN_BM;
                float2 ml = make_float2(-INFINITY, 0.f);
                if (i < np) ml = __ldcg(p.part_ml + pr);
                const int e = min(32, (np - b + wpr - 1) / wpr);
                float wgt = 0.f;
                for (int i0 = 0; i0 < e; i0 += NB) {
                    float x[NB][V];
#pragma unroll
                    for (int q = 0; q < NB; ++q) {
                        const long long ri = __shfl_sync(0xffffffffu, pr, (i0 + q) & 31);
                        if (i0 + q < e) {
                            const float* src = p.part_o + ri * D + lane * V;
                            if (V == 2) {
                                *reinterpret_cast<float2*>(x[q]) = __ldcg(reinterpret_cast<const float2*>(src));
                            } else {
#pragma unroll
                                for (int j = 0; j + 3 < V; j += 4)
                                    *reinterpret_cast<float4*>(x[q] + j) = __ldcg(reinterpret_cast<const float4*>(src + j));
                            }
                        }
                    }
                    if (i0 == 0) {  // the statistics arrive while the first values are on their way
                        float mb = ml.x;
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, o));
                        const float Mn = fmaxf(M, mb), ref = Mn == -INFINITY ? 0.f : Mn;
                        const float f = ex2(M - ref);
                        wgt = ex2(ml.x - ref);
                        den = den * f + wgt * ml.y;
#pragma unroll
                        for (int j = 0; j < V; ++j) acc[j] *= f;
                        M = Mn;
                    }
#pragma unroll
                    for (int q = 0; q < NB; ++q) {
                        const float wi = __shfl_sync(0xffffffffu, wgt, (i0 + q) & 31);
                        if (i0 + q < e) {
#pragma unroll
                            for (int j = 0; j < V; ++j) acc[j] += wi * x[q][j];
                        }
                    }
                }
            }
            den = ft::warp_sum(den);
        }
        if (wpr > 1) {
#pragma unroll
            for (int j = 0; j < V; ++j) s_acc[wid * D + lane * V + j] = acc[j];
            if (lane == 0) s_md[wid] = make_float2(M, den);
            __syncthreads();
            if (on && share == 0) {
                for (int q = 1; q < wpr; ++q) {
                    const float2 md = s_md[wid + q];
                    const float Mn = fmaxf(M, md.x), ref = Mn == -INFINITY ? 0.f : Mn;
                    const float f = ex2(M - ref), h = ex2(md.x - ref);
                    den = den * f + md.y * h;
#pragma unroll
                    for (int j = 0; j < V; ++j) acc[j] = acc[j] * f + s_acc[(wid + q) * D + lane * V + j] * h;
                    M = Mn;
                }
            }
            __syncthreads();
        }
        if (on && share == 0) {
            const float inv = den > 0.f ? 1.f / den : (den == 0.f ? 0.f : den);
            uint16_t* dst = p.out + (long long)tok * p.ld_o + (k.head * p.G + gh) * D;
#pragma unroll
            for (int j = 0; j < V; j += 2)
                *reinterpret_cast<uint32_t*>(dst + part_column(lane * V + j)) = pack2<BF>(acc[j] * inv, acc[j + 1] * inv);
        }
    }
}

template <int D, bool BF, bool FEW>
__global__ void __launch_bounds__(G_THREADS, Cfg<D>::CTAS) attn_kernel(const __grid_constant__ CUtensorMap map,
                                                                       const AttnArgs p) {
    using C = Cfg<D>;
    constexpr int NK = C::NK, NV = C::NV, NS = C::NS;
    extern __shared__ __align__(1024) unsigned char smQ[];  // Q, then the rings of K and V
    __shared__ uint64_t k_full[NK], k_empty[NK], v_full[NV], v_empty[NV], s_full[NS], p_full[NS], pv_done[2], q_full, o_full, o_empty, w_full,
        done;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_fail;
    __shared__ __align__(16) AttnWork s_work[NWORK];
    __shared__ __align__(16) float s_red[NQ][4];  // transposed form: a value of each query and softmax warp
    unsigned char *ring_k = smQ + C::QBYTES, *ring_v = ring_k + NK * C::STAGE;
    unsigned char* smP = smQ + 64 * 128;  // transposed form: NS x 4 KB in rows of Q that its items do not have
    const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31;

    if (tid == 128) {
        for (int s = 0; s < NK; ++s) {
            ft::mbar_init(&k_full[s], 1);
            ft::mbar_init(&k_empty[s], 1);
        }
        for (int s = 0; s < NV; ++s) {
            ft::mbar_init(&v_full[s], 1);
            ft::mbar_init(&v_empty[s], 1);
        }
        for (int b = 0; b < NS; ++b) {
            ft::mbar_init(&s_full[b], 1);
            ft::mbar_init(&p_full[b], 4);
        }
        for (int b = 0; b < 2; ++b) ft::mbar_init(&pv_done[b], 1);
        ft::mbar_init(&q_full, 4);
        ft::mbar_init(&o_full, 1);
        ft::mbar_init(&o_empty, 4);
        ft::mbar_init(&w_full, 1);
        ft::mbar_init(&done, 1);
        ft::mbar_fence_init();
        s_fail = 0;
        tc::prefetch_map(&map);
    }
    if (wid == 5) tc::tmem_alloc(&s_tmem, C::TCOLS);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;
    ft::grid_dep_launch();  // (its TMEM is allocated: no CTA of a later kernel can hold what this one needs)
    // up to here nothing touched global memory: it ran beside the end of the kernel before this one
    ft::grid_dep_wait();
    const AttnCta mine0 = p.ctas[blockIdx.x];
    const int w0 = mine0.w0, w1 = mine0.w1;
    auto load_q = [&](const AttnWork& k) {
        constexpr int CH = D / 8, RS = 128 / CH;  // 16-byte chunks of a row, rows of a step
        const int ch = tid % CH, rr0 = tid / CH, R = k.r0 + rr0;
        const int dt = RS / p.G, dg = RS % p.G;   // a step in tokens and heads: no division in the loop
        int gh = R % p.G;
        const uint16_t* src = p.q + (long long)(k.tok0 + R / p.G) * p.ld_q + (k.head * p.G + gh) * D + ch * 8;
        const long long step = dt * p.ld_q + dg * D, wrap = p.ld_q - p.G * D;
        unsigned char* dst = smQ + (ch >> 3) * (ATTN_BM * 128);
        for (int rr = rr0; rr < k.nrows; rr += RS) {
            ft::cp_async16(dst + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4), src);
            src += step;
            gh += dg;
            if (gh >= p.G) {
                gh -= p.G;
                src += wrap;
            }
        }
    };
    // the first item came with the range for what starts at once (its queries and pages); all arrive by a bulk copy
    // that the first use waits for
    const int nw = min(w1 - w0, NWORK);
    if (tid == 160 && nw > 0) {
        ft::mbar_arrive_expect_tx(&w_full, nw * (uint32_t)sizeof(AttnWork));
        ft::bulk_g2s(s_work, p.works + w0, nw * (uint32_t)sizeof(AttnWork), &w_full);
    }
    auto work = [&](int w) -> AttnWork { return w - w0 < NWORK ? s_work[w - w0] : p.works[w]; };

    if (wid >= 4) {
        if (C::CTAS == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
        if (wid == 4 || wid == 6) {
        // ---------------------------------------------------- TMA warps: keys, values
        const int kv = wid == 4 ? 0 : 1, NST = kv ? NV : NK;
        uint64_t *full = kv ? v_full : k_full, *empty = kv ? v_empty : k_empty;
        unsigned char* ring = kv ? ring_v : ring_k;
        constexpr int NB = D / 64, H = C::HALVES;            // blocks of 64 values across a row
        const int rows = min(p.page, 64), nsub = ATTN_BN / rows;  // a box is 64 values of a page's rows, at most 64
        const int oob = p.n_pages * p.L * 2 * p.Hkv;         // a box past the map's end reads zeros
        // lane i < nsub reads the page of the tile's i-th run of rows, two tiles ahead, across items; it is looked at
        // only when a box of it is issued
        constexpr int NONE = 0x7fffffff;                     // no key of the item there: reads zeros
        int st = 0, n = 0, rw = w0, ri = 0;  // st, par: next stage, parity of its phase; n stages issued
        uint32_t par = 0;
        bool ok = true;
        AttnWork kr = mine0.first;
        auto read = [&]() {
            if (rw < w1 && ri == kr.ntile) {                 // the next item, if there is one
                ri = 0;
                if (++rw < w1) kr = work(rw);
            }
            if (rw >= w1) return NONE;
            const int pos = kr.pos0 + ri * ATTN_BN + lane * rows;
            ++ri;
            return lane >= nsub || pos >= kr.kend ? NONE : p.table[(size_t)kr.trow * p.row_pages + (pos >> p.page_log)];
        };
        // the first tile's pages need the first item only: they are read while the items are still on their way
        int cur = read();
        if (nw > 0) ok = __all_sync(0xffffffffu, ft::mbar_wait(&w_full, 0, p.err));
        int next = ok ? read() : NONE;
        for (int w = w0; w < w1 && ok && !__any_sync(0xffffffffu, s_fail); ++w) {
            const AttnWork k = work(w);
            // one stage: boxes of runs [sub0, sub0 + ns) by blocks [blk0, blk0 + nb), a block `bytes` after the other
            auto stage = [&](int id, int sub0, int ns, int blk0, int nb, uint32_t bytes) {
                // (a new barrier passes for the phase before its first)
                if (!__all_sync(0xffffffffu, ft::mbar_wait(&empty[st], par ^ 1u, p.err))) {
                    ok = false;
                    return;
                }
                if (lane == 0) ft::mbar_arrive_expect_tx(&full[st], C::STAGE);
                const int sub = lane / nb, blk = lane % nb, mine = __shfl_sync(0xffffffffu, id, sub0 + sub);
                if (sub < ns) {
                    int z = oob;
                    if ((unsigned)mine < (unsigned)p.n_pages)
                        z = ((mine * p.L + p.layer) * 2 + kv) * p.Hkv + k.head;
                    else if (mine != NONE)
                        atomicOr(p.err, FT_DEVERR_ARG);
                    tc::tma_load_3d(ring + (size_t)st * C::STAGE + blk * bytes + sub * rows * 128, &map, (blk0 + blk) * 64,
                                    ((sub0 + sub) * rows) & (p.page - 1), z, &full[st]);
                }
                ++n;
                if (++st == NST) {
                    st = 0;
                    par ^= 1u;
                }
            };
            for (int i = 0; i < k.ntile && ok; ++i) {
                const int next2 = read();
                if (kv == 0) {
                    for (int h = 0; h < H && ok; ++h) stage(cur, 0, nsub, h * (NB / H), NB / H, ATTN_BN * 128);
                } else {  // an upper half without keys is left out
                    const int halves = H == 2 && k.kend - (k.pos0 + i * ATTN_BN) <= 64 ? 1 : H;
                    for (int h = 0; h < halves && ok; ++h) stage(cur, h * (nsub / H), nsub / H, 0, NB, ATTN_BN / H * 128);
                }
                cur = next;
                next = next2;
            }
        }
        if (!ok) s_fail = 1;
        for (int j = max(0, n - NST); j < n; ++j)  // nothing in flight into shared memory at exit
            ft::mbar_wait(&full[j % NST], (j / NST) & 1, p.err);
    } else if (wid == 5) {
        // ------------------------------------------------------------ MMA warp
        {
            constexpr uint32_t id_s = idesc_of(BF, ATTN_BN, false, false), id_o = idesc_of(BF, D, false, true);
            constexpr uint32_t id_st = idesc_of(BF, NQ, false, false), id_ot = idesc_of(BF, NQ, true, false);
            constexpr int H = C::HALVES;
            const uint32_t pdesc = desc_k(smP), kdesc = desc_k(ring_k), vdesc = desc_v(ring_v, ATTN_BN / H * 128), qdesc = desc_k(smQ);
            constexpr uint32_t SW = C::STAGE / 16, QW = (D / 64) / H * (ATTN_BM * 128 / 16);
            int g = 0, n = 0;
            Slot rk, rv;
            bool ok = true;
            auto wait = [&](uint64_t* b, uint32_t phase) {
                if (!__all_sync(0xffffffffu, ft::mbar_wait(b, phase & 1u, p.err))) ok = false;
            };
            Slot sc;  // score buffer of the next tile
            auto release_v = [&]() {
                mma_commit(&v_empty[rv.st]);
                advance<NV>(rv);
            };
            int sb = 0;
            // an item; the two forms have loops of their own, so that neither's operands are selected at run time
            auto item = [&](const AttnWork& k, auto form) {
                constexpr bool few = decltype(form)::value;
                const int nt = k.ntile, keys = k.kend - k.pos0;
                auto scores = [&]() {  // S = Q K^T, or S^T = K Q^T, with the next tile of the ring
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        wait(&k_full[rk.st], rk.ph);
                        tc::fence_after_sync();
                        const uint32_t s = tmem + (uint32_t)(D + sc.st * ATTN_BN), kd = kdesc + rk.st * SW, qd = qdesc + h * QW;
                        mma_scores<(D / 64) / H>(s, few ? kd : qd, few ? qd : kd, few ? id_st : id_s, h ? 1u : 0u);
                        if (h == H - 1) mma_commit(&s_full[sc.st]);
                        mma_commit(&k_empty[rk.st]);
                        advance<NK>(rk);
                    }
                    advance<NS>(sc);
                };
                auto values = [&](int half, uint32_t v, uint32_t accumulate) {
                    if (few) {
#pragma unroll
                        for (int d = 0; d < D; d += 128)
                            mma_values_t(tmem + (uint32_t)(d / 128 * NQ), v + d / 64 * (ATTN_BN / H * 128 / 16),
                                         pdesc + (uint32_t)(sb * 256 + half * 128), id_ot, accumulate);
                    } else {
                        mma_values(tmem, tmem + (uint32_t)(D + sb * ATTN_BN + 32 * half), v, id_o, accumulate);
                    }
                };
                wait(&q_full, n);
                scores();
                for (int i = 0; i < nt && ok; ++i, ++g) {
                    if (NS == 2 && i + 1 < nt) scores();
                    if (i == 0 && n > 0) wait(&o_empty, n - 1);
                    wait(&v_full[rv.st], rv.ph);
                    wait(&p_full[sb], g / NS);
                    tc::fence_after_sync();
                    values(0, vdesc + rv.st * SW, i ? 1u : 0u);
                    if (keys - i * ATTN_BN > 64) {
                        if (H == 2) {
                            release_v();
                            wait(&v_full[rv.st], rv.ph);
                            tc::fence_after_sync();
                        }
                        values(1, vdesc + rv.st * SW + (H == 2 ? 0 : 512), 1u);
                    }
                    release_v();
                    if (NS == 2) mma_commit(&pv_done[g & 1]);
                    if (i == nt - 1) mma_commit(&o_full);
                    if (NS == 2) sb ^= 1;
                    if (NS == 1 && i + 1 < nt) scores();
                }
            };
            if (nw > 0) wait(&w_full, 0);
            for (int w = w0; w < w1 && ok && !__any_sync(0xffffffffu, s_fail); ++w, ++n) {
                const AttnWork k = work(w);
                if (FEW && k.nrows <= NQ)
                    item(k, std::true_type());
                else
                    item(k, std::false_type());
            }
            if (!ok) s_fail = 1;
            mma_commit(&done);
            ft::mbar_wait(&done, 0, p.err);
        }
        }
    } else {
        if (C::CTAS == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
        // ------------------------------------------------------- softmax warps
        constexpr int H = C::HALVES;
        const int r = tid;  // row of the item: TMEM lane
        const uint32_t lane_base = tmem + ((uint32_t)(wid * 32) << 16);
        auto publish_q = [&]() {
            ft::cp_async_wait_all();
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) ft::mbar_arrive(&q_full);
        };
        // the whole warp goes on or gives up: what follows a wait is executed by all its lanes together
        auto wait = [&](uint64_t* b, int ph) {
            return __all_sync(0xffffffffu, ft::mbar_wait(b, (uint32_t)ph & 1u, p.err));
        };
        int g = 0, it0 = 0, n = 0;
        bool ok = true;
        // what the pool holds past the keys of a tile may be anything: its weights are 0, its values are made 0
        auto clear_values = [&](int valid, int i) {
            if (valid >= ATTN_BN || (H == 2 && valid == 64)) return;
            const bool two = valid > 64;
            const int vit = it0 + H * i + (H == 2 && two), st = vit % NV;
            if (!wait(&v_full[st], vit / NV)) ok = false;
            unsigned char* vt = ring_v + (size_t)st * C::STAGE;
            // rows of this stage (of 64 keys, or of the whole tile) that hold no key
            const int z0 = max(H == 2 && two ? valid - 64 : valid, 0), nz = ((H == 1 && two ? ATTN_BN : 64) - z0) * 8;
            for (int x = tid; x < nz * (D / 64); x += 128) {
                const int b = x / nz, y = x % nz;
                *reinterpret_cast<uint4*>(vt + b * (ATTN_BN / H * 128) + z0 * 128 + y * 16) = make_uint4(0, 0, 0, 0);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        };
        auto next_item = [&](const AttnWork& k) {
            it0 += H * k.ntile - (H == 2 && k.kend - (k.pos0 + (k.ntile - 1) * ATTN_BN) <= 64);
        };
        // The transposed form, for few rows: a thread has a key, its scores with all the queries, their weights on
        // a reference of each query that the four warps agree on, as long as no weight on it is larger than MAX_SUM: the
        // score of the item's first key or, in f16, whose weights have room for less, the largest of the first 32 (64
        // requests of up to 512 keys 14.2 us; with the first key's 15.1).
        auto few_rows = [&](const AttnWork& k, int w) {
            int t = r;
            asm volatile("" : "+r"(t));  // what follows from t stays in here: the other form needs the registers
            float ref[NQ], l[NQ], x[NQ];  // reference of the weights (0: no key seen yet), sums of this thread's keys
#pragma unroll
            for (int j = 0; j < NQ; ++j) l[j] = ref[j] = 0.f;
            const uint32_t rows = (1u << k.nrows) - 1;
            const bool more = w + 1 < w1;
            unsigned unseen = 0;  // queries whose first key scored -inf
            bool held = false;    // the next item's queries have to wait for the last product: they lie over its weights
            for (int i = 0; i < k.ntile; ++i, ++g) {
                if (!wait(&s_full[g % NS], g / NS)) ok = false;
                tc::fence_after_sync();
                tmem_ld16(lane_base + (uint32_t)(D + (g % NS) * ATTN_BN), reinterpret_cast<uint32_t*>(x));
                if (i == k.ntile - 1 && more) {
                    held = work(w + 1).nrows > 64;
                    if (!held) load_q(work(w + 1));
                }
                const int pos = k.pos0 + i * ATTN_BN + t;
                // the queries that see this key: all but those of tokens that it is behind
                const int past = k.vis0 == ATTN_NOMASK ? 0 : pos - k.vis0 + 1;
                const uint32_t vis = pos >= k.kend ? 0u : past <= 0 ? rows : rows & (0xffffffffu << min(max(past * p.G - k.r0, 0), 31));
                if (i == 0) {
                    if constexpr (BF) {
                        if (t == 0) {
#pragma unroll
                            for (int j = 0; j < NQ; ++j) s_red[j >> 2][j & 3] = vis >> j & 1 ? x[j] * p.c : 0.f;
                        }
                    } else if (wid == 0) {
                        float y[NQ];
#pragma unroll
                        for (int j = 0; j < NQ; ++j) y[j] = vis >> j & 1 ? x[j] * p.c : -INFINITY;
                        const float m0 = warp_columns(y, t, [](float a, float b) { return fmaxf(a, b); });
                        if (!(t & 1)) s_red[t >> 3][(t >> 1) & 3] = m0 - SHIFT<BF>;
                    }
                    if (any_of_128(!ok)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int j = 0; j < NQ; j += 4) *reinterpret_cast<float4*>(ref + j) = *reinterpret_cast<const float4*>(s_red[j >> 2]);
#pragma unroll
                    for (int j = 0; j < NQ; ++j) {
                        if (ref[j] == -INFINITY) {
                            unseen |= 1u << j;
                            ref[j] = 0.f;
                        }
                    }
                }
                float e[NQ], top = 0.f;
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    const float y = ex2(fmaf(x[j], p.c, -ref[j]));
                    e[j] = vis >> j & 1 ? y : 0.f;
                    top = fmaxf(top, e[j]);
                }
                if (any_of_128(top > MAX_SUM<BF> || (unseen & vis) || !ok)) {
                    // the maxima of the queries over the tile
                    float y[NQ];
#pragma unroll
                    for (int j = 0; j < NQ; ++j) y[j] = x[j] = vis >> j & 1 ? x[j] * p.c : -INFINITY;
                    const float m1 = warp_columns(y, t & 31, [](float a, float b) { return fmaxf(a, b); });
                    if (!(t & 1)) s_red[(t & 31) >> 1][wid] = m1;
                    if (any_of_128(!ok)) {
                        ok = false;
                        break;
                    }
                    if (i > 0) {
                        if (NS == 2 && !wait(&pv_done[(g - 1) & 1], (g - 1) >> 1)) ok = false;
                        tc::fence_after_sync();
                    }
#pragma unroll
                    for (int j = 0; j < NQ; ++j) {
                        const float4 m4 = *reinterpret_cast<const float4*>(s_red[j]);
                        const float m = max3(fmaxf(m4.x, m4.y), m4.z, m4.w) - SHIFT<BF>;
                        const bool first = unseen >> j & 1;
                        if (m != -INFINITY) unseen &= ~(1u << j);
                        const float now = first ? (m == -INFINITY ? 0.f : m) : fmaxf(m, ref[j]);
                        y[j] = first ? 1.f : ex2(ref[j] - now);
                        ref[j] = now;
                        l[j] *= y[j];
                        e[j] = ex2(x[j] - now);
                    }
                    any_of_128(false);  // s_red is read
                    if (i > 0) {
#pragma unroll
                        for (int d = 0; d < D; d += 128) {
                            uint32_t o[NQ];
                            tmem_ld16(lane_base + (uint32_t)(d / 128 * NQ), o);
#pragma unroll
                            for (int j = 0; j < NQ; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * y[j]);
                            tmem_st16(lane_base + (uint32_t)(d / 128 * NQ), o);
                        }
                        tmem_wait_st();
                    }
                }
                // P^T: 16 rows of 64 keys, 128 bytes each with the swizzle, a half of the tile after the other
                const uint32_t pt = ft::smem_addr(smP) + (g % NS) * 4096 + (t >> 6) * 2048 + (t & 63) * 2;
#pragma unroll
                for (int j = 0; j < NQ; j += 2) {
                    const uint32_t v = pack2<BF>(e[j], e[j + 1]);
                    l[j] += e[j];
                    l[j + 1] += e[j + 1];
                    st_shared16((pt ^ ((j & 7) << 4)) + j * 128, v);
                    st_shared16((pt ^ (((j + 1) & 7) << 4)) + (j + 1) * 128, v >> 16);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                clear_values(k.kend - (pos - t), i);
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) ft::mbar_arrive(&p_full[g % NS]);
            }
            if (more && !held) publish_q();
            const float sum1 = warp_columns(l, t & 31, [](float a, float b) { return a + b; });
            if (!(t & 1)) s_red[(t & 31) >> 1][wid] = sum1;
            if (any_of_128(!ok)) {
                ok = false;
                return;
            }
            if (!wait(&o_full, n)) {
                ok = false;
                return;
            }
            tc::fence_after_sync();
            if (more && held) {
                load_q(work(w + 1));
                publish_q();
            }
            const float4 s4 = *reinterpret_cast<const float4*>(s_red[t & 15]);
            const float sum = (s4.x + s4.y) + (s4.z + s4.w);  // of query lane % 16
            const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
#pragma unroll
            for (int d = 0; d < D; d += 128) {
                tmem_ld16(lane_base + (uint32_t)(d / 128 * NQ), reinterpret_cast<uint32_t*>(x));
                if (k.prow < 0) {
                    int gh = k.r0 % p.G;
                    uint16_t* dst = p.out + (long long)(k.tok0 + k.r0 / p.G) * p.ld_o + (k.head * p.G + gh) * D + d + t;
#pragma unroll
                    for (int j = 0; j < NQ; ++j) {
                        const float f = __shfl_sync(0xffffffffu, inv, j);
                        if (j < k.nrows) *dst = (uint16_t)pack2<BF>(x[j] * f, 0.f);
                        dst += D;
                        if (++gh == p.G) {
                            gh = 0;
                            dst += p.ld_o - p.G * D;
                        }
                    }
                } else {
                    float* dst = p.part_o + (size_t)k.prow * D + part_column(d + t);
#pragma unroll
                    for (int j = 0; j < NQ; ++j)
                        if (j < k.nrows) dst[j * D] = x[j];
                }
            }
            if (k.prow >= 0) {
                float mine = ref[0];
#pragma unroll
                for (int j = 1; j < NQ; ++j) mine = t == j ? ref[j] : mine;
                if (t < k.nrows) p.part_ml[k.prow + t] = make_float2(sum == 0.f ? -INFINITY : mine, sum);
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) ft::mbar_arrive(&o_empty);
            next_item(k);
        };
        if (w0 < w1) {
            load_q(mine0.first);
            publish_q();
            ok = wait(&w_full, 0);
        }
        for (int w = w0; w < w1; ++w, ++n) {
            // the transposed form's barriers have no time limit: there the four warps go on or stop together
            if (FEW ? any_of_128(!ok || s_fail) : !ok || __any_sync(0xffffffffu, s_fail)) {
                ok = false;
                break;
            }
            const AttnWork k = work(w);
            if constexpr (FEW) {
                if (k.nrows <= NQ) {
                    few_rows(k, w);
                    continue;
                }
            }
            const bool rows_here = wid * 32 < k.nrows;
            const int tok = (k.r0 + min(r, k.nrows - 1)) / p.G;
            const int lim = min(k.kend, k.vis0 == ATTN_NOMASK ? k.kend : k.vis0 + tok);  // this row sees positions < lim
            float m = -INFINITY, l = 0.f;
            for (int i = 0; i < k.ntile; ++i, ++g) {
                if (!wait(&s_full[g % NS], g / NS)) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                const int pos = k.pos0 + i * ATTN_BN;
                if (i == k.ntile - 1 && w + 1 < w1) load_q(work(w + 1));  // every product with this Q is done
                const int valid = k.kend - pos;
                const bool two = valid > 64;  // keys in the upper half
                const uint32_t sa = lane_base + (uint32_t)(D + (g % NS) * ATTN_BN);
                uint32_t s[ATTN_BN];  // scores, then (in the first half of each half) the weights in the cache's type
                float* f = reinterpret_cast<float*>(s);
                const uint64_t c2 = f2(p.c, p.c);
                float mc = 0.f, lt = 0.f;
                auto load = [&](int h) {
                    tc::tmem_ld32(sa + 64 * h, s + 64 * h);
                    tc::tmem_ld32(sa + 64 * h + 32, s + 64 * h + 32);
                };
                auto loaded = [&](int h) {  // ... and masked
                    tc::tmem_wait_ld(s + 64 * h);
                    tc::tmem_wait_ld(s + 64 * h + 32);
                    const int left = lim - (pos + 64 * h);
                    if (left < 64) {
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            if (j >= left) f[64 * h + j] = -INFINITY;
                    }
                };
                // weights of 64 keys on the reference mc; returns their sum.  The weights go to the product in the
                // cache's own type; l keeps their fp32 values.
                auto weights = [&](int h) {
                    const uint64_t mc2 = f2(-mc, -mc);
                    uint64_t l4[4] = {0, 0, 0, 0};  // pairs of sums
#pragma unroll
                    for (int j = 0; j < 64; j += 2) {
                        float2 e = unf2(fma2(f2(f[64 * h + j], f[64 * h + j + 1]), c2, mc2));
                        e.x = ex2(e.x);
                        e.y = ex2(e.y);
                        l4[(j >> 1) & 3] = add2(l4[(j >> 1) & 3], f2(e.x, e.y));
                        s[64 * h + (j >> 1)] = pack2<BF>(e.x, e.y);
                    }
                    const float2 ls = unf2(add2(add2(l4[0], l4[1]), add2(l4[2], l4[3])));
                    return ls.x + ls.y;
                };
                auto reference = [&]() { mc = m == -INFINITY ? 0.f : m * p.c - SHIFT<BF>; };  // -inf: a row that has seen no key yet
                if (rows_here) {
                    load(0);
                    bool exact = i == 0;
                    if (!exact) {
                        // the reference of the tiles before is almost always good enough; whether it is, the sum tells
                        reference();
                        loaded(0);
                        if (two) load(1);
                        lt = weights(0);
                        if (two) {
                            loaded(1);
                            lt += weights(1);
                        }
                        // (lanes past the rows hold anything)
                        exact = __any_sync(0xffffffffu, r < k.nrows && (lt > MAX_SUM<BF> || m == -INFINITY));
                        if (exact) load(0);
                    }
                    if (exact) {
                        if (two) load(1);
                        loaded(0);
                        float mx[4] = {m, m, m, m};  // four chains
#pragma unroll
                        for (int j = 0; j < 64; j += 2) mx[(j >> 1) & 3] = max3(mx[(j >> 1) & 3], f[j], f[j + 1]);
                        if (two) {
                            loaded(1);
#pragma unroll
                            for (int j = 64; j < ATTN_BN; j += 2) mx[(j >> 1) & 3] = max3(mx[(j >> 1) & 3], f[j], f[j + 1]);
                        }
                        const float mn = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
                        if (i == 0) {
                            m = mn;
                        } else {
                            const bool lag = r < k.nrows && (lt > MAX_SUM<BF> || m == -INFINITY) && mn > m;
                            // with one S the scores' own barrier has told that the product before them is done
                            if (NS == 2 && !wait(&pv_done[(g - 1) & 1], (g - 1) >> 1)) ok = false;
                            tc::fence_after_sync();
                            const float fac = lag ? ex2((m - mn) * p.c) : 1.f;
                            l *= fac;
                            if (lag) m = mn;
#pragma unroll 1
                            for (int cc = 0; cc < D; cc += 32) {
                                uint32_t o[32];
                                tc::tmem_ld32(lane_base + (uint32_t)cc, o);
                                tc::tmem_wait_ld(o);
#pragma unroll
                                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * fac);
                                tmem_st32(lane_base + (uint32_t)cc, o);
                            }
                        }
                        reference();
                        lt = weights(0);
                        if (two) lt += weights(1);
                    }
                    l += lt;
                    tmem_st32(sa, s);
                    if (two) tmem_st32(sa + 32, s + 64);
                }
                clear_values(valid, i);
                if (rows_here) tmem_wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) ft::mbar_arrive(&p_full[g % NS]);
            }
            if (!ok) continue;
            if (w + 1 < w1) publish_q();
            if (!wait(&o_full, n)) {
                ok = false;
                continue;
            }
            tc::fence_after_sync();
            if (rows_here) {
                const bool in = r < k.nrows;
                const int R = k.r0 + min(r, k.nrows - 1);
                if (k.prow < 0) {
                    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // no key seen: zeros; NaN stays
                    uint16_t* dst = p.out + (long long)(k.tok0 + R / p.G) * p.ld_o + (k.head * p.G + R % p.G) * D;
                    const bool wide = (uintptr_t)dst % 32 == 0;
#pragma unroll
                    for (int cc = 0; cc < D; cc += 32) {
                        uint32_t o[32], v[16];
                        tc::tmem_ld32(lane_base + (uint32_t)cc, o);
                        tc::tmem_wait_ld(o);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            v[j] = pack2<BF>(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
                        if (in && wide) {
                            st_global32(dst + cc, v);
                            st_global32(dst + cc + 16, v + 8);
                        } else if (in) {
#pragma unroll
                            for (int j = 0; j < 16; j += 4)
                                *reinterpret_cast<uint4*>(dst + cc + 2 * j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                        }
                    }
                } else {
                    const int r4 = wid * 32 + (lane >> 2);
                    float* dst = p.part_o + (size_t)(k.prow + r4) * D + (lane & 3) * 8;
#pragma unroll
                    for (int cc = 0; cc < D; cc += 32) {
                        uint32_t o[32];
                        tmem_ld_quads(lane_base + (uint32_t)cc, o);
                        tmem_ld_quads(lane_base + (uint32_t)(cc + (16 << 16)), o + 16);
                        tc::tmem_wait_ld(o);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {  // rows r4, + 8, + 16, + 24
                            const uint32_t* s = o + (j >> 1) * 16 + (j & 1) * 2;
                            const uint32_t v[8] = {s[0], s[1], s[4], s[5], s[8], s[9], s[12], s[13]};
                            if (r4 + 8 * j < k.nrows) st_global32(dst + cc + (size_t)(8 * j) * D, v);
                        }
                    }
                    if (in) p.part_ml[k.prow + r] = make_float2(m * p.c - SHIFT<BF>, l);
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) ft::mbar_arrive(&o_empty);
            next_item(k);
        }
        if (!ok) s_fail = 1;
        ft::cp_async_wait_all();
    }
    tc::fence_before_sync();
    __syncthreads();
    if (wid == 5) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, C::TCOLS);
    }
}

// ------------------------------------------------------------------ the plan

constexpr int PT = ATTN_MAX_B;  // threads: one per request

constexpr int CHOICES = PT / 32;  // chunk sizes that are looked at, one a warp
constexpr int CUM = 2048;       // segments whose running cost is kept in shared memory

struct PlanArgs {
    AttnPlan pl;
    int B, T, n_groups, G, Hkv, page, n_rows, row_pages, merge_nb, merge_warps, per_sm;
    const int *cu_q, *rows, *group_start, *group_tokens, *lens, *table;
    unsigned* err;
};

// What the plan kernel keeps of a segment.
struct SegRec {
    int b, r0, nrows, ntile, kend;
    attnline::cost_t cum;  // cost of the segments before it
};

__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

__device__ __forceinline__ int block_max(int v, int (&ws)[32]) {
    v = __reduce_max_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) ws[threadIdx.x >> 5] = v;
    __syncthreads();
    v = __reduce_max_sync(0xffffffffu, ws[threadIdx.x & 31]);
    __syncthreads();
    return v;
}

// Lowers cut[g] to the tokens of the whole pages that the rows of group g share, of the claim[g] that are claimed: a warp
// compares 256 pages of a request with those of the group's first at a time.  Bound by what one SM reads from L2 once
// there are many rows, by latency else: 64 requests of 128 claimed pages 1.8 us, 6 of 1024 1.3, 130 of 512 6.0 (7.1 page
// by page, which is left for rows that do not start on 16 bytes; with the loads of two requests under way 6.8).
template <class V>
__device__ __forceinline__ void cut_claims(const PlanArgs& p, int most, const int* group, const int* row, const int* first,
                                           const int* claim, int* cut) {
    constexpr int W = sizeof(V) / 4, N = 8 / W;
    const int lane = threadIdx.x & 31, plog = __ffs(p.page) - 1;
    for (int u = threadIdx.x >> 5; u < p.B * cdiv(most, 256); u += PT / 32) {
        const int b = u % p.B, g = group[b], j0 = u / p.B * 256 + lane * W;
        if (g < 0 || b == first[g]) continue;
        const int pages = claim[g] >> plog;
        const int *mine = p.table + (size_t)row[b] * p.row_pages, *ref = p.table + (size_t)row[first[g]] * p.row_pages;
        V x[N], y[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int j = j0 + i * 32 * W;
            if (j < pages) {
                x[i] = *reinterpret_cast<const V*>(mine + j);
                y[i] = *reinterpret_cast<const V*>(ref + j);
            }
        }
        int bad = INT_MAX;
#pragma unroll
        for (int i = N - 1; i >= 0; --i) {
            const int j = j0 + i * 32 * W;
#pragma unroll
            for (int k = W - 1; k >= 0; --k)
                if (j + k < pages && reinterpret_cast<const int*>(&x[i])[k] != reinterpret_cast<const int*>(&y[i])[k]) bad = j + k;
        }
        bad = __reduce_min_sync(0xffffffffu, bad);
        if (lane == 0 && bad != INT_MAX) atomicMin(&cut[g], bad << plog);
    }
}

__global__ void __launch_bounds__(PT) attn_plan_kernel(const PlanArgs p) {
    __shared__ int s_n[PT], s_len[PT], s_row[PT], s_P[PT], s_pre[PT], s_sb[PT];  // per request
    __shared__ int g_min[PT], g_rows[PT], g_solo[PT], g_first[PT];               // per group
    __shared__ int q_g[PT / 2], q_off[PT / 2];  // per group taken together (it has two requests at least)
    __shared__ int ws[32];
    __shared__ attnline::cost_t wl[32];
    __shared__ long long s_end[CHOICES];  // per choice of the chunk: what it costs
    __shared__ int s_c[CHOICES], s_iph;
    extern __shared__ __align__(16) attnline::cost_t s_cum[];      // [CUM]
    int4* s_cta = reinterpret_cast<int4*>(s_cum + CUM);            // [n_cta] first item, first and last segment
    ft::grid_dep_launch();
    ft::grid_dep_wait();
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int B = p.B, G = p.G, n_cta = p.pl.n_cta;
    SegRec* seg = reinterpret_cast<SegRec*>(p.pl.seg);

    // ---- requests and groups
    bool ok = true;
    int n = 0, len = 0, row = 0, gi = -1;
    if (tid < B) {
        const int a = p.cu_q[tid], e = p.cu_q[tid + 1];
        n = e - a;
        row = p.rows ? p.rows[tid] : tid;
        if (a < 0 || e < a || e > p.T || (tid == 0 && a != 0) || row < 0 || row >= p.n_rows) ok = false;
        if (ok) {
            len = p.lens[row];
            if (len < 0 || len > (long long)p.row_pages * p.page) ok = false;
        }
    }
    if (tid < p.n_groups) {
        const int a = p.group_start[tid], e = p.group_start[tid + 1];
        if (a < 0 || e < a || e > B || p.group_tokens[tid] < 0) ok = false;
    }
    if (!__syncthreads_and(ok)) {
        if (tid == 0) {
            atomicOr(p.err, FT_DEVERR_ARG);
            *p.pl.hdr = AttnHdr{0, 0};
        }
        for (int i = tid; i < n_cta; i += PT) p.pl.ctas[i].w0 = p.pl.ctas[i].w1 = 0;
        return;
    }
    g_min[tid] = 0x7fffffff;
    g_rows[tid] = 0;
    g_solo[tid] = 0;
    g_first[tid] = 0x7fffffff;
    s_n[tid] = n;
    s_len[tid] = len;
    s_row[tid] = row;
    __syncthreads();
    if (tid < B && n > 0 && p.n_groups > 0) {
        if (p.group_start[0] <= tid) {
            gi = upper(p.n_groups, tid, [&](int i) { return p.group_start[i]; });
            if (tid >= p.group_start[gi + 1]) gi = -1;
        }
        if (gi >= 0) {
            atomicMin(&g_min[gi], max(0, len - n));
            atomicAdd(&g_rows[gi], n * G);
            atomicAdd(&g_solo[gi], cdiv(n * G, ATTN_BM));
            atomicMin(&g_first[gi], tid);
        }
    }
    __syncthreads();
    // a group's shared tokens: whole pages before every query; taken together only where that saves at
    // least a fifth of the row tiles that run over them (else the join costs more than it saves)
    int P = 0;
    if (tid < p.n_groups && g_rows[tid] > 0) {
        P = min(p.group_tokens[tid], g_min[tid]) / p.page * p.page;
        if (5 * cdiv(g_rows[tid], ATTN_BM) > 4 * g_solo[tid]) P = 0;
    }
    // ... and cut to the pages that all its rows really share
    g_min[tid] = g_solo[tid] = P;
    s_pre[tid] = gi;
    const int most = __syncthreads_or(P) ? block_max(P / p.page, ws) : 0;
    if (p.row_pages % 4 == 0 && (uintptr_t)p.table % 16 == 0)
        cut_claims<int4>(p, most, s_pre, s_row, g_first, g_min, g_solo);
    else
        cut_claims<int>(p, most, s_pre, s_row, g_first, g_min, g_solo);
    __syncthreads();
    P = g_solo[tid];
    int n_pre;
    const int my_pre = ft::block_scan(P > 0 ? 1 : 0, ws, n_pre);
    g_min[tid] = P;  // from here on: the shared tokens taken
    if (P > 0) q_g[my_pre] = tid;
    g_solo[tid] = my_pre;
    __syncthreads();
    s_P[tid] = gi >= 0 ? g_min[gi] : 0;
    s_pre[tid] = gi >= 0 && g_min[gi] > 0 ? g_solo[gi] : -1;

    // ---- chunks of the shared ranges: of up to four rounds over the CTAs, the one that ends first
    int n_seg;
    const int my_segs = cdiv(n * G, ATTN_BM);
    s_sb[tid] = ft::block_scan(my_segs, ws, n_seg);
    __syncthreads();
    attnline::cost_t cost = 0;
    for (int base = 0; base < n_seg; base += PT) {
        const int s = base + tid;
        SegRec r{};
        if (s < n_seg) {
            r.b = upper(B, s, [&](int i) { return s_sb[i]; });
            // requests without queries share the next one's start: upper() takes the last of them,
            // which is the one that has rows
            r.r0 = (s - s_sb[r.b]) * ATTN_BM;
            r.nrows = min(ATTN_BM, s_n[r.b] * G - r.r0);
            const int last = (r.r0 + r.nrows - 1) / G;
            r.kend = max(0, min(s_len[r.b], s_len[r.b] - s_n[r.b] + 1 + last));
            r.ntile = max(1, cdiv(r.kend - s_P[r.b], ATTN_BN));
        }
        attnline::cost_t total;
        r.cum = cost + ft::block_scan(s < n_seg ? attnline::segment_cost(r.ntile) : 0, wl, total);
        if (s < n_seg) {
            seg[s] = r;
            if (s < CUM) s_cum[s] = r.cum;
        }
        cost += total;
    }
    const long long S = cost * p.Hkv;
    // Items for so many sixteenths of the CTAs, the rest left to the other work, up to four rounds over all of them: a
    // warp looks at each choice.  What it costs, in eighths of a tile's time: the end of an even share or of the longest
    // chain of prefix items (1.3 times that where an SM has two such CTAs), and the join, 20000 pieces of a row in a
    // tile's time.  Against the five choices 1/4, 1/2, 1, 2, 4 by the end alone: 64 requests behind 8192 keys 28.1 ->
    // 26.6 us, with 64 keys of their own at head size 256 22.3 -> 20.5, 130 behind 16384 58.0 -> 56.4, 65 of one head a
    // row 38.4 -> 36.6; the worst of 24 others 256 behind 8192 at 256, 45.5 -> 47.7.
    if (n_pre > 0) {
        int rts = 0, mt = 1;
        for (int i = lane; i < n_pre; i += 32) {
            rts += cdiv(g_rows[q_g[i]], ATTN_BM);
            mt = max(mt, cdiv(g_min[q_g[i]], ATTN_BN));
        }
        rts = __reduce_add_sync(0xffffffffu, rts);
        mt = __reduce_max_sync(0xffffffffu, mt);
        auto total = [&](int c, auto rows) {  // of the row tiles, or the rows, times the chunks that they run over
            int x = 0;
            for (int i = lane; i < n_pre; i += 32) x += rows(g_rows[q_g[i]]) * cdiv(cdiv(g_min[q_g[i]], ATTN_BN), c);
            return (int)__reduce_add_sync(0xffffffffu, x) * p.Hkv;
        };
        auto items = [&](int c) { return total(c, [](int r) { return cdiv(r, ATTN_BM); }); };
        {
            const int k = wid, cap = max((k < 16 ? k + 1 : 16 + 3 * (k - 15)) * n_cta / 16, rts * p.Hkv);
            int lo = 1, hi = mt;  // smallest c with items(c) <= cap
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (items(mid) <= cap) hi = mid; else lo = mid + 1;
            }
            const int ni = items(lo), pieces = total(lo, [](int r) { return r; });
            const long long each = lo + OVP, chain = 8 * cdiv(ni, n_cta) * each;
            const bool beside = p.per_sm == 2 && ni > n_cta / 2 * 17 / 16;
            if (lane == 0) {
                s_end[k] = max((S + ni * each) * 8 / n_cta, beside ? chain * 13 / 10 : chain) + pieces / 2500;
                s_c[k] = lo;
            }
        }
    }
    __syncthreads();
    int c = 1;
    if (n_pre > 0) {
        int best = 0;
        for (int i = 1; i < CHOICES; ++i)
            if (s_end[i] < s_end[best]) best = i;
        c = s_c[best];
    }
    {
        int x = 0;
        if (tid < n_pre) x = cdiv(g_rows[q_g[tid]], ATTN_BM) * cdiv(cdiv(g_min[q_g[tid]], ATTN_BN), c);
        int iph;
        const int off = ft::block_scan(x, ws, iph);
        if (tid < n_pre) q_off[tid] = off;
        if (tid == 0) s_iph = iph;
    }
    __syncthreads();
    const int iph = s_iph, n_items = iph * p.Hkv;

    // ---- parts of the line of tiles: CTAs with one prefix item more get less
    const attnline::Line line(cost, p.Hkv, n_seg, n_cta, n_items, c);
    const int k0 = line.k0, n1 = line.n1;
    auto cum_of = [&](int i) { return i < CUM ? s_cum[i] : seg[i].cum; };
    __syncthreads();  // seg is complete

    int n_works = 0;
    for (int base = 0; base < n_cta; base += PT) {
        const int i = base + tid;
        int cnt = 0;
        if (i < n_cta) {
            cnt = k0 + (i < n1 ? 1 : 0);
            const long long x0 = line.start_of(i), x1 = line.start_of(i + 1);
            if (x1 > x0) {
                const int l0 = line.at(x0, cum_of), l1 = line.at(x1 - 1, cum_of);
                cnt += attnline::Line::items(l0, l1, line.begin_of(l1, cum_of), x1);
                s_cta[i].y = l0;
                s_cta[i].z = l1;
            }
        }
        int total;
        const int at = n_works + ft::block_scan(cnt, ws, total);
        if (i < n_cta) {
            p.pl.ctas[i].w0 = s_cta[i].x = at;
            p.pl.ctas[i].w1 = at + cnt;
            s_cta[i].w = cnt;
        }
        n_works += total;
    }
    __syncthreads();
    // eight lanes per CTA write its items
    for (int i = tid >> 3; i < n_cta; i += PT / 8) {
        const int4 mine = s_cta[i];
        const int w0 = mine.x, k = k0 + (i < n1 ? 1 : 0), sl = tid & 7;
        // one CTA an SM: every other block of CTAs has its own keys' items first and the shared ones after, so that the
        // products of the one kind run beside the reads of the other (blocks, so that a shared chunk's row tiles still
        // run together): 130 requests behind 16384 keys 65.5 -> 62.8 us.  With two CTAs an SM it cost 4%
        const bool late = p.per_sm == 1 && (i >> 4 & 1);
        const int jp = late ? mine.w - k : 0, js = late ? 0 : k;
        auto put = [&](int j, const AttnWork& w) {
            p.pl.works[w0 + j] = w;
            if (j == 0) p.pl.ctas[i].first = w;
        };
        for (int j = sl; j < k; j += 8) {
            const int idx = j * n_cta + i, h = idx / iph, rem = idx % iph;
            const int q = upper(n_pre, rem, [&](int a) { return q_off[a]; });
            const int gg = q_g[q], nrt = cdiv(g_rows[gg], ATTN_BM), nt = cdiv(g_min[gg], ATTN_BN);
            const int nch = cdiv(nt, c), ch = (rem - q_off[q]) / nrt, rt = (rem - q_off[q]) % nrt;
            const int t0 = (int)((long long)ch * nt / nch), t1 = (int)((long long)(ch + 1) * nt / nch);
            AttnWork w;
            w.head = h;
            w.trow = s_row[g_first[gg]];
            w.pos0 = t0 * ATTN_BN;
            w.ntile = t1 - t0;
            w.kend = min(g_min[gg], t1 * ATTN_BN);
            w.vis0 = ATTN_NOMASK;
            w.tok0 = p.cu_q[p.group_start[gg]];
            w.r0 = rt * ATTN_BM;
            w.nrows = min(ATTN_BM, g_rows[gg] - w.r0);
            w.prow = idx * ATTN_BM;
            put(jp + j, w);
        }
        const long long x0 = line.start_of(i), x1 = line.start_of(i + 1);
        if (x1 <= x0) continue;
        const int l0 = mine.y, l1 = mine.z;
        for (int l = l0 + sl; l <= l1; l += 8) {
            const SegRec r = seg[l % n_seg];
            int t0, t1;
            attnline::Line::tiles(line.begin_of(l, cum_of), r.ntile, x0, x1, t0, t1);
            if (t0 >= t1) continue;  // (only ever the last one)
            AttnWork w;
            w.head = l / n_seg;
            w.trow = s_row[r.b];
            w.pos0 = s_P[r.b] + t0 * ATTN_BN;
            w.ntile = t1 - t0;
            w.kend = r.kend;
            w.vis0 = s_len[r.b] - s_n[r.b] + 1;
            w.tok0 = p.cu_q[r.b];
            w.r0 = r.r0;
            w.nrows = r.nrows;
            const bool whole = t0 == 0 && t1 == r.ntile;
            w.prow = whole && s_pre[r.b] < 0 ? -1
                     : t0 == 0 ? (int)(p.pl.b_row + (long long)w.head * p.T * G + (long long)w.tok0 * G + r.r0)
                               : (int)(p.pl.c_row + (long long)i * ATTN_BM);
            put(js + (l - l0), w);
        }
    }
    // ---- rows with more than one piece
    auto pieces_of = [&](int l, const SegRec& r, int& c0, int& c1) {  // the CTAs that have some of its tiles
        line.holders(line.begin_of(l, cum_of), r.ntile, c0, c1);
        return c0 != c1 || s_pre[r.b] >= 0;
    };
    int rows = 0;
    for (int l = tid; l < n_seg * p.Hkv; l += PT) {
        const SegRec r = seg[l % n_seg];
        int c0, c1;
        if (pieces_of(l, r, c0, c1)) rows += r.nrows;
    }
    ft::block_scan(rows, ws, rows);
    // several warps share a row's pieces as long as all warps run at once
    const int warps = max(1, p.merge_warps / max(1, rows));
    int n_merge = 0;
    for (int base = 0; base < n_seg * p.Hkv; base += PT) {
        const int l = base + tid;
        int cnt = 0, c0 = 0, c1 = 0;
        SegRec r{};
        AttnMerge m{};
        if (l < n_seg * p.Hkv) {
            r = seg[l % n_seg];
            const int q = s_pre[r.b];
            if (pieces_of(l, r, c0, c1)) {
                m.head = l / n_seg;
                m.tok0 = p.cu_q[r.b];
                m.brow = (int)(p.pl.b_row + (long long)m.head * p.T * G + (long long)m.tok0 * G + r.r0);
                m.c0 = c0 + 1;
                m.nc = c1 - c0;
                m.ptok0 = -1;
                m.pitem = m.pnrt = m.pnch = 0;
                if (q >= 0) {
                    const int gg = q_g[q];
                    m.ptok0 = p.cu_q[p.group_start[gg]];
                    m.pnrt = cdiv(g_rows[gg], ATTN_BM);
                    m.pnch = cdiv(cdiv(g_min[gg], ATTN_BN), c);
                    m.pitem = m.head * iph + q_off[q];
                }
                const int np = m.pnch + 1 + m.nc, most = min(warps, cdiv(np, p.merge_nb));
                m.wpr = most >= 8 ? 8 : most >= 4 ? 4 : most >= 2 ? 2 : 1;
                cnt = cdiv(r.nrows, 8 / m.wpr);
            }
        }
        int total;
        const int at = n_merge + ft::block_scan(cnt, ws, total);
        const int step = cnt ? 8 / m.wpr : 0, brow = m.brow;
        for (int j = 0; j < cnt; ++j) {
            m.r0 = r.r0 + j * step;
            m.nrows = min(step, r.nrows - j * step);
            m.brow = brow + j * step;
            p.pl.merges[at + j] = m;
        }
        n_merge += total;
    }
    if (tid == 0) *p.pl.hdr = AttnHdr{n_merge, n_works};
}

// -------------------------------------------------------------- host side

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The kernels of a head size and type.
struct Kernels {
    const void *attn, *attn_few, *merge;
    size_t smem;
};
template <int D, bool BF>
Kernels kernels() {
    return Kernels{(const void*)attn_kernel<D, BF, false>, (const void*)attn_kernel<D, BF, D != 64>,
                   (const void*)attn_merge_kernel<D, BF>, Cfg<D>::SMEM};
}
Kernels kernels_of(const ft_kv* kv) {
    const bool bf = kv->dtype == FT_KV_BF16;
    if (kv->D == 64) return bf ? kernels<64, true>() : kernels<64, false>();
    if (kv->D == 128) return bf ? kernels<128, true>() : kernels<128, false>();
    return bf ? kernels<256, true>() : kernels<256, false>();
}
size_t plan_smem(const ft_kv* kv) { return CUM * sizeof(attnline::cost_t) + (size_t)kv->plan.n_cta * 16; }

}  // namespace

void attn_plan_sizes(int Hq, int Hkv, int D, int T_max, int B_max, int num_sms, AttnPlan& p) {
    const int G = Hq / Hkv;
    const int rts = (int)(((long long)T_max * G + ATTN_BM - 1) / ATTN_BM);
    p.n_cta = num_sms * (D != 256 ? 2 : 1);
    p.cap_segs = rts + B_max;                          // a request's last tile may be short
    p.cap_items = 4 * p.n_cta + Hkv * (rts + B_max);   // four rounds, or a chunk for each row tile
    p.cap_works = p.cap_items + Hkv * p.cap_segs + p.n_cta;
    // a row each, a short last record of a segment, and what each CTA of the join reads first
    p.cap_merges = T_max * Hq + Hkv * p.cap_segs + 4 * num_sms;
    p.b_row = (long long)p.cap_items * ATTN_BM;
    p.c_row = p.b_row + (long long)T_max * Hq;  // (kv_api.cu refuses sizes whose rows pass 2^31)
    p.part_rows = p.c_row + (long long)p.n_cta * ATTN_BM;
}

size_t attn_seg_bytes(const AttnPlan& p) { return (size_t)p.cap_segs * sizeof(SegRec); }

// The pool as [n_pages*L*2*Hkv][page][D], read in boxes of 64 values by a
// page's rows (at most 64) with 128-byte swizzle.
bool attn_encode_map(ft_kv* kv) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
        return false;
    const cuuint64_t dims[3] = {(cuuint64_t)kv->D, (cuuint64_t)kv->page, (cuuint64_t)kv->n_pages * kv->L * 2 * kv->Hkv};
    const cuuint64_t strides[2] = {(cuuint64_t)kv->D * 2, (cuuint64_t)kv->D * 2 * kv->page};
    const cuuint32_t box[3] = {64, (cuuint32_t)(kv->page < 64 ? kv->page : 64), 1};
    const cuuint32_t es[3] = {1, 1, 1};
    return reinterpret_cast<EncodeTiledFn>(f)(
               &kv->map, kv->dtype == FT_KV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
               kv->pool, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t attn_setup(ft_kv* kv) {
    const Kernels k = kernels_of(kv);
    cudaError_t e = ensure_dynamic_smem(k.attn, k.smem);
    if (e == cudaSuccess) e = ensure_dynamic_smem(k.attn_few, k.smem);
    return e == cudaSuccess ? ensure_dynamic_smem((const void*)attn_plan_kernel, plan_smem(kv)) : e;
}

cudaError_t launch_attn_plan(ft_kv* kv, int B, int T, const int* cu_q, const int* rows, int n_groups,
                             const int* group_start, const int* group_tokens) {
    kv->few_rows = n_groups == 0 && (long long)T * (kv->Hq / kv->Hkv) <= (long long)NQ * B;
    PlanArgs a{kv->plan, B, T, n_groups, kv->Hq / kv->Hkv, kv->Hkv, kv->page, kv->n_rows, kv->row_pages,
               MERGE_NB(kv->D), kv->num_sms * 8 * MERGE_CTAS(kv->D), kv->plan.n_cta / kv->num_sms, cu_q, rows, group_start, group_tokens, kv->lens, kv->table, kv->err};
    void* args[] = {&a};
    return launch_dependent((const void*)attn_plan_kernel, 1, PT, plan_smem(kv), kv->stream, args);
}

cudaError_t launch_attn_forward(ft_kv* kv, int layer, const void* q, long long ld_q, void* out, long long ld_o,
                                float scale) {
    AttnArgs a{};
    a.works = kv->plan.works;
    a.hdr = kv->plan.hdr;
    a.ctas = kv->plan.ctas;
    a.merges = kv->plan.merges;
    a.c_row = kv->plan.c_row;
    a.q = static_cast<const uint16_t*>(q);
    a.ld_q = ld_q;
    a.out = static_cast<uint16_t*>(out);
    a.ld_o = ld_o;
    a.table = kv->table;
    a.row_pages = kv->row_pages; a.page = kv->page; a.page_log = __builtin_ctz(kv->page); a.n_pages = kv->n_pages; a.L = kv->L; a.Hkv = kv->Hkv;
    a.G = kv->Hq / kv->Hkv;
    a.layer = layer;
    a.c = scale * LOG2E;
    a.part_o = kv->part_o;
    a.part_ml = kv->part_ml;
    a.err = kv->err;
    const Kernels k = kernels_of(kv);
    void* args[] = {&kv->map, &a};
    const cudaError_t e = launch_dependent(kv->few_rows ? k.attn_few : k.attn, kv->plan.n_cta, G_THREADS, k.smem, kv->stream, args);
    return e == cudaSuccess ? launch_dependent(k.merge, kv->num_sms * 4, 256, 0, kv->stream, args + 1) : e;
}

// ft_block_norm: the norms before and after a block with its gate and the
// residual sum, in one pass.
//
//   z = a * rsqrt(mean(a^2) + eps) * w_post       (or z = a)
//   h = rs * r + bs * g * z
//   y = h * rsqrt(mean(h^2) + eps) * w_pre
//
// Bound: HBM for prompts (a and r are read, h and y written, once each; the
// weights stay in L2), latency for a few tokens.  A row lives in the registers
// of its threads, NV vectors of 8 values each, between the loads and the stores,
// so nothing is read twice.  Each CTA takes one row and ends: the loads of the
// CTAs that follow fill the gaps that its barriers leave, so registers (that is,
// CTAs an SM) decide.  Measured against that: CTAs that stay and ask for the next
// row's values a row ahead, 2 x 512 threads an SM, 96 us instead of 67.6 for 8192
// tokens of 4096; a gate of [T, H] held in registers from the start instead of
// brought into L2, 18.4 us instead of 17.9 for 4001 tokens of 2048.
//
// Measured (a stream of calls on buffers larger than L2): 8192 tokens of 4096 in
// fp32, out bf16, 67.6 us, 6.95 TB/s (the copy rate); 4001 of 2048 in f16 with
// both norms and a full gate 17.9 us, 4.6 TB/s; one token of 2048 1.8 us.
#include "ft_kv.cuh"
#include "../../include/ft_gen.h"

#include <cmath>
#include <cstdio>
#include <cstdlib>

namespace {

struct NormParams {
    int T, H, nvec;           // nvec = H / 8
    int tpr;                  // threads of a row: 32 (rows are warps) or the whole CTA
    int gate_kind, post_norm;
    int w32, g32;             // weights, gate are fp32
    const void *block, *gate, *resid, *pre, *post;
    void *resid_out, *out;
    long long ld_b, ld_g, ld_r, ld_ro, ld_o;
    float eps, rs, bs;
};

// 8 values in memory's form, and as fp32.
template <bool F32>
struct Raw {
    uint4 v[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ void load_raw(const void* p, long long i, Raw<F32>& r) {  // at element offset i
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + i * (F32 ? 4 : 2));
    r.v[0] = q[0];
    if (F32) r.v[F32 ? 1 : 0] = q[1];
}
template <bool F32, bool BF>
__device__ __forceinline__ void widen(const Raw<F32>& r, float* f) {
    if (F32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4& v = r.v[F32 ? h : 0];
            f[4 * h] = __uint_as_float(v.x);
            f[4 * h + 1] = __uint_as_float(v.y);
            f[4 * h + 2] = __uint_as_float(v.z);
            f[4 * h + 3] = __uint_as_float(v.w);
        }
    } else {
        const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (BF) {
                f[2 * k] = __uint_as_float(w[k] << 16);
                f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
            } else {
                const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
                f[2 * k] = t.x;
                f[2 * k + 1] = t.y;
            }
        }
    }
}

template <bool F32, bool BF>
__device__ __forceinline__ void store8(void* p, long long i, const float* f) {
    if (F32) {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        q[0] = make_float4(f[0], f[1], f[2], f[3]);
        q[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        uint4 v;
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (BF) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
                w[k] = *reinterpret_cast<const uint32_t*>(&b);
            } else {
                const __half2 b = __floats2half2_rn(f[2 * k], f[2 * k + 1]);
                w[k] = *reinterpret_cast<const uint32_t*>(&b);
            }
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = v;
    }
}

template <bool F32, bool BF>
__device__ __forceinline__ void load8(const void* p, long long i, float* f) {
    Raw<F32> r;
    load_raw<F32>(p, i, r);
    widen<F32, BF>(r, f);
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Values whose type the kernel is not compiled for.  With AHEAD those of 16 bits are fetched ahead of their use, all others
// at it.
template <bool AHEAD>
struct Later {
    Raw<false> r;
    __device__ __forceinline__ void fetch(bool f32, const void* p, long long i) {
        if (AHEAD && !f32) load_raw<false>(p, i, r);
    }
    template <bool BF>
    __device__ __forceinline__ void get(bool f32, const void* p, long long i, float* f) {
        if (f32) {
            Raw<true> q;
            load_raw<true>(p, i, q);
            widen<true, BF>(q, f);
        } else {
            if (!AHEAD) load_raw<false>(p, i, r);
            widen<false, BF>(r, f);
        }
    }
};

// Sum over the threads of a row, the same in all of them.
__device__ __forceinline__ float row_sum(float v, bool cta, float* ws) {
    v = ft::warp_sum(v);
    if (!cta) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) ws[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < (int)(blockDim.x >> 5) ? ws[lane] : 0.f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);  // (at most 16 warps)
    return __shfl_sync(0xffffffffu, v, 0);
}

// BF: the 16-bit type is bf16, else f16; B32, R32, O32: block, residual, out are fp32.
template <bool BF, bool B32, bool R32, bool O32, int NV>
__global__ void __launch_bounds__(512, NV == 1 ? 3 : 1) block_norm_kernel(const NormParams p) {
    __shared__ float ws[2][32];
    ft::grid_dep_launch();
    const bool cta = p.tpr != 32;
    const long long t = cta ? blockIdx.x : (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int tid = cta ? threadIdx.x : threadIdx.x & 31;
    ft::grid_dep_wait();
    if (t >= p.T) return;  // whole warps
    const long long rb = t * p.ld_b, rr = t * p.ld_r, rg = p.gate_kind == FT_GATE_FULL ? t * p.ld_g : 0;
    // Of long rows the weights are asked for at once as well; of shorter ones their registers cost more CTAs than the wait for
    // them (8192 tokens of 2048 30.0 us instead of 23.8; 2048 of 16384 69.0 instead of 83.8).
    constexpr bool W_AHEAD = NV == 4;
    Later<W_AHEAD> post_in[NV], pre_in[NV];
    float a[NV][8], h[NV][8];
    if constexpr (W_AHEAD) {
        Raw<B32> b_in[NV];
        Raw<R32> r_in[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = v * p.tpr + tid;
            if (i >= p.nvec) continue;
            load_raw<R32>(p.resid, rr + 8 * i, r_in[v]);
            if (p.block) load_raw<B32>(p.block, rb + 8 * i, b_in[v]);
            if (p.post) post_in[v].fetch(p.w32, p.post, 8 * i);
            if (p.pre && p.out) pre_in[v].fetch(p.w32, p.pre, 8 * i);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int k = 0; k < 8; ++k) h[v][k] = a[v][k] = 0.f;
            if (v * p.tpr + tid < p.nvec) {
                widen<R32, BF>(r_in[v], h[v]);
                if (p.block) widen<B32, BF>(b_in[v], a[v]);
            }
        }
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = v * p.tpr + tid;
            if (i < p.nvec) {
                load8<R32, BF>(p.resid, rr + 8 * i, h[v]);
                if (p.block) load8<B32, BF>(p.block, rb + 8 * i, a[v]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) h[v][k] = a[v][k] = 0.f;
            }
        }
    }
    if (p.gate_kind == FT_GATE_FULL)  // (into L2: no registers)
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = v * p.tpr + tid;
            if (i < p.nvec) prefetch_l2(static_cast<const uint8_t*>(p.gate) + (rg + 8 * i) * (p.g32 ? 4 : 2));
        }
    if (p.block) {
        float f = p.bs;
        if (p.post_norm) {
            float ss = 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int k = 0; k < 8; ++k) ss = fmaf(a[v][k], a[v][k], ss);
            ss = row_sum(ss, cta, ws[0]);
            const float r = rsqrtf(ss / p.H + p.eps);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int i = v * p.tpr + tid;
                float w[8];
                if (p.post && i < p.nvec) {
                    post_in[v].template get<BF>(p.w32, p.post, 8 * i, w);
#pragma unroll
                    for (int k = 0; k < 8; ++k) a[v][k] = a[v][k] * r * w[k];
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) a[v][k] *= r;
                }
            }
        }
        if (p.gate_kind == FT_GATE_TOKEN) {
            float g;
            if (p.g32) g = static_cast<const float*>(p.gate)[t];
            else if (BF) g = __bfloat162float(static_cast<const __nv_bfloat16*>(p.gate)[t]);
            else g = __half2float(static_cast<const __half*>(p.gate)[t]);
            f *= g;
        } else if (p.gate_kind != FT_GATE_NONE) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int i = v * p.tpr + tid;
                float g[8];
                if (i < p.nvec) {
                    Later<false>().get<BF>(p.g32, p.gate, rg + 8 * i, g);
#pragma unroll
                    for (int k = 0; k < 8; ++k) a[v][k] *= g[k];
                }
            }
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int k = 0; k < 8; ++k) h[v][k] = fmaf(f, a[v][k], p.rs * h[v][k]);
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int k = 0; k < 8; ++k) h[v][k] *= p.rs;
    }
    if (p.resid_out) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = v * p.tpr + tid;
            if (i < p.nvec) store8<R32, BF>(p.resid_out, t * p.ld_ro + 8 * i, h[v]);
        }
    }
    if (!p.out) return;
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = fmaf(h[v][k], h[v][k], ss);
    ss = row_sum(ss, cta, ws[1]);
    const float r = rsqrtf(ss / p.H + p.eps);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int i = v * p.tpr + tid;
        if (i >= p.nvec) continue;
        float w[8];
        if (p.pre) {
            pre_in[v].template get<BF>(p.w32, p.pre, 8 * i, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) h[v][k] = h[v][k] * r * w[k];
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) h[v][k] *= r;
        }
        store8<O32, BF>(p.out, t * p.ld_o + 8 * i, h[v]);
    }
}

template <bool BF, bool B32, bool R32, bool O32>
const void* kernel_nv(int nv) {
    return nv == 1 ? (const void*)block_norm_kernel<BF, B32, R32, O32, 1>
         : nv == 2 ? (const void*)block_norm_kernel<BF, B32, R32, O32, 2>
                   : (const void*)block_norm_kernel<BF, B32, R32, O32, 4>;
}
template <bool BF>
const void* kernel_of(bool b32, bool r32, bool o32, int nv) {
    if (b32) {
        if (r32) return o32 ? kernel_nv<BF, true, true, true>(nv) : kernel_nv<BF, true, true, false>(nv);
        return o32 ? kernel_nv<BF, true, false, true>(nv) : kernel_nv<BF, true, false, false>(nv);
    }
    if (r32) return o32 ? kernel_nv<BF, false, true, true>(nv) : kernel_nv<BF, false, true, false>(nv);
    return o32 ? kernel_nv<BF, false, false, true>(nv) : kernel_nv<BF, false, false, false>(nv);
}

// T rows of w bytes, ld bytes apart (ld = 0: one row).
struct Span {
    uintptr_t p;
    long long ld, w, n;
    uintptr_t end() const { return p + (uintptr_t)(ld * (n - 1) + w); }
};

// Whether two spans may share a byte: they overlap and are not different columns of the rows of one buffer.
bool may_touch(const Span& a, const Span& b) {
    if (!a.p || !b.p || a.p >= b.end() || b.p >= a.end()) return false;
    if (a.ld != b.ld || a.ld == 0) return true;
    const uintptr_t row = (uintptr_t)a.ld, off = b.p >= a.p ? (b.p - a.p) % row : (row - (a.p - b.p) % row) % row;
    return off < (uintptr_t)a.w || off + (uintptr_t)b.w > row;
}

bool same(const Span& a, const Span& b) { return a.p == b.p && a.ld == b.ld && a.w == b.w; }

int size_of(int type) { return type == FT_T_F32 ? 4 : 2; }

}  // namespace

extern "C" ft_status ft_block_norm(const ft_norm_desc* d, int32_t T, const void* block, int64_t ld_b, const void* gate,
                                   int64_t ld_g, const void* resid, int64_t ld_r, void* resid_out, int64_t ld_ro,
                                   void* out, int64_t ld_o, void* stream) {
    if (!d || T < 0 || d->H < 8 || d->H > 16384 || d->H % 8 || (d->post_norm != 0 && d->post_norm != 1) ||
        d->gate < FT_GATE_NONE || d->gate > FT_GATE_FULL || !(d->eps >= 0.f) || !std::isfinite(d->eps) ||
        !std::isfinite(d->resid_scale) || !std::isfinite(d->block_scale))
        return FT_ERR_ARG;
    // the 16-bit types of what the call has are one
    int small = -1;
    const struct { int type; bool used; } types[] = {{d->block_type, block != nullptr}, {d->resid_type, true},
                                                     {d->out_type, out != nullptr}, {d->w_type, d->pre || d->post},
                                                     {d->gate_type, d->gate != FT_GATE_NONE}};
    for (const auto& t : types) {
        if (t.type < FT_T_BF16 || t.type > FT_T_F32) return FT_ERR_ARG;
        if (t.type == FT_T_F32 || !t.used) continue;
        if (small >= 0 && t.type != small) return FT_ERR_ARG;
        small = t.type;
    }
    if (T == 0) return FT_OK;
    const bool full = d->gate == FT_GATE_FULL;
    const long long H = d->H;
    // (rows whose last byte has no 62-bit offset are refused)
    auto bad_rows = [&](const void* p, long long ld) { return p && ((uintptr_t)p % 16 || ld < H || ld % 8 || ld > (1ll << 60) / T); };
    if (!resid || (!resid_out && !out) || bad_rows(block, ld_b) || bad_rows(resid, ld_r) || bad_rows(resid_out, ld_ro) ||
        bad_rows(out, ld_o) || (full && bad_rows(gate, ld_g)) || (uintptr_t)d->post % 16 || (uintptr_t)d->pre % 16 ||
        (!block && (d->post_norm || d->gate != FT_GATE_NONE)) || (d->gate != FT_GATE_NONE && !gate) ||
        (d->gate == FT_GATE_CHANNEL && (uintptr_t)gate % 16) ||
        (d->gate == FT_GATE_TOKEN && (uintptr_t)gate % size_of(d->gate_type)))
        return FT_ERR_ARG;
    const int sb = size_of(d->block_type), sr = size_of(d->resid_type), so = size_of(d->out_type), sg = size_of(d->gate_type),
              sw = size_of(d->w_type);
    const Span in[] = {{(uintptr_t)block, ld_b * sb, H * sb, T}, {(uintptr_t)resid, ld_r * sr, H * sr, T}};
    Span g{0, 0, 0, 1};
    if (d->gate == FT_GATE_FULL) g = {(uintptr_t)gate, ld_g * sg, H * sg, T};
    else if (d->gate == FT_GATE_CHANNEL) g = {(uintptr_t)gate, 0, H * sg, 1};
    else if (d->gate == FT_GATE_TOKEN) g = {(uintptr_t)gate, 0, (long long)T * sg, 1};
    const Span fixed[] = {g, {(uintptr_t)d->post, 0, H * sw, 1}, {(uintptr_t)d->pre, 0, H * sw, 1}};
    const Span outs[] = {{(uintptr_t)resid_out, ld_ro * sr, H * sr, T}, {(uintptr_t)out, ld_o * so, H * so, T}};
    for (const Span& o : outs) {
        for (const Span& i : in)
            if (may_touch(o, i) && !same(o, i)) return FT_ERR_ARG;
        for (const Span& i : fixed)
            if (may_touch(o, i)) return FT_ERR_ARG;
    }
    if (may_touch(outs[0], outs[1])) return FT_ERR_ARG;

    NormParams p{};
    p.T = T; p.H = d->H; p.nvec = d->H / 8;
    p.gate_kind = d->gate; p.post_norm = d->post_norm;
    p.w32 = d->w_type == FT_T_F32; p.g32 = d->gate_type == FT_T_F32;
    p.block = block; p.gate = gate; p.resid = resid; p.pre = d->pre; p.post = d->post;
    p.resid_out = resid_out; p.out = out;
    p.ld_b = ld_b; p.ld_g = ld_g; p.ld_r = ld_r; p.ld_ro = ld_ro; p.ld_o = ld_o;
    p.eps = d->eps; p.rs = d->resid_scale; p.bs = d->block_scale;
    // a row of at most 64 vectors is a warp's, a longer one a CTA's (8192 tokens of 1024: a warp 21.4 us, a CTA 16.3; 16384 of
    // 512: 16.8 and 19.0)
    int nv, threads, grid;
    if (p.nvec <= 64) {
        p.tpr = 32;
        nv = p.nvec <= 32 ? 1 : 2;
        threads = 128;
        grid = (int)(((long long)T + 3) / 4);
    } else {
        nv = p.nvec <= 512 ? 1 : p.nvec <= 1024 ? 2 : 4;
        threads = ((p.nvec + nv - 1) / nv + 31) / 32 * 32;
        p.tpr = threads;
        grid = T;
    }
    const bool b32 = d->block_type == FT_T_F32, r32 = d->resid_type == FT_T_F32, o32 = d->out_type == FT_T_F32;
    const void* k = small == FT_T_F16 ? kernel_of<false>(b32, r32, o32, nv) : kernel_of<true>(b32, r32, o32, nv);
    void* args[] = {&p};
    const cudaError_t e = launch_dependent(k, grid, threads, 0, (cudaStream_t)stream, args);
    if (e == cudaSuccess) return FT_OK;
    if (getenv("FT_DEBUG")) fprintf(stderr, "libft: launch -> %s\n", cudaGetErrorString(e));
    return FT_ERR_CUDA;
}

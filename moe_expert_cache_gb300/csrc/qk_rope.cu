// ft_qk_rope_store: RMS norm and rotation of query and key heads, and the
// store of keys and values into their pages, in one pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * w        per head, over its D values
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)   for the rot/2 pairs
//
// Bound: HBM for prompts (each value is read once and written once, 4 bytes a
// value plus the angles' table), latency for a few tokens.  D/16 lanes hold a
// head, 16 values each as two 16-byte vectors.  In the half form lane j takes
// vector j of the first half and its partner of the second, so a pair never
// leaves its lane; in the pair form it takes 16 neighbours.  Either way it
// needs the angles 8j..8j+7.  Norm weights and angles are multiplied once for a
// token, y = (x r) C + (partner r) S with r = rsqrt(...), and kept in registers
// over all the heads of one kind that the warp works on; the arithmetic runs two
// values an instruction.
//
// Measured: 8191 tokens of 32 + 2*4 heads of 128, 33.7 us, 5.1 TB/s (75% of the
// copy rate; DRAM sees 86 MB in and 33 MB out, the rest of the writes stays in
// L2); one token 2.4 us, the latency of three dependent reads (token, page,
// values) and a launch.
#include "ft_kv.cuh"

namespace {

struct RopeParams {
    RopeArgs a;
    int Hq, Hkv, page, page_log, n_pages, n_rows, row_pages, L;
    int steps;   // warp steps per token: 32*16/D heads each
    int spw;     // steps of one warp
    int parts;   // warps per token
    const int* table;
    uint8_t* pool;
    unsigned* err;
};

// Pairs of fp32 values in 64-bit registers.
typedef uint64_t f32x2;
__device__ __forceinline__ f32x2 pk(float a, float b) {
    f32x2 v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ float2 un(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// 8 values of a 16-byte vector as four pairs.
template <bool BF>
__device__ __forceinline__ void unpack8(const uint4& v, f32x2* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF) {
            f[i] = pk(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        } else {
            const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[i] = pk(t.x, t.y);
        }
    }
}

template <bool BF>
__device__ __forceinline__ uint4 pack8(const f32x2* f) {
    uint4 v;
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = un(f[i]);
        if (BF) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(t.x, t.y);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        } else {
            const __half2 b = __floats2half2_rn(t.x, t.y);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
    }
    return v;
}

// heads whose loads a lane has in flight, at 128 threads and 4 CTAs an SM (8191 tokens: 33.7 us; 2 at 256 threads 35.8,
// 4 46.4, whose registers spill)
constexpr int U = 3;

template <int D, bool BF, bool PAIR>
__global__ void __launch_bounds__(128, 4) qk_rope_store_kernel(const RopeParams p) {
    constexpr int GL = D / 16;      // lanes of a head
    constexpr int HPW = 32 / GL;    // heads of a warp step
    ft::grid_dep_launch();
    const int lane = threadIdx.x & 31, j = lane % GL, sub = lane / GL;
    const long long w = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int t = (int)(w / p.parts), part = (int)(w % p.parts);
    ft::grid_dep_wait();
    if (t >= p.a.T) return;
    const int rot = p.a.rot, half = rot / 2;
    // offsets of this lane's two vectors within a head
    const bool turns = 16 * j < rot;
    const int o0 = turns && !PAIR ? 8 * j : 16 * j;
    const int o1 = turns && !PAIR ? half + 8 * j : 16 * j + 8;
    const int HT = p.Hq + 2 * p.Hkv;
    const uint16_t* x = static_cast<const uint16_t*>(p.a.qkv) + (long long)t * p.a.ld;
    const int step0 = part * p.spw, step1 = min(step0 + p.spw, p.steps);

    uint4 va[U], vb[U];
    auto load = [&](int s0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = (s0 + u) * HPW + sub;
            if (s0 + u < step1 && h < HT) {
                va[u] = *reinterpret_cast<const uint4*>(x + (long long)h * D + o0);
                vb[u] = *reinterpret_cast<const uint4*>(x + (long long)h * D + o1);
            }
        }
    };
    load(step0);

    const int row = p.a.row_of[t], pos = p.a.pos[t];
    bool live = row >= 0;
    int pg = -1;
    if (row >= 0 && row < p.n_rows && pos >= 0 && pos < p.a.max_pos && (pos >> p.page_log) < p.row_pages)
        pg = p.table[(size_t)row * p.row_pages + (pos >> p.page_log)];
    if (live && (pg < 0 || pg >= p.n_pages)) {
        live = false;
        if (lane == 0) atomicOr(p.err, FT_DEVERR_ARG);
    }
    if (row < -1 && lane == 0) atomicOr(p.err, FT_DEVERR_ARG);

    // factors of the values and of their partners for the heads of one kind (0: queries, 1: keys)
    f32x2 ca[4], cb[4], sa[4], sb[4];
    int kind = -1;
    auto factors = [&](int k) {
        kind = k;
        const uint16_t* nw = static_cast<const uint16_t*>(k ? p.a.k_norm : p.a.q_norm);
        const f32x2 one = pk(1.f, 1.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) ca[i] = cb[i] = one;
        if (nw) {
            unpack8<BF>(*reinterpret_cast<const uint4*>(nw + o0), ca);
            unpack8<BF>(*reinterpret_cast<const uint4*>(nw + o1), cb);
        }
        if (!turns) return;
        const float* cs = p.a.cos_sin + (long long)pos * rot + 8 * j;
        float c[8], s[8];
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            *reinterpret_cast<float4*>(c + i) = *reinterpret_cast<const float4*>(cs + i);
            *reinterpret_cast<float4*>(s + i) = *reinterpret_cast<const float4*>(cs + half + i);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!PAIR) {  // values 2i, 2i+1 of the first half turn with the same ones of the second
                const f32x2 cc = pk(c[2 * i], c[2 * i + 1]);
                sa[i] = mul2(cb[i], pk(-s[2 * i], -s[2 * i + 1]));
                sb[i] = mul2(ca[i], pk(s[2 * i], s[2 * i + 1]));
                ca[i] = mul2(ca[i], cc);
                cb[i] = mul2(cb[i], cc);
            } else {      // value 2i turns with 2i+1
                const float2 wa = un(ca[i]), wb = un(cb[i]);
                sa[i] = pk(-wa.y * s[i], wa.x * s[i]);
                sb[i] = pk(-wb.y * s[4 + i], wb.x * s[4 + i]);
                ca[i] = mul2(ca[i], pk(c[i], c[i]));
                cb[i] = mul2(cb[i], pk(c[4 + i], c[4 + i]));
            }
        }
    };
    // first value of this token in the page's banks of the layer
    uint16_t* bank = nullptr;
    if (live)
        bank = reinterpret_cast<uint16_t*>(p.pool) +
               (((size_t)pg * p.L + p.a.layer) * 2 * p.Hkv * p.page + (pos & (p.page - 1))) * D;
    const size_t head_stride = (size_t)p.page * D;
    uint16_t* qo = static_cast<uint16_t*>(p.a.q_out) + (long long)t * p.a.ld_q;

    for (int s0 = step0; s0 < step1; s0 += U) {
        uint4 xa[U], xb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            xa[u] = va[u];
            xb[u] = vb[u];
        }
        if (s0 + U < step1) load(s0 + U);  // (a head is read before its place in a shared buffer is written)
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = (s0 + u) * HPW + sub;
            if (s0 + u >= step1) break;  // warp-uniform
            const bool in = h < HT, is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
            f32x2 a[4], b[4];
            unpack8<BF>(in ? xa[u] : make_uint4(0, 0, 0, 0), a);
            unpack8<BF>(in ? xb[u] : make_uint4(0, 0, 0, 0), b);
            f32x2 q = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) q = fma2(b[i], b[i], fma2(a[i], a[i], q));
            const float2 q2 = un(q);
            float ss = q2.x + q2.y;
#pragma unroll
            for (int o = GL / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (!in) continue;
            uint16_t* dst = is_q ? qo + (long long)h * D : bank + (size_t)(h - p.Hq) * head_stride;
            if (!live) {
                if (is_q) {
                    *reinterpret_cast<uint4*>(dst + o0) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4*>(dst + o1) = make_uint4(0, 0, 0, 0);
                }
                continue;
            }
            if (is_v) {
                *reinterpret_cast<uint4*>(dst + o0) = xa[u];
                *reinterpret_cast<uint4*>(dst + o1) = xb[u];
                continue;
            }
            if (kind != (is_q ? 0 : 1)) factors(is_q ? 0 : 1);
            if (is_q ? p.a.q_norm != nullptr : p.a.k_norm != nullptr) {
                const float r = rsqrtf(ss * (1.f / D) + p.a.eps);
                const f32x2 r2 = pk(r, r);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = mul2(a[i], r2);
                    b[i] = mul2(b[i], r2);
                }
            }
            f32x2 ya[4], yb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ya[i] = mul2(a[i], ca[i]);
                yb[i] = mul2(b[i], cb[i]);
            }
            if (turns) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (!PAIR) {
                        ya[i] = fma2(b[i], sa[i], ya[i]);
                        yb[i] = fma2(a[i], sb[i], yb[i]);
                    } else {
                        const float2 u2 = un(a[i]), v2 = un(b[i]);
                        ya[i] = fma2(pk(u2.y, u2.x), sa[i], ya[i]);
                        yb[i] = fma2(pk(v2.y, v2.x), sb[i], yb[i]);
                    }
                }
            }
            *reinterpret_cast<uint4*>(dst + o0) = pack8<BF>(ya);
            *reinterpret_cast<uint4*>(dst + o1) = pack8<BF>(yb);
        }
    }
}

template <int D>
const void* kernel_of(bool bf, bool pair) {
    if (bf) return pair ? (const void*)qk_rope_store_kernel<D, true, true> : (const void*)qk_rope_store_kernel<D, true, false>;
    return pair ? (const void*)qk_rope_store_kernel<D, false, true> : (const void*)qk_rope_store_kernel<D, false, false>;
}

}  // namespace

cudaError_t launch_qk_rope_store(ft_kv* kv, const RopeArgs& a) {
    RopeParams p{};
    p.a = a;
    p.Hq = kv->Hq; p.Hkv = kv->Hkv; p.page = kv->page; p.page_log = __builtin_ctz(kv->page); p.n_pages = kv->n_pages; p.n_rows = kv->n_rows;
    p.row_pages = kv->row_pages; p.L = kv->L;
    p.table = kv->table; p.pool = kv->pool; p.err = kv->err;
    const int hpw = 32 / (kv->D / 16);
    p.steps = (kv->Hq + 2 * kv->Hkv + hpw - 1) / hpw;
    // few tokens: a warp per step, so that the whole call is one round of
    // loads; many: a warp keeps its token's angles over as many steps as leave
    // 32 warps for every SM, two rounds of the 16 that its registers hold
    const long long per = (long long)a.T * p.steps / ((long long)kv->num_sms * 32);
    p.spw = per < 1 ? 1 : per > p.steps ? p.steps : (int)per;
    p.parts = (p.steps + p.spw - 1) / p.spw;
    const long long warps = (long long)a.T * p.parts;
    const int grid = (int)((warps + 3) / 4);
    const bool bf = kv->dtype == FT_KV_BF16;
    const bool pair = a.pair != 0;
    const void* k = kv->D == 64 ? kernel_of<64>(bf, pair) : kv->D == 128 ? kernel_of<128>(bf, pair) : kernel_of<256>(bf, pair);
    void* args[] = {&p};
    return launch_dependent(k, grid, 128, 0, kv->stream, args);
}

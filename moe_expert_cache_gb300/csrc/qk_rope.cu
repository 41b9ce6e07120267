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
// needs the angles 8j..8j+7, which it keeps in registers over all the heads of
// a token that its warp works on.
#include "ft_kv.cuh"

namespace {

struct RopeParams {
    RopeArgs a;
    int Hq, Hkv, page, n_pages, n_rows, row_pages, L;
    int steps;   // warp steps per token: 32*16/D heads each
    int spw;     // steps of one warp
    int parts;   // warps per token
    const int* table;
    uint8_t* pool;
    unsigned* err;
};

template <bool BF>
__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
    if (BF) {
        ft::bf16x8_to_f32(v, f);
    } else {
        const __half2* h = reinterpret_cast<const __half2*>(&v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = __half22float2(h[i]);
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        }
    }
}

template <bool BF>
__device__ __forceinline__ uint4 pack8(const float* f) {
    uint4 v;
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        } else {
            const __half2 b = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
    }
    return v;
}

constexpr int U = 4;  // heads whose loads a lane has in flight

template <int D, bool BF>
__global__ void __launch_bounds__(256) qk_rope_store_kernel(const RopeParams p) {
    ft::grid_dep_launch();
    constexpr int GL = D / 16;      // lanes of a head
    constexpr int HPW = 32 / GL;    // heads of a warp step
    const int lane = threadIdx.x & 31, j = lane % GL, sub = lane / GL;
    const long long w = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int t = (int)(w / p.parts), part = (int)(w % p.parts);
    if (t >= p.a.T) {
        ft::grid_dep_wait();
        return;
    }
    const int rot = p.a.rot, half = rot / 2;
    // offsets of this lane's two vectors within a head
    const bool turns = 16 * j < rot;
    const int o0 = turns && !p.a.pair ? 8 * j : 16 * j;
    const int o1 = turns && !p.a.pair ? half + 8 * j : 16 * j + 8;
    const int HT = p.Hq + 2 * p.Hkv;
    const uint16_t* x = static_cast<const uint16_t*>(p.a.qkv) + (long long)t * p.a.ld;
    const int step0 = part * p.spw, step1 = min(step0 + p.spw, p.steps);

    ft::grid_dep_wait();
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
    if (row >= 0 && row < p.n_rows && pos >= 0 && pos < p.a.max_pos && pos / p.page < p.row_pages)
        pg = p.table[(size_t)row * p.row_pages + pos / p.page];
    if (live && (pg < 0 || pg >= p.n_pages)) {
        live = false;
        if (lane == 0) atomicOr(p.err, FT_DEVERR_ARG);
    }
    if (row < -1 && lane == 0) atomicOr(p.err, FT_DEVERR_ARG);

    float c[8], s[8];
    if (live && turns) {
        const float* cs = p.a.cos_sin + (long long)pos * rot + 8 * j;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            *reinterpret_cast<float4*>(c + i) = *reinterpret_cast<const float4*>(cs + i);
            *reinterpret_cast<float4*>(s + i) = *reinterpret_cast<const float4*>(cs + half + i);
        }
    }
    // first value of this token in the page's banks of the layer
    uint16_t* bank = nullptr;
    if (live)
        bank = reinterpret_cast<uint16_t*>(p.pool) +
               (((size_t)pg * p.L + p.a.layer) * 2 * p.Hkv * p.page + pos % p.page) * D;
    const size_t head_stride = (size_t)p.page * D;
    uint16_t* qo = static_cast<uint16_t*>(p.a.q_out) + (long long)t * p.a.ld_q;

    for (int s0 = step0; s0 < step1; s0 += U) {
        if (s0 > step0) load(s0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = (s0 + u) * HPW + sub;
            if (s0 + u >= step1) break;  // warp-uniform
            const bool in = h < HT, is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
            float a[8], b[8];
            if (in) {
                unpack8<BF>(va[u], a);
                unpack8<BF>(vb[u], b);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) a[i] = b[i] = 0.f;
            }
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss += a[i] * a[i] + b[i] * b[i];
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
                *reinterpret_cast<uint4*>(dst + o0) = va[u];
                *reinterpret_cast<uint4*>(dst + o1) = vb[u];
                continue;
            }
            const uint16_t* nw = static_cast<const uint16_t*>(is_q ? p.a.q_norm : p.a.k_norm);
            if (nw) {
                const float r = rsqrtf(ss * (1.f / D) + p.a.eps);
                float wa[8], wb[8];
                unpack8<BF>(*reinterpret_cast<const uint4*>(nw + o0), wa);
                unpack8<BF>(*reinterpret_cast<const uint4*>(nw + o1), wb);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    a[i] = a[i] * r * wa[i];
                    b[i] = b[i] * r * wb[i];
                }
            }
            if (turns) {
                if (!p.a.pair) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float ya = a[i], yb = b[i];
                        a[i] = ya * c[i] - yb * s[i];
                        b[i] = yb * c[i] + ya * s[i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float a0 = a[i], a1 = a[i + 1], b0 = b[i], b1 = b[i + 1];
                        a[i] = a0 * c[i / 2] - a1 * s[i / 2];
                        a[i + 1] = a1 * c[i / 2] + a0 * s[i / 2];
                        b[i] = b0 * c[4 + i / 2] - b1 * s[4 + i / 2];
                        b[i + 1] = b1 * c[4 + i / 2] + b0 * s[4 + i / 2];
                    }
                }
            }
            *reinterpret_cast<uint4*>(dst + o0) = pack8<BF>(a);
            *reinterpret_cast<uint4*>(dst + o1) = pack8<BF>(b);
        }
    }
}

}  // namespace

cudaError_t launch_qk_rope_store(ft_kv* kv, const RopeArgs& a) {
    RopeParams p{};
    p.a = a;
    p.Hq = kv->Hq; p.Hkv = kv->Hkv; p.page = kv->page; p.n_pages = kv->n_pages; p.n_rows = kv->n_rows;
    p.row_pages = kv->row_pages; p.L = kv->L;
    p.table = kv->table; p.pool = kv->pool; p.err = kv->err;
    const int hpw = 32 / (kv->D / 16);
    p.steps = (kv->Hq + 2 * kv->Hkv + hpw - 1) / hpw;
    // few tokens: a warp per step, so that the whole call is one round of
    // loads; many: a warp keeps its token's angles over as many steps as leave
    // every SM 32 warps
    const long long per = (long long)a.T * p.steps / ((long long)kv->num_sms * 32);
    p.spw = per < 1 ? 1 : per > p.steps ? p.steps : (int)per;
    p.parts = (p.steps + p.spw - 1) / p.spw;
    const long long warps = (long long)a.T * p.parts;
    const int grid = (int)((warps + 7) / 8);
    const bool bf = kv->dtype == FT_KV_BF16;
    const void* k = kv->D == 64    ? (bf ? (const void*)qk_rope_store_kernel<64, true> : (const void*)qk_rope_store_kernel<64, false>)
                    : kv->D == 128 ? (bf ? (const void*)qk_rope_store_kernel<128, true> : (const void*)qk_rope_store_kernel<128, false>)
                                   : (bf ? (const void*)qk_rope_store_kernel<256, true> : (const void*)qk_rope_store_kernel<256, false>);
    void* args[] = {&p};
    return launch_dependent(k, grid, 256, 0, kv->stream, args);
}

// block_norm.cuh -- the residual sum and the norms between two blocks,
// forward and backward ("DiffuMamba: High-Throughput Diffusion LMs with
// Mamba Backbone", App. A.1 Eq. (10)-(12)).
//
// Per token row:  un = N(u) post_w,  x_out = res_scale x + gate un (rounded to
// the stream's type),  y = gamma N(x_out) + beta.  With n = N(x_out),
// m = N(u), rs = 1/sigma and means over the row:
//   dn = gamma dy,  D = dx_out + rs (dn - n mean(dn n) - mean(dn))
//   dx = res_scale D,  g = gate D,  dgate = sum D un,  dpost_w = sum g m
//   du = rs_u (g post_w - m mean(g post_w m) - mean(g post_w))   (or g)
//   dgamma = sum dy n,  dbeta = sum dy
// (a root-mean-square norm drops the plain means).
//
// The work is one read and one write of each row: bound by memory.  A thread
// owns K groups of V neighbouring columns for every row it visits, so the
// row stays in registers between its passes (mean, then the centred squares:
// never a difference of large sums), and the backward's column sums stay in
// registers over all rows of a block.  Row sums are fp32, through warp
// shuffles and, for rows wider than a warp, shared memory.
//
// Three forms.  Rows of 256 to 8192 columns in whole groups of eight: a block
// walks a run of one batch row's tokens, every thread copying its own columns
// of the rows ahead into shared memory (cp.async; a thread reads back only what
// it copied, so no barrier), with the vectors in registers for the whole run.
// Odd and narrow rows, and those whose copies ahead do not fit: tiles of neighbouring rows as flat runs of bytes.  What
// neither takes: a warp or a block a row, straight from memory.
//
// 16,384 rows of 2048 bf16 (268 MB, 41 us at 6.56 TB/s): forward 71 us straight
// from memory, 58 copied ahead, 54 with one barrier for mean and variance in
// packed arithmetic, 50 with two column groups a thread.  Backward (403 MB, 61
// us): 168, 105, 83 with packed arithmetic and the statistics asked for a row ahead,
// 80 with fp32 rows in whole sectors (which took 65,536 rows of 1920 with an fp32
// stream from 313 us to 249-280, from run to run, of 230).  What is left is the
// chain of a row's sums.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "tma_util.cuh"

namespace bimamba {

constexpr int kBlockNormThreads = 512;  // at most; 128 registers a thread

struct BlockNormParams {
    const void* x;         // forward: the stream entering; backward: x_out as stored
    const void* u;         // or null
    const float* gate;     // or null
    const float* post_w;   // or null
    const float* gamma;    // or null
    const float* beta;     // or null (forward)
    void* x_out;           // forward, or null
    void* y;               // forward, or null
    float* stats;          // [rows][4]; forward: or null
    const void* dy;        // backward, or null
    const void* dx_out;    // backward, or null
    void* dx;
    void* du;
    float* part;           // backward: [batch * nseg][4][d] column sums (dgate, dpost_w, dgamma, dbeta), or null
    float res_scale, eps;
    int64_t L;
    int batch, d;
    int gate_bs, gamma_bs;  // floats between batch rows: d, or 0 when shared
    int rms;
    int nseg;               // row segments per batch row (backward, and the copying form)
};

// V neighbouring elements <-> fp32 (V = 8: 16- or 32-byte rows of a 16-byte
// aligned pointer; V = 1: any).
template <int V>
__device__ __forceinline__ void bn_load(const __nv_bfloat16* p, float* v) {
    if constexpr (V == 8) {
        const uint4 q = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(w[e] << 16);
            v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
    } else {
        v[0] = __bfloat162float(*p);
    }
}
template <int V>
__device__ __forceinline__ void bn_load(const float* p, float* v) {
    if constexpr (V == 8) {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        v[0] = *p;
    }
}
template <int V>
__device__ __forceinline__ void bn_store(__nv_bfloat16* p, const float* v) {
    if constexpr (V == 8) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        *p = __float2bfloat16_rn(v[0]);
    }
}
template <int V>
__device__ __forceinline__ void bn_store(float* p, const float* v) {
    if constexpr (V == 8) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *p = v[0];
    }
}
// The value as the stream's type holds it.
template <typename T>
__device__ __forceinline__ float bn_round(float v) {
    if constexpr (sizeof(T) == 2) return __bfloat162float(__float2bfloat16_rn(v));
    return v;
}
// V entries of an optional fp32 vector, `other` without it.
template <int V>
__device__ __forceinline__ void bn_vec(const float* p, int c, float other, float* v) {
    if (p) {
        bn_load<V>(p + c, v);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = other;
    }
}

// The sum of v over the row's threads (WARP: the warp; else the block, by
// the two buffers of `red` in turn, so one barrier a sum is enough).
template <bool WARP>
__device__ __forceinline__ float bn_row_sum(float v, float (*red)[32], int& turn) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if constexpr (WARP) return v;
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    float* r = red[turn];
    turn ^= 1;
    if (lane == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < nw ? r[lane] : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Mean (0 with rms) and 1/sigma of the row held in v[K][V].
template <int V, int K, bool WARP>
__device__ __forceinline__ void bn_stats(const float (&v)[K][V], int col0, int step, int d, int rms, float eps,
                                         float (*red)[32], int& turn, float& mu, float& rs) {
    mu = 0.f;
    if (!rms) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) s += v[k][e];  // columns past d hold 0
        mu = bn_row_sum<WARP>(s, red, turn) / (float)d;
    }
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (col0 + k * step < d) {
#pragma unroll
            for (int e = 0; e < V; ++e) q = fmaf(v[k][e] - mu, v[k][e] - mu, q);
        }
    rs = rsqrtf(bn_row_sum<WARP>(q, red, turn) / (float)d + eps);
}

// One row per block (blockDim.x threads of K groups), or with WARP a row per
// warp.  V == 8: d % 8 == 0 and every pointer 16-byte aligned.
template <typename TS, typename TU, int V, int K, bool WARP>
__global__ void __launch_bounds__(kBlockNormThreads) block_norm_fwd_kernel(const BlockNormParams p) {
    __shared__ float red[2][32];
    int turn = 0;
    const int64_t row = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= p.batch * p.L) return;  // whole warps (WARP) or no block at all
    const int64_t b = row / p.L;
    const int d = p.d, lane = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int col0 = lane * V, step = (WARP ? 32 : blockDim.x) * V;
    float x[K][V], u[K][V];
    float4 st = make_float4(0.f, 1.f, 0.f, 1.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = col0 + k * step;
#pragma unroll
        for (int e = 0; e < V; ++e) x[k][e] = u[k][e] = 0.f;
        if (c < d) {
            bn_load<V>(static_cast<const TS*>(p.x) + row * d + c, x[k]);
            if (p.u) bn_load<V>(static_cast<const TU*>(p.u) + row * d + c, u[k]);
        }
    }
    if (p.post_w) bn_stats<V, K, WARP>(u, col0, step, d, p.rms, p.eps, red, turn, st.z, st.w);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = col0 + k * step;
        if (c >= d) continue;
        float g[V], w[V];
        bn_vec<V>(p.gate ? p.gate + b * p.gate_bs : nullptr, c, 1.f, g);
        if (p.post_w) {
            bn_vec<V>(p.post_w, c, 1.f, w);
#pragma unroll
            for (int e = 0; e < V; ++e) u[k][e] = (u[k][e] - st.z) * st.w * w[e];
        }
#pragma unroll
        for (int e = 0; e < V; ++e) x[k][e] = bn_round<TS>(fmaf(g[e], u[k][e], p.res_scale * x[k][e]));
        if (p.x_out) bn_store<V>(static_cast<TS*>(p.x_out) + row * d + c, x[k]);
    }
    if (p.y) {
        bn_stats<V, K, WARP>(x, col0, step, d, p.rms, p.eps, red, turn, st.x, st.y);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = col0 + k * step;
            if (c >= d) continue;
            float g[V], be[V];
            bn_vec<V>(p.gamma ? p.gamma + b * p.gamma_bs : nullptr, c, 1.f, g);
            bn_vec<V>(p.beta ? p.beta + b * p.gamma_bs : nullptr, c, 0.f, be);
#pragma unroll
            for (int e = 0; e < V; ++e) x[k][e] = fmaf(g[e], (x[k][e] - st.x) * st.y, be[e]);
            bn_store<V>(static_cast<TU*>(p.y) + row * d + c, x[k]);
        }
    }
    if (p.stats && lane == 0) {
        float* s = p.stats + row * 4;
        s[0] = st.x, s[1] = st.y, s[2] = st.z, s[3] = st.w;
    }
}

// A block (or with WARP each warp) walks the rows of one segment of one batch
// row and keeps the column sums in registers.
template <typename TS, typename TU, int V, int K, bool WARP>
__global__ void __launch_bounds__(kBlockNormThreads) block_norm_bwd_kernel(const BlockNormParams p) {
    __shared__ float red[2][32];
    int turn = 0;
    const int64_t b = blockIdx.y;
    const int seg = WARP ? blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (seg >= p.nseg) return;  // whole warps (WARP) or no block at all
    const int d = p.d, lane = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int col0 = lane * V, step = (WARP ? 32 : blockDim.x) * V;
    float sg[K][V], sw[K][V], sm[K][V], sb[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) sg[k][e] = sw[k][e] = sm[k][e] = sb[k][e] = 0.f;
    const int64_t t0 = p.L * seg / p.nseg, t1 = p.L * (seg + 1) / p.nseg;
    for (int64_t t = t0; t < t1; ++t) {
        const int64_t row = b * p.L + t;
        const float* sp = p.stats + row * 4;
        const float mu = sp[0], rs = sp[1], mu_u = sp[2], rs_u = sp[3];
        float n[K][V], dy[K][V], D[K][V], u[K][V];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = col0 + k * step;
#pragma unroll
            for (int e = 0; e < V; ++e) n[k][e] = dy[k][e] = D[k][e] = u[k][e] = 0.f;
            if (c >= d) continue;
            if (p.dy) {
                bn_load<V>(static_cast<const TS*>(p.x) + row * d + c, n[k]);
                bn_load<V>(static_cast<const TU*>(p.dy) + row * d + c, dy[k]);
            }
            if (p.dx_out) bn_load<V>(static_cast<const TS*>(p.dx_out) + row * d + c, D[k]);
            if (p.u) bn_load<V>(static_cast<const TU*>(p.u) + row * d + c, u[k]);
        }
        if (p.dy) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = col0 + k * step;
                if (c >= d) continue;
                float ga[V];
                bn_vec<V>(p.gamma ? p.gamma + b * p.gamma_bs : nullptr, c, 1.f, ga);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    n[k][e] = (n[k][e] - mu) * rs;
                    sm[k][e] = fmaf(dy[k][e], n[k][e], sm[k][e]);
                    sb[k][e] += dy[k][e];
                    dy[k][e] *= ga[e];
                    s1 += dy[k][e];
                    s2 = fmaf(dy[k][e], n[k][e], s2);
                }
            }
            s2 = bn_row_sum<WARP>(s2, red, turn) / (float)d;
            s1 = p.rms ? 0.f : bn_row_sum<WARP>(s1, red, turn) / (float)d;
        }
        float t1s = 0.f, t2s = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = col0 + k * step;
            if (c >= d) continue;
            if (p.dy) {
#pragma unroll
                for (int e = 0; e < V; ++e) D[k][e] = fmaf(rs, dy[k][e] - fmaf(n[k][e], s2, s1), D[k][e]);
            }
            float o[V];
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = p.res_scale * D[k][e];
            bn_store<V>(static_cast<TS*>(p.dx) + row * d + c, o);
            if (!p.u) continue;
            float ga[V], w[V];
            bn_vec<V>(p.gate ? p.gate + b * p.gate_bs : nullptr, c, 1.f, ga);
            if (p.post_w) {
                bn_vec<V>(p.post_w, c, 1.f, w);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float m = (u[k][e] - mu_u) * rs_u, g = ga[e] * D[k][e], gw = g * w[e];
                    sg[k][e] = fmaf(D[k][e], m * w[e], sg[k][e]);
                    sw[k][e] = fmaf(g, m, sw[k][e]);
                    t1s += gw;
                    t2s = fmaf(gw, m, t2s);
                    u[k][e] = m;
                    D[k][e] = gw;
                }
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    sg[k][e] = fmaf(D[k][e], u[k][e], sg[k][e]);
                    o[e] = ga[e] * D[k][e];
                }
                bn_store<V>(static_cast<TU*>(p.du) + row * d + c, o);
            }
        }
        if (p.u && p.post_w) {
            t2s = bn_row_sum<WARP>(t2s, red, turn) / (float)d;
            t1s = p.rms ? 0.f : bn_row_sum<WARP>(t1s, red, turn) / (float)d;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = col0 + k * step;
                if (c >= d) continue;
                float o[V];
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] = rs_u * (D[k][e] - fmaf(u[k][e], t2s, t1s));
                bn_store<V>(static_cast<TU*>(p.du) + row * d + c, o);
            }
        }
    }
    if (!p.part) return;
    float* q = p.part + ((int64_t)b * p.nseg + seg) * 4 * d;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = col0 + k * step;
        if (c >= d) continue;
        bn_store<V>(q + c, sg[k]);
        bn_store<V>(q + d + c, sw[k]);
        bn_store<V>(q + 2 * (int64_t)d + c, sm[k]);
        bn_store<V>(q + 3 * (int64_t)d + c, sb[k]);
    }
}

// ---------------------------------------------------------------- rows copied ahead

// Pairs of columns in packed f32x2 arithmetic.
__device__ __forceinline__ float2 bn_f2(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 bn_mul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 bn_add(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 bn_fma(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// Eight columns of one thread.
struct Bn8 {
    float2 v[4];
};
__device__ __forceinline__ Bn8 bn_fill(float v) { return {{bn_f2(v), bn_f2(v), bn_f2(v), bn_f2(v)}}; }
__device__ __forceinline__ float2 bn_sum4(const Bn8& a) { return bn_add(bn_add(a.v[0], a.v[1]), bn_add(a.v[2], a.v[3])); }
__device__ __forceinline__ Bn8 bn_unpack(uint4 q) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    Bn8 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) r.v[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
    return r;
}
__device__ __forceinline__ uint4 bn_pack(const Bn8& a) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a.v[e].x, a.v[e].y);
        w[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// Stores; the value returned is what the type holds.
__device__ __forceinline__ Bn8 bn_store8(__nv_bfloat16* p, const Bn8& a, bool store) {
    const uint4 q = bn_pack(a);
    if (store) *reinterpret_cast<uint4*>(p) = q;
    return bn_unpack(q);
}
__device__ __forceinline__ Bn8 bn_store8(float* p, const Bn8& a, bool store) {
    if (store)  // 32 bytes at once: two halves would write every sector in two parts
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(a.v[0].x), "f"(a.v[0].y),
                     "f"(a.v[1].x), "f"(a.v[1].y), "f"(a.v[2].x), "f"(a.v[2].y), "f"(a.v[3].x), "f"(a.v[3].y)
                     : "memory");
    return a;
}
__device__ __forceinline__ Bn8 bn_load8(const float* p, float other) {
    if (!p) return bn_fill(other);
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    return {{make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)}};
}

__device__ __forceinline__ float bn_warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}
// What a block's warps hand one another for row sums: two buffers in turn, so
// that one barrier a sum is enough.  At most 16 warps, the absent ones zeros;
// every thread adds the warps' values itself, in order (a read of two warps'
// pairs is one broadcast; shuffles would cost more).
struct BnShared {
    float4 part[2][8];  // (sum, squares) of each warp
    float4 count[8];    // (columns, 1 / columns) of each warp
};
// `columns` of this warp; before the block's first sum.
__device__ __forceinline__ void bn_share(BnShared& sh, float columns) {
    const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    float2* part = reinterpret_cast<float2*>(sh.part);
    float2* count = reinterpret_cast<float2*>(sh.count);
    if (threadIdx.x < 32) part[threadIdx.x] = make_float2(0.f, 0.f);
    if (threadIdx.x >= nw && threadIdx.x < 16) count[threadIdx.x] = make_float2(0.f, 0.f);
    if ((threadIdx.x & 31) == 0) count[warp] = make_float2(columns, columns > 0.f ? 1.f / columns : 0.f);
    __syncthreads();
}
// The block's sums of a pair.
__device__ __forceinline__ float2 bn_block_sum2(float2 v, BnShared& sh, int& turn) {
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    // even lanes take x over, odd ones y: one shuffle a step for both
    float t = (lane & 1 ? v.y : v.x) + __shfl_xor_sync(0xffffffffu, lane & 1 ? v.x : v.y, 1);
#pragma unroll
    for (int off = 2; off <= 16; off <<= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    if (nw == 1) return make_float2(__shfl_sync(0xffffffffu, t, 0), __shfl_sync(0xffffffffu, t, 1));
    float4* r = sh.part[turn];
    turn ^= 1;
    if (lane < 2) reinterpret_cast<float*>(r)[(threadIdx.x >> 5) * 2 + lane] = t;
    __syncthreads();
    v = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        if (2 * w >= nw) break;
        const float4 a = r[w];
        v = bn_add(bn_add(v, make_float2(a.x, a.y)), make_float2(a.z, a.w));
    }
    return v;
}

// 16-byte pieces of eight elements.
template <typename T>
constexpr int kBnPieces = (int)sizeof(T) / 2;

// A warp's 256 columns of a row, in its part of piece q of a stage, and a
// lane's eight of them back.  bf16: each lane copies its own 16 bytes.  fp32:
// lane l copies the chunks l and l + 32 of the warp's 64, so that a copy's
// sectors are whole; chunk c goes to place c ^ (c / 8 & 1), which spreads a
// read of 32 bytes a lane over all banks.  (So a warp's copies are waited for,
// and its reads finished, by the whole warp.)
__device__ __forceinline__ int bn_place(int c) { return c ^ (c >> 3 & 1); }
template <typename T>
__device__ __forceinline__ void bn_fetch(unsigned char* stage, int q, const T* row, int c0, int d) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned char* to = stage + (q * blockDim.x + warp * 32 * kBnPieces<T>) * 16;
#pragma unroll
    for (int h = 0; h < kBnPieces<T>; ++h) {
        const int c = lane + 32 * h, col = c0 + c * (16 / (int)sizeof(T));
        if (col < d) cp_async<16>(to + (sizeof(T) == 2 ? c : bn_place(c)) * 16, row + col, true);
    }
}
template <typename T>
__device__ __forceinline__ Bn8 bn_fetched(const unsigned char* stage, int q) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned char* from = stage + (q * blockDim.x + warp * 32 * kBnPieces<T>) * 16;
    if constexpr (sizeof(T) == 2) {
        return bn_unpack(*reinterpret_cast<const uint4*>(from + lane * 16));
    } else {
        const float4 a = *reinterpret_cast<const float4*>(from + bn_place(2 * lane) * 16);
        const float4 b = *reinterpret_cast<const float4*>(from + bn_place(2 * lane + 1) * 16);
        return {{make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)}};
    }
}

// The block's stages start as zeros: what no copy fills (columns past d, an
// absent tensor) reads as that.
__device__ __forceinline__ void bn_clear(unsigned char* smem, int bytes) {
    for (int q = threadIdx.x * 16; q < bytes; q += blockDim.x * 16) *reinterpret_cast<uint4*>(smem + q) = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
}

// Vectors of a thread's columns: held in registers, or (where there are too
// many columns) read again a row; they stay in L1.
template <int K, bool HOLD>
struct BnVec {
    const float* p;
    float other;
    Bn8 v[HOLD ? K : 1];
    __device__ __forceinline__ void start(const float* q, float without, int col0, int step, int d) {
        p = q;
        other = without;
        if constexpr (HOLD) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = col0 + k * step;
                v[k] = bn_load8(p && c < d ? p + c : nullptr, c < d ? other : 0.f);  // zeros keep zeros past d
            }
        }
    }
    __device__ __forceinline__ Bn8 get(int k, int c) const {
        if constexpr (HOLD) return v[k];
        return bn_load8(p ? p + c : p, other);
    }
};

// Rows ahead, and the 16-byte pieces of one: what fits in shared memory.
template <typename TS, typename TU>
constexpr int kBnFwdStages = sizeof(TU) == 4 ? 3 : 4;
template <typename TS, typename TU, int K>
constexpr int kBnFwdPieces = K * (kBnPieces<TS> + kBnPieces<TU>);
template <typename TU, int K>
constexpr int kBnBwdStages = K == 1 ? 4 : (sizeof(TU) == 4 ? 1 : 2);
template <typename TS, typename TU, int K>
constexpr int kBnBwdPieces = K * 2 * (kBnPieces<TS> + kBnPieces<TU>);

// Mean (0 with rms) and 1/sigma of the row held in v, one barrier: each warp
// has the mean and the centred squares of its own columns, and with means m_w
// of n_w columns the row's squares are sum_w M2_w + n_w (m_w - mean)^2: no
// difference of large sums.
template <int K>
__device__ __forceinline__ float bn_warp_columns(int d) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < K; ++k)
        n += max(0, min(256, d - (int)((threadIdx.x >> 5) * 256 + k * blockDim.x * 8)));
    return (float)n;
}
template <int K>
__device__ __forceinline__ float2 bn_row_stats(const Bn8 (&v)[K], const bool (&in)[K], const BlockNormParams& p, float own_inv, BnShared& sh,
                                               int& turn) {
    const int nw = blockDim.x >> 5;
    const float per = 1.f / (float)p.d;
    float sum = 0.f, own = 0.f;  // the warp's sum and its mean
    if (!p.rms) {
        float2 s = bn_sum4(v[0]);
#pragma unroll
        for (int k = 1; k < K; ++k) s = bn_add(s, bn_sum4(v[k]));  // columns past d hold 0
        sum = bn_warp_sum(s.x + s.y);
        own = sum * own_inv;
    }
    float2 q = bn_f2(0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (!in[k]) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 c = bn_add(v[k].v[e], bn_f2(-own));
            q = bn_fma(c, c, q);
        }
    }
    const float squares = bn_warp_sum(q.x + q.y);
    if (nw == 1) return make_float2(own, rsqrtf(squares * per + p.eps));
    float4* r = sh.part[turn];
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) reinterpret_cast<float2*>(r)[threadIdx.x >> 5] = make_float2(sum, squares);
    __syncthreads();
    float2 total = bn_f2(0.f);
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        if (2 * w >= nw) break;
        const float4 a = r[w];
        total = bn_add(bn_add(total, make_float2(a.x, a.y)), make_float2(a.z, a.w));
    }
    const float mu = total.x * per;
    if (!p.rms) {
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            if (2 * w >= nw) break;
            const float4 a = r[w], n = sh.count[w];
            const float o0 = fmaf(a.x, n.y, -mu), o1 = fmaf(a.z, n.w, -mu);
            total.y = fmaf(n.x * o0, o0, fmaf(n.z * o1, o1, total.y));
        }
    }
    return make_float2(p.rms ? 0.f : mu, rsqrtf(total.y * per + p.eps));
}

template <typename TS, typename TU, int K, bool POST>
__global__ void __launch_bounds__(kBlockNormThreads) block_norm_fwd_run_kernel(const BlockNormParams p) {
    constexpr int NS = kBnFwdStages<TS, TU>, PIECES = kBnFwdPieces<TS, TU, K>, PS = kBnPieces<TS>, PU = kBnPieces<TU>;
    extern __shared__ __align__(16) unsigned char bn_smem[];
    __shared__ BnShared sh;
    int turn = 0;
    const int64_t b = blockIdx.y;
    const int seg = blockIdx.x, d = p.d, col0 = threadIdx.x * 8, step = blockDim.x * 8;
    // rows seg, seg + nseg, ...: the blocks move through memory together
    const int64_t r0 = b * p.L + seg, hop = (int64_t)p.nseg * d;
    const int rows = (int)((p.L - seg + p.nseg - 1) / p.nseg);
    const int stage_bytes = PIECES * blockDim.x * 16;
    const TS* x_in = static_cast<const TS*>(p.x) + r0 * d;   // the next row to copy
    const TU* u_in = p.u ? static_cast<const TU*>(p.u) + r0 * d : nullptr;
    bool in[K];
#pragma unroll
    for (int k = 0; k < K; ++k) in[k] = col0 + k * step < d;
    const int warp_col = (threadIdx.x >> 5) * 256;
    if (d != K * step || !p.u) bn_clear(bn_smem, NS * stage_bytes);
    auto fetch = [&](int row, int s) {
        if (row < rows) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                bn_fetch(bn_smem + s * stage_bytes, k * (PS + PU), x_in, warp_col + k * step, d);
                if (u_in) bn_fetch(bn_smem + s * stage_bytes, k * (PS + PU) + PS, u_in, warp_col + k * step, d);
            }
            x_in += hop;
            if (u_in) u_in += hop;
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < NS; ++s) fetch(s, s);
    BnVec<K, true> gate, post_w, gamma, beta;
    gate.start(p.gate ? p.gate + b * p.gate_bs : nullptr, 1.f, col0, step, d);
    if (POST) post_w.start(p.post_w, 1.f, col0, step, d);
    gamma.start(p.gamma ? p.gamma + b * p.gamma_bs : nullptr, 1.f, col0, step, d);
    beta.start(p.beta ? p.beta + b * p.gamma_bs : nullptr, 0.f, col0, step, d);
    const float2 res = bn_f2(p.res_scale);
    const float columns = bn_warp_columns<K>(d), own_inv = 1.f / fmaxf(columns, 1.f);
    bn_share(sh, columns);
    TS* x_out = p.x_out ? static_cast<TS*>(p.x_out) + r0 * d + col0 : nullptr;
    TU* y = p.y ? static_cast<TU*>(p.y) + r0 * d + col0 : nullptr;
    int s = 0;
    for (int row = 0; row < rows; ++row) {
        const unsigned char* const stage = bn_smem + s * stage_bytes;
        cp_async_wait_pending<NS - 1>();
        __syncwarp();
        Bn8 x[K], u[K];
        float2 sx = make_float2(0.f, 1.f), su = make_float2(0.f, 1.f);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            x[k] = bn_fetched<TS>(stage, k * (PS + PU));
            u[k] = bn_fetched<TU>(stage, k * (PS + PU) + PS);
        }
        __syncwarp();
        fetch(row + NS, s);
        s = s + 1 == NS ? 0 : s + 1;
        if constexpr (POST) su = bn_row_stats<K>(u, in, p, own_inv, sh, turn);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = col0 + k * step;
            const Bn8 g = gate.get(k, c);
            if constexpr (POST) {
                const Bn8 w = post_w.get(k, c);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    u[k].v[e] = bn_mul(bn_mul(bn_add(u[k].v[e], bn_f2(-su.x)), bn_f2(su.y)), w.v[e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) x[k].v[e] = bn_fma(g.v[e], u[k].v[e], bn_mul(res, x[k].v[e]));
            x[k] = bn_store8(x_out + k * step, x[k], x_out && in[k]);
        }
        if (y) {
            sx = bn_row_stats<K>(x, in, p, own_inv, sh, turn);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = col0 + k * step;
                const Bn8 g = gamma.get(k, c), be = beta.get(k, c);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[k].v[e] = bn_fma(g.v[e], bn_mul(bn_add(x[k].v[e], bn_f2(-sx.x)), bn_f2(sx.y)), be.v[e]);
                bn_store8(y + k * step, x[k], in[k]);
            }
            y += hop;
        }
        if (x_out) x_out += hop;
        if (p.stats && threadIdx.x == 0)
            reinterpret_cast<float4*>(p.stats)[r0 + (int64_t)row * p.nseg] = make_float4(sx.x, sx.y, su.x, su.y);
    }
    cp_async_wait_all();
}

template <typename TS, typename TU, int K, bool POST>
__global__ void __launch_bounds__(kBlockNormThreads) block_norm_bwd_run_kernel(const BlockNormParams p) {
    constexpr int NS = kBnBwdStages<TU, K>, PIECES = kBnBwdPieces<TS, TU, K>, PS = kBnPieces<TS>, PU = kBnPieces<TU>;
    extern __shared__ __align__(16) unsigned char bn_smem[];
    __shared__ BnShared sh;
    int turn = 0;
    const int64_t b = blockIdx.y;
    const int seg = blockIdx.x, d = p.d, col0 = threadIdx.x * 8, step = blockDim.x * 8;
    // rows seg, seg + nseg, ...: the blocks move through memory together
    const int64_t r0 = b * p.L + seg, hop = (int64_t)p.nseg * d;
    const int rows = (int)((p.L - seg + p.nseg - 1) / p.nseg);
    const int warp_col = (threadIdx.x >> 5) * 256;
    const int stage_bytes = PIECES * blockDim.x * 16;
    int64_t at = r0 * d;  // the next row to copy
    auto fetch = [&](int row, int s) {
        if (row < rows) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int q = k * 2 * (PS + PU), c = warp_col + k * step;
                unsigned char* const stage = bn_smem + s * stage_bytes;
                if (p.dy) {
                    bn_fetch(stage, q, static_cast<const TS*>(p.x) + at, c, d);
                    bn_fetch(stage, q + PS, static_cast<const TU*>(p.dy) + at, c, d);
                }
                if (p.dx_out) bn_fetch(stage, q + PS + PU, static_cast<const TS*>(p.dx_out) + at, c, d);
                if (p.u) bn_fetch(stage, q + 2 * PS + PU, static_cast<const TU*>(p.u) + at, c, d);
            }
            at += hop;
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < NS; ++s) fetch(s, s);
    BnVec<K, K == 1> gate, post_w, gamma;
    gate.start(p.gate ? p.gate + b * p.gate_bs : nullptr, 1.f, col0, step, d);
    if (POST) post_w.start(p.post_w, 1.f, col0, step, d);
    gamma.start(p.gamma ? p.gamma + b * p.gamma_bs : nullptr, 1.f, col0, step, d);
    const float per = 1.f / (float)d;
    const float2 res = bn_f2(p.res_scale);
    bn_share(sh, 0.f);
    Bn8 sg[K], sw[K], sm[K], sb[K];
#pragma unroll
    for (int k = 0; k < K; ++k) sg[k] = sw[k] = sm[k] = sb[k] = bn_fill(0.f);
    TS* dx = static_cast<TS*>(p.dx) + r0 * d + col0;
    TU* du = p.u ? static_cast<TU*>(p.du) + r0 * d + col0 : nullptr;
    const float4* stats = reinterpret_cast<const float4*>(p.stats) + r0;
    float4 ahead = rows > 0 ? stats[0] : make_float4(0.f, 0.f, 0.f, 0.f);
    int s = 0;
    for (int row = 0; row < rows; ++row) {
        const unsigned char* const stage = bn_smem + s * stage_bytes;
        const float4 st = ahead;
        if (row + 1 < rows) ahead = stats[(int64_t)(row + 1) * p.nseg];
        cp_async_wait_pending<NS - 1>();
        __syncwarp();
        Bn8 n[K], dy[K], D[K];
        float2 sum = bn_f2(0.f);
        if (p.dy) {
            float2 s1 = bn_f2(0.f), s2 = bn_f2(0.f);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = col0 + k * step, q = k * 2 * (PS + PU);
                if (c >= d) continue;
                n[k] = bn_fetched<TS>(stage, q);
                dy[k] = bn_fetched<TU>(stage, q + PS);
                const Bn8 ga = gamma.get(k, c);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    n[k].v[e] = bn_mul(bn_add(n[k].v[e], bn_f2(-st.x)), bn_f2(st.y));
                    sm[k].v[e] = bn_fma(dy[k].v[e], n[k].v[e], sm[k].v[e]);
                    sb[k].v[e] = bn_add(sb[k].v[e], dy[k].v[e]);
                    dy[k].v[e] = bn_mul(dy[k].v[e], ga.v[e]);
                    s1 = bn_add(s1, dy[k].v[e]);
                    s2 = bn_fma(dy[k].v[e], n[k].v[e], s2);
                }
            }
            sum = bn_block_sum2(make_float2(s1.x + s1.y, s2.x + s2.y), sh, turn);
            sum = make_float2(p.rms ? 0.f : sum.x * per, sum.y * per);
        }
        float2 t1 = bn_f2(0.f), t2 = bn_f2(0.f);
        Bn8 u[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = col0 + k * step, q = k * 2 * (PS + PU);
            if (c >= d) continue;
            D[k] = p.dx_out ? bn_fetched<TS>(stage, q + PS + PU) : bn_fill(0.f);
            if (p.dy) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    D[k].v[e] = bn_fma(bn_f2(st.y),
                                       bn_add(dy[k].v[e], bn_fma(n[k].v[e], bn_f2(-sum.y), bn_f2(-sum.x))), D[k].v[e]);
            }
            Bn8 o;
#pragma unroll
            for (int e = 0; e < 4; ++e) o.v[e] = bn_mul(res, D[k].v[e]);
            bn_store8(dx + k * step, o, true);
            if (!du) continue;
            u[k] = bn_fetched<TU>(stage, q + 2 * PS + PU);
            const Bn8 ga = gate.get(k, c);
            if constexpr (POST) {
                const Bn8 w = post_w.get(k, c);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 m = bn_mul(bn_add(u[k].v[e], bn_f2(-st.z)), bn_f2(st.w));
                    const float2 g = bn_mul(ga.v[e], D[k].v[e]), gw = bn_mul(g, w.v[e]);
                    sg[k].v[e] = bn_fma(D[k].v[e], bn_mul(m, w.v[e]), sg[k].v[e]);
                    sw[k].v[e] = bn_fma(g, m, sw[k].v[e]);
                    t1 = bn_add(t1, gw);
                    t2 = bn_fma(gw, m, t2);
                    u[k].v[e] = m;
                    D[k].v[e] = gw;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sg[k].v[e] = bn_fma(D[k].v[e], u[k].v[e], sg[k].v[e]);
                    o.v[e] = bn_mul(ga.v[e], D[k].v[e]);
                }
                bn_store8(du + k * step, o, true);
            }
        }
        __syncwarp();
        fetch(row + NS, s);
        s = s + 1 == NS ? 0 : s + 1;
        if constexpr (POST) {
            float2 tu = bn_block_sum2(make_float2(t1.x + t1.y, t2.x + t2.y), sh, turn);
            tu = make_float2(p.rms ? 0.f : tu.x * per, tu.y * per);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (col0 + k * step >= d) continue;
                Bn8 o;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o.v[e] = bn_mul(bn_f2(st.w), bn_add(D[k].v[e], bn_fma(u[k].v[e], bn_f2(-tu.y), bn_f2(-tu.x))));
                bn_store8(du + k * step, o, true);
            }
        }
        dx += hop;
        if (du) du += hop;
    }
    cp_async_wait_all();
    if (!p.part) return;
    float* q = p.part + ((int64_t)b * p.nseg + seg) * 4 * d;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = col0 + k * step;
        if (c >= d) continue;
        bn_store8(q + c, sg[k], true);
        bn_store8(q + d + c, sw[k], true);
        bn_store8(q + 2 * (int64_t)d + c, sm[k], true);
        bn_store8(q + 3 * (int64_t)d + c, sb[k], true);
    }
}

// ---------------------------------------------------------------- rows of any width, packed

// Rows that are no whole groups of eight, or too narrow for a warp.  A block
// takes a tile of neighbouring rows as the flat run of bytes that it is:
// 16-byte chunks copied ahead into one of two stages and, with the results
// in the places of the inputs, written back the same way, whatever the width.  A
// group of G lanes (4 to 32, or the whole block) has a row, E elements a lane,
// P of them (2 for even widths) in one access: lane g's j-th access is
// column (g + G j) P.

// A tile's bytes of one tensor: [at, at + bytes) from the 16-byte aligned base;
// in shared memory the chunk that holds `at` comes first.
struct BnRun {
    int64_t at;
    int bytes;
    __device__ __forceinline__ int head() const { return (int)(at & 15); }
    __device__ __forceinline__ int chunks() const { return (head() + bytes + 15) >> 4; }
};
// `end`: the tensor's bytes, past which nothing is read.
__device__ __forceinline__ void bn_copy_run(unsigned char* to, const void* base, BnRun r, int64_t end) {
    const char* from = static_cast<const char*>(base) + (r.at & ~15LL);
    const int64_t left = end - (r.at & ~15LL);
    for (int k = threadIdx.x; k < r.chunks(); k += blockDim.x) {
        const int n = left - 16LL * k < 16 ? (int)(left - 16LL * k) : 16;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(to) + 16 * k), "l"(from + 16LL * k),
                     "r"(n)
                     : "memory");
    }
}
template <typename T>
__device__ __forceinline__ void bn_store_run(const unsigned char* from, void* base, BnRun r) {
    char* to = static_cast<char*>(base) + (r.at & ~15LL);
    const int head = r.head(), tail = head + r.bytes;  // the chunks' bytes [head, tail) are the run's
    for (int k = threadIdx.x; k < r.chunks(); k += blockDim.x) {
        if (16 * k >= head && 16 * k + 16 <= tail) {
            *reinterpret_cast<uint4*>(to + 16LL * k) = *reinterpret_cast<const uint4*>(from + 16 * k);
        } else {
#pragma unroll
            for (int e = 0; e < 16; e += (int)sizeof(T))
                if (16 * k + e >= head && 16 * k + e < tail)
                    *reinterpret_cast<T*>(to + 16LL * k + e) = *reinterpret_cast<const T*>(from + 16 * k + e);
        }
    }
}

template <int P>
__device__ __forceinline__ void bn_get(const __nv_bfloat16* p, float* v) {
    if constexpr (P == 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
        v[0] = __uint_as_float(w << 16), v[1] = __uint_as_float(w & 0xffff0000u);
    } else {
        v[0] = __bfloat162float(*p);
    }
}
template <int P>
__device__ __forceinline__ void bn_get(const float* p, float* v) {
    if constexpr (P == 2) {
        const float2 w = *reinterpret_cast<const float2*>(p);
        v[0] = w.x, v[1] = w.y;
    } else {
        v[0] = *p;
    }
}
template <int P>
__device__ __forceinline__ void bn_set(__nv_bfloat16* p, const float* v) {
    if constexpr (P == 2)
        *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v[0], v[1]);
    else
        *p = __float2bfloat16_rn(v[0]);
}
template <int P>
__device__ __forceinline__ void bn_set(float* p, const float* v) {
    if constexpr (P == 2)
        *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    else
        *p = v[0];
}

// A lane's E elements of a row that starts for it at `from`, or of an fp32
// vector (`other` without it, 0 past d).  It has `mine` accesses, `step`
// elements apart; the elements of the others are 0.
template <int E, int P, typename T>
__device__ __forceinline__ void bn_gather(const T* from, float (&v)[E], int step, int mine) {
#pragma unroll
    for (int j = 0; j < E / P; ++j) {
#pragma unroll
        for (int e = 0; e < P; ++e) v[j * P + e] = 0.f;
        if (j < mine) bn_get<P>(from, v + j * P);
        from += step;
    }
}
template <int E, int P, typename T>
__device__ __forceinline__ void bn_scatter(T* to, const float (&v)[E], int step, int mine) {
#pragma unroll
    for (int j = 0; j < E / P; ++j) {
        if (j < mine) bn_set<P>(to, v + j * P);
        to += step;
    }
}
template <int E, int P>
__device__ __forceinline__ void bn_gather_vec(const float* p, float other, float (&v)[E], int g, int G, int d) {
#pragma unroll
    for (int j = 0; j < E / P; ++j)
#pragma unroll
        for (int e = 0; e < P; ++e) {
            const int c = (g + G * j) * P + e;
            v[j * P + e] = c < d ? (p ? p[c] : other) : 0.f;
        }
}
// The row's sums of a pair: G lanes, or (G = the block) through shared memory.
__device__ __forceinline__ float2 bn_group_sum2(float2 v, int G, BnShared& sh, int& turn) {
    if (G > 32) return bn_block_sum2(v, sh, turn);
    for (int off = G >> 1; off > 0; off >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, off);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, off);
    }
    return v;
}
template <int E, int P>
__device__ __forceinline__ float2 bn_group_stats(const float (&v)[E], const BlockNormParams& p, int mine, int G,
                                                 BnShared& sh, int& turn) {
    const float per = 1.f / (float)p.d;
    float mu = 0.f, q = 0.f;
    if (!p.rms) {
        float t = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) t += v[e];  // columns past d hold 0
        mu = bn_group_sum2(make_float2(t, 0.f), G, sh, turn).x * per;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float c = v[e] - mu;
        if (e / P < mine) q = fmaf(c, c, q);
    }
    return make_float2(mu, rsqrtf(bn_group_sum2(make_float2(q, 0.f), G, sh, turn).x * per + p.eps));
}

constexpr int kBnPackFwd = 16, kBnPackBwd = 8;  // E
// Bytes of a stage: `rows` rows of each tensor (chunks at both ends may be partial).
__host__ __device__ __forceinline__ int bn_pack_bytes(int rows, int d, int esz) { return (rows * d * esz + 31 + 15) / 16 * 16; }

template <typename TS, typename TU, int P, bool POST>
__global__ void __launch_bounds__(256, 2) block_norm_fwd_pack_kernel(const BlockNormParams p, const int G, const int R) {
    constexpr int E = kBnPackFwd;
    extern __shared__ __align__(16) unsigned char bn_smem[];
    __shared__ BnShared sh;
    int turn = 0;
    const int d = p.d, g = threadIdx.x % G, group = threadIdx.x / G, groups = blockDim.x / G;
    const int step = G * P, accesses = d > g * P ? (d - g * P + step - 1) / step : 0;
    const int64_t b = blockIdx.y, tiles = (p.L + R - 1) / R;
    const int xs = bn_pack_bytes(R, d, sizeof(TS)), us = bn_pack_bytes(R, d, sizeof(TU));
    const int64_t all = p.batch * p.L * d;
    const auto run = [&](int64_t tile, int esz) {
        const int64_t t0 = tile * R, n = p.L - t0 < R ? p.L - t0 : R;
        return BnRun{(b * p.L + t0) * d * esz, (int)n * d * esz};
    };
    const auto fetch = [&](int64_t tile, int s) {
        if (tile < tiles) {
            bn_copy_run(bn_smem + s * (xs + us), p.x, run(tile, sizeof(TS)), all * (int)sizeof(TS));
            if (p.u) bn_copy_run(bn_smem + s * (xs + us) + xs, p.u, run(tile, sizeof(TU)), all * (int)sizeof(TU));
        }
        cp_async_commit();
    };
    fetch(blockIdx.x, 0);
    float gate[E], gamma[E], beta[E], post_w[POST ? E : 1];
    bn_gather_vec<E, P>(p.gate ? p.gate + b * p.gate_bs : nullptr, 1.f, gate, g, G, d);
    if constexpr (POST) bn_gather_vec<E, P>(p.post_w, 1.f, post_w, g, G, d);
    bn_gather_vec<E, P>(p.gamma ? p.gamma + b * p.gamma_bs : nullptr, 1.f, gamma, g, G, d);
    bn_gather_vec<E, P>(p.beta ? p.beta + b * p.gamma_bs : nullptr, 0.f, beta, g, G, d);
    bn_share(sh, 0.f);
    int s = 0;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, s ^= 1) {
        const BnRun rx = run(tile, sizeof(TS)), ru = run(tile, sizeof(TU));
        const int n = rx.bytes / (d * (int)sizeof(TS));
        unsigned char* const stage = bn_smem + s * (xs + us);
        TS* const xt = reinterpret_cast<TS*>(stage + rx.head());
        TU* const ut = reinterpret_cast<TU*>(stage + xs + ru.head());
        cp_async_wait_all();
        __syncthreads();  // and the other stage's results are written back
        fetch(tile + gridDim.x, s ^ 1);
        // whole warps (or the block) go round together: a group without a row has one of no columns
        for (int r0 = 0; r0 < n; r0 += groups) {
            const bool own = r0 + group < n;
            const int r = own ? r0 + group : n - 1, mine = own ? accesses : 0;
            TS* const xr = xt + r * d + g * P;
            TU* const ur = ut + r * d + g * P;
            float x[E], u[E];
            float2 sx = make_float2(0.f, 1.f), su = make_float2(0.f, 1.f);
            bn_gather<E, P>(xr, x, step, mine);
            if (p.u) {
                bn_gather<E, P>(ur, u, step, mine);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) u[e] = 0.f;
            }
            if constexpr (POST) {
                su = bn_group_stats<E, P>(u, p, accesses, G, sh, turn);
#pragma unroll
                for (int e = 0; e < E; ++e) u[e] = (u[e] - su.x) * su.y * post_w[e];
            }
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = bn_round<TS>(fmaf(gate[e], u[e], p.res_scale * x[e]));
            if (p.x_out) bn_scatter<E, P>(xr, x, step, mine);
            if (p.y) {
                sx = bn_group_stats<E, P>(x, p, accesses, G, sh, turn);
#pragma unroll
                for (int e = 0; e < E; ++e) x[e] = fmaf(gamma[e], (x[e] - sx.x) * sx.y, beta[e]);
                bn_scatter<E, P>(ur, x, step, mine);
            }
            if (own && p.stats && g == 0) {
                float* st = p.stats + (b * p.L + tile * R + r) * 4;
                st[0] = sx.x, st[1] = sx.y, st[2] = su.x, st[3] = su.y;
            }
        }
        __syncthreads();
        if (p.x_out) bn_store_run<TS>(stage, p.x_out, rx);
        if (p.y) bn_store_run<TU>(stage + xs, p.y, ru);
    }
    cp_async_wait_all();
}

template <typename TS, typename TU, int P, bool POST>
__global__ void __launch_bounds__(512, 1) block_norm_bwd_pack_kernel(const BlockNormParams p, const int G, const int R) {
    constexpr int E = kBnPackBwd;
    extern __shared__ __align__(16) unsigned char bn_smem[];
    __shared__ BnShared sh;
    int turn = 0;
    const int d = p.d, g = threadIdx.x % G, group = threadIdx.x / G, groups = blockDim.x / G;
    const int step = G * P, accesses = d > g * P ? (d - g * P + step - 1) / step : 0;
    const int64_t b = blockIdx.y, tiles = (p.L + R - 1) / R;
    const int xs = bn_pack_bytes(R, d, sizeof(TS)), us = bn_pack_bytes(R, d, sizeof(TU));
    const int64_t all = p.batch * p.L * d;
    const auto run = [&](int64_t tile, int esz) {
        const int64_t t0 = tile * R, n = p.L - t0 < R ? p.L - t0 : R;
        return BnRun{(b * p.L + t0) * d * esz, (int)n * d * esz};
    };
    // x_out (then dx), dx_out, u (then du), dy
    const auto fetch = [&](int64_t tile, int s) {
        if (tile < tiles) {
            unsigned char* const stage = bn_smem + s * 2 * (xs + us);
            const BnRun rx = run(tile, sizeof(TS)), ru = run(tile, sizeof(TU));
            if (p.dy) bn_copy_run(stage, p.x, rx, all * (int)sizeof(TS));
            if (p.dx_out) bn_copy_run(stage + xs, p.dx_out, rx, all * (int)sizeof(TS));
            if (p.u) bn_copy_run(stage + 2 * xs, p.u, ru, all * (int)sizeof(TU));
            if (p.dy) bn_copy_run(stage + 2 * xs + us, p.dy, ru, all * (int)sizeof(TU));
        }
        cp_async_commit();
    };
    fetch(blockIdx.x, 0);
    float gate[E], gamma[E], post_w[POST ? E : 1], sg[E], sw[E], sm[E], sb[E];
    bn_gather_vec<E, P>(p.gate ? p.gate + b * p.gate_bs : nullptr, 1.f, gate, g, G, d);
    if constexpr (POST) bn_gather_vec<E, P>(p.post_w, 1.f, post_w, g, G, d);
    bn_gather_vec<E, P>(p.gamma ? p.gamma + b * p.gamma_bs : nullptr, 1.f, gamma, g, G, d);
#pragma unroll
    for (int e = 0; e < E; ++e) sg[e] = sw[e] = sm[e] = sb[e] = 0.f;
    bn_share(sh, 0.f);
    const float per = 1.f / (float)d;
    int s = 0;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, s ^= 1) {
        const BnRun rx = run(tile, sizeof(TS)), ru = run(tile, sizeof(TU));
        const int n = rx.bytes / (d * (int)sizeof(TS));
        unsigned char* const stage = bn_smem + s * 2 * (xs + us);
        TS* const xt = reinterpret_cast<TS*>(stage + rx.head());
        const TS* const dxt = reinterpret_cast<const TS*>(stage + xs + rx.head());
        TU* const ut = reinterpret_cast<TU*>(stage + 2 * xs + ru.head());
        const TU* const dyt = reinterpret_cast<const TU*>(stage + 2 * xs + us + ru.head());
        cp_async_wait_all();
        __syncthreads();
        fetch(tile + gridDim.x, s ^ 1);
        for (int r0 = 0; r0 < n; r0 += groups) {
            const bool own = r0 + group < n;
            const int r = own ? r0 + group : n - 1, mine = own ? accesses : 0, at = r * d + g * P;
            const float* st = p.stats + (b * p.L + tile * R + r) * 4;
            const float mu = st[0], rs = st[1], mu_u = st[2], rs_u = st[3];
            float D[E], u[E];
            if (p.dx_out) {
                bn_gather<E, P>(dxt + at, D, step, mine);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) D[e] = 0.f;
            }
            if (p.u) bn_gather<E, P>(ut + at, u, step, mine);
            if (p.dy) {
                float v[E], dy[E];
                float2 sum = make_float2(0.f, 0.f);
                bn_gather<E, P>(xt + at, v, step, mine);
                bn_gather<E, P>(dyt + at, dy, step, mine);  // 0 past d, and so is what follows from it
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    v[e] = (v[e] - mu) * rs;
                    sm[e] = fmaf(own ? dy[e] : 0.f, v[e], sm[e]);
                    sb[e] += own ? dy[e] : 0.f;
                    dy[e] *= gamma[e];
                    sum.x += dy[e];
                    sum.y = fmaf(dy[e], v[e], sum.y);
                }
                sum = bn_group_sum2(sum, G, sh, turn);
                sum = make_float2(p.rms ? 0.f : sum.x * per, sum.y * per);
#pragma unroll
                for (int e = 0; e < E; ++e) D[e] = fmaf(rs, dy[e] - fmaf(v[e], sum.y, sum.x), D[e]);
            }
            float o[E];
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = p.res_scale * D[e];
            bn_scatter<E, P>(xt + at, o, step, mine);
            if (!p.u) continue;
            if constexpr (POST) {
                float2 t = make_float2(0.f, 0.f);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float m = (u[e] - mu_u) * rs_u, q = gate[e] * D[e], w = post_w[e];  // gate, post_w 0 past d
                    if (own) {
                        sg[e] = fmaf(D[e], m * w, sg[e]);
                        sw[e] = fmaf(q, m, sw[e]);
                    }
                    t.x = fmaf(q, w, t.x);
                    t.y = fmaf(q * w, m, t.y);
                    u[e] = m;
                    D[e] = q * w;
                }
                t = bn_group_sum2(t, G, sh, turn);
                t = make_float2(p.rms ? 0.f : t.x * per, t.y * per);
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = rs_u * (D[e] - fmaf(u[e], t.y, t.x));
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    if (own) sg[e] = fmaf(D[e], u[e], sg[e]);
                    o[e] = gate[e] * D[e];
                }
            }
            bn_scatter<E, P>(ut + at, o, step, mine);
        }
        __syncthreads();
        bn_store_run<TS>(stage, p.dx, rx);
        if (p.u) bn_store_run<TU>(stage + 2 * xs, p.du, ru);
    }
    cp_async_wait_all();
    if (!p.part) return;
    // the groups' column sums, in order
    __syncthreads();
    float* const sums = reinterpret_cast<float*>(bn_smem);  // [groups][4][d]
    bn_scatter<E, P>(sums + (group * 4 + 0) * d + g * P, sg, step, accesses);
    bn_scatter<E, P>(sums + (group * 4 + 1) * d + g * P, sw, step, accesses);
    bn_scatter<E, P>(sums + (group * 4 + 2) * d + g * P, sm, step, accesses);
    bn_scatter<E, P>(sums + (group * 4 + 3) * d + g * P, sb, step, accesses);
    __syncthreads();
    float* q = p.part + ((int64_t)b * p.nseg + blockIdx.x) * 4 * d;
    for (int c = threadIdx.x; c < 4 * d; c += blockDim.x) {
        float t = 0.f;
        for (int k = 0; k < groups; ++k) t += sums[k * 4 * d + c];
        q[c] = t;
    }
}

// The column sums over the partial rows: of one batch row (blockIdx.z), or
// of all for the shared vectors.  blockIdx.y: which vector.  A block takes 32
// columns, each of its warps every sixteenth row; their sums are added in order.
constexpr int kBnSumWarps = 16;
__global__ void __launch_bounds__(kBnSumWarps * 32)
    block_norm_sums_kernel(const float* part, int nseg, int batch, int d, float* dgate, float* dpost_w, float* dgamma,
                           float* dbeta, int gate_shared, int gamma_shared) {
    __shared__ float sum[kBnSumWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane, which = blockIdx.y;
    float* out = which == 0 ? dgate : which == 1 ? dpost_w : which == 2 ? dgamma : dbeta;
    const bool shared = which == 1 || (which == 0 ? gate_shared : gamma_shared);
    const int64_t b = blockIdx.z;
    if (!out || (shared && b > 0)) return;
    const int64_t k0 = shared ? 0 : b * nseg, k1 = shared ? (int64_t)batch * nseg : k0 + nseg;
    float s = 0.f;
    if (c < d) {
#pragma unroll 4
        for (int64_t k = k0 + warp; k < k1; k += kBnSumWarps) s += part[(k * 4 + which) * d + c];
    }
    sum[warp][lane] = s;
    __syncthreads();
    if (warp || c >= d) return;
    s = 0.f;
    for (int w = 0; w < kBnSumWarps; ++w) s += sum[w][lane];
    out[(shared ? 0 : b * d) + c] = s;
}

}  // namespace bimamba

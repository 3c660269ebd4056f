// glr.cuh -- the gated linear recurrence, forward and backward.
//
// Per batch row and channel, over the row's tokens in scan order:
//   rg = sigmoid(r + r_bias), ig = sigmoid(i + i_bias), la = A rg (<= 0)
//   a = e^la,  beta = sqrt(1 - a^2),  h <- a h + beta ig x
//   out = (h + add) silu(z)
// and with dh = dout silu(z) and G_s = dh_s + a_{s+1} G_{s+1} (the state's
// gradient, scanned from the last step to the first), w = beta ig x:
//   dx = G beta ig              di = G w (1 - ig)
//   dla = G (a h_{s-1} - (a^2 / beta^2) w)    dr = A dla rg (1 - rg)
//   dA = sum rg dla             dr_bias = sum dr,  di_bias = sum di
//   dadd = dh                   dz = dout (h + add) silu'(z)
// (d beta / d la = -a^2 / beta, so that part of dla is (a^2 / beta^2) w).
//
// The backward recomputes the gates and the states from the inputs and the
// state that the forward saved every kGlrChunk steps (fp32, 4 / 64 bytes an
// element) instead of reading a stored h: that is less traffic than bf16
// states would be, and exact.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace bimamba {

constexpr int kGlrChunk = 64;
constexpr float kGlrLog2e = 1.4426950408889634f;

// Rows of one tensor: element (b, t, d) at p[b * bs + t * ts + d].
struct GlrRows {
    void* p;
    int64_t bs, ts;
};

struct GlrParams {
    GlrRows x, r, i, add, z, out;          // add.p, z.p may be null
    GlrRows dout, dx, dr, di, dadd, dz;    // backward
    const float* A;
    const float* r_bias;   // or null
    const float* i_bias;   // or null
    const int* lengths;    // or null
    const float* h_in;     // forward: state entering; or null
    float* h_out;          // or null
    float* chunk;          // [batch][nchunk][D]: forward writes (or null), backward reads
    const float* dh_out;   // or null
    float* dh_in;          // or null
    float* part;           // backward: [batch rows of partial sums][3][D]
    int64_t L;
    int D, batch, reverse;
    int64_t nchunk;        // ceil(L / kGlrChunk)
};

// ---------------------------------------------------------------- math

__device__ __forceinline__ float glr_ex2(float v) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
}
__device__ __forceinline__ float glr_rcp(float v) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
}
__device__ __forceinline__ float glr_sqrt(float v) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
}

// 1 / (1 + e^-v): e^-v may be +inf, whose reciprocal is 0.
__device__ __forceinline__ float glr_sigmoid(float v) { return glr_rcp(1.f + glr_ex2(-v * kGlrLog2e)); }

// 1 - a^2 = -expm1(t), t = 2 la <= 0, a = e^la.  Near 0 the difference would
// cancel, so down to t = -1/4 the Taylor series of expm1 to t^6 is taken (first
// omitted term t^6 / 5040 of the sum: 4.8e-8 at most); below, a^2 <= 0.78 and
// the subtraction loses two bits at most.
__device__ __forceinline__ float glr_one_minus_a2(float t, float a) {
    float s = fmaf(t, 1.f / 720.f, 1.f / 120.f);
    s = fmaf(t, s, 1.f / 24.f);
    s = fmaf(t, s, 1.f / 6.f);
    s = fmaf(t, s, 0.5f);
    s = fmaf(t, s, 1.f);
    return t > -0.25f ? -t * s : fmaf(-a, a, 1.f);
}

struct GlrGate {
    float rg, ig, a, b2;  // b2 = beta^2
};

__device__ __forceinline__ GlrGate glr_gate(float r, float i, float A) {
    GlrGate g;
    g.rg = glr_sigmoid(r);
    g.ig = glr_sigmoid(i);
    const float la = A * g.rg;
    g.a = glr_ex2(la * kGlrLog2e);
    g.b2 = glr_one_minus_a2(2.f * la, g.a);
    return g;
}

// ---------------------------------------------------------------- element I/O

template <typename T>
__device__ __forceinline__ float glr_ld(const GlrRows& q, int64_t b, int64_t t, int d) {
    const T* p = static_cast<const T*>(q.p) + b * q.bs + t * q.ts + d;
    return static_cast<float>(*p);
}
template <typename T>
__device__ __forceinline__ void glr_st(const GlrRows& q, int64_t b, int64_t t, int d, float v) {
    static_cast<T*>(q.p)[b * q.bs + t * q.ts + d] = static_cast<T>(v);  // bf16: to nearest even
}

__device__ __forceinline__ int64_t glr_len(const GlrParams& p, int64_t b) {
    if (!p.lengths) return p.L;
    const int64_t n = p.lengths[b];
    return n < 0 ? 0 : (n > p.L ? p.L : n);
}

// ---------------------------------------------------------------- one thread per channel

// The scan as the formula says it: a thread walks one channel of one batch row.
template <typename T>
__global__ void glr_fwd_kernel(const GlrParams p) {
    const int d = blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t b = blockIdx.y;
    if (d >= p.D) return;
    const int64_t len = glr_len(p, b);
    const float A = p.A[d], rb = p.r_bias ? p.r_bias[d] : 0.f, ib = p.i_bias ? p.i_bias[d] : 0.f;
    float h = p.h_in ? p.h_in[b * p.D + d] : 0.f;
    for (int64_t s = 0; s < len; ++s) {
        const int64_t t = p.reverse ? len - 1 - s : s;
        if (p.chunk && s % kGlrChunk == 0) p.chunk[(b * p.nchunk + s / kGlrChunk) * p.D + d] = h;
        const GlrGate g = glr_gate(glr_ld<T>(p.r, b, t, d) + rb, glr_ld<T>(p.i, b, t, d) + ib, A);
        h = fmaf(g.a, h, glr_sqrt(g.b2) * g.ig * glr_ld<T>(p.x, b, t, d));
        float y = h;
        if (p.add.p) y += glr_ld<T>(p.add, b, t, d);
        if (p.z.p) {
            const float z = glr_ld<T>(p.z, b, t, d);
            y *= z * glr_sigmoid(z);
        }
        glr_st<T>(p.out, b, t, d, y);
    }
    for (int64_t t = len; t < p.L; ++t) glr_st<T>(p.out, b, t, d, 0.f);
    if (p.h_out) p.h_out[b * p.D + d] = h;
}

// Chunk by chunk from the last: the states of the chunk from its saved first
// one, then the gradients from its last step to its first.
template <typename T>
__global__ void glr_bwd_kernel(const GlrParams p) {
    const int d = blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t b = blockIdx.y;
    if (d >= p.D) return;
    const int64_t len = glr_len(p, b);
    const float A = p.A[d], rb = p.r_bias ? p.r_bias[d] : 0.f, ib = p.i_bias ? p.i_bias[d] : 0.f;
    float q = p.dh_out ? p.dh_out[b * p.D + d] : 0.f;  // a_{s+1} G_{s+1}
    float sA = 0.f, sr = 0.f, si = 0.f;
    float hp[kGlrChunk];  // the state before each step
    for (int64_t c = (len + kGlrChunk - 1) / kGlrChunk - 1; c >= 0; --c) {
        const int64_t s0 = c * kGlrChunk;
        const int n = (int)(len - s0 < kGlrChunk ? len - s0 : kGlrChunk);
        float h = p.chunk[(b * p.nchunk + c) * p.D + d];
        for (int j = 0; j < n; ++j) {
            const int64_t t = p.reverse ? len - 1 - (s0 + j) : s0 + j;
            const GlrGate g = glr_gate(glr_ld<T>(p.r, b, t, d) + rb, glr_ld<T>(p.i, b, t, d) + ib, A);
            hp[j] = h;
            h = fmaf(g.a, h, glr_sqrt(g.b2) * g.ig * glr_ld<T>(p.x, b, t, d));
        }
        for (int j = n - 1; j >= 0; --j) {
            const int64_t t = p.reverse ? len - 1 - (s0 + j) : s0 + j;
            const GlrGate g = glr_gate(glr_ld<T>(p.r, b, t, d) + rb, glr_ld<T>(p.i, b, t, d) + ib, A);
            const float beta = glr_sqrt(g.b2), bi = beta * g.ig, w = bi * glr_ld<T>(p.x, b, t, d);
            float dh = glr_ld<T>(p.dout, b, t, d);
            if (p.add.p || p.z.p) {
                const float hs = fmaf(g.a, hp[j], w) + (p.add.p ? glr_ld<T>(p.add, b, t, d) : 0.f);
                if (p.z.p) {
                    const float z = glr_ld<T>(p.z, b, t, d), sz = glr_sigmoid(z);
                    glr_st<T>(p.dz, b, t, d, dh * hs * (sz * fmaf(z, 1.f - sz, 1.f)));
                    dh *= z * sz;
                }
                if (p.add.p) glr_st<T>(p.dadd, b, t, d, dh);
            }
            const float G = dh + q;
            const float ratio = beta > 0.f ? g.a * g.a * glr_rcp(g.b2) : 0.f;  // beta is 0 for a denormal b2 too
            const float dla = G * fmaf(g.a, hp[j], -ratio * w);
            const float dr = A * dla * g.rg * (1.f - g.rg), di = G * w * (1.f - g.ig);
            glr_st<T>(p.dx, b, t, d, G * bi);
            glr_st<T>(p.dr, b, t, d, dr);
            glr_st<T>(p.di, b, t, d, di);
            sA = fmaf(g.rg, dla, sA);
            sr += dr;
            si += di;
            q = g.a * G;
        }
    }
    for (int64_t t = len; t < p.L; ++t) {
        glr_st<T>(p.dx, b, t, d, 0.f);
        glr_st<T>(p.dr, b, t, d, 0.f);
        glr_st<T>(p.di, b, t, d, 0.f);
        if (p.add.p) glr_st<T>(p.dadd, b, t, d, 0.f);
        if (p.z.p) glr_st<T>(p.dz, b, t, d, 0.f);
    }
    if (p.dh_in) p.dh_in[b * p.D + d] = q;
    float* part = p.part + b * 3 * p.D + d;
    part[0] = sA;
    part[p.D] = sr;
    part[2 * p.D] = si;
}

// The three sums over the partial rows [n][3][D], in row order.
__global__ void glr_sums_kernel(const float* part, int64_t n, int D, float* dA, float* dr_bias, float* di_bias) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= 3 * D) return;
    float s = 0.f;
    for (int64_t k = 0; k < n; ++k) s += part[k * 3 * D + c];
    float* to = c < D ? dA : (c < 2 * D ? dr_bias : di_bias);
    if (to) to[c % D] = s;
}

}  // namespace bimamba

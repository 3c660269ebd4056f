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
    float* part;           // backward: [batch * nchunk][3][D] partial sums
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

// 0 for 0 and for what flushes to it, where beta = v * this is 0 as well
__device__ __forceinline__ float glr_rsqrt(float v) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return v < 1.17549435e-38f ? 0.f : y;
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

// ---------------------------------------------------------------- element I/O

__device__ __forceinline__ int64_t glr_len(const GlrParams& p, int64_t b) {
    if (!p.lengths) return p.L;
    const int64_t n = p.lengths[b];
    return n < 0 ? 0 : (n > p.L ? p.L : n);
}

// ---------------------------------------------------------------- pairs of channels

// A lane owns two neighbouring channels; its arithmetic is packed f32x2.
__device__ __forceinline__ float2 glr_f2(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 glr_mul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 glr_add(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 glr_fma(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// Two channels as they lie in memory: packed for bf16, so that a tile's
// loads in flight cost one register a pair.
template <typename T>
struct GlrRaw;
template <>
struct GlrRaw<__nv_bfloat16> {
    uint32_t v;
    __device__ __forceinline__ float2 get() const {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    }
};
template <>
struct GlrRaw<float> {
    float2 v;
    __device__ __forceinline__ float2 get() const { return v; }
};

// VEC: one access for the pair (channel count and strides even, pointers
// aligned to the pair); else one per channel, `n` (0..2) of them in range.
template <bool VEC>
__device__ __forceinline__ GlrRaw<__nv_bfloat16> glr_ld2(const __nv_bfloat16* p, int n) {
    GlrRaw<__nv_bfloat16> r;
    r.v = 0u;
    if constexpr (VEC) {
        if (n) r.v = __ldcs(reinterpret_cast<const unsigned int*>(p));
    } else {
        const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
        if (n > 0) r.v = q[0];
        if (n > 1) r.v |= (uint32_t)q[1] << 16;
    }
    return r;
}
template <bool VEC>
__device__ __forceinline__ GlrRaw<float> glr_ld2(const float* p, int n) {
    GlrRaw<float> r;
    r.v = make_float2(0.f, 0.f);
    if constexpr (VEC) {
        if (n) r.v = __ldcs(reinterpret_cast<const float2*>(p));
    } else {
        if (n > 0) r.v.x = p[0];
        if (n > 1) r.v.y = p[1];
    }
    return r;
}
template <bool VEC>
__device__ __forceinline__ void glr_st2(__nv_bfloat16* p, float2 v, int n) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);  // to nearest even
    if constexpr (VEC) {
        if (n) *reinterpret_cast<__nv_bfloat162*>(p) = h;
    } else {
        if (n > 0) p[0] = h.x;
        if (n > 1) p[1] = h.y;
    }
}
template <bool VEC>
__device__ __forceinline__ void glr_st2(float* p, float2 v, int n) {
    if constexpr (VEC) {
        if (n) *reinterpret_cast<float2*>(p) = v;
    } else {
        if (n > 0) p[0] = v.x;
        if (n > 1) p[1] = v.y;
    }
}
// fp32 vectors (parameters, states): always element by element, `n` of them.
__device__ __forceinline__ float2 glr_vec2(const float* p, int n) {
    return make_float2(p && n > 0 ? p[0] : 0.f, p && n > 1 ? p[1] : 0.f);
}
__device__ __forceinline__ void glr_put2(float* p, float2 v, int n) {
    if (n > 0) p[0] = v.x;
    if (n > 1) p[1] = v.y;
}

__device__ __forceinline__ float2 glr_sigmoid2(float2 v) { return make_float2(glr_sigmoid(v.x), glr_sigmoid(v.y)); }

struct GlrGate2 {
    float2 rg, ig, a, b2;
};
// r, i: raw activations; nr, ni: -bias log2 e.
__device__ __forceinline__ GlrGate2 glr_gate2(float2 r, float2 i, float2 nr, float2 ni, float2 A) {
    GlrGate2 g;
    const float2 er = glr_fma(r, glr_f2(-kGlrLog2e), nr), ei = glr_fma(i, glr_f2(-kGlrLog2e), ni);
    const float2 dr = glr_add(make_float2(glr_ex2(er.x), glr_ex2(er.y)), glr_f2(1.f));
    const float2 di = glr_add(make_float2(glr_ex2(ei.x), glr_ex2(ei.y)), glr_f2(1.f));
    g.rg = make_float2(glr_rcp(dr.x), glr_rcp(dr.y));
    g.ig = make_float2(glr_rcp(di.x), glr_rcp(di.y));
    const float2 la = glr_mul(A, g.rg), l2 = glr_mul(la, glr_f2(kGlrLog2e));
    g.a = make_float2(glr_ex2(l2.x), glr_ex2(l2.y));
    // glr_one_minus_a2, packed
    const float2 t = glr_add(la, la);
    float2 s = glr_fma(t, glr_f2(1.f / 720.f), glr_f2(1.f / 120.f));
    s = glr_fma(t, s, glr_f2(1.f / 24.f));
    s = glr_fma(t, s, glr_f2(1.f / 6.f));
    s = glr_fma(t, s, glr_f2(0.5f));
    s = glr_fma(t, s, glr_f2(1.f));
    const float2 mt = glr_mul(t, glr_f2(-1.f));
    const float2 near0 = glr_mul(mt, s), far = glr_fma(glr_mul(g.a, glr_f2(-1.f)), g.a, glr_f2(1.f));
    g.b2 = make_float2(t.x > -0.25f ? near0.x : far.x, t.y > -0.25f ? near0.y : far.y);
    return g;
}

// ---------------------------------------------------------------- tiles in scan order

// A block scans one tile: 64 channels (a lane has two) of NW warps x TOK
// steps.  Each warp scans its TOK steps from a zero state and keeps, per
// step, the decay since its first step and the state; the warps' affine maps
// (P, h) meet in shared memory, and with the state that enters the tile every
// output is P * state + h.  So the inputs are read once, all of a warp's
// loads are in flight together, and the chain over the sequence is one
// product-and-add per tile.
//
// Tiles of one row and channel slab hand over through the workspace, in groups
// of kGlrGroup: every tile publishes its map; the last of a group also
// publishes the state that enters the next group.  A tile reads that state
// and the maps of its group's earlier tiles and applies them in order, so the
// result is bit for bit that of the plain chain whatever the timing, while
// only one hop in kGlrGroup waits on another tile's wait.  A published pair is one
// 64-bit word (or a float each), written once over an all-ones fill that no
// result has (a NaN of that pattern is replaced), so it needs no flag and no
// fence.  Tiles are taken in ticket order, so whatever a tile waits for has
// started; every wait is bounded.
constexpr int kGlrSlab = 64;
constexpr int kGlrGroup = 8;
constexpr unsigned kGlrErrTimeout = 4u;  // a wait for an earlier tile gave up

static __device__ unsigned int g_glr_error;

struct GlrSync {
    unsigned int* ticket;        // all ones before the launch; null: one tile a row, nothing to hand over
    unsigned long long* map;     // [batch * slabs][tiles][64]: (P, h) of each channel
    float* state;                // [batch * slabs][groups][64]: state entering each group
    int64_t tiles, groups;
    long long wait_limit;
    int starve;                  // test aid: publish nothing
};

__device__ __forceinline__ unsigned glr_bits(float v) {
    const unsigned u = __float_as_uint(v);
    return u == 0xffffffffu ? 0x7fffffffu : u;
}
__device__ __forceinline__ void glr_publish_map(unsigned long long* q, float2 P, float2 h) {
    const unsigned long long v0 = (unsigned long long)glr_bits(h.x) << 32 | glr_bits(P.x);
    const unsigned long long v1 = (unsigned long long)glr_bits(h.y) << 32 | glr_bits(P.y);
    asm volatile("st.relaxed.gpu.global.v2.b64 [%0], {%1, %2};" ::"l"(q), "l"(v0), "l"(v1) : "memory");
}
__device__ __forceinline__ void glr_publish_state(float* q, float2 h) {
    asm volatile("st.relaxed.gpu.global.v2.b32 [%0], {%1, %2};" ::"l"(q), "r"(glr_bits(h.x)), "r"(glr_bits(h.y))
                 : "memory");
}

// The state entering tile `ti`: the group's entering state carried through
// the group's earlier maps.  map, state: of this row and slab, at the lane's
// pair.  Each lane waits for its own two channels.
__device__ __forceinline__ float2 glr_lookback(const GlrSync& y, const unsigned long long* map, const float* state,
                                               int64_t ti) {
    const int64_t g = ti / kGlrGroup, first = g * kGlrGroup;
    const int n = (int)(ti - first);
    unsigned long long m[kGlrGroup - 1][2];
    unsigned s0, s1;
    const long long t0 = clock64();
    bool ready = false;
    while (!ready) {
        asm volatile("ld.relaxed.gpu.global.v2.b32 {%0, %1}, [%2];"
                     : "=r"(s0), "=r"(s1)
                     : "l"(state + g * kGlrSlab)
                     : "memory");
        ready = s0 != 0xffffffffu && s1 != 0xffffffffu;
#pragma unroll
        for (int k = 0; k < kGlrGroup - 1; ++k) {
            if (k >= n) continue;
            asm volatile("ld.relaxed.gpu.global.v2.b64 {%0, %1}, [%2];"
                         : "=l"(m[k][0]), "=l"(m[k][1])
                         : "l"(map + (first + k) * kGlrSlab)
                         : "memory");
            // P lies in [0, 1] (or is NaN, 0x7fffffff): never the fill
            ready = ready && (unsigned)m[k][0] != 0xffffffffu && (unsigned)m[k][1] != 0xffffffffu;
        }
        if (!ready && clock64() - t0 > y.wait_limit) {
            atomicOr(&g_glr_error, kGlrErrTimeout);
            break;
        }
    }
    __syncwarp();
    float2 c = ready ? make_float2(__uint_as_float(s0), __uint_as_float(s1)) : make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kGlrGroup - 1; ++k) {
        if (k >= n || !ready) continue;
        const float2 P = make_float2(__uint_as_float((unsigned)m[k][0]), __uint_as_float((unsigned)m[k][1]));
        const float2 h = make_float2(__uint_as_float((unsigned)(m[k][0] >> 32)), __uint_as_float((unsigned)(m[k][1] >> 32)));
        c = glr_fma(P, c, h);
    }
    return c;
}

// Steps a warp scans: what its registers hold with two blocks of 256 threads on an SM.
template <typename T>
constexpr int kGlrTok = sizeof(T) == 2 ? 16 : 8;
constexpr int kGlrWarps = 8;

// The rest of a row behind its length: zeros from token t0 up to t1.
template <typename T, bool VEC>
__device__ __forceinline__ void glr_zero_rows(const GlrRows& q, int64_t b, int64_t t0, int64_t t1, int c0, int nch,
                                              int warp, int nwarp) {
    for (int64_t t = t0 + warp; t < t1; t += nwarp)
        glr_st2<VEC>(static_cast<T*>(q.p) + b * q.bs + t * q.ts + c0, make_float2(0.f, 0.f), nch);
}

template <typename T, bool VEC, bool EPI>
__global__ void __launch_bounds__(kGlrWarps * 32, 2) glr_tile_fwd_kernel(const GlrParams p, const GlrSync y) {
    constexpr int TOK = kGlrTok<T>;
    __shared__ float4 agg[kGlrWarps][32];
    __shared__ float2 enter[32];
    __shared__ unsigned ticket;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarp = blockDim.x >> 5;
    unsigned id = blockIdx.x;
    if (y.ticket) {
        if (threadIdx.x == 0) ticket = atomicAdd(y.ticket, 1u) + 1u;
        __syncthreads();
        id = ticket;
    }
    const int slabs = (p.D + kGlrSlab - 1) / kGlrSlab;
    const unsigned chains = (unsigned)slabs * p.batch, rs = id % chains;
    const int64_t ti = id / chains, b = rs / slabs;
    const int c0 = (int)(rs % slabs) * kGlrSlab + 2 * lane;
    const int nch = p.D - c0 > 1 ? 2 : (p.D - c0 > 0 ? 1 : 0);
    const int64_t len = glr_len(p, b), s0 = ti * (nwarp * TOK);
    const int64_t s1 = s0 + nwarp * TOK;  // the tile's steps [s0, s1)
    if (len < s1) glr_zero_rows<T, VEC>(p.out, b, len > s0 ? len : s0, s1 < p.L ? s1 : p.L, c0, nch, warp, nwarp);
    if (len <= s0) {  // nothing to scan, and no later tile of this row has anything either
        if (ti == 0 && warp == 0 && p.h_out)
            glr_put2(p.h_out + b * p.D + c0, glr_vec2(p.h_in ? p.h_in + b * p.D + c0 : nullptr, nch), nch);
        return;
    }

    const int64_t ws = s0 + warp * TOK;
    const int n = len - ws >= TOK ? TOK : (len > ws ? (int)(len - ws) : 0);
    const int64_t t0 = p.reverse ? len - 1 - ws : ws;  // the token of the warp's first step
    const int step = p.reverse ? -1 : 1;
    float2 Ps[TOK], hs[TOK];
    {
        GlrRaw<T> rx[TOK], rr[TOK], ri[TOK];
        const T* px = static_cast<const T*>(p.x.p) + b * p.x.bs + t0 * p.x.ts + c0;
        const T* pr = static_cast<const T*>(p.r.p) + b * p.r.bs + t0 * p.r.ts + c0;
        const T* pi = static_cast<const T*>(p.i.p) + b * p.i.bs + t0 * p.i.ts + c0;
        const int64_t ax = step * p.x.ts, ar = step * p.r.ts, ai = step * p.i.ts;
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
            const int m = j < n ? nch : 0;
            rx[j] = glr_ld2<VEC>(px + j * ax, m);
            rr[j] = glr_ld2<VEC>(pr + j * ar, m);
            ri[j] = glr_ld2<VEC>(pi + j * ai, m);
        }
        const float2 A = glr_vec2(p.A + c0, nch);
        const float2 nr = glr_mul(glr_vec2(p.r_bias ? p.r_bias + c0 : nullptr, nch), glr_f2(-kGlrLog2e));
        const float2 ni = glr_mul(glr_vec2(p.i_bias ? p.i_bias + c0 : nullptr, nch), glr_f2(-kGlrLog2e));
        float2 P = glr_f2(1.f), h = glr_f2(0.f);
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
            const GlrGate2 g = glr_gate2(rr[j].get(), ri[j].get(), nr, ni, A);
            const float2 beta = make_float2(glr_sqrt(g.b2.x), glr_sqrt(g.b2.y));
            float2 a = g.a, w = glr_mul(glr_mul(beta, g.ig), rx[j].get());
            if (j >= n) a = glr_f2(1.f), w = glr_f2(0.f);  // past the end: the state stays
            P = glr_mul(P, a);
            h = glr_fma(a, h, w);
            Ps[j] = P;
            hs[j] = h;
        }
        agg[warp][lane] = make_float4(P.x, h.x, P.y, h.y);
    }
    GlrRaw<T> ra[EPI ? TOK : 1], rz[EPI ? TOK : 1];
    if constexpr (EPI) {
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
            const int m = j < n ? nch : 0;
            const int64_t t = t0 + step * j;
            ra[j] = glr_ld2<VEC>(static_cast<const T*>(p.add.p) + b * p.add.bs + t * p.add.ts + c0, p.add.p ? m : 0);
            rz[j] = glr_ld2<VEC>(static_cast<const T*>(p.z.p) + b * p.z.bs + t * p.z.ts + c0, p.z.p ? m : 0);
        }
    }
    __syncthreads();
    if (warp == 0) {
        float2 P = glr_f2(1.f), h = glr_f2(0.f);
        for (int w = 0; w < nwarp; ++w) {
            const float4 q = agg[w][lane];
            const float2 Pw = make_float2(q.x, q.z);
            P = glr_mul(P, Pw);
            h = glr_fma(Pw, h, make_float2(q.y, q.w));
        }
        const bool last = s1 >= len, publish = y.ticket && !last && !y.starve;
        unsigned long long* map = y.map + (int64_t)rs * y.tiles * kGlrSlab + 2 * lane;
        float* state = y.state + (int64_t)rs * y.groups * kGlrSlab + 2 * lane;
        if (publish) glr_publish_map(map + ti * kGlrSlab, P, h);
        float2 c;
        if (ti == 0) {
            // the other tiles take it from here, not from h_in, which may be h_out
            c = glr_vec2(p.h_in ? p.h_in + b * p.D + c0 : nullptr, nch);
            if (publish) glr_publish_state(state, c);
        } else {
            c = glr_lookback(y, map, state, ti);
        }
        enter[lane] = c;
        const float2 end = glr_fma(P, c, h);
        if (publish && (ti + 1) % kGlrGroup == 0) glr_publish_state(state + (ti + 1) / kGlrGroup * kGlrSlab, end);
        if (last && p.h_out) glr_put2(p.h_out + b * p.D + c0, end, nch);
    }
    __syncthreads();
    float2 c = enter[lane];
    for (int w = 0; w < warp; ++w) {
        const float4 q = agg[w][lane];
        c = glr_fma(make_float2(q.x, q.z), c, make_float2(q.y, q.w));
    }
    if (p.chunk && n > 0 && ws % kGlrChunk == 0) glr_put2(p.chunk + (b * p.nchunk + ws / kGlrChunk) * p.D + c0, c, nch);
    T* po = static_cast<T*>(p.out.p) + b * p.out.bs + t0 * p.out.ts + c0;
    const int64_t ao = step * p.out.ts;
#pragma unroll
    for (int j = 0; j < TOK; ++j) {
        float2 h = glr_fma(Ps[j], c, hs[j]);
        if constexpr (EPI) {
            h = glr_add(h, ra[j].get());
            if (p.z.p) {
                const float2 z = rz[j].get();
                h = glr_mul(h, glr_mul(z, glr_sigmoid2(z)));
            }
        }
        glr_st2<VEC>(po + j * ao, h, j < n ? nch : 0);
    }
}

// Backward, one tile of kGlrChunk steps: the tiles are walked from the last
// step to the first (tile tj from the end of the row's own tiles), and what
// they hand over is q = a G, which the affine map of a tile takes from its
// right end to its left.  A warp's steps share one product P for both
// scans, the recomputed states (ascending, from the saved state that enters the tile)
// and q (descending).
constexpr int kGlrBwdTok = kGlrChunk / kGlrWarps;

template <typename T, bool VEC, bool EPI>
__global__ void __launch_bounds__(kGlrWarps * 32, 2) glr_tile_bwd_kernel(const GlrParams p, const GlrSync y) {
    constexpr int TOK = kGlrBwdTok;
    __shared__ float2 aggP[kGlrWarps][32], aggh[kGlrWarps][32], aggq[kGlrWarps][32];
    __shared__ float2 enter[32];
    __shared__ unsigned ticket;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned id = blockIdx.x;
    if (y.ticket) {
        if (threadIdx.x == 0) ticket = atomicAdd(y.ticket, 1u) + 1u;
        __syncthreads();
        id = ticket;
    }
    const int slabs = (p.D + kGlrSlab - 1) / kGlrSlab;
    const unsigned chains = (unsigned)slabs * p.batch, rs = id % chains;
    const int64_t tj = id / chains, b = rs / slabs;
    const int c0 = (int)(rs % slabs) * kGlrSlab + 2 * lane;
    const int nch = p.D - c0 > 1 ? 2 : (p.D - c0 > 0 ? 1 : 0);
    const int64_t len = glr_len(p, b), used = (len + kGlrChunk - 1) / kGlrChunk;  // the row's own tiles
    const int64_t ti = tj < used ? used - 1 - tj : tj;
    const int64_t s0 = ti * kGlrChunk, s1 = s0 + kGlrChunk;
    float* part = p.part + ((int64_t)b * p.nchunk + ti) * 3 * p.D + c0;
    if (len < s1) {
        const int64_t z0 = len > s0 ? len : s0, z1 = s1 < p.L ? s1 : p.L;
        glr_zero_rows<T, VEC>(p.dx, b, z0, z1, c0, nch, warp, kGlrWarps);
        glr_zero_rows<T, VEC>(p.dr, b, z0, z1, c0, nch, warp, kGlrWarps);
        glr_zero_rows<T, VEC>(p.di, b, z0, z1, c0, nch, warp, kGlrWarps);
        if (EPI && p.add.p) glr_zero_rows<T, VEC>(p.dadd, b, z0, z1, c0, nch, warp, kGlrWarps);
        if (EPI && p.z.p) glr_zero_rows<T, VEC>(p.dz, b, z0, z1, c0, nch, warp, kGlrWarps);
    }
    if (len <= s0) {
        if (warp < 3) glr_put2(part + (int64_t)warp * p.D, glr_f2(0.f), nch);
        if (tj == 0 && warp == 0 && p.dh_in)
            glr_put2(p.dh_in + b * p.D + c0, glr_vec2(p.dh_out ? p.dh_out + b * p.D + c0 : nullptr, nch), nch);
        return;
    }

    const int64_t ws = s0 + warp * TOK;
    const int n = len - ws >= TOK ? TOK : (len > ws ? (int)(len - ws) : 0);
    const int64_t t0 = p.reverse ? len - 1 - ws : ws;
    const int step = p.reverse ? -1 : 1;
    GlrRaw<T> rx[TOK], rd[TOK], ra[EPI ? TOK : 1], rz[EPI ? TOK : 1];
    float2 rg[TOK], ig[TOK], a[TOK], hp[TOK];
    const float2 A = glr_vec2(p.A + c0, nch);
    {
        GlrRaw<T> rr[TOK], ri[TOK];
        const T* px = static_cast<const T*>(p.x.p) + b * p.x.bs + t0 * p.x.ts + c0;
        const T* pr = static_cast<const T*>(p.r.p) + b * p.r.bs + t0 * p.r.ts + c0;
        const T* pi = static_cast<const T*>(p.i.p) + b * p.i.bs + t0 * p.i.ts + c0;
        const T* pd = static_cast<const T*>(p.dout.p) + b * p.dout.bs + t0 * p.dout.ts + c0;
        const int64_t ax = step * p.x.ts, ar = step * p.r.ts, ai = step * p.i.ts, ad = step * p.dout.ts;
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
            const int m = j < n ? nch : 0;
            rx[j] = glr_ld2<VEC>(px + j * ax, m);
            rr[j] = glr_ld2<VEC>(pr + j * ar, m);
            ri[j] = glr_ld2<VEC>(pi + j * ai, m);
            rd[j] = glr_ld2<VEC>(pd + j * ad, m);
            if constexpr (EPI) {
                const int64_t t = t0 + step * j;
                ra[j] = glr_ld2<VEC>(static_cast<const T*>(p.add.p) + b * p.add.bs + t * p.add.ts + c0, p.add.p ? m : 0);
                rz[j] = glr_ld2<VEC>(static_cast<const T*>(p.z.p) + b * p.z.bs + t * p.z.ts + c0, p.z.p ? m : 0);
            }
        }
        const float2 nr = glr_mul(glr_vec2(p.r_bias ? p.r_bias + c0 : nullptr, nch), glr_f2(-kGlrLog2e));
        const float2 ni = glr_mul(glr_vec2(p.i_bias ? p.i_bias + c0 : nullptr, nch), glr_f2(-kGlrLog2e));
        float2 P = glr_f2(1.f), h = glr_f2(0.f);
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
            const GlrGate2 g = glr_gate2(rr[j].get(), ri[j].get(), nr, ni, A);
            const float2 beta = make_float2(glr_sqrt(g.b2.x), glr_sqrt(g.b2.y));
            float2 w = glr_mul(glr_mul(beta, g.ig), rx[j].get());
            rg[j] = g.rg;
            ig[j] = g.ig;
            a[j] = g.a;
            if (j >= n) a[j] = glr_f2(1.f), w = glr_f2(0.f);
            hp[j] = h;  // the state before step j, from a zero state at the warp's first
            P = glr_mul(P, a[j]);
            h = glr_fma(a[j], h, w);
        }
        float2 q = glr_f2(0.f);
#pragma unroll
        for (int j = TOK - 1; j >= 0; --j) {
            float2 dh = rd[j].get();
            if constexpr (EPI) {
                if (p.z.p) dh = glr_mul(dh, glr_mul(rz[j].get(), glr_sigmoid2(rz[j].get())));
            }
            q = glr_mul(a[j], glr_add(q, dh));  // past the end dout reads as 0 and a is 1
        }
        aggP[warp][lane] = P;
        aggh[warp][lane] = h;
        aggq[warp][lane] = q;
    }
    __syncthreads();
    if (warp == 0) {
        float2 P = glr_f2(1.f), q = glr_f2(0.f);
        for (int w = kGlrWarps - 1; w >= 0; --w) {
            P = glr_mul(P, aggP[w][lane]);
            q = glr_fma(aggP[w][lane], q, aggq[w][lane]);
        }
        const bool last = ti == 0, publish = y.ticket && !last && !y.starve;
        unsigned long long* map = y.map + (int64_t)rs * y.tiles * kGlrSlab + 2 * lane;
        float* state = y.state + (int64_t)rs * y.groups * kGlrSlab + 2 * lane;
        if (publish) glr_publish_map(map + tj * kGlrSlab, P, q);
        float2 c;
        if (tj == 0) {
            c = glr_vec2(p.dh_out ? p.dh_out + b * p.D + c0 : nullptr, nch);
            if (publish) glr_publish_state(state, c);
        } else {
            c = glr_lookback(y, map, state, tj);
        }
        enter[lane] = c;
        const float2 end = glr_fma(P, c, q);
        if (publish && (tj + 1) % kGlrGroup == 0) glr_publish_state(state + (tj + 1) / kGlrGroup * kGlrSlab, end);
        if (last && p.dh_in) glr_put2(p.dh_in + b * p.D + c0, end, nch);
    }
    {
        // the states before the warp's steps, from the one that enters the tile
        float2 c = glr_vec2(p.chunk + (b * p.nchunk + ti) * p.D + c0, nch);
        for (int w = 0; w < warp; ++w) c = glr_fma(aggP[w][lane], c, aggh[w][lane]);
        float2 P = c;
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
            hp[j] = glr_add(P, hp[j]);
            P = glr_mul(P, a[j]);
        }
    }
    __syncthreads();
    float2 q = enter[lane];
    for (int w = kGlrWarps - 1; w > warp; --w) q = glr_fma(aggP[w][lane], q, aggq[w][lane]);
    __syncthreads();  // the maps are read: their place takes the sums below
    float2 sA = glr_f2(0.f), sr = glr_f2(0.f), si = glr_f2(0.f);
    const float2 one = glr_f2(1.f);
#pragma unroll
    for (int j = TOK - 1; j >= 0; --j) {
        const int m = j < n ? nch : 0;
        const int64_t t = t0 + step * j;
        const float2 la = glr_mul(A, rg[j]), t2 = glr_add(la, la);
        const float2 b2 = make_float2(glr_one_minus_a2(t2.x, a[j].x), glr_one_minus_a2(t2.y, a[j].y));
        const float2 rs2 = make_float2(glr_rsqrt(b2.x), glr_rsqrt(b2.y));
        const float2 bi = glr_mul(glr_mul(b2, rs2), ig[j]), w = glr_mul(bi, rx[j].get());
        float2 dh = rd[j].get();
        if constexpr (EPI) {
            if (p.z.p) {
                const float2 z = rz[j].get(), sz = glr_sigmoid2(z);
                const float2 h = glr_add(glr_fma(a[j], hp[j], w), ra[j].get());
                // silu'(z) = s (1 + z (1 - s))
                const float2 ds = glr_mul(sz, glr_fma(z, glr_fma(sz, glr_f2(-1.f), one), one));
                glr_st2<VEC>(static_cast<T*>(p.dz.p) + b * p.dz.bs + t * p.dz.ts + c0, glr_mul(glr_mul(dh, h), ds), m);
                dh = glr_mul(dh, glr_mul(z, sz));
            }
            if (p.add.p) glr_st2<VEC>(static_cast<T*>(p.dadd.p) + b * p.dadd.bs + t * p.dadd.ts + c0, dh, m);
        }
        const float2 G = glr_add(dh, q);
        q = glr_mul(a[j], G);
        // (a / beta)^2 w, with beta = 0 giving 0 (its 1/beta below is then 0 too)
        const float2 ar = glr_mul(a[j], rs2);
        const float2 dla = glr_mul(G, glr_fma(a[j], hp[j], glr_mul(glr_mul(ar, ar), glr_mul(w, glr_f2(-1.f)))));
        const float2 dr = glr_mul(glr_mul(A, dla), glr_mul(rg[j], glr_fma(rg[j], glr_f2(-1.f), one)));
        const float2 di = glr_mul(glr_mul(G, w), glr_fma(ig[j], glr_f2(-1.f), one));
        glr_st2<VEC>(static_cast<T*>(p.dx.p) + b * p.dx.bs + t * p.dx.ts + c0, glr_mul(G, bi), m);
        glr_st2<VEC>(static_cast<T*>(p.dr.p) + b * p.dr.bs + t * p.dr.ts + c0, dr, m);
        glr_st2<VEC>(static_cast<T*>(p.di.p) + b * p.di.bs + t * p.di.ts + c0, di, m);
        if (j < n) {
            sA = glr_fma(rg[j], dla, sA);
            sr = glr_add(sr, dr);
            si = glr_add(si, di);
        }
    }
    aggP[warp][lane] = sA;
    aggh[warp][lane] = sr;
    aggq[warp][lane] = si;
    __syncthreads();
    if (warp < 3) {
        const float2(*from)[32] = warp == 0 ? aggP : (warp == 1 ? aggh : aggq);
        float2 v = glr_f2(0.f);
        for (int w = 0; w < kGlrWarps; ++w) v = glr_add(v, from[w][lane]);
        glr_put2(part + (int64_t)warp * p.D, v, nch);
    }
}

// The three sums over the partial rows [n][3][D]: a block takes 32 columns, each
// of its 32 warps every 32nd row, and the warps' sums are added in order.
__global__ void __launch_bounds__(1024) glr_sums_kernel(const float* part, int64_t n, int D, float* dA, float* dr_bias,
                                                        float* di_bias) {
    __shared__ float sum[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane, wide = 3LL * D;
    float s = 0.f;
    if (c < wide) {
#pragma unroll 4
        for (int64_t k = warp; k < n; k += 32) s += part[k * wide + c];
    }
    sum[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < wide) {
        float v = 0.f;
        for (int w = 0; w < 32; ++w) v += sum[w][lane];
        float* to = c < D ? dA : (c < 2LL * D ? dr_bias : di_bias);
        if (to) to[c % D] = v;
    }
}

}  // namespace bimamba

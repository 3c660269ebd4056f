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

#include "tma_util.cuh"

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
    int copy;              // bytes of one asynchronous copy: 16, a pair of elements, or 0 (none possible)
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
__device__ __forceinline__ float glr_rsqrt(float v) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
}
// The larger of two, NaN if either is.
__device__ __forceinline__ float glr_max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// 1 / (1 + e^-v): e^-v may be +inf, whose reciprocal is 0.
__device__ __forceinline__ float glr_sigmoid(float v) { return glr_rcp(1.f + glr_ex2(-v * kGlrLog2e)); }

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

// u = 1 - 2^l for l <= 0, to fp32's relative accuracy however small |l| is, on
// the FP32 pipe (the special-function unit is the forward's scarcest): l =
// n + f with |f| <= 1/2 (n by adding and subtracting 1.5 2^23), 2^f - 1 = f p(f)
// with p of degree 5 (minimax of the relative error by Remez exchange, 1.1e-8),
// and u = (1 - 2^n) - 2^n (2^f - 1), where 1 - 2^n is exact or far from
// cancelling.  Below l = -126 the power is as good as 0.
__device__ __forceinline__ float2 glr_one_minus_ex2(float2 l) {
    constexpr float kMagic = 12582912.f;
    l = make_float2(glr_max_nan(l.x, -126.f), glr_max_nan(l.y, -126.f));
    const float2 m = glr_add(l, glr_f2(kMagic));
    const float2 f = glr_fma(glr_add(m, glr_f2(-kMagic)), glr_f2(-1.f), l);
    float2 q = glr_fma(f, glr_f2(0.00015403512225020677f), glr_f2(0.0013390735257416964f));
    q = glr_fma(f, q, glr_f2(0.009618237614631653f));
    q = glr_fma(f, q, glr_f2(0.05550357326865196f));
    q = glr_fma(f, q, glr_f2(0.24022649228572845f));
    q = glr_fma(f, q, glr_f2(0.6931471824645996f));
    q = glr_mul(f, q);
    // -2^n, its exponent from the low bits of m
    const float2 s = make_float2(__uint_as_float((__float_as_uint(m.x) << 23) + 0xbf800000u),
                                 __uint_as_float((__float_as_uint(m.y) << 23) + 0xbf800000u));
    return glr_fma(q, s, glr_add(s, glr_f2(1.f)));
}

// The gates of a pair: r, i raw activations; nr, ni: -bias log2 e; A2: A log2 e.
struct GlrGate2 {
    float2 rg, u, a, b2, di;  // a = 1 - u, b2 = beta^2 = 1 - a^2 = u (1 + a), ig = 1 / di
};
__device__ __forceinline__ GlrGate2 glr_gate2(float2 r, float2 i, float2 nr, float2 ni, float2 A2) {
    GlrGate2 g;
    const float2 er = glr_fma(r, glr_f2(-kGlrLog2e), nr), ei = glr_fma(i, glr_f2(-kGlrLog2e), ni);
    const float2 dr = glr_add(make_float2(glr_ex2(er.x), glr_ex2(er.y)), glr_f2(1.f));
    g.di = glr_add(make_float2(glr_ex2(ei.x), glr_ex2(ei.y)), glr_f2(1.f));
    g.rg = make_float2(glr_rcp(dr.x), glr_rcp(dr.y));
    g.u = glr_one_minus_ex2(glr_mul(A2, g.rg));
    g.a = glr_fma(g.u, glr_f2(-1.f), glr_f2(1.f));
    g.b2 = glr_mul(g.u, glr_add(g.a, glr_f2(1.f)));
    return g;
}
// The smallest normal, added under every 1 / beta: 0 / 0 becomes 0, and down to
// beta^2 = 1e-31 nothing else changes.
constexpr float kGlrTiny = 1.17549435e-38f;
// beta ig with one special function: b2 / sqrt(b2 di^2) = sqrt(b2) / di (where
// di^2 overflows, an input gate below e^-44, it counts as closed).
__device__ __forceinline__ float2 glr_beta_ig(float2 b2, float2 di) {
    const float2 v = glr_mul(glr_mul(glr_add(b2, glr_f2(kGlrTiny)), di), di);
    return glr_mul(b2, make_float2(glr_rsqrt(v.x), glr_rsqrt(v.y)));
}

// ---------------------------------------------------------------- tiles in scan order

// A block scans one tile at a time: 64 channels (a lane has two) of 8 warps x
// TOK steps.  Each warp scans its TOK steps from a zero state and keeps, per
// step, the decay since its first step and the state; the warps' affine maps
// (P, h) meet in shared memory, and with the state that enters the tile every
// output is P * state + h.  So the inputs are read once, and the chain over
// the sequence is one product-and-add per tile.
//
// Tiles of one row and channel slab hand over through the workspace, in groups
// of kGlrGroup: every tile publishes its map; the last of a group also
// publishes the state that enters the next group.  A tile reads that state
// and the maps of its group's earlier tiles and applies them in order, so the
// result is bit for bit that of the plain chain whatever the timing, while
// only one hop in kGlrGroup waits on another tile's wait.  A published pair is one
// 64-bit word (or a float each), written once over an all-ones fill that no
// result has (a NaN of that pattern is replaced), so it needs no flag and no
// fence.  Tiles are taken in ticket order and a block works through its own in
// that order, so whatever a tile waits for is being worked on; every wait is
// bounded, and once one has run out the launch's other waits end as well.
//
// Blocks stay (as many as the GPU holds) and take the next tile's ticket while
// they work on one.  Each warp copies the rows of its own steps into its own
// part of shared memory (cp.async, 16 bytes a lane), NS tiles ahead, so the
// copies overlap the arithmetic without a barrier: a warp waits for its own
// copies only.
constexpr int kGlrSlab = 64;
constexpr int kGlrGroup = 8;
constexpr unsigned kGlrErrTimeout = 4u;  // a wait for an earlier tile gave up

static __device__ unsigned int g_glr_error;

struct GlrSync {
    unsigned int* ticket;        // [0] the tickets, [1] set once a wait ran out; all ones before the launch.
                                 // Null: one tile a row, nothing to hand over
    unsigned long long* map;     // [batch * slabs][tiles][64]: (P, h) of each channel
    float* state;                // [batch * slabs][groups][64]: state entering each group
    int64_t tiles, groups;
    unsigned total;              // tiles of all rows and slabs
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
        if (ready) break;
        unsigned gone;
        asm volatile("ld.relaxed.gpu.global.b32 %0, [%1];" : "=r"(gone) : "l"(y.ticket + 1) : "memory");
        if (gone == 0u || clock64() - t0 > y.wait_limit) {
            atomicExch(y.ticket + 1, 0u);
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

// Where a tile lies.  `at` counts tiles along the row in the order in which
// they are walked.
struct GlrTile {
    unsigned rs;     // row * slabs + slab
    int64_t at, b, len;
    int c;           // first channel
};
__device__ __forceinline__ GlrTile glr_tile(const GlrParams& p, unsigned id) {
    const unsigned slabs = (unsigned)(p.D + kGlrSlab - 1) / kGlrSlab, chains = slabs * (unsigned)p.batch;
    GlrTile t;
    t.at = id / chains;
    t.rs = id % chains;
    t.b = t.rs / slabs;
    t.c = (int)(t.rs % slabs) * kGlrSlab;
    t.len = glr_len(p, t.b);
    return t;
}
// Steps of a row of `len` that start at ws, at most `most`.
__device__ __forceinline__ int glr_steps(int64_t len, int64_t ws, int most) {
    return len - ws >= most ? most : (len > ws ? (int)(len - ws) : 0);
}

// A warp's copy of n rows (of TOK) of one tensor into its place: row j is the
// token t0 + step * j.  The widest copies that the launch found possible;
// what lies past n or past the last channel becomes 0.
template <typename T, int TOK>
__device__ __forceinline__ void glr_copy_rows(T* to, const GlrRows& q, const GlrTile& t, int64_t t0, int step, int n,
                                              int D, int bytes) {
    const int lane = threadIdx.x & 31, left = D - t.c;
    const T* from = static_cast<const T*>(q.p) + t.b * q.bs + t0 * q.ts + t.c;
    const int64_t ts = step * q.ts;
    if (bytes == 16) {
        constexpr int E = 16 / sizeof(T), PER = kGlrSlab / E, ROWS = 32 / PER;  // elements a copy, copies a row
        const int c = lane % PER * E, r = lane / PER;
        const bool in = c < left;
#pragma unroll
        for (int k = 0; k < TOK / ROWS; ++k) {
            const int j = r + k * ROWS;
            const bool ok = in && j < n;
            cp_async<16>(to + j * kGlrSlab + c, ok ? from + j * ts + c : static_cast<const T*>(q.p), ok);
        }
    } else if (bytes) {
        const int c = 2 * lane;
#pragma unroll 4
        for (int j = 0; j < TOK; ++j) {
            const bool ok = c < left && j < n;
            cp_async<2 * sizeof(T)>(to + j * kGlrSlab + c, ok ? from + j * ts + c : static_cast<const T*>(q.p), ok);
        }
    } else {
        GlrRaw<T> v[TOK];
        const int c = 2 * lane, nch = left - c > 1 ? 2 : (left - c > 0 ? 1 : 0);
#pragma unroll
        for (int j = 0; j < TOK; ++j) v[j] = glr_ld2<false>(from + j * ts + c, j < n ? nch : 0);
#pragma unroll
        for (int j = 0; j < TOK; ++j) *reinterpret_cast<GlrRaw<T>*>(to + j * kGlrSlab + c) = v[j];
    }
}
// The lane's pair of row j.
template <typename T>
__device__ __forceinline__ float2 glr_row(const T* rows, int j) {
    return reinterpret_cast<const GlrRaw<T>*>(rows + j * kGlrSlab)[threadIdx.x & 31].get();
}

// Takes the block's first NS tiles; `slot` is shared memory.
template <int NS>
__device__ __forceinline__ void glr_first(const GlrSync& y, unsigned (&id)[NS], unsigned* slot) {
    if (y.ticket) {
        if (threadIdx.x == 0) {
#pragma unroll
            for (int k = 0; k < NS; ++k) slot[k] = atomicAdd(y.ticket, 1u) + 1u;
        }
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < NS; ++k) id[k] = y.ticket ? slot[k] : blockIdx.x + k * gridDim.x;
    __syncthreads();
}

// Stages of a block's copies: what two blocks on an SM leave room for.
template <bool EPI>
constexpr int kGlrFwdStages = EPI ? 1 : 2;
template <typename T, bool EPI>
constexpr int kGlrFwdWarpBytes = (3 * kGlrFwdStages<EPI> + (EPI ? 2 : 0)) * kGlrTok<T> * kGlrSlab * (int)sizeof(T);

template <typename T, bool VEC, bool EPI>
__global__ void __launch_bounds__(kGlrWarps * 32, 2) glr_tile_fwd_kernel(const GlrParams p, const GlrSync y) {
    constexpr int TOK = kGlrTok<T>, NS = kGlrFwdStages<EPI>, ROWS = TOK * kGlrSlab;
    extern __shared__ __align__(16) unsigned char glr_smem[];
    __shared__ float4 aggs[2][kGlrWarps][32];
    __shared__ float2 enter[32];
    __shared__ unsigned slot[2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarp = blockDim.x >> 5;
    T* const mine = reinterpret_cast<T*>(glr_smem + warp * kGlrFwdWarpBytes<T, EPI>);
    T* const epi = mine + 3 * NS * ROWS;
    const int step = p.reverse ? -1 : 1;
    const int tile_steps = nwarp * TOK;

    auto copy_inputs = [&](unsigned id, int stage) {
        if (id < y.total) {
            const GlrTile t = glr_tile(p, id);
            const int64_t ws = t.at * tile_steps + warp * TOK;
            const int n = glr_steps(t.len, ws, TOK);
            if (n) {
                const int64_t t0 = p.reverse ? t.len - 1 - ws : ws;
                T* to = mine + stage * 3 * ROWS;
                glr_copy_rows<T, TOK>(to, p.r, t, t0, step, n, p.D, p.copy);
                glr_copy_rows<T, TOK>(to + ROWS, p.i, t, t0, step, n, p.D, p.copy);
                glr_copy_rows<T, TOK>(to + 2 * ROWS, p.x, t, t0, step, n, p.D, p.copy);
            }
        }
        cp_async_commit();
    };

    unsigned ids[NS];
    glr_first<NS>(y, ids, slot);
#pragma unroll
    for (int k = 0; k < NS; ++k) copy_inputs(ids[k], k);
    int stage = 0, par = 0;
    while (ids[0] < y.total) {
        const GlrTile t = glr_tile(p, ids[0]);
        unsigned ahead = ids[NS - 1] + gridDim.x;
        if (y.ticket && threadIdx.x == 0) ahead = atomicAdd(y.ticket, 1u) + 1u;
        const int c0 = t.c + 2 * lane;
        const int nch = p.D - c0 > 1 ? 2 : (p.D - c0 > 0 ? 1 : 0);
        const int64_t b = t.b, len = t.len, s0 = t.at * tile_steps, s1 = s0 + tile_steps;  // the tile's steps [s0, s1)
        const int64_t ws = s0 + warp * TOK;
        const int n = glr_steps(len, ws, TOK);
        const int64_t t0 = p.reverse ? len - 1 - ws : ws;  // the token of the warp's first step
        if (len < s1) glr_zero_rows<T, VEC>(p.out, b, len > s0 ? len : s0, s1 < p.L ? s1 : p.L, c0, nch, warp, nwarp);
        if (len == 0 && s0 == 0 && warp == 0 && p.h_out)
            glr_put2(p.h_out + b * p.D + c0, glr_vec2(p.h_in ? p.h_in + b * p.D + c0 : nullptr, nch), nch);
        float4(*agg)[32] = aggs[par];
        float2 Ps[TOK], hs[TOK];
        cp_async_wait_pending<NS - 1>();
        __syncwarp();
        if constexpr (EPI) {
            // every lane is past its last tile's phase 2
            if (n && p.add.p) glr_copy_rows<T, TOK>(epi, p.add, t, t0, step, n, p.D, p.copy);
            if (n && p.z.p) glr_copy_rows<T, TOK>(epi + ROWS, p.z, t, t0, step, n, p.D, p.copy);
            cp_async_commit();
        }
        {
            const T* in = mine + stage * 3 * ROWS;
            const float2 A2 = glr_mul(glr_vec2(p.A + c0, nch), glr_f2(kGlrLog2e));
            const float2 nr = glr_mul(glr_vec2(p.r_bias ? p.r_bias + c0 : nullptr, nch), glr_f2(-kGlrLog2e));
            const float2 ni = glr_mul(glr_vec2(p.i_bias ? p.i_bias + c0 : nullptr, nch), glr_f2(-kGlrLog2e));
            float2 P = glr_f2(1.f), h = glr_f2(0.f);
#pragma unroll
            for (int j = 0; j < TOK; ++j) {
                const GlrGate2 g = glr_gate2(glr_row(in, j), glr_row(in + ROWS, j), nr, ni, A2);
                float2 a = g.a, w = glr_mul(glr_beta_ig(g.b2, g.di), glr_row(in + 2 * ROWS, j));
                if (j >= n) a = glr_f2(1.f), w = glr_f2(0.f);  // past the end: the state stays
                P = glr_mul(P, a);
                h = glr_fma(a, h, w);
                Ps[j] = P;
                hs[j] = h;
            }
            agg[warp][lane] = make_float4(P.x, h.x, P.y, h.y);
        }
        if (threadIdx.x == 0) slot[par] = ahead;
        __syncthreads();
        ahead = slot[par];
        if (len > s0 && warp == 0) {
            float2 P = glr_f2(1.f), h = glr_f2(0.f);
            for (int w = 0; w < nwarp; ++w) {
                const float4 q = agg[w][lane];
                const float2 Pw = make_float2(q.x, q.z);
                P = glr_mul(P, Pw);
                h = glr_fma(Pw, h, make_float2(q.y, q.w));
            }
            const bool last = s1 >= len, publish = y.ticket && !last && !y.starve;
            unsigned long long* map = y.map + (int64_t)t.rs * y.tiles * kGlrSlab + 2 * lane;
            float* state = y.state + (int64_t)t.rs * y.groups * kGlrSlab + 2 * lane;
            if (publish) glr_publish_map(map + t.at * kGlrSlab, P, h);
            float2 c;
            if (t.at == 0) {
                // the other tiles take it from here, not from h_in, which may be h_out
                c = glr_vec2(p.h_in ? p.h_in + b * p.D + c0 : nullptr, nch);
                if (publish) glr_publish_state(state, c);
            } else {
                c = glr_lookback(y, map, state, t.at);
            }
            enter[lane] = c;
            const float2 end = glr_fma(P, c, h);
            if (publish && (t.at + 1) % kGlrGroup == 0) glr_publish_state(state + (t.at + 1) / kGlrGroup * kGlrSlab, end);
            if (last && p.h_out) glr_put2(p.h_out + b * p.D + c0, end, nch);
        }
        copy_inputs(ahead, stage);
        if (len > s0) {
            __syncthreads();
            float2 c = enter[lane];
            for (int w = 0; w < warp; ++w) {
                const float4 q = agg[w][lane];
                c = glr_fma(make_float2(q.x, q.z), c, make_float2(q.y, q.w));
            }
            if (p.chunk && n > 0 && ws % kGlrChunk == 0)
                glr_put2(p.chunk + (b * p.nchunk + ws / kGlrChunk) * p.D + c0, c, nch);
            if constexpr (EPI) {
                cp_async_wait_pending<1>();  // all but the next tile's inputs
                __syncwarp();
            }
            T* po = static_cast<T*>(p.out.p) + b * p.out.bs + t0 * p.out.ts + c0;
            const int64_t ao = step * p.out.ts;
#pragma unroll
            for (int j = 0; j < TOK; ++j) {
                float2 h = glr_fma(Ps[j], c, hs[j]);
                if constexpr (EPI) {
                    if (p.add.p) h = glr_add(h, glr_row(epi, j));
                    if (p.z.p) {
                        const float2 z = glr_row(epi + ROWS, j);
                        h = glr_mul(h, glr_mul(z, glr_sigmoid2(z)));
                    }
                }
                glr_st2<VEC>(po + j * ao, h, j < n ? nch : 0);
            }
        }
        par ^= 1;
        if constexpr (NS == 2) {
            ids[0] = ids[1];
            stage ^= 1;
        }
        ids[NS - 1] = ahead;
    }
    cp_async_wait_all();
}

// Backward, tiles of kGlrChunk steps: they are walked from the last step to
// the first (tile `at` from the end of the row's own tiles), and what they
// hand over is q = a G, which the affine map of a tile takes from its right
// end to its left.  A warp's steps share one product P for both scans, the
// recomputed states (ascending, from the saved state that enters the tile)
// and q (descending).  The second half reads x, dout, add and z again from
// shared memory, so a warp's next copies start after it.
constexpr int kGlrBwdTok = kGlrChunk / kGlrWarps;
template <typename T>
constexpr int kGlrBwdStages = sizeof(T) == 2 ? 2 : 1;
template <typename T, bool EPI>
constexpr int kGlrBwdWarpBytes = (EPI ? 6 : 4) * kGlrBwdStages<T> * kGlrBwdTok * kGlrSlab * (int)sizeof(T);

template <typename T, bool VEC, bool EPI>
__global__ void __launch_bounds__(kGlrWarps * 32, 2) glr_tile_bwd_kernel(const GlrParams p, const GlrSync y) {
    constexpr int TOK = kGlrBwdTok, NS = kGlrBwdStages<T>, ROWS = TOK * kGlrSlab, NT = EPI ? 6 : 4;
    extern __shared__ __align__(16) unsigned char glr_smem[];
    __shared__ float2 aggP[kGlrWarps][32], aggh[kGlrWarps][32], aggq[kGlrWarps][32];
    __shared__ float2 sums[3][kGlrWarps][32];
    __shared__ float2 enter[32];
    __shared__ unsigned slot[2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    T* const mine = reinterpret_cast<T*>(glr_smem + warp * kGlrBwdWarpBytes<T, EPI>);
    const int step = p.reverse ? -1 : 1;
    const float2 one = glr_f2(1.f), minus = glr_f2(-1.f);

    // the tile's place along the row, in steps' order
    auto index_of = [](const GlrTile& t) {
        const int64_t used = (t.len + kGlrChunk - 1) / kGlrChunk;  // the row's own tiles
        return t.at < used ? used - 1 - t.at : t.at;
    };
    auto copy_inputs = [&](unsigned id, int stage) {
        if (id < y.total) {
            const GlrTile t = glr_tile(p, id);
            const int64_t ws = index_of(t) * kGlrChunk + warp * TOK;
            const int n = glr_steps(t.len, ws, TOK);
            if (n) {
                const int64_t t0 = p.reverse ? t.len - 1 - ws : ws;
                T* to = mine + stage * NT * ROWS;
                glr_copy_rows<T, TOK>(to, p.r, t, t0, step, n, p.D, p.copy);
                glr_copy_rows<T, TOK>(to + ROWS, p.i, t, t0, step, n, p.D, p.copy);
                glr_copy_rows<T, TOK>(to + 2 * ROWS, p.x, t, t0, step, n, p.D, p.copy);
                glr_copy_rows<T, TOK>(to + 3 * ROWS, p.dout, t, t0, step, n, p.D, p.copy);
                if (EPI && p.add.p) glr_copy_rows<T, TOK>(to + 4 * ROWS, p.add, t, t0, step, n, p.D, p.copy);
                if (EPI && p.z.p) glr_copy_rows<T, TOK>(to + 5 * ROWS, p.z, t, t0, step, n, p.D, p.copy);
            }
        }
        cp_async_commit();
    };

    unsigned ids[NS];
    glr_first<NS>(y, ids, slot);
#pragma unroll
    for (int k = 0; k < NS; ++k) copy_inputs(ids[k], k);
    int stage = 0, par = 0;
    while (ids[0] < y.total) {
        const GlrTile t = glr_tile(p, ids[0]);
        unsigned ahead = ids[NS - 1] + gridDim.x;
        if (y.ticket && threadIdx.x == 0) ahead = atomicAdd(y.ticket, 1u) + 1u;
        const int c0 = t.c + 2 * lane;
        const int nch = p.D - c0 > 1 ? 2 : (p.D - c0 > 0 ? 1 : 0);
        const int64_t b = t.b, len = t.len, ti = index_of(t), s0 = ti * kGlrChunk, s1 = s0 + kGlrChunk;
        const int64_t ws = s0 + warp * TOK;
        const int n = glr_steps(len, ws, TOK);
        const int64_t t0 = p.reverse ? len - 1 - ws : ws;
        float* part = p.part + (b * p.nchunk + ti) * 3 * p.D + c0;
        if (len < s1) {
            const int64_t z0 = len > s0 ? len : s0, z1 = s1 < p.L ? s1 : p.L;
            glr_zero_rows<T, VEC>(p.dx, b, z0, z1, c0, nch, warp, kGlrWarps);
            glr_zero_rows<T, VEC>(p.dr, b, z0, z1, c0, nch, warp, kGlrWarps);
            glr_zero_rows<T, VEC>(p.di, b, z0, z1, c0, nch, warp, kGlrWarps);
            if (EPI && p.add.p) glr_zero_rows<T, VEC>(p.dadd, b, z0, z1, c0, nch, warp, kGlrWarps);
            if (EPI && p.z.p) glr_zero_rows<T, VEC>(p.dz, b, z0, z1, c0, nch, warp, kGlrWarps);
        }
        const bool active = len > s0;
        if (!active) {
            if (warp < 3) glr_put2(part + (int64_t)warp * p.D, glr_f2(0.f), nch);
            if (t.at == 0 && warp == 0 && p.dh_in)
                glr_put2(p.dh_in + b * p.D + c0, glr_vec2(p.dh_out ? p.dh_out + b * p.D + c0 : nullptr, nch), nch);
        }
        const T* in = mine + stage * NT * ROWS;
        const T *in_x = in + 2 * ROWS, *in_d = in + 3 * ROWS, *in_add = in + 4 * ROWS, *in_z = in + 5 * ROWS;
        float2 rg[TOK], ig[TOK], u[TOK], hp[TOK];
        const float2 A = glr_vec2(p.A + c0, nch);
        float2 entering = glr_f2(0.f);
        if (active) entering = glr_vec2(p.chunk + (b * p.nchunk + ti) * p.D + c0, nch);
        cp_async_wait_pending<NS - 1>();
        __syncwarp();
        {
            const float2 nr = glr_mul(glr_vec2(p.r_bias ? p.r_bias + c0 : nullptr, nch), glr_f2(-kGlrLog2e));
            const float2 ni = glr_mul(glr_vec2(p.i_bias ? p.i_bias + c0 : nullptr, nch), glr_f2(-kGlrLog2e));
            const float2 A2 = glr_mul(A, glr_f2(kGlrLog2e));
            float2 P = one, h = glr_f2(0.f);
#pragma unroll
            for (int j = 0; j < TOK; ++j) {
                const GlrGate2 g = glr_gate2(glr_row(in, j), glr_row(in + ROWS, j), nr, ni, A2);
                float2 w = glr_mul(glr_beta_ig(g.b2, g.di), glr_row(in_x, j)), a = g.a;
                rg[j] = g.rg;
                ig[j] = make_float2(glr_rcp(g.di.x), glr_rcp(g.di.y));
                u[j] = g.u;
                if (j >= n) a = one, u[j] = w = glr_f2(0.f);
                hp[j] = h;  // the state before step j, from a zero state at the warp's first
                P = glr_mul(P, a);
                h = glr_fma(a, h, w);
            }
            float2 q = glr_f2(0.f);
#pragma unroll
            for (int j = TOK - 1; j >= 0; --j) {
                float2 dh = glr_row(in_d, j);
                if constexpr (EPI) {
                    if (p.z.p) {
                        const float2 z = glr_row(in_z, j);
                        dh = glr_mul(dh, glr_mul(z, glr_sigmoid2(z)));
                    }
                }
                if (j >= n) dh = glr_f2(0.f);
                const float2 G = glr_add(q, dh);
                q = glr_fma(u[j], glr_mul(G, minus), G);  // a G; past the end u is 0
            }
            aggP[warp][lane] = P;
            aggh[warp][lane] = h;
            aggq[warp][lane] = q;
        }
        if (threadIdx.x == 0) slot[par] = ahead;
        __syncthreads();
        ahead = slot[par];
        if (active) {
            if (warp == 0) {
                float2 P = one, q = glr_f2(0.f);
                for (int w = kGlrWarps - 1; w >= 0; --w) {
                    P = glr_mul(P, aggP[w][lane]);
                    q = glr_fma(aggP[w][lane], q, aggq[w][lane]);
                }
                const bool last = ti == 0, publish = y.ticket && !last && !y.starve;
                unsigned long long* map = y.map + (int64_t)t.rs * y.tiles * kGlrSlab + 2 * lane;
                float* state = y.state + (int64_t)t.rs * y.groups * kGlrSlab + 2 * lane;
                if (publish) glr_publish_map(map + t.at * kGlrSlab, P, q);
                float2 c;
                if (t.at == 0) {
                    c = glr_vec2(p.dh_out ? p.dh_out + b * p.D + c0 : nullptr, nch);
                    if (publish) glr_publish_state(state, c);
                } else {
                    c = glr_lookback(y, map, state, t.at);
                }
                enter[lane] = c;
                const float2 end = glr_fma(P, c, q);
                if (publish && (t.at + 1) % kGlrGroup == 0)
                    glr_publish_state(state + (t.at + 1) / kGlrGroup * kGlrSlab, end);
                if (last && p.dh_in) glr_put2(p.dh_in + b * p.D + c0, end, nch);
            }
            {
                // the states before the warp's steps, from the one that enters the tile
                float2 c = entering;
                for (int w = 0; w < warp; ++w) c = glr_fma(aggP[w][lane], c, aggh[w][lane]);
#pragma unroll
                for (int j = 0; j < TOK; ++j) {
                    hp[j] = glr_add(c, hp[j]);
                    c = glr_fma(u[j], glr_mul(c, minus), c);
                }
            }
            __syncthreads();
            float2 q = enter[lane];
            for (int w = kGlrWarps - 1; w > warp; --w) q = glr_fma(aggP[w][lane], q, aggq[w][lane]);
            float2 sA = glr_f2(0.f), sr = glr_f2(0.f), si = glr_f2(0.f);
#pragma unroll
            for (int j = TOK - 1; j >= 0; --j) {
                const int m = j < n ? nch : 0;
                const int64_t tk = t0 + step * j;
                const float2 a = glr_fma(u[j], minus, one), b2 = glr_mul(u[j], glr_add(a, one));
                const float2 b2t = glr_add(b2, glr_f2(kGlrTiny));
                const float2 rb = make_float2(glr_rsqrt(b2t.x), glr_rsqrt(b2t.y));  // 1 / beta
                const float2 bi = glr_mul(glr_mul(b2, rb), ig[j]), w = glr_mul(bi, glr_row(in_x, j));
                float2 dh = glr_row(in_d, j);
                if constexpr (EPI) {
                    if (p.z.p) {
                        const float2 z = glr_row(in_z, j), sz = glr_sigmoid2(z);
                        float2 h = glr_fma(a, hp[j], w);
                        if (p.add.p) h = glr_add(h, glr_row(in_add, j));
                        // silu'(z) = s (1 + z (1 - s))
                        const float2 ds = glr_mul(sz, glr_fma(z, glr_fma(sz, minus, one), one));
                        glr_st2<VEC>(static_cast<T*>(p.dz.p) + b * p.dz.bs + tk * p.dz.ts + c0,
                                     glr_mul(glr_mul(dh, h), ds), m);
                        dh = glr_mul(dh, glr_mul(z, sz));
                    }
                    if (p.add.p) glr_st2<VEC>(static_cast<T*>(p.dadd.p) + b * p.dadd.bs + tk * p.dadd.ts + c0, dh, m);
                }
                if (j >= n) continue;
                const float2 G = glr_add(dh, q);
                q = glr_mul(a, G);
                const float2 ab = glr_mul(a, rb);  // (a^2 / beta^2) w below
                const float2 dla = glr_mul(G, glr_fma(a, hp[j], glr_mul(glr_mul(ab, ab), glr_mul(w, minus))));
                const float2 dr = glr_mul(glr_mul(A, dla), glr_mul(rg[j], glr_fma(rg[j], minus, one)));
                const float2 di = glr_mul(glr_mul(G, w), glr_fma(ig[j], minus, one));
                glr_st2<VEC>(static_cast<T*>(p.dx.p) + b * p.dx.bs + tk * p.dx.ts + c0, glr_mul(G, bi), m);
                glr_st2<VEC>(static_cast<T*>(p.dr.p) + b * p.dr.bs + tk * p.dr.ts + c0, dr, m);
                glr_st2<VEC>(static_cast<T*>(p.di.p) + b * p.di.bs + tk * p.di.ts + c0, di, m);
                sA = glr_fma(rg[j], dla, sA);
                sr = glr_add(sr, dr);
                si = glr_add(si, di);
            }
            sums[0][warp][lane] = sA;
            sums[1][warp][lane] = sr;
            sums[2][warp][lane] = si;
        }
        __syncwarp();  // every lane has read its rows
        copy_inputs(ahead, stage);
        if (active) {
            __syncthreads();
            if (warp < 3) {
                float2 v = glr_f2(0.f);
                for (int w = 0; w < kGlrWarps; ++w) v = glr_add(v, sums[warp][w][lane]);
                glr_put2(part + (int64_t)warp * p.D, v, nch);
            }
        }
        par ^= 1;
        if constexpr (NS == 2) {
            ids[0] = ids[1];
            stage ^= 1;
        }
        ids[NS - 1] = ahead;
    }
    cp_async_wait_all();
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

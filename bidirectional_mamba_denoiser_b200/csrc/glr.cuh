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
// states would be, and rounds none of them to bf16.  A decay may be anything
// down to 0, and what it multiplies is as small, so a comes with its own
// relative accuracy and dla from the terms above, which both have a factor a
// (as h - w / beta^2 they would cancel to it, and leave the rounding of h).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include <type_traits>

#include "tma_util.cuh"

namespace bimamba {

constexpr int kGlrChunk = 64;
constexpr float kGlrLog2e = 1.4426950408889634f;

// Rows of one tensor: the element of channel 0 of (b, t) is at p + b * bs +
// t * |ts| bytes, and the next step's ts bytes on (ts < 0 in reverse).
struct GlrRows {
    char* p;
    int64_t bs;
    int ts;
};
enum {
    kGlrR, kGlrI, kGlrX, kGlrDout, kGlrAdd, kGlrZ,
    kGlrOut, kGlrDx = kGlrOut, kGlrDr, kGlrDi, kGlrDadd, kGlrDz, kGlrTensors
};

// Maps of the inputs and the backward's outputs: [batch][L][D], boxes of one warp's rows.
struct GlrMaps {
    CUtensorMap m[kGlrTensors];
};

struct GlrParams {
    GlrRows rows[kGlrTensors];  // p null where the call has none
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
    int copy;              // bytes of one cp.async: 16, a pair of elements, or 0 (none possible)
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
// The larger and the smaller of two, NaN if either is.
__device__ __forceinline__ float glr_max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float glr_min_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
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
__device__ __forceinline__ float2 glr_fma(float2 a, float2 b, float c) { return glr_fma(a, b, glr_f2(c)); }
__device__ __forceinline__ float2 glr_add(float2 a, float b) { return glr_add(a, glr_f2(b)); }
__device__ __forceinline__ float2 glr_sub(float2 a, float2 b) { return glr_fma(b, glr_f2(-1.f), a); }

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
    __device__ __forceinline__ float2 neg() const {
        return make_float2(__uint_as_float((v << 16) + 0x80000000u), __uint_as_float((v & 0xffff0000u) ^ 0x80000000u));
    }
};
template <>
struct GlrRaw<float> {
    float2 v;
    __device__ __forceinline__ float2 get() const { return v; }
    __device__ __forceinline__ float2 neg() const { return make_float2(-v.x, -v.y); }
};

// Stores of n (0..2) channels of a pair.  VEC: one access (channel count and
// strides even, pointers aligned to the pair, so n is 0 or 2).
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
// A pair of an fp32 vector, zeros where it is null.
template <bool VEC>
__device__ __forceinline__ float2 glr_vec2(const float* p, int64_t c, int n) {
    if (!p || n == 0) return make_float2(0.f, 0.f);
    if constexpr (VEC) return *reinterpret_cast<const float2*>(p + c);
    return make_float2(p[c], n > 1 ? p[c + 1] : 0.f);
}

__device__ __forceinline__ float2 glr_sigmoid2(float2 v) { return make_float2(glr_sigmoid(v.x), glr_sigmoid(v.y)); }

// 2^l - 1 for l <= 0, to fp32's relative accuracy however small |l| is, on the
// FP32 pipe (the special-function unit is the forward's scarcest): l = n + f
// with |f| <= 1/2 (n by adding and subtracting 1.5 2^23), 2^f - 1 = f p(f) with
// p of degree 5 (minimax of the relative error by Remez exchange, with its
// coefficients as fp32 holds them within 2.2e-8), and 2^l - 1 = (2^n - 1) + 2^n
// (2^f - 1), where 2^n - 1 is exact or far from cancelling.  `pow` is 2^l itself
// = 2^n + 2^n (2^f - 1): of 2^l - 1 it could not be had, whose rounding is all
// that is left of a small power.  Below l = -126.5 it is 0 (n = -127, whose 2^n
// has no bits).
__device__ __forceinline__ float2 glr_ex2m1(float2 l, float2& pow) {
    constexpr float kMagic = 12582912.f;
    l = make_float2(glr_max_nan(l.x, -127.f), glr_max_nan(l.y, -127.f));
    const float2 m = glr_add(l, kMagic);
    const float2 f = glr_sub(l, glr_add(m, -kMagic));
    float2 q = glr_fma(f, glr_f2(0.00015403512225020677f), 0.0013390735257416964f);
    q = glr_fma(f, q, 0.009618237614631653f);
    q = glr_fma(f, q, 0.05550357326865196f);
    q = glr_fma(f, q, 0.24022649228572845f);
    q = glr_fma(f, q, 0.6931471824645996f);
    q = glr_mul(f, q);
    // 2^n, its exponent from the low bits of m
    const float2 s = make_float2(__uint_as_float((__float_as_uint(m.x) << 23) + 0x3f800000u),
                                 __uint_as_float((__float_as_uint(m.y) << 23) + 0x3f800000u));
    pow = glr_fma(q, s, s);
    return glr_fma(q, s, glr_add(s, -1.f));
}

// The gates of a pair, most of them negated: so the products and sums below
// need no operand of ones, which costs two registers or two moves each time.
// r, i: raw activations; nr, ni: -bias log2 e; nA2: -A log2 e.
struct GlrGate2 {
    float2 nrg, a, nb2, di;  // -rg, a, -beta^2 = a^2 - 1, 1 / ig
};
__device__ __forceinline__ GlrGate2 glr_gate2(float2 r, float2 i, float2 nr, float2 ni, float2 nA2) {
    GlrGate2 g;
    const float2 er = glr_fma(r, glr_f2(-kGlrLog2e), nr), ei = glr_fma(i, glr_f2(-kGlrLog2e), ni);
    const float2 dr = glr_add(make_float2(glr_ex2(er.x), glr_ex2(er.y)), 1.f);
    g.di = glr_add(make_float2(glr_ex2(ei.x), glr_ex2(ei.y)), 1.f);
    g.nrg = make_float2(glr_rcp(-dr.x), glr_rcp(-dr.y));
    const float2 nu = glr_ex2m1(glr_mul(nA2, g.nrg), g.a);  // a - 1
    g.nb2 = glr_fma(nu, g.a, nu);
    return g;
}
// The smallest normal, added under every 1 / beta: 0 / 0 becomes 0, and down to
// beta^2 = 1e-31 nothing else changes.
constexpr float kGlrTiny = 1.17549435e-38f;
// a once more, from what the backward keeps of a gate.
__device__ __forceinline__ float2 glr_decay(float2 nA2, float2 nrg) {
    const float2 l = glr_mul(nA2, nrg);
    return make_float2(glr_ex2(l.x), glr_ex2(l.y));
}
// -beta ig with one special function: b2 / sqrt(b2 di^2) = sqrt(b2) / di (where
// di^2 overflows, an input gate below e^-44, it counts as closed).
__device__ __forceinline__ float2 glr_minus_beta_ig(float2 nb2, float2 di) {
    const float2 v = glr_mul(glr_mul(make_float2(kGlrTiny - nb2.x, kGlrTiny - nb2.y), di), di);
    return glr_mul(nb2, make_float2(glr_rsqrt(v.x), glr_rsqrt(v.y)));
}
// -beta alone, and 1 / beta of it (0 times it stays 0).
__device__ __forceinline__ float2 glr_minus_beta(float2 nb2) {
    return glr_mul(nb2, make_float2(glr_rsqrt(kGlrTiny - nb2.x), glr_rsqrt(kGlrTiny - nb2.y)));
}
__device__ __forceinline__ float2 glr_over_beta(float2 nb) {
    return make_float2(glr_rcp(1e-24f - nb.x), glr_rcp(1e-24f - nb.y));
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
// only one hop in kGlrGroup waits on another tile's wait.  Each warp fetches one
// of the eight pieces, asked for before its steps and looked at after them, so
// what is there already costs no latency.  Where rows and slabs are so many
// that a tile's predecessor is done long before its turn, a group is one tile:
// only states are handed over.  A published pair is one 64-bit word
// (or a float each), written once over an all-ones fill that no result has (a
// NaN of that pattern is replaced), so it needs no flag and no fence.  Tiles
// are taken in ticket order and a block works through its own in that order,
// so whatever a tile waits for is being worked on; every wait is bounded, and
// once one has run out the launch's other waits end as well.
//
// Blocks stay (as many as the GPU holds) and take the next tile's ticket while
// they work on one.  Each warp copies the rows of its own steps into its own
// part of shared memory, NS tiles ahead, so the copies overlap the arithmetic
// without a block barrier: a warp waits for its own copies only.  Long calls
// copy by tensor maps, one box a tensor that one lane asks for (in reverse the
// box's rows are the steps backwards); others by cp.async, whose addresses cost
// the warp some 20 instructions a tensor.
//
// What bounds it and what the choices measured (b 8, L 2048, D 4096 bf16; its
// 537 MB take 82 us at 6.56 TB/s):
//   one thread a channel, step after step                    1339 us
//   a block a tile, loads to registers                        360
//   blocks that stay, rows copied ahead                        234
//   pieces asked for early, offsets a tile once, full tiles
//   without selects                                            151
//   copies by maps                                             137
//   states alone handed over, one barrier                      131
// Special functions take 59 us, the copies alone 109 us with the gates left
// out; issue slots are 60 % used by 16 warps of 128 registers, some 30 of 81
// instructions a pair and step being the gates'.  Shorter warps' runs would
// spread a tile's fixed instructions (some 300 a warp) over fewer steps, longer
// ones do not fit the registers.  Scalar constants in place of packed ones: the
// same time.
constexpr int kGlrSlab = 64;
constexpr int kGlrGroup = 8;
static_assert(kGlrGroup == 8, "a piece for each warp");
constexpr unsigned kGlrErrTimeout = 4u;  // a wait for an earlier tile gave up

static __device__ unsigned int g_glr_error;

constexpr int kGlrPad = 16, kGlrGone = 32;  // other sectors

struct GlrSync {
    unsigned int* ticket;        // [0] the tickets, [kGlrPad] those of glr_pad, [kGlrGone] zero once a wait ran
                                 // out; all ones before the launch.  Null: one tile a row, nothing to hand over
    unsigned long long* map;     // [batch * slabs][tiles][64]: (P, h) of each channel
    float* state;                // [batch * slabs][groups][64]: state entering each group
    int64_t tiles, groups;
    int shift;                   // a group is 1 << shift tiles: kGlrGroup, or one
    unsigned total;              // tiles of all rows and slabs
    int4* plan;                  // padded batches with a hand-over: [0] {count}, then the tiles that have steps in
                                 // ticket order, {at, row, length}; else null
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

// Steps a warp scans: what its registers hold with two blocks of 256 threads on an SM.
template <typename T>
constexpr int kGlrTok = sizeof(T) == 2 ? 16 : 8;
constexpr int kGlrWarps = 8;

// Where a tile lies: `at` counts tiles along the row in the order in which
// they are walked (below 0: there is none), rs is row * slabs + slab.
struct GlrTile {
    int at, rs, b, len;
};
__device__ __forceinline__ int glr_slabs(const GlrParams& p) { return (p.D + kGlrSlab - 1) / kGlrSlab; }
__device__ __forceinline__ GlrTile glr_tile(const GlrParams& p, const GlrSync& y, unsigned id) {
    if (id >= y.total) return {-1, 0, 0, 0};
    const unsigned slabs = glr_slabs(p), chains = slabs * (unsigned)p.batch;
    GlrTile t;
    if (y.plan) {
        const int4 e = y.plan[1 + id / slabs];  // (in range: id < total)
        if (id / slabs >= (unsigned)y.plan[0].x) return {-1, 0, 0, 0};
        t.at = e.x, t.b = e.y, t.len = e.z;
        t.rs = t.b * (int)slabs + (int)(id % slabs);
        return t;
    }
    t.at = (int)(id / chains);
    t.rs = (int)(id % chains);
    t.b = t.rs / (int)slabs;
    t.len = (int)glr_len(p, t.b);
    return t;
}
__device__ __forceinline__ int glr_channel(const GlrParams& p, const GlrTile& t) {
    return (t.rs - t.b * glr_slabs(p)) * kGlrSlab;
}
// What a warp fetches for a tile that is not its row's first: warp w < 7 the
// map of the group's tile w, warp 7 the state that enters the group.
struct GlrPiece {
    unsigned long long v[2];
};
// The lane's place in the map of the row's tile `at`, and in the state that enters its group.
__device__ __forceinline__ unsigned long long* glr_map(const GlrSync& y, const GlrTile& t, int at) {
    return y.map + (t.rs * y.tiles + at) * kGlrSlab + 2 * (threadIdx.x & 31);
}
__device__ __forceinline__ float* glr_state(const GlrSync& y, const GlrTile& t, int at) {
    return y.state + (t.rs * y.groups + (at >> y.shift)) * kGlrSlab + 2 * (threadIdx.x & 31);
}
// Tiles of t's group before it.
__device__ __forceinline__ int glr_before(const GlrSync& y, const GlrTile& t) { return t.at & ((1 << y.shift) - 1); }
__device__ __forceinline__ void glr_ask(GlrPiece& q, const GlrSync& y, const GlrTile& t, int warp) {
    if (warp == kGlrGroup - 1) {
        unsigned s0, s1;
        asm volatile("ld.relaxed.gpu.global.v2.b32 {%0, %1}, [%2];"
                     : "=r"(s0), "=r"(s1)
                     : "l"(glr_state(y, t, t.at))
                     : "memory");
        q.v[0] = s0, q.v[1] = s1;
    } else if (warp < glr_before(y, t)) {
        asm volatile("ld.relaxed.gpu.global.v2.b64 {%0, %1}, [%2];"
                     : "=l"(q.v[0]), "=l"(q.v[1])
                     : "l"(glr_map(y, t, t.at - glr_before(y, t) + warp))
                     : "memory");
    } else {
        q.v[0] = q.v[1] = 0x3f800000ull;  // no such tile: P = 1, h = 0
    }
}
// The piece as (P, h) of the lane's two channels (the state as P = 0): waits
// until both are written.  P lies in [0, 1] (or is NaN, 0x7fffffff): never the fill.
__device__ __forceinline__ float4 glr_wait_piece(const GlrSync& y, GlrPiece q, const GlrTile& t, int warp) {
    if ((unsigned)q.v[0] == 0xffffffffu || (unsigned)q.v[1] == 0xffffffffu) {
        const long long t0 = clock64();
        for (int tries = 1;; ++tries) {
            glr_ask(q, y, t, warp);
            if ((unsigned)q.v[0] != 0xffffffffu && (unsigned)q.v[1] != 0xffffffffu) break;
            if (tries % 64) continue;  // the word that all waits share is looked at rarely
            unsigned gone;
            asm volatile("ld.relaxed.gpu.global.b32 %0, [%1];" : "=r"(gone) : "l"(y.ticket + kGlrGone) : "memory");
            if (gone == 0u || clock64() - t0 > y.wait_limit) {
                atomicExch(y.ticket + kGlrGone, 0u);
                atomicOr(&g_glr_error, kGlrErrTimeout);
                q.v[0] = q.v[1] = 0;
                break;
            }
        }
    }
    if (warp == kGlrGroup - 1)
        return make_float4(0.f, __uint_as_float((unsigned)q.v[0]), 0.f, __uint_as_float((unsigned)q.v[1]));
    return make_float4(__uint_as_float((unsigned)q.v[0]), __uint_as_float((unsigned)(q.v[0] >> 32)),
                       __uint_as_float((unsigned)q.v[1]), __uint_as_float((unsigned)(q.v[1] >> 32)));
}
// (P, h) of two channels applied to c.
__device__ __forceinline__ float2 glr_apply(float4 q, float2 c) {
    return glr_fma(make_float2(q.x, q.z), c, make_float2(q.y, q.w));
}

// c through the first n (at most 7) maps (all read at once).
__device__ __forceinline__ float2 glr_through(const float4 (*maps)[32], float2 c, int n) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int w = 0; w < 7; ++w) {
        const float4 q = maps[w][lane];
        if (w < n) c = glr_apply(q, c);
    }
    return c;
}

// The tile's first step (a row without tokens has one empty tile, or none).
// BWD: tiles are walked from the row's last to its first.
template <bool BWD>
__device__ __forceinline__ int64_t glr_first_step(const GlrTile& t, int tile_steps) {
    if constexpr (!BWD) return (int64_t)t.at * tile_steps;
    const int64_t used = t.len > 0 ? ((int64_t)t.len + tile_steps - 1) / tile_steps : 1;
    return (used - 1 - t.at) * tile_steps;
}

// The tiles of a block, in shared memory, a few ahead, each with the byte
// offset of its first step in every tensor (an offset: of an address out of
// shared memory the compiler would not know that it is global).  Warp 0 looks
// them up (each lane one tensor's offset) and takes a ticket a turn before it
// is looked up.
constexpr int kGlrQueue = 4;
struct GlrEntry {
    GlrTile t;
    int64_t off[kGlrTensors];
};
template <bool BWD, int ESZ>
struct GlrQueue {
    GlrEntry* q;
    int tile_steps;
    unsigned id;  // thread 0: the ticket to look up next
    __device__ __forceinline__ unsigned ticket(const GlrSync& y) {
        return y.ticket ? atomicAdd(y.ticket, 1u) + 1u : id + gridDim.x;
    }
    __device__ __forceinline__ void put(const GlrParams& p, const GlrSync& y, unsigned k) {
        if (threadIdx.x >= 32) return;
        GlrEntry& e = q[k % kGlrQueue];
        const GlrTile t = glr_tile(p, y, __shfl_sync(0xffffffffu, id, 0));
        if (threadIdx.x == 0) {
            id = ticket(y);
            e.t = t;
        }
        if (threadIdx.x < kGlrTensors && t.at >= 0) {
            const GlrRows& r = p.rows[threadIdx.x];
            const int64_t s = glr_first_step<BWD>(t, tile_steps);
            // in reverse the token of step s is len - 1 - s, and ts < 0
            const int64_t off = p.reverse ? (s - (t.len - 1)) * r.ts : s * r.ts;
            e.off[threadIdx.x] = t.b * r.bs + off + (int64_t)glr_channel(p, t) * ESZ;
        }
    }
    __device__ __forceinline__ void start(const GlrParams& p, const GlrSync& y, int n) {
        id = blockIdx.x - gridDim.x;
        if (threadIdx.x == 0) id = ticket(y);
        for (int k = 0; k < n; ++k) put(p, y, k);
        __syncthreads();
    }
};

// Before the tiles of a padded batch: the hand-over workspace's fill (`bytes`
// of ones), the states of rows without tokens, and the plan, which lists level
// by level the rows that have a tile there: before tile `at` of row b stand
// sum_j min(tiles_j, at) + #{j < b: tiles_j > at}.
__global__ void __launch_bounds__(256)
    glr_plan_kernel(const __grid_constant__ GlrParams p, uint4* fill, int64_t bytes, int4* plan, int64_t tiles,
                    int tile_steps) {
    __shared__ int before, count;
    for (int64_t k = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; k < bytes / 16; k += (int64_t)gridDim.x * blockDim.x)
        fill[k] = make_uint4(~0u, ~0u, ~0u, ~0u);
    for (int64_t item = blockIdx.x; item < p.batch * tiles; item += gridDim.x) {
        const int64_t b = item / tiles, len = glr_len(p, b);
        const int here = (int)(item % tiles);
        const bool there = len > (int64_t)here * tile_steps;
        if (plan && (there || item == 0)) {
            if (threadIdx.x == 0) before = count = 0;
            __syncthreads();
            int stand = 0, all = 0;
            for (int j = threadIdx.x; j < p.batch; j += blockDim.x) {
                const int own = (int)((glr_len(p, j) + tile_steps - 1) / tile_steps);
                stand += min(own, here) + (j < b && own > here);
                all += own;
            }
            atomicAdd(&before, stand);
            atomicAdd(&count, all);
            __syncthreads();
            if (threadIdx.x == 0) {
                if (there) plan[1 + before] = make_int4(here, (int)b, (int)len, 0);
                if (item == 0) plan[0] = make_int4(count, 0, 0, 0);
            }
            __syncthreads();
        }
        if (here == 0 && len == 0) {
            const float* from = p.part ? p.dh_out : p.h_in;
            float* to = p.part ? p.dh_in : p.h_out;
            if (to)
                for (int64_t k = threadIdx.x; k < p.D; k += blockDim.x) to[b * p.D + k] = from ? from[b * p.D + k] : 0.f;
        }
    }
}

// Zeros behind a padded row's length, kGlrPadTokens of one row at a time
// (`item` counts them), in every output and in the backward's partial sums: the
// work of blocks that find no more tiles, while the last chains still run.
constexpr int kGlrPadTokens = 16;
template <typename T>
__device__ __noinline__ void glr_pad_rows(const GlrParams& p, int64_t item) {
    const int64_t per_row = (p.L + kGlrPadTokens - 1) / kGlrPadTokens;
    const int64_t b = item / per_row, s0 = item % per_row * kGlrPadTokens, len = glr_len(p, b);
    const int64_t t0 = len > s0 ? len : s0, t1 = s0 + kGlrPadTokens < p.L ? s0 + kGlrPadTokens : p.L;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarp = blockDim.x >> 5;
    for (int q = kGlrOut; q < kGlrTensors; ++q) {
        const GlrRows& r = p.rows[q];
        if (!r.p) continue;
        const int64_t ts = r.ts < 0 ? -(int64_t)r.ts : r.ts;
        const bool wide = p.D * sizeof(T) % 16 == 0 && (reinterpret_cast<uintptr_t>(r.p) | r.bs | ts) % 16 == 0;
        for (int64_t t = t0 + warp; t < t1; t += nwarp) {
            char* const to = r.p + b * r.bs + t * ts;
            if (wide) {
                for (int k = lane; k < p.D / (16 / (int)sizeof(T)); k += 32)
                    reinterpret_cast<uint4*>(to)[k] = make_uint4(0u, 0u, 0u, 0u);
            } else {
                for (int k = lane; k < p.D; k += 32) reinterpret_cast<T*>(to)[k] = T(0.f);
            }
        }
    }
    if (p.part && len <= s0 && s0 % kGlrChunk == 0) {
        float* const part = p.part + (b * p.nchunk + s0 / kGlrChunk) * 3 * p.D;
        for (int64_t k = threadIdx.x; k < 3LL * p.D; k += blockDim.x) part[k] = 0.f;
    }
}
template <typename T>
__device__ __forceinline__ void glr_pad(const GlrParams& p, const GlrSync& y, unsigned* slot) {
    const int64_t items = p.batch * ((p.L + kGlrPadTokens - 1) / kGlrPadTokens);
    __syncthreads();
    for (int64_t k = blockIdx.x;; k += gridDim.x) {
        if (y.ticket) {
            if (threadIdx.x == 0) *slot = atomicAdd(y.ticket + kGlrPad, 1u) + 1u;
            __syncthreads();
            k = *slot;
            __syncthreads();
        }
        if (k >= items) break;
        glr_pad_rows<T>(p, k);
    }
}
// Steps of a row of `len` that start at ws, at most `most`.
__device__ __forceinline__ int glr_steps(int64_t len, int64_t ws, int most) {
    return len - ws >= most ? most : (len > ws ? (int)(len - ws) : 0);
}

// A warp's copy of n rows (of TOK) of some tensors into their places, one
// behind the other: row j is the tile's step first + j, `left` channels wide.
// The widest copies that the launch found possible; what lies past n or past
// the last channel becomes 0.
template <typename T, int TOK, int... TENSORS>
__device__ __forceinline__ void glr_copy_rows(T* to, const GlrParams& p, const GlrEntry& e, int first, int n, int left) {
    const int lane = threadIdx.x & 31;
    constexpr int E = 16 / sizeof(T), PER = kGlrSlab / E, ROWS = 32 / PER;  // elements a copy, copies a row
    if (p.copy == 16 && n == TOK && left >= kGlrSlab) {
        const int r = first + lane / PER, col = lane % PER * 16;
        uint32_t dst = smem_addr(to) + lane * 16;
        const auto one = [&](int tensor) {
            const int64_t ts = p.rows[tensor].ts;
            const char* from = p.rows[tensor].p + (e.off[tensor] + col) + r * ts;
#pragma unroll
            for (int k = 0; k < TOK / ROWS; ++k) {
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + k * 512), "l"(from) : "memory");
                from += ROWS * ts;
            }
            dst += TOK * kGlrSlab * sizeof(T);
        };
        (one(TENSORS), ...);
        return;
    }
    const auto one = [&](int tensor) {
        const char* const tile = p.rows[tensor].p + e.off[tensor];
        const int64_t ts = p.rows[tensor].ts;
        const int col = 2 * lane;
        if (p.copy == 16) {
            const int col = lane % PER * E, r = lane / PER;
            const char* from = tile + (first + r) * ts + col * sizeof(T);
            for (int k = 0; k < TOK / ROWS; ++k) {
                const bool ok = col < left && r + k * ROWS < n;
                cp_async<16>(to + (r + k * ROWS) * kGlrSlab + col, ok ? from + k * ROWS * ts : tile, ok);
            }
        } else if (p.copy) {
            const char* from = tile + first * ts + col * sizeof(T);
#pragma unroll 4
            for (int j = 0; j < TOK; ++j) {
                const bool ok = col < left && j < n;
                cp_async<2 * sizeof(T)>(to + j * kGlrSlab + col, ok ? from + j * ts : tile, ok);
            }
        } else {
            T v[TOK][2];
            const char* from = tile + first * ts + col * sizeof(T);
#pragma unroll
            for (int j = 0; j < TOK; ++j) {
                const T* q = reinterpret_cast<const T*>(from + j * ts);
                v[j][0] = j < n && col < left ? q[0] : T(0.f);
                v[j][1] = j < n && col + 1 < left ? q[1] : T(0.f);
            }
#pragma unroll
            for (int j = 0; j < TOK; ++j) to[j * kGlrSlab + col] = v[j][0], to[j * kGlrSlab + col + 1] = v[j][1];
        }
        to += TOK * kGlrSlab;
    };
    (one(TENSORS), ...);
}
// The same by maps, from step `first` of the row on, completing on `bar`; a
// warp without steps completes it with nothing.
template <typename T, int TOK, int... TENSORS>
__device__ __forceinline__ void glr_copy_boxes(T* to, const GlrMaps& maps, const GlrParams& p, const GlrTile& t,
                                               int64_t first, int n, int c, uint64_t* bar) {
    if ((threadIdx.x & 31) != 0) return;
    if (n == 0) {
        mbar_arrive(bar);
        return;
    }
    constexpr int BYTES = TOK * kGlrSlab * (int)sizeof(T);
    mbar_arrive_expect_tx(bar, ((p.rows[TENSORS].p ? BYTES : 0) + ...));
    const int t0 = (int)(p.reverse ? t.len - first - TOK : first);  // below 0: zeros
    const auto one = [&](int tensor) {
        if (p.rows[tensor].p) tma_load_3d(to, &maps.m[tensor], bar, c, t0, t.b);
        to += TOK * kGlrSlab;
    };
    (one(TENSORS), ...);
}
// Rows of results, from shared memory by one lane; a whole warp's steps only.
template <typename T>
__device__ __forceinline__ void glr_store_box(const T* from, const CUtensorMap& map, int c, int t0, int b) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(&map)),
                 "r"(smem_addr(from)), "r"(c), "r"(t0), "r"(b)
                 : "memory");
}
// The lane's boxes are read (its shared memory may be written again).
__device__ __forceinline__ void glr_boxes_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// Bounded, like every wait.
__device__ __forceinline__ void glr_wait_boxes(uint64_t* bar, unsigned parity) {
    if (mbar_try_wait(bar, parity)) return;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (clock64() - t0 > 4000000000LL) {
            atomicOr(&g_glr_error, kErrTmaTimeout);
            return;
        }
    }
}

// How a kernel's inputs come: by cp.async, or by maps forward or in reverse.
enum { kGlrAsync, kGlrMapForward, kGlrMapReverse };
// Where the row of a warp's step j lies: the rows of a box run with the tokens.
template <int TOK, int MODE>
struct GlrOrder {
    __device__ __forceinline__ constexpr int operator()(int j) const {
        return (MODE == kGlrMapReverse ? TOK - 1 - j : j) * kGlrSlab;
    }
};

// Steps past a warp's last keep the state: their rows in all NT tensors become
// zeros, but r = -inf, a closed gate, so that a = 1 and w = 0 without a select
// in the scan.
template <typename T, int TOK, int NT, int MODE>
__device__ __forceinline__ void glr_close_rows(T* rows, GlrOrder<TOK, MODE> at, int n) {
    const int lane = threadIdx.x & 31;
    for (int j = n; j < TOK; ++j)
        for (int q = 0; q < NT; ++q) {
            T* const to = rows + q * TOK * kGlrSlab + at(j);
            if constexpr (sizeof(T) == 2)
                reinterpret_cast<uint32_t*>(to)[lane] = q == 0 ? 0xff80ff80u : 0u;
            else
                reinterpret_cast<uint2*>(to)[lane] = q == 0 ? make_uint2(0xff800000u, 0xff800000u) : make_uint2(0u, 0u);
        }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // a box may overwrite them
}
// -bias log2 e, -A log2 e or -A of a pair, kept finite so that a closed gate wins.
__device__ __forceinline__ float2 glr_finite(float2 v) {
    return make_float2(glr_min_nan(glr_max_nan(v.x, -3.4e38f), 3.4e38f), glr_min_nan(glr_max_nan(v.y, -3.4e38f), 3.4e38f));
}
template <bool VEC>
__device__ __forceinline__ float2 glr_scaled(const float* v, int c, int nch, float by) {
    return glr_finite(glr_mul(glr_vec2<VEC>(v, c, nch), glr_f2(by)));
}
// The lane's pair of a row, and its negative.
template <typename T>
__device__ __forceinline__ float2 glr_minus_row(const T* row) {
    return reinterpret_cast<const GlrRaw<T>*>(row)[threadIdx.x & 31].neg();
}
template <typename T>
__device__ __forceinline__ float2 glr_row(const T* row) {
    return reinterpret_cast<const GlrRaw<T>*>(row)[threadIdx.x & 31].get();
}

// EPI: 0 out = h, 1 with add, 2 with z (an absent add is zero rows).
// Stages of a block's copies: what two blocks on an SM leave room for.
template <int EPI>
constexpr int kGlrFwdStages = EPI ? 1 : 2;
template <typename T, int EPI>
constexpr int kGlrFwdWarpBytes = (3 * kGlrFwdStages<EPI> + EPI) * kGlrTok<T> * kGlrSlab * (int)sizeof(T);

template <typename T, bool VEC, int EPI, int MODE>
__global__ void __launch_bounds__(kGlrWarps * 32, 2)
    glr_tile_fwd_kernel(const __grid_constant__ GlrParams p, const __grid_constant__ GlrSync y,
                        const __grid_constant__ GlrMaps maps) {
    constexpr int TOK = kGlrTok<T>, NS = kGlrFwdStages<EPI>, ROWS = TOK * kGlrSlab;
    extern __shared__ __align__(128) unsigned char glr_smem[];
    __shared__ float4 aggs[2][kGlrWarps][32];      // (P, h) of each warp
    __shared__ float4 pieces[2][kGlrGroup][32];    // what glr_ask fetched; [7] the state entering the group (or the row)
    __shared__ GlrEntry queue[kGlrQueue];
    __shared__ uint64_t bars[kGlrWarps][NS + 1];  // a warp's stages, and its add and z
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarp = blockDim.x >> 5;
    T* const mine = reinterpret_cast<T*>(glr_smem + warp * kGlrFwdWarpBytes<T, EPI>);
    T* const epi = mine + 3 * NS * ROWS;  // z, then add
    const int tile_steps = nwarp * TOK;
    constexpr bool by_map = MODE != kGlrAsync;
    constexpr GlrOrder<TOK, MODE> at;
    uint64_t* const bar = bars[warp];

    auto copy_inputs = [&](const GlrEntry& e, int stage) {
        const GlrTile t = e.t;
        const int64_t ws = (int64_t)t.at * tile_steps + warp * TOK;
        const int n = t.at < 0 ? 0 : glr_steps(t.len, ws, TOK);
        if constexpr (by_map) {
            glr_copy_boxes<T, TOK, kGlrR, kGlrI, kGlrX>(mine + stage * 3 * ROWS, maps, p, t, ws, n, glr_channel(p, t),
                                                        bar + stage);
        } else {
            const int left = p.D - glr_channel(p, t);
            if (n) glr_copy_rows<T, TOK, kGlrR, kGlrI, kGlrX>(mine + stage * 3 * ROWS, p, e, warp * TOK, n, left);
            cp_async_commit();
        }
    };

    if (by_map && threadIdx.x == 0) {
        for (int w = 0; w < nwarp; ++w)
            for (int k = 0; k <= NS; ++k) mbar_init(&bars[w][k], 1);
        fence_barrier_init();
    }
    GlrQueue<false, sizeof(T)> tiles{queue, tile_steps};
    tiles.start(p, y, NS);
    if (EPI == 2 && !p.rows[kGlrAdd].p) {
        for (int j = lane; j < ROWS; j += 32) epi[ROWS + j] = T(0.f);
    }
#pragma unroll
    for (int k = 0; k < NS; ++k) copy_inputs(queue[k], k);
    for (unsigned k = 0;; ++k) {
        const GlrEntry& e = queue[k % kGlrQueue];
        GlrTile t = e.t;
        if (t.at < 0) break;
        tiles.put(p, y, k + NS);  // over entry k + NS - 4, which every warp has left behind
        const int stage = NS == 2 ? k & 1 : 0;
        const int c0 = glr_channel(p, t) + 2 * lane;
        const int nch = p.D - c0 > 1 ? 2 : (p.D - c0 > 0 ? 1 : 0);
        const int64_t s0 = (int64_t)t.at * tile_steps, s1 = s0 + tile_steps;  // the tile's steps [s0, s1)
        const int64_t ws = s0 + warp * TOK, row = (int64_t)t.b * p.D + c0;
        const int n = glr_steps(t.len, ws, TOK);
        GlrPiece piece;
        if (t.at) glr_ask(piece, y, t, warp);
        float4(*agg)[32] = aggs[k & 1];
        float4(*got)[32] = pieces[k & 1];
        float2 Ps[TOK], hs[TOK];
        if constexpr (by_map)
            glr_wait_boxes(bar + stage, (k / NS) & 1);
        else
            cp_async_wait_pending<NS - 1>();
        __syncwarp();
        if constexpr (EPI > 0 && by_map) {
            const int c = c0 - 2 * lane;
            if constexpr (EPI == 1) glr_copy_boxes<T, TOK, kGlrAdd>(epi, maps, p, t, ws, n, c, bar + NS);
            if constexpr (EPI == 2) glr_copy_boxes<T, TOK, kGlrZ, kGlrAdd>(epi, maps, p, t, ws, n, c, bar + NS);
        } else if constexpr (EPI > 0) {
            // every lane is past its last tile's outputs
            const int left = p.D - (c0 - 2 * lane);
            if (EPI == 2 && n) glr_copy_rows<T, TOK, kGlrZ>(epi, p, e, warp * TOK, n, left);
            if (n && p.rows[kGlrAdd].p)
                glr_copy_rows<T, TOK, kGlrAdd>(epi + (EPI - 1) * ROWS, p, e, warp * TOK, n, left);
            cp_async_commit();
        }
        if (n) {
            T* in = mine + stage * 3 * ROWS;
            if (n < TOK) glr_close_rows<T, TOK, 3, MODE>(in, at, n);
            const float2 nA2 = glr_scaled<VEC>(p.A, c0, nch, -kGlrLog2e);
            const float2 nr = glr_scaled<VEC>(p.r_bias, c0, nch, -kGlrLog2e);
            const float2 ni = glr_scaled<VEC>(p.i_bias, c0, nch, -kGlrLog2e);
            float2 P = glr_f2(1.f), h = glr_f2(0.f);
#pragma unroll
            for (int j = 0; j < TOK; ++j) {
                const GlrGate2 g = glr_gate2(glr_row(in + at(j)), glr_row(in + ROWS + at(j)), nr, ni, nA2);
                const float2 w = glr_mul(glr_minus_beta_ig(g.nb2, g.di), glr_minus_row(in + 2 * ROWS + at(j)));
                P = glr_mul(P, g.a);
                h = glr_fma(g.a, h, w);
                Ps[j] = P;
                hs[j] = h;
            }
            agg[warp][lane] = make_float4(P.x, h.x, P.y, h.y);
        } else {
            agg[warp][lane] = make_float4(1.f, 0.f, 1.f, 0.f);
        }
        if (t.at == 0 && warp == nwarp - 1) {
            const float2 c = glr_vec2<VEC>(p.h_in, row, nch);
            got[kGlrGroup - 1][lane] = make_float4(0.f, c.x, 0.f, c.y);
        } else if (t.at && !y.shift && warp == kGlrGroup - 1) {
            // no map to publish first: the state is waited for before the barrier, the only one then
            got[kGlrGroup - 1][lane] = glr_wait_piece(y, piece, t, warp);
        }
        __syncthreads();
        t = e.t;  // (read again rather than kept)
        const bool last = s1 >= t.len, publish = y.ticket && !last && !y.starve;
        float2 P = glr_f2(1.f), h = glr_f2(0.f);
        if (warp == 0) {
#pragma unroll
            for (int w = 0; w < kGlrWarps; ++w) {
                const float4 q = agg[w][lane];
                if (w >= nwarp) continue;
                P = glr_mul(P, make_float2(q.x, q.z));
                h = glr_apply(q, h);
            }
            if (publish && y.shift) glr_publish_map(glr_map(y, t, t.at), P, h);
        }
        if (t.at && y.shift) {
            got[warp][lane] = glr_wait_piece(y, piece, t, warp);
            __syncthreads();
        }
        const float4 from = got[kGlrGroup - 1][lane];
        float2 c = make_float2(from.y, from.w);
        if (y.shift) c = glr_through(got, c, glr_before(y, t));
        if (warp == 0) {
            const float2 end = glr_fma(P, c, h);
            // the other tiles take a row's first state from here, not from h_in, which may be h_out
            if (publish && t.at == 0) glr_publish_state(glr_state(y, t, 0), c);
            if (publish && ((t.at + 1) & ((1 << y.shift) - 1)) == 0)
                glr_publish_state(glr_state(y, t, t.at + 1), end);
            if (last && p.h_out) glr_st2<VEC>(p.h_out + row, end, nch);
        }
        c = glr_through(agg, c, warp);
        copy_inputs(queue[(k + NS) % kGlrQueue], stage);
        if (p.chunk && n > 0 && ws % kGlrChunk == 0)
            glr_st2<VEC>(p.chunk + ((int64_t)t.b * p.nchunk + ws / kGlrChunk) * p.D + c0, c, nch);
        if constexpr (EPI > 0) {
            if constexpr (by_map)
                glr_wait_boxes(bar + NS, k & 1);
            else
                cp_async_wait_pending<1>();  // all but the next tile's inputs
            __syncwarp();
        }
        const int64_t ts = p.rows[kGlrOut].ts;
        char* po = p.rows[kGlrOut].p + e.off[kGlrOut] + warp * TOK * ts + 2 * lane * (int)sizeof(T);
        auto outputs = [&](auto full) {
#pragma unroll
            for (int j = 0; j < TOK; ++j) {
                float2 h = glr_fma(Ps[j], c, hs[j]);
                if constexpr (EPI > 0) h = glr_add(h, glr_row(epi + (EPI - 1) * ROWS + at(j)));
                if constexpr (EPI == 2) {
                    const float2 z = glr_row(epi + at(j));
                    h = glr_mul(h, glr_mul(z, glr_sigmoid2(z)));
                }
                if (decltype(full)::value || j < n) glr_st2<VEC>(reinterpret_cast<T*>(po), h, nch);
                po += ts;
            }
        };
        if (n == TOK)
            outputs(std::true_type{});
        else
            outputs(std::false_type{});
    }
    cp_async_wait_all();
    if (p.lengths) glr_pad<T>(p, y, reinterpret_cast<unsigned*>(queue));
}

// Backward, tiles of kGlrChunk steps: they are walked from the last step to
// the first (tile `at` from the end of the row's own tiles), and what they
// hand over is q = a G, which the affine map of a tile takes from its right
// end to its left.  A warp's steps share one running product P for both scans,
// the recomputed states (from the saved state that enters the tile) and q,
// which at the warp's first step is sum_s P_s dh_s.  Of each step the registers
// keep rg, ig, beta and the state before it; a is one more ex2 where it is wanted
// again (a small a cannot be had from beta, nor a small beta from a, and there
// is no room for both).  The second half reads x, dout, add and z again from
// shared memory, and by maps it leaves its results in the rows that it has
// read, from where a lane sends them as boxes; so a stage is filled again once
// they are out.  b 8, L 2048, D 4096 bf16: 285 us of 143 us for its 940 MB; issue
// slots 61 % used, special functions 42 %, some 180 instructions a pair and step
// (68 the second half's, 30 the gates', 40 a tile's fixed ones over 8 steps); the
// registers hold no more steps.  (One thread a channel: 2956 us with the forward;
// a block a tile: 465.)
constexpr int kGlrBwdTok = kGlrChunk / kGlrWarps;
template <typename T>
constexpr int kGlrBwdStages = sizeof(T) == 2 ? 2 : 1;
template <typename T, int EPI>
constexpr int kGlrBwdWarpBytes = (EPI == 2 ? 6 : 4) * kGlrBwdStages<T> * kGlrBwdTok * kGlrSlab * (int)sizeof(T);

template <typename T, bool VEC, int EPI, int MODE>
__global__ void __launch_bounds__(kGlrWarps * 32, 2)
    glr_tile_bwd_kernel(const __grid_constant__ GlrParams p, const __grid_constant__ GlrSync y,
                        const __grid_constant__ GlrMaps maps) {
    constexpr int TOK = kGlrBwdTok, NS = kGlrBwdStages<T>, ROWS = TOK * kGlrSlab, NT = EPI == 2 ? 6 : 4;
    extern __shared__ __align__(128) unsigned char glr_smem[];
    __shared__ float4 agg[kGlrWarps][32];   // (P, q) of each warp
    __shared__ float2 aggh[kGlrWarps][32];  // its h
    __shared__ float4 pieces[kGlrGroup][32];
    __shared__ float2 sums[3][kGlrWarps][32];
    __shared__ GlrEntry queue[kGlrQueue];
    __shared__ uint64_t bars[kGlrWarps][NS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    T* const mine = reinterpret_cast<T*>(glr_smem + warp * kGlrBwdWarpBytes<T, EPI>);

    constexpr bool by_map = MODE != kGlrAsync;
    constexpr GlrOrder<TOK, MODE> at;
    uint64_t* const bar = bars[warp];

    auto copy_inputs = [&](const GlrEntry& e, int stage) {
        const GlrTile t = e.t;
        const int64_t ws = glr_first_step<true>(t, kGlrChunk) + warp * TOK;
        const int n = t.at < 0 ? 0 : glr_steps(t.len, ws, TOK);
        T* to = mine + stage * NT * ROWS;
        if constexpr (by_map) {
            const int c = glr_channel(p, t);
            if (lane == 0) glr_boxes_read();  // the stage's results
            if constexpr (EPI == 2)
                glr_copy_boxes<T, TOK, kGlrR, kGlrI, kGlrX, kGlrDout, kGlrZ, kGlrAdd>(to, maps, p, t, ws, n, c, bar + stage);
            else
                glr_copy_boxes<T, TOK, kGlrR, kGlrI, kGlrX, kGlrDout>(to, maps, p, t, ws, n, c, bar + stage);
        } else {
            if (n) {
                const int left = p.D - glr_channel(p, t);
                if constexpr (EPI == 2) {
                    glr_copy_rows<T, TOK, kGlrR, kGlrI, kGlrX, kGlrDout, kGlrZ>(to, p, e, warp * TOK, n, left);
                    if (p.rows[kGlrAdd].p) glr_copy_rows<T, TOK, kGlrAdd>(to + 5 * ROWS, p, e, warp * TOK, n, left);
                } else {
                    glr_copy_rows<T, TOK, kGlrR, kGlrI, kGlrX, kGlrDout>(to, p, e, warp * TOK, n, left);
                }
            }
            cp_async_commit();
        }
    };
    // the parameters' sums of the tile before, once a barrier has passed
    float* part = nullptr;
    int part_n = 0;
    auto put_sums = [&]() {
        if (part_n && warp < 3) {
            float2 v = glr_f2(0.f);
#pragma unroll
            for (int w = 0; w < kGlrWarps; ++w) v = glr_add(v, sums[warp][w][lane]);
            glr_st2<VEC>(part + (int64_t)warp * p.D, v, part_n);
        }
    };

    if (by_map && threadIdx.x == 0) {
        for (int w = 0; w < kGlrWarps; ++w)
            for (int k = 0; k < NS; ++k) mbar_init(&bars[w][k], 1);
        fence_barrier_init();
    }
    GlrQueue<true, sizeof(T)> tiles{queue, kGlrChunk};
    tiles.start(p, y, NS);
    if (EPI == 2 && !p.rows[kGlrAdd].p) {
        for (int k = 0; k < NS; ++k)
            for (int j = lane; j < ROWS; j += 32) mine[(k * NT + 5) * ROWS + j] = T(0.f);
    }
#pragma unroll
    for (int k = 0; k < NS; ++k) copy_inputs(queue[k], k);
    for (unsigned k = 0;; ++k) {
        const GlrEntry& e = queue[k % kGlrQueue];
        GlrTile t = e.t;
        if (t.at < 0) break;
        tiles.put(p, y, k + NS);  // over entry k + NS - 4, which every warp has left behind
        const int stage = NS == 2 ? k & 1 : 0;
        const int c0 = glr_channel(p, t) + 2 * lane;
        const int nch = p.D - c0 > 1 ? 2 : (p.D - c0 > 0 ? 1 : 0);
        const int64_t s0 = glr_first_step<true>(t, kGlrChunk), row = (int64_t)t.b * p.D + c0;
        const int64_t chunk = ((int64_t)t.b * p.nchunk + s0 / kGlrChunk) * p.D;
        const int n = glr_steps(t.len, s0 + warp * TOK, TOK);
        GlrPiece piece;
        if (t.at) glr_ask(piece, y, t, warp);
        T* in = mine + stage * NT * ROWS;
        const T *in_x = in + 2 * ROWS, *in_d = in + 3 * ROWS, *in_z = in + 4 * ROWS, *in_add = in + 5 * ROWS;
        float2 nrg[TOK], nig[TOK], nb[TOK], hp[TOK];  // -rg, -ig, -beta, a state
        const float2 entering = glr_vec2<VEC>(p.chunk, chunk + c0, nch);
        if constexpr (by_map)
            glr_wait_boxes(bar + stage, (k / NS) & 1);
        else
            cp_async_wait_pending<NS - 1>();
        __syncwarp();
        float2 P = glr_f2(1.f), q = glr_f2(0.f), h = glr_f2(0.f);
        if (n) {
            if (n < TOK) glr_close_rows<T, TOK, NT, MODE>(in, at, n);
            const float2 nA2 = glr_scaled<VEC>(p.A, c0, nch, -kGlrLog2e);
            const float2 nr = glr_scaled<VEC>(p.r_bias, c0, nch, -kGlrLog2e);
            const float2 ni = glr_scaled<VEC>(p.i_bias, c0, nch, -kGlrLog2e);
#pragma unroll
            for (int j = 0; j < TOK; ++j) {
                const GlrGate2 g = glr_gate2(glr_row(in + at(j)), glr_row(in + ROWS + at(j)), nr, ni, nA2);
                nrg[j] = g.nrg;
                nig[j] = make_float2(glr_rcp(-g.di.x), glr_rcp(-g.di.y));
                nb[j] = glr_minus_beta(g.nb2);
                const float2 w = glr_mul(glr_mul(nb[j], nig[j]), glr_row(in_x + at(j)));
                hp[j] = h;  // the state before step j, from a zero state at the warp's first
                P = glr_mul(P, g.a);
                h = glr_fma(g.a, h, w);
                float2 dh = glr_row(in_d + at(j));
                if constexpr (EPI == 2) {
                    const float2 z = glr_row(in_z + at(j));
                    dh = glr_mul(dh, glr_mul(z, glr_sigmoid2(z)));
                }
                q = glr_fma(P, dh, q);  // what the step's dh is at the warp's first
            }
        }
        aggh[warp][lane] = h;
        agg[warp][lane] = make_float4(P.x, q.x, P.y, q.y);
        __syncthreads();
        t = e.t;  // (read again rather than kept)
        // by maps a stage's results go out from it, so it is filled again half a tile later
        if (by_map && NS == 2 && k > 0) copy_inputs(queue[(k + 1) % kGlrQueue], stage ^ 1);
        put_sums();
        part = p.part + chunk * 3 + c0;
        part_n = nch;
        float2 sA = glr_f2(0.f), sr = glr_f2(0.f), si = glr_f2(0.f);
        const bool last = s0 == 0, publish = y.ticket && !last && !y.starve;
        // the map from the tile's end to the warp's, and for warp 0 to the tile's start
        float2 Pw = glr_f2(1.f), qw = glr_f2(0.f);
#pragma unroll
        for (int w = kGlrWarps - 1; w > 0; --w) {
            const float4 a = agg[w][lane];
            if (w <= warp) continue;
            Pw = glr_mul(Pw, make_float2(a.x, a.z));
            qw = glr_apply(a, qw);
        }
        q = glr_fma(P, qw, q);
        P = glr_mul(P, Pw);
        if (publish && y.shift && warp == 0) glr_publish_map(glr_map(y, t, t.at), P, q);
        float4 mypiece = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t.at) {
            mypiece = glr_wait_piece(y, piece, t, warp);
        } else if (warp == kGlrGroup - 1) {
            const float2 c = glr_vec2<VEC>(p.dh_out, row, nch);
            mypiece = make_float4(0.f, c.x, 0.f, c.y);
        }
        pieces[warp][lane] = mypiece;
        // the states before the warp's steps, from the one that enters the tile
        const float2 nA2 = glr_scaled<VEC>(p.A, c0, nch, -kGlrLog2e);
        if (n) {
            float2 c = entering;
#pragma unroll
            for (int w = 0; w < kGlrWarps - 1; ++w) {
                const float4 a = agg[w][lane];
                const float2 hw = aggh[w][lane];
                if (w < warp) c = glr_fma(make_float2(a.x, a.z), c, hw);
            }
#pragma unroll
            for (int j = 0; j < TOK; ++j) {
                hp[j] = glr_add(c, hp[j]);
                c = glr_mul(glr_decay(nA2, nrg[j]), c);
            }
        }
        __syncthreads();
        const float4 from = pieces[kGlrGroup - 1][lane];
        float2 c = make_float2(from.y, from.w);
        if (y.shift) c = glr_through(pieces, c, glr_before(y, t));
        if (warp == 0) {
            const float2 end = glr_fma(P, c, q);
            // the other tiles take the last state's gradient from here, not from dh_out, which may be dh_in
            if (publish && t.at == 0) glr_publish_state(glr_state(y, t, 0), c);
            if (publish && ((t.at + 1) & ((1 << y.shift) - 1)) == 0)
                glr_publish_state(glr_state(y, t, t.at + 1), end);
            if (last && p.dh_in) glr_st2<VEC>(p.dh_in + row, end, nch);
        }
        q = glr_fma(Pw, c, qw);
        const float2 nA = glr_scaled<VEC>(p.A, c0, nch, -1.f);  // finite: where A is infinite a factor beside it is 0
        // where the warp's steps go, from its last to its first
        char* to[kGlrDz - kGlrDx + 1];
#pragma unroll
        for (int k = kGlrDx; k <= kGlrDz; ++k)
            to[k - kGlrDx] = p.rows[k].p + e.off[k] + (int64_t)p.rows[k].ts * (warp * TOK + TOK - 1) +
                             2 * lane * (int)sizeof(T);
        // BOXES: into the row of the input that is read by now (dr for r, di for i, dx for x, dz for z, dadd for add)
        auto put = [&](auto boxes, int tensor, int j, float2 v) {
            if constexpr (decltype(boxes)::value) {
                const int q = tensor == kGlrDr ? 0 : tensor == kGlrDi ? 1 : tensor == kGlrDx ? 2 : tensor == kGlrDz ? 4 : 5;
                if (EPI == 1 && tensor == kGlrDadd) return;  // it is dout, as it lies there
                glr_st2<true>(in + q * ROWS + at(j) + 2 * lane, v, 2);
            } else {
                glr_st2<VEC>(reinterpret_cast<T*>(to[tensor - kGlrDx] - (TOK - 1 - j) * (int64_t)p.rows[tensor].ts), v, nch);
            }
        };
        auto outputs = [&](auto full, auto boxes) {
#pragma unroll
            for (int j = TOK - 1; j >= 0; --j) {
                if (!decltype(full)::value && j >= n) continue;
                const float2 a = glr_decay(nA2, nrg[j]);
                const float2 bi = glr_mul(nb[j], nig[j]), w = glr_mul(bi, glr_row(in_x + at(j)));
                const float2 ah = glr_mul(a, hp[j]);
                float2 dh = glr_row(in_d + at(j));
                if constexpr (EPI == 2) {
                    const float2 z = glr_row(in_z + at(j)), sz = glr_sigmoid2(z);
                    // silu'(z) = s (1 + z (1 - s))
                    const float2 ds = glr_fma(glr_mul(sz, z), make_float2(1.f - sz.x, 1.f - sz.y), sz);
                    put(boxes, kGlrDz, j, glr_mul(glr_mul(dh, glr_add(glr_add(ah, w), glr_row(in_add + at(j)))), ds));
                    dh = glr_mul(dh, glr_mul(z, sz));
                }
                if (EPI == 1 || (EPI == 2 && p.rows[kGlrDadd].p)) put(boxes, kGlrDadd, j, dh);
                const float2 G = glr_add(dh, q);
                q = glr_mul(a, G);
                // a h_{s-1} - (a / beta)^2 w
                const float2 ab = glr_mul(a, glr_over_beta(nb[j])), wab = glr_mul(w, ab);
                const float2 dla = glr_mul(G, make_float2(fmaf(-wab.x, ab.x, ah.x), fmaf(-wab.y, ab.y, ah.y)));
                const float2 dr = glr_mul(glr_mul(nA, glr_fma(nrg[j], nrg[j], nrg[j])), dla);
                const float2 Gw = glr_mul(G, w), di = glr_fma(Gw, nig[j], Gw);
                put(boxes, kGlrDx, j, glr_mul(G, bi));
                put(boxes, kGlrDr, j, dr);
                put(boxes, kGlrDi, j, di);
                sA = glr_fma(nrg[j], dla, sA);
                sr = glr_add(sr, dr);
                si = glr_add(si, di);
            }
        };
        if (n == TOK) {
            outputs(std::true_type{}, std::bool_constant<by_map>{});
            if constexpr (by_map) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    const int c = c0, first = (int)(glr_first_step<true>(t, kGlrChunk)) + warp * TOK;
                    const int token = p.reverse ? t.len - first - TOK : first;
                    glr_store_box(in, maps.m[kGlrDr], c, token, t.b);
                    glr_store_box(in + ROWS, maps.m[kGlrDi], c, token, t.b);
                    glr_store_box(in + 2 * ROWS, maps.m[kGlrDx], c, token, t.b);
                    if (EPI == 2) glr_store_box(in + 4 * ROWS, maps.m[kGlrDz], c, token, t.b);
                    if (EPI && p.rows[kGlrDadd].p)
                        glr_store_box(in + (EPI == 1 ? 3 : 5) * ROWS, maps.m[kGlrDadd], c, token, t.b);
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                }
            }
        } else {
            outputs(std::false_type{}, std::false_type{});
        }
        sums[0][warp][lane] = make_float2(-sA.x, -sA.y);
        sums[1][warp][lane] = sr;
        sums[2][warp][lane] = si;
        __syncwarp();  // every lane has read its rows
        if (!by_map || NS == 1) copy_inputs(queue[(k + NS) % kGlrQueue], stage);
    }
    __syncthreads();
    put_sums();
    if constexpr (by_map)
        glr_boxes_read();
    else
        cp_async_wait_all();
    if (p.lengths) glr_pad<T>(p, y, reinterpret_cast<unsigned*>(queue));
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

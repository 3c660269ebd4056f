// glr_api.cu -- the C ABI of the gated linear recurrence (include/bimamba.h):
// argument checks, launch shapes and dispatch.  The arithmetic is in glr.cuh.
#include <cuda_runtime.h>

#include <algorithm>

#include "api_util.h"
#include "bimamba.h"
#include "glr.cuh"

namespace {

using bimamba::GlrParams;
using bimamba::GlrRows;
using bf16 = __nv_bfloat16;

static_assert(bimamba::kGlrChunk == BIMAMBA_GLR_CHUNK, "the header's chunk is the kernels'");

bool sizes_ok(int batch, int64_t L, int D) {
    return batch > 0 && batch <= kMaxBatch && L > 0 && L <= 0x7fffffffLL && D > 0;
}

// Rows that are read: any strides from 0; the kernels step through a row in 32 bits.
int check_in(const bimamba_rows_t& q, size_t esz, int64_t L, bool optional) {
    if (!q.ptr) return optional ? BIMAMBA_OK : BIMAMBA_ERR_INVALID_ARG;
    if (q.batch_stride < 0 || q.token_stride < 0) return BIMAMBA_ERR_INVALID_ARG;
    if (L > 1 && q.token_stride > BIMAMBA_GLR_MAX_TOKEN_STRIDE) return BIMAMBA_ERR_UNSUPPORTED;
    return aligned(q.ptr, esz) ? BIMAMBA_OK : BIMAMBA_ERR_MISALIGNED;
}

// Rows that are written: no two of them may overlap, so the strides have to
// nest one way or the other ([batch][L] or [L][batch] order).
int check_out(const bimamba_rows_t& q, size_t esz, int batch, int64_t L, int D) {
    int rc = check_in(q, esz, L, false);
    if (rc) return rc;
    const bool tok = L == 1 || q.token_stride >= D, bat = batch == 1 || q.batch_stride >= D;
    if (!tok || !bat) return BIMAMBA_ERR_INVALID_ARG;
    if (batch > 1 && L > 1) {
        const bool batch_outer = (q.batch_stride - D) / q.token_stride >= L - 1;
        const bool token_outer = (q.token_stride - D) / q.batch_stride >= batch - 1;
        if (!batch_outer && !token_outer) return BIMAMBA_ERR_INVALID_ARG;
    }
    return BIMAMBA_OK;
}

int check_common(const bimamba_glr_inputs_t* in, const bimamba_glr_params_t* p, int batch, int64_t L, int D,
                 unsigned flags) {
    if (!in || !p || !sizes_ok(batch, L, D)) return BIMAMBA_ERR_INVALID_ARG;
    if (flags & ~(BIMAMBA_GLR_REVERSE | BIMAMBA_TEST_STARVE)) return BIMAMBA_ERR_UNSUPPORTED;
    if (!dtype_ok(in->dtype)) return BIMAMBA_ERR_UNSUPPORTED;
    const size_t e = elem_size(in->dtype);
    int rc = check_in(in->x, e, L, false);
    if (!rc) rc = check_in(in->r, e, L, false);
    if (!rc) rc = check_in(in->i, e, L, false);
    if (!rc) rc = check_in(in->add, e, L, true);
    if (!rc) rc = check_in(in->z, e, L, true);
    if (rc) return rc;
    if (!p->A) return BIMAMBA_ERR_INVALID_ARG;
    if (!aligned(p->A, 4) || !aligned(p->r_bias, 4) || !aligned(p->i_bias, 4) || !aligned(in->lengths, 4))
        return BIMAMBA_ERR_MISALIGNED;
    return BIMAMBA_OK;
}

// Strides in bytes, the token's with the sign of the walk (0 where there is one token).
void set_rows(GlrParams& k, int tensor, const bimamba_rows_t& q, size_t esz) {
    const int ts = k.L > 1 ? (int)(q.token_stride * (int64_t)esz) : 0;
    k.rows[tensor] = {static_cast<char*>(q.ptr), q.batch_stride * (int64_t)esz, k.reverse ? -ts : ts};
}

void fill_common(GlrParams& k, const bimamba_glr_inputs_t* in, const bimamba_glr_params_t* p, int batch, int64_t L,
                 int D, unsigned flags) {
    k.lengths = in->lengths;
    k.A = p->A;
    k.r_bias = p->r_bias;
    k.i_bias = p->i_bias;
    k.L = L;
    k.D = D;
    k.batch = batch;
    k.reverse = (flags & BIMAMBA_GLR_REVERSE) ? 1 : 0;
    k.nchunk = (L + bimamba::kGlrChunk - 1) / bimamba::kGlrChunk;
    const size_t e = elem_size(in->dtype);
    set_rows(k, bimamba::kGlrX, in->x, e);
    set_rows(k, bimamba::kGlrR, in->r, e);
    set_rows(k, bimamba::kGlrI, in->i, e);
    if (in->add.ptr) set_rows(k, bimamba::kGlrAdd, in->add, e);
    if (in->z.ptr) set_rows(k, bimamba::kGlrZ, in->z, e);
}

int check_workspace(const void* ws, size_t have, size_t need) {
    return !ws || !aligned(ws, 256) || have < need ? BIMAMBA_ERR_WORKSPACE : BIMAMBA_OK;
}

}  // namespace

namespace bimamba {

int glr_error_word(int reset, unsigned int* word) {
    if (cudaMemcpyFromSymbol(word, g_glr_error, sizeof(*word)) != cudaSuccess) return BIMAMBA_ERR_CUDA;
    const unsigned int zero = 0;
    if (reset && cudaMemcpyToSymbol(g_glr_error, &zero, sizeof(zero)) != cudaSuccess) return BIMAMBA_ERR_CUDA;
    return BIMAMBA_OK;
}

}  // namespace bimamba

namespace {

// The smallest tile of a launch (fp32); the workspace is sized for it.
constexpr int kSmallTile = bimamba::kGlrTok<float> * bimamba::kGlrWarps;
static_assert(kSmallTile <= bimamba::kGlrChunk, "the backward's tiles are no smaller");

// The hand-over workspace of a launch whose rows have `tiles` tiles: the
// ticket (256 bytes), the maps, the groups' entering states.
size_t sync_bytes(int batch, int D, int64_t tiles) {
    const size_t chains = (size_t)batch * ((D + bimamba::kGlrSlab - 1) / bimamba::kGlrSlab);
    const size_t groups = (size_t)(tiles + bimamba::kGlrGroup - 1) / bimamba::kGlrGroup;
    return 256 + chains * bimamba::kGlrSlab * ((size_t)tiles * 8 + groups * 4);
}

// With the plan of a padded batch behind it.
size_t handover_bytes(int batch, int D, int64_t tiles) {
    return sync_bytes(batch, D, tiles) + 16 * ((size_t)batch * tiles + 1);
}

// Points y at the workspace and enqueues the all-ones fill (a row of one tile
// hands nothing over and gets neither), and what a padded batch needs first.
int make_sync(bimamba::GlrSync& y, const GlrParams& k, int64_t tiles, int tile_steps, bool grouped, unsigned flags,
              void* ws, cudaStream_t st) {
    const int batch = k.batch, D = k.D;
    const size_t chains = (size_t)batch * ((D + bimamba::kGlrSlab - 1) / bimamba::kGlrSlab);
    const size_t maps = grouped ? chains * bimamba::kGlrSlab * (size_t)tiles * 8 : 0;
    const size_t groups = grouped ? (size_t)(tiles + bimamba::kGlrGroup - 1) / bimamba::kGlrGroup : (size_t)tiles;
    const size_t bytes = tiles > 1 ? 256 + maps + chains * bimamba::kGlrSlab * groups * 4 : 0;  // sync_bytes at most
    int4* plan = k.lengths && tiles > 1 ? reinterpret_cast<int4*>(static_cast<char*>(ws) + bytes) : nullptr;
    if (plan) {
        const int64_t blocks = std::max<int64_t>(k.batch * tiles, (int64_t)(bytes / 16384));
        bimamba::glr_plan_kernel<<<(unsigned)std::min<int64_t>(blocks, 8 * kSms), 256, 0, st>>>(
            k, static_cast<uint4*>(ws), (int64_t)bytes, plan, tiles, tile_steps);
        const int rc = launch_status();
        if (rc) return rc;
    }
    y = {};
    y.tiles = tiles;
    y.shift = grouped ? 3 : 0;
    y.groups = (int64_t)groups;
    if (tiles <= 1) return BIMAMBA_OK;
    y.plan = plan;
    y.starve = (flags & BIMAMBA_TEST_STARVE) ? 1 : 0;
    y.wait_limit = y.starve ? kStarveWaitCycles : kWaitCycles;
    unsigned char* q = static_cast<unsigned char*>(ws);
    y.ticket = reinterpret_cast<unsigned int*>(q);
    y.map = reinterpret_cast<unsigned long long*>(q + 256);
    y.state = reinterpret_cast<float*>(q + 256 + maps);
    if (plan) return BIMAMBA_OK;
    return cudaMemsetAsync(ws, 0xff, bytes, st) == cudaSuccess ? BIMAMBA_OK : BIMAMBA_ERR_CUDA;
}

// Every row of the tensors from first to last starts at a multiple of `bytes`.
bool starts_at(const GlrParams& k, int first, int last, int bytes) {
    for (int q = first; q <= last; ++q) {
        const GlrRows& r = k.rows[q];
        if (r.p && (!aligned(r.p, bytes) || r.bs % bytes || r.ts % bytes)) return false;
    }
    return true;
}

// Bytes of one asynchronous copy that the inputs allow: 16, a pair, or 0 (single elements).
int copy_bytes(const GlrParams& k, int esz) {
    if (k.D * (int64_t)esz % 16 == 0 && starts_at(k, bimamba::kGlrR, bimamba::kGlrZ, 16)) return 16;
    return k.D % 2 == 0 && starts_at(k, bimamba::kGlrR, bimamba::kGlrZ, 2 * esz) ? 2 * esz : 0;
}

// Outputs, and all fp32 vectors, in pairs.
bool pairs(const GlrParams& k, int esz) {
    for (const void* v : {(const void*)k.A, (const void*)k.r_bias, (const void*)k.i_bias, (const void*)k.h_in,
                          (const void*)k.h_out, (const void*)k.chunk, (const void*)k.dh_out, (const void*)k.dh_in})
        if (!aligned(v, 8)) return false;
    return k.D % 2 == 0 && starts_at(k, bimamba::kGlrOut, bimamba::kGlrDz, 2 * esz);
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Maps of the inputs that the call has, and of the backward's outputs; false
// where one cannot be mapped (rows shared by tokens or by the batch, outputs
// that start between 16 bytes).
bool make_maps(bimamba::GlrMaps& maps, const GlrParams& k, int esz, int rows) {
    static const EncodeFn encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeFn>(f);
    }();
    const int last = k.part ? bimamba::kGlrDz : bimamba::kGlrZ;
    if (!encode || (k.part && !starts_at(k, bimamba::kGlrDx, bimamba::kGlrDz, 16))) return false;
    for (int q = bimamba::kGlrR; q <= last; ++q) {
        const GlrRows& r = k.rows[q];
        if (!r.p) continue;
        const int64_t ts = r.ts < 0 ? -(int64_t)r.ts : r.ts, bs = k.batch > 1 ? r.bs : ts * k.L;
        if (ts <= 0 || bs <= 0 || bs >= (1LL << 40)) return false;
        const cuuint64_t dims[3] = {(cuuint64_t)k.D, (cuuint64_t)k.L, (cuuint64_t)k.batch};
        const cuuint64_t strides[2] = {(cuuint64_t)ts, (cuuint64_t)bs};
        const cuuint32_t box[3] = {(cuuint32_t)bimamba::kGlrSlab, (cuuint32_t)rows, 1}, one[3] = {1, 1, 1};
        if (encode(&maps.m[q], esz == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, r.p, dims,
                   strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
    }
    return true;
}

// Blocks that stay: what the SMs hold at 128 registers a thread.
using TilesFn = void (*)(GlrParams, bimamba::GlrSync, bimamba::GlrMaps);
// fns: by mode; without the maps' kernels where they cannot be used.
int launch_tiles(const TilesFn (&fns)[3], GlrParams& k, int esz, int64_t tiles, int tile_steps, int warps,
                 size_t warp_bytes, unsigned flags, void* ws, cudaStream_t st) {
    const int64_t total = tiles * k.batch * ((k.D + bimamba::kGlrSlab - 1) / bimamba::kGlrSlab);
    // tickets run past the total by what the blocks take ahead
    if (total > 0x7fffffffLL) return BIMAMBA_ERR_UNSUPPORTED;
    const size_t smem = warps * warp_bytes;
    constexpr size_t kFixed = 17 * 1024 + 1024;  // static shared memory and the 1 KB that the system keeps
    const int by_regs = 16 / warps, by_smem = (int)(228 * 1024 / (smem + kFixed));
    const int64_t held = (int64_t)kSms * std::max(1, std::min(by_regs, by_smem));
    // A tile's predecessor was taken as many tickets ago as there are rows times slabs: at half as many again as the
    // blocks hold tiles it is done, and states alone are handed over (not in a padded batch, whose last tiles may be
    // of one row).
    bimamba::GlrSync y;
    int rc = make_sync(y, k, tiles, tile_steps, k.lengths || 2 * (total / tiles) < 3 * held, flags, ws, st);
    if (rc) return rc;
    y.total = (unsigned)total;
    // maps take the host some microseconds: where every block has several tiles
    bimamba::GlrMaps maps = {};
    int mode = bimamba::kGlrAsync;
    if (fns[1] && k.copy == 16 && total >= 4 * held && make_maps(maps, k, esz, tile_steps / bimamba::kGlrWarps))
        mode = k.reverse ? bimamba::kGlrMapReverse : bimamba::kGlrMapForward;
    const TilesFn fn = fns[mode];
    if ((rc = ensure_smem(reinterpret_cast<const void*>(fn), bimamba::kGlrWarps * warp_bytes))) return rc;
    fn<<<(unsigned)std::min(total, held), warps * 32, smem, st>>>(k, y, maps);
    return launch_status();
}

template <typename T, bool VEC, int EPI>
int launch_fwd_epi(GlrParams& k, unsigned flags, void* ws, cudaStream_t st) {
    constexpr int TOK = bimamba::kGlrTok<T>, TILE = TOK * bimamba::kGlrWarps;
    const int64_t tiles = (k.L + TILE - 1) / TILE;
    const int warps = tiles > 1 ? bimamba::kGlrWarps : (int)((k.L + TOK - 1) / TOK);
    using namespace bimamba;
    TilesFn fns[3] = {glr_tile_fwd_kernel<T, VEC, EPI, kGlrAsync>, nullptr, nullptr};
    if constexpr (VEC) {  // (inputs of whole 16 bytes hardly come with outputs of unpaired elements)
        fns[1] = glr_tile_fwd_kernel<T, VEC, EPI, kGlrMapForward>;
        fns[2] = glr_tile_fwd_kernel<T, VEC, EPI, kGlrMapReverse>;
    }
    return launch_tiles(fns, k, (int)sizeof(T), tiles, TILE, warps, bimamba::kGlrFwdWarpBytes<T, EPI>,
                        flags, ws, st);
}

template <typename T, bool VEC, int EPI>
int launch_bwd_epi(GlrParams& k, unsigned flags, void* ws, cudaStream_t st) {
    using namespace bimamba;
    TilesFn fns[3] = {glr_tile_bwd_kernel<T, VEC, EPI, kGlrAsync>, nullptr, nullptr};
    if constexpr (VEC) {  // (inputs of whole 16 bytes hardly come with outputs of unpaired elements)
        fns[1] = glr_tile_bwd_kernel<T, VEC, EPI, kGlrMapForward>;
        fns[2] = glr_tile_bwd_kernel<T, VEC, EPI, kGlrMapReverse>;
    }
    return launch_tiles(fns, k, (int)sizeof(T), k.nchunk, bimamba::kGlrChunk, bimamba::kGlrWarps,
                        bimamba::kGlrBwdWarpBytes<T, EPI>, flags, ws, st);
}

template <bool BWD, typename T, bool VEC>
int launch_vec(GlrParams& k, unsigned flags, void* ws, cudaStream_t st) {
    const int epi = k.rows[bimamba::kGlrZ].p ? 2 : (k.rows[bimamba::kGlrAdd].p ? 1 : 0);
    if constexpr (BWD) {
        if (epi == 2) return launch_bwd_epi<T, VEC, 2>(k, flags, ws, st);
        return epi ? launch_bwd_epi<T, VEC, 1>(k, flags, ws, st) : launch_bwd_epi<T, VEC, 0>(k, flags, ws, st);
    } else {
        if (epi == 2) return launch_fwd_epi<T, VEC, 2>(k, flags, ws, st);
        return epi ? launch_fwd_epi<T, VEC, 1>(k, flags, ws, st) : launch_fwd_epi<T, VEC, 0>(k, flags, ws, st);
    }
}

template <bool BWD>
int launch(GlrParams& k, bimamba_dtype_t dtype, unsigned flags, void* ws, cudaStream_t st) {
    const int e = (int)elem_size(dtype);
    k.copy = copy_bytes(k, e);
    const bool vec = pairs(k, e);
    if (dtype == BIMAMBA_BF16)
        return vec ? launch_vec<BWD, bf16, true>(k, flags, ws, st) : launch_vec<BWD, bf16, false>(k, flags, ws, st);
    return vec ? launch_vec<BWD, float, true>(k, flags, ws, st) : launch_vec<BWD, float, false>(k, flags, ws, st);
}

// The backward's partial sums, one row of 3 D per chunk, in whole 256 bytes.
size_t part_bytes(int batch, int64_t L, int D) {
    const size_t rows = (size_t)batch * (size_t)((L + bimamba::kGlrChunk - 1) / bimamba::kGlrChunk);
    return (rows * 3 * (size_t)D * sizeof(float) + 255) / 256 * 256;
}

}  // namespace

extern "C" {

size_t bimamba_glr_workspace_bytes(int batch, int64_t L, int d_inner, int backward) {
    if (!sizes_ok(batch, L, d_inner)) return 0;
    const size_t sync = handover_bytes(batch, d_inner, (L + kSmallTile - 1) / kSmallTile);
    return backward ? part_bytes(batch, L, d_inner) + sync : sync;
}

int bimamba_glr_fwd(const bimamba_glr_inputs_t* in, const bimamba_glr_params_t* p, const float* h_in,
                    const bimamba_rows_t* out, float* h_out, float* chunk_states, int batch, int64_t L, int d_inner,
                    unsigned flags, void* workspace, size_t workspace_bytes, void* cuda_stream) {
    int rc = check_common(in, p, batch, L, d_inner, flags);
    if (rc) return rc;
    if (!out) return BIMAMBA_ERR_INVALID_ARG;
    if ((rc = check_out(*out, elem_size(in->dtype), batch, L, d_inner))) return rc;
    if (!aligned(h_in, 4) || !aligned(h_out, 4) || !aligned(chunk_states, 4)) return BIMAMBA_ERR_MISALIGNED;
    if (L > BIMAMBA_GLR_CHUNK &&
        (rc = check_workspace(workspace, workspace_bytes, bimamba_glr_workspace_bytes(batch, L, d_inner, 0))))
        return rc;

    GlrParams k = {};
    fill_common(k, in, p, batch, L, d_inner, flags);
    set_rows(k, bimamba::kGlrOut, *out, elem_size(in->dtype));
    k.h_in = h_in;
    k.h_out = h_out;
    k.chunk = chunk_states;
    return launch<false>(k, in->dtype, flags, workspace, static_cast<cudaStream_t>(cuda_stream));
}

int bimamba_glr_bwd(const bimamba_glr_inputs_t* in, const bimamba_glr_params_t* p, const bimamba_rows_t* dout,
                    const float* chunk_states, const float* dh_out, const bimamba_glr_grads_t* grads, int batch,
                    int64_t L, int d_inner, unsigned flags, void* workspace, size_t workspace_bytes,
                    void* cuda_stream) {
    int rc = check_common(in, p, batch, L, d_inner, flags);
    if (rc) return rc;
    if (!dout || !chunk_states || !grads) return BIMAMBA_ERR_INVALID_ARG;
    const size_t e = elem_size(in->dtype);
    if ((rc = check_in(*dout, e, L, false))) return rc;
    if ((rc = check_out(grads->dx, e, batch, L, d_inner))) return rc;
    if ((rc = check_out(grads->dr, e, batch, L, d_inner))) return rc;
    if ((rc = check_out(grads->di, e, batch, L, d_inner))) return rc;
    if (in->add.ptr && (rc = check_out(grads->dadd, e, batch, L, d_inner))) return rc;
    if (in->z.ptr && (rc = check_out(grads->dz, e, batch, L, d_inner))) return rc;
    if (!aligned(chunk_states, 4) || !aligned(dh_out, 4) || !aligned(grads->dA, 4) || !aligned(grads->dr_bias, 4) ||
        !aligned(grads->di_bias, 4) || !aligned(grads->dh_in, 4))
        return BIMAMBA_ERR_MISALIGNED;
    if ((rc = check_workspace(workspace, workspace_bytes, bimamba_glr_workspace_bytes(batch, L, d_inner, 1)))) return rc;

    GlrParams k = {};
    fill_common(k, in, p, batch, L, d_inner, flags);
    set_rows(k, bimamba::kGlrDout, *dout, e);
    set_rows(k, bimamba::kGlrDx, grads->dx, e);
    set_rows(k, bimamba::kGlrDr, grads->dr, e);
    set_rows(k, bimamba::kGlrDi, grads->di, e);
    if (in->add.ptr) set_rows(k, bimamba::kGlrDadd, grads->dadd, e);
    if (in->z.ptr) set_rows(k, bimamba::kGlrDz, grads->dz, e);
    k.chunk = const_cast<float*>(chunk_states);
    k.dh_out = dh_out;
    k.dh_in = grads->dh_in;
    k.part = static_cast<float*>(workspace);
    unsigned char* sync = static_cast<unsigned char*>(workspace) + part_bytes(batch, L, d_inner);
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    rc = launch<true>(k, in->dtype, flags, sync, st);
    if (rc || !(grads->dA || grads->dr_bias || grads->di_bias)) return rc;
    bimamba::glr_sums_kernel<<<(unsigned)((3LL * d_inner + 31) / 32), 1024, 0, st>>>(
        k.part, batch * k.nchunk, d_inner, grads->dA, grads->dr_bias, grads->di_bias);
    return launch_status();
}

}  // extern "C"

// block_norm_api.cu -- the C ABI of the block norm (include/bimamba.h):
// argument checks, launch shapes and dispatch.  The arithmetic is in block_norm.cuh.
#include <cuda_runtime.h>

#include <algorithm>

#include "api_util.h"
#include "bimamba.h"
#include "block_norm.cuh"

namespace {

using bimamba::BlockNormParams;
using bf16 = __nv_bfloat16;

constexpr int kMaxD = 16384;  // the widest row a block of 512 threads holds, 32 columns each

bool sizes_ok(int batch, int64_t L, int d) {
    return batch > 0 && batch <= kMaxBatch && L > 0 && d > 0 && L <= 0x7fffffffLL / batch;
}

int check_common(const bimamba_block_norm_params_t* p, bimamba_dtype_t ts, bimamba_dtype_t tu, int batch, int64_t L,
                 int d, unsigned flags) {
    if (!p || !sizes_ok(batch, L, d)) return BIMAMBA_ERR_INVALID_ARG;
    if (flags & ~(BIMAMBA_NORM_RMS | BIMAMBA_NORM_GATE_SHARED | BIMAMBA_NORM_GAMMA_SHARED))
        return BIMAMBA_ERR_UNSUPPORTED;
    if (!dtype_ok(ts) || !dtype_ok(tu) || (ts == BIMAMBA_BF16 && tu == BIMAMBA_F32)) return BIMAMBA_ERR_UNSUPPORTED;
    if (d > kMaxD) return BIMAMBA_ERR_UNSUPPORTED;
    if (!aligned(p->gate, 4) || !aligned(p->post_w, 4) || !aligned(p->gamma, 4) || !aligned(p->beta, 4))
        return BIMAMBA_ERR_MISALIGNED;
    return BIMAMBA_OK;
}

void fill_common(BlockNormParams& k, const bimamba_block_norm_params_t* p, int batch, int64_t L, int d,
                 unsigned flags) {
    k.gate = p->gate;
    k.post_w = p->post_w;
    k.gamma = p->gamma;
    k.res_scale = p->res_scale;
    k.L = L;
    k.batch = batch;
    k.d = d;
    k.gate_bs = (flags & BIMAMBA_NORM_GATE_SHARED) ? 0 : d;
    k.gamma_bs = (flags & BIMAMBA_NORM_GAMMA_SHARED) ? 0 : d;
    k.rms = (flags & BIMAMBA_NORM_RMS) ? 1 : 0;
}

// How a row is spread over threads.  8 columns a thread (16-byte accesses)
// where the width and every pointer allow it, else one; rows of at most
// 1024 columns to a warp (no barrier), wider ones to a block.
struct Shape {
    int vec, k, threads;
    bool warp;
};

Shape shape_for(int d, bool vec) {
    const int groups = vec ? d / 8 : d;
    if (groups <= 128) return {vec ? 8 : 1, groups <= 32 ? 1 : 4, 256, true};
    const int most = bimamba::kBlockNormThreads, k = (groups + most - 1) / most;  // vec: up to 4; else up to 32
    const int per = (groups + k - 1) / k;
    return {vec ? 8 : 1, vec ? (k == 1 ? 1 : 4) : (k <= 4 ? 4 : 32), (per + 31) / 32 * 32, false};
}

template <bool BWD, typename TS, typename TU, int V, int K, bool WARP>
int launch_one(const BlockNormParams& k, const Shape& s, cudaStream_t st) {
    if constexpr (BWD) {
        const int per = WARP ? s.threads / 32 : 1;
        const dim3 grid((unsigned)((k.nseg + per - 1) / per), (unsigned)k.batch);
        bimamba::block_norm_bwd_kernel<TS, TU, V, K, WARP><<<grid, s.threads, 0, st>>>(k);
    } else {
        const int per = WARP ? s.threads / 32 : 1;
        const unsigned grid = (unsigned)((k.batch * k.L + per - 1) / per);
        bimamba::block_norm_fwd_kernel<TS, TU, V, K, WARP><<<grid, s.threads, 0, st>>>(k);
    }
    return launch_status();
}

template <bool BWD, typename TS, typename TU>
int launch_shape(const BlockNormParams& k, const Shape& s, cudaStream_t st) {
    if (s.warp) {
        if (s.vec == 8) return s.k == 1 ? launch_one<BWD, TS, TU, 8, 1, true>(k, s, st)
                                        : launch_one<BWD, TS, TU, 8, 4, true>(k, s, st);
        return s.k == 1 ? launch_one<BWD, TS, TU, 1, 1, true>(k, s, st)
                        : launch_one<BWD, TS, TU, 1, 4, true>(k, s, st);
    }
    if (s.vec == 8) return s.k == 1 ? launch_one<BWD, TS, TU, 8, 1, false>(k, s, st)
                                    : launch_one<BWD, TS, TU, 8, 4, false>(k, s, st);
    return s.k == 4 ? launch_one<BWD, TS, TU, 1, 4, false>(k, s, st)
                    : launch_one<BWD, TS, TU, 1, 32, false>(k, s, st);
}

template <bool BWD>
int launch_rows(const BlockNormParams& k, const Shape& s, bimamba_dtype_t ts, bimamba_dtype_t tu, cudaStream_t st) {
    if (ts == BIMAMBA_BF16) return launch_shape<BWD, bf16, bf16>(k, s, st);
    if (tu == BIMAMBA_BF16) return launch_shape<BWD, float, bf16>(k, s, st);
    return launch_shape<BWD, float, float>(k, s, st);
}

constexpr size_t kMaxRunSmem = 200 * 1024;

int run_threads(int d, int k) { return ((d / 8 + k - 1) / k + 31) / 32 * 32; }

// The copying form: 32 to 512 threads of K = 1 or 2 groups of eight columns.
// False where the copies ahead would not fit: the backward of fp32 rows of 3080 to
// 4096 columns with an fp32 branch (above, K = 2 has fewer stages).
template <bool BWD, typename TS, typename TU, int K>
bool launch_run_k(BlockNormParams& k, cudaStream_t st, int& rc) {
    constexpr int pieces = BWD ? bimamba::kBnBwdPieces<TS, TU, K> : bimamba::kBnFwdPieces<TS, TU, K>;
    constexpr int stages = BWD ? bimamba::kBnBwdStages<TU, K> : bimamba::kBnFwdStages<TS, TU>;
    const int threads = run_threads(k.d, K);
    const size_t smem = (size_t)stages * pieces * threads * 16;
    if (smem > kMaxRunSmem) return false;
    void (*fn)(BlockNormParams);
    if constexpr (BWD)
        fn = k.post_w ? bimamba::block_norm_bwd_run_kernel<TS, TU, K, true>
                      : bimamba::block_norm_bwd_run_kernel<TS, TU, K, false>;
    else
        fn = k.post_w ? bimamba::block_norm_fwd_run_kernel<TS, TU, K, true>
                      : bimamba::block_norm_fwd_run_kernel<TS, TU, K, false>;
    // one limit for all widths: it is raised once a kernel
    if ((rc = ensure_smem(reinterpret_cast<const void*>(fn), kMaxRunSmem))) return true;
    if (!BWD) {  // one run a block that an SM holds (up to 96 registers a thread, 128 for K = 2)
        const int held = (int)std::min<size_t>(std::min((K == 1 ? 640 : 512) / threads, 24), 220 * 1024 / (smem + 2048));
        k.nseg = (int)std::max<int64_t>(1, std::min<int64_t>(k.L, (int64_t)kSms * std::max(held, 1) / k.batch));
    }
    fn<<<dim3((unsigned)k.nseg, (unsigned)k.batch), threads, smem, st>>>(k);
    rc = launch_status();
    return true;
}

// Groups of eight columns a thread.  The forward holds two above a warp's 256
// columns: half the row sums' work (16,384 rows of 2048 bf16: 50 us, with one
// group 54; 65,536 of 352: 40 and 66).  The backward's column sums leave room for
// one, up to 512 threads.
template <bool BWD, typename TS, typename TU>
bool launch_run(BlockNormParams& k, cudaStream_t st, int& rc) {
    const bool one = BWD ? k.d <= 8 * bimamba::kBlockNormThreads : k.d <= 256;
    return one ? launch_run_k<BWD, TS, TU, 1>(k, st, rc) : launch_run_k<BWD, TS, TU, 2>(k, st, rc);
}

// The packed form: G lanes a row, as few as E elements each allow.
int pack_lanes(int d, bool bwd) {
    const int e = bwd ? bimamba::kBnPackBwd : bimamba::kBnPackFwd;
    int g = 4;
    while (g < 32 && g * e < d) g *= 2;
    return g * e < d ? (d + 32 * e - 1) / (32 * e) * 32 : g;
}
constexpr int kPackMaxD = 4096;  // 512 threads of 8 in the backward
constexpr size_t kPackSmem = 100 * 1024;

template <bool BWD, typename TS, typename TU, int P>
int launch_pack_p(BlockNormParams& k, cudaStream_t st) {
    const int G = pack_lanes(k.d, BWD), threads = std::max(256, G), groups = G > 32 ? 1 : threads / G;
    const int block = G > 32 ? G : threads, row = k.d * (int)(sizeof(TS) + sizeof(TU)) * (BWD ? 2 : 1);
    // about 16 KB a stage (24 in the backward), whole rounds of the groups
    int R = (BWD ? 24576 : 16384) / row / groups * groups;
    R = (int)std::min<int64_t>(std::max(R, groups), (k.L + groups - 1) / groups * groups);
    size_t smem = 2 * (size_t)(bimamba::bn_pack_bytes(R, k.d, sizeof(TS)) + bimamba::bn_pack_bytes(R, k.d, sizeof(TU)));
    if (BWD) smem = std::max(2 * smem, (size_t)groups * 4 * k.d * sizeof(float));
    void (*fn)(BlockNormParams, int, int);
    if constexpr (BWD)
        fn = k.post_w ? bimamba::block_norm_bwd_pack_kernel<TS, TU, P, true>
                      : bimamba::block_norm_bwd_pack_kernel<TS, TU, P, false>;
    else
        fn = k.post_w ? bimamba::block_norm_fwd_pack_kernel<TS, TU, P, true>
                      : bimamba::block_norm_fwd_pack_kernel<TS, TU, P, false>;
    if (smem > 2 * kPackSmem) return BIMAMBA_ERR_UNSUPPORTED;  // (no width reaches it)
    int rc = ensure_smem(reinterpret_cast<const void*>(fn), 2 * kPackSmem);
    if (rc) return rc;
    if (!BWD) {
        const int64_t tiles = (k.L + R - 1) / R;
        const int held = (int)std::max<size_t>(1, std::min<size_t>(512 / block, 220 * 1024 / (smem + 2048)));
        k.nseg = (int)std::max<int64_t>(1, std::min<int64_t>(tiles, (int64_t)kSms * held / k.batch));
    }
    fn<<<dim3((unsigned)k.nseg, (unsigned)k.batch), block, smem, st>>>(k, G, R);
    return launch_status();
}

template <bool BWD, typename TS, typename TU>
int launch_pack(BlockNormParams& k, cudaStream_t st) {
    return k.d % 2 ? launch_pack_p<BWD, TS, TU, 1>(k, st) : launch_pack_p<BWD, TS, TU, 2>(k, st);
}

// Which form.  The copying one where a row fills a warp and is whole groups of
// eight, if its copies ahead fit; the packed one for other rows up to kPackMaxD
// columns (8192 fp32 rows of 4096 in the backward: 220 us of 123; 65,536 rows of 129
// bf16: forward 44 us, backward 61, the plain form 111 and 638; of 56: 17 and 26,
// plain 31 and 49); the plain one for wider odd rows, for pointers that no 16-byte
// access can use, and for batch rows of a few tokens that have vectors of their
// own (a block a batch row would be idle).
template <bool BWD>
int launch(BlockNormParams& k, bool vec, bool chunks, bimamba_dtype_t ts, bimamba_dtype_t tu, cudaStream_t st) {
    // the copying form's fp32 stores are of 32 bytes
    const bool wide = (ts == BIMAMBA_BF16 || (aligned(k.x_out, 32) && aligned(k.dx, 32))) &&
                      (tu == BIMAMBA_BF16 || (aligned(k.y, 32) && aligned(k.du, 32)));
    if (vec && wide && k.d >= 256 && k.d <= 16 * bimamba::kBlockNormThreads) {
        int rc = BIMAMBA_OK;
        if (ts == BIMAMBA_BF16 ? launch_run<BWD, bf16, bf16>(k, st, rc)
                               : (tu == BIMAMBA_BF16 ? launch_run<BWD, float, bf16>(k, st, rc)
                                                     : launch_run<BWD, float, float>(k, st, rc)))
            return rc;
    }
    if (chunks && k.d <= kPackMaxD && (k.L >= 16 || k.batch == 1)) {
        if (ts == BIMAMBA_BF16) return launch_pack<BWD, bf16, bf16>(k, st);
        return tu == BIMAMBA_BF16 ? launch_pack<BWD, float, bf16>(k, st) : launch_pack<BWD, float, float>(k, st);
    }
    return launch_rows<BWD>(k, shape_for(k.d, vec), ts, tu, st);
}

// Row segments of the backward per batch row, each with its own column sums:
// one for each block that the SMs hold at 128 registers a thread, but at least
// 8 rows a segment.  (In fp32 shared memory holds fewer, and the rest follow:
// 16,384 rows of 2048 take 148 us of 123.)
int segments(int batch, int64_t L, int d) {
    const int threads = d % 8 == 0 && d >= 256 ? std::min(512, (d / 8 + 31) / 32 * 32) : std::max(256, pack_lanes(d, true));
    const int held = std::max(1, std::min(16, 512 / threads));
    const int64_t want = std::max<int64_t>(1, (int64_t)held * kSms / batch), most = std::max<int64_t>(1, L / 8);
    return (int)std::min(want, most);
}

template <typename... P>
bool all_aligned16(P... p) {
    return (aligned(p, 16) && ...);
}

}  // namespace

extern "C" {

int bimamba_block_norm_fwd(const void* x, const void* u, const bimamba_block_norm_params_t* p, void* x_out, void* y,
                           float* stats, bimamba_dtype_t stream_dtype, bimamba_dtype_t dtype, int batch, int64_t L,
                           int d, unsigned flags, void* cuda_stream) {
    int rc = check_common(p, stream_dtype, dtype, batch, L, d, flags);
    if (rc) return rc;
    if (!x || (!x_out && !y) || !(p->eps > 0.f)) return BIMAMBA_ERR_INVALID_ARG;
    if (!u && (p->gate || p->post_w)) return BIMAMBA_ERR_INVALID_ARG;
    const size_t es = elem_size(stream_dtype), eu = elem_size(dtype);
    if (!aligned(x, es) || !aligned(x_out, es) || !aligned(u, eu) || !aligned(y, eu) || !aligned(stats, 4))
        return BIMAMBA_ERR_MISALIGNED;

    BlockNormParams k = {};
    fill_common(k, p, batch, L, d, flags);
    k.beta = p->beta;
    k.eps = p->eps;
    k.x = x;
    k.u = u;
    k.x_out = x_out;
    k.y = y;
    k.stats = stats;
    const bool chunks = all_aligned16(x, u, x_out, y);
    const bool vec = chunks && d % 8 == 0 && all_aligned16(stats, p->gate, p->post_w, p->gamma, p->beta);
    // vectors that all rows share make the batch one long row
    if ((!k.gate || !k.gate_bs) && ((!k.gamma && !k.beta) || !k.gamma_bs)) k.L *= batch, k.batch = 1;
    return launch<false>(k, vec, chunks, stream_dtype, dtype, static_cast<cudaStream_t>(cuda_stream));
}

size_t bimamba_block_norm_workspace_bytes(int batch, int64_t L, int d) {
    if (!sizes_ok(batch, L, d)) return 0;
    return (size_t)batch * segments(batch, L, d) * 4 * (size_t)d * sizeof(float);
}

int bimamba_block_norm_bwd(const void* dy, const void* dx_out, const void* x_out, const void* u, const float* stats,
                           const bimamba_block_norm_params_t* p, const bimamba_block_norm_grads_t* g,
                           bimamba_dtype_t stream_dtype, bimamba_dtype_t dtype, int batch, int64_t L, int d,
                           unsigned flags, void* workspace, size_t workspace_bytes, void* cuda_stream) {
    int rc = check_common(p, stream_dtype, dtype, batch, L, d, flags);
    if (rc) return rc;
    if (!g || !x_out || !stats || (!dy && !dx_out) || !g->dx) return BIMAMBA_ERR_INVALID_ARG;
    if (!u && (p->gate || p->post_w)) return BIMAMBA_ERR_INVALID_ARG;
    if ((u == nullptr) != (g->du == nullptr)) return BIMAMBA_ERR_INVALID_ARG;
    if ((g->dgate && !p->gate) || (g->dpost_w && !p->post_w) || (g->dgamma && !p->gamma))
        return BIMAMBA_ERR_INVALID_ARG;
    if (!dy && (g->dgamma || g->dbeta)) return BIMAMBA_ERR_INVALID_ARG;
    const size_t es = elem_size(stream_dtype), eu = elem_size(dtype);
    if (!aligned(dy, eu) || !aligned(dx_out, es) || !aligned(x_out, es) || !aligned(u, eu) || !aligned(stats, 4) ||
        !aligned(g->dx, es) || !aligned(g->du, eu) || !aligned(g->dgate, 4) || !aligned(g->dpost_w, 4) ||
        !aligned(g->dgamma, 4) || !aligned(g->dbeta, 4))
        return BIMAMBA_ERR_MISALIGNED;
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < bimamba_block_norm_workspace_bytes(batch, L, d))
        return BIMAMBA_ERR_WORKSPACE;

    BlockNormParams k = {};
    fill_common(k, p, batch, L, d, flags);
    k.x = x_out;
    k.u = u;
    k.stats = const_cast<float*>(stats);
    k.dy = dy;
    k.dx_out = dx_out;
    k.dx = g->dx;
    k.du = g->du;
    k.nseg = segments(batch, L, d);
    const bool sums = g->dgate || g->dpost_w || g->dgamma || g->dbeta;
    k.part = sums ? static_cast<float*>(workspace) : nullptr;
    const bool chunks = all_aligned16(dy, dx_out, x_out, u, (const void*)g->dx, (const void*)g->du);
    const bool vec = chunks && d % 8 == 0 && all_aligned16(stats, p->gate, p->post_w, p->gamma);
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    if ((rc = launch<true>(k, vec, chunks, stream_dtype, dtype, st)) || !sums) return rc;
    const dim3 grid((unsigned)((d + 31) / 32), 4, (unsigned)batch);
    bimamba::block_norm_sums_kernel<<<grid, 32 * bimamba::kBnSumWarps, 0, st>>>(
        k.part, k.nseg, batch, d, g->dgate, g->dpost_w, g->dgamma, g->dbeta, (flags & BIMAMBA_NORM_GATE_SHARED) != 0,
        (flags & BIMAMBA_NORM_GAMMA_SHARED) != 0);
    return launch_status();
}

}  // extern "C"

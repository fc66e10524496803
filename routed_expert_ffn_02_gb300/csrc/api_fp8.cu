// api_fp8.cu -- the C ABI of the 8-bit operators and of the balance loss
// (include/moe.h): argument validation, workspace layout and the launch
// sequence of each entry point.  Nothing here allocates or throws.

#include "api_common.cuh"
#include "fp8.cuh"
#include "moe_internal.cuh"

using namespace moe;

namespace {

constexpr int kSide = 128;   // columns of a block of scales

moe_status check_blocks(const char* name, int32_t n) {
    if (n < kSide || n % kSide)
        return fail(MOE_ERR_INVALID_ARG, "%s = %d is not a positive multiple of 128", name, n);
    if (n > kMaxHidden) return fail(MOE_ERR_UNSUPPORTED, "%s is limited to %d", name, kMaxHidden);
    return MOE_OK;
}

// ---- the planner's tile lists ----

struct Lists {
    WsHeader* hdr;
    FatTile *tiles, *solo, *thin;
};
void take_lists(Carver* c, int64_t rows, int E, Lists* l) {
    l->hdr = c->take<WsHeader>(1);
    l->tiles = c->take<FatTile>((size_t)max_fat_tiles(rows, E));
    l->solo = c->take<FatTile>((size_t)E);
    l->thin = c->take<FatTile>((size_t)E);
}
// Every expert that holds rows is a pair-tile, solo or tensor-core streaming
// expert: at most 32 rows, at most 128, or more.
Plan plan_of(const Lists& l, int E) {
    return Plan{l.tiles, l.solo, nullptr, l.thin, l.hdr, kThinMaxTokens + 1, 1, 1, nullptr, E};
}
Fp8Args args_of(const Lists& l, int64_t rows, int K, int N, bool gated) {
    Fp8Args a = {};
    a.tiles = l.tiles;
    a.solo_tiles = l.solo;
    a.thin_tiles = l.thin;
    a.hdr = l.hdr;
    a.rows = (int)rows;
    a.k_blocks = K / kSide;
    a.n_rows = N;
    a.n_blocks_n = gated ? N / kSide : (N + 255) / 256;
    a.ld_out = N;
    a.wait_cycles = main_wait_cycles();
    return a;
}

// ---- workspaces ----

struct FfnBufs {
    Lists l;
    uint8_t *xq, *xs, *hq, *hs;
    int32_t* inv_perm;
};
void take_ffn(Carver* c, const moe_shape* sh, FfnBufs* b) {
    const int64_t P = (int64_t)sh->T * sh->k;
    take_lists(c, P, sh->E, &b->l);
    b->xq = c->take<uint8_t>((size_t)(P * sh->H));
    b->xs = c->take<uint8_t>((size_t)(P * (sh->H / kSide)));
    b->hq = c->take<uint8_t>((size_t)(P * sh->I));
    b->hs = c->take<uint8_t>((size_t)(P * (sh->I / kSide)));
    b->inv_perm = c->take<int32_t>((size_t)P);
}
size_t carve_ffn(const moe_shape* sh, void* ws, FfnBufs* b) {
    Carver c(ws);
    take_ffn(&c, sh, b);
    return align_up(c.off, 256);
}

struct FwdBufs {
    FfnBufs f;
    int32_t *idx, *counts, *offsets, *perm, *chunk;
    float* gates;
    uint8_t* y;   // [P, H] bf16, or fp32 (fp32_y)
};
// y of a batch that cannot have pair tiles stays in L2 (at most 128 tokens),
// where four bytes a value cost nothing measurable (decode batch 24: 160.7 us
// either way), and the output is then rounded once instead of twice.
bool fp32_y(const moe_shape* sh) { return sh->T <= kTileM; }
size_t carve_fwd(const moe_shape* sh, void* ws, FwdBufs* b) {
    const int64_t P = (int64_t)sh->T * sh->k;
    Carver c(ws);
    take_ffn(&c, sh, &b->f);
    b->idx = c.take<int32_t>((size_t)P);
    b->gates = c.take<float>((size_t)P);
    b->counts = c.take<int32_t>((size_t)sh->E);
    b->offsets = c.take<int32_t>((size_t)sh->E + 1);
    b->perm = c.take<int32_t>((size_t)P);
    b->chunk = c.take<int32_t>(permute_scratch_ints(P, sh->E));
    b->y = c.take<uint8_t>((size_t)(P * sh->H) * (fp32_y(sh) ? 4 : 2));
    return align_up(c.off, 256);
}

// Places the scratch of the balance loss; returns its bytes.
size_t carve_balance(void* ws, BalanceArgs* a) {
    Carver c(ws);
    a->hdr = c.take<WsHeader>(1);
    a->shares = c.take<float>((size_t)balance_shares(a->E, a->S));
    a->part = c.take<float2>((size_t)(balance_partial_rows(a->T, a->S) * a->E));
    return align_up(c.off, 256);
}

moe_status check_experts(const moe_fp8_experts* w) {
    if (!w) return fail(MOE_ERR_INVALID_ARG, "experts is NULL");
    CHECK_PTR(w->gate); CHECK_PTR(w->up); CHECK_PTR(w->down);
    CHECK_PTR(w->gate_scales); CHECK_PTR(w->up_scales); CHECK_PTR(w->down_scales);
    return MOE_OK;
}

// Which kernels run, from sizes the host knows: `most` bounds any expert's
// rows.  A single expert takes one kernel by its rows.  With several, small
// experts cannot be ruled out, so the pair kernel is a launch more, and up to
// kPairRows rows the one-CTA kernel takes the pair tiles as well.  Measured, us
// without / with the pair kernel, rows x (N, K) over E experts:
//   777 x (640, 1152) over 48: 15.3 / 26.5      4096 x (4096, 2048) over 16: 53.5 / 56.6
//   4000 x (2048, 2048) over 2: 26.8 / 28.4     4000 x (2048, 1024) over 4: 20.7 / 23.4
//   4000 x (4096, 2048) over 8: 45.4 / 44.6     8192 x (4096, 2048) over 16: 78.6 / 67.6
//   layer of 512 tokens, 64 experts, 2048 x 1024: 134 / 163
// A few experts with many rows each and long K would gain from pairs below the
// limit (2000 x (4096, 4096) over 2: 36.4 / 32.6, 4000 over 2: 68.5 / 60.1,
// over 4: 69.3 / 61.7); the host does not know the rows of each expert.
struct Kernels {
    bool pair, solo;
};
constexpr int64_t kPairRows = 4096;
Kernels kernels_for(int64_t rows, int64_t most, int E) {
    const bool pair = most > kTileM && (E == 1 || rows > kPairRows);
    return {pair, !(E == 1 && pair)};
}

// The grouped product y = A W^T (plain) over the planner's lists.
moe_status run_product(const uint8_t* x, const uint8_t* W, const Fp8Args& a, const Kernels& kn,
                       int E, int num_sms, cudaStream_t s) {
    if (kn.pair) CUDA_TRY(launch_fp8_pair(x, a.rows, W, a, E, num_sms, s), "8-bit product (pairs)");
    if (kn.solo) CUDA_TRY(launch_fp8_solo(x, a.rows, W, a, E, num_sms, s), "8-bit product (one-CTA)");
    return MOE_OK;
}

// Quantised rows in place (xq, xs): gate/up, then down into y [P, H], or y32
// where no expert can have pair tiles.
moe_status run_ffn(const moe_shape* sh, const FfnBufs& b, const moe_fp8_experts* w,
                   __nv_bfloat16* y, float* y32, int64_t most, int num_sms, cudaStream_t s) {
    const int64_t P = (int64_t)sh->T * sh->k;
    Fp8Args a = args_of(b.l, P, sh->H, sh->I, true);
    a.a_scales = b.xs;
    a.b0_scales = w->gate_scales;
    a.b1_scales = w->up_scales;
    a.out_q = b.hq;
    a.out_scales = b.hs;
    const Kernels kn = kernels_for(P, most, sh->E);
    a.with_pairs = !kn.pair;
    if (kn.pair)
        CUDA_TRY(launch_fp8_pair_gate_up(b.xq, P, w->gate, w->up, a, sh->E, num_sms, s),
                 "8-bit gate/up (pairs)");
    if (kn.solo)
        CUDA_TRY(launch_fp8_solo_gate_up(b.xq, P, w->gate, w->up, a, sh->E, num_sms, s),
                 "8-bit gate/up (one-CTA)");
    Fp8Args d = args_of(b.l, P, sh->I, sh->H, false);
    d.with_pairs = !kn.pair;
    d.early_weights = 1;   // the lists were complete before the gate/up kernels started
    d.a_scales = b.hs;
    d.b0_scales = w->down_scales;
    d.out = y;
    d.out32 = y32;
    return run_product(b.hq, w->down, d, kn, sh->E, num_sms, s);
}

moe_status check_balance_args(int32_t T, int32_t E, int32_t k, int32_t S, bool have_seq) {
    if (T < 0) return fail(MOE_ERR_INVALID_ARG, "T = %d < 0", T);
    if (E < 1 || E > kMaxE) return fail(MOE_ERR_INVALID_ARG, "E = %d outside [1, %d]", E, kMaxE);
    if (k < 1 || k > kMaxK || k > E)
        return fail(MOE_ERR_INVALID_ARG, "k = %d outside [1, min(E, %d)]", k, kMaxK);
    if ((int64_t)T * k > (int64_t)INT32_MAX - kTileM)
        return fail(MOE_ERR_INVALID_ARG, "T*k = %lld too large", (long long)T * k);
    if (S < 1) return fail(MOE_ERR_INVALID_ARG, "S = %d < 1", S);
    if (S > INT32_MAX / 2)
        return fail(MOE_ERR_INVALID_ARG, "S = %d too large", S);
    if (!have_seq && S != 1)
        return fail(MOE_ERR_INVALID_ARG, "S = %d without seq_offsets", S);
    return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_quantize_rows(const moe_bf16* x, int32_t rows, int32_t K, uint8_t* q,
                             uint8_t* scales, moe_stream_t stream) {
    if (rows < 0) return fail(MOE_ERR_INVALID_ARG, "rows = %d < 0", rows);
    STATUS_TRY(check_blocks("K", K));
    if (rows == 0) return ok();
    CHECK_PTR(x); CHECK_PTR(q);
    if (!scales) return fail(MOE_ERR_INVALID_ARG, "scales is NULL");
    int sms = 0;
    STATUS_TRY(current_device(&sms));
    CUDA_TRY(launch_quantize_rows((const __nv_bfloat16*)x, rows, K, nullptr, 1, 0, q, scales, sms,
                                  (cudaStream_t)stream), "quantize rows");
    return ok();
}

moe_status moe_quantize_weights(const moe_bf16* W, int32_t n, int32_t N, int32_t K, uint8_t* q,
                                uint8_t* scales, moe_stream_t stream) {
    if (n < 0) return fail(MOE_ERR_INVALID_ARG, "n = %d < 0", n);
    STATUS_TRY(check_blocks("N", N));
    STATUS_TRY(check_blocks("K", K));
    if ((int64_t)n * (N / kSide) * (K / kSide) > INT32_MAX)
        return fail(MOE_ERR_INVALID_ARG, "n = %d matrices are too many blocks", n);
    if (n == 0) return ok();
    CHECK_PTR(W); CHECK_PTR(q);
    if (!scales) return fail(MOE_ERR_INVALID_ARG, "scales is NULL");
    int sms = 0;
    STATUS_TRY(current_device(&sms));
    CUDA_TRY(launch_quantize_matrices((const __nv_bfloat16*)W, n, N, K, q, scales,
                                      (cudaStream_t)stream), "quantize weights");
    return ok();
}

size_t moe_grouped_gemm_fp8_workspace_size(int32_t rows, int32_t E) {
    if (rows < 0 || rows > INT32_MAX - kTileM || E < 1 || E > kMaxE) return 0;
    Carver c(nullptr);
    Lists l;
    take_lists(&c, rows, E, &l);
    return align_up(c.off, 256);
}

moe_status moe_grouped_gemm_fp8(const uint8_t* x, const uint8_t* x_scales, int32_t rows,
                                const int32_t* offsets, int32_t E, int32_t N, int32_t K,
                                const uint8_t* W, const uint8_t* W_scales, moe_bf16* y, void* ws,
                                size_t ws_bytes, moe_stream_t stream) {
    if (rows < 0 || rows > INT32_MAX - kTileM)
        return fail(MOE_ERR_INVALID_ARG, "rows = %d out of range", rows);
    if (E < 1 || E > kMaxE) return fail(MOE_ERR_INVALID_ARG, "E = %d outside [1, %d]", E, kMaxE);
    STATUS_TRY(check_blocks("N", N));
    STATUS_TRY(check_blocks("K", K));
    if (rows == 0) return ok();
    CHECK_PTR(x); CHECK_PTR(x_scales); CHECK_PTR(W); CHECK_PTR(W_scales); CHECK_PTR(y);
    if (!offsets) return fail(MOE_ERR_INVALID_ARG, "offsets is NULL");
    STATUS_TRY(check_ws(ws, ws_bytes, moe_grouped_gemm_fp8_workspace_size(rows, E)));
    int sms = 0;
    STATUS_TRY(current_device(&sms));
    cudaStream_t s = (cudaStream_t)stream;
    Carver c(ws);
    Lists l;
    take_lists(&c, rows, E, &l);
    const PdlScope pdl(rows <= kPermChunk);
    Fp8Args a = args_of(l, rows, K, N, false);
    if (E == 1) a.group = offsets;
    else CUDA_TRY(launch_plan_groups(offsets, rows, E, plan_of(l, E), s), "plan");
    a.a_scales = x_scales;
    a.b0_scales = W_scales;
    a.out = (__nv_bfloat16*)y;
    const Kernels kn = kernels_for(rows, rows, E);
    a.with_pairs = !kn.pair;
    STATUS_TRY(run_product(x, W, a, kn, E, sms, s));
    return ok();
}

size_t moe_expert_ffn_fp8_workspace_size(const moe_shape* shape) {
    if (check_shape_status(shape) != MOE_OK) return 0;
    FfnBufs b;
    return carve_ffn(shape, nullptr, &b);
}

moe_status moe_expert_ffn_fp8(const moe_shape* shape, const moe_bf16* x, const int32_t* perm,
                              const int32_t* offsets, const moe_fp8_experts* experts,
                              moe_bf16* y_sorted, void* ws, size_t ws_bytes,
                              moe_stream_t stream) {
    STATUS_TRY(check_shape_status(shape));
    if (shape->T == 0) return ok();
    CHECK_PTR(x); CHECK_PTR(y_sorted);
    if (!perm || !offsets) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
    STATUS_TRY(check_experts(experts));
    FfnBufs b;
    STATUS_TRY(check_ws(ws, ws_bytes, carve_ffn(shape, nullptr, &b)));
    carve_ffn(shape, ws, &b);
    int sms = 0;
    STATUS_TRY(current_device(&sms));
    cudaStream_t s = (cudaStream_t)stream;
    const int64_t P = (int64_t)shape->T * shape->k;
    const PdlScope pdl(P <= kPermChunk);
    CUDA_TRY(launch_plan_groups(offsets, (int)P, shape->E, plan_of(b.l, shape->E), s), "plan");
    CUDA_TRY(launch_invert_perm(perm, P, b.inv_perm, sms, s), "invert perm");
    CUDA_TRY(launch_quantize_rows((const __nv_bfloat16*)x, shape->T, shape->H, b.inv_perm,
                                  shape->k, P, b.xq, b.xs, sms, s), "quantize rows");
    STATUS_TRY(run_ffn(shape, b, experts, (__nv_bfloat16*)y_sorted, nullptr, P, sms, s));
    return ok();
}

size_t moe_fp8_workspace_size(const moe_shape* shape) {
    if (check_shape_status(shape) != MOE_OK) return 0;
    FwdBufs b;
    return carve_fwd(shape, nullptr, &b);
}

moe_status moe_forward_fp8(const moe_shape* shape, const float* logits, const moe_bf16* x,
                           const moe_fp8_experts* experts, moe_bf16* out, int32_t* topk_idx,
                           float* gates, void* ws, size_t ws_bytes, moe_stream_t stream) {
    STATUS_TRY(check_shape_status(shape));
    if (shape->T == 0) return ok();
    if (!logits) return fail(MOE_ERR_INVALID_ARG, "logits is NULL");
    CHECK_PTR(x); CHECK_PTR(out);
    STATUS_TRY(check_experts(experts));
    FwdBufs b;
    STATUS_TRY(check_ws(ws, ws_bytes, carve_fwd(shape, nullptr, &b)));
    carve_fwd(shape, ws, &b);
    int sms = 0;
    STATUS_TRY(current_device(&sms));
    cudaStream_t s = (cudaStream_t)stream;
    const int T = shape->T, E = shape->E, k = shape->k;
    const int64_t P = (int64_t)T * k;
    const PdlScope pdl(P <= kPermChunk);
    int32_t* idx = topk_idx ? topk_idx : b.idx;
    float* g = gates ? gates : b.gates;
    const Plan plan = plan_of(b.f.l, E);
    const int64_t nch = (P + kPermChunk - 1) / kPermChunk;
    if (fp8_prologue_fits(T)) {
        CUDA_TRY(launch_fp8_prologue(logits, (const __nv_bfloat16*)x, T, E, k, shape->H, idx, g,
                                     b.f.inv_perm, b.f.l.thin, b.f.l.hdr, b.f.xq, b.f.xs, s),
                 "prologue");
    } else {
        CUDA_TRY(launch_route(logits, T, E, k, idx, g, s), "route");
        CUDA_TRY(launch_permute(idx, T, E, k, b.counts, b.offsets, b.perm, b.f.inv_perm, b.chunk,
                                b.chunk + nch * E, b.f.l.hdr, &plan, s), "permute");
        CUDA_TRY(launch_quantize_rows((const __nv_bfloat16*)x, T, shape->H, b.f.inv_perm, k, P,
                                      b.f.xq, b.f.xs, sms, s), "quantize rows");
    }
    __nv_bfloat16* y = (__nv_bfloat16*)b.y;
    float* y32 = fp32_y(shape) ? (float*)b.y : nullptr;
    STATUS_TRY(run_ffn(shape, b.f, experts, y, y32, T, sms, s));
    if (y32)
        CUDA_TRY(launch_combine_f32(y32, b.f.inv_perm, g, T, k, shape->H, (__nv_bfloat16*)out, s),
                 "combine");
    else
        CUDA_TRY(launch_combine(y, b.f.inv_perm, g, T, k, shape->H, (__nv_bfloat16*)out, sms, s),
                 "combine");
    return ok();
}

size_t moe_balance_workspace_size(int32_t T, int32_t E, int32_t S) {
    if (check_balance_args(T, E, 1, S, true) != MOE_OK) return 0;
    BalanceArgs a = {};
    a.T = T;
    a.E = E;
    a.S = S;
    return carve_balance(nullptr, &a);
}

moe_status moe_balance(const float* logits, const int32_t* topk_idx, int32_t T, int32_t E,
                       int32_t k, const int32_t* seq_offsets, int32_t S, float coef, float* loss,
                       int32_t* counts, float* stats, void* ws, size_t ws_bytes,
                       moe_stream_t stream) {
    STATUS_TRY(check_balance_args(T, E, k, S, seq_offsets != nullptr));
    if (!loss || !counts || (T > 0 && (!logits || !topk_idx || !stats)))
        return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
    if (!aligned(stats, 8)) return fail(MOE_ERR_INVALID_ARG, "stats is not 8-byte aligned");
    BalanceArgs a = {};
    a.T = T;
    a.E = E;
    a.k = k;
    a.S = S;
    a.seq = seq_offsets;
    a.coef = coef;
    a.loss = loss;
    a.counts = counts;
    STATUS_TRY(check_ws(ws, ws_bytes, carve_balance(nullptr, &a)));
    carve_balance(ws, &a);
    int sms = 0;
    STATUS_TRY(current_device(&sms));
    const PdlScope pdl(true);
    CUDA_TRY(launch_balance(logits, topk_idx, (float2*)stats, a, sms, (cudaStream_t)stream),
             "balance");
    return ok();
}

moe_status moe_balance_backward(const float* logits, const float* stats, const int32_t* counts,
                                const int32_t* seq_offsets, int32_t T, int32_t E, int32_t k,
                                int32_t S, float coef, const float* d_loss,
                                const int32_t* topk_idx, const float* gates, const float* d_gates,
                                float* d_logits, moe_stream_t stream) {
    STATUS_TRY(check_balance_args(T, E, k, S, seq_offsets != nullptr));
    if (T == 0) return ok();
    if (!logits || !stats || !counts || !d_logits) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
    if (!aligned(stats, 8)) return fail(MOE_ERR_INVALID_ARG, "stats is not 8-byte aligned");
    if ((d_gates != nullptr) != (topk_idx != nullptr) || (d_gates != nullptr) != (gates != nullptr))
        return fail(MOE_ERR_INVALID_ARG, "topk_idx, gates and d_gates come together");
    int sms = 0;
    STATUS_TRY(current_device(&sms));
    BalanceArgs a = {};
    a.T = T;
    a.E = E;
    a.k = k;
    a.S = S;
    a.seq = seq_offsets;
    a.coef = coef;
    a.counts = const_cast<int32_t*>(counts);   // read only there
    const PdlScope pdl(true);
    CUDA_TRY(launch_balance_backward(logits, (const float2*)stats, d_loss, topk_idx, gates,
                                     d_gates, d_logits, a, sms, (cudaStream_t)stream),
             "balance backward");
    return ok();
}

}  // extern "C"

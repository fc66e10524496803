// api_train.cu -- the C ABI of the experts' training passes and of the product
// with an epilogue (include/moe.h): argument validation, workspace layout and
// the launch sequence of each entry point.  Nothing here allocates or throws.

#include "api_common.cuh"
#include "train.cuh"

using namespace moe;

namespace {

// Rows of B per CTA of the tile kernel: the narrow build where the groups hold
// at most 3/4 of a narrow chunk (128 rows) on average, else the wide one.
int rows_per_cta(int64_t rows, int E) { return rows <= (int64_t)96 * E ? kThinRows : kWideRows; }

// Whether a kernel may start while the one before it finishes.  It gains at the
// ends of short launches and costs long ones (E, H, I, tokens; backward, us
// with / without): 1, 4096, 2048, 8192: 482 / 506; 32, 2048, 1024, 1999: 267 /
// 282; 384, 4096, 2048, 16384: 13300 / 12750.  Counted in weight tiles per SM.
bool overlap(const moe_shape* sh, int num_sms) {
    return (int64_t)sh->E * 3 * (sh->H / 256) * (sh->I / 256) <= (int64_t)64 * num_sms;
}

struct Lists {
    WsHeader* hdr;
    RowLists l;
};
void take_lists(Carver* c, int64_t rows, int E, int most, Lists* l) {
    l->hdr = c->take<WsHeader>(1);
    l->l.n_chunks = c->take<int32_t>(1);
    l->l.ends = c->take<int32_t>(2);
    l->l.groups = c->take<RowChunk>((size_t)E);
    l->l.chunks = c->take<RowChunk>((size_t)max_chunks(rows, E, most));
}

// The tile kernel's arguments over the lists, or (dense) over one group.
TileArgs args_of(const Lists& l, bool dense, int64_t rows, int E) {
    TileArgs a = {};
    a.hdr = l.hdr;
    a.rows = (int)rows;
    a.E = E;
    if (!dense) {
        a.chunks = l.l.chunks;
        a.groups = l.l.groups;
        a.n_chunks = l.l.n_chunks;
    }
    a.wait_cycles = main_wait_cycles();
    return a;
}

struct FwdBufs {
    Lists l;
    __nv_bfloat16 *xs, *h;
};
size_t carve_fwd(const moe_shape* sh, void* ws, FwdBufs* b) {
    const int64_t P = (int64_t)sh->T * sh->k;
    Carver c(ws);
    take_lists(&c, P, sh->E, 2 * rows_per_cta(P, sh->E), &b->l);
    b->xs = c.take<__nv_bfloat16>((size_t)(P * sh->H));
    b->h = c.take<__nv_bfloat16>((size_t)(P * sh->I));
    return align_up(c.off, 256);
}

struct BwdBufs {
    Lists l;
    __nv_bfloat16 *x, *d;          // padded rows of x and d_out
    float* dx;                     // each slot's part of d_x
    __nv_bfloat16 *h, *dg, *du;    // padded
    float* parts;
};
size_t carve_bwd(const moe_shape* sh, void* ws, BwdBufs* b) {
    const int64_t P = (int64_t)sh->T * sh->k, pad = padded_rows(P, sh->E);
    Carver c(ws);
    take_lists(&c, P, sh->E, 2 * rows_per_cta(P, sh->E), &b->l);
    b->x = c.take<__nv_bfloat16>((size_t)(pad * sh->H));
    b->d = c.take<__nv_bfloat16>((size_t)(pad * sh->H));
    b->dx = c.take<float>((size_t)(P * sh->H));
    b->h = c.take<__nv_bfloat16>((size_t)(pad * sh->I));
    b->dg = c.take<__nv_bfloat16>((size_t)(pad * sh->I));
    b->du = c.take<__nv_bfloat16>((size_t)(pad * sh->I));
    b->parts = c.take<float>((size_t)(P * (sh->I / 32)));
    return align_up(c.off, 256);
}

// Lists and gates are read four bytes at a time (a slice of a longer list will do).
#define CHECK_WORDS(p)                                                            \
    do {                                                                          \
        if (!aligned((p), 4)) return fail(MOE_ERR_INVALID_ARG, "%s is not 4-byte aligned", #p); \
    } while (0)

// Route lists given together, or a dense block.
moe_status check_lists(const moe_shape* sh, const int32_t* perm, const int32_t* offsets, bool* dense) {
    *dense = !perm && !offsets;
    if (!*dense && (!perm || !offsets))
        return fail(MOE_ERR_INVALID_ARG, "perm and offsets come together");
    if (*dense && (sh->E != 1 || sh->k != 1))
        return fail(MOE_ERR_INVALID_ARG, "no route lists with E = %d, k = %d (a dense block has 1, 1)",
                    sh->E, sh->k);
    CHECK_WORDS(perm); CHECK_WORDS(offsets);
    return MOE_OK;
}

// need_x: the call reads or writes the record's x.
moe_status check_saved(const moe_saved* v, bool need_x) {
    if (!v) return fail(MOE_ERR_INVALID_ARG, "saved is NULL");
    CHECK_PTR(v->gate); CHECK_PTR(v->up);
    if (need_x) CHECK_PTR(v->x);
    if (v->fp8 && ((need_x && !v->x_scales) || !v->gate_scales || !v->up_scales))
        return fail(MOE_ERR_INVALID_ARG, "8-bit checkpoints without scales");
    return MOE_OK;
}

moe_status check_product(int32_t rows, int32_t E, int32_t N, int32_t K) {
    constexpr int kMost = 65536;
    if (rows < 0 || rows > INT32_MAX - kTileM)
        return fail(MOE_ERR_INVALID_ARG, "rows = %d out of range", rows);
    if (E < 1 || E > kMaxE) return fail(MOE_ERR_INVALID_ARG, "E = %d outside [1, %d]", E, kMaxE);
    if (N < 1) return fail(MOE_ERR_INVALID_ARG, "N = %d is not positive", N);
    if (K < 8 || K % 8) return fail(MOE_ERR_INVALID_ARG, "K = %d is not a positive multiple of 8", K);
    if (N > kMost || K > kMost) return fail(MOE_ERR_UNSUPPORTED, "N and K are limited to %d", kMost);
    return MOE_OK;
}
size_t carve_product(int32_t rows, int32_t E, void* ws, Lists* l) {
    Carver c(ws);
    take_lists(&c, rows, E, 2 * rows_per_cta(rows, E), l);
    return align_up(c.off, 256);
}

}  // namespace

extern "C" {

size_t moe_expert_ffn_train_workspace_size(const moe_shape* shape) {
    if (check_shape_status(shape) != MOE_OK) return 0;
    FwdBufs b;
    return carve_fwd(shape, nullptr, &b);
}

moe_status moe_expert_ffn_train(const moe_shape* shape, const moe_bf16* x, const int32_t* perm,
                                const int32_t* offsets, const moe_bf16* W_gate,
                                const moe_bf16* W_up, const moe_bf16* W_down, moe_bf16* y_sorted,
                                const moe_saved* saved, void* ws, size_t ws_bytes,
                                moe_stream_t stream) {
    STATUS_TRY(check_shape_status(shape));
    if (shape->T == 0) return ok();
    bool dense;
    STATUS_TRY(check_lists(shape, perm, offsets, &dense));
    CHECK_PTR(x); CHECK_PTR(W_gate); CHECK_PTR(W_up); CHECK_PTR(W_down); CHECK_PTR(y_sorted);
    STATUS_TRY(check_saved(saved, saved && saved->fp8));
    FwdBufs b;
    STATUS_TRY(check_ws(ws, ws_bytes, carve_fwd(shape, nullptr, &b)));
    carve_fwd(shape, ws, &b);
    int sms = 0;
    STATUS_TRY(current_device(&sms));
    cudaStream_t s = (cudaStream_t)stream;
    const int T = shape->T, E = shape->E, k = shape->k, H = shape->H, I = shape->I;
    const int64_t P = (int64_t)T * k;
    const int nb = rows_per_cta(P, E), most = 2 * nb;
    const PdlScope pdl(overlap(shape, sms));
    const __nv_bfloat16* xs = (const __nv_bfloat16*)x;
    if (saved->fp8)
        CUDA_TRY(launch_quantize_rows(xs, T, H, nullptr, 1, 0, (uint8_t*)saved->x, saved->x_scales,
                                      sms, s), "quantize rows");
    if (!dense) {
        CUDA_TRY(launch_forward_rows(xs, perm, k, H, offsets, (int)P, E, most, b.xs, b.l.l, b.l.hdr, sms, s),
                 "sorted rows");
        xs = b.xs;
    }
    TileArgs a = args_of(b.l, dense, P, E);
    a.out = b.h;
    a.gate = saved->gate;
    a.up = saved->up;
    a.gate_scales = saved->gate_scales;
    a.up_scales = saved->up_scales;
    CUDA_TRY(launch_train_gate_up(xs, P, (const __nv_bfloat16*)W_gate, (const __nv_bfloat16*)W_up,
                                  H, I, saved->fp8 != 0, nb, a, sms, s), "gate/up");
    a.out = (__nv_bfloat16*)y_sorted;
    CUDA_TRY(launch_train_down(b.h, P, (const __nv_bfloat16*)W_down, H, I, nb, a, sms, s), "down");
    return ok();
}

size_t moe_expert_ffn_backward_workspace_size(const moe_shape* shape) {
    if (check_shape_status(shape) != MOE_OK) return 0;
    BwdBufs b;
    return carve_bwd(shape, nullptr, &b);
}

moe_status moe_expert_ffn_backward(const moe_shape* shape, const moe_bf16* d_out,
                                   const float* gates, const moe_saved* saved,
                                   const int32_t* perm, const int32_t* offsets,
                                   const int32_t* inv_perm, const moe_bf16* W_gate,
                                   const moe_bf16* W_up, const moe_bf16* W_down, moe_bf16* d_x,
                                   float* d_gates, moe_bf16* dW_gate, moe_bf16* dW_up,
                                   moe_bf16* dW_down, void* ws, size_t ws_bytes,
                                   moe_stream_t stream) {
    STATUS_TRY(check_shape_status(shape));
    const bool weights = dW_gate || dW_up || dW_down;
    if (weights) {
        CHECK_PTR(dW_gate); CHECK_PTR(dW_up); CHECK_PTR(dW_down);
    }
    const int T = shape->T, E = shape->E, k = shape->k, H = shape->H, I = shape->I;
    cudaStream_t s = (cudaStream_t)stream;
    int sms = 0;
    if (T == 0) {       // no row: the weights' gradients are zero
        if (!weights) return ok();
        STATUS_TRY(current_device(&sms));
        for (moe_bf16* w : {dW_gate, dW_up, dW_down})
            CUDA_TRY(cudaMemsetAsync(w, 0, (size_t)E * H * I * 2, s), "clear weight gradients");
        return ok();
    }
    bool dense;
    STATUS_TRY(check_lists(shape, perm, offsets, &dense));
    if (dense != !inv_perm) return fail(MOE_ERR_INVALID_ARG, "perm, offsets and inv_perm come together");
    if (d_gates && !gates) return fail(MOE_ERR_INVALID_ARG, "d_gates without gates");
    CHECK_WORDS(inv_perm); CHECK_WORDS(gates); CHECK_WORDS(d_gates);
    CHECK_PTR(d_out); CHECK_PTR(W_gate); CHECK_PTR(W_up); CHECK_PTR(W_down);
    if (d_x) CHECK_PTR(d_x);
    STATUS_TRY(check_saved(saved, weights));
    BwdBufs b;
    STATUS_TRY(check_ws(ws, ws_bytes, carve_bwd(shape, nullptr, &b)));
    carve_bwd(shape, ws, &b);
    STATUS_TRY(current_device(&sms));
    const int64_t P = (int64_t)T * k, pad = padded_rows(P, E);
    const int nb = rows_per_cta(P, E), most = 2 * nb;
    const PdlScope pdl(overlap(shape, sms));
    // x (for the weights' gradients alone) and d_out by sorted row: the caller's
    // own where the block is dense
    const __nv_bfloat16 *x = (const __nv_bfloat16*)saved->x, *d = (const __nv_bfloat16*)d_out;
    const int64_t xd_rows = dense ? T : pad;
    if (!dense) {
        const BackwardRows q = {saved->x, saved->fp8 ? saved->x_scales : nullptr, d, perm, inv_perm, offsets,
                                weights ? b.x : nullptr, b.d, b.l.l, b.l.hdr, T, k, H, E, most};
        CUDA_TRY(launch_backward_rows(q, sms, s), "sorted rows");
        x = b.x;
        d = b.d;
    } else if (saved->fp8 && weights) {
        CUDA_TRY(launch_dequantize_rows((const uint8_t*)saved->x, saved->x_scales, T, H, b.x, sms, s),
                 "dequantize rows");
        x = b.x;
    }
    TileArgs a = args_of(b.l, dense, P, E);
    a.padded = !dense;
    a.gate = saved->gate;
    a.up = saved->up;
    a.gate_scales = saved->gate_scales;
    a.up_scales = saved->up_scales;
    a.gates = gates;
    a.perm = perm;
    a.out = b.h;
    a.d_gate = b.dg;
    a.d_up = b.du;
    a.gate_parts = d_gates ? b.parts : nullptr;
    CUDA_TRY(launch_hidden_grad(d, xd_rows, (const __nv_bfloat16*)W_down, H, I, saved->fp8 != 0, nb,
                                pad, a, sms, s), "gradient of the projections");
    // The weights' gradients and that of x need nothing of one another: the
    // second starts as the first one's CTAs run out of items (the first waits
    // for the hidden gradients, so they are complete when the second starts).
    if (weights) {
        TileArgs w = a;
        w.out = (__nv_bfloat16*)dW_down;
        w.d_gate = (__nv_bfloat16*)dW_gate;
        w.d_up = (__nv_bfloat16*)dW_up;
        CUDA_TRY(launch_weight_grad(b.h, b.dg, b.du, pad, x, d, xd_rows, H, I, w, sms, s),
                 "gradients of the weights");
    }
    if (d_x) {
        a.out = dense ? (__nv_bfloat16*)d_x : nullptr;
        a.out32 = dense ? nullptr : b.dx;
        a.early = weights && overlap(shape, sms);
        CUDA_TRY(launch_input_grad(b.dg, b.du, pad, (const __nv_bfloat16*)W_gate,
                                   (const __nv_bfloat16*)W_up, H, I, nb, a, sms, s), "gradient of x");
    }
    __nv_bfloat16* sums = d_x && !dense ? (__nv_bfloat16*)d_x : nullptr;
    if (sums || d_gates)
        CUDA_TRY(launch_finish(b.dx, sums, b.parts, I / 32, d_gates, inv_perm, dense ? nullptr : b.l.l.ends, T, k, H,
                               sms, s), "sums over slots");
    return ok();
}

moe_status moe_dequantize_rows(const uint8_t* q, const uint8_t* scales, int32_t rows, int32_t K,
                               moe_bf16* x, moe_stream_t stream) {
    if (rows < 0) return fail(MOE_ERR_INVALID_ARG, "rows = %d < 0", rows);
    if (K < 128 || K % 128) return fail(MOE_ERR_INVALID_ARG, "K = %d is not a positive multiple of 128", K);
    if (K > kMaxHidden) return fail(MOE_ERR_UNSUPPORTED, "K is limited to %d", kMaxHidden);
    if (rows == 0) return ok();
    CHECK_PTR(q); CHECK_PTR(x);
    if (!scales) return fail(MOE_ERR_INVALID_ARG, "scales is NULL");
    int sms = 0;
    STATUS_TRY(current_device(&sms));
    CUDA_TRY(launch_dequantize_rows(q, scales, rows, K, (__nv_bfloat16*)x, sms, (cudaStream_t)stream),
             "dequantize rows");
    return ok();
}

size_t moe_grouped_gemm_workspace_size(int32_t rows, int32_t E, int32_t N, int32_t K) {
    if (check_product(rows, E, N, K) != MOE_OK) return 0;
    Lists l;
    return carve_product(rows, E, nullptr, &l);
}

moe_status moe_grouped_gemm(const moe_bf16* x, int32_t rows, const int32_t* offsets, int32_t E,
                            int32_t N, int32_t K, const moe_bf16* W, const float* bias,
                            int32_t activation, const moe_bf16* residual, void* y, int32_t y_fp32,
                            void* ws, size_t ws_bytes, moe_stream_t stream) {
    STATUS_TRY(check_product(rows, E, N, K));
    if (activation < MOE_ACT_NONE || activation > MOE_ACT_SILU)
        return fail(MOE_ERR_INVALID_ARG, "activation = %d is none of moe_activation", activation);
    if (!offsets && E != 1) return fail(MOE_ERR_INVALID_ARG, "offsets is NULL with E = %d", E);
    if (rows == 0) return ok();
    CHECK_PTR(x); CHECK_PTR(W); CHECK_PTR(y);
    CHECK_WORDS(offsets); CHECK_WORDS(bias);
    if (!aligned(residual, 2)) return fail(MOE_ERR_INVALID_ARG, "residual is not 2-byte aligned");
    Lists l;
    STATUS_TRY(check_ws(ws, ws_bytes, carve_product(rows, E, nullptr, &l)));
    carve_product(rows, E, ws, &l);
    int sms = 0;
    STATUS_TRY(current_device(&sms));
    cudaStream_t s = (cudaStream_t)stream;
    const int nb = rows_per_cta(rows, E), most = 2 * nb;
    const PdlScope pdl(rows <= kPermChunk);
    if (!offsets && rows <= kFewRows) {
        const ProductEpilogue e = {bias, (const __nv_bfloat16*)residual, y_fp32 ? nullptr : (__nv_bfloat16*)y,
                                   y_fp32 ? (float*)y : nullptr, activation};
        CUDA_TRY(launch_product_rows((const __nv_bfloat16*)x, rows, (const __nv_bfloat16*)W, N, K, e, s),
                 "product of few rows");
        return ok();
    }
    if (offsets) CUDA_TRY(launch_plan_rows(offsets, rows, E, most, l.l, l.hdr, s), "plan");
    TileArgs a = args_of(l, !offsets, rows, E);
    a.out = y_fp32 ? nullptr : (__nv_bfloat16*)y;
    a.out32 = y_fp32 ? (float*)y : nullptr;
    a.bias = bias;
    a.residual = (const __nv_bfloat16*)residual;
    a.act = activation;
    a.vec = N % 8 == 0 && aligned(residual, 16);
    CUDA_TRY(launch_product((const __nv_bfloat16*)x, rows, (const __nv_bfloat16*)W, N, K, nb, a, sms, s),
             "product");
    return ok();
}

}  // extern "C"

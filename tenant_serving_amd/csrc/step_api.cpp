// C ABI of the operators between the linears of a step: argument validation
// and dispatch.  See include/bitdelta_step.h for the contract.
#include <hip/hip_runtime.h>

#include <cmath>

#include "step_internal.h"

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr float kMaxScale = 1152921504606846976.0f;  // 2^60: times log2(e) it stays far from infinity

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool in_type(int32_t t) { return t == BD_BF16 || t == BD_FP32; }

bd_status finish(hipError_t e) {
    if (e == hipSuccess) return BD_OK;
    bd::note_hip_error(e);
    return BD_ERR_HIP;
}

bd_status check_kv(const bd_kv* kv) {
    if (!kv || !kv->k || !kv->v) return BD_ERR_NULL;
    if (kv->type != BD_BF16 && kv->type != BD_E4M3 && kv->type != BD_E2M1) return BD_ERR_MODE;
    const bool codes = kv->type != BD_BF16;
    if (codes && (!kv->k_scales || !kv->v_scales)) return BD_ERR_NULL;
    if (kv->num_heads < 1 || kv->num_heads > 65535 || kv->head_dim < 16 || kv->head_dim > 256 ||
        kv->head_dim % (kv->type == BD_E2M1 ? bd::kGroup4 : 16) != 0 || kv->page_size < 8 || kv->page_size > 4096 || kv->page_size % 8 != 0 ||
        kv->num_pages < 1 || kv->num_pages > kMaxRows / kv->page_size)
        return BD_ERR_SHAPE;
    const int64_t unit = codes ? 16 : 8;  // elements of 16 bytes
    for (const int64_t s : {kv->page_stride, kv->head_stride, kv->token_stride}) {
        if (s < 0 || s / unit >= int64_t(1) << 32) return BD_ERR_SHAPE;
        if (s % unit != 0) return BD_ERR_ALIGN;
    }
    if (!aligned(kv->k, 16) || !aligned(kv->v, 16)) return BD_ERR_ALIGN;
    if (codes && (!aligned(kv->k_scales, 8) || !aligned(kv->v_scales, 8))) return BD_ERR_ALIGN;
    return BD_OK;
}

bd_status check_strides(const int64_t* s, int32_t type) {
    const int64_t unit = type == BD_FP32 ? 4 : 8;
    for (int i = 0; i < 2; ++i) {
        if (s[i] < 0) return BD_ERR_SHAPE;
        if (s[i] % unit != 0) return BD_ERR_ALIGN;
    }
    return BD_OK;
}

// A cap of scores: none, or one whose inverse and square are ordinary numbers.
bool cap_ok(float cap) { return cap == 0.0f || (cap >= 1.0f / kMaxScale && cap <= kMaxScale); }

// Sizes of an attention call that its kernels can index.
bool attend_shape(int64_t B, int64_t Hq, int64_t H, int64_t D, int64_t page_size, int64_t max_pages) {
    if (B < 1 || B > kMaxRows || H < 1 || H > 65535 || Hq < H || Hq > 65535 || Hq % H != 0) return false;
    if (D < 16 || D > 256 || D % 16 != 0 || page_size < 8 || page_size > 4096 || page_size % 8 != 0) return false;
    if (max_pages < 1 || max_pages > bd::kAttendMaxTokens / page_size) return false;
    const int64_t rows = B * H * ((Hq / H + 15) / 16);  // of units of 128 tokens
    const int64_t units = (max_pages * page_size + 127) / 128;
    return rows <= int64_t(1) << 23 && (units + 4) * rows <= int64_t(1) << 30;
}

// The same of a prompt's: rows and workgroups below 2^31 and 2^23.
bool prompt_shape(int64_t T, int64_t B, int64_t Hq, int64_t H, int64_t D, int64_t page_size, int64_t max_pages) {
    if (T < 1 || B < 1 || H < 1 || H > 65535 || Hq < H || Hq > 65535 || Hq % H != 0) return false;
    if (D < 16 || D > 256 || D % 16 != 0 || page_size < 8 || page_size > 4096 || page_size % 8 != 0) return false;
    if (max_pages < 1 || max_pages > bd::kAttendMaxTokens / page_size) return false;
    return T <= (int64_t(1) << 29) / Hq && B <= (int64_t(1) << 22) / H;
}

}  // namespace

extern "C" {

bd_status bd_rms_norm(const void* x, int32_t x_type, const void* residual, void* residual_out,
                      int32_t residual_type, const void* gain, int32_t gain_type, int32_t num_gains,
                      const int32_t* variant_ids, float eps, void* out, int32_t out_type, uint8_t* scales,
                      int64_t M, int64_t d, void* stream) {
    if (!gain) return BD_ERR_NULL;
    if (M > 0 && (!x || !out || (out_type == BD_E4M3 && !scales))) return BD_ERR_NULL;
    if (M > 0 && (residual == nullptr) != (residual_out == nullptr)) return BD_ERR_NULL;
    if (!in_type(x_type) || !in_type(gain_type) || (out_type != BD_BF16 && out_type != BD_E4M3)) return BD_ERR_MODE;
    if (residual && !in_type(residual_type)) return BD_ERR_MODE;
    if (M < 0 || M > kMaxRows || d < 8 || d > bd::kNormMaxD || d % 8 != 0 || num_gains < 1 || !(eps >= 0.0f))
        return BD_ERR_SHAPE;
    if (!aligned(gain, 16) || !aligned(x, 16) || !aligned(residual, 16) || !aligned(residual_out, 16) ||
        !aligned(out, out_type == BD_E4M3 ? 8 : 16) || !aligned(variant_ids, 4))
        return BD_ERR_ALIGN;
    if (M == 0) return BD_OK;
    const bd_status st = bd::check_current_device(nullptr);
    if (st != BD_OK) return st;
    const bd::NormArgs a{x, residual, residual_out, gain, variant_ids, out, scales, eps, num_gains,
                         gain_type == BD_FP32, (int32_t)d, M};
    return finish(bd::launch_norm(a, x_type == BD_FP32, !residual ? 0 : residual_type == BD_FP32 ? 2 : 1,
                                  out_type == BD_E4M3, static_cast<hipStream_t>(stream)));
}

bd_status bd_rotary(const bd_rotary_rows* rows, int32_t count, int32_t x_type, int32_t out_type, int32_t head_dim,
                    int32_t turned, int32_t interleaved, const int32_t* positions, const uint64_t* steps,
                    float gain, int64_t T, void* stream) {
    if (!rows || !steps || (T > 0 && !positions)) return BD_ERR_NULL;
    if (!in_type(x_type) || !in_type(out_type)) return BD_ERR_MODE;
    if (count < 1 || count > 2 || head_dim < 16 || head_dim > 256 || head_dim % 16 != 0 || turned < 2 ||
        turned > head_dim || turned % 2 != 0 || !std::isfinite(gain) || T < 0 || T > kMaxRows)
        return BD_ERR_SHAPE;
    bd::RotaryArgs a{};
    for (int i = 0; i < count; ++i) {
        const bd_rotary_rows& r = rows[i];
        if (T > 0 && (!r.x || !r.out)) return BD_ERR_NULL;
        if (r.heads < 1 || r.heads > 65535) return BD_ERR_SHAPE;
        bd_status st = check_strides(r.x_strides, x_type);
        if (st != BD_OK || (st = check_strides(r.out_strides, out_type)) != BD_OK) return st;
        if (!aligned(r.x, 16) || !aligned(r.out, 16)) return BD_ERR_ALIGN;
        a.x[i] = r.x, a.out[i] = r.out, a.heads[i] = r.heads;
        a.xs[i] = {r.x_strides[0], r.x_strides[1]};
        a.os[i] = {r.out_strides[0], r.out_strides[1]};
    }
    if (!aligned(positions, 4) || !aligned(steps, 8)) return BD_ERR_ALIGN;
    if (T == 0) return BD_OK;
    const bd_status st = bd::check_current_device(nullptr);
    if (st != BD_OK) return st;
    a.positions = positions, a.steps = steps, a.gain = gain, a.dim = head_dim, a.turned = turned, a.T = T;
    return finish(bd::launch_rotary(a, x_type == BD_FP32, out_type == BD_FP32, interleaved != 0,
                                    static_cast<hipStream_t>(stream)));
}

bd_status bd_kv_write(const bd_kv* kv, const void* k, const int64_t* k_strides, const void* v,
                      const int64_t* v_strides, int32_t type, const int32_t* slots, int64_t T, void* stream) {
    bd_status st = check_kv(kv);
    if (st != BD_OK) return st;
    if (!k_strides || !v_strides || (T > 0 && (!k || !v || !slots))) return BD_ERR_NULL;
    if (!in_type(type)) return BD_ERR_MODE;
    if (T < 0 || T > int64_t(1) << 28) return BD_ERR_SHAPE;
    if ((st = check_strides(k_strides, type)) != BD_OK || (st = check_strides(v_strides, type)) != BD_OK) return st;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4)) return BD_ERR_ALIGN;
    if (T == 0) return BD_OK;
    if ((st = bd::check_current_device(nullptr)) != BD_OK) return st;
    return finish(bd::launch_kv_write(*kv, k, {k_strides[0], k_strides[1]}, v, {v_strides[0], v_strides[1]},
                                      type == BD_FP32, slots, T, static_cast<hipStream_t>(stream)));
}

bd_status bd_kv_read(const bd_kv* kv, const int32_t* slots, int64_t T, uint16_t* k_out, uint16_t* v_out,
                     void* stream) {
    bd_status st = check_kv(kv);
    if (st != BD_OK) return st;
    if (T > 0 && (!slots || !k_out || !v_out)) return BD_ERR_NULL;
    if (T < 0 || T > kMaxRows) return BD_ERR_SHAPE;
    if (!aligned(slots, 4) || !aligned(k_out, 16) || !aligned(v_out, 16)) return BD_ERR_ALIGN;
    if (T == 0) return BD_OK;
    if ((st = bd::check_current_device(nullptr)) != BD_OK) return st;
    return finish(bd::launch_kv_read(*kv, slots, T, k_out, v_out, static_cast<hipStream_t>(stream)));
}

size_t bd_attend_workspace_bytes(int64_t B, int64_t num_q_heads, int64_t num_heads, int64_t head_dim,
                                 int64_t page_size, int64_t max_pages) {
    if (!attend_shape(B, num_q_heads, num_heads, head_dim, page_size, max_pages)) return 0;
    return bd::attend_workspace_bytes(B, num_q_heads, num_heads, head_dim, page_size, max_pages);
}

bd_status bd_attend_scores(const bd_kv* kv, const void* q, int32_t q_type, const int64_t* q_strides,
                    int32_t num_q_heads, const int32_t* page_table, int64_t table_stride, int64_t max_pages,
                    const int32_t* lengths, int64_t B, float scale, const bd_scores* scores,
                    uint16_t* out, float* lse,
                    void* workspace, size_t workspace_bytes, void* stream) {
    bd_status st = check_kv(kv);
    if (st != BD_OK) return st;
    if (!q_strides || (B > 0 && (!q || !page_table || !lengths || !out))) return BD_ERR_NULL;
    if (!in_type(q_type)) return BD_ERR_MODE;
    if (B < 0 || table_stride < 0 || !(std::fabs(scale) <= kMaxScale) ||
        !attend_shape(B > 0 ? B : 1, num_q_heads, kv->num_heads, kv->head_dim, kv->page_size, max_pages))
        return BD_ERR_SHAPE;
    const bd_scores form = scores ? *scores : bd_scores{};
    if (form.last) return BD_ERR_MODE;
    if (!cap_ok(form.cap)) return BD_ERR_SHAPE;
    if (!aligned(form.slopes, 4) || !aligned(form.first, 4)) return BD_ERR_ALIGN;
    if ((st = check_strides(q_strides, q_type)) != BD_OK) return st;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(page_table, 4) || !aligned(lengths, 4) || !aligned(lse, 4))
        return BD_ERR_ALIGN;
    if (B == 0) return BD_OK;
    const size_t need = bd::attend_workspace_bytes(B, num_q_heads, kv->num_heads, kv->head_dim, kv->page_size,
                                                   max_pages);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return BD_ERR_WORKSPACE;
    if ((st = bd::check_current_device(nullptr)) != BD_OK) return st;
    const bd::AttendArgs a{*kv, q, {q_strides[0], q_strides[1]}, page_table, lengths, out, lse,
                           need > 0 ? static_cast<float*>(workspace) : nullptr, table_stride, (int32_t)max_pages, (int32_t)B,
                           num_q_heads, scale, form.cap, form.slopes, form.first};
    return finish(bd::launch_attend(a, q_type == BD_FP32, static_cast<hipStream_t>(stream)));
}

bd_status bd_attend(const bd_kv* kv, const void* q, int32_t q_type, const int64_t* q_strides,
                    int32_t num_q_heads, const int32_t* page_table, int64_t table_stride, int64_t max_pages,
                    const int32_t* lengths, int64_t B, float scale, uint16_t* out, float* lse,
                    void* workspace, size_t workspace_bytes, void* stream) {
    return bd_attend_scores(kv, q, q_type, q_strides, num_q_heads, page_table, table_stride, max_pages, lengths, B,
                            scale, nullptr, out, lse, workspace, workspace_bytes, stream);
}

size_t bd_attend_prompt_workspace_bytes(int64_t T, int64_t B, int64_t num_q_heads, int64_t num_heads,
                                        int64_t head_dim, int64_t page_size, int64_t max_pages) {
    if (!prompt_shape(T, B, num_q_heads, num_heads, head_dim, page_size, max_pages)) return 0;
    return bd::prompt_workspace_bytes(T, B, num_q_heads, num_heads, head_dim, page_size * max_pages);
}

bd_status bd_attend_prompt(const bd_kv* kv, const uint16_t* q, const int64_t* q_strides, int32_t num_q_heads,
                           int64_t T, const int32_t* page_table, int64_t table_stride, int64_t max_pages,
                           const int32_t* lengths, const int32_t* starts, int64_t B, float scale,
                           const bd_scores* scores, uint16_t* out, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream) {
    bd_status st = check_kv(kv);
    if (st != BD_OK) return st;
    const bool some = B > 0 && T > 0;
    if (!q_strides || (some && (!q || !page_table || !lengths || !starts || !out))) return BD_ERR_NULL;
    const bd_scores form = scores ? *scores : bd_scores{};
    if (B < 0 || T < 0 || table_stride < 0 || !(std::fabs(scale) <= kMaxScale) || !cap_ok(form.cap) ||
        !prompt_shape(T > 0 ? T : 1, B > 0 ? B : 1, num_q_heads, kv->num_heads, kv->head_dim, kv->page_size, max_pages))
        return BD_ERR_SHAPE;
    if ((st = check_strides(q_strides, BD_BF16)) != BD_OK) return st;
    for (const void* x : {static_cast<const void*>(page_table), static_cast<const void*>(lengths),
                          static_cast<const void*>(starts), static_cast<const void*>(lse),
                          static_cast<const void*>(form.slopes), static_cast<const void*>(form.first),
                          static_cast<const void*>(form.last)})
        if (!aligned(x, 4)) return BD_ERR_ALIGN;
    if (!aligned(q, 16) || !aligned(out, 16)) return BD_ERR_ALIGN;
    if (!some) return BD_OK;
    const size_t need = bd::prompt_workspace_bytes(T, B, num_q_heads, kv->num_heads, kv->head_dim,
                                                   kv->page_size * max_pages);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return BD_ERR_WORKSPACE;
    if ((st = bd::check_current_device(nullptr)) != BD_OK) return st;
    const bd::PromptArgs a{*kv, q, {q_strides[0], q_strides[1]}, page_table, lengths, starts, out, lse,
                           need > 0 ? static_cast<float*>(workspace) : nullptr, table_stride, (int32_t)max_pages,
                           (int32_t)B, (int32_t)T, num_q_heads, scale, form.cap, form.slopes, form.first, form.last};
    return finish(bd::launch_prompt(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

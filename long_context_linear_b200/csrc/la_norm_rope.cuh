// C entry points of the query/key norm with rotation (norm_rope.cuh); part of
// la_lib.cu's translation unit.
#pragma once

extern "C++" {
namespace {

constexpr int kNropeBlocksPerSm = 4;  // backward: resident blocks whose partial weight gradients are joined

bool nrope_strides_ok(const la_view* v, size_t esz) {
    const auto ok = [&](int64_t s) { return (s * (int64_t)esz) % 16 == 0; };
    return ok(v->stride_b) && ok(v->stride_h) && ok(v->stride_n);
}

la_status nrope_view(nrope::View* out, const la_view* v, const char* name, size_t esz) {
    if (!v || !v->data) return fail(LA_ERR_INVALID_ARG, "%s must be non-null", name);
    if (!aligned16(v->data) || !nrope_strides_ok(v, esz))
        return fail(LA_ERR_INVALID_ARG, "%s: the pointer and the strides must be multiples of 16 bytes", name);
    out->p = v->data;
    out->sb = v->stride_b;
    out->sh = v->stride_h;
    out->sn = v->stride_n;
    return LA_OK;
}

// Checks shared by both directions; fills everything but the views.
la_status nrope_common(nrope::Params* p, const void* q_weight, const void* k_weight, const float* inv_freq,
                       const void* positions, int pos64, int64_t pos_sb, int64_t pos_sn, int B, int N, int Hq, int Hk,
                       int d, int rot, float eps, la_dtype dt, la_dtype wdt) {
    la_status s = check_dims(d, d, dt);
    if (s != LA_OK) return s;
    if (wdt != LA_FP32 && wdt != dt)
        return fail(LA_ERR_UNSUPPORTED, "weights must be fp32 or of the inputs' type");
    if (B < 0 || N < 0 || Hq < 0 || Hk < 0)
        return fail(LA_ERR_INVALID_ARG, "negative size B=%d N=%d Hq=%d Hk=%d", B, N, Hq, Hk);
    if (rot < 0 || rot > d || rot % 16)
        return fail(LA_ERR_UNSUPPORTED, "rot = %d must be a multiple of 16 in [0, %d]", rot, d);
    if (!(eps >= 0.f) || eps > 1e30f) return fail(LA_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if ((long)Hq + Hk > (1L << 20) || (long)B * N > (1L << 36)) return fail(LA_ERR_INVALID_ARG, "problem too large");
    if ((Hq && !q_weight) || (Hk && !k_weight)) return fail(LA_ERR_INVALID_ARG, "the weights must be non-null");
    if (!aligned16(q_weight) || !aligned16(k_weight)) return fail(LA_ERR_INVALID_ARG, "the weights must be 16-byte aligned");
    if (rot && !inv_freq) return fail(LA_ERR_INVALID_ARG, "inv_freq must be non-null when rot > 0");
    if ((reinterpret_cast<uintptr_t>(inv_freq) & 3u) || (reinterpret_cast<uintptr_t>(positions) & (pos64 ? 7u : 3u)))
        return fail(LA_ERR_INVALID_ARG, "inv_freq or positions is misaligned");
    p->w[0] = q_weight;
    p->w[1] = k_weight;
    p->w32 = wdt == LA_FP32;
    p->Hq = Hq;
    p->HT = Hq + Hk;
    p->N = N;
    p->rows = (long)B * N * (Hq + Hk);
    p->pos = positions;
    p->pos64 = pos64 != 0;
    p->pos_sb = pos_sb;
    p->pos_sn = pos_sn;
    p->inv_freq = inv_freq;
    p->half = rot / 2;
    p->eps = eps;
    return LA_OK;
}

template <typename T, int D>
long nrope_blocks(long rows) {
    return (rows + nrope::block_rows<T, D>() - 1) / nrope::block_rows<T, D>();
}

template <typename T, int D>
void nrope_launch(const nrope::Params& p, bool inter, bool backward, int blocks, cudaStream_t st) {
    const size_t smem = p.half ? (size_t)nrope::block_tokens<T, D>(p.HT) * p.half * sizeof(float2) : 0;
    auto go = [&](auto kern) { kern<<<blocks, nrope::NUM_THREADS, smem, st>>>(p); };
    if (backward) {
        if (inter) go(nrope::norm_rope_backward_kernel<T, D, true>);
        else go(nrope::norm_rope_backward_kernel<T, D, false>);
    } else {
        if (inter) go(nrope::norm_rope_kernel<T, D, true>);
        else go(nrope::norm_rope_kernel<T, D, false>);
    }
}

template <typename F>
auto nrope_by_type(la_dtype dt, int d, F f) {
    if (dt == LA_BF16) return d == 128 ? f((__nv_bfloat16*)nullptr, std::integral_constant<int, 128>())
                                       : f((__nv_bfloat16*)nullptr, std::integral_constant<int, 64>());
    return d == 128 ? f((float*)nullptr, std::integral_constant<int, 128>())
                    : f((float*)nullptr, std::integral_constant<int, 64>());
}

long nrope_total_blocks(la_dtype dt, int d, long rows) {
    return nrope_by_type(dt, d, [&](auto* t, auto D) {
        return nrope_blocks<std::remove_pointer_t<decltype(t)>, decltype(D)::value>(rows);
    });
}

void nrope_go(const nrope::Params& p, la_dtype dt, int d, bool inter, bool backward, int blocks, cudaStream_t st) {
    nrope_by_type(dt, d, [&](auto* t, auto D) {
        nrope_launch<std::remove_pointer_t<decltype(t)>, decltype(D)::value>(p, inter, backward, blocks, st);
        return 0;
    });
}

}  // namespace
}  // extern "C++"

la_status la_qk_norm_rope(const la_view* q, const la_view* k, const la_view* q_out, const la_view* k_out,
                          const void* q_weight, const void* k_weight, const float* inv_freq, const void* positions,
                          int pos64, int64_t pos_stride_b, int64_t pos_stride_n, int B, int N, int Hq, int Hk, int d,
                          int rot, float eps, int interleaved, la_dtype dt, la_dtype wdt, la_stream_t stream) {
    g_last_error[0] = 0;
    nrope::Params p{};
    la_status s = nrope_common(&p, q_weight, k_weight, inv_freq, positions, pos64, pos_stride_b, pos_stride_n, B, N, Hq,
                               Hk, d, rot, eps, dt, wdt);
    if (s != LA_OK) return s;
    if (p.rows == 0) return LA_OK;
    const size_t esz = dt == LA_FP32 ? 4 : 2;
    if (Hq && ((s = nrope_view(&p.x[0], q, "q", esz)) != LA_OK || (s = nrope_view(&p.y[0], q_out, "q_out", esz)) != LA_OK))
        return s;
    if (Hk && ((s = nrope_view(&p.x[1], k, "k", esz)) != LA_OK || (s = nrope_view(&p.y[1], k_out, "k_out", esz)) != LA_OK))
        return s;
    const long blocks = nrope_total_blocks(dt, d, p.rows);
    if (blocks > (1L << 31) - 1) return fail(LA_ERR_INVALID_ARG, "problem too large");
    DeviceInfo* di;
    if ((s = device_info(&di)) != LA_OK) return s;
    nrope_go(p, dt, d, interleaved != 0, false, (int)blocks, reinterpret_cast<cudaStream_t>(stream));
    return after_launch("norm_rope launch");
}

size_t la_qk_norm_rope_backward_workspace_size(int d) {
    DeviceInfo* di;
    const int sms = device_info(&di) == LA_OK ? di->sms : 148;
    return d > 0 ? (size_t)sms * kNropeBlocksPerSm * 2 * d * sizeof(float) : 0;
}

la_status la_qk_norm_rope_backward(const la_view* dq_out, const la_view* dk_out, const la_view* q, const la_view* k,
                                   const void* q_weight, const void* k_weight, const float* inv_freq,
                                   const void* positions, int pos64, int64_t pos_stride_b, int64_t pos_stride_n,
                                   const la_view* dq, const la_view* dk, float* dq_weight, float* dk_weight, int B, int N,
                                   int Hq, int Hk, int d, int rot, float eps, int interleaved, la_dtype dt, la_dtype wdt,
                                   void* workspace, size_t ws_bytes, la_stream_t stream) {
    g_last_error[0] = 0;
    nrope::Params p{};
    la_status s = nrope_common(&p, q_weight, k_weight, inv_freq, positions, pos64, pos_stride_b, pos_stride_n, B, N, Hq,
                               Hk, d, rot, eps, dt, wdt);
    if (s != LA_OK) return s;
    if ((reinterpret_cast<uintptr_t>(dq_weight) & 3u) || (reinterpret_cast<uintptr_t>(dk_weight) & 3u))
        return fail(LA_ERR_INVALID_ARG, "the weight gradients must be 4-byte aligned");
    const size_t esz = dt == LA_FP32 ? 4 : 2;
    if (p.rows) {
        if (Hq && ((s = nrope_view(&p.x[0], q, "q", esz)) != LA_OK ||
                   (s = nrope_view(&p.dy[0], dq_out, "dq_out", esz)) != LA_OK ||
                   (s = nrope_view(&p.y[0], dq, "dq", esz)) != LA_OK))
            return s;
        if (Hk && ((s = nrope_view(&p.x[1], k, "k", esz)) != LA_OK ||
                   (s = nrope_view(&p.dy[1], dk_out, "dk_out", esz)) != LA_OK ||
                   (s = nrope_view(&p.y[1], dk, "dk", esz)) != LA_OK))
            return s;
    }
    const size_t need = la_qk_norm_rope_backward_workspace_size(d);
    if (!workspace || !aligned16(workspace) || ws_bytes < need)
        return fail(LA_ERR_INVALID_ARG, "workspace of %zu bytes (16-byte aligned) required, got %zu", need, ws_bytes);
    DeviceInfo* di;
    if ((s = device_info(&di)) != LA_OK) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int blocks = (int)std::min<long>(nrope_total_blocks(dt, d, p.rows), (long)di->sms * kNropeBlocksPerSm);
    p.partial = reinterpret_cast<float*>(workspace);
    if (blocks) {
        nrope_go(p, dt, d, interleaved != 0, true, blocks, st);
        if ((s = after_launch("norm_rope backward launch")) != LA_OK) return s;
    }
    if (dq_weight || dk_weight) {
        nrope::weight_grad_kernel<<<2 * d / 32, nrope::NUM_THREADS, 0, st>>>(p.partial, blocks, d, dq_weight, dk_weight);
        return after_launch("norm_rope weight gradient launch");
    }
    return LA_OK;
}

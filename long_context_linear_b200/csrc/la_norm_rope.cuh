// C entry points of the query/key norm with rotation (norm_rope.cuh); part of
// la_lib.cu's translation unit.
#pragma once

extern "C++" {
namespace {

constexpr int kNropeBlocksPerSm = 8;  // backward: blocks whose partial weight gradients are joined

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

// An output whose entries share memory would be written by several blocks.
la_status nrope_distinct(const nrope::View& v, const char* name, int B, int H, int N) {
    if ((B > 1 && v.sb == 0) || (H > 1 && v.sh == 0) || (N > 1 && v.sn == 0))
        return fail(LA_ERR_INVALID_ARG, "%s: stride 0 in a dimension of more than one entry", name);
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
    // (B * N * heads itself may pass 64 bits)
    const long heads = (long)Hq + Hk;
    if (Hq > (1 << 20) || Hk > (1 << 20) || N > (1 << 30) || (heads && (long)B * N > (1L << 34) / heads))
        return fail(LA_ERR_INVALID_ARG, "problem too large");
    if ((Hq && !q_weight) || (Hk && !k_weight)) return fail(LA_ERR_INVALID_ARG, "the weights must be non-null");
    if (!aligned16(q_weight) || !aligned16(k_weight)) return fail(LA_ERR_INVALID_ARG, "the weights must be 16-byte aligned");
    if (rot && !inv_freq) return fail(LA_ERR_INVALID_ARG, "inv_freq must be non-null when rot > 0");
    if ((reinterpret_cast<uintptr_t>(inv_freq) & 3u) || (reinterpret_cast<uintptr_t>(positions) & (pos64 ? 7u : 3u)))
        return fail(LA_ERR_INVALID_ARG, "inv_freq or positions is misaligned");
    p->side[0].w = q_weight;
    p->side[1].w = k_weight;
    p->side[0].H = Hq;
    p->side[1].H = Hk;
    for (nrope::Side& sd : p->side) sd.rows = (long)B * N * sd.H;
    p->w32 = wdt == LA_FP32;
    p->N = N;
    p->pos = positions;
    p->pos64 = pos64 != 0;
    p->pos_sb = pos_sb;
    p->pos_sn = pos_sn;
    p->inv_freq = inv_freq;
    p->half = rot / 2;
    p->eps = eps;
    return LA_OK;
}

// Rows per thread: 4 (backward 2), or 1 when that leaves SMs without a block
// (norm + rotation of 64 tokens of 64 + 64 heads of 128: 5.1 us with 4, 3.9 with
// 1), and forward for a side of one head, whose rows are as many tokens with
// angles of their own (4 x 8192 tokens of 64 + 1 heads of 128: 270 us with 1, 281
// with 4; 3 + 3 fp32 heads 56 and 48; backward 603 and 518 with 2).

// Launches a direction; `most`: at most this many blocks (0: one per pass).
// On the way it fixes the number of blocks of either side.
template <typename T, int D>
void nrope_launch(nrope::Params& p, bool inter, bool backward, long most, int sms, cudaStream_t st) {
    const long rows = p.side[0].rows + p.side[1].rows;
    bool few = rows <= (long)sms * nrope::block_rows<T, D, 4>();
    for (const nrope::Side& sd : p.side) few = few || (!backward && sd.rows && sd.H == 1);
    const int per = few ? nrope::block_rows<T, D, 1>() : nrope::block_rows<T, D, 4>() / (backward ? 2 : 1);
    size_t smem = 0;
    long n[2];
    for (int k = 0; k < 2; ++k) {
        n[k] = (p.side[k].rows + per - 1) / per;
        if (n[k] && p.half) smem = std::max(smem, (size_t)nrope::block_tokens(per, p.side[k].H) * p.half * sizeof(float2));
    }
    if (most && n[0] + n[1] > most) {
        // resident blocks shared out by rows, at least one for a side that has any
        const long q = n[0] ? std::max<long>(1, std::min<long>(most - (n[1] > 0), most * n[0] / (n[0] + n[1]))) : 0;
        n[1] = n[1] ? std::min(n[1], most - q) : 0;
        n[0] = std::min(n[0], q);
    }
    p.side[0].blocks = (int)n[0];
    p.side[1].blocks = (int)n[1];
    auto go = [&](auto kern) { kern<<<(unsigned)(n[0] + n[1]), nrope::NUM_THREADS, smem, st>>>(p); };
    if (backward) {
        if (inter) few ? go(nrope::norm_rope_backward_kernel<T, D, true, 1>) : go(nrope::norm_rope_backward_kernel<T, D, true, 2>);
        else few ? go(nrope::norm_rope_backward_kernel<T, D, false, 1>) : go(nrope::norm_rope_backward_kernel<T, D, false, 2>);
    } else {
        if (inter) few ? go(nrope::norm_rope_kernel<T, D, true, 1>) : go(nrope::norm_rope_kernel<T, D, true, 4>);
        else few ? go(nrope::norm_rope_kernel<T, D, false, 1>) : go(nrope::norm_rope_kernel<T, D, false, 4>);
    }
}

void nrope_go(nrope::Params& p, la_dtype dt, int d, bool inter, bool backward, long most, int sms, cudaStream_t st) {
    if (dt == LA_BF16) {
        if (d == 128) nrope_launch<__nv_bfloat16, 128>(p, inter, backward, most, sms, st);
        else nrope_launch<__nv_bfloat16, 64>(p, inter, backward, most, sms, st);
    } else {
        if (d == 128) nrope_launch<float, 128>(p, inter, backward, most, sms, st);
        else nrope_launch<float, 64>(p, inter, backward, most, sms, st);
    }
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
    if (p.side[0].rows + p.side[1].rows == 0) return LA_OK;
    const size_t esz = dt == LA_FP32 ? 4 : 2;
    if (Hq && ((s = nrope_view(&p.side[0].x, q, "q", esz)) != LA_OK || (s = nrope_view(&p.side[0].y, q_out, "q_out", esz)) != LA_OK ||
               (s = nrope_distinct(p.side[0].y, "q_out", B, Hq, N)) != LA_OK))
        return s;
    if (Hk && ((s = nrope_view(&p.side[1].x, k, "k", esz)) != LA_OK || (s = nrope_view(&p.side[1].y, k_out, "k_out", esz)) != LA_OK ||
               (s = nrope_distinct(p.side[1].y, "k_out", B, Hk, N)) != LA_OK))
        return s;
    DeviceInfo* di;
    if ((s = device_info(&di)) != LA_OK) return s;
    nrope_go(p, dt, d, interleaved != 0, false, 0, di->sms, reinterpret_cast<cudaStream_t>(stream));
    return after_launch("norm_rope launch");
}

size_t la_qk_norm_rope_backward_workspace_size(int d) {
    DeviceInfo* di;
    const int sms = device_info(&di) == LA_OK ? di->sms : 148;
    return d > 0 ? (size_t)sms * kNropeBlocksPerSm * d * sizeof(float) : 0;
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
    const bool any = p.side[0].rows + p.side[1].rows > 0;
    if (any) {
        if (Hq && ((s = nrope_view(&p.side[0].x, q, "q", esz)) != LA_OK ||
                   (s = nrope_view(&p.side[0].dy, dq_out, "dq_out", esz)) != LA_OK ||
                   (s = nrope_view(&p.side[0].y, dq, "dq", esz)) != LA_OK ||
                   (s = nrope_distinct(p.side[0].y, "dq", B, Hq, N)) != LA_OK))
            return s;
        if (Hk && ((s = nrope_view(&p.side[1].x, k, "k", esz)) != LA_OK ||
                   (s = nrope_view(&p.side[1].dy, dk_out, "dk_out", esz)) != LA_OK ||
                   (s = nrope_view(&p.side[1].y, dk, "dk", esz)) != LA_OK ||
                   (s = nrope_distinct(p.side[1].y, "dk", B, Hk, N)) != LA_OK))
            return s;
    }
    const size_t need = la_qk_norm_rope_backward_workspace_size(d);
    if (!workspace || !aligned16(workspace) || ws_bytes < need)
        return fail(LA_ERR_INVALID_ARG, "workspace of %zu bytes (16-byte aligned) required, got %zu", need, ws_bytes);
    DeviceInfo* di;
    if ((s = device_info(&di)) != LA_OK) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    p.partial = reinterpret_cast<float*>(workspace);
    if (any) {
        nrope_go(p, dt, d, interleaved != 0, true, (long)di->sms * kNropeBlocksPerSm, di->sms, st);
        if ((s = after_launch("norm_rope backward launch")) != LA_OK) return s;
    }
    if (dq_weight || dk_weight) {
        nrope::weight_grad_kernel<<<dim3(d / 32, 2), nrope::NUM_THREADS, 0, st>>>(p.partial, p.side[0].blocks, p.side[1].blocks,
                                                                               d, dq_weight, dk_weight);
        return after_launch("norm_rope weight gradient launch");
    }
    return LA_OK;
}

// Norm of every query and key head with the rotation by the token's position,
// in one pass over q and k (and its gradients).
//
//   r = (mean_i x_i^2 + eps)^(-1/2),  xh = r x,  y = R(p) (w * xh)
//
// where R(p) turns the pair (a, b) of frequency i by the angle p f_i:
// (a cos - b sin, b cos + a sin).  Pairs are (i, i + rot/2), or (2i, 2i + 1)
// when interleaved; dims from rot on are not turned.  Backward, with
// g = R(-p) dy:
//   dx = r (w g - xh mean(w g xh)),   dw = sum over tokens and heads of g xh.
//
// Bound by the bytes of q and k: a row (one head of one token, d values) is
// held by LPR = d sizeof(T) / 16 lanes with one 16-byte vector each; statistics
// are fp32 sums over those lanes, the partner of a pair sits in another lane
// of the row (or in the same vector when interleaved).  A block of 256 threads
// takes ROWS consecutive rows in (token, head) order, every thread's loads
// issued before any use, and forms the cosines and sines of its tokens once in
// shared memory meanwhile.
//
// Angles: p f is formed in double, in turns, and reduced to [-1/2, 1/2] before
// it is rounded to fp32 for sincospi: a position of 2^20 is 10^5 radians, where
// an fp32 product is 0.01 rad off.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace lcl {
namespace nrope {

constexpr int NUM_THREADS = 256;
constexpr int UNROLL = 4;  // rows per thread and pass

struct View {
    const void* p;
    long sb, sh, sn;  // strides in elements
};

struct Params {
    View x[2];        // q, k
    View dy[2];       // backward: gradients of the outputs
    View y[2];        // outputs (backward: gradients of q, k)
    const void* w[2];
    int w32;          // weights are fp32 (else the element type)
    int Hq, HT;       // query heads, query + key heads
    long N;           // tokens per batch entry
    long rows;        // B * N * HT
    const void* pos;  // int32 or int64, or null (token index n)
    int pos64;
    long pos_sb, pos_sn;
    const float* inv_freq;
    int half;         // rot / 2
    float eps;
    float* partial;   // backward: [gridDim.x][2][d]
};

template <typename T> struct Elem;
template <> struct Elem<float> {
    static constexpr int VEC = 4;
    __device__ __forceinline__ static void unpack(const uint4& r, float (&f)[4]) {
        f[0] = __uint_as_float(r.x); f[1] = __uint_as_float(r.y); f[2] = __uint_as_float(r.z); f[3] = __uint_as_float(r.w);
    }
    __device__ __forceinline__ static uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <> struct Elem<__nv_bfloat16> {
    static constexpr int VEC = 8;
    __device__ __forceinline__ static void unpack(const uint4& r, float (&f)[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ static uint4 pack(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <typename T, int D> constexpr int lanes_per_row() { return D / Elem<T>::VEC; }
// rows per block and pass
template <typename T, int D> constexpr int block_rows() { return NUM_THREADS / lanes_per_row<T, D>() * UNROLL; }
// most tokens that a block's rows belong to
template <typename T, int D> int block_tokens(int HT) { return (block_rows<T, D>() + HT - 2) / HT + 1; }

__device__ __forceinline__ float row_sum(float s, int lpr) {
    for (int o = lpr >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// cos and sin of position * inv_freq for `tokens` tokens from token tok0 on
__device__ __forceinline__ void fill_angles(const Params& p, long tok0, int tokens, long all_tokens, float2* cs) {
    constexpr double INV_2PI = 0.15915494309189533576888;
    for (int e = threadIdx.x; e < tokens * p.half; e += NUM_THREADS) {
        const int tt = e / p.half, i = e - tt * p.half;
        const long tok = tok0 + tt;
        if (tok >= all_tokens) break;
        const long b = tok / p.N, n = tok - b * p.N;
        double pos;
        if (!p.pos) pos = static_cast<double>(n);
        else if (p.pos64) pos = static_cast<double>(reinterpret_cast<const long long*>(p.pos)[b * p.pos_sb + n * p.pos_sn]);
        else pos = static_cast<double>(reinterpret_cast<const int*>(p.pos)[b * p.pos_sb + n * p.pos_sn]);
        const double turns = pos * (static_cast<double>(p.inv_freq[i]) * INV_2PI);
        float s, c;
        sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
        cs[e] = make_float2(c, s);
    }
}

// The row's vector turned by its token's angles (sgn = 1) or back (sgn = -1);
// every lane of the warp takes part.
template <int VEC, int LPR, bool kInter>
__device__ __forceinline__ void rotate(float (&f)[VEC], const float2* cs, int lane, int half, float sgn) {
    if constexpr (kInter) {
        if (lane * VEC < 2 * half) {
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                const float2 t = cs[lane * (VEC / 2) + i];
                const float a = f[2 * i], b = f[2 * i + 1], s = sgn * t.y;
                f[2 * i] = a * t.x - b * s;
                f[2 * i + 1] = b * t.x + a * s;
            }
        }
    } else {
        const int hl = half / VEC;
        const bool first = lane < hl, turned = lane < 2 * hl;
        const int partner = !turned ? lane : (first ? lane + hl : lane - hl);
        const float2* t = cs + (first ? lane : lane - hl) * VEC;
        const float ss = first ? -sgn : sgn;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float other = __shfl_sync(0xffffffffu, f[i], partner, LPR);
            if (turned) f[i] = f[i] * t[i].x + other * (ss * t[i].y);
        }
    }
}

template <int VEC, typename T>
__device__ __forceinline__ void load_weight(const Params& p, int side, int lane, float (&w)[VEC]) {
    if (p.w32) {
        const float4* src = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.w[side]) + lane * VEC);
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const float4 x = __ldg(src + i);
            w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
        }
    } else {
        Elem<T>::unpack(__ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(p.w[side]) + lane * VEC)), w);
    }
}

template <typename T, int D, bool kInter>
__global__ void __launch_bounds__(NUM_THREADS)
norm_rope_kernel(const __grid_constant__ Params p) {
    constexpr int VEC = Elem<T>::VEC, LPR = lanes_per_row<T, D>(), RB = NUM_THREADS / LPR, ROWS = RB * UNROLL;
    extern __shared__ float2 cs[];
    const int lane = threadIdx.x % LPR, slot = threadIdx.x / LPR;
    const long row0 = static_cast<long>(blockIdx.x) * ROWS;
    const long tok0 = row0 / p.HT;
    uint4 r[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const long row = row0 + slot + u * RB;
        r[u] = make_uint4(0u, 0u, 0u, 0u);
        if (row < p.rows) {
            const long tok = row / p.HT;
            const int h = static_cast<int>(row - tok * p.HT), side = h >= p.Hq, hs = side ? h - p.Hq : h;
            const long b = tok / p.N, n = tok - b * p.N;
            const View& x = p.x[side];
            r[u] = __ldcs(reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(x.p) + b * x.sb + hs * x.sh + n * x.sn +
                                                         lane * VEC));
        }
    }
    if (p.half) {
        const long last = min(row0 + ROWS, p.rows) - 1;
        fill_angles(p, tok0, static_cast<int>(last / p.HT - tok0) + 1, p.rows / p.HT, cs);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const long row = row0 + slot + u * RB;
        const bool live = row < p.rows;
        const long tok = (live ? row : row0) / p.HT;
        const int h = live ? static_cast<int>(row - tok * p.HT) : 0, side = h >= p.Hq, hs = side ? h - p.Hq : h;
        float f[VEC], w[VEC];
        Elem<T>::unpack(r[u], f);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) ss = fmaf(f[i], f[i], ss);
        const float rs = rsqrtf(row_sum(ss, LPR) * (1.f / D) + p.eps);
        load_weight<VEC, T>(p, side, lane, w);
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = f[i] * rs * w[i];
        if (p.half) rotate<VEC, LPR, kInter>(f, cs + (tok - tok0) * p.half, lane, p.half, 1.f);
        if (live) {
            const long b = tok / p.N, n = tok - b * p.N;
            const View& y = p.y[side];
            T* dst = reinterpret_cast<T*>(const_cast<void*>(y.p)) + b * y.sb + hs * y.sh + n * y.sn + lane * VEC;
            *reinterpret_cast<uint4*>(dst) = Elem<T>::pack(f);
        }
    }
}

// Gradients of q and k, and per block the sums of g xh over its rows (fixed
// order: a block's rows depend on the grid alone).
template <typename T, int D, bool kInter>
__global__ void __launch_bounds__(NUM_THREADS)
norm_rope_backward_kernel(const __grid_constant__ Params p) {
    constexpr int VEC = Elem<T>::VEC, LPR = lanes_per_row<T, D>(), RB = NUM_THREADS / LPR, ROWS = RB * UNROLL;
    extern __shared__ float2 cs[];
    __shared__ float red[2][RB][D];
    const int lane = threadIdx.x % LPR, slot = threadIdx.x / LPR;
    float dw[2][VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) dw[0][i] = dw[1][i] = 0.f;
    for (long row0 = static_cast<long>(blockIdx.x) * ROWS; row0 < p.rows; row0 += static_cast<long>(gridDim.x) * ROWS) {
        const long tok0 = row0 / p.HT;
        uint4 rx[UNROLL], rd[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const long row = row0 + slot + u * RB;
            rx[u] = rd[u] = make_uint4(0u, 0u, 0u, 0u);
            if (row < p.rows) {
                const long tok = row / p.HT;
                const int h = static_cast<int>(row - tok * p.HT), side = h >= p.Hq, hs = side ? h - p.Hq : h;
                const long b = tok / p.N, n = tok - b * p.N;
                const View &x = p.x[side], &d = p.dy[side];
                rx[u] = __ldcs(reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(x.p) + b * x.sb + hs * x.sh +
                                                              n * x.sn + lane * VEC));
                rd[u] = __ldcs(reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(d.p) + b * d.sb + hs * d.sh +
                                                              n * d.sn + lane * VEC));
            }
        }
        __syncthreads();  // the angles of the previous pass have been read
        if (p.half) {
            const long last = min(row0 + ROWS, p.rows) - 1;
            fill_angles(p, tok0, static_cast<int>(last / p.HT - tok0) + 1, p.rows / p.HT, cs);
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const long row = row0 + slot + u * RB;
            const bool live = row < p.rows;
            const long tok = (live ? row : row0) / p.HT;
            const int h = live ? static_cast<int>(row - tok * p.HT) : 0, side = h >= p.Hq, hs = side ? h - p.Hq : h;
            float f[VEC], g[VEC], w[VEC];
            Elem<T>::unpack(rx[u], f);
            Elem<T>::unpack(rd[u], g);
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < VEC; ++i) ss = fmaf(f[i], f[i], ss);
            const float rs = rsqrtf(row_sum(ss, LPR) * (1.f / D) + p.eps);
            if (p.half) rotate<VEC, LPR, kInter>(g, cs + (tok - tok0) * p.half, lane, p.half, -1.f);
            load_weight<VEC, T>(p, side, lane, w);
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                f[i] *= rs;  // xh
                const float gx = live ? g[i] * f[i] : 0.f;
                if (side) dw[1][i] += gx;
                else dw[0][i] += gx;
                w[i] *= g[i];
                dot = fmaf(w[i], f[i], dot);
            }
            dot = row_sum(dot, LPR) * (1.f / D);
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[i] = rs * (w[i] - f[i] * dot);
            if (live) {
                const long b = tok / p.N, n = tok - b * p.N;
                const View& y = p.y[side];
                T* dst = reinterpret_cast<T*>(const_cast<void*>(y.p)) + b * y.sb + hs * y.sh + n * y.sn + lane * VEC;
                *reinterpret_cast<uint4*>(dst) = Elem<T>::pack(f);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        red[0][slot][lane * VEC + i] = dw[0][i];
        red[1][slot][lane * VEC + i] = dw[1][i];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * D; e += NUM_THREADS) {
        const int side = e / D, i = e - side * D;
        float s = 0.f;
        for (int r = 0; r < RB; ++r) s += red[side][r][i];
        p.partial[static_cast<long>(blockIdx.x) * 2 * D + e] = s;
    }
}

// dw = sum of the blocks' partial sums, [blocks][2][d] -> dq_weight, dk_weight:
// 32 columns per block, 8 warps over the partial rows, joined in a fixed order.
__global__ void __launch_bounds__(NUM_THREADS)
weight_grad_kernel(const float* __restrict__ partial, int blocks, int d, float* __restrict__ dwq, float* __restrict__ dwk) {
    __shared__ float red[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    float s = 0.f;
    for (int b = warp; b < blocks; b += 8) s += partial[static_cast<long>(b) * 2 * d + col];
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0) {
        for (int w = 1; w < 8; ++w) s += red[w][lane];
        float* dst = col < d ? dwq : dwk;
        if (dst) dst[col < d ? col : col - d] = s;
    }
}

}  // namespace nrope
}  // namespace lcl

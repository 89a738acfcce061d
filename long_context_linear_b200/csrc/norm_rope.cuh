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
// Bound by the bytes of q and k.  A row (one head of one token, d values) is
// held by d / (2 VEC) lanes with two 16-byte vectors each; with pairs (i, i +
// rot/2) a lane's two vectors are the two halves of its pairs, so that the
// rotation needs no exchange between lanes.  A block takes consecutive rows of q
// or of k in (token, head) order, every thread's loads issued before any use,
// and forms the cosines and sines of its tokens once in shared memory meanwhile;
// its weights stay in registers.
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

constexpr int NUM_THREADS = 128;  // (256: 211 instead of 199 us forward, 356 instead of 349 backward at the size below)

struct View {
    const void* p;
    long sb, sh, sn;  // strides in elements
};

struct Side {         // q or k
    View x;
    View dy;          // backward: gradient of the output
    View y;           // output (backward: gradient of x)
    const void* w;
    long rows;        // B * N * H
    int H;
    int blocks;
};

struct Params {
    Side side[2];     // blocks of q first
    int w32;          // weights are fp32 (else the element type)
    int N;            // tokens per batch entry
    const void* pos;  // int32 or int64, or null (token index n)
    int pos64;
    long pos_sb, pos_sn;
    const float* inv_freq;
    int half;         // rot / 2
    float eps;
    float* partial;   // backward: [blocks][d]
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

template <typename T, int D> constexpr int lanes_per_row() { return D / Elem<T>::VEC / 2; }
// rows per block and pass, U of them per thread
template <typename T, int D, int U> constexpr int block_rows() { return NUM_THREADS / lanes_per_row<T, D>() * U; }
// most tokens that `rows` consecutive rows of H heads belong to
inline int block_tokens(int rows, int H) { return (rows + H - 2) / H + 1; }

// A block's rows in (token, head) order, from one division by H per block:
// everything per row is 32-bit.  (With 64-bit divisions per row the first
// version spent most of its instructions on them.)
struct Rows {
    long b0;     // batch entry of the first row
    int n0, h0;  // its token within the entry, its head
};
__device__ __forceinline__ Rows first_row(int N, int H, long row0) {
    Rows r;
    if (row0 < (1l << 31)) {
        const unsigned row = static_cast<unsigned>(row0), tok = row / static_cast<unsigned>(H);
        r.h0 = static_cast<int>(row - tok * H);
        const unsigned b = tok / static_cast<unsigned>(N);
        r.n0 = static_cast<int>(tok - b * N);
        r.b0 = b;
    } else {
        const long tok = row0 / H;
        r.h0 = static_cast<int>(row0 - tok * H);
        r.b0 = tok / N;
        r.n0 = static_cast<int>(tok - r.b0 * N);
    }
    return r;
}
// Token tt after the block's first one: batch entry and token within it.
__device__ __forceinline__ void token_at(const Rows& r, int N, int tt, long& b, int& n) {
    const unsigned nn = static_cast<unsigned>(r.n0 + tt);
    const unsigned over = nn < static_cast<unsigned>(N) ? 0u : nn / static_cast<unsigned>(N);
    b = r.b0 + over;
    n = static_cast<int>(nn - over * N);
}
// Row i of the block: its token's distance from the first one, and where it is.
struct At {
    int tt, h, n;
    long b;
    __device__ __forceinline__ long in(const View& v) const { return b * v.sb + h * v.sh + n * v.sn; }
};
__device__ __forceinline__ At row_at(const Rows& r, int N, int H, int i) {
    At a;
    const unsigned h = static_cast<unsigned>(r.h0 + i);
    a.tt = h < static_cast<unsigned>(H) ? 0 : static_cast<int>(h / static_cast<unsigned>(H));
    a.h = static_cast<int>(h) - a.tt * H;
    token_at(r, N, a.tt, a.b, a.n);
    return a;
}

__device__ __forceinline__ float row_sum(float s, int lpr) {
    for (int o = lpr >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// cos and sin of position * inv_freq for the tokens of the block's `rows` rows.
// A lane reads the F frequencies of its vector as F / 2 float4s; the i-th float4
// of every vector lie side by side, so that lanes read neighbouring ones
// (frequency by frequency their stride was F x 8 bytes: four-way bank conflicts,
// 16 % of the pass).
template <int F>
__device__ __forceinline__ void fill_angles(const Params& p, const Rows& r, int H, int rows, float2* cs) {
    constexpr double INV_2PI = 0.15915494309189533576888;
    const int tokens = (r.h0 + rows - 1) / H + 1;
    for (int e = threadIdx.x; e < tokens * p.half; e += NUM_THREADS) {
        const int tt = e / p.half, i = e - tt * p.half;
        long b;
        int n;
        token_at(r, p.N, tt, b, n);
        double pos;
        if (!p.pos) pos = static_cast<double>(n);
        else if (p.pos64) pos = static_cast<double>(reinterpret_cast<const long long*>(p.pos)[b * p.pos_sb + n * p.pos_sn]);
        else pos = static_cast<double>(reinterpret_cast<const int*>(p.pos)[b * p.pos_sb + n * p.pos_sn]);
        const double turns = pos * (static_cast<double>(p.inv_freq[i]) * INV_2PI);
        float s, c;
        sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
        cs[tt * p.half + ((i % F) / 2 * (p.half / F) + i / F) * 2 + (i & 1)] = make_float2(c, s);
    }
}

// The two vectors (indices in units of VEC values) of lane l of a row.  With
// pairs (i, i + half): lane l < half / VEC holds the l-th vector of either half,
// the others the vectors behind them, which are not turned.  Interleaved: l
// and l + LPR (a row's 16-byte loads then cover whole 128-byte lines).
template <int VEC, int LPR, bool kInter>
__device__ __forceinline__ void lane_vectors(int l, int half, int (&vec)[2]) {
    if constexpr (kInter) {
        vec[0] = l;
        vec[1] = l + LPR;
    } else {
        const int hl = half / VEC;
        vec[0] = l < hl ? l : 2 * l;
        vec[1] = l < hl ? l + hl : 2 * l + 1;
    }
}

// A lane's 2 VEC values turned by their token's angles (sgn = 1) or back (-1).
template <int VEC, int LPR, bool kInter>
__device__ __forceinline__ void rotate(float (&f)[2][VEC], const float2* cs, int l, int half, float sgn) {
    if constexpr (kInter) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const int e0 = (l + v * LPR) * VEC;
            if (e0 < 2 * half) {
                const float4* t = reinterpret_cast<const float4*>(cs) + l + v * LPR;
#pragma unroll
                for (int i = 0; i < VEC / 4; ++i) {
                    const float4 x = t[i * (2 * half / VEC)];  // cos, sin of two pairs
                    float a = f[v][4 * i], b = f[v][4 * i + 1];
                    f[v][4 * i] = a * x.x - b * (sgn * x.y);
                    f[v][4 * i + 1] = b * x.x + a * (sgn * x.y);
                    a = f[v][4 * i + 2], b = f[v][4 * i + 3];
                    f[v][4 * i + 2] = a * x.z - b * (sgn * x.w);
                    f[v][4 * i + 3] = b * x.z + a * (sgn * x.w);
                }
            }
        }
    } else if (l * VEC < half) {
        const float4* t = reinterpret_cast<const float4*>(cs) + l;
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const float4 x = t[i * (half / VEC)];
            float a = f[0][2 * i], b = f[1][2 * i];
            f[0][2 * i] = a * x.x - b * (sgn * x.y);
            f[1][2 * i] = b * x.x + a * (sgn * x.y);
            a = f[0][2 * i + 1], b = f[1][2 * i + 1];
            f[0][2 * i + 1] = a * x.z - b * (sgn * x.w);
            f[1][2 * i + 1] = b * x.z + a * (sgn * x.w);
        }
    }
}

template <typename T>
__device__ __forceinline__ void load_weight(const Params& p, const void* weight, int vec, float (&w)[Elem<T>::VEC]) {
    constexpr int VEC = Elem<T>::VEC;
    if (p.w32) {
        const float4* src = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(weight) + vec * VEC);
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const float4 x = __ldg(src + i);
            w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
        }
    } else {
        Elem<T>::unpack(__ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(weight) + vec * VEC)), w);
    }
}

// U rows per thread: 4 for many rows (bytes in flight), 1 for few.  4 x 8192
// tokens of 32 + 32 bf16 heads of 128, from the projection's layout to the
// attention's, all dims turned: 0.199 ms, 5.4 TB/s = 0.83 of a copy, for calls in
// a row (norm alone 0.188; 2 rows per thread 0.208); 0.213 to 0.219 ms between
// other work.
template <typename T, int D, bool kInter, int U>
__global__ void __launch_bounds__(NUM_THREADS, 6)
norm_rope_kernel(const __grid_constant__ Params p) {
    constexpr int VEC = Elem<T>::VEC, LPR = lanes_per_row<T, D>(), RB = NUM_THREADS / LPR, ROWS = RB * U;
    extern __shared__ float4 cs4[];
    float2* cs = reinterpret_cast<float2*>(cs4);
    const bool second = static_cast<int>(blockIdx.x) >= p.side[0].blocks;
    const Side& sd = p.side[second];
    const int lane = threadIdx.x % LPR, slot = threadIdx.x / LPR;
    const long row0 = static_cast<long>(blockIdx.x - (second ? p.side[0].blocks : 0)) * ROWS;
    const int rows = static_cast<int>(min(static_cast<long>(ROWS), sd.rows - row0));
    const Rows first = first_row(p.N, sd.H, row0);
    int vec[2];
    lane_vectors<VEC, LPR, kInter>(lane, p.half, vec);
    uint4 r[U][2];
    long out[U];
    int tt[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = slot + u * RB;
        const At at = row_at(first, p.N, sd.H, i < rows ? i : 0);
        const T* src = reinterpret_cast<const T*>(sd.x.p) + at.in(sd.x);
        out[u] = at.in(sd.y);
        tt[u] = at.tt;
#pragma unroll
        for (int v = 0; v < 2; ++v)
            r[u][v] = i < rows ? __ldcs(reinterpret_cast<const uint4*>(src + vec[v] * VEC)) : make_uint4(0u, 0u, 0u, 0u);
    }
    if (p.half) fill_angles<kInter ? VEC / 2 : VEC>(p, first, sd.H, rows, cs);
    float w[2][VEC];
#pragma unroll
    for (int v = 0; v < 2; ++v) load_weight<T>(p, sd.w, vec[v], w[v]);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float f[2][VEC];
        float ss = 0.f;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            Elem<T>::unpack(r[u][v], f[v]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) ss = fmaf(f[v][i], f[v][i], ss);
        }
        const float rs = rsqrtf(row_sum(ss, LPR) * (1.f / D) + p.eps);
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[v][i] = f[v][i] * rs * w[v][i];
        rotate<VEC, LPR, kInter>(f, cs + tt[u] * p.half, lane, p.half, 1.f);
        if (slot + u * RB < rows) {
            T* dst = reinterpret_cast<T*>(const_cast<void*>(sd.y.p)) + out[u];
#pragma unroll
            for (int v = 0; v < 2; ++v) *reinterpret_cast<uint4*>(dst + vec[v] * VEC) = Elem<T>::pack(f[v]);
        }
    }
}

// Gradients of q or k, and per block the sums of g xh over its rows (fixed
// order: a block's rows depend on the grid alone).  The same size, with the join
// of the sums below: 0.349 ms in a row, 4.6 TB/s = 0.70 of a copy (2 x 4096 tokens,
// half turned: 0.105 ms, 0.58): 32 accumulators and weights leave 128 registers and
// 16 warps per SM, whose loads and arithmetic overlap across blocks only
// (1 row per thread 0.44, fewer blocks per SM 0.39).
template <typename T, int D, bool kInter, int U>
__global__ void __launch_bounds__(NUM_THREADS, 4)
norm_rope_backward_kernel(const __grid_constant__ Params p) {
    constexpr int VEC = Elem<T>::VEC, LPR = lanes_per_row<T, D>(), RB = NUM_THREADS / LPR, ROWS = RB * U;
    constexpr int WARPS = NUM_THREADS / 32;
    extern __shared__ float4 cs4[];
    float2* cs = reinterpret_cast<float2*>(cs4);
    __shared__ float red[WARPS][D];
    const bool second = static_cast<int>(blockIdx.x) >= p.side[0].blocks;
    const Side& sd = p.side[second];
    const int lane = threadIdx.x % LPR, slot = threadIdx.x / LPR;
    int vec[2];
    lane_vectors<VEC, LPR, kInter>(lane, p.half, vec);
    float w[2][VEC], dw[2][VEC];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        load_weight<T>(p, sd.w, vec[v], w[v]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) dw[v][i] = 0.f;
    }
    for (long row0 = static_cast<long>(blockIdx.x - (second ? p.side[0].blocks : 0)) * ROWS; row0 < sd.rows;
         row0 += static_cast<long>(sd.blocks) * ROWS) {
        const int rows = static_cast<int>(min(static_cast<long>(ROWS), sd.rows - row0));
        const Rows first = first_row(p.N, sd.H, row0);
        uint4 rx[U][2], rd[U][2];
        long out[U];
        int tt[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = slot + u * RB;
            const At at = row_at(first, p.N, sd.H, i < rows ? i : 0);
            const T* x = reinterpret_cast<const T*>(sd.x.p) + at.in(sd.x);
            const T* d = reinterpret_cast<const T*>(sd.dy.p) + at.in(sd.dy);
            out[u] = at.in(sd.y);
            tt[u] = at.tt;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                rx[u][v] = i < rows ? __ldcs(reinterpret_cast<const uint4*>(x + vec[v] * VEC)) : make_uint4(0u, 0u, 0u, 0u);
                rd[u][v] = i < rows ? __ldcs(reinterpret_cast<const uint4*>(d + vec[v] * VEC)) : make_uint4(0u, 0u, 0u, 0u);
            }
        }
        __syncthreads();  // the angles of the pass before have been read
        if (p.half) fill_angles<kInter ? VEC / 2 : VEC>(p, first, sd.H, rows, cs);
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool live = slot + u * RB < rows;
            float f[2][VEC], g[2][VEC];
            float ss = 0.f;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                Elem<T>::unpack(rx[u][v], f[v]);
                Elem<T>::unpack(rd[u][v], g[v]);
#pragma unroll
                for (int i = 0; i < VEC; ++i) ss = fmaf(f[v][i], f[v][i], ss);
            }
            const float rs = rsqrtf(row_sum(ss, LPR) * (1.f / D) + p.eps);
            rotate<VEC, LPR, kInter>(g, cs + tt[u] * p.half, lane, p.half, -1.f);
            float dot = 0.f;
#pragma unroll
            for (int v = 0; v < 2; ++v)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    f[v][i] *= rs;  // xh
                    if (live) dw[v][i] = fmaf(g[v][i], f[v][i], dw[v][i]);
                    g[v][i] *= w[v][i];
                    dot = fmaf(g[v][i], f[v][i], dot);
                }
            dot = row_sum(dot, LPR) * (1.f / D);
            if (live) {
                T* dst = reinterpret_cast<T*>(const_cast<void*>(sd.y.p)) + out[u];
#pragma unroll
                for (int v = 0; v < 2; ++v) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) f[v][i] = rs * (g[v][i] - f[v][i] * dot);
                    *reinterpret_cast<uint4*>(dst + vec[v] * VEC) = Elem<T>::pack(f[v]);
                }
            }
        }
    }
    // the rows of a warp, then of the block
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            float s = dw[v][i];
            for (int o = LPR; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (threadIdx.x % 32 < LPR) red[threadIdx.x / 32][vec[v] * VEC + i] = s;
        }
    __syncthreads();
    for (int e = threadIdx.x; e < D; e += NUM_THREADS) {
        float s = 0.f;
        for (int k = 0; k < WARPS; ++k) s += red[k][e];
        p.partial[static_cast<long>(blockIdx.x) * D + e] = s;
    }
}

// dw = sum of the blocks' partial sums [blocks_q + blocks_k][d]: block (x, side)
// takes 32 columns, 4 warps over the partial rows, joined in a fixed order.  With
// the full grid of partial rows (1184) 29 us of a profiled (cold) call of 2 x 4096
// tokens, beside 84 of the first kernel: d / 32 x 2 blocks on an empty GPU, each
// warp's 148 loads one after another.
__global__ void __launch_bounds__(NUM_THREADS)
weight_grad_kernel(const float* __restrict__ partial, int blocks_q, int blocks_k, int d, float* __restrict__ dwq,
                   float* __restrict__ dwk) {
    __shared__ float red[4][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    const int b0 = blockIdx.y ? blocks_q : 0, b1 = blockIdx.y ? blocks_q + blocks_k : blocks_q;
    float* dst = blockIdx.y ? dwk : dwq;
    float s = 0.f;
    for (int b = b0 + warp; b < b1; b += 4) s += partial[static_cast<long>(b) * d + col];
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && dst) {
        for (int k = 1; k < 4; ++k) s += red[k][lane];
        dst[col] = s;
    }
}

}  // namespace nrope
}  // namespace lcl

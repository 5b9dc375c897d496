// dense.cuh -- dense attention: differential attention with its gradients, and
// attention over a shared prefix.
#pragma once
#include "common.cuh"

namespace sla {

// Row-major tensor [batch, head, token, d]: element strides (0 where a dimension
// is broadcast or has one entry).
struct DenseT {
    long long b, h, n;
    __host__ __device__ __forceinline__ long long at(long long ib, long long ih, long long in) const {
        return ib * b + ih * h + in * n;
    }
};

struct DenseArgs {
    const void *q, *k, *v, *kp, *vp, *dout;
    void *out, *out2, *dq, *dk, *dv, *dlam;
    float* lse;
    const void* lam;
    const int32_t *q_len, *kv_len;
    DenseT qs, ks, vs, kps, vps, os, dos, dqs, dks, dvs;
    int B, H, Hk, G, Nq, Nk, P;
    int causal;
    float scale;                  // tau
    float scale_log2;             // tau * log2(e)
    float* delta;                 // backward: [2][B * H * Nq]
};

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f<__half>(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }

// A sequence's length: within [0, most], out-of-range values flagged.
__device__ __forceinline__ int dense_len(const int32_t* len, int b, int most) {
    if (!len) return most;
    const int n = len[b];
    if (n < 0 || n > most) {
        report(kStatusBadData);
        return n < 0 ? 0 : most;
    }
    return n;
}

// ------------------------------------------------------------------ one warp a row
// Forward: lane = key for the logits, lane = D/32 columns for the products.
template <int D, typename T, bool DIFF>
__global__ void __launch_bounds__(128) dense_fwd_rows_kernel(const DenseArgs a) {
    constexpr int C = D / 32, M = DIFF ? 2 : 1, E = D / M;
    __shared__ float qs[4][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * 4 + warp;
    if (row >= static_cast<long long>(a.B) * a.H * a.Nq) return;
    const int i = row % a.Nq, h = row / a.Nq % a.H, b = row / a.Nq / a.H, hk = h / a.G;
    const int qn = dense_len(a.q_len, b, a.Nq), kn = dense_len(a.kv_len, b, a.Nk);
    float m[M], l[M], acc[M][C];
    for (int x = 0; x < M; ++x) {
        m[x] = -INFINITY;
        l[x] = 0.f;
        for (int c = 0; c < C; ++c) acc[x][c] = 0.f;
    }
    if (i < qn) {
        for (int c = lane; c < D; c += 32)
            qs[warp][c] = to_f<T>(static_cast<const T*>(a.q)[a.qs.at(b, h, i) + c]);
        __syncwarp();
        const int own = a.causal ? min(kn, max(0, i + kn - qn + 1)) : kn;
        for (int part = 0; part < 2; ++part) {
            const int n = part ? own : a.P;
            const T* kb = static_cast<const T*>(part ? a.k : a.kp) + (part ? a.ks.at(b, hk, 0) : a.kps.at(0, hk, 0));
            const T* vb = static_cast<const T*>(part ? a.v : a.vp) + (part ? a.vs.at(b, hk, 0) : a.vps.at(0, hk, 0));
            const long long kst = part ? a.ks.n : a.kps.n, vst = part ? a.vs.n : a.vps.n;
            for (int j0 = 0; j0 < n; j0 += 32) {
                const int j = j0 + lane;
                float s[M], p[M];
                for (int x = 0; x < M; ++x) {
                    s[x] = -INFINITY;
                    if (j < n) {
                        s[x] = 0.f;
                        for (int c = 0; c < E; ++c)
                            s[x] = fmaf(qs[warp][x * E + c], to_f<T>(kb[j * kst + x * E + c]), s[x]);
                        s[x] *= a.scale_log2;
                    }
                    float mx = s[x];
                    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
                    mx = fmaxf(mx, m[x]);
                    const float r = exp2f(m[x] - mx);
                    p[x] = exp2f(s[x] - mx);
                    m[x] = mx;
                    float sum = p[x];
                    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
                    l[x] = l[x] * r + sum;
                    for (int c = 0; c < C; ++c) acc[x][c] *= r;
                }
                for (int t = 0; t < min(32, n - j0); ++t)
                    for (int c = 0; c < C; ++c) {
                        const float vv = to_f<T>(vb[(j0 + t) * vst + lane + 32 * c]);
                        for (int x = 0; x < M; ++x)
                            acc[x][c] = fmaf(__shfl_sync(~0u, p[x], t), vv, acc[x][c]);
                    }
            }
        }
    }
    const float lam = DIFF ? to_f<T>(static_cast<const T*>(a.lam)[h]) : 0.f;
    for (int x = 0; x < M; ++x) {
        const float inv = l[x] > 0.f ? 1.f / l[x] : 0.f;
        for (int c = 0; c < C; ++c) acc[x][c] *= inv;
        if (a.lse && lane == 0)
            a.lse[((static_cast<long long>(b) * a.H + h) * M + x) * a.Nq + i] =
                l[x] > 0.f ? (m[x] + log2f(l[x])) * 0.6931471805599453f : -INFINITY;
    }
    for (int c = 0; c < C; ++c) {
        static_cast<T*>(a.out)[a.os.at(b, h, i) + lane + 32 * c] =
            from_f<T>(DIFF ? acc[0][c] - lam * acc[M - 1][c] : acc[0][c]);
        if (DIFF && a.out2) static_cast<T*>(a.out2)[row * D + lane + 32 * c] = from_f<T>(acc[M - 1][c]);
    }
}

// delta_1 = dout . (out + lambda out2), delta_2 = dout . out2, one warp a row.
template <int D, typename T>
__global__ void __launch_bounds__(128) dense_delta_kernel(const DenseArgs a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long rows = static_cast<long long>(a.B) * a.H * a.Nq;
    const long long row = static_cast<long long>(blockIdx.x) * 4 + warp;
    if (row >= rows) return;
    const int i = row % a.Nq, h = row / a.Nq % a.H, b = row / a.Nq / a.H;
    float d1 = 0.f, d2 = 0.f;
    if (i < dense_len(a.q_len, b, a.Nq)) {
        const float lam = to_f<T>(static_cast<const T*>(a.lam)[h]);
        for (int c = lane; c < D; c += 32) {
            const float g = to_f<T>(static_cast<const T*>(a.dout)[a.dos.at(b, h, i) + c]);
            const float o = to_f<T>(static_cast<const T*>(a.out)[a.os.at(b, h, i) + c]);
            const float o2 = to_f<T>(static_cast<const T*>(a.out2)[row * D + c]);
            d1 = fmaf(g, fmaf(lam, o2, o), d1);
            d2 = fmaf(g, o2, d2);
        }
    }
    for (int o = 16; o; o >>= 1) {
        d1 += __shfl_xor_sync(~0u, d1, o);
        d2 += __shfl_xor_sync(~0u, d2, o);
    }
    if (lane == 0) {
        a.delta[row] = d1;
        a.delta[rows + row] = d2;
    }
}

// dlambda_h = -sum over batch and queries of delta_2, one block a head, a fixed order.
template <typename T>
__global__ void __launch_bounds__(256) dense_dlambda_kernel(const DenseArgs a) {
    __shared__ double part[256];
    const int h = blockIdx.x;
    const long long rows = static_cast<long long>(a.B) * a.H * a.Nq;
    double s = 0.0;
    for (int b = 0; b < a.B; ++b)
        for (int i = threadIdx.x; i < a.Nq; i += 256)
            s += a.delta[rows + (static_cast<long long>(b) * a.H + h) * a.Nq + i];
    part[threadIdx.x] = s;
    __syncthreads();
    for (int o = 128; o; o >>= 1) {
        if (threadIdx.x < o) part[threadIdx.x] += part[threadIdx.x + o];
        __syncthreads();
    }
    if (threadIdx.x == 0) static_cast<T*>(a.dlam)[h] = from_f<T>(static_cast<float>(-part[0]));
}

// dq (KEYS = false, a warp a query) or dk and dv (KEYS = true, a warp a key).
template <int D, typename T, bool KEYS>
__global__ void __launch_bounds__(128) dense_bwd_rows_kernel(const DenseArgs a) {
    constexpr int C = D / 32, E = D / 2;
    __shared__ float xs[4][2 * D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int heads = KEYS ? a.Hk : a.H, len = KEYS ? a.Nk : a.Nq;
    const long long rows = static_cast<long long>(a.B) * a.H * a.Nq;
    const long long row = static_cast<long long>(blockIdx.x) * 4 + warp;
    if (row >= static_cast<long long>(a.B) * heads * len) return;
    const int r = row % len, hh = row / len % heads, b = row / len / heads;
    const int qn = dense_len(a.q_len, b, a.Nq), kn = dense_len(a.kv_len, b, a.Nk);
    const T *q = static_cast<const T*>(a.q), *k = static_cast<const T*>(a.k), *v = static_cast<const T*>(a.v),
            *g = static_cast<const T*>(a.dout);
    float acc[2][C];
    for (int c = 0; c < C; ++c) acc[0][c] = acc[1][c] = 0.f;
    if (r < (KEYS ? kn : qn)) {
        const T* x0 = KEYS ? k + a.ks.at(b, hh, r) : q + a.qs.at(b, hh, r);
        const T* x1 = KEYS ? v + a.vs.at(b, hh, r) : g + a.dos.at(b, hh, r);
        for (int c = lane; c < D; c += 32) {
            xs[warp][c] = to_f<T>(x0[c]);
            xs[warp][D + c] = to_f<T>(x1[c]);
        }
        __syncwarp();
        for (int gg = 0; gg < (KEYS ? a.G : 1); ++gg) {
            const int h = KEYS ? hh * a.G + gg : hh, hk = KEYS ? hh : hh / a.G;
            const float lam = to_f<T>(static_cast<const T*>(a.lam)[h]);
            const int first = KEYS && a.causal ? max(0, r - kn + qn) : 0;
            const int last = KEYS ? qn : (a.causal ? min(kn, max(0, r + kn - qn + 1)) : kn);
            for (int j0 = first; j0 < last; j0 += 32) {
                const int j = j0 + lane;
                float w0 = 0.f, ds1 = 0.f, ds2 = 0.f;
                if (j < last) {
                    const T* y0 = KEYS ? q + a.qs.at(b, h, j) : k + a.ks.at(b, hk, j);
                    const T* y1 = KEYS ? g + a.dos.at(b, h, j) : v + a.vs.at(b, hk, j);
                    float s1 = 0.f, s2 = 0.f, dp = 0.f;
                    for (int c = 0; c < E; ++c) {
                        s1 = fmaf(xs[warp][c], to_f<T>(y0[c]), s1);
                        s2 = fmaf(xs[warp][E + c], to_f<T>(y0[E + c]), s2);
                    }
                    for (int c = 0; c < D; ++c) dp = fmaf(xs[warp][D + c], to_f<T>(y1[c]), dp);
                    const int qi = KEYS ? j : r;
                    const long long at = (static_cast<long long>(b) * a.H + h) * a.Nq + qi;
                    const float* ls = a.lse + (static_cast<long long>(b) * a.H + h) * 2 * a.Nq + qi;
                    const float p1 = expf(s1 * a.scale - ls[0]), p2 = expf(s2 * a.scale - ls[a.Nq]);
                    w0 = p1 - lam * p2;
                    ds1 = a.scale * p1 * (dp - a.delta[at]);
                    ds2 = -lam * a.scale * p2 * (dp - a.delta[rows + at]);
                }
                for (int t = 0; t < min(32, last - j0); ++t) {
                    const float t0 = __shfl_sync(~0u, w0, t), t1 = __shfl_sync(~0u, ds1, t),
                                t2 = __shfl_sync(~0u, ds2, t);
                    const T* y0 = KEYS ? q + a.qs.at(b, h, j0 + t) : k + a.ks.at(b, hk, j0 + t);
                    const T* y1 = g + (KEYS ? a.dos.at(b, h, j0 + t) : 0);
                    for (int c = 0; c < C; ++c) {
                        acc[0][c] = fmaf(lane + 32 * c < E ? t1 : t2, to_f<T>(y0[lane + 32 * c]), acc[0][c]);
                        if (KEYS) acc[1][c] = fmaf(t0, to_f<T>(y1[lane + 32 * c]), acc[1][c]);
                    }
                }
            }
        }
    }
    for (int c = 0; c < C; ++c) {
        if (KEYS) {
            static_cast<T*>(a.dk)[a.dks.at(b, hh, r) + lane + 32 * c] = from_f<T>(acc[0][c]);
            static_cast<T*>(a.dv)[a.dvs.at(b, hh, r) + lane + 32 * c] = from_f<T>(acc[1][c]);
        } else {
            static_cast<T*>(a.dq)[a.dqs.at(b, hh, r) + lane + 32 * c] = from_f<T>(acc[0][c]);
        }
    }
}

}  // namespace sla

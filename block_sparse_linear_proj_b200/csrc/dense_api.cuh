// dense_api.cuh -- host side of the dense attention calls (part of sla_api.cu's
// translation unit): validation, workspace, launches.
#pragma once

namespace {

sla_status_t dense_check(const sla_dense_params_t* p) {
    if (!p) return SLA_ERR_INVALID_ARG;
    if (p->B <= 0 || p->H <= 0 || p->Hk <= 0 || p->Nq <= 0 || p->Nk < 0 || p->P < 0 || p->d <= 0)
        return SLA_ERR_INVALID_ARG;
    if (p->H % p->Hk != 0) return SLA_ERR_INVALID_ARG;
    if (p->io_dtype != SLA_IO_BF16 && p->io_dtype != SLA_IO_FP16) return SLA_ERR_INVALID_ARG;
    if ((p->causal != 0 && p->causal != 1) || (p->differential != 0 && p->differential != 1))
        return SLA_ERR_INVALID_ARG;
    if (!std::isfinite(p->sm_scale)) return SLA_ERR_INVALID_ARG;
    if (p->d != 64 && p->d != 128) return SLA_ERR_UNSUPPORTED;
    if (p->B > 65535 || p->H > 65535) return SLA_ERR_UNSUPPORTED;
    if (static_cast<long long>(p->B) * p->H > (1LL << 30) / p->Nq) return SLA_ERR_UNSUPPORTED;
    if (static_cast<long long>(p->Nk) + p->P >= (1LL << 30)) return SLA_ERR_UNSUPPORTED;
    return SLA_OK;
}

// A tensor's strides, checked: `st` has nd (2: head, token; 3: batch, head, token)
// values, NULL for a dense tensor.  A dimension of one entry gets stride 0.
sla_status_t dense_strides(const int64_t* st, int nd, int B, int H, int N, int d, bool output, sla::DenseT& t) {
    const long long size[3] = {nd == 3 ? B : 1, H, N};
    t = {0, 0, 0};
    if (N == 0) return SLA_OK;           // no entries: nothing to reach, nothing to overlap
    long long s[3] = {static_cast<long long>(H) * N * d, static_cast<long long>(N) * d, d};
    if (st)
        for (int x = 0; x < nd; ++x) s[3 - nd + x] = st[x];
    for (int x = 0; x < 3; ++x) {
        if (size[x] <= 1) { s[x] = 0; continue; }
        if (s[x] < 0 || s[x] % 8 != 0 || s[x] >= (1LL << 36)) return SLA_ERR_INVALID_ARG;
        if (s[x] == 0 && (output || x == 2)) return SLA_ERR_INVALID_ARG;
    }
    if (output) {      // entries apart: in the order of the strides, each at least the extent below it
        int o[3] = {0, 1, 2};
        std::sort(o, o + 3, [&](int x, int y) { return s[x] < s[y]; });
        long long extent = d;
        for (int x : o) {
            if (size[x] <= 1) continue;
            if (s[x] < extent) return SLA_ERR_INVALID_ARG;
            // (no address space has 2^60 elements; and the sum stays within 64 bits)
            if (s[x] > (1LL << 60) / size[x] || (extent += s[x] * (size[x] - 1)) > (1LL << 60)) return SLA_ERR_INVALID_ARG;
        }
    }
    t = {s[0], s[1], s[2]};
    return SLA_OK;
}

// How the forward call splits its work over CTAs (one an SM: 148 at once).
struct DensePlan {
    int tiles_g, splits_g, two_g, slots_g;   // gathered: every sequence's rows against the prefix
    int tiles_b, splits_b, two_b, slots_b;   // the rows of one sequence
    int gathered_items, items, prefix_b, direct;
    long long rows;
};

DensePlan dense_plan(const sla_dense_params_t* p) {
    DensePlan x{};
    const long long G = p->H / p->Hk, seq = G * p->Nq, all = seq * p->B;
    const bool diff = p->differential != 0;
    constexpr long long SMS = 148;          // a B200's
    auto cdiv = [](long long u, long long v) { return (u + v - 1) / v; };
    const long long nP = cdiv(p->P, sla::kDenseBN), nK = cdiv(p->Nk, sla::kDenseBN);
    x.rows = all * p->Hk;
    // The prefix is taken for all sequences at once where a sequence alone leaves most of a row tile empty.
    const bool gather = p->P > 0 && p->B > 1 && seq < 128;
    x.prefix_b = !gather;
    auto shape = [&](long long rows, int& tiles, int& two) {
        two = !diff && rows > 128;
        tiles = static_cast<int>(cdiv(rows, two ? 256 : 128));
    };
    shape(seq, x.tiles_b, x.two_b);
    if (gather) shape(all, x.tiles_g, x.two_g);
    const long long tb = nK + (gather ? 0 : nP);                       // key tiles of a unit
    const long long cb = gather && nK == 0 ? 0 : static_cast<long long>(p->B) * p->Hk * x.tiles_b,
                    cg = gather ? static_cast<long long>(p->Hk) * x.tiles_g : 0;
    const long long work = cb * tb + cg * nP;
    // Ranges of key tiles that give the gathered and the own units up to one CTA an SM each, of eight tiles at least
    // where there is that much work (a CTA's start, about 2.5 us, its end and the join cost as much as about that
    // many), else three: a step of 257 tokens and 2 heads / 16 x 5 drafted tokens on 4099 + 333 keys took 35.0 / 20.5 us
    // so, 37.2 / 24.2 with ranges of two tiles, 34.8 / 22.4 of four and 35.1 / 71.7 unsplit. (The join grows with the
    // rows, which the rule does not see: 512 tokens of 8 heads, 26.0 us in two ranges, take 16.4 in one.)  More ranges,
    // to even out sequences of different lengths, gave nothing with CTAs that each pay a start: 32 such caches, 1 range
    // each 118 us, 2 and 4: 116, 6: 121.
    const long long least = std::max<long long>(work >= 8 * SMS ? 8 : 3, cdiv(work, SMS));
    auto ranges = [&](long long units, long long tiles) {
        return units == 0 ? 0 : units >= SMS ? 1 : static_cast<int>(std::max<long long>(1, std::min(cdiv(tiles, least), SMS / units)));
    };
    x.splits_b = ranges(cb, tb);
    x.splits_g = ranges(cg, nP);
    // a stream of every second tile is a part of its own
    x.slots_b = x.splits_b * (!diff && !x.two_b ? 2 : 1);
    x.slots_g = x.splits_g * (!diff && !x.two_g ? 2 : 1);
    x.gathered_items = static_cast<int>(cg * x.splits_g);
    x.items = x.gathered_items + static_cast<int>(cb * x.splits_b);
    x.direct = x.slots_b + x.slots_g == 1;
    return x;
}

struct DenseWs {
    size_t rowdata, ext, dlam_part, dlam_done, bound, vnorm, opart, lpart, total;
};

DenseWs dense_layout(const sla_dense_params_t* p) {
    DenseWs w{};
    const DensePlan x = dense_plan(p);
    const size_t maps = p->differential ? 2 : 1;
    // the forward's parts and the backward's sums are never in use together
    size_t off = 0;
    auto take = [&](size_t bytes) { size_t o = off; off = align_up(off + bytes); return o; };
    if (!x.direct) {
        const size_t n = static_cast<size_t>(x.slots_b + x.slots_g) * maps * static_cast<size_t>(x.rows);
        w.opart = take(n * p->d * 4);
        w.lpart = take(n * 4);
    }
    w.total = off;
    off = 0;
    if (p->differential && p->P == 0) {        // (with a prefix no backward call can follow)
        const size_t tiles = static_cast<size_t>(p->B) * p->H * ((p->Nq + sla::kDenseRowTile - 1) / sla::kDenseRowTile);
        w.rowdata = take(tiles * sla::kDenseRowFloats * 4);
        w.ext = take(tiles * sla::kDenseExt);
        w.dlam_part = take(tiles * 4);         // (a place for each 128 queries; one for each 64 are enough)
        w.dlam_done = take(static_cast<size_t>(p->H) * 4);
        if (p->io_dtype == SLA_IO_FP16) {
            w.bound = take(tiles * 8);
            w.vnorm = take(static_cast<size_t>(p->B) * p->Hk * ((p->Nk + 127) / 128) * 4);
        }
    }
    w.total = std::max<size_t>(std::max(w.total, off), kAlign);
    return w;
}

// A launch; `early`: it may start before the kernel ahead of it in the stream has ended (and waits inside for that).
template <typename... P, typename... A>
cudaError_t dense_go(void (*kern)(P...), unsigned grid, unsigned threads, int smem, cudaStream_t st, bool early,
                     const A&... args) {
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(grid), c.blockDim = dim3(threads), c.dynamicSmemBytes = static_cast<size_t>(smem), c.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &at, c.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&c, kern, args...);
}

// Shared memory above the default is asked for once a kernel and device, and again if a launch says it is not there
// (a context that was reset).
template <typename... P, typename... A>
sla_status_t dense_launch(void (*kern)(P...), std::atomic<unsigned long long>& asked, unsigned grid, int smem,
                          cudaStream_t st, bool early, const A&... args) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SLA_ERR_CUDA;
    const unsigned long long bit = 1ull << (dev & 63);
    for (int tries = 0; tries < 2; ++tries) {
        const bool fresh = tries || dev > 63 || !(asked.load(std::memory_order_relaxed) & bit);
        if (fresh) {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
                return SLA_ERR_CUDA;
            asked.fetch_or(bit, std::memory_order_relaxed);
        }
        if (dense_go(kern, grid, sla::kDenseThreads, smem, st, early, args...) == cudaSuccess) return SLA_OK;
        cudaGetLastError();
        if (fresh) break;
    }
    return SLA_ERR_CUDA;
}

// 4-D map over a [B, Hk, N, d] tensor of 16-bit values, box 64 x tokens (128-byte swizzle).  A dimension of
// stride 0 has one entry in the map; the kernel's coordinate there is 0.
bool dense_map(CUtensorMap* m, const void* base, const sla::DenseT& t, int B, int Hk, int N, int d, bool half,
               int tokens = sla::kDenseBN) {
    EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N),
                                static_cast<cuuint64_t>(t.h ? Hk : 1), static_cast<cuuint64_t>(t.b ? B : 1)};
    const cuuint64_t row = static_cast<cuuint64_t>(d) * 2;
    const cuuint64_t strides[3] = {t.n ? static_cast<cuuint64_t>(t.n) * 2 : row,
                                   t.h ? static_cast<cuuint64_t>(t.h) * 2 : row,
                                   t.b ? static_cast<cuuint64_t>(t.b) * 2 : row};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(tokens), 1, 1}, one[4] = {1, 1, 1, 1};
    return fn(m, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base),
              dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

sla_status_t dense_check_ws(const sla_dense_params_t* p, void* ws, size_t ws_bytes, DenseWs& w) {
    w = dense_layout(p);
    if (!ws || !aligned(ws, kAlign) || ws_bytes < w.total) return SLA_ERR_WORKSPACE;
    return SLA_OK;
}

void dense_fill(const sla_dense_params_t* p, sla::DenseArgs& a) {
    a.B = p->B, a.H = p->H, a.Hk = p->Hk, a.G = p->H / p->Hk;
    a.Nq = p->Nq, a.Nk = p->Nk, a.P = p->P;
    a.causal = p->causal;
    const double tau = p->sm_scale > 0.f ? static_cast<double>(p->sm_scale)
                                         : 1.0 / std::sqrt(static_cast<double>(p->differential ? p->d / 2 : p->d));
    a.scale = static_cast<float>(tau);
    a.scale_log2 = static_cast<float>(tau * 1.4426950408889634);
}

// lambda, lengths and lse: small arrays without strides.
sla_status_t dense_small(const sla_dense_params_t* p, const void* lambda, const int32_t* q_len, const int32_t* kv_len,
                         const float* lse) {
    if (p->differential ? !lambda || !aligned(lambda, 2) : lambda != nullptr) return SLA_ERR_INVALID_ARG;
    if (!aligned(q_len, 4) || !aligned(kv_len, 4) || !aligned(lse, 4)) return SLA_ERR_INVALID_ARG;
    return SLA_OK;
}

template <int D, typename T, bool DIFF>
sla_status_t dense_fwd_t(const sla_dense_params_t* p, const sla::DenseArgs& a, void* ws, const DenseWs& w,
                         cudaStream_t st) {
    using L = sla::DenseFwdLayout<D, DIFF>;
    const DensePlan x = dense_plan(p);
    sla::DenseFwdArgs f{};
    f.a = a;
    f.k_b = a.ks.b != 0, f.k_h = a.ks.h != 0, f.v_b = a.vs.b != 0, f.v_h = a.vs.h != 0;
    f.kp_h = a.kps.h != 0, f.vp_h = a.vps.h != 0;
    f.gathered_items = x.gathered_items, f.tiles_g = x.tiles_g, f.splits_g = x.splits_g, f.two_g = x.two_g;
    f.tiles_b = x.tiles_b, f.splits_b = x.splits_b, f.two_b = x.two_b, f.prefix_b = x.prefix_b, f.direct = x.direct;
    f.slots_g = x.slots_g, f.slots_b = x.slots_b, f.rows = x.rows;
    f.opart = at<float>(ws, w.opart), f.lpart = at<float>(ws, w.lpart);
    f.wait_ns = wait_limit_ns();
    f.debug_stall = debug_stall() ? 1 : 0;
    sla::DenseMaps tm{};
    constexpr bool half = std::is_same<T, __half>::value;
    if (p->Nk && (!dense_map(&tm.k, a.k, a.ks, p->B, p->Hk, p->Nk, D, half) ||
                  !dense_map(&tm.v, a.v, a.vs, p->B, p->Hk, p->Nk, D, half)))
        return SLA_ERR_CUDA;
    if (p->P && (!dense_map(&tm.kp, a.kp, a.kps, 1, p->Hk, p->P, D, half) ||
                 !dense_map(&tm.vp, a.vp, a.vps, 1, p->Hk, p->P, D, half)))
        return SLA_ERR_CUDA;
    static std::atomic<unsigned long long> asked{0};
    {
        Span sp(SLA_KERNEL_DENSE, st);
        const sla_status_t s = dense_launch(sla::dense_fwd_kernel<D, T, DIFF>, asked, static_cast<unsigned>(x.items),
                                            L::SMEM, st, false, tm, f);
        if (s != SLA_OK) return s;
    }
    if (!x.direct) {
        Span sp(SLA_KERNEL_DENSE, st);
        if (dense_go(sla::dense_merge_kernel<D, T, DIFF>, static_cast<unsigned>((x.rows + 3) / 4), 128, 0, st, true, f) !=
            cudaSuccess)
            return SLA_ERR_CUDA;
    }
    return launch_status();
}

template <int D, typename T>
sla_status_t dense_fwd(const sla_dense_params_t* p, const sla::DenseArgs& a, void* ws, const DenseWs& w,
                       cudaStream_t st) {
    return p->differential ? dense_fwd_t<D, T, true>(p, a, ws, w, st) : dense_fwd_t<D, T, false>(p, a, ws, w, st);
}

template <int D, typename T>
sla_status_t dense_bwd(const sla_dense_params_t* p, const sla::DenseArgs& a, void* ws, const DenseWs& w,
                       cudaStream_t st) {
    using L = sla::DenseBwdLayout<D>;
    sla::DenseBwdArgs f{};
    f.a = a;
    f.q_b = a.qs.b != 0, f.q_h = a.qs.h != 0, f.do_b = a.dos.b != 0, f.do_h = a.dos.h != 0;
    f.k_b = a.ks.b != 0, f.k_h = a.ks.h != 0, f.v_b = a.vs.b != 0, f.v_h = a.vs.h != 0;
    f.key_tiles = (p->Nk + 127) / 128;
    f.query_tiles = (p->Nq + 127) / 128;
    f.row_tiles = (p->Nq + sla::kDenseRowTile - 1) / sla::kDenseRowTile;
    f.key_items = p->B * p->Hk * f.key_tiles;
    f.rowdata = at<float>(ws, w.rowdata), f.ext = at<unsigned char>(ws, w.ext);
    f.dlam_part = at<float>(ws, w.dlam_part), f.dlam_done = at<unsigned>(ws, w.dlam_done);
    f.bound = at<float2>(ws, w.bound), f.vnorm = at<float>(ws, w.vnorm);
    f.wait_ns = wait_limit_ns();
    f.debug_stall = debug_stall() ? 1 : 0;
    sla::DenseBwdMaps tm{};
    constexpr bool half = std::is_same<T, __half>::value;
    if (!dense_map(&tm.q, a.q, a.qs, p->B, p->H, p->Nq, D, half, 64) ||
        !dense_map(&tm.dout, a.dout, a.dos, p->B, p->H, p->Nq, D, half, 64) ||
        (p->Nk && (!dense_map(&tm.k, a.k, a.ks, p->B, p->Hk, p->Nk, D, half, 64) ||
                   !dense_map(&tm.v, a.v, a.vs, p->B, p->Hk, p->Nk, D, half, 64))))
        return SLA_ERR_CUDA;
    static std::atomic<unsigned long long> asked{0};
    {
        Span sp(SLA_KERNEL_DENSE_BWD, st);
        const unsigned rows = static_cast<unsigned>(p->B) * p->H * f.row_tiles;
        sla::dense_rows_kernel<D, T><<<rows + (half ? static_cast<unsigned>(f.key_items) : 0u), 256, 0, st>>>(f);
    }
    {
        Span sp(SLA_KERNEL_DENSE_BWD, st);
        const sla_status_t s = dense_launch(sla::dense_bwd_kernel<D, T>, asked,
                                            static_cast<unsigned>(f.key_items + p->B * p->H * f.query_tiles), L::SMEM, st,
                                            true, tm, f);
        if (s != SLA_OK) return s;
    }
    return launch_status();
}

template <typename F>
sla_status_t dense_dispatch(const sla_dense_params_t* p, F f) {
    if (p->io_dtype == SLA_IO_BF16)
        return p->d == 128 ? f(std::integral_constant<int, 128>{}, __nv_bfloat16{})
                           : f(std::integral_constant<int, 64>{}, __nv_bfloat16{});
    return p->d == 128 ? f(std::integral_constant<int, 128>{}, __half{})
                       : f(std::integral_constant<int, 64>{}, __half{});
}

}  // namespace

extern "C" size_t sla_dense_workspace_size(const sla_dense_params_t* p) {
    if (dense_check(p) != SLA_OK) return 0;
    return dense_layout(p).total;
}

extern "C" sla_status_t sla_diff_forward(const sla_dense_params_t* p, const int64_t* strides, const void* q,
                                         const void* k, const void* v, const void* lambda, const int32_t* q_len,
                                         const int32_t* kv_len, void* out, void* out2, float* lse, void* workspace,
                                         size_t ws_bytes, sla_stream_t stream) {
    sla_status_t s = dense_check(p);
    if (s != SLA_OK) return s;
    if (p->differential != 1 || p->P != 0) return SLA_ERR_INVALID_ARG;
    if ((s = check_tensor(q, 16)) || (s = check_tensor(out, 16)) || (p->Nk && (s = check_tensor(k, 16))) ||
        (p->Nk && (s = check_tensor(v, 16))) || (s = dense_small(p, lambda, q_len, kv_len, lse)))
        return s;
    if (!aligned(out2, 16)) return SLA_ERR_INVALID_ARG;
    sla::DenseArgs a{};
    if ((s = dense_strides(strides, 3, p->B, p->H, p->Nq, p->d, false, a.qs)) ||
        (s = dense_strides(strides ? strides + 3 : nullptr, 3, p->B, p->Hk, p->Nk, p->d, false, a.ks)) ||
        (s = dense_strides(strides ? strides + 6 : nullptr, 3, p->B, p->Hk, p->Nk, p->d, false, a.vs)) ||
        (s = dense_strides(strides ? strides + 9 : nullptr, 3, p->B, p->H, p->Nq, p->d, true, a.os)))
        return s;
    DenseWs w;
    if ((s = dense_check_ws(p, workspace, ws_bytes, w))) return s;
    dense_fill(p, a);
    a.q = q, a.k = k, a.v = v, a.lam = lambda, a.q_len = q_len, a.kv_len = kv_len;
    a.out = out, a.out2 = out2, a.lse = lse;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return finish(dense_dispatch(p, [&](auto d, auto t) { return dense_fwd<d(), decltype(t)>(p, a, workspace, w, st); }), st);
}

extern "C" sla_status_t sla_diff_backward(const sla_dense_params_t* p, const int64_t* strides, const void* q,
                                          const void* k, const void* v, const void* lambda, const int32_t* q_len,
                                          const int32_t* kv_len, const void* out, const void* out2, const float* lse,
                                          const void* dout, void* dq, void* dk, void* dv, void* dlambda,
                                          void* workspace, size_t ws_bytes, sla_stream_t stream) {
    sla_status_t s = dense_check(p);
    if (s != SLA_OK) return s;
    if (p->differential != 1 || p->P != 0) return SLA_ERR_INVALID_ARG;
    if ((s = check_tensor(q, 16)) || (s = check_tensor(out, 16)) || (s = check_tensor(out2, 16)) ||
        (s = check_tensor(lse, 4)) || (s = check_tensor(dout, 16)) || (s = check_tensor(dq, 16)) ||
        (s = check_tensor(dlambda, 2)) || (s = dense_small(p, lambda, q_len, kv_len, lse)))
        return s;
    if (p->Nk && ((s = check_tensor(k, 16)) || (s = check_tensor(v, 16)) || (s = check_tensor(dk, 16)) ||
                  (s = check_tensor(dv, 16))))
        return s;
    // (a scale at which log-sum-exps over it leave the range of the kernel's parts: 2^-20, 2^-100)
    if (p->sm_scale > 0.f && p->sm_scale < (p->io_dtype == SLA_IO_FP16 ? 9.5367431640625e-7f : 7.888609e-31f))
        return SLA_ERR_UNSUPPORTED;
    // (broadcast keys of a size that no gradient has room for)
    if (static_cast<long long>(p->B) * p->Hk * ((p->Nk + 127) / 128) > (1LL << 30)) return SLA_ERR_UNSUPPORTED;
    sla::DenseArgs a{};
    struct { sla::DenseT* t; int h, n; bool output; } const want[8] = {
        {&a.qs, p->H, p->Nq, false}, {&a.ks, p->Hk, p->Nk, false}, {&a.vs, p->Hk, p->Nk, false},
        {&a.os, p->H, p->Nq, false}, {&a.dos, p->H, p->Nq, false}, {&a.dqs, p->H, p->Nq, true},
        {&a.dks, p->Hk, p->Nk, true}, {&a.dvs, p->Hk, p->Nk, true}};
    for (int x = 0; x < 8; ++x)
        if ((s = dense_strides(strides ? strides + 3 * x : nullptr, 3, p->B, want[x].h, want[x].n, p->d,
                               want[x].output, *want[x].t)))
            return s;
    DenseWs w;
    if ((s = dense_check_ws(p, workspace, ws_bytes, w))) return s;
    dense_fill(p, a);
    a.q = q, a.k = k, a.v = v, a.lam = lambda, a.q_len = q_len, a.kv_len = kv_len;
    a.out = const_cast<void*>(out), a.out2 = const_cast<void*>(out2), a.lse = const_cast<float*>(lse);
    a.dout = dout, a.dq = dq, a.dk = dk, a.dv = dv, a.dlam = dlambda;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return finish(dense_dispatch(p, [&](auto d, auto t) { return dense_bwd<d(), decltype(t)>(p, a, workspace, w, st); }), st);
}

extern "C" sla_status_t sla_prefix_forward(const sla_dense_params_t* p, const int64_t* strides, const void* q,
                                           const void* k_prefix, const void* v_prefix, const void* k, const void* v,
                                           const void* lambda, const int32_t* q_len, const int32_t* kv_len, void* out,
                                           float* lse, void* workspace, size_t ws_bytes, sla_stream_t stream) {
    sla_status_t s = dense_check(p);
    if (s != SLA_OK) return s;
    if ((s = check_tensor(q, 16)) || (s = check_tensor(out, 16)) || (s = dense_small(p, lambda, q_len, kv_len, lse)))
        return s;
    if (p->Nk && ((s = check_tensor(k, 16)) || (s = check_tensor(v, 16)))) return s;
    if (p->P && ((s = check_tensor(k_prefix, 16)) || (s = check_tensor(v_prefix, 16)))) return s;
    sla::DenseArgs a{};
    if ((s = dense_strides(strides, 3, p->B, p->H, p->Nq, p->d, false, a.qs)) ||
        (s = dense_strides(strides ? strides + 3 : nullptr, 2, 1, p->Hk, p->P, p->d, false, a.kps)) ||
        (s = dense_strides(strides ? strides + 5 : nullptr, 2, 1, p->Hk, p->P, p->d, false, a.vps)) ||
        (s = dense_strides(strides ? strides + 7 : nullptr, 3, p->B, p->Hk, p->Nk, p->d, false, a.ks)) ||
        (s = dense_strides(strides ? strides + 10 : nullptr, 3, p->B, p->Hk, p->Nk, p->d, false, a.vs)) ||
        (s = dense_strides(strides ? strides + 13 : nullptr, 3, p->B, p->H, p->Nq, p->d, true, a.os)))
        return s;
    DenseWs w;
    if ((s = dense_check_ws(p, workspace, ws_bytes, w))) return s;
    dense_fill(p, a);
    a.q = q, a.k = k, a.v = v, a.kp = k_prefix, a.vp = v_prefix, a.lam = lambda;
    a.q_len = q_len, a.kv_len = kv_len, a.out = out, a.lse = lse;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return finish(dense_dispatch(p, [&](auto d, auto t) { return dense_fwd<d(), decltype(t)>(p, a, workspace, w, st); }), st);
}

// dense.cuh -- dense attention: differential attention with its gradients, and
// attention over a shared prefix.
#pragma once
#include <type_traits>

#include "attn.cuh"
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
__device__ __forceinline__ int dense_len_in(int n, int most) {
    if (n < 0 || n > most) {
        report(kStatusBadData);
        return n < 0 ? 0 : most;
    }
    return n;
}
__device__ __forceinline__ int dense_len(const int32_t* len, int b, int most) {
    return len ? dense_len_in(len[b], most) : most;
}

// ------------------------------------------------------------------ forward
// One CTA owns up to 256 query rows of one key/value head and walks a range of
// 128-key tiles with two softmax streams, a warpgroup each:
//   plain, many rows  stream s = rows [128 s, 128 s + 128), every tile
//   plain, <= 128     both streams the same rows, stream s the tiles of parity s
//   differential      stream s = map s of the same 128 rows, every tile
// Stream s: S_s = Q K^T (tcgen05, M = N = 128, fp32 in tensor memory; map s
// contracts its half of the head), one row a thread: running maximum and sum in
// fp32, P in 16 bits written over the first columns of S_s, O_s += P V, its first
// half while the second half's weights are formed.  While one stream is in its
// softmax the tensor core works for the other:
//   S_s(0) | P_s(u) V  S_s(u+1) | ...
// (in issue order, so S_s(u+1) may overwrite P_s(u), and S_s(u+1) complete means
// that O_s holds tile u).  A row rescales O_s only when its maximum has grown by
// 2^8 (P stays below 2^8, exact in the sum; the reference maximum cancels in
// O / l).  fp16 weights are lifted by a further 2^7, so that they fill the type's
// range: beside a dominating key the many others' 2^-25 would be 0 in the product,
// though not in l.  The bound is the special function unit (8 cycles a warp and ex2,
// 2048 for a tile of both streams) beside the tensor core (1536, plain 2048).
// Other forms of it, each measured once on the 10400-token differential forward when
// this one took 1.04 ms: 64-key tiles with two buffers of S 1.15, three eighths of
// the exponentials as polynomials on the FMA pipe 1.13.  (This one has taken 1.04 to
// 1.13 ms on different boxes; 64-key tiles with four warpgroups, 1.10, one issuing
// warp for both streams, 1.08, and a quarter of the exponentials as polynomials,
// 1.06, lie within that.)
// Rows are (query i, head g of the group) in the order i * G + g, so a causal
// tile ends early and the heads of a group share each key tile.  Key tiles come
// from the prefix first, then the sequence's own keys.  Where sequences have few
// rows, "gathered" CTAs take the rows of all sequences against the prefix, and
// the prefix is read once; their parts and those of split ranges are joined by
// dense_merge_kernel.
// Value rows past a sequence's length may hold anything (and 0 * NaN is NaN):
// they are zeroed in shared memory.
// Warps: w0 TMA producer, w1 and w2 MMA issuers of the streams, w4-11 the streams.
constexpr int kDenseBN = 128;
constexpr int kDenseThreads = 384;

struct DenseMaps {
    CUtensorMap k, v, kp, vp;      // [B, Hk, N, D] 16-bit, box 64 x 128 tokens
};

struct DenseFwdArgs {
    DenseArgs a;
    int k_b, k_h, v_b, v_h, kp_h, vp_h;   // 0: that dimension is broadcast in the map
    int gathered_items, tiles_g, splits_g, two_g;  // gathered CTAs: prefix only
    int tiles_b, splits_b, two_b;                  // CTAs of one sequence
    int prefix_b;                                  // these walk the prefix too
    int direct;                                    // one part: results, else parts
    float* opart;                                  // [slot][map][row][D] fp32
    float* lpart;                                  // [slot][map][row] log2 units
    int slots_g, slots_b;
    long long rows;                                // B * Hk * G * Nq
    unsigned long long wait_ns;
    int debug_stall;                               // test hook: load no tiles, so the consumers' waits run out
};

template <int D, bool DIFF>
struct DenseFwdLayout {
    static constexpr int NQ = DIFF ? 1 : 2;
    static constexpr int QBOX = 128 * 128;                // 64 columns of 128 rows
    static constexpr int QTILE = 128 * D * 2;
    static constexpr int BOX = kDenseBN * 128;            // 64 columns of a key tile
    static constexpr int TILE = kDenseBN * D * 2;
    static constexpr int SLOTS = D == 128 ? (DIFF ? 6 : 5) : 8;
    static constexpr int OFF_RING = NQ * QTILE;
    static constexpr int OFF_MISC = OFF_RING + SLOTS * TILE;
    static constexpr int SMEM = 1024 + OFF_MISC + 512;
    static_assert(SMEM <= 232448, "shared memory of an SM");
};

// Bounded wait of a converged warp: all of its lanes, without a branch on the lane (a
// wait inside one took some 250 cycles longer, measured).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
    return __all_sync(~0u, mbar_wait(bar, parity, abort, limit_ns)) != 0;
}
// A place in a ring of mbarrier-guarded slots.  (Kept as slot and phase: quotients
// and remainders of a running index are long chains of dependent instructions in
// the issuing warps, whose step time bounds the pipeline.)
template <int SLOTS>
struct RingPos {
    int slot;
    uint32_t phase;
    __device__ __forceinline__ void step(int d) {
        slot += d;
        if (slot >= SLOTS) {
            slot -= SLOTS;
            phase ^= 1u;
        }
    }
};
// Named barriers between the two streams' warps of a scheduler (ids 2..9).
__device__ __forceinline__ void turn_wait(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void turn_give(int id) { asm volatile("bar.arrive %0, 64;" ::"r"(id) : "memory"); }
// One lane of a converged warp (always the same one).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int n, int h,
                                            int b) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(n), "r"(h), "r"(b)
        : "memory");
}
// Programmatic dependent launch: a kernel lets the next one of its stream start early, and that one waits here for
// all of the first's work before it touches any of it.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) { return pack_bf16(lo, hi); }
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) { return pack_half2(lo, hi); }
template <typename T>
__host__ __device__ constexpr uint32_t idesc_t(int M, int N, int a_mn, int b_mn) {
    return std::is_same<T, __half>::value ? idesc_f16(M, N, a_mn, b_mn) : idesc_bf16(M, N, a_mn, b_mn);
}

// 2^x for two values.
__device__ __forceinline__ uint64_t exp2_2(uint64_t x) {
    float a, b;
    f2unpack(x, a, b);
    return f2pack(fast_exp2(a), fast_exp2(b));
}
// The streams' weights are P 2^lift: to 2^15 of fp16's 65504, and down to 2^-31.
template <typename T>
constexpr float kDenseLift = std::is_same<T, __half>::value ? 7.f : 0.f;
// Own keys that query i of a sequence sees: [0, this).
__device__ __forceinline__ int dense_own(int i, int qn, int kn, int causal) {
    return causal ? min(kn, max(0, i + kn - qn + 1)) : kn;
}

template <int D, typename T, bool DIFF>
__global__ void __launch_bounds__(kDenseThreads, 1)
    dense_fwd_kernel(const __grid_constant__ DenseMaps tm, const __grid_constant__ DenseFwdArgs f) {
    using L = DenseFwdLayout<D, DIFF>;
    constexpr int NBOX = D / 64, SLOTS = L::SLOTS;
    constexpr uint32_t COL_O = 256;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const DenseArgs& a = f.a;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::OFF_MISC);   // [SLOTS]
    uint64_t* empty = full + SLOTS;                                     // [SLOTS]
    uint64_t* q_full = empty + SLOTS;
    uint64_t* s_full = q_full + 1;                                      // [stream]
    uint64_t* p_full = s_full + 2;                                      // [stream][half]
    uint64_t* v_here = p_full + 4;                                      // [stream] the dirty tile's values have landed
    uint64_t* o_full = v_here + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(o_full + 1);
    volatile int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
    float* xl = reinterpret_cast<float*>(smem + L::OFF_RING);           // [2][128] row sums, after the last product

    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;

    let_next_start();
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    // ------------------------------------------------------------ which rows, which keys
    const bool gathered = static_cast<int>(blockIdx.x) < f.gathered_items;
    int it = gathered ? blockIdx.x : blockIdx.x - f.gathered_items;
    const int splits = gathered ? f.splits_g : f.splits_b, tiles = gathered ? f.tiles_g : f.tiles_b;
    const bool two = DIFF ? false : (gathered ? f.two_g : f.two_b) != 0;       // two row tiles
    const int sp = it % splits;
    it /= splits;
    int tile, hk, b0;
    if (gathered) {
        tile = it % tiles, hk = it / tiles, b0 = 0;
    } else {           // a head's key tiles stay in L2 while its row tiles run; the longest causal rows first
        tile = tiles - 1 - it % tiles;
        it /= tiles;
        hk = it % a.Hk, b0 = it / a.Hk;
    }
    const int per_seq = a.G * a.Nq;
    const int rows = gathered ? a.B * per_seq : per_seq;
    const int row0 = tile * (two ? 256 : 128);
    // (both lengths are asked for before either is looked at)
    const int q_raw = !gathered && a.q_len ? a.q_len[b0] : a.Nq, k_raw = !gathered && a.kv_len ? a.kv_len[b0] : a.Nk;
    const int qn0 = gathered ? 0 : dense_len_in(q_raw, a.Nq), kn0 = gathered ? 0 : dense_len_in(k_raw, a.Nk);
    const int nP = (gathered || f.prefix_b) ? (a.P + kDenseBN - 1) / kDenseBN : 0;
    int own = 0;                                   // own keys that the last query of these rows sees
    if (!gathered) {
        const int i_last = min(min(rows, row0 + (two ? 256 : 128)) - 1, rows - 1) / a.G;
        own = dense_own(min(i_last, qn0 - 1), qn0, kn0, a.causal);
    }
    const bool any_row = gathered || row0 / a.G < qn0;
    const int total = any_row ? nP + (own + kDenseBN - 1) / kDenseBN : 0;
    const int t_begin = static_cast<int>(static_cast<long long>(total) * sp / splits),
              n = static_cast<int>(static_cast<long long>(total) * (sp + 1) / splits) - t_begin;
    // the one tile that holds value rows past the sequence's length
    const int dirty = (!gathered && kn0 < a.Nk && kn0 % kDenseBN != 0) ? nP + kn0 / kDenseBN - t_begin : -1;

    if (tid == 0) {
        for (int s = 0; s < SLOTS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], DIFF || two ? 2 : 1);
        }
        mbar_init(q_full, 8);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&p_full[2 * s], 4);
            mbar_init(&p_full[2 * s + 1], 4);
            mbar_init(&v_here[s], 1);
        }
        mbar_init(o_full, 2);
        *abort_flag = 0;
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const unsigned long long lim = f.wait_ns;
    auto fail = [&]() {
        *abort_flag = 1;
        report(kStatusTimeout);
    };
    // Tiles are loaded in the order of their use, K(0) .. K(lead - 1), then V(i), K(i + lead), ...; a K(i + lead) past
    // the last tile leaves its place empty.  So V(i) has place 2 i + lead, K(i) place i < lead ? i : 2 i - lead + 1.
    const bool every = DIFF || two;                 // each stream takes every tile
    const int lead = every ? 1 : 2;

    if (warp < 4) reg_dec<72>();
    if (warp == 0) {
        // ==================================================== producer (the whole warp waits, one lane issues)
        const bool leader = elect_one();
        RingPos<SLOTS> rp{0, 1u};           // (phase of the wait for an empty slot: the first round passes)
        uint32_t used = 0u, last = 0u;      // slots loaded, and the phases of their last loads
        bool ok = true;
        auto load = [&](int i, bool val) {
            if (!warp_wait(&empty[rp.slot], rp.phase, abort_flag, lim)) return false;
            const int t = t_begin + i;
            const bool pre = t < nP;
            if (leader) {
                const CUtensorMap* m = pre ? (val ? &tm.vp : &tm.kp) : (val ? &tm.v : &tm.k);
                const int tok = (pre ? t : t - nP) * kDenseBN;
                const int h = hk * (pre ? (val ? f.vp_h : f.kp_h) : (val ? f.v_h : f.k_h));
                const int b = pre ? 0 : b0 * (val ? f.v_b : f.k_b);
                mbar_arrive_expect_tx(&full[rp.slot], L::TILE);
                for (int c = 0; c < NBOX; ++c)
                    tma_load_4d(smem + L::OFF_RING + rp.slot * L::TILE + c * L::BOX, m, &full[rp.slot], c * 64, tok, h, b);
            }
            __syncwarp();
            used |= 1u << rp.slot;
            last = (last & ~(1u << rp.slot)) | ((rp.phase ^ 1u) << rp.slot);
            return true;
        };
        const int n_load = f.debug_stall ? 0 : n;
        for (int i = 0; ok && i < lead; ++i, rp.step(1))
            if (i < n_load) ok = load(i, false);
        for (int i = 0; ok && i < n_load; ++i) {
            ok = load(i, true);
            rp.step(1);
            if (ok && i + lead < n_load) ok = load(i + lead, false);
            rp.step(1);
        }
        if (!ok) fail();
        for (int y = 0; y < SLOTS; ++y)     // every load has landed before the CTA exits
            if ((used >> y) & 1u) mbar_drain(&full[y], (last >> y) & 1u, abort_flag);
    } else if (warp == 1 || warp == 2) {
        // ==================================================== MMA issuers (the whole warp waits, one lane issues)
        // One a stream: an issue blocks until the tensor core takes it, and a wait after it starts only then, so one
        // issuer for both streams leaves the tensor core idle between them.  Every issuer waits for every load in
        // order, so that it sees each phase of a slot; where the streams take different tiles that is one issuer for
        // both (two of them, each with its own tiles alone, would mistake a slot's phases for each other).
        constexpr uint32_t ID_S = idesc_t<T>(128, kDenseBN, 0, 0), ID_O = idesc_t<T>(128, D, 0, 1);
        const bool leader = elect_one();
        auto wait = [&](uint64_t* bar, uint32_t par) { return warp_wait(bar, par, abort_flag, lim); };
        const uint64_t q0 = sdesc(sbase, 16, 1024, kSwizzle128B), k0 = sdesc(sbase + L::OFF_RING, 16, 1024, kSwizzle128B),
                       v0 = sdesc(sbase + L::OFF_RING, L::BOX, 1024, kSwizzle128B);
        const uint32_t q_step = two ? L::QTILE >> 4 : 0;
        RingPos<SLOTS> rp{0, 0u};
        // S of stream s from the key tile at rp
        auto qk = [&](int s) {
            if (!wait(&full[rp.slot], rp.phase)) return false;
            if (leader) {
                const uint64_t qd = q0 + s * q_step, kd = k0 + rp.slot * (L::TILE >> 4);
                constexpr int STEPS = DIFF ? D / 32 : D / 16;
#pragma unroll
                for (int k = 0; k < STEPS; ++k) {
                    const int kk = k + (DIFF ? s * STEPS : 0);
                    umma_f16_ss(tmem + s * 128, qd + (((kk >> 2) * L::QBOX + (kk & 3) * 32) >> 4),
                                kd + (((kk >> 2) * L::BOX + (kk & 3) * 32) >> 4), ID_S, k > 0 ? 1u : 0u);
                }
                umma_commit(&s_full[s]);
                umma_commit(&empty[rp.slot]);
            }
            __syncwarp();
            return true;
        };
        // O_s += P_s V with the value tile i at rp, the stream's u-th, each half once its weights are there
        auto pv = [&](int s, int i, uint32_t u) {
            if (!wait(&full[rp.slot], rp.phase)) return false;
            if (i == dirty && leader) mbar_arrive(&v_here[s]);
            const uint64_t vd = v0 + rp.slot * (L::TILE >> 4);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (!wait(&p_full[2 * s + half], u & 1)) return false;
                tc_fence_after();
                if (leader)
#pragma unroll
                    for (int k = half * 4; k < half * 4 + 4; ++k)
                        umma_f16_ts(tmem + COL_O + s * D, tmem + s * 128 + k * 8, vd + ((k * 2048) >> 4), ID_O,
                                    (u > 0 || k > 0) ? 1u : 0u);
            }
            if (leader) umma_commit(&empty[rp.slot]);
            __syncwarp();
            return true;
        };
        bool ok = n == 0 || wait(q_full, 0);
        tc_fence_after();
        if (every) {
            const int s = warp - 1;
            if (ok && n > 0) ok = qk(s);
            rp.step(1);
            for (int i = 0; ok && i < n; ++i) {
                if (!(ok = pv(s, i, i))) break;
                rp.step(1);
                if (i + 1 < n) ok = qk(s);
                rp.step(1);
            }
        } else if (warp == 1) {
            for (int i = 0; ok && i < min(n, 2); ++i, rp.step(1)) ok = qk(i);
            if (n < 2) rp.step(2 - n);
            for (int i = 0; ok && i < n; ++i) {
                if (!(ok = pv(i & 1, i, i >> 1))) break;
                rp.step(1);
                if (i + 2 < n) ok = qk(i & 1);
                rp.step(1);
            }
        }
        if (!ok) fail();
        if (leader) umma_commit(o_full);   // also: every MMA has completed before tensor memory is released
        mbar_drain(o_full, 0, abort_flag);
    } else if (warp >= 4) {
        reg_inc<216>();
        // ==================================================== streams
        const int q4 = warp & 3, s = (warp - 4) >> 2, r = q4 * 32 + lane;
        const uint32_t tl = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
        auto wwait = [&](uint64_t* bar, uint32_t par) { return warp_wait(bar, par, abort_flag, lim); };
        // a row of the CTA's (this thread's is asked for again after the loop, which has few registers left)
        struct Row {
            int b, lr, qi, h;
            bool in, real;
        };
        auto row_of = [&](int rr) {
            const int gr = row0 + rr;
            Row x;
            x.in = gr < rows;
            x.b = gathered ? (x.in ? gr / per_seq : 0) : b0;
            x.lr = gathered ? gr % per_seq : gr;
            x.qi = x.lr / a.G;
            x.h = hk * a.G + x.lr % a.G;
            x.real = x.in && x.qi < (gathered ? dense_len(a.q_len, x.b, a.Nq) : qn0);
            return x;
        };
        const int my_row = (two ? s * 128 : 0) + r;
        if (n > 0) {
            // the query rows, zeros where there is no query: a lane finds the place of one row, D/8 lanes load a row, and
            // four of a lane's loads are in flight at once (a 16-byte chunk of a row of its own for each lane took up to
            // 6 us for 256 gathered rows)
            constexpr int LANES = D / 8;                        // 16-byte chunks a row
            const int per_warp = two ? 32 : 16, first = (warp - 4) * per_warp;
            const Row x = row_of(first + lane % per_warp);
            const T* mine = x.real ? static_cast<const T*>(a.q) + a.qs.at(x.b, x.h, x.qi) : nullptr;
            const int c = lane % LANES;
#pragma unroll 1
            for (int y0 = 0; y0 < per_warp; y0 += 4 * (32 / LANES)) {
                uint4 v[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const char* src = reinterpret_cast<const char*>(__shfl_sync(
                        ~0u, reinterpret_cast<unsigned long long>(mine), y0 + z * (32 / LANES) + lane / LANES));
                    v[z] = src ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int rr = first + y0 + z * (32 / LANES) + lane / LANES;
                    *reinterpret_cast<uint4*>(smem + (rr >> 7) * L::QTILE + (c >> 3) * L::QBOX + sw128(rr & 127, c & 7)) = v[z];
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }
        const int own_r = gathered ? 0 : dense_own(row_of(my_row).qi, qn0, kn0, a.causal);
        const float c = a.scale_log2, grow = 8.f / c;
        float m = -INFINITY, l = 0.f;                           // reference maximum (raw logits), sum
        bool ok = true;
        const int step = every ? 1 : 2;
        // The streams' warps of a scheduler take turns at the exponentials: in lockstep they would share the special
        // function unit there, and the tensor core elsewhere, and leave each idle half of the time.  A stream that
        // gave up keeps taking its turns.
        const int my_turn = 2 + s * 4 + q4, other_turn = 2 + (1 - s) * 4 + q4;
        if (every && s == 1 && n > 0) turn_give(other_turn);
        int u = 0;
        for (int i = step == 2 ? s : 0; i < n; i += step, ++u) {
            const uint32_t sc = tl + s * 128;              // this thread's S, and its P over it
            uint32_t sv[2][64];
            ok = ok && wwait(&s_full[s], u & 1);
            if (ok) {
                tc_fence_after();
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    tmem_ld32(sc + x * 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[x >> 1][(x & 1) * 32]));
                tmem_ld_wait();
                // columns that this row sees
                const int t = t_begin + i, see = t < nP ? a.P - t * kDenseBN : own_r - (t - nP) * kDenseBN;
                if (__any_sync(~0u, see < kDenseBN)) {
#pragma unroll
                    for (int y = 0; y < kDenseBN; ++y)
                        if (y >= see) sv[y >> 6][y & 63] = 0xFF800000u;       // -inf
                }
                const float mx = fmaxf(max64_bits(sv[0]), max64_bits(sv[1]));
                const bool up = mx > m + grow || (m == -INFINITY && mx > m);
                if (__any_sync(~0u, up)) {
                    const float to = up ? mx : m, k = up ? fast_exp2((m - to) * c) : 1.f;      // 0 from -inf
                    l *= k;
                    m = to;
                    if (u > 0) {
#pragma unroll 1
                        for (int x = 0; x < D; x += 32) {
                            uint32_t o[32];
                            tmem_ld32(tl + COL_O + s * D + x, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * k);
                            tmem_st32(tl + COL_O + s * D + x, o);
                        }
                    }
                }
                if (i == dirty && (ok = wwait(&v_here[s], 0))) {
                    // value rows past the sequence's length to zero, before this stream's P is announced (each
                    // stream does it for its own products)
                    const int x = (2 * i + lead) % SLOTS, r0 = kn0 % kDenseBN;
                    unsigned char* vt = smem + L::OFF_RING + x * L::TILE + r0 * 128;
                    for (int y = r; y < (kDenseBN - r0) * 8; y += 128)
#pragma unroll
                        for (int bx = 0; bx < NBOX; ++bx)
                            *reinterpret_cast<uint4*>(vt + bx * L::BOX + y * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
            }
            if (every) turn_wait(my_turn);
            if (ok) {
                const float nm = m == -INFINITY ? 0.f : fmaf(-m, c, kDenseLift<T>);
                const uint64_t c2 = f2pack(c, c), nm2 = f2pack(nm, nm);
                uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t pw[32];
#pragma unroll
                    for (int y = 0; y < 32; ++y) {
                        const uint64_t e =
                            ffma2(f2pack(__uint_as_float(sv[x][2 * y]), __uint_as_float(sv[x][2 * y + 1])), c2, nm2);
                        const uint64_t w = exp2_2(e);
                        if (y & 1) sum1 = fadd2(sum1, w);
                        else sum0 = fadd2(sum0, w);
                        float lo, hi;
                        f2unpack(w, lo, hi);
                        pw[y] = pack2<T>(lo, hi);
                    }
                    if (x == 1 && every && (s == 0 || i + 1 < n)) turn_give(other_turn);
                    tmem_st32(sc + x * 32, pw);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[2 * s + x]);
                }
                float s0, s1;
                f2unpack(fadd2(sum0, sum1), s0, s1);
                l += s0 + s1;
            } else if (every && (s == 0 || i + 1 < n)) {
                turn_give(other_turn);
            }
        }
        if (!ok) fail();
        // ---------------------------------------------------- results
        ok = wwait(o_full, 0) && ok;
        tc_fence_after();
        int again = my_row;
        asm volatile("" : "+r"(again));
        const Row me = row_of(again);
        const int b = me.b, lr = me.lr, qi = me.qi, h = me.h;
        const bool in = me.in, real = me.real;
        if (!real || m == -INFINITY) l = 0.f;
        const float lse2 = l > 0.f ? m * c + (log2f(l) - kDenseLift<T>) : -INFINITY;
        const long long prow = (static_cast<long long>(b) * a.Hk + hk) * per_seq + lr;
        constexpr int M = DIFF ? 2 : 1;
        // parts: [slot][map][row]; a plain stream of its own tiles is a slot of its own
        const int slot = (gathered ? 0 : f.slots_g) + (step == 2 ? 2 * sp + s : sp);
        const long long part = (static_cast<long long>(slot) * M + (DIFF ? s : 0)) * f.rows + prow;
        if (in) {
            if (!f.direct)
                f.lpart[part] = lse2;
            else if (a.lse)
                a.lse[((static_cast<long long>(b) * a.H + h) * M + (DIFF ? s : 0)) * a.Nq + qi] =
                    lse2 * 0.6931471805599453f;
        }
        // Rows go out through shared memory, so that a warp writes whole rows: put() stages 16 bytes of this thread's
        // row, flush() writes the warp's 32 rows to their places (null: none).
        unsigned char* stage = smem + L::OFF_RING + 1024 + (warp - 4) * (32 * D * 4);
        auto put = [&](int at, int row_bytes, int chunk, uint4 v) {
            *reinterpret_cast<uint4*>(stage + at + lane * row_bytes + ((chunk ^ (lane & 3)) << 4)) = v;
        };
        auto flush = [&](int at, auto row_bytes, void* dst) {
            constexpr int RB = decltype(row_bytes)::value, LANES = RB / 16, AT_ONCE = 32 / LANES;
            const unsigned wanted = __ballot_sync(~0u, dst != nullptr);
            const int c = lane % LANES;
#pragma unroll 4
            for (int y = 0; y < LANES; ++y) {
                if (!((wanted >> (y * AT_ONCE)) & ((1u << AT_ONCE) - 1u))) continue;
                const int rr = y * AT_ONCE + lane / LANES;
                char* to = reinterpret_cast<char*>(__shfl_sync(~0u, reinterpret_cast<unsigned long long>(dst), rr));
                const uint4 v = *reinterpret_cast<const uint4*>(stage + at + rr * RB + ((c ^ (rr & 3)) << 4));
                if (to) reinterpret_cast<uint4*>(to)[c] = v;
            }
        };
        if (DIFF && f.direct) {
            // both maps' sums of this row (every product and load is complete: the ring is free), then half of its
            // columns a warpgroup
            xl[s * 128 + r] = l;
            named_bar(1, 256);
            const float l1 = xl[r], l2 = xl[128 + r];
            const float i1 = l1 > 0.f ? 1.f / l1 : 0.f, i2 = l2 > 0.f ? 1.f / l2 : 0.f;
            const float lam = to_f<T>(static_cast<const T*>(a.lam)[h]);
            const bool second = a.out2 != nullptr;
#pragma unroll 1
            for (int x = 0; x < D / 2; x += 32) {
                uint32_t o1[32], o2[32], w1[16], w2[16];
                tmem_ld32(tl + COL_O + s * (D / 2) + x, o1);
                tmem_ld32(tl + COL_O + D + s * (D / 2) + x, o2);
                tmem_ld_wait();
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                    const float a0 = l2 > 0.f ? __uint_as_float(o2[2 * y]) * i2 : 0.f,
                                a1 = l2 > 0.f ? __uint_as_float(o2[2 * y + 1]) * i2 : 0.f,
                                b0_ = l1 > 0.f ? __uint_as_float(o1[2 * y]) * i1 : 0.f,
                                b1_ = l1 > 0.f ? __uint_as_float(o1[2 * y + 1]) * i1 : 0.f;
                    w1[y] = pack2<T>(fmaf(-lam, a0, b0_), fmaf(-lam, a1, b1_));
                    w2[y] = pack2<T>(a0, a1);
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    put(0, D, x / 8 + y, make_uint4(w1[4 * y], w1[4 * y + 1], w1[4 * y + 2], w1[4 * y + 3]));
                    if (second) put(32 * D, D, x / 8 + y, make_uint4(w2[4 * y], w2[4 * y + 1], w2[4 * y + 2], w2[4 * y + 3]));
                }
            }
            __syncwarp();
            const bool write = in && ok;
            flush(0, std::integral_constant<int, D>{}, write ? static_cast<T*>(a.out) + a.os.at(b, h, qi) + s * (D / 2) : nullptr);
            if (second)
                flush(32 * D, std::integral_constant<int, D>{},
                      write ? static_cast<T*>(a.out2) + ((static_cast<long long>(b) * a.H + h) * a.Nq + qi) * D + s * (D / 2)
                            : nullptr);
        } else if (__any_sync(~0u, in && ok && (f.direct || l > 0.f))) {
            const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll 1
            for (int x = 0; x < D; x += 64) {
                uint32_t o[64];
                tmem_ld32(tl + COL_O + s * D + x, *reinterpret_cast<uint32_t(*)[32]>(o));
                tmem_ld32(tl + COL_O + s * D + x + 32, *reinterpret_cast<uint32_t(*)[32]>(o + 32));
                tmem_ld_wait();
#pragma unroll
                for (int y = 0; y < 64; ++y) o[y] = l > 0.f ? __float_as_uint(__uint_as_float(o[y]) * inv) : 0u;
                if (f.direct) {
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        uint32_t w[4];
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            w[z] = pack2<T>(__uint_as_float(o[8 * y + 2 * z]), __uint_as_float(o[8 * y + 2 * z + 1]));
                        put(0, 2 * D, x / 8 + y, make_uint4(w[0], w[1], w[2], w[3]));
                    }
                } else {
#pragma unroll
                    for (int y = 0; y < 16; ++y)
                        put(0, 4 * D, x / 4 + y, make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]));
                }
            }
            __syncwarp();
            if (f.direct)
                flush(0, std::integral_constant<int, 2 * D>{}, in && ok ? static_cast<T*>(a.out) + a.os.at(b, h, qi) : nullptr);
            else      // (a row that saw nothing has no part)
                flush(0, std::integral_constant<int, 4 * D>{}, in && ok && l > 0.f ? f.opart + part * D : nullptr);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8], __nv_bfloat16) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = bf16lo(u[i]), x[2 * i + 1] = bf16hi(u[i]);
}
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8], __half) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = half_lo(u[i]), x[2 * i + 1] = half_hi(u[i]);
}

// Joins the parts of each row, a warp a row: weights 2^(lse_p - max), their sum,
// the weighed mean of the parts' outputs.  A lane takes the log-sum-exps of every
// 32nd part, and the outputs of eight parts are in flight at once (one part after
// the other, 16 parts of 288 rows took 18 us).
template <int D, typename T, bool DIFF>
__global__ void __launch_bounds__(128) dense_merge_kernel(const __grid_constant__ DenseFwdArgs f) {
    constexpr int C = D / 32, M = DIFF ? 2 : 1;
    const DenseArgs& a = f.a;
    const int lane = threadIdx.x & 31;
    const int row = static_cast<int>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= f.rows) return;
    const int per_seq = a.G * a.Nq, lr = row % per_seq, hk = row / per_seq % a.Hk, b = row / per_seq / a.Hk;
    const int qi = lr / a.G, h = hk * a.G + lr % a.G;
    const int slots = f.slots_g + f.slots_b;
    wait_for_previous();
    float o[M][C];
#pragma unroll
    for (int x = 0; x < M; ++x) {
        float mx = -INFINITY, sum = 0.f;
        for (int p = lane; p < slots; p += 32) mx = fmaxf(mx, f.lpart[(static_cast<long long>(p) * M + x) * f.rows + row]);
#pragma unroll
        for (int y = 16; y; y >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, y));
#pragma unroll
        for (int c = 0; c < C; ++c) o[x][c] = 0.f;
        if (mx > -INFINITY) {
            for (int p0 = 0; p0 < slots; p0 += 32) {
                float mine = 0.f;                              // this lane's part's weight, 0 past the last
                if (p0 + lane < slots)
                    mine = fast_exp2(f.lpart[(static_cast<long long>(p0 + lane) * M + x) * f.rows + row] - mx);
                sum += mine;
                for (int y0 = 0; y0 < min(32, slots - p0); y0 += 8) {
                    float w[8];
                    float2 v[8][C / 2];
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        w[y] = __shfl_sync(~0u, mine, y0 + y);
                        const float2* src = reinterpret_cast<const float2*>(
                            f.opart + ((static_cast<long long>(p0 + y0 + y) * M + x) * f.rows + row) * D + lane * C);
#pragma unroll
                        for (int c = 0; c < C / 2; ++c)        // (a part that saw nothing was not written)
                            v[y][c] = w[y] > 0.f ? src[c] : make_float2(0.f, 0.f);
                    }
#pragma unroll
                    for (int y = 0; y < 8; ++y)
#pragma unroll
                        for (int c = 0; c < C / 2; ++c) {
                            o[x][2 * c] = fmaf(w[y], v[y][c].x, o[x][2 * c]);
                            o[x][2 * c + 1] = fmaf(w[y], v[y][c].y, o[x][2 * c + 1]);
                        }
                }
            }
#pragma unroll
            for (int y = 16; y; y >>= 1) sum += __shfl_xor_sync(~0u, sum, y);
            const float inv = 1.f / sum;
#pragma unroll
            for (int c = 0; c < C; ++c) o[x][c] *= inv;
        }
        if (a.lse && lane == 0)
            a.lse[((static_cast<long long>(b) * a.H + h) * M + x) * a.Nq + qi] =
                mx > -INFINITY ? (mx + log2f(sum)) * 0.6931471805599453f : -INFINITY;
    }
    const float lam = DIFF ? to_f<T>(static_cast<const T*>(a.lam)[h]) : 0.f;
    T* op = static_cast<T*>(a.out) + a.os.at(b, h, qi) + lane * C;
    T* o2p = DIFF && a.out2 ? static_cast<T*>(a.out2) + ((static_cast<long long>(b) * a.H + h) * a.Nq + qi) * D + lane * C : nullptr;
#pragma unroll
    for (int c = 0; c < C; c += 2) {
        float v0 = o[0][c], v1 = o[0][c + 1];
        if (DIFF) {
            v0 = fmaf(-lam, o[M - 1][c], v0);
            v1 = fmaf(-lam, o[M - 1][c + 1], v1);
            if (o2p) *reinterpret_cast<uint32_t*>(o2p + c) = pack2<T>(o[M - 1][c], o[M - 1][c + 1]);
        }
        *reinterpret_cast<uint32_t*>(op + c) = pack2<T>(v0, v1);
    }
}

// ------------------------------------------------------------------ gradients
// Rows the gradient kernel streams past its resident tile, and what it reads of
// each query: kDenseRowFloats values for 64 queries, in the order
//   -lse_1 log2 e + shift | -lse_2 log2 e + shift | -delta_1 | -delta_2 | delta_1 - delta_2
// (-inf, 0 for padding and queries that see nothing, whose weights so become 0).
//
// fp16 has 15 powers of two above 1 and 24 below, and weights of 2^-12 times
// gradients of 2^-16 lie below those, so what is packed is scaled by powers of two
// that place its largest possible value between 2^14 and 2^15; the results are
// scaled back in fp32.
//   W = P_1 - lambda P_2 by 2^shift, shift = 14 - max(0, e) with every |lambda| of
//       the heads that share a key below 2^e;
//   dS_1 by 2^sigma, dS_2 (which holds lambda on the key side) by 2^(sigma - e):
//       |P (dP - delta)| <= |dout|_2 |v|_2 + |delta|, largest over what a CTA meets.
// dense_rows_kernel leaves the largest |dout|_2 and |delta| of its 64 queries and the
// largest |v|_2 of 128 keys (a further read of v). With the scales a step of 4 x 1531
// ragged tokens, d = 64, takes 200 us, without 195.5; 2 x 2048, d = 128: 365 and 361.
// bf16 has fp32's range: no scales.
constexpr int kDenseRowTile = 64, kDenseRowFloats = 5 * kDenseRowTile;
template <typename T>
constexpr bool kDenseScaled = std::is_same<T, __half>::value;
// The smallest e with |x| < 2^e (-126 for 0, 129 for no finite x), and 2^e.
__device__ __forceinline__ int exp_above(float x) { return ((__float_as_int(x) >> 23) & 255) - 126; }
__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }
// The largest of a warp's values, none negative (their bits order as they do).
__device__ __forceinline__ float warp_max(float x) {
    return __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(x)));
}
// This lane's largest |lambda| of a group of n heads, and e of the warp's.
template <typename T>
__device__ __forceinline__ float dense_lam_max(const T* lam, int n, int lane) {
    float x = 0.f;
    for (int y = lane; y < n; y += 32) x = fmaxf(x, fabsf(to_f<T>(lam[y])));
    return x;
}
__device__ __forceinline__ int dense_lam_exp(float x) { return min(17, max(-20, exp_above(warp_max(x)))); }
__device__ __forceinline__ int dense_shift(int lam_exp) { return 14 - max(0, lam_exp); }

// For the key side the same values of a tile also lie as an operand of the S and dP
// products, 64 rows of 128 bytes in the 128-byte swizzle: elements 0-2, 16-18 and
// 32-34 of a query's row are -lse_1, -lse_2 (as above, over tau log2 e) and -delta_1
// in three parts of the I/O type each.  One further step of 16 against rows of the
// parts' weights adds them, where reading them from shared memory for every lane
// took 1024 of a tile's 2500 cycles.  bf16: weights 1, the parts hold 24 bits.
// fp16: weights 2^14, 2^3, 2^-8; values to 2^29 (a part's remainder is at most 2^-11
// of it: 2^18 fits 2^3 x 65504, 2^7 fits 2^-8 x 65504), to 2^-33 of 1 or of the value.
constexpr int kDenseExt = 64 * 128;
template <typename T>
__device__ __forceinline__ float dense_ext_weight(int part) {
    if (!std::is_same<T, __half>::value) return 1.f;
    return part == 0 ? 16384.f : part == 1 ? 8.f : 1.f / 256.f;
}

struct DenseBwdArgs {
    DenseArgs a;
    int q_b, q_h, do_b, do_h, k_b, k_h, v_b, v_h;   // 0: that dimension is broadcast in the map
    int key_items, key_tiles, query_tiles;          // CTAs of 128 keys, then CTAs of 128 queries
    int row_tiles;                                  // ceil(Nq / 64)
    float* rowdata;                                 // [B * H][row_tiles][kDenseRowFloats]
    float2* bound;                                  // fp16: [B * H][row_tiles] largest |dout|_2, largest |delta|
    float* vnorm;                                   // fp16: [B * Hk][key_tiles] largest |v|_2
    unsigned char* ext;                             // [B * H][row_tiles][kDenseExt]
    float* dlam_part;                               // [H][B][query_tiles] sums of delta_2
    unsigned* dlam_done;                            // [H] how many of a head's are there
    unsigned long long wait_ns;
    int debug_stall;                                // test hook, as above
};

struct DenseBwdMaps {
    CUtensorMap q, dout, k, v;                      // box 64 x 64 tokens
};

// The per-query values above, from one read of dout, out and out2:
//   delta_2 = dout . out2,  delta_1 = dout . O_1 = dout . out + lambda delta_2.
// out and out2 are rounded to 16 bits, which puts about 0.1% of bf16 gradients'
// size on dq and dk beside the 0.24% of the roundings of dS and of the results.
// (Unrounded deltas take the outputs in 32 bits, which the calls do not pass on, or
// the sum of P dP over all keys before the first dS: another S, dP and exponentials
// of every pair.)
// One CTA a tile of 64 queries of a head, 8 lanes a row; for fp16 then one a tile of
// 128 keys of a key/value head, for its largest |v|_2.
template <int D, typename T>
__global__ void __launch_bounds__(256) dense_rows_kernel(const __grid_constant__ DenseBwdArgs f) {
    const DenseArgs& a = f.a;
    const int lane8 = threadIdx.x & 7, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __shared__ float2 most[8];
    if (kDenseScaled<T> && blockIdx.x >= static_cast<unsigned>(a.B) * a.H * f.row_tiles) {
        const int it = blockIdx.x - static_cast<unsigned>(a.B) * a.H * f.row_tiles;
        const int t = it % f.key_tiles, hk = it / f.key_tiles % a.Hk, b = it / f.key_tiles / a.Hk;
        const int kn = dense_len(a.kv_len, b, a.Nk);
        let_next_start();
        float x = 0.f;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int j = t * 128 + y * 32 + (threadIdx.x >> 3);
            float sq = 0.f;
            if (j < kn) {
                const T* v = static_cast<const T*>(a.v) + a.vs.at(b, hk, j);
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    float e[8];
                    unpack8(__ldg(reinterpret_cast<const uint4*>(v + (c * 8 + lane8) * 8)), e, T{});
#pragma unroll
                    for (int z = 0; z < 8; ++z) sq = fmaf(e[z], e[z], sq);
                }
            }
#pragma unroll
            for (int z = 4; z; z >>= 1) sq += __shfl_xor_sync(~0u, sq, z);
            x = fmaxf(x, sq);
        }
        x = warp_max(x);
        if (lane == 0) most[warp].x = x;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int z = 1; z < 8; ++z) x = fmaxf(x, most[z].x);
            f.vnorm[it] = sqrtf(x);
        }
        return;
    }
    const int t = blockIdx.x % f.row_tiles, bh = blockIdx.x / f.row_tiles, h = bh % a.H, b = bh / a.H;
    const int qn = dense_len(a.q_len, b, a.Nq);
    const float lam = to_f<T>(static_cast<const T*>(a.lam)[h]);
    if (b == 0 && t == 0 && threadIdx.x == 0) f.dlam_done[h] = 0u;
    let_next_start();
    const float lm = kDenseScaled<T> ? dense_lam_max(static_cast<const T*>(a.lam) + h / a.G * a.G, a.G, lane) : 0.f;
    const float shift = kDenseScaled<T> ? static_cast<float>(dense_shift(dense_lam_exp(lm))) : 0.f;
    float top = 0.f, topd = 0.f;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const int c = y * 32 + (threadIdx.x >> 3), i = t * kDenseRowTile + c;
        float d1 = 0.f, d2 = 0.f, sq = 0.f;
        if (i < qn) {
            const T* g = static_cast<const T*>(a.dout) + a.dos.at(b, h, i);
            const T* o = static_cast<const T*>(a.out) + a.os.at(b, h, i);
            const T* o2 = static_cast<const T*>(a.out2) + (static_cast<long long>(bh) * a.Nq + i) * D;
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
                const int at = (x * 8 + lane8) * 8;
                float gv[8], ov[8], o2v[8];
                unpack8(__ldg(reinterpret_cast<const uint4*>(g + at)), gv, T{});
                unpack8(__ldg(reinterpret_cast<const uint4*>(o + at)), ov, T{});
                unpack8(__ldg(reinterpret_cast<const uint4*>(o2 + at)), o2v, T{});
#pragma unroll
                for (int z = 0; z < 8; ++z) {
                    d1 = fmaf(gv[z], ov[z], d1);
                    d2 = fmaf(gv[z], o2v[z], d2);
                    if (kDenseScaled<T>) sq = fmaf(gv[z], gv[z], sq);
                }
            }
        }
#pragma unroll
        for (int x = 4; x; x >>= 1) {
            d1 += __shfl_xor_sync(~0u, d1, x);
            d2 += __shfl_xor_sync(~0u, d2, x);
            if (kDenseScaled<T>) sq += __shfl_xor_sync(~0u, sq, x);
        }
        top = fmaxf(top, sq), topd = fmaxf(topd, fmaxf(fabsf(fmaf(lam, d2, d1)), fabsf(d2)));
        if (lane8 == 0) {
            float l1 = -INFINITY, l2 = -INFINITY;
            if (i < qn) {
                const float* ls = a.lse + static_cast<long long>(bh) * 2 * a.Nq + i;
                l1 = ls[0], l2 = ls[a.Nq];
            }
            const bool some = l1 > -INFINITY;
            float* row = f.rowdata + (static_cast<long long>(bh) * f.row_tiles + t) * kDenseRowFloats + c;
            row[0] = some ? shift - l1 * 1.4426950408889634f : -INFINITY;
            row[64] = some ? shift - l2 * 1.4426950408889634f : -INFINITY;
            row[128] = -fmaf(lam, d2, d1);
            row[192] = -d2;
            row[256] = fmaf(lam, d2, d1) - d2;
            unsigned char* e = f.ext + (static_cast<long long>(bh) * f.row_tiles + t) * kDenseExt;
            const float v[3] = {row[0] / a.scale_log2, row[64] / a.scale_log2, -fmaf(lam, d2, d1)};
            if (kDenseScaled<T> && some && fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fabsf(v[2])) > 536870912.f)
                report(kStatusRange);          // past what the parts hold
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                uint4 w = make_uint4(0, 0, 0, 0);
                if (z < 3) {
                    const float x = v[z];
                    const float w0 = dense_ext_weight<T>(0), w1 = dense_ext_weight<T>(1), w2 = dense_ext_weight<T>(2);
                    const T p0 = from_f<T>(x / w0);
                    const float r1 = isinf(x) ? 0.f : x - to_f<T>(p0) * w0;
                    const T p1 = from_f<T>(r1 / w1);
                    w.x = pack2<T>(to_f<T>(p0), to_f<T>(p1));
                    w.y = pack2<T>((r1 - to_f<T>(p1) * w1) / w2, 0.f);
                }
                *reinterpret_cast<uint4*>(e + sw128(c, 2 * z)) = w;
                *reinterpret_cast<uint4*>(e + sw128(c, 2 * z + 1)) = make_uint4(0, 0, 0, 0);
            }
        }
    }
    if (kDenseScaled<T>) {
        top = warp_max(top), topd = warp_max(topd);
        if (lane == 0) most[warp] = make_float2(top, topd);
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int z = 1; z < 8; ++z) top = fmaxf(top, most[z].x), topd = fmaxf(topd, most[z].y);
            f.bound[blockIdx.x] = make_float2(sqrtf(top), topd);
        }
    }
}

// One CTA holds 128 rows of one side (X, Y) and streams 64-row tiles of the other
// (x, y) past them; S_m and dP are recomputed by each side:
//   keys     X = K, Y = V, x = Q, y = dout:   dv += W^T y,  dk_m += dS_m^T x_m
//   queries  X = Q, Y = dout, x = K, y = V:   dq_m += dS_m x_m
// so no sums cross CTAs and the gradients are the same bits every time.  In both
// the tile is held with the resident row in the tensor-memory lane (for keys
// that is S^T), so W and dS, written by the thread of their row in 16 bits, are
// the A operands of the accumulating products: from tensor memory, but dS_2 of the
// keys for d = 128, whose accumulators leave no columns for it, from shared memory.
//   S_m = X_m x_m^T, dP = Y y^T      tcgen05 M = 128, N = 64
// X and Y are A operands too: for queries they lie in tensor memory beside the
// accumulators, and the products run at full rate (32 cycles a step of 16, where
// both from shared memory, as for keys, take 48: its bandwidth is the bound there,
// with the loads and dS_2; the row values as an operand took 2 x 2048 tokens, d =
// 128, with their forward from 361 to 353 us, 4 x 1531 ragged ones, d = 64, from
// 211 to 203, and K and dS_2 in tensor memory, which d = 64 has room for, to 196).
// S(i+1) is issued once both warpgroups have read S(i) into registers, and runs
// while they form the weights of tile i: a warpgroup takes 32 of the 64 columns.
// The queries also sum P_2 (.) dP, which is delta_2 without the rounding of out2:
// dlambda needs it, a sum of both signs in which those roundings would show.
// Warps: w0 TMA producer, w1 issuer of S and dP, w2 issuer of the accumulating
// products (an issue blocks until the tensor core takes it, so waits of the one
// overlap issues of the other), w4-11 two warpgroups.
template <int D>
struct DenseBwdLayout {
    static constexpr int RBOX = 128 * 128, SBOX = 64 * 128;   // 64 columns of 128 / 64 rows
    static constexpr int RES = 128 * D * 2;                    // a resident tile
    static constexpr int STR = 64 * D * 2;                     // a streamed tile
    static constexpr int STAGE = 2 * STR + kDenseExt + 1024;   // x, y, keys: the rows' values as an operand and as such
    static constexpr int SLOTS = D == 128 ? 3 : 5;
    static constexpr int OFF_DS2 = 2 * RES;                    // keys: dS_2, 128 rows of 64 values
    static constexpr int OFF_ONE = OFF_DS2 + 16384;            // keys: 128 rows of 128 bytes, the parts' weights, zeros
    static constexpr int OFF_RING = OFF_ONE + 16384;
    static constexpr int OFF_MISC = OFF_RING + SLOTS * STAGE;
    static constexpr int SMEM = 1024 + OFF_MISC + 256;
    static_assert(SMEM <= 232448, "shared memory of an SM");
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

template <int D, typename T, bool KEYS>
__device__ __forceinline__ void dense_bwd_cta(const DenseBwdMaps& tm, const DenseBwdArgs& f, unsigned char* smem,
                                              int item) {
    using L = DenseBwdLayout<D>;
    constexpr int NBOX = D / 64, SLOTS = L::SLOTS;
    // tensor memory: S_1 | S_2 | dP | W (keys) or dS_2 | dS_1 | accumulators (| queries: Q, dout)
    constexpr uint32_t COL_DP = 128, COL_W = 192, COL_DS1 = 224, COL_ACC = 256, COL_X = 384, COL_Y = 448;
    // accumulators: keys dv first; then dk or dq: for d = 128 one of D columns (map m in its half), for d = 64
    // one for each map over all 64 columns of x, of which its half is the result (N = 64 either way)
    constexpr uint32_t COL_G = COL_ACC + (KEYS ? D : 0);
    // d = 64 leaves the keys columns behind their accumulators: for dS_2, and for K, then the A operand of S
    constexpr bool ROOM = KEYS && D == 64;
    constexpr uint32_t COL_DS2 = KEYS ? 448 : COL_W, COL_K = 480;
    const uint32_t sbase = smem_u32(smem);
    const DenseArgs& a = f.a;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::OFF_MISC);   // [SLOTS]
    uint64_t* empty = full + SLOTS;                                     // [SLOTS]
    uint64_t* r_full = empty + SLOTS;     // resident tiles
    uint64_t* s_full = r_full + 1;        // S, dP of a tile
    uint64_t* s_free = s_full + 1;        // read by the warpgroups
    uint64_t* p_full = s_free + 1;        // W, dS written
    uint64_t* p_free = p_full + 1;        // and consumed
    uint64_t* end_bar = p_free + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(end_bar + 1);
    volatile int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
    float* part = reinterpret_cast<float*>(smem + L::OFF_RING);         // [8] after the last product

    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
    const int tiles = KEYS ? f.key_tiles : f.query_tiles, heads = KEYS ? a.Hk : a.H;
    // the tiles with the most visible partners first: early keys, late queries
    const int tile = KEYS ? item % tiles : tiles - 1 - item % tiles;
    const int hr = item / tiles % heads, b = item / tiles / heads;
    const int hk = KEYS ? hr : hr / a.G;
    const int row0 = tile * 128;
    const int q_raw = a.q_len ? a.q_len[b] : a.Nq, k_raw = a.kv_len ? a.kv_len[b] : a.Nk;
    const int qn = dense_len_in(q_raw, a.Nq), kn = dense_len_in(k_raw, a.Nk), off = kn - qn;
    int t0 = 0, per = 0;                  // streamed tiles [t0, t0 + per) of each head
    if (KEYS) {
        if (row0 < kn) {
            const int first = a.causal ? max(0, row0 - off) : 0;
            t0 = first / 64;
            per = max(0, (qn + 63) / 64 - t0);
        }
    } else if (row0 < qn) {
        per = (dense_own(min(row0 + 127, qn - 1), qn, kn, a.causal) + 63) / 64;
    }
    const int n = per * (KEYS ? a.G : 1);
    // the streamed tile that holds rows past the sequence's length
    const int slen = KEYS ? qn : kn;
    const int dirty = slen < (KEYS ? a.Nq : a.Nk) && slen % 64 != 0 ? slen / 64 : -1;

    if (tid == 0) {
        for (int s = 0; s < SLOTS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(r_full, ROOM ? 5 : KEYS ? 1 : 8);
        mbar_init(s_full, 1);
        mbar_init(s_free, 8);
        mbar_init(p_full, 8);
        mbar_init(p_free, 1);
        mbar_init(end_bar, 2);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (KEYS) {
        for (int x = tid; x < 1024; x += kDenseThreads) {
            const uint32_t w = pack2<T>(dense_ext_weight<T>(0), dense_ext_weight<T>(1)), w2 = pack2<T>(dense_ext_weight<T>(2), 0.f);
            *reinterpret_cast<uint4*>(smem + L::OFF_ONE + sw128(x >> 3, x & 7)) =
                x & 7 ? make_uint4(0, 0, 0, 0) : make_uint4(w, w2, 0, 0);
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    wait_for_previous();                  // the row values
    const uint32_t tmem = *tmem_slot;
    const unsigned long long lim = f.wait_ns;
    auto fail = [&]() {
        *abort_flag = 1;
        report(kStatusTimeout);
    };
    auto wait = [&](uint64_t* bar, uint32_t par) { return warp_wait(bar, par, abort_flag, lim); };

    if (warp == 0) {
        // ==================================================== producer (the whole warp waits, one lane issues)
        const bool leader = elect_one();
        const CUtensorMap *mx = KEYS ? &tm.q : &tm.k, *my = KEYS ? &tm.dout : &tm.v;
        const int n_load = f.debug_stall ? 0 : n;
        if (KEYS && n_load > 0 && leader) {
            mbar_arrive_expect_tx(r_full, (ROOM ? 1 : 2) * L::RES);
            for (int c = 0; c < NBOX; ++c)
                for (int z = 0; z < 2; ++z) {
                    if (!ROOM)
                        tma_load_4d(smem + c * L::RBOX + z * L::SBOX, &tm.k, r_full, c * 64, row0 + z * 64, hr * f.k_h,
                                    b * f.k_b);
                    tma_load_4d(smem + L::RES + c * L::RBOX + z * L::SBOX, &tm.v, r_full, c * 64, row0 + z * 64,
                                hr * f.v_h, b * f.v_b);
                }
        }
        __syncwarp();
        const int xb = b * (KEYS ? f.q_b : f.k_b), yb = b * (KEYS ? f.do_b : f.v_b);
        RingPos<SLOTS> rp{0, 1u};           // (phase of the wait for an empty slot: the first round passes)
        bool ok = true;
        int i = 0, t = t0, h = KEYS ? hr * a.G : hk;
        for (; i < n_load; ++i) {
            if (!(ok = wait(&empty[rp.slot], rp.phase))) break;
            if (leader) {
                unsigned char* st = smem + L::OFF_RING + rp.slot * L::STAGE;
                uint64_t* bar = &full[rp.slot];
                mbar_arrive_expect_tx(bar, 2 * L::STR + (KEYS ? kDenseExt + 256 : 0));
                const int xh = h * (KEYS ? f.q_h : f.k_h), yh = h * (KEYS ? f.do_h : f.v_h);
                for (int c = 0; c < NBOX; ++c) {
                    tma_load_4d(st + c * L::SBOX, mx, bar, c * 64, t * 64, xh, xb);
                    tma_load_4d(st + L::STR + c * L::SBOX, my, bar, c * 64, t * 64, yh, yb);
                }
                if (KEYS) {
                    const long long at = (static_cast<long long>(b) * a.H + h) * f.row_tiles + t;
                    bulk_load(st + 2 * L::STR, f.ext + at * kDenseExt, kDenseExt, bar);
                    bulk_load(st + 2 * L::STR + kDenseExt, f.rowdata + at * kDenseRowFloats + 256, 256, bar);
                }
            }
            __syncwarp();
            rp.step(1);
            if (++t == t0 + per) t = t0, ++h;
        }
        if (!ok) fail();
        // every load has landed before the CTA exits
        if (KEYS && n_load > 0) mbar_drain(r_full, 0, abort_flag);   // (with the warps' own arrivals)
        for (int y = max(0, i - SLOTS); y < i; ++y) mbar_drain(&full[y % SLOTS], (y / SLOTS) & 1, abort_flag);
    } else if (warp == 1) {
        // ==================================================== issuer of S and dP
        constexpr uint32_t ID_S = idesc_t<T>(128, 64, 0, 0);
        constexpr int STEPS = D / 32;
        const bool leader = elect_one();
        const uint64_t X0 = sdesc(sbase, 16, 1024, kSwizzle128B), Y0 = sdesc(sbase + L::RES, 16, 1024, kSwizzle128B),
                       x0 = sdesc(sbase + L::OFF_RING, 16, 1024, kSwizzle128B),
                       one = sdesc(sbase + L::OFF_ONE, 16, 1024, kSwizzle128B);
        RingPos<SLOTS> rp{0, 0u};
        bool ok = n == 0 || wait(r_full, 0);
        for (int i = 0; ok && i < n; ++i) {
            if (!(ok = wait(&full[rp.slot], rp.phase))) break;
            if (i > 0 && !(ok = wait(s_free, (i - 1) & 1))) break;
            tc_fence_after();
            if (leader) {
                const uint64_t xd = x0 + rp.slot * (L::STAGE >> 4), yd = xd + (L::STR >> 4), ed = yd + (L::STR >> 4);
#pragma unroll
                for (int kk = 0; kk < 2 * STEPS; ++kk) {
                    const uint64_t bd = xd + (((kk >> 2) * L::SBOX + (kk & 3) * 32) >> 4);
                    if (KEYS && !ROOM)
                        umma_f16_ss(tmem + (kk / STEPS) * 64, X0 + (((kk >> 2) * L::RBOX + (kk & 3) * 32) >> 4), bd, ID_S,
                                    kk % STEPS ? 1u : 0u);
                    else
                        umma_f16_ts(tmem + (kk / STEPS) * 64, tmem + (KEYS ? COL_K : COL_X) + kk * 8, bd, ID_S,
                                    kk % STEPS ? 1u : 0u);
                }
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint64_t bd = yd + (((kk >> 2) * L::SBOX + (kk & 3) * 32) >> 4);
                    if (KEYS)
                        umma_f16_ss(tmem + COL_DP, Y0 + (((kk >> 2) * L::RBOX + (kk & 3) * 32) >> 4), bd, ID_S, kk ? 1u : 0u);
                    else
                        umma_f16_ts(tmem + COL_DP, tmem + COL_Y + kk * 8, bd, ID_S, kk ? 1u : 0u);
                }
                if (KEYS)      // - lse_1, - lse_2, - delta_1 of the columns
#pragma unroll
                    for (int z = 0; z < 3; ++z) umma_f16_ss(tmem + z * 64, one, ed + z * 2, ID_S, 1u);
                umma_commit(s_full);
            }
            __syncwarp();
            rp.step(1);
        }
        if (!ok) fail();
        if (leader) umma_commit(end_bar);      // also: every MMA has completed before tensor memory is released
        mbar_drain(end_bar, 0, abort_flag);
    } else if (warp == 2) {
        // ==================================================== issuer of the accumulating products
        constexpr uint32_t ID_V = idesc_t<T>(128, D, 0, 1), ID_G = idesc_t<T>(128, 64, 0, 1);
        const bool leader = elect_one();
        const uint64_t x0 = sdesc(sbase + L::OFF_RING, L::SBOX, 1024, kSwizzle128B),
                       ds2 = sdesc(sbase + L::OFF_DS2, 16, 1024, kSwizzle128B);
        RingPos<SLOTS> rp{0, 0u};
        bool ok = true;
        for (int i = 0; ok && i < n; ++i) {
            if (!(ok = wait(&full[rp.slot], rp.phase)) || !(ok = wait(p_full, i & 1))) break;
            tc_fence_after();
            if (leader) {
                const uint64_t xd = x0 + rp.slot * (L::STAGE >> 4), yd = xd + (L::STR >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t acc = i > 0 || k > 0 ? 1u : 0u;
                    const uint64_t x1 = xd + ((k * 2048) >> 4), x2 = x1 + (D == 128 ? L::SBOX >> 4 : 0);
                    if (KEYS) umma_f16_ts(tmem + COL_ACC, tmem + COL_W + k * 8, yd + ((k * 2048) >> 4), ID_V, acc);
                    umma_f16_ts(tmem + COL_G, tmem + COL_DS1 + k * 8, x1, ID_G, acc);
                    if (KEYS && !ROOM)
                        umma_f16_ss(tmem + COL_G + 64, ds2 + ((k * 32) >> 4), x2, ID_G, acc);
                    else
                        umma_f16_ts(tmem + COL_G + 64, tmem + COL_DS2 + k * 8, x2, ID_G, acc);
                }
                umma_commit(p_free);
                umma_commit(&empty[rp.slot]);
            }
            __syncwarp();
            rp.step(1);
        }
        if (!ok) fail();
        if (leader) umma_commit(end_bar);
        mbar_drain(end_bar, 0, abort_flag);
    } else if (warp >= 4) {
        // ==================================================== warpgroups
        const int q4 = warp & 3, w = (warp - 4) >> 2, r = q4 * 32 + lane;
        const uint32_t tl = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
        const int row = row0 + r;
        // what the scales come from, asked for before the resident rows (after them: 205 us a step of 4 x 1531 ragged
        // tokens, d = 64, against 200)
        float dn = 0.f, dl = 0.f, vn = 0.f, lm = 0.f;
        if (kDenseScaled<T> && n > 0) {
            lm = dense_lam_max(static_cast<const T*>(a.lam) + hk * a.G, a.G, lane);
            if (KEYS) {
                vn = f.vnorm[(static_cast<long long>(b) * a.Hk + hr) * f.key_tiles + tile];
#pragma unroll 4
                for (int y = lane; y < n; y += 32) {
                    const float2 x = f.bound[(static_cast<long long>(b) * a.H + hr * a.G + y / per) * f.row_tiles + t0 + y % per];
                    dn = fmaxf(dn, x.x), dl = fmaxf(dl, x.y);
                }
            } else {
                const int y = row0 / kDenseRowTile + (lane & 1);
                if (y < f.row_tiles) {
                    const float2 x = f.bound[(static_cast<long long>(b) * a.H + hr) * f.row_tiles + y];
                    dn = x.x, dl = x.y;
                }
                const float* p = f.vnorm + (static_cast<long long>(b) * a.Hk + hk) * f.key_tiles;
#pragma unroll 4
                for (int z = lane; z < (per + 1) / 2; z += 32) vn = fmaxf(vn, p[z]);
            }
        }
        if ((ROOM ? w == 0 : !KEYS) && n > 0) {
            // the resident rows to tensor memory: queries (w = 0) and dout (w = 1), or keys; zeros for padding
            const bool have = row < (KEYS ? kn : qn);
            const T* src = static_cast<const T*>(KEYS ? a.k : w ? a.dout : a.q) +
                           (!have ? 0 : KEYS ? a.ks.at(b, hr, row) : w ? a.dos.at(b, hr, row) : a.qs.at(b, hr, row));
#pragma unroll
            for (int x = 0; x < NBOX; ++x) {
                uint32_t v[32];
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    const uint4 u = have ? __ldg(reinterpret_cast<const uint4*>(src + x * 64) + y) : make_uint4(0, 0, 0, 0);
                    v[4 * y] = u.x, v[4 * y + 1] = u.y, v[4 * y + 2] = u.z, v[4 * y + 3] = u.w;
                }
                tmem_st32(tl + (KEYS ? COL_K : w ? COL_Y : COL_X) + x * 32, v);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(r_full);
        }
        const float c = a.scale_log2;
        const T* lams = static_cast<const T*>(a.lam) + (KEYS ? hr * a.G : hr);
        // the weights' scale 2^shift, and those of dS_1 and dS_2 (queries: one for both, lambda comes in the end)
        int shift = 0, up1 = 0, up2 = 0;
        if (kDenseScaled<T> && n > 0) {
            const int e = dense_lam_exp(lm);
            shift = dense_shift(e);
            up1 = min(60, max(-60, 15 - exp_above(fmaf(warp_max(dn), warp_max(vn), warp_max(dl)))));
            up2 = KEYS ? up1 - e : up1;
        }
        const float un1 = exp2_int(up1 - shift), un2 = exp2_int(up2 - shift);
        const uint64_t c2 = f2pack(c, c), un12 = f2pack(un1, un1), un22 = f2pack(un2, un2);
        uint64_t nl1 = 0, nl2 = 0, nd1 = 0, nd2 = 0;          // queries: this row's values
        if (!KEYS && n > 0) {
            const int t = row >> 6;
            const bool have = t < f.row_tiles;
            const float* rd = f.rowdata + ((static_cast<long long>(b) * a.H + hr) * f.row_tiles + (have ? t : 0)) *
                                              kDenseRowFloats + (row & 63);
            const float v0 = have ? rd[0] : -INFINITY, v1 = have ? rd[64] : -INFINITY, v2 = have ? rd[128] : 0.f,
                        v3 = have ? rd[192] : 0.f;
            nl1 = f2pack(v0, v0), nl2 = f2pack(v1, v1);
            nd1 = f2pack(v2 * un1, v2 * un1), nd2 = f2pack(v3 * un1, v3 * un1);
        }
        const int own = dense_own(row, qn, kn, a.causal);     // queries
        float lam = to_f<T>(lams[0]);
        uint64_t delta2 = 0;                                  // queries: the sum of P_2 dP, scaled as P
        RingPos<SLOTS> rp{0, 0u};
        bool ok = true;
        int t = t0;
        for (int i = 0; i < n; ++i) {
            // (keys: this thread reads the tile's row values itself, so it also waits for their load)
            ok = ok && wait(s_full, i & 1) && (!KEYS || wait(&full[rp.slot], rp.phase));
            uint32_t s1[32], s2[32], dp[32];
            if (ok) {
                tc_fence_after();
                tmem_ld32(tl + w * 32, s1);
                tmem_ld32(tl + 64 + w * 32, s2);
                tmem_ld32(tl + COL_DP + w * 32, dp);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free);
            }
            if (!ok) break;
            const int base = t * 64 + w * 32;
            // columns [lo, hi) count; the others may hold anything
            const int lo = KEYS && a.causal ? row - off - base : 0;
            const int hi = KEYS ? (t == dirty ? qn - base : 32) : own - base;
            if (__any_sync(~0u, lo > 0 || hi < 32)) {
#pragma unroll
                for (int x = 0; x < 32; ++x)
                    if (x < lo || x >= hi) {
                        s1[x] = s2[x] = 0xFF800000u;          // -inf: weight 0
                        dp[x] = 0u;
                    }
            }
            const uint64_t nlam2 = f2pack(-lam, -lam);
            unsigned char* st = smem + L::OFF_RING + rp.slot * L::STAGE;
            // keys: S and dP hold - lse and - delta_1 already; delta_1 - delta_2 of the columns is read here
            const float* rd = reinterpret_cast<const float*>(st + 2 * L::STR + kDenseExt) + w * 32;
            uint32_t ww[16], d1[16], d2[16];
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                uint64_t dd[2] = {0, 0};
                if (KEYS) {
                    const ulonglong2 u1 = *reinterpret_cast<const ulonglong2*>(rd + 4 * x);
                    dd[0] = u1.x, dd[1] = u1.y;
                }
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const int y = 2 * x + z, k = 2 * y;
                    float u, v;
                    const uint64_t z1 = f2pack(__uint_as_float(s1[k]), __uint_as_float(s1[k + 1])),
                                   z2 = f2pack(__uint_as_float(s2[k]), __uint_as_float(s2[k + 1])),
                                   g = f2pack(__uint_as_float(dp[k]), __uint_as_float(dp[k + 1]));
                    if (KEYS) {
                        const uint64_t p1 = exp2_2(fmul2(z1, c2)), p2 = fmul2(exp2_2(fmul2(z2, c2)), nlam2);   // P_1, -lambda P_2
                        uint64_t w1 = fmul2(p1, g), w2 = fmul2(p2, fadd2(g, dd[z]));
                        if (kDenseScaled<T>) w1 = fmul2(w1, un12), w2 = fmul2(w2, un22);
                        f2unpack(w1, u, v);
                        d1[y] = pack2<T>(u, v);
                        f2unpack(w2, u, v);
                        d2[y] = pack2<T>(u, v);
                        f2unpack(fadd2(p1, p2), u, v);
                        ww[y] = pack2<T>(u, v);
                    } else {                                           // (dq_2 takes -lambda in the end)
                        const uint64_t p1 = exp2_2(ffma2(z1, c2, nl1)), p2 = exp2_2(ffma2(z2, c2, nl2));
                        delta2 = ffma2(p2, g, delta2);
                        f2unpack(fmul2(p1, kDenseScaled<T> ? ffma2(g, un12, nd1) : fadd2(g, nd1)), u, v);
                        d1[y] = pack2<T>(u, v);
                        f2unpack(fmul2(p2, kDenseScaled<T> ? ffma2(g, un12, nd2) : fadd2(g, nd2)), u, v);
                        d2[y] = pack2<T>(u, v);
                    }
                }
            }
            // the last tile's products have read W and dS
            if (i > 0) {
                if (!(ok = wait(p_free, (i - 1) & 1))) break;
                tc_fence_after();
            }
            tmem_st16(tl + COL_DS1 + w * 16, d1);
            if (KEYS) tmem_st16(tl + COL_W + w * 16, ww);
            if (KEYS && !ROOM) {
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    *reinterpret_cast<uint4*>(smem + L::OFF_DS2 + sw128(r, w * 4 + y)) =
                        make_uint4(d2[4 * y], d2[4 * y + 1], d2[4 * y + 2], d2[4 * y + 3]);
            } else {
                tmem_st16(tl + COL_DS2 + w * 16, d2);
            }
            if (t == dirty) {      // rows past the length to zero: they are B operands of the products below
                if (!KEYS && !(ok = wait(&full[rp.slot], rp.phase))) break;
                const int rz = slen % 64;
                for (int y = w * 128 + r; y < (64 - rz) * 8; y += 256)
#pragma unroll
                    for (int bx = 0; bx < 2 * NBOX; ++bx)
                        *reinterpret_cast<uint4*>(st + bx * L::SBOX + rz * 128 + y * 16) = make_uint4(0, 0, 0, 0);
            }
            if ((KEYS && !ROOM) || t == dirty) fence_proxy_async_smem();
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);
            rp.step(1);
            if (++t == t0 + per) {
                t = t0;
                if (KEYS && i + 1 < n) lam = to_f<T>(*++lams);
            }
        }
        if (!ok) fail();
        ok = wait(end_bar, 0) && ok;
        tc_fence_after();
        // ---------------------------------------------------- results: keys dv (w = 0) and dk (w = 1), queries halves of dq
        const bool in = row < (KEYS ? a.Nk : a.Nq), some = n > 0 && row < (KEYS ? kn : qn);
        const int x0 = KEYS ? 0 : w * (D / 2), x1 = KEYS ? D : x0 + D / 2;
        const bool is_v = KEYS && w == 0;
        // (w = 1 of the queries holds the second map's half)
        const float unshift = exp2_int(-shift), down1 = a.scale * exp2_int(-up1), down2 = a.scale * exp2_int(-up2);
        T* dst = static_cast<T*>(KEYS ? (is_v ? a.dv : a.dk) : a.dq) +
                 (in ? (KEYS ? (is_v ? a.dvs.at(b, hr, row) : a.dks.at(b, hr, row)) : a.dqs.at(b, hr, row)) : 0);
#pragma unroll 1
        for (int x = x0; x < x1; x += 32) {
            uint32_t o[32];
            const float k = is_v ? unshift : !KEYS ? (w == 1 ? -lam * down1 : down1) : x < D / 2 ? down1 : down2;
            // d = 64: the second map's half lies in its own accumulator
            tmem_ld32(tl + (is_v ? COL_ACC : COL_G + (D == 64 && x >= 32 ? 64 : 0)) + x, o);
            tmem_ld_wait();
            if (in && ok)
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    uint32_t u[4];
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        u[z] = some ? pack2<T>(__uint_as_float(o[8 * y + 2 * z]) * k, __uint_as_float(o[8 * y + 2 * z + 1]) * k)
                                    : 0u;
                    reinterpret_cast<uint4*>(dst + x)[y] = make_uint4(u[0], u[1], u[2], u[3]);
                }
        }
        if (!KEYS) {
            // delta_2 of the CTA's rows, its place among the head's, and the head's sum from whoever is last: the
            // places are added in one order
            float u, v;
            f2unpack(delta2, u, v);
            float s = some ? (u + v) * unshift : 0.f;
#pragma unroll
            for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
            if (lane == 0) part[warp - 4] = s;
            named_bar(1, 256);
            if (warp == 4) {
                const long long places = static_cast<long long>(a.B) * f.query_tiles;
                float* mine = f.dlam_part + hr * places;
                unsigned before = 0u;
                if (lane == 0) {
                    float sum = 0.f;
                    for (int x = 0; x < 8; ++x) sum += part[x];
                    mine[static_cast<long long>(b) * f.query_tiles + tile] = sum;
                    __threadfence();
                    before = atomicAdd(&f.dlam_done[hr], 1u);
                }
                if (__shfl_sync(~0u, before, 0) == places - 1) {
                    __threadfence();
                    double sum = 0.0;
                    for (long long x = lane; x < places; x += 32) sum += __ldcg(mine + x);
#pragma unroll
                    for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(~0u, sum, x);
                    if (lane == 0) static_cast<T*>(a.dlam)[hr] = from_f<T>(static_cast<float>(-sum));
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int D, typename T>
__global__ void __launch_bounds__(kDenseThreads, 1)
    dense_bwd_kernel(const __grid_constant__ DenseBwdMaps tm, const __grid_constant__ DenseBwdArgs f) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    if (static_cast<int>(blockIdx.x) < f.key_items)
        dense_bwd_cta<D, T, true>(tm, f, smem, blockIdx.x);
    else
        dense_bwd_cta<D, T, false>(tm, f, smem, blockIdx.x - f.key_items);
}

}  // namespace sla

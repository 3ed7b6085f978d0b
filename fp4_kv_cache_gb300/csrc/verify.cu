// verify.cu -- csa2d_tree_verify: which drafted tokens stay, and the token behind them.
//
// A cluster of CTAs takes a request.  Every CTA goes down the tree for itself, on the same numbers:
// the drafts' own probabilities p(x) and q(x) are fetched for all nodes at once, so that a node that is
// accepted costs no further load.  Only where a draft is turned down, or at the end, is a row of the
// vocabulary read: the cluster shares it out, each warp sums the weights of a run of tokens, and the
// CTAs tell one another their sums.  With c and m as in csa2_draft.h, what is left after k rejections
// is max(p - c q, 0) / m of the rows themselves, so nothing is written between the rejections.
//
// Weights are summed as whole numbers of 2^-40, so that neither the order nor the number of CTAs
// decides about a token.  A weight w is taken apart without 64-bit conversions (which run at a fraction
// of the rate here): h = w 2^20 rounded to a whole number, and the rest times 2^20, rounded; adding
// 1.5 2^23 leaves either number in the low bits of a float.  h 2^20 + rest is w 2^40 rounded, ties to
// even, since h 2^20 is even.  Two weights go through this at a time (add, multiply and fma of two
// floats are one instruction here); what has to be looked at one by one -- values below 0, above 1 or
// not finite -- is found by the largest bit pattern of a load.
//
// What bounds it: each rejection is a pass over a row of the vocabulary that needs the pass before, so the
// request with most of them sets the time (64 trees of up to 16 nodes over 131,072 float32 tokens 26.6 us, of
// which 9.9 are their last rows at the copy rate; half the warps' time is waiting for loads and barriers
// by profile); one chain of six 10.2 us.  Behind the last pass one warp looks for the token, a load, a scan
// and a branch at a time through its run: the same calls with r = 0, where the first turn finds it, take 22.0 and
// 9.8 us, with r = 1, where the last one does, 28.7 and 12.3.  Weights one at a time, with 64-bit bookkeeping
// of what is not finite, took 35.5 and 12.3.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "draft.cuh"
#include "internal.h"

namespace csa2 {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kMaxCtas = 8;
constexpr int kMaxNodes = 32 * CSA2D_MAX_WORDS;
constexpr float kMagic = 12582912.0f;               // 1.5 x 2^23
// A lane's part of a run stays below 2^11 weights, so that its 32-bit sums hold: the vocabulary over
// one CTA's warps and lanes, and the loads that a last round makes too many.
static_assert(CSA2D_MAX_VOCAB / kThreads + 64 < 2048, "sums of a lane");

__device__ __forceinline__ float value(float v) { return v; }
__device__ __forceinline__ float value(__half v) { return __half2float(v); }
__device__ __forceinline__ float value(__nv_bfloat16 v) { return __bfloat162float(v); }

// A probability as it counts: 0 where it is below 0 or not finite.
__device__ __forceinline__ float clean(float v, bool &bad)
{
    const bool fine = v >= 0.0f && v < INFINITY;
    bad |= !fine;
    return fine ? v : 0.0f;
}
// What is left of p: max(p - c q, 0), at most 1.
__device__ __forceinline__ float rest_of(float p, float q, float c) { return fminf(fmaxf(__fsub_rn(p, __fmul_rn(c, q)), 0.0f), 1.0f); }

// Two floats, each operation rounded once for either.
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ void apart(uint64_t v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t v;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}

struct Sum {
    uint32_t high, low;                     // with the offsets of kMagic still in them
};
__device__ __forceinline__ void add(Sum &s, float w)
{
    const float t = __fmul_rn(w, 1048576.0f), h = __fadd_rn(t, kMagic);
    const float l = __fmaf_rn(__fsub_rn(t, __fsub_rn(h, kMagic)), 1048576.0f, kMagic);
    s.high += __float_as_uint(h);
    s.low += __float_as_uint(l);
}
// The same for two weights.
__device__ __forceinline__ void add(Sum &s, float w0, float w1)
{
    const uint64_t k20 = pair(1048576.0f, 1048576.0f), magic = pair(kMagic, kMagic), back = pair(-kMagic, -kMagic), minus = pair(-1.0f, -1.0f);
    const uint64_t t = mul2(pair(w0, w1), k20), h = add2(t, magic);
    const uint64_t l = fma2(fma2(add2(h, back), minus, t), k20, magic);       // t - (h - magic), exact
    float a, b, c, d;
    apart(h, a, b);
    apart(l, c, d);
    s.high += __float_as_uint(a) + __float_as_uint(b);
    s.low += __float_as_uint(c) + __float_as_uint(d);
}
__device__ __forceinline__ int64_t whole(const Sum &s, uint32_t n)
{
    const uint32_t off = n * 0x4b400000u;
    return (int64_t)(int32_t)(s.high - off) * 1048576 + (int32_t)(s.low - off);
}
__device__ __forceinline__ int64_t whole(float w)
{
    Sum s{0, 0};
    add(s, w);
    return whole(s, 1);
}
__device__ __forceinline__ int64_t warp_sum(int64_t v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void to_peer(int64_t *p, uint32_t rank, int64_t v)
{
    uint32_t at = (uint32_t)__cvta_generic_to_shared(p);
    asm volatile("mapa.shared::cluster.u32 %0, %0, %1;\n\tst.shared::cluster.b64 [%0], %2;" : "+r"(at) : "r"(rank), "l"(v) : "memory");
}

// N values of a row, as floats.
template <typename T, int N>
__device__ __forceinline__ void load_values(const T *from, float (&v)[N])
{
    if constexpr (N == 1) {
        v[0] = value(*from);
    } else {
        const uint4 raw = *reinterpret_cast<const uint4 *>(from);
        const T *t = reinterpret_cast<const T *>(&raw);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = value(t[i]);
    }
}

struct VerifySmem {
    int32_t parent[kMaxNodes], token[kMaxNodes], path[kMaxNodes];
    float u[kMaxNodes], p[kMaxNodes], q[kMaxNodes];      // the number given, p and q of the node's token at its parent
    uint32_t again[CSA2D_MAX_WORDS];                      // nodes whose token an earlier child of the same parent has
    int64_t warp[kWarps], cta[2][kMaxCtas];
};

// VEC: values a load; more than one where rows begin on 16 bytes.
template <typename T, bool DRAWN, int VEC>
__global__ void __launch_bounds__(kThreads) tree_verify_kernel(const csa2d_verify_args P, const int ctas, uint32_t *d_status)
{
    __shared__ VerifySmem M;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = ctas > 1 ? (int)cluster_rank() : 0, b = blockIdx.x / ctas;
    if (ctas > 1) cluster_arrive();                       // waited for before a peer is written to
    pdl_wait();
    pdl_allow_dependents();
    const T *all_p = static_cast<const T *>(P.p), *all_q = static_cast<const T *>(P.q);
    const int64_t c0 = P.cu[b], n64 = P.cu[b + 1] - c0;
    uint32_t flags = 0;
    auto leave_out = [&] {
        if (ctas > 1) cluster_wait();
        if (rank > 0) return;
        for (int i = tid; i < P.max_path; i += kThreads) P.path[(int64_t)b * P.max_path + i] = -1;
        if (tid == 0) {
            P.keep[b] = 0;
            P.next_token[b] = -1;
            P.delta[b] = P.pos && n64 > 0 ? -(int32_t)min(n64, (int64_t)INT32_MAX) : 0;
            if (n64 > 0) dev_flag(d_status, CSA2_DEV_BAD_INDEX);
        }
    };
    if (n64 <= 0 || c0 < 0 || c0 + n64 > P.n_tokens || n64 > kMaxNodes) {
        leave_out();
        return;
    }
    const int32_t root = P.pos ? P.pos[c0] : 0;           // looked at once the nodes have been read
    const int n = (int)n64;
    if (tid < CSA2D_MAX_WORDS) M.again[tid] = 0u;
    for (int i = tid; i < n; i += kThreads) {
        int32_t up = -1, x = -1;
        float u = 0.0f, p = 0.0f, q = 0.0f;
        if (i > 0) {
            up = P.parent[c0 + i];
            x = P.token[c0 + i];
            u = P.u[c0 + i];
            if (up < -1 || up >= i) {
                flags |= CSA2_DEV_BAD_INDEX;
                up = -1;
            }
            if (up >= 0 && x >= 0 && x < P.vocab) {
                p = value(all_p[(c0 + up) * P.p_row + x]);
                if (DRAWN) q = value(all_q[(c0 + up) * P.q_row + x]);
            }
        }
        M.parent[i] = up;
        M.token[i] = x;
        M.u[i] = u;
        M.p[i] = p;
        M.q[i] = q;
    }
    if (root < 0) {
        leave_out();
        return;
    }
    __syncthreads();
    if (!DRAWN) {
        for (int i = tid; i < n; i += kThreads) {
            bool is = false;
            for (int k = 1; k < i; ++k) is |= M.parent[k] == M.parent[i] && M.token[k] == M.token[i];
            if (is) atomicOr(&M.again[i >> 5], 1u << (i & 31));
        }
        __syncthreads();
    }
    if (ctas > 1) cluster_wait();

    // this warp's run of tokens: whole loads of a warp, but for the vocabulary's end
    const int64_t per = ((int64_t)P.vocab + ctas * kWarps - 1) / (ctas * kWarps);
    const int64_t run = (per + 32 * VEC - 1) / (32 * VEC) * (32 * VEC);
    const int32_t x0 = (int32_t)min((rank * kWarps + warp) * run, (int64_t)P.vocab), x1 = (int32_t)min(x0 + run, (int64_t)P.vocab);
    uint32_t round = 0;
    bool bad = false;
    int at = 0, tried = 0;                                // tried: children of `at` below this one have been
    float c = 0.0f, m = 1.0f;

    // Weights of the kept node's tokens x ..: what is left of p, or p itself.
    const T *row_p = all_p + c0 * P.p_row, *row_q = DRAWN ? all_q + c0 * P.q_row : nullptr;
    auto load = [&](int32_t x, float cc, float (&w)[VEC]) {
        float p[VEC], q[VEC];
        if (VEC == 1 || x + VEC <= x1) {
            load_values<T, VEC>(row_p + x, p);
            if (DRAWN && cc > 0.0f) load_values<T, VEC>(row_q + x, q);
        } else {
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                p[k] = x + k < x1 ? value(row_p[x + k]) : 0.0f;
                if (DRAWN && cc > 0.0f) q[k] = x + k < x1 ? value(row_q[x + k]) : 0.0f;
            }
        }
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            w[k] = clean(p[k], bad);
            w[k] = DRAWN && cc > 0.0f ? rest_of(w[k], clean(q[k], bad), cc) : fminf(w[k], 1.0f);
        }
    };
    // Without q: nodes whose tokens have lost their weight, the kept node's children below `tried`.
    auto gone = [&](int i) { return M.parent[i] == at && M.token[i] >= 0 && M.token[i] < P.vocab && !(M.again[i >> 5] >> (i & 31) & 1u); };
    // The sum of all weights (take: without the tokens that lost theirs); this warp's and the CTAs' are
    // left in M.
    auto sum_row = [&](float cc, bool take) -> int64_t {
        Sum s{0, 0};
        uint32_t count = 0;
        constexpr int kAhead = VEC == 1 ? 8 : VEC == 4 ? 4 : 2;      // loads of a lane under way
        const bool two = DRAWN && cc > 0.0f;
        const uint64_t c2 = pair(-cc, -cc);
#pragma unroll 1
        for (int32_t x = x0 + VEC * lane; x < x1; x += 32 * VEC * kAhead) {
            float p[kAhead][VEC], q[kAhead][VEC];
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int32_t at_x = x + 32 * VEC * k;
#pragma unroll
                for (int i = 0; i < VEC; ++i) p[k][i] = q[k][i] = 0.0f;
                if (at_x + VEC <= x1) {
                    load_values<T, VEC>(row_p + at_x, p[k]);
                    if (two) load_values<T, VEC>(row_q + at_x, q[k]);
                } else if (VEC > 1) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        if (at_x + i < x1) p[k][i] = value(row_p[at_x + i]);
                        if (at_x + i < x1 && two) q[k][i] = value(row_q[at_x + i]);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
#pragma unroll
                for (int i = 0; i < VEC; ++i) top = max(top, max(__float_as_uint(p[k][i]), __float_as_uint(q[k][i])));
            if (top > 0x3f800000u) {                      // one by one
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        p[k][i] = clean(p[k][i], bad);
                        p[k][i] = two ? rest_of(p[k][i], clean(q[k][i], bad), cc) : fminf(p[k][i], 1.0f);
                        q[k][i] = 0.0f;
                    }
            }
#pragma unroll
            for (int k = 0; k < kAhead * VEC; k += 2) {
                float w0 = p[k / VEC][k % VEC], w1 = p[(k + 1) / VEC][(k + 1) % VEC];
                if (two) {                                // p + (-(c q)), each rounded: p - c q
                    apart(add2(pair(w0, w1), mul2(c2, pair(q[k / VEC][k % VEC], q[(k + 1) / VEC][(k + 1) % VEC]))), w0, w1);
                    w0 = fmaxf(w0, 0.0f);
                    w1 = fmaxf(w1, 0.0f);
                }
                add(s, w0, w1);
            }
            count += kAhead * VEC;
        }
        int64_t mine = whole(s, count);
        if (!DRAWN && take)
            for (int i = 1 + lane; i < tried; i += 32)
                if (gone(i) && M.token[i] >= x0 && M.token[i] < x1) {
                    bool none = false;
                    mine -= whole(fminf(clean(M.p[i], none), 1.0f));
                }
        mine = warp_sum(mine);
        __syncthreads();                                  // the sums before have been read
        if (lane == 0) M.warp[warp] = mine;
        __syncthreads();
        int64_t total = 0;
        for (int w = 0; w < kWarps; ++w) total += M.warp[w];
        const int side = round & 1;
        ++round;
        if (ctas > 1) {
            if (tid < ctas) to_peer(&M.cta[side][rank], tid, total);
            cluster_arrive();
            cluster_wait();
            total = 0;
            for (int k = 0; k < ctas; ++k) total += M.cta[side][k];
        }
        return total;
    };

    // ---- down the tree
    int keep = 1;
    int64_t total = -1;                                   // the weights' sum, once it is known
    if (tid == 0) M.path[0] = 0;
    for (int w = 0; w < (n + 31) >> 5 && keep < P.max_path;) {
        const int i32 = 32 * w + lane;
        const uint32_t is = __ballot_sync(0xffffffffu, i32 < n && i32 >= tried && i32 > 0 && M.parent[i32] == at);
        if (is == 0) {
            ++w;
            continue;
        }
        const int i = 32 * w + __ffs((int)is) - 1;
        tried = i + 1;
        const int32_t x = M.token[i];
        if (x < 0 || x >= P.vocab) {
            flags |= CSA2_DEV_BAD_INDEX;
            continue;
        }
        float p = clean(M.p[i], bad);
        bool yes;
        if (DRAWN) {
            const float q = clean(M.q[i], bad);
            yes = __fmul_rn(__fmul_rn(M.u[i], q), m) < fmaxf(__fsub_rn(p, __fmul_rn(c, q)), 0.0f);
        } else {
            if (M.again[i >> 5] >> (i & 31) & 1u) p = 0.0f;
            yes = __fmul_rn(M.u[i], m) < p;
        }
        if (yes) {
            if (tid == 0) M.path[keep] = i;
            ++keep;
            at = i;
            row_p = all_p + (c0 + at) * P.p_row;
            if (DRAWN) row_q = all_q + (c0 + at) * P.q_row;
            c = 0.0f;
            m = 1.0f;
            total = -1;
        } else if (DRAWN) {
            c = __fadd_rn(c, m);
            total = sum_row(c, false);
            m = __ll2float_rn(total) * 9.094947017729282e-13f;
        } else {
            m = fmaxf(__fsub_rn(m, p), 0.0f);
        }
    }

    // ---- the token behind them
    bool left = true;                                     // drawn from what is left
    if (total < 0) total = sum_row(c, true);
    if (total == 0) {
        left = false;
        total = sum_row(0.0f, false);
    }
    const int64_t M24 = min(max(__float2int_rd(__fmul_rn(P.r[b], 16777216.0f)), 0), (1 << 24) - 1);
    int64_t aim = (total >> 24) * M24 + (((total & ((1 << 24) - 1)) * M24) >> 24);
    const int side = (round - 1) & 1;
    for (int k = 0; k < rank; ++k) aim -= M.cta[side][k];
    for (int k = 0; k < warp; ++k) aim -= M.warp[k];
    if (total > 0 && aim >= 0 && aim < M.warp[warp]) {    // one warp of the cluster
        const float cc = left ? c : 0.0f;
        for (int32_t at_x = x0; at_x < x1; at_x += 32 * VEC) {
            const int32_t x = at_x + VEC * lane;
            float w[VEC];
            int64_t each[VEC], sum = 0;
            if (x < x1) {
                load(x, cc, w);
            } else {
#pragma unroll
                for (int k = 0; k < VEC; ++k) w[k] = 0.0f;
            }
            if (!DRAWN && left)
                for (int i = 1; i < tried; ++i)
                    if (gone(i))
#pragma unroll
                        for (int k = 0; k < VEC; ++k)
                            if (M.token[i] == x + k) w[k] = 0.0f;
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                each[k] = whole(w[k]);
                sum += each[k];
            }
            int64_t upto = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, upto > aim);
            if (past) {
                if (lane == __ffs((int)past) - 1) {
                    int64_t before = upto - sum;
                    int k = 0;
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {       // the first whose sum passes the aim
                        before += each[i];
                        k += before <= aim;
                    }
                    P.next_token[b] = x + k;
                }
                break;
            }
            aim -= __shfl_sync(0xffffffffu, upto, 31);
        }
    }
    if (bad) flags |= CSA2_DEV_NONFINITE;
    if (rank == 0) {
        __syncthreads();                                  // the path
        for (int i = tid; i < P.max_path; i += kThreads) P.path[(int64_t)b * P.max_path + i] = i < keep ? M.path[i] : -1;
        if (tid == 0) {
            P.keep[b] = keep;
            P.delta[b] = keep - n;
            if (total == 0) {
                P.next_token[b] = -1;
                flags |= CSA2D_DEV_NO_TOKEN;
            }
        }
    }
    if (flags) dev_flag(d_status, flags);
}

template <typename T, bool DRAWN>
cudaError_t launch(const csa2d_verify_args &a, int ctas, uint32_t *d_status, cudaStream_t s)
{
    constexpr int kVec = 16 / sizeof(T);
    const bool vec = (uintptr_t)a.p % 16 == 0 && a.p_row % kVec == 0 && (!DRAWN || ((uintptr_t)a.q % 16 == 0 && a.q_row % kVec == 0));
    const dim3 grid((unsigned)(a.batch * ctas));
    if (vec) return launch_pdl(tree_verify_kernel<T, DRAWN, kVec>, grid, dim3(kThreads), 0, s, ctas, a, ctas, d_status);
    return launch_pdl(tree_verify_kernel<T, DRAWN, 1>, grid, dim3(kThreads), 0, s, ctas, a, ctas, d_status);
}

} // namespace

cudaError_t launch_tree_verify(const csa2d_verify_args &a, uint32_t *d_status, cudaStream_t s)
{
    // CTAs a request: a power of two of them, while all requests' fit the GPU at once (two an SM; 64 trees
    // of up to 16 nodes over 131,072 tokens: 26.6 us with four, 28.8 with eight, 41 with two; one chain of six:
    // 10.2 us with eight, 14.4 with four) and each has a few thousand tokens.  CTAs of 256 threads, four an SM
    // and so eight a request of that batch, take 24.4 us for it, but 14.4 for the chain and 16.4 where this
    // takes 14.3 (33 trees over 32,003 bf16 tokens); both sizes would be twice the instances.
    int ctas = kMaxCtas;
    while (ctas > 1 && ((int64_t)a.batch * ctas > 2 * (int64_t)device_sm_count() || a.vocab < 2048 * ctas)) ctas /= 2;
    switch (a.type) {
    case CSA2D_F32: return a.q ? launch<float, true>(a, ctas, d_status, s) : launch<float, false>(a, ctas, d_status, s);
    case CSA2D_F16: return a.q ? launch<__half, true>(a, ctas, d_status, s) : launch<__half, false>(a, ctas, d_status, s);
    default: return a.q ? launch<__nv_bfloat16, true>(a, ctas, d_status, s) : launch<__nv_bfloat16, false>(a, ctas, d_status, s);
    }
}

} // namespace csa2

// Gradients of the factors of a pool of adapters, on the sm_100a tensor cores.
//
// Method: "LoRA 与 QLoRA" section LoRA (only A and B are trained); deck
// "3 QLoRA Finetuning" card 1.  For adapter a, over its tokens t:
//   dB_a [dout][r] = s_a sum_t dY_t^T U_t,   dA_a [r][din] = s_a sum_t G_t^T X_t,
// both as C[m][j] = s_a sum_t P[t][m] Q[t][j] with (P, Q) = (dY, U) and (X, G),
// dA stored transposed.
//
// HBM-bound (P is read once, Q is narrow), so everything else has to stay out
// of the way of the loads.  A CTA owns 128 MT rows m of one adapter over all of
// its tokens, K in steps of 64 gathered tokens: four producer warps copy the
// token rows by cp.async into swizzled tiles (a row of P or Q is one K of an
// MN-major operand, so nothing is transposed), one thread issues the MMAs, four
// warps add up.  Q enters as three bf16 parts (what an fp32 value holds), three
// MMAs each.  The accumulators alternate between two sets of TMEM columns and
// are added into fp32 registers every 512 tokens, because the tensor cores'
// running sums truncate and the error would grow with the sequence; the sums
// have one order whatever the timing.  On the register-level mma.sync path the
// same three parts took 2.5 to 8 times as long: their issue, not the loads, was
// the bound.
// Adapters without tokens get zeros, and so do columns past an adapter's rank.
// Every wait is bounded; on give-up the CTA records QLN_ERR_TIMEOUT, drains its
// copies and MMAs, frees TMEM and exits.
#include "qln_common.cuh"
#include "qln_internal.h"
#include "tc_ptx.cuh"

namespace qln {

constexpr int kGrBK = 64;      // tokens per step
constexpr int kGrGroup = 8;    // steps per accumulation in TMEM
constexpr uint64_t kGrWaitNs = 4000000000ull;

template <int NB, int MT>  // columns (r padded), 128-row sub-tiles
struct GrCfg {
    static constexpr int kRowB = NB >= 64 ? 128 : 2 * NB;  // bytes of a swizzled Q row
    static constexpr int kQBlocks = NB > 64 ? NB / 64 : 1;
    static constexpr uint32_t kPBytes = MT * 16384u;
    static constexpr uint32_t kQPart = kQBlocks * kGrBK * kRowB;
    static constexpr uint32_t kStage = kPBytes + 3 * kQPart;
    static constexpr int kSumWarps = 4 * MT;        // a TMEM lane quadrant of a sub-tile each; then 4 producers, 1 issuer
    static constexpr int kThreads = (kSumWarps + 5) * 32;
    static constexpr int kCtas = NB <= 32 ? 2 : 1;  // per SM
    static constexpr int kStages = NB == 16 ? 4 : NB == 32 ? 3 : NB == 64 ? 4 : 3;
    static constexpr uint32_t kTmemCols = 2 * MT * NB < 32 ? 32 : 2 * MT * NB;
    static constexpr uint32_t kOffBar = kStages * kStage;  // full[S], empty[S], acc_full[2], acc_empty[2]
    static constexpr uint32_t kOffMisc = kOffBar + (2 * kStages + 4) * 8;
    static constexpr uint32_t kSmem = kOffMisc + 16 + 1024;  // + alignment slack
    static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
    static_assert(kTmemCols * kCtas <= 512, "TMEM of an SM");
};

struct GradArgs {
    const uint16_t *P[2], *Q[2];  // 0: dB, 1: dA; Q: three planes of n * r
    int64_t M[2];
    float *C[2];
    const int32_t *order, *start, *rank;
    const float *scale;
    int64_t plane;
    int r, tilesB;
    int *status;
};

template <int NB, int MT>
__global__ void __launch_bounds__(GrCfg<NB, MT>::kThreads, GrCfg<NB, MT>::kCtas) adapter_grad_kernel(const GradArgs p) {
    using C = GrCfg<NB, MT>;
    constexpr int S = C::kStages, kProd = C::kSumWarps, kIssuer = kProd + 4;  // first producer warp, issuer warp
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem), bar0 = sbase + C::kOffBar;
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (S + s); };
    auto acc_full = [&](int b) { return bar0 + 8u * (2 * S + b); };
    auto acc_empty = [&](int b) { return bar0 + 8u * (2 * S + 2 + b); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 4);
    pdl_wait();
    pdl_trigger();
    const int which = (int)blockIdx.x < p.tilesB ? 0 : 1;
    const int a = blockIdx.y, r = p.r;
    const int64_t M = which ? p.M[1] : p.M[0], m0 = (int64_t)((int)blockIdx.x - (which ? p.tilesB : 0)) * 128 * MT;
    const int p0 = __ldg(p.start + a), cnt = __ldg(p.start + a + 1) - p0;
    const int steps = (cnt + kGrBK - 1) / kGrBK, groups = (steps + kGrGroup - 1) / kGrGroup;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    uint32_t tmem_d = 0;
    if (steps > 0) {  // uniform over the CTA
        if (tid == 0) {
            for (int s = 0; s < S; ++s) {
                tc::mbar_init(full(s), 128);
                tc::mbar_init(empty(s), 1);
            }
            for (int b = 0; b < 2; ++b) {
                tc::mbar_init(acc_full(b), 1);
                tc::mbar_init(acc_empty(b), 32 * C::kSumWarps);
            }
            *abort_flag = 0;
            tc::mbar_fence_init();
        }
        if (warp == kIssuer) {
            tc::tmem_alloc(tc::smem_addr(tmem_slot), C::kTmemCols);
            tc::tmem_relinquish();
        }
        tc::tc_fence_before();
        __syncthreads();
        tc::tc_fence_after();
        tmem_d = *tmem_slot;
    }
    auto give_up = [&]() {
        *abort_flag = 1;
        atomicExch(p.status, (int)QLN_ERR_TIMEOUT);
    };

    if (warp >= kProd && warp < kIssuer) {
        // ------------------------------------------------------------ producers
        // Sixteen threads per token row: thread (c, r0) copies chunk c of the rows r0 + 8 i.  A stage is handed over
        // once its copies have landed, two steps after their issue.
        constexpr int kLag = S - 2;
        const int pt = tid - 32 * kProd, c = pt & 15, r0 = pt >> 4;
        const uint16_t *P = which ? p.P[1] : p.P[0], *Q = which ? p.Q[1] : p.Q[0];
        int tok[8];
        auto tokens = [&](int st) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int q = st * kGrBK + r0 + 8 * i;
                tok[i] = q < cnt ? __ldg(p.order + p0 + q) : -1;
            }
        };
        auto hand_over = [&](int st) {
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(full(st % S));
        };
        if (steps > 0) tokens(0);
        int done = 0;  // steps handed over
        bool ok = true;
        for (int st = 0; st < steps; ++st) {
            const int s = st % S;
            ok = tc::mbar_wait_bounded(empty(s), ((uint32_t)(st / S) & 1u) ^ 1u, abort_flag, kGrWaitNs);
            if (!ok) {
                give_up();
                break;
            }
            const uint32_t sP = sbase + s * C::kStage, sQ = sP + C::kPBytes;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int row = r0 + 8 * i;  // row % 8 == r0
                const bool in = tok[i] >= 0;
                const uint16_t *src = P + (in ? (int64_t)tok[i] * M + m0 + 8 * c : 0);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const bool ok16 = in && m0 + 128 * mt + 8 * c < M;
                    // 64-wide blocks of m, 8192 bytes each
                    const uint32_t dst = sP + mt * 16384 + (c >> 3) * 8192 + row * 128 + (((c & 7) ^ r0) << 4);
                    cp_async16_to(dst, ok16 ? src + 128 * mt : P, ok16 ? 16 : 0);
                }
#pragma unroll
                for (int k = c; k < 3 * (NB / 8); k += 16) {
                    const int part = k / (NB / 8), ck = k % (NB / 8);
                    const bool ok16 = in && 8 * ck < r;
                    const int swz = C::kRowB == 128 ? r0 : C::kRowB == 64 ? (row >> 1) & 3 : (row >> 2) & 1;
                    const uint32_t dst = sQ + part * C::kQPart + (ck >> 3) * (kGrBK * 128) + row * C::kRowB +
                                         (((ck & 7) ^ swz) << 4);
                    cp_async16_to(dst, ok16 ? Q + part * p.plane + (int64_t)tok[i] * r + 8 * ck : Q, ok16 ? 16 : 0);
                }
            }
            cp_async_commit();
            if (st + 1 < steps) tokens(st + 1);
            if (st >= kLag) {
                cp_async_wait<kLag>();
                hand_over(done++);
            }
        }
        cp_async_wait<0>();
        for (; ok && done < steps; ++done) hand_over(done);
    } else if (warp == kIssuer) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0 && steps > 0) {
            const uint32_t idesc = tc::idesc_bf16_f32(128, NB, true, true);
            for (int st = 0; st < steps; ++st) {
                const int s = st % S, grp = st / kGrGroup, b = grp & 1;
                const bool first = st % kGrGroup == 0;
                if ((first && grp >= 2 &&
                     !tc::mbar_wait_bounded(acc_empty(b), (uint32_t)(grp / 2 - 1) & 1u, abort_flag, kGrWaitNs)) ||
                    !tc::mbar_wait_bounded(full(s), (uint32_t)(st / S) & 1u, abort_flag, kGrWaitNs)) {
                    give_up();
                    break;
                }
                tc::tc_fence_after();
                const uint32_t sP = sbase + s * C::kStage, sQ = sP + C::kPBytes;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int k = 0; k < kGrBK / 16; ++k)
#pragma unroll
                        for (int part = 0; part < 3; ++part)
                            tc::tc_mma_ss(tmem_d + (b * MT + mt) * NB,
                                          tc::smem_desc_mn<128>(sP + mt * 16384 + k * 2048, 8192),
                                          tc::smem_desc_mn<C::kRowB>(sQ + part * C::kQPart + k * 16 * C::kRowB, kGrBK * 128),
                                          idesc, first && k == 0 && part == 0 ? 0u : 1u);
                tc::tc_commit(empty(s));
                if (st % kGrGroup == kGrGroup - 1 || st == steps - 1) tc::tc_commit(acc_full(b));
            }
        }
    } else {
        // ------------------------------------------------------------ sums and results
        const int mt = warp >> 2, quad = warp & 3;
        float sum[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) sum[j] = 0.f;
        bool ok = true;
        for (int grp = 0; grp < groups; ++grp) {
            const int b = grp & 1;
            ok = tc::mbar_wait_bounded(acc_full(b), (uint32_t)(grp / 2) & 1u, abort_flag, kGrWaitNs);
            if (!ok) give_up();
            ok = __all_sync(0xffffffffu, ok);  // tcgen05.ld is warp-collective
            if (!ok) break;
            tc::tc_fence_after();
#pragma unroll
            for (int j0 = 0; j0 < NB; j0 += 16) {
                uint32_t v[16];
                tc::tmem_ld_32x32b_x16(tmem_d + ((uint32_t)(quad * 32) << 16) + (uint32_t)((b * MT + mt) * NB + j0), v);
                tc::tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) sum[j0 + j] = __fadd_rn(sum[j0 + j], __uint_as_float(v[j]));
            }
            tc::tc_fence_before();
            tc::mbar_arrive(acc_empty(b));
        }
        if (ok) {
            const int rk0 = p.rank ? __ldg(p.rank + a) : r, rk = cnt > 0 ? min(max(rk0, 0), r) : 0;
            const float s = __ldg(p.scale + a);
            float *out = (which ? p.C[1] : p.C[0]) + (int64_t)a * M * r;
            const int64_t m = m0 + 128 * mt + quad * 32 + lane;
            if (m < M && which) {  // dA [r][din]: consecutive m per j
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    if (j < r) out[(int64_t)j * M + m] = j < rk ? __fmul_rn(s, sum[j]) : 0.f;
            } else if (m < M) {    // dB [dout][r]: a row of r per m (r is a multiple of 8)
#pragma unroll
                for (int j = 0; j < NB; j += 4)
                    if (j < r) {
                        float4 v;
                        v.x = j < rk ? __fmul_rn(s, sum[j]) : 0.f;
                        v.y = j + 1 < rk ? __fmul_rn(s, sum[j + 1]) : 0.f;
                        v.z = j + 2 < rk ? __fmul_rn(s, sum[j + 2]) : 0.f;
                        v.w = j + 3 < rk ? __fmul_rn(s, sum[j + 3]) : 0.f;
                        *reinterpret_cast<float4 *>(out + m * r + j) = v;
                    }
            }
        }
    }

    if (steps > 0) {
        // Teardown: every MMA has retired before TMEM is released.
        tc::tc_fence_before();
        __syncthreads();
        if (warp == kIssuer) {
            if (lane == 0 && *abort_flag) {  // the last commit covers all MMAs issued; its phase is not known after an abort
                tc::tc_commit(acc_full(0));
                const uint64_t t0 = tc::global_timer_ns();
                while (tc::global_timer_ns() - t0 < 2000000ull) {}  // 2 ms: far longer than the MMAs of a ring
            }
            __syncwarp();
            tc::tc_fence_after();
            tc::tmem_dealloc(tmem_d, C::kTmemCols);
        }
    }
}

template <int NB, int MT>
static cudaError_t launch_grad(GradArgs &a, int count, cudaStream_t st) {
    using C = GrCfg<NB, MT>;
    auto kern = adapter_grad_kernel<NB, MT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    a.tilesB = (int)((a.M[0] + 128 * MT - 1) / (128 * MT));
    const unsigned tilesA = (unsigned)((a.M[1] + 128 * MT - 1) / (128 * MT));
    return launch_pdl(kern, dim3((unsigned)a.tilesB + tilesA, (unsigned)count), dim3(C::kThreads), (size_t)C::kSmem, st, a);
}

cudaError_t launch_adapter_grads(const uint16_t *dY, const uint16_t *U3, int64_t dout, const uint16_t *X,
                                 const uint16_t *G3, int64_t din, int64_t n, const qln_adapter_pool *pool,
                                 const AdapterPlan &p, float *dA, float *dB, int *status, cudaStream_t st) {
    GradArgs a;
    a.P[0] = dY, a.P[1] = X;
    a.Q[0] = U3, a.Q[1] = G3;
    a.M[0] = dout, a.M[1] = din;
    a.C[0] = dB, a.C[1] = dA;
    a.order = p.order, a.start = p.start, a.rank = pool->rank;
    a.scale = pool->scale;
    a.plane = n * pool->r;
    a.r = pool->r;
    a.status = status;
    if (a.r <= 16) return launch_grad<16, 1>(a, pool->count, st);
    if (a.r <= 32) return launch_grad<32, 1>(a, pool->count, st);
    if (a.r <= 64) return launch_grad<64, 2>(a, pool->count, st);
    return launch_grad<128, 1>(a, pool->count, st);
}

}  // namespace qln

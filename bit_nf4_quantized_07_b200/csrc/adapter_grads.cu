// Gradients of the factors of a pool of adapters, on the sm_100a tensor cores.
//
// Method: "LoRA 与 QLoRA" section LoRA (only A and B are trained); deck
// "3 QLoRA Finetuning" card 1.  For adapter a, over its tokens t:
//   dB_a [dout][r] = s_a sum_t dY_t^T U_t,   dA_a [r][din] = s_a sum_t G_t^T X_t,
// both as C[m][j] = s_a sum_t P[t][m] Q[t][j] with (P, Q) = (dY, U) and (X, G),
// dA stored transposed.
//
// HBM-bound (P is read once, Q is narrow), so everything else has to stay out
// of the way of the loads.  An item is 128 MT rows m of one adapter over all of
// its tokens, K in steps of 64 gathered tokens; a CTA works through every
// gridDim.x-th item without draining its ring in between.  Producer warps copy
// the token rows by cp.async into swizzled tiles (a row of P or Q is one K of an
// MN-major operand, so nothing is transposed), their token numbers read two
// steps ahead; one thread issues the MMAs; four warps or eight add up and store.  Q
// enters as three bf16 parts (what an fp32 value holds), three MMAs each; the
// first part has an accumulator of its own, because the tensor cores' running
// sums truncate at every addition.  For the same reason the accumulators, two
// sets in turn, are added into fp32 registers every 512 tokens: the error does
// not grow with the sequence.  The sums have one order whatever the timing.
// 2048 tokens of 4 adapters, 11008 + 4096 columns, rank 16, cold: 29 us, 2.1 TB/s
// (rows of 256 bytes gathered from tokens 22 KB apart; the longest adapter's
// items take 1.3 times the mean); 4096 tokens, 28672 + 8192, rank 64: 113 us.
// On the register-level mma.sync path the same three parts took 2.5 to 4 times
// as long: their issue, not the loads, was the bound.
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
    static constexpr int kCols = NB > 64 ? 64 : NB;  // columns that a sum warp keeps in registers
    static constexpr int kSumWarps = 4 * MT * (NB / kCols);  // a TMEM lane quadrant of a sub-tile (or half of its columns) each
    static constexpr int kProdWarps = 8;            // then the producers, then the issuer
    static constexpr int kThreads = (kSumWarps + kProdWarps + 1) * 32;
    static constexpr int kCtas = NB <= 32 ? 2 : 1;  // per SM
    static constexpr int kStages = NB == 16 ? 4 : NB == 32 ? 3 : NB == 64 ? 4 : 3;
    static constexpr uint32_t kTmemCols = 4 * MT * NB;  // two sets of (first part, the other two)
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
    int r, count, tiles, tilesB;  // tiles: of 128 MT rows, dB's then dA's
    int *status;
};

template <int NB, int MT>
__global__ void __launch_bounds__(GrCfg<NB, MT>::kThreads, GrCfg<NB, MT>::kCtas) adapter_grad_kernel(const GradArgs p) {
    using C = GrCfg<NB, MT>;
    constexpr int S = C::kStages, kProd = C::kSumWarps, kIssuer = kProd + C::kProdWarps;  // first producer warp, issuer warp
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
    const int r = p.r, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int items = p.tiles * p.count;
    // Up to 32 adapters are taken in the order of their token counts, the longest first: the last round's items are then
    // the shortest, and the tail of the grid is short.
    __shared__ int s_order[32];
    if (warp == 0 && p.count <= 32) {
        const int c = lane < p.count ? __ldg(p.start + lane + 1) - __ldg(p.start + lane) : -1;
        int ahead = 0;
        for (int b = 0; b < 32; ++b) {
            const int o = __shfl_sync(0xffffffffu, c, b);
            ahead += o > c || (o == c && b < lane);
        }
        s_order[ahead] = lane;
    }
    struct Item {  // 128 MT rows of one adapter: tile counts dB's, then dA's
        int a, p0, cnt, tile;
        __device__ bool dA(const GradArgs &p) const { return tile >= p.tilesB; }
        __device__ int64_t M(const GradArgs &p) const { return dA(p) ? p.M[1] : p.M[0]; }
        __device__ int64_t m0(const GradArgs &p) const { return (int64_t)(dA(p) ? tile - p.tilesB : tile) * (128 * MT); }
    };
    auto item_at = [&](int i) {
        Item t{0, 0, 0, 0};
        if (i < items) {
            t.a = i / p.tiles;
            t.tile = i - t.a * p.tiles;
            if (p.count <= 32) t.a = s_order[t.a];
            t.p0 = __ldg(p.start + t.a);
            t.cnt = __ldg(p.start + t.a + 1) - t.p0;
        }
        return t;
    };
    auto steps_of = [](const Item &t) { return (t.cnt + kGrBK - 1) / kGrBK; };

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            tc::mbar_init(full(s), 32 * C::kProdWarps);
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
    const uint32_t tmem_d = *tmem_slot;
    auto give_up = [&]() {
        *abort_flag = 1;
        atomicExch(p.status, (int)QLN_ERR_TIMEOUT);
    };

    if (warp >= kProd && warp < kIssuer) {
        // ------------------------------------------------------------ producers
        // Sixteen threads per token row: thread (c, r0) copies chunk c of the rows r0 + 16 i.  A stage is handed over
        // once its copies have landed, two steps after their issue.
        constexpr int kLag = S - 2;
        const int pt = tid - 32 * kProd, c = pt & 15, r0 = pt >> 4;
        struct Step {  // one step: its tokens (-1: none) and its item's tile (-1: no step)
            int tok[4], tile;
        };
        int next_item = blockIdx.x, st = 0, left = 0;  // the look-ahead: its item's next step, steps left
        Item it = item_at(next_item), nx = item_at(next_item + gridDim.x);
        left = steps_of(it);
        auto look = [&](Step &x) {
            while (left == 0 && next_item < items) {
                next_item += gridDim.x;
                it = nx;
                nx = item_at(next_item + gridDim.x);
                left = steps_of(it);
                st = 0;
            }
            x.tile = left > 0 ? it.tile : -1;
            if (left == 0) return;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int q = st * kGrBK + r0 + 16 * i;
                x.tok[i] = q < it.cnt ? __ldg(p.order + it.p0 + q) : -1;
            }
            ++st;
            --left;
        };
        auto hand_over = [&](int k) {
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(full(k % S));
        };
        Step cur, n1;
        look(cur);
        look(n1);
        int k = 0, done = 0;  // steps issued, handed over
        bool ok = true;
        while (cur.tile >= 0) {
            const int s = k % S;
            ok = tc::mbar_wait_bounded(empty(s), ((uint32_t)(k / S) & 1u) ^ 1u, abort_flag, kGrWaitNs);
            if (!ok) {
                give_up();
                break;
            }
            const uint32_t sP = sbase + s * C::kStage, sQ = sP + C::kPBytes;
            const Item of{0, 0, 0, cur.tile};
            const bool dA = of.dA(p);
            const int64_t M = of.M(p), m = of.m0(p) + 8 * c;  // this thread's columns of P: m, and 128 further
            const uint16_t *const P = (dA ? p.P[1] : p.P[0]) + m, *const Q = dA ? p.Q[1] : p.Q[0];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = r0 + 16 * i, t = cur.tok[i], r7 = r0 & 7;  // row % 8
                const bool in = t >= 0;
                const uint16_t *src = P + (int64_t)t * M;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const bool ok16 = in && m + 128 * mt < M;
                    // 64-wide blocks of m, 8192 bytes each
                    const uint32_t dst = sP + mt * 16384 + (c >> 3) * 8192 + row * 128 + (((c & 7) ^ r7) << 4);
                    cp_async16_to(dst, ok16 ? src + 128 * mt : p.P[0], ok16 ? 16 : 0);
                }
#pragma unroll
                for (int u = 0; u < (3 * (NB / 8) + 15) / 16; ++u) {
                    const int kq = c + 16 * u;
                    if (kq >= 3 * (NB / 8)) break;
                    const int part = kq / (NB / 8), ck = kq % (NB / 8);
                    const bool ok16 = in && 8 * ck < r;
                    const int swz = C::kRowB == 128 ? r7 : C::kRowB == 64 ? (row >> 1) & 3 : (row >> 2) & 1;
                    const uint32_t dst = sQ + part * C::kQPart + (ck >> 3) * (kGrBK * 128) + row * C::kRowB +
                                         (((ck & 7) ^ swz) << 4);
                    cp_async16_to(dst, ok16 ? Q + part * p.plane + (int64_t)t * r + 8 * ck : p.P[0], ok16 ? 16 : 0);
                }
            }
            cp_async_commit();
            cur = n1;
            look(n1);
            if (k++ >= kLag) {
                cp_async_wait<kLag>();
                hand_over(done++);
            }
        }
        cp_async_wait<0>();
        for (; ok && done < k; ++done) hand_over(done);
    } else if (warp == kIssuer) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            const uint32_t idesc = tc::idesc_bf16_f32(128, NB, true, true);
            int k = 0, grp = 0;  // steps and groups so far
            bool ok = true;
            Item nx = item_at(blockIdx.x);
            for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
                const int steps = steps_of(nx);
                nx = item_at(i + gridDim.x);
                for (int st = 0; st < steps; ++st, ++k) {
                    const int s = k % S, b = grp & 1;
                    const bool first = st % kGrGroup == 0, last = st % kGrGroup == kGrGroup - 1 || st == steps - 1;
                    ok = (!first || grp < 2 ||
                          tc::mbar_wait_bounded(acc_empty(b), (uint32_t)(grp / 2 - 1) & 1u, abort_flag, kGrWaitNs)) &&
                         tc::mbar_wait_bounded(full(s), (uint32_t)(k / S) & 1u, abort_flag, kGrWaitNs);
                    if (!ok) {
                        give_up();
                        break;
                    }
                    tc::tc_fence_after();
                    const uint32_t sP = sbase + s * C::kStage, sQ = sP + C::kPBytes;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int kk = 0; kk < kGrBK / 16; ++kk)
#pragma unroll
                            for (int part = 0; part < 3; ++part)
                                tc::tc_mma_ss(tmem_d + ((b * MT + mt) * 2 + (part ? 1 : 0)) * NB,
                                              tc::smem_desc_mn<128>(sP + mt * 16384 + kk * 2048, 8192),
                                              tc::smem_desc_mn<C::kRowB>(sQ + part * C::kQPart + kk * 16 * C::kRowB, kGrBK * 128),
                                              idesc, first && kk == 0 && part < 2 ? 0u : 1u);
                    tc::tc_commit(empty(s));
                    if (last) {
                        tc::tc_commit(acc_full(b));
                        ++grp;
                    }
                }
            }
        }
    } else {
        // ------------------------------------------------------------ sums and results
        constexpr int NC = C::kCols;
        const int mt = (warp >> 2) % MT, quad = warp & 3, col0 = (warp >> 2) / MT * NC;
        int grp = 0;
        bool ok = true;
        Item nx = item_at(blockIdx.x);
        for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const Item t = nx;
            nx = item_at(i + gridDim.x);
            const int rk0 = p.rank ? __ldg(p.rank + t.a) : r;
            const float s = __ldg(p.scale + t.a);
            float sum[NC];
#pragma unroll
            for (int j = 0; j < NC; ++j) sum[j] = 0.f;
            for (int g = (steps_of(t) + kGrGroup - 1) / kGrGroup; g > 0; --g, ++grp) {
                const int b = grp & 1;
                ok = tc::mbar_wait_bounded(acc_full(b), (uint32_t)(grp / 2) & 1u, abort_flag, kGrWaitNs);
                if (!ok) give_up();
                ok = __all_sync(0xffffffffu, ok);  // tcgen05.ld is warp-collective
                if (!ok) break;
                tc::tc_fence_after();
                const uint32_t base = tmem_d + ((uint32_t)(quad * 32) << 16) + (uint32_t)((b * MT + mt) * 2 * NB + col0);
#pragma unroll
                for (int j0 = 0; j0 < NC; j0 += 8) {
                    uint32_t v[8], w[8];
                    tc::tmem_ld_32x32b_x8(base + j0, v);
                    tc::tmem_ld_32x32b_x8(base + NB + j0, w);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        sum[j0 + j] = __fadd_rn(sum[j0 + j], __fadd_rn(__uint_as_float(v[j]), __uint_as_float(w[j])));
                }
                tc::tc_fence_before();
                tc::mbar_arrive(acc_empty(b));
            }
            if (!ok) break;
            const int rk = t.cnt > 0 ? min(max(rk0, 0), r) : 0;
            const int64_t M = t.M(p), m = t.m0(p) + 128 * mt + quad * 32 + lane;
            float *out = (t.dA(p) ? p.C[1] : p.C[0]) + (int64_t)t.a * M * r;
            if (m < M && t.dA(p)) {  // dA [r][din]: consecutive m per j
#pragma unroll
                for (int j = 0; j < NC; ++j)
                    if (col0 + j < r) out[(int64_t)(col0 + j) * M + m] = col0 + j < rk ? __fmul_rn(s, sum[j]) : 0.f;
            } else if (m < M) {   // dB [dout][r]: a row of r per m (r is a multiple of 8)
#pragma unroll
                for (int j = 0; j < NC; j += 4)
                    if (col0 + j < r) {
                        float4 v;
                        v.x = col0 + j < rk ? __fmul_rn(s, sum[j]) : 0.f;
                        v.y = col0 + j + 1 < rk ? __fmul_rn(s, sum[j + 1]) : 0.f;
                        v.z = col0 + j + 2 < rk ? __fmul_rn(s, sum[j + 2]) : 0.f;
                        v.w = col0 + j + 3 < rk ? __fmul_rn(s, sum[j + 3]) : 0.f;
                        *reinterpret_cast<float4 *>(out + m * r + col0 + j) = v;
                    }
            }
        }
    }

    // Teardown: every MMA has retired before TMEM is released (the sums have waited for the last of them).
    tc::tc_fence_before();
    __syncthreads();
    if (warp == kIssuer) {
        if (lane == 0 && *abort_flag) {  // after an abort the barriers' phases are not known
            const uint64_t t0 = tc::global_timer_ns();
            while (tc::global_timer_ns() - t0 < 2000000ull) {}  // 2 ms: far longer than a ring's MMAs take
        }
        __syncwarp();
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem_d, C::kTmemCols);
    }
}

template <int NB, int MT>
static cudaError_t launch_grad(GradArgs &a, cudaStream_t st, int num_sms) {
    using C = GrCfg<NB, MT>;
    auto kern = adapter_grad_kernel<NB, MT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    a.tilesB = (int)((a.M[0] + 128 * MT - 1) / (128 * MT));
    a.tiles = a.tilesB + (int)((a.M[1] + 128 * MT - 1) / (128 * MT));
    // One wave that walks the items: their rings do not drain in between, and no CTA starts late.  A CTA per item instead
    // (whole calls, us): 4096 x 4096, 100 tokens of 8 adapters 37.4 / 35.1; 1000 tokens of 40 adapters, rank 32: 161 / 144;
    // 4096 x 11008, 2048 tokens of 16 adapters, rank 64: 265 / 242.
    const int64_t items = (int64_t)a.tiles * a.count, wave = (int64_t)num_sms * C::kCtas;
    return launch_pdl(kern, dim3((unsigned)(items < wave ? items : wave)), dim3(C::kThreads), (size_t)C::kSmem, st, a);
}

cudaError_t launch_adapter_grads(const uint16_t *dY, const uint16_t *U3, int64_t dout, const uint16_t *X,
                                 const uint16_t *G3, int64_t din, int64_t n, const qln_adapter_pool *pool,
                                 const AdapterPlan &p, float *dA, float *dB, int *status, cudaStream_t st,
                                 int num_sms) {
    GradArgs a;
    a.P[0] = dY, a.P[1] = X;
    a.Q[0] = U3, a.Q[1] = G3;
    a.M[0] = dout, a.M[1] = din;
    a.C[0] = dB, a.C[1] = dA;
    a.order = p.order, a.start = p.start, a.rank = pool->rank;
    a.scale = pool->scale;
    a.plane = n * pool->r;
    a.r = pool->r;
    a.count = pool->count;
    a.status = status;
    if (a.r <= 16) return launch_grad<16, 1>(a, st, num_sms);
    if (a.r <= 32) return launch_grad<32, 1>(a, st, num_sms);
    if (a.r <= 64) return launch_grad<64, 2>(a, st, num_sms);
    return launch_grad<128, 1>(a, st, num_sms);
}

}  // namespace qln

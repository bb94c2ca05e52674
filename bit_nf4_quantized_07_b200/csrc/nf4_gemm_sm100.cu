// Fused NF4 doubleDequant + GEMM on the sm_100a tensor cores (tcgen05, TMEM
// accumulators, TMA operand loads).  W' is decoded tile by tile into shared
// memory and never reaches HBM.
//
// Method: "LoRA 与 QLoRA" section QLoRA 1 (4-bit weight -> dequant -> BF16 ->
// GEMM) and section LoRA (y = W0 x + s B(A x), A x formed first); jjjymmm.cn
// "QLoRA" (doubleDequant: restore the block constant, then the weight); deck
// "3 QLoRA Finetuning" card 1 (the matmul sees the dequantized BF16 weight and
// gradients flow through it).
//
//   forward (TRANS = false): out[t][m] = sum_k X[t][k] W'[m][k]  + sum_j sU[t][j] B[m][j]
//   dX      (TRANS = true) : out[t][m] = sum_k dY[t][k] W'[k][m] + sum_j sG[t][j] A[j][m]
//
// One CTA computes a (128*MT) (m) x (NT*BN) (tokens) tile as MT*NT <= 2
// accumulators of 128 TMEM lanes x BN columns, K in steps of 64.  MT = 2 lets
// two 128-row weight tiles share every activation tile (half the activation
// bytes per FLOP); NT = 2 lets every decoded weight tile serve two token
// tiles (half the decode work per FLOP, the integer-pipe bound of the
// decoders).  The shape is chosen per call.
//   A_op (weights): decoded by 128*MT threads (one 64-wide row block each)
//     into the canonical 128-byte-swizzled layout, K-major for the forward
//     (W' rows along K) and MN-major for dX (W' rows are the K index, their
//     consecutive columns the M index);
//   B_op (activations X / dY, K-major): TMA tiles with 128-byte swizzle;
//   the adapter term is extra K steps whose A_op (B or A, zero-padded to 64)
//     and B_op (s*U or s*G) both arrive by TMA.
// MULTI: each token has an adapter of its own from a pool.  The adapter term
// goes by chunks of 16 columns: the first 16 of every adapter present among the
// tile's tokens (warp 1 lists them while the pipeline fills), then the next 16
// of those with a larger rank, and so on; a k-step takes the next four chunks,
// whichever adapters they belong to.  A chunk's A_op is 16 columns of the
// adapter's factor by TMA in 32-byte rows (dX: 16 rows of it, as in a weight
// step; 3-D maps, so what lies past the factor reads as zero).  Its B_op is
// written by the decoders: s*U or s*G of the adapter's own tokens, copied
// asynchronously one k-step ahead, zero for the others; a stage's zeros stay
// where they are from step to step.  (One warp per scheduler has nothing to
// hide its instructions behind: writing every row in every step took 1.5 us per
// k-step.)  All MMAs keep one shape: only
// then do they run in the order of their issue.  A zero times an infinity would
// still be a NaN, so the decoders also replace what is not finite in the
// factor's tile by 1 with its sign, and the epilogue adds those products to
// their own tokens one by one (a path that finite factors never take; what the 1
// brings is nothing beside an infinity, and of its sign where s U is infinite
// too, where a zero would make it NaN).  A k-step of
// chunks costs about as much as a weight step; a prefill tile of packed
// sequences has one or two.
// A MULTI kernel reads its activations and weights before the kernel ahead of
// it on the stream has completed, and waits for that one only before the
// adapter steps.  This is safe because the call's first kernel waits for all
// earlier work, and every kernel of the call lets its dependents start only
// after its own wait.
// Warp roles: warp 0 TMA producer, warp 1 TMEM owner + single-thread MMA
// issuer, warps 2.. decoders and then the epilogue (TMEM -> BF16 -> HBM).
// Every barrier wait is bounded; on give-up the CTA records QLN_ERR_TIMEOUT
// in the status word, drains its own copies and MMAs, frees TMEM and exits.
#include <cuda.h>

#include "qln_common.cuh"
#include "qln_internal.h"
#include "tc_ptx.cuh"

namespace qln {
namespace tc {

constexpr int kBM = 128;   // rows per accumulator (TMEM lanes)
constexpr int kBK = 64;
constexpr uint64_t kWaitLimitNs = 4000000000ull;  // 4 s

template <int MT, int NT, bool MULTI>
struct Cfg {
    static_assert(MT * NT <= 2, "two TMEM accumulators of up to 256 columns at most");
    static constexpr int kStages = MT * NT == 1 ? 4 : 3;
    static constexpr int kMaxBN = NT == 1 ? 256 : 208;     // tokens per accumulator
    // One decoder per 64-wide row block of the weight tile; MULTI: always 256, so that with MT = 1 there are two groups,
    // which take the weight steps in turn: a step's chain of waits, decoding and fences is longer than its MMAs where
    // there are few tokens, and two chains run side by side.  In the steps of chunks two threads share a row.
    static constexpr int kDecThreads = MULTI ? 256 * MT : 128 * MT;
    static constexpr int kShare = kDecThreads / (128 * MT);  // groups, or threads per row of a chunk
    static constexpr int kThreads = 64 + kDecThreads;
    static constexpr uint32_t kABytes = 16384u * MT;        // MT x (128 rows x 64 K) bf16
    static constexpr uint32_t kBBytes = NT * kMaxBN * kBK * 2;
    static constexpr uint32_t kCBytes = 4096u * MT;         // codes of the A tile
    static constexpr uint32_t kTmemCols = 256u * MT * NT;
    static constexpr uint32_t kOffA = 0;
    static constexpr uint32_t kOffB = kOffA + kStages * kABytes;
    static constexpr uint32_t kOffC = kOffB + kStages * kBBytes;
    static constexpr uint32_t kOffBar = kOffC + kStages * kCBytes;
    // barriers: tma_full[S], code_full[S], dec_full[S], empty[S], accum_full, list_full (MULTI)
    static constexpr uint32_t kNumBars = 4 * kStages + 2;
    static_assert(MT * NT == 1 || kOffBar == 221184u, "one size for both");
    static constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;  // tmem base, abort flag, epilogue go
    static constexpr uint32_t kSmemBytes = kOffMisc + 16 + 1024;  // + alignment slack
    // MULTI: the tile's list of adapters (one word each), the adapter of each token, and the list's place of every
    // adapter of the pool (16 bits each)
    static constexpr int kTok = NT * kMaxBN;
    static constexpr uint32_t kOffList = kOffMisc + 16;
    static constexpr uint32_t kListBytes = kTok * 6 + QLN_MAX_ADAPTERS * 2 + 16;
    static constexpr uint32_t kSmemBytesMulti = kSmemBytes + kListBytes;
    static_assert(kSmemBytesMulti <= 232448, "shared memory of one CTA");
};

// The pool's side of a MULTI call.
struct MultiParams {
    const int32_t *ids, *rank;
    const uint16_t *lact;  // [n][r] bf16: s U or s G
    const uint16_t *lw;    // the pool's factors
    int count, r;
};

// ---- cluster (K split of a MULTI call) ----
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_map(uint32_t saddr, uint32_t rank) {
    uint32_t d;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(saddr), "r"(rank));
    return d;
}
__device__ __forceinline__ void cluster_st_u32(uint32_t a, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// Columns (tokens) of a tile that each CTA of a K split finishes: a multiple of 8.
__host__ __device__ constexpr int split_cols(int ntok, int ks) { return ((ntok + ks - 1) / ks + 7) & ~7; }

// What the products of a factor's non-finite elements add to one output (m, t)
// of adapter a: lw rows of m with stride 1 over j (forward) or columns with
// stride M (dX).
__device__ __noinline__ float nonfinite_products(const MultiParams &mp, int a, int64_t m, int64_t t, int64_t M, bool trans) {
    float v = 0.f;
    const int rk = mp.rank ? min(max(__ldg(mp.rank + a), 0), mp.r) : mp.r;
    for (int j = 0; j < rk; ++j) {
        const uint32_t f = mp.lw[trans ? ((int64_t)a * mp.r + j) * M + m : ((int64_t)a * M + m) * mp.r + j];
        if ((f & 0x7f80u) == 0x7f80u) v += bf16lo_to_f32(f) * bf16lo_to_f32(mp.lact[t * mp.r + j]);
    }
    return v;
}

struct Params {
    const int8_t *qabs;
    bool e4m3;  // qabs holds E4M3 codes (QLN_DQ_E4M3), else int8
    const float *absmax;
    const float *dq_scale;
    const float *dq_mean;
    int64_t cols;      // W columns (din)
    int64_t n;         // tokens
    uint16_t *out;     // [n][out_ld]
    int64_t out_ld;
    int *status;
    int KT;            // weight k-steps
    int RT;            // adapter k-steps
    int BN;            // tokens per accumulator (multiple of 16)
};

template <bool TRANS, int MT, int NT, bool MULTI>
__global__ void __launch_bounds__(Cfg<MT, NT, MULTI>::kThreads, 1)
nf4_tc_gemm_kernel(const __grid_constant__ CUtensorMap tm_codes, const __grid_constant__ CUtensorMap tm_act,
                   const __grid_constant__ CUtensorMap tm_lw, const __grid_constant__ CUtensorMap tm_lact,
                   const Params p, const __grid_constant__ MultiParams mp) {
    using C = Cfg<MT, NT, MULTI>;
    constexpr int S = C::kStages;
    constexpr int TM = kBM * MT;  // rows of the CTA tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_addr(smem);
    const uint32_t bar0 = sbase + C::kOffBar;
    auto tma_full = [&](int s) { return bar0 + 8u * s; };
    auto code_full = [&](int s) { return bar0 + 8u * (S + s); };
    auto dec_full = [&](int s) { return bar0 + 8u * (2 * S + s); };
    auto empty = [&](int s) { return bar0 + 8u * (3 * S + s); };
    const uint32_t accum_full = bar0 + 8u * (4 * S);
    const uint32_t list_full = bar0 + 8u * (4 * S + 1);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 4);
    volatile int *epi_go = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 8);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t0 = (int64_t)blockIdx.x * NT * p.BN;  // NT accumulators of BN tokens each
    const int64_t m0 = (int64_t)blockIdx.y * TM;
    // MULTI: the cluster's CTAs share the K steps (and the steps of chunks) of one tile
    const int ks = MULTI ? (int)gridDim.z : 1, kz = MULTI ? (int)blockIdx.z : 0;
    const int k0 = MULTI ? p.KT * kz / ks : 0;                              // this CTA's first weight step
    const int nweight = MULTI ? p.KT * (kz + 1) / ks - k0 : p.KT;           // and how many it has
    const int nsteps = nweight + (MULTI ? 0 : p.RT);
    // MULTI: the tile's adapters
    uint32_t *s_list = reinterpret_cast<uint32_t *>(smem + C::kOffList);  // adapter | rank << 12 | sub-tiles << 24
    int16_t *s_tok = reinterpret_cast<int16_t *>(s_list + C::kTok);
    int16_t *s_place = s_tok + C::kTok;
    volatile int *s_count = reinterpret_cast<volatile int *>(s_place + QLN_MAX_ADAPTERS);  // adapters of the tile
    volatile int *s_bad = s_count + 1;                                                     // a factor is not finite
    // The chunks in their order, for a whole warp.  A batch covers E = 2^k entries of the list (all of them, up to 32)
    // and 32 / E columns-of-16; lane i holds its i-th chunk: entry | (first column / 16) << 26.
    struct Chunks {
        int na, E, e0, j0, cnt, pos, batch, step;  // batch: its number; step: of all steps of chunks
        uint32_t d, mask;  // mask: which of the batch's E x 32 / E places are chunks
    };
    auto refill = [&](Chunks &k) -> bool {  // to the next batch with a chunk; false past the last
        for (;;) {
            k.e0 += k.E;
            if (k.e0 >= k.na) {
                k.e0 = 0;
                k.j0 += 16 * (32 / k.E);
                if (k.j0 >= mp.r) return false;
            }
            const int e = k.e0 + (lane & (k.E - 1)), j = k.j0 + 16 * (lane / k.E);
            const uint32_t own = (e < k.na ? s_list[e] : 0u) | (uint32_t)(j >> 4) << 26;
            const uint32_t mask = __ballot_sync(0xffffffffu, (int)((own >> 12) & 0xffu) > j && j < mp.r);
            if (!mask) continue;
            int src = 0;  // the lane of the mask's lane-th bit
#pragma unroll
            for (int h = 16; h > 0; h >>= 1)
                if (__popc(mask & ((1u << (src + h)) - 1u)) <= lane) src += h;
            k.d = __shfl_sync(0xffffffffu, own, src);
            k.mask = mask;
            k.cnt = __popc(mask);
            k.pos = 0;
            ++k.batch;
            return true;
        }
    };
    auto begin = [&](Chunks &k) -> bool {
        k.na = *s_count;
        k.E = k.na <= 1 ? 1 : (k.na > 16 ? 32 : 1 << (32 - __clz(k.na - 1)));
        k.e0 = -k.E;
        k.j0 = k.batch = k.step = 0;
        return k.na > 0 && refill(k);
    };
    auto take = [&](Chunks &k, uint32_t (&ent)[4]) -> bool {  // the next step's chunks (0: none); whether more follow
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t d = __shfl_sync(0xffffffffu, k.d, (k.pos + q) & 31);
            ent[q] = k.pos + q < k.cnt ? d : 0u;
        }
        k.pos += 4;
        ++k.step;
        return k.pos < k.cnt || refill(k);
    };
    auto skip = [&](Chunks &k, bool more) -> bool {  // past the steps of the cluster's other CTAs
        while (more && k.step % ks != kz) {
            ++k.step;
            k.pos += 4;
            more = k.pos < k.cnt || refill(k);
        }
        return more;
    };
    auto ent_who = [](uint32_t d) { return (int)(d & 0xfffu); };
    auto ent_col = [](uint32_t d) { return (int)(d >> 26) * 16; };
    auto ent_left = [](uint32_t d) { return (int)((d >> 12) & 0xffu) - (int)(d >> 26) * 16; };  // columns to the rank's end
    constexpr uint32_t kAChunk = 4096u * MT;               // TM rows of 32 bytes
    const uint32_t bchunk = (uint32_t)(NT * p.BN) * 32u;   // the tile's tokens, 32 bytes each
    if (MULTI)
        for (int i = threadIdx.x; i < QLN_MAX_ADAPTERS; i += C::kThreads) s_place[i] = -1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(tma_full(s), 1);
            mbar_init(code_full(s), 1);
            mbar_init(dec_full(s), C::kDecThreads);
            mbar_init(empty(s), 1);
        }
        mbar_init(accum_full, 1);
        *abort_flag = 0;
        if (MULTI) {
            mbar_init(list_full, 1);
            *s_bad = 0;
        }
        mbar_fence_init();
        tma_prefetch_map(&tm_codes);
        tma_prefetch_map(&tm_act);
        tma_prefetch_map(&tm_lw);
        if (!MULTI) tma_prefetch_map(&tm_lact);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_d = *tmem_slot;
    // Barriers, descriptors and TMEM are set up while the previous kernel on
    // the stream finishes; every global access comes after this wait.
    if (!MULTI) {
        qln::pdl_wait();
        qln::pdl_trigger();
    }

    auto give_up = [&]() {
        *abort_flag = 1;
        atomicExch(p.status, (int)QLN_ERR_TIMEOUT);
    };

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        int issued = 0;
        if (lane == 0) {
            const uint32_t bsub = (uint32_t)p.BN * kBK * 2;  // one token sub-tile
            const uint32_t bbytes = NT * bsub;
            for (int kt = 0; kt < nsteps; ++kt) {
                const int s = kt % S;
                const uint32_t ph = (uint32_t)(kt / S) & 1u;
                if (!mbar_wait_bounded(empty(s), ph ^ 1u, abort_flag, kWaitLimitNs)) {
                    give_up();
                    break;
                }
                const uint32_t sA = sbase + C::kOffA + s * C::kABytes;
                const uint32_t sB = sbase + C::kOffB + s * C::kBBytes;
                const uint32_t sC = sbase + C::kOffC + s * C::kCBytes;
                if (kt < nweight) {
                    mbar_arrive_expect_tx(code_full(s), C::kCBytes);
                    if (!TRANS) {  // TM rows x 32 bytes
                        tma_load_2d(sC, &tm_codes, (k0 + kt) * 32, (int32_t)m0, code_full(s));
                    } else {       // 2*MT boxes of 64 rows x 32 bytes: [column block][row][32 B]
#pragma unroll
                        for (int d = 0; d < 2 * MT; ++d)
                            tma_load_2d(sC + 2048 * d, &tm_codes, (int32_t)(m0 / 2) + 32 * d, (k0 + kt) * kBK, code_full(s));
                    }
                    mbar_arrive_expect_tx(tma_full(s), bbytes);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        tma_load_2d(sB + nt * bsub, &tm_act, (k0 + kt) * kBK, (int32_t)(t0 + nt * p.BN), tma_full(s));
                } else {
                    const int a = kt - p.KT;
                    mbar_arrive_expect_tx(tma_full(s), C::kABytes + bbytes);
                    if (!TRANS) {
                        tma_load_2d(sA, &tm_lw, a * kBK, (int32_t)m0, tma_full(s));  // TM rows x 64
                    } else {
#pragma unroll
                        for (int d = 0; d < 2 * MT; ++d)
                            tma_load_2d(sA + 8192 * d, &tm_lw, (int32_t)m0 + 64 * d, a * kBK, tma_full(s));
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        tma_load_2d(sB + nt * bsub, &tm_lact, a * kBK, (int32_t)(t0 + nt * p.BN), tma_full(s));
                }
                issued = kt + 1;
            }
        }
        if constexpr (MULTI) {
            bool ok = true;
            if (lane == 0) {
                qln::pdl_wait();  // s U or s G is there
                qln::pdl_trigger();
                ok = issued == nsteps && mbar_wait_bounded(list_full, 0, abort_flag, kWaitLimitNs);
                if (!ok) give_up();
            }
            issued = __shfl_sync(0xffffffffu, issued, 0);
            __syncwarp();  // the list, which lane 0 has waited for
            Chunks k;
            bool more = __shfl_sync(0xffffffffu, ok, 0) && begin(k);
            while ((more = skip(k, more))) {
                const int s = issued % S;
                const uint32_t sA = sbase + C::kOffA + s * C::kABytes;
                uint32_t ent[4];
                more = take(k, ent);
                if (lane == 0) {
                    ok = mbar_wait_bounded(empty(s), ((uint32_t)(issued / S) & 1u) ^ 1u, abort_flag, kWaitLimitNs);
                    if (ok) {
                        mbar_arrive_expect_tx(tma_full(s), (1 + (ent[1] != 0) + (ent[2] != 0) + (ent[3] != 0)) * kAChunk);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if (!ent[q]) break;
                            const int who = ent_who(ent[q]), col = ent_col(ent[q]);
                            if (!TRANS) {
                                tma_load_3d(sA + q * kAChunk, &tm_lw, col, (int32_t)m0, who, tma_full(s));
                            } else {
#pragma unroll
                                for (int d = 0; d < 2 * MT; ++d)
                                    tma_load_3d(sA + 8192 * d + 2048 * q, &tm_lw, (int32_t)m0 + 64 * d, col, who, tma_full(s));
                            }
                        }
                    } else {
                        give_up();
                    }
                }
                if (!__shfl_sync(0xffffffffu, ok, 0)) break;
                ++issued;
            }
        }
        if (lane == 0) {
            // Drain: every issued copy has landed before the CTA may exit.
            for (int kt = (issued > S ? issued - S : 0); kt < issued; ++kt) {
                const int s = kt % S;
                const uint32_t ph = (uint32_t)(kt / S) & 1u;
                if (!mbar_wait_bounded(tma_full(s), ph, nullptr, kWaitLimitNs)) give_up();
                if (kt < nweight && !mbar_wait_bounded(code_full(s), ph, nullptr, kWaitLimitNs)) give_up();
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if constexpr (MULTI) {
            // the tile's adapters, in the order of their first tokens
            int id[(C::kTok + 31) / 32];
            const int ntok = NT * p.BN;
#pragma unroll
            for (int i = 0; i < (C::kTok + 31) / 32; ++i) {
                const int k = 32 * i + lane;
                const int a = k < ntok && t0 + k < p.n ? __ldg(mp.ids + t0 + k) : -1;
                id[i] = (unsigned)a < (unsigned)mp.count ? a : -1;
                if (k < ntok) s_tok[k] = (int16_t)id[i];
            }
            int na = 0;
#pragma unroll
            for (int i = 0; i < (C::kTok + 31) / 32; ++i) {
                const uint32_t same = __match_any_sync(0xffffffffu, id[i]);
                const uint32_t first = __ballot_sync(0xffffffffu, 32 * i + lane < p.BN);  // tokens of sub-tile 0
                const bool lead = id[i] >= 0 && (same & ((1u << lane) - 1u)) == 0;
                int at = lead ? s_place[id[i]] : 0;
                const uint32_t fresh = __ballot_sync(0xffffffffu, lead && at < 0);
                if (lead) {
                    const uint32_t subs = ((same & first) ? 1u << 24 : 0u) | ((same & ~first) ? 1u << 25 : 0u);
                    if (at < 0) {
                        at = na + __popc(fresh & ((1u << lane) - 1u));
                        s_place[id[i]] = (int16_t)at;
                        const int k = mp.rank ? __ldg(mp.rank + id[i]) : mp.r;
                        s_list[at] = (uint32_t)id[i] | (uint32_t)min(max(k, 0), mp.r) << 12 | subs;
                    } else {
                        s_list[at] |= subs;
                    }
                }
                na += __popc(fresh);
                __syncwarp();
            }
            if (lane == 0) {
                *s_count = na;
                mbar_arrive(list_full);  // release: the list above is visible to its waiters
            }
            __syncwarp();
        }
        // The whole warp runs the loop and one lane issues: the descriptors are warp-uniform values then, which is how the
        // instruction takes them.
        const uint32_t idesc = idesc_bf16_f32(kBM, p.BN, TRANS, false);
        const uint64_t adesc0 = smem_desc_sw128(sbase + C::kOffA, TRANS ? 8192 : 16, 1024);
        const uint64_t bdesc0 = smem_desc_sw128(sbase + C::kOffB, 16, 1024);
        int s = 0;
        uint32_t ph = 0;
        for (int kt = 0; kt < nsteps; ++kt) {
            const bool ok = mbar_wait_bounded(tma_full(s), ph, abort_flag, kWaitLimitNs) &&
                            mbar_wait_bounded(dec_full(s), ph, abort_flag, kWaitLimitNs);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) give_up();
                break;
            }
            tc_fence_after();
            const uint64_t ad = adesc0 + (uint32_t)s * (C::kABytes >> 4), bd = bdesc0 + (uint32_t)s * (C::kBBytes >> 4);
            if (lane == 0) {
#pragma unroll
                for (int sub = 0; sub < MT; ++sub) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int k = 0; k < kBK / 16; ++k) {
                            // K-major: next 16 K elements are 32 bytes further inside the
                            // swizzled 128-byte rows.  MN-major: next two 8-row K groups.
                            tc_mma_ss(tmem_d + (sub * NT + nt) * 256, ad + ((sub * 16384 + k * (TRANS ? 2048 : 32)) >> 4),
                                      bd + (uint32_t)(nt * p.BN * 8) + (k * 32 >> 4), idesc, (kt | k) != 0 ? 1u : 0u);
                        }
                    }
                }
                tc_commit(empty(s));
            }
            __syncwarp();
            if (++s == S) {
                s = 0;
                ph ^= 1u;
            }
        }
        if constexpr (MULTI) {
            __syncwarp();
            Chunks k;
            bool more = begin(k);
            for (int kt = nsteps; (more = skip(k, more)); ++kt) {
                const int s = kt % S;
                const uint32_t ph = (uint32_t)(kt / S) & 1u;
                uint32_t ent[4];
                more = take(k, ent);
                bool ok = true;
                if (lane == 0) {
                    ok = mbar_wait_bounded(tma_full(s), ph, abort_flag, kWaitLimitNs) &&
                         mbar_wait_bounded(dec_full(s), ph, abort_flag, kWaitLimitNs);
                    if (ok) {
                        tc_fence_after();
                        const uint32_t sA = sbase + C::kOffA + s * C::kABytes;
                        const uint32_t sB = sbase + C::kOffB + s * C::kBBytes;
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                if (!((ent[q] >> (24 + nt)) & 1u)) continue;  // none of its tokens, or no chunk
                                const uint64_t bdesc = smem_desc_sw32(sB + q * bchunk + nt * p.BN * 32);
#pragma unroll
                                for (int sub = 0; sub < MT; ++sub) {
                                    const uint64_t adesc = TRANS ? smem_desc_sw128(sA + sub * 16384 + q * 2048, 8192, 1024)
                                                                 : smem_desc_sw32(sA + q * kAChunk + sub * 4096);
                                    tc_mma_ss(tmem_d + (sub * NT + nt) * 256, adesc, bdesc, idesc, 1u);
                                }
                            }
                        tc_commit(empty(s));
                    } else {
                        give_up();
                    }
                }
                if (!__shfl_sync(0xffffffffu, ok, 0)) break;
            }
        }
        if (lane == 0) {
            tc_commit(accum_full);
        }
    } else {
        // ------------------------------------------------------------ decoders
        // One thread per 64-wide row block of the A tile.
        //   fwd: block = W row m0 + dt, column block kt.
        //   dX : block = W row 64*kt + dt%64, column block m0/64 + dt/64.
        const int dt = threadIdx.x - 64;
        const int64_t bpr = p.cols / 64;
        const int db = dt & (128 * MT - 1), share = dt / (128 * MT);  // block, and which of its threads
        const int drow = TRANS ? (db & 63) : db;
        const int dcol = TRANS ? (db >> 6) : 0;
        const float mu = p.qabs ? __ldg(p.dq_mean) : 0.f;
        auto block_index = [&](int kt) -> int64_t {
            return TRANS ? ((int64_t)kt * kBK + drow) * bpr + (m0 / 64) + dcol : (m0 + drow) * bpr + kt;
        };
        // Raw block constants are fetched two k-steps before use so that their
        // L2 latency hides behind the decode of the steps in between.
        struct Raw {
            float v;     // absmax (plain) or DQ scale b_g
            int32_t q;   // DQ code rhat_j
        };
        auto fetch = [&](int kt) -> Raw {
            Raw r{0.f, 0};
            if (kt < nweight) {
                const int64_t jb = block_index(k0 + kt);
                if (p.qabs) {
                    r.q = __ldg(p.qabs + jb);
                    r.v = __ldg(p.dq_scale + (jb >> 8));
                } else {
                    r.v = __ldg(p.absmax + jb);
                }
            }
            return r;
        };
        Raw r0 = fetch(share), r1 = fetch(share + C::kShare);
        // This thread's 32 code bytes sit at a 32-byte stride; the two 16-byte
        // halves are read in an order that keeps each 8-thread phase on
        // distinct banks (half `cfirst` first).
        const uint32_t cfirst = (drow >> 2) & 1;
        const uint32_t code_off = (TRANS ? dcol * 2048 : 0) + drow * 32;
        const uint32_t r8 = drow & 7;
        // fwd (K-major): row drow at (drow/8)*1024 + (drow%8)*128, chunk c (K 8c..8c+7).
        // dX (MN-major): atom (dcol, drow/8) at dcol*8192 + (drow/8)*1024, K-row drow%8,
        //   chunk c = M elements 8c..8c+7.  Both: chunk c at byte (c ^ (row % 8)) * 16
        // of the row.  Bits 4-6 of the row's address are zero, so the chunk
        // address is (row address + 16*r8) XOR 16*c; the half read first
        // holds chunks 4*cfirst.. , folded into the XOR base as well.
        const uint32_t row_off = (TRANS ? dcol * 8192 : 0) + (drow >> 3) * 1024 + r8 * 128;
        const uint32_t sA0 = smem_addr(smem + C::kOffA) + row_off + (r8 << 4);
        // A group that takes every second step leaves out phases of the barriers; it never falls two behind one, since the
        // MMAs end in their order and it has waited for one of the last S + 2 steps.
        for (int kt = share; kt < nsteps; kt += C::kShare) {
            const int s = kt % S;
            const uint32_t ph = (uint32_t)(kt / S) & 1u;
            const float ah = p.qabs ? dq_restore((uint32_t)r0.q, r0.v, mu, p.e4m3) : r0.v;
            r0 = r1;
            r1 = fetch(kt + 2 * C::kShare);
            if (!mbar_wait_bounded(empty(s), ph ^ 1u, abort_flag, kWaitLimitNs)) {
                give_up();
                break;
            }
            if (kt < nweight) {
                if (!mbar_wait_bounded(code_full(s), ph, abort_flag, kWaitLimitNs)) {
                    give_up();
                    break;
                }
                const uint8_t *cptr = smem + C::kOffC + s * C::kCBytes + code_off;
                const uint4 ca = *reinterpret_cast<const uint4 *>(cptr + 16 * cfirst);
                const uint4 cb = *reinterpret_cast<const uint4 *>(cptr + 16 * (cfirst ^ 1));
                const NF4Table tab = nf4_table(ah);
                const uint32_t xa = (sA0 + s * C::kABytes) ^ (cfirst << 6);  // chunks of ca: 4*cfirst + i
                const uint32_t xb = xa ^ 64u;                                  // chunks of cb
                st_shared_v4(xa ^ 0u, nf4_decode8(ca.x, tab));
                st_shared_v4(xa ^ 16u, nf4_decode8(ca.y, tab));
                st_shared_v4(xa ^ 32u, nf4_decode8(ca.z, tab));
                st_shared_v4(xa ^ 48u, nf4_decode8(ca.w, tab));
                st_shared_v4(xb ^ 0u, nf4_decode8(cb.x, tab));
                st_shared_v4(xb ^ 16u, nf4_decode8(cb.y, tab));
                st_shared_v4(xb ^ 32u, nf4_decode8(cb.z, tab));
                st_shared_v4(xb ^ 48u, nf4_decode8(cb.w, tab));
                fence_proxy_async_smem();
            }
            mbar_arrive_n(dec_full(s), C::kShare);
        }
        if constexpr (MULTI) {
            if (!*abort_flag && !mbar_wait_bounded(list_full, 0, abort_flag, kWaitLimitNs)) give_up();
            qln::pdl_wait();  // s U or s G is there
            constexpr int kRows = (C::kTok + C::kDecThreads - 1) / C::kDecThreads;
            // This thread's tokens: their adapters' places in the list (-1: none); the next chunk of the batch that is
            // theirs, as its place and its number (kNone: none left); and the chunks of each stage that hold values of
            // them (4 bits a stage).
            constexpr int kNone = 1 << 20;
            int place[kRows], at[kRows], num[kRows], batch = -1;
            uint32_t held[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int row = dt + i * C::kDecThreads, tok = row < NT * p.BN ? s_tok[row] : -1;
                place[i] = tok >= 0 ? s_place[tok] : -1;
                held[i] = 0u;
            }
            Chunks k{};
            auto seek = [&](int i, int to) {  // token i's chunk at the batch's place `to`, or none
                at[i] = to;
                num[i] = to < 32 && ((k.mask >> to) & 1u) ? __popc(k.mask & ((1u << to) - 1u)) : kNone;
            };
            // B_op of the next step, kt: s U or s G of each chunk's own tokens (asynchronous copies), zeros for the
            // others.  A stage is cleared on its first use; later, only what its last step held is.
            auto put = [&](int kt) {
                const int s = kt % S, step = k.pos >> 2;
                const uint32_t sB = sbase + C::kOffB + s * C::kBBytes;
                if (batch != k.batch) {
                    batch = k.batch;
#pragma unroll
                    for (int i = 0; i < kRows; ++i) {
                        const int to = place[i] - k.e0;
                        seek(i, place[i] >= 0 && to >= 0 && to < k.E ? to : 32);
                    }
                }
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    if (i * C::kDecThreads >= NT * p.BN) break;  // no rows left
                    const int row = dt + i * C::kDecThreads;
                    uint32_t old = (held[i] >> (4 * s)) & 15u, now = 0u;
                    if (kt - nsteps < S) old = row < NT * p.BN ? 15u : 0u;
                    const uint32_t to = sB + row * 32 + (((row >> 2) & 1) << 4);  // 32-byte swizzle: halves at `to` and to ^ 16
                    while ((num[i] >> 2) < step) seek(i, at[i] + k.E);  // chunks of the cluster's other CTAs
                    while ((num[i] >> 2) == step) {
                        const int q = num[i] & 3, j = k.j0 + 16 * (at[i] / k.E);
                        const uint16_t *src = mp.lact + (t0 + row) * mp.r + j;
                        const int half2 = j + 8 < mp.r ? 16 : 0;  // r = 8: the second half is zero
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to + q * bchunk), "l"(src) : "memory");
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"((to + q * bchunk) ^ 16u),
                                     "l"(half2 ? src + 8 : src), "r"(half2)
                                     : "memory");
                        now |= 1u << q;
                        seek(i, at[i] + k.E);
                    }
                    held[i] = (held[i] & ~(15u << (4 * s))) | now << (4 * s);
                    for (old &= ~now; old; old &= old - 1) {
                        const uint32_t d = to + (__ffs(old) - 1) * bchunk;
                        st_shared_v4(d, make_uint4(0u, 0u, 0u, 0u));
                        st_shared_v4(d ^ 16u, make_uint4(0u, 0u, 0u, 0u));
                    }
                }
                qln::cp_async_commit();
            };
            // the stage's MMAs of S steps before have read it
            auto free_stage = [&](int kt) -> bool {
                const bool ok = mbar_wait_bounded(empty(kt % S), ((uint32_t)(kt / S) & 1u) ^ 1u, abort_flag, kWaitLimitNs);
                if (!ok) give_up();
                return __all_sync(0xffffffffu, ok);
            };
            // One step is written while the copies of the one before are on their way.  ent: its chunks, nq their count;
            // with equal ranks only the count is needed (nothing lies past a rank but the map's own zeros).
            uint32_t ent[4] = {0u, 0u, 0u, 0u}, nxt[4] = {0u, 0u, 0u, 0u};
            int nq = 0, nxq = 0;
            bool more = __all_sync(0xffffffffu, !*abort_flag) && begin(k);
            more = skip(k, more);
            auto advance = [&](int kt) -> bool {  // puts step kt and moves on
                if (!free_stage(kt)) return false;
                put(kt);
                nxq = min(4, k.cnt - k.pos);
                if (mp.rank) {
                    more = take(k, nxt);
                } else {
                    k.pos += 4;
                    ++k.step;
                    more = k.pos < k.cnt || refill(k);
                }
                more = skip(k, more);
                return true;
            };
            bool live = more && advance(nsteps);
            for (int kt = nsteps; live; ++kt) {
                const int s = kt % S;
                nq = nxq;
#pragma unroll
                for (int q = 0; q < 4; ++q) ent[q] = nxt[q];
                live = more;
                if (more) {
                    if (!advance(kt + 1)) break;
                    qln::cp_async_wait<1>();
                } else {
                    qln::cp_async_wait<0>();
                }
                const bool ok = mbar_wait_bounded(tma_full(s), (uint32_t)(kt / S) & 1u, abort_flag, kWaitLimitNs);
                if (!ok) give_up();
                if (!__all_sync(0xffffffffu, ok)) break;
                // The factors' chunks: zero past the rank, and where they are not finite.  A thread takes the
                // columns of one m in all chunks (32 bytes each), or one row j of a chunk (128 bytes of m).
                uint8_t *sA = smem + C::kOffA + s * C::kABytes;
                const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
                // x 0 added up: NaN exactly if an element is not finite
                __nv_bfloat162 o0 = zero, o1 = zero, o2 = zero, o3 = zero;
                auto look = [&](const uint4 &v) {
                    o0 = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&v.x), zero, o0);
                    o1 = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&v.y), zero, o1);
                    o2 = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&v.z), zero, o2);
                    o3 = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&v.w), zero, o3);
                };
                auto odd = [&]() { return __hadd2(__hadd2(o0, o1), __hadd2(o2, o3)); };
                auto is_odd = [](const __nv_bfloat162 &v) { return __hisnan(__low2bfloat16(v)) || __hisnan(__high2bfloat16(v)); };
                auto clear = [](uint4 *q, int n) {  // the non-finite of n vectors of 8: to 1 or -1
                    uint16_t *w = reinterpret_cast<uint16_t *>(q);
                    for (int h = 0; h < 8 * n; ++h)
                        if ((w[h] & 0x7f80u) == 0x7f80u) w[h] = (uint16_t)((w[h] & 0x8000u) | 0x3f80u);
                };
                bool bad = false;
                if (!TRANS) {
                    // row drow: its two 16-byte halves change places where bit 7 of the address is set; the threads of
                    // a row share its chunks
                    constexpr int kQ = 4 / C::kShare;
                    const int q0 = share * kQ;
                    uint4 *row = reinterpret_cast<uint4 *>(sA + q0 * kAChunk + drow * 32);
                    if (mp.rank) {
                        const int swap = (drow >> 2) & 1;
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            for (int h = ent[q] && q / kQ == share ? ent_left(ent[q]) : 16; h < 16; ++h)
                                reinterpret_cast<uint16_t *>(row + (q % kQ) * (kAChunk / 16) + ((h >> 3) ^ swap))[h & 7] = 0;
                    }
                    uint4 v[kQ][2];
#pragma unroll
                    for (int q = 0; q < kQ; ++q)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            v[q][h] = q0 + q < nq ? row[q * (kAChunk / 16) + h] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int q = 0; q < kQ; ++q) {
                        look(v[q][0]);
                        look(v[q][1]);
                    }
                    if (is_odd(odd())) {
                        bad = true;
#pragma unroll
                        for (int q = 0; q < kQ; ++q)
                            if (q0 + q < nq) clear(row + q * (kAChunk / 16), 2);
                    }
                } else {
                    constexpr int kV = 8 / C::kShare;  // of a row's eight 16-byte pieces
                    const int q = drow >> 4;
                    uint4 *row = reinterpret_cast<uint4 *>(sA + dcol * 8192 + drow * 128);
                    const uint32_t e = q == 0 ? ent[0] : q == 1 ? ent[1] : q == 2 ? ent[2] : ent[3];
                    if (q < nq) {
                        if (mp.rank && (drow & 15) >= ent_left(e)) {  // past the rank
#pragma unroll
                            for (int c = 0; c < kV; ++c) row[(share * kV + c) ^ r8] = make_uint4(0u, 0u, 0u, 0u);
                        } else {
                            uint4 v[kV];
#pragma unroll
                            for (int c = 0; c < kV; ++c) v[c] = row[(share * kV + c) ^ r8];
#pragma unroll
                            for (int c = 0; c < kV; ++c) look(v[c]);
                            if (is_odd(odd())) {
                                bad = true;
                                for (int c = 0; c < kV; ++c) clear(row + ((share * kV + c) ^ r8), 1);
                            }
                        }
                    }
                }
                if (bad) *s_bad = 1;
                fence_proxy_async_smem();
                mbar_arrive(dec_full(s));
            }
            qln::cp_async_wait<0>();
        }

        // ------------------------------------------------------------ epilogue
        // The go / no-go decision is made uniform across the decoder threads
        // (tcgen05.ld is warp-collective, named barrier 1 counts all of them).
        if (*abort_flag || !mbar_wait_bounded(accum_full, 0, abort_flag, kWaitLimitNs)) give_up();
        asm volatile("bar.sync 1, %0;" ::"n"(C::kDecThreads) : "memory");
        if (dt == 0) *epi_go = *abort_flag ? 0 : 1;
        asm volatile("bar.sync 1, %0;" ::"n"(C::kDecThreads) : "memory");
        if (*epi_go && ks == 1) {
            tc_fence_after();
            const int q = warp & 3;              // TMEM lane quadrant of this warp
            const int sub = MT == 2 ? ((warp - 2) >> 2) & 1 : 0;    // weight sub-tile of this warp
            const int part = ((warp - 2) >> 2) / MT;                // which of the warps of its quadrant it is
            uint16_t *Os = reinterpret_cast<uint16_t *>(smem);  // [NT*BN][TM] bf16; all MMAs are done
            const int m = sub * kBM + q * 32 + lane;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                for (int c0 = 0; c0 < p.BN; c0 += 32) {
                    if (C::kShare == 2 && ((nt + c0 / 32) & 1) != part) continue;
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(tmem_d + ((uint32_t)(q * 32) << 16) + (uint32_t)((sub * NT + nt) * 256 + c0), v);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (c0 + j < p.BN)
                            Os[(nt * p.BN + c0 + j) * TM + m] =
                                __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(v[j])));
                }
            }
            if constexpr (MULTI) {
                if (*s_bad) {  // once more, with the products of the factors' non-finite elements
                    qln::pdl_wait();
                    for (int k = 0; k < NT * p.BN; ++k) {
                        const int a = s_tok[k], nt = k >= p.BN ? 1 : 0;
                        if (a < 0 || (C::kShare == 2 && ((nt + (k - nt * p.BN) / 32) & 1) != part)) continue;
                        uint32_t v;
                        asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];"
                                     : "=r"(v)
                                     : "r"(tmem_d + ((uint32_t)(q * 32) << 16) + (uint32_t)((sub * NT + nt) * 256 + k - nt * p.BN)));
                        tmem_wait_ld();
                        const float y = __uint_as_float(v) + nonfinite_products(mp, a, m0 + m, t0 + k, p.out_ld, TRANS);
                        Os[k * TM + m] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
                    }
                }
            }
            asm volatile("bar.sync 1, %0;" ::"n"(C::kDecThreads) : "memory");
            constexpr int kChunksPerRow = TM / 8;
            const int chunks = NT * p.BN * kChunksPerRow;
            for (int idx = dt; idx < chunks; idx += C::kDecThreads) {
                const int row = idx / kChunksPerRow, ch = idx % kChunksPerRow;
                const int64_t t = t0 + row;
                if (t < p.n)
                    *reinterpret_cast<uint4 *>(p.out + t * p.out_ld + m0 + 8 * ch) =
                        *reinterpret_cast<const uint4 *>(Os + row * TM + 8 * ch);
            }
        }
    }

    // K split: CTA q of the cluster finishes every cq-th part of the tile's columns (tokens).  Every CTA sends its
    // accumulators there (fp32, into the stages, which nobody uses any more), and they are added in the CTAs' order.
    if constexpr (MULTI) {
        if (ks > 1) {
            const int ntok = NT * p.BN, cq = split_cols(ntok, ks), c_lo = kz * cq, c_n = min(cq, ntok - c_lo);
            __syncthreads();
            const bool go = *epi_go != 0;
            cluster_sync();  // every CTA's copies have landed, its MMAs have retired
            if (warp >= 2 && go) {
                // Eight columns at a time in a short loop: this code runs once, and unrolled over 32 columns its
                // instructions took longer to fetch (8 us) than its data to move.
                tc_fence_after();
                const int q = warp & 3, sub = MT == 2 ? ((warp - 2) >> 2) & 1 : 0, part = ((warp - 2) >> 2) / MT;
                const uint32_t mine = sbase + (uint32_t)((kz * cq) * TM + sub * kBM + q * 32 + lane) * 4u;
#pragma unroll 1
                for (int col = 8 * part; col < ntok; col += 8 * C::kShare) {
                    const int nt = NT == 2 && col >= p.BN ? 1 : 0, to = col / cq;
                    uint32_t v[8];
                    tmem_ld_32x32b_x8(tmem_d + ((uint32_t)(q * 32) << 16) + (uint32_t)((sub * NT + nt) * 256 + col - nt * p.BN), v);
                    const uint32_t d = cluster_map(mine + (uint32_t)((col - to * cq) * TM) * 4u, (uint32_t)to);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j) cluster_st_u32(d + j * TM * 4u, v[j]);
                }
                tc_fence_before();
                if (threadIdx.x == 64 && *s_bad)
                    for (int z = 0; z < ks; ++z)
                        cluster_st_u32(cluster_map(smem_addr(const_cast<const int *>(s_bad)), (uint32_t)z), 1u);
            }
            __syncwarp();
            cluster_sync();  // all parts are here
            if (warp >= 2 && go) {
                const float *part_s = reinterpret_cast<const float *>(smem);
                const bool bad = *s_bad != 0;
                constexpr int kCh = TM / 8;
                for (int idx = threadIdx.x - 64; idx < c_n * kCh; idx += C::kDecThreads) {
                    const int col = idx / kCh, m = (idx % kCh) * 8, k = c_lo + col;
                    const int64_t t = t0 + k;
                    if (t >= p.n) continue;
                    float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                    for (int z = 0; z < ks; ++z) {
                        const float4 *src = reinterpret_cast<const float4 *>(part_s + (z * cq + col) * TM + m);
                        const float4 u = src[0], w = src[1];
                        y[0] += u.x, y[1] += u.y, y[2] += u.z, y[3] += u.w;
                        y[4] += w.x, y[5] += w.y, y[6] += w.z, y[7] += w.w;
                    }
                    if (bad && s_tok[k] >= 0)
                        for (int j = 0; j < 8; ++j) y[j] += nonfinite_products(mp, s_tok[k], m0 + m + j, t, p.out_ld, TRANS);
                    *reinterpret_cast<uint4 *>(p.out + t * p.out_ld + m0 + m) =
                        make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
                }
            }
        }
    }

    // Teardown: all MMAs must have retired before TMEM is released.
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        if (lane == 0 && !mbar_wait_bounded(accum_full, 0, nullptr, kWaitLimitNs)) give_up();
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_d, C::kTmemCols);
    }
}

// ---------------------------------------------------------------------------
// Host side: tensor maps (driver entry point fetched through the runtime, so
// the library does not link libcuda), tile-shape choice, launch.
// ---------------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    }
    return fn;
}

// 3D map over a row-major bf16 [outer][mid][inner] array, boxes of one outer index.
static bool make_map_3d(CUtensorMap *m, const void *base, uint64_t inner, uint64_t mid, uint64_t outer,
                        uint32_t box_inner, uint32_t box_mid, CUtensorMapSwizzle sw) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {inner, mid, outer};
    cuuint64_t strides[2] = {inner * 2, inner * mid * 2};
    cuuint32_t box[3] = {box_inner, box_mid, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2D map over a row-major [outer][inner] array.
static bool make_map(CUtensorMap *m, CUtensorMapDataType dt, int esize, const void *base, uint64_t inner,
                     uint64_t outer, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle sw) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {inner, outer};
    cuuint64_t strides[1] = {inner * (uint64_t)esize};
    cuuint32_t box[2] = {box_inner, box_outer};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, dt, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tc

bool make_tensor_map_2d(CUtensorMap *m, CUtensorMapDataType dt, int esize, const void *base, uint64_t inner,
                        uint64_t outer, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle sw) {
    return tc::make_map(m, dt, esize, base, inner, outer, box_inner, box_outer, sw);
}

namespace tc {

// Tile shape per call.  Candidates: MT weight sub-tiles of 128 rows and NT
// token sub-tiles of BN tokens (MT * NT <= 2, BN a multiple of 16).  A simple
// cost model picks the fastest: one CTA per SM; a k-step costs the larger of
// its tensor time (at the measured dense rate, about 5700 FLOP per cycle per
// SM) and its decode time (about 0.12 cycle per decoded weight, integer-pipe
// bound), plus a fixed cost per tile; waves are counted whole.
struct TileShape {
    int MT, NT, BN;
};

static TileShape choose_shape(int64_t M, int64_t K, int64_t n, int num_sms) {
    const int64_t ksteps = K / kBK + 1;
    TileShape best{1, 1, 128};
    double best_cost = 1e300;
    const int shapes[3][2] = {{2, 1}, {1, 2}, {1, 1}};
    for (const auto &sh : shapes) {
        const int MT = sh[0], NT = sh[1];
        if ((M % (kBM * MT)) != 0) continue;
        const int maxbn = NT == 1 ? 256 : 208;
        for (int bn = maxbn; bn >= 16; bn -= 16) {
            if (bn < 128 && (int64_t)NT * bn < n) break;  // narrow tiles only for small n
            const int64_t tile_tok = (int64_t)NT * bn;
            const int64_t ttiles = (n + tile_tok - 1) / tile_tok;
            const int64_t tiles = ttiles * (M / (kBM * MT));
            const int64_t rounds = (tiles + num_sms - 1) / num_sms;
            const double mma = 2.0 * kBM * MT * tile_tok * kBK / 5700.0;
            const double dec = 0.12 * 8192.0 * MT;
            const double tile = ksteps * (mma > dec ? mma : dec) + 4000.0;
            // ties go to the fewest padded tokens
            const double cost = rounds * tile * (1.0 + 1e-4 * (double)(ttiles * tile_tok - n) / (double)n);
            if (cost < best_cost * 0.999) {
                best_cost = cost;
                best = TileShape{MT, NT, bn};
            }
        }
    }
    return best;
}

// Tile shape and K split of a MULTI call, by a cost in cycles that was fitted to 274 measured calls (13 sizes, every shape;
// it meets them within 5 % and its choices are within 2 % of the best).  A k-step takes its chain of copy, decoding and
// MMA through the ring plus 0.18 of its tensor time, or the tensor time where that is more; a tile its start and, per
// column, its epilogue; a split the exchange, and in four slower steps besides.  CTAs of clusters find fewer places.
// Splitting fills the SMs where there are few tiles: 4096 x 4096 and 64 tokens, rank 16: 21 us split in three, 37 us
// unsplit; 333 tokens: 33 us split in two, 40 us unsplit.
struct MultiShape {
    TileShape t;
    int ks;
};

static MultiShape choose_multi(int64_t M, int64_t K, int64_t n, int num_sms) {
    const int KT = (int)(K / kBK);
    MultiShape best{{1, 1, 128}, 1};
    double best_cost = 1e300;
    const int shapes[3][2] = {{2, 1}, {1, 2}, {1, 1}};
    for (const auto &sh : shapes) {
        const int MT = sh[0], NT = sh[1];
        if ((M % (kBM * MT)) != 0) continue;
        for (int bn = NT == 1 ? 256 : 208; bn >= 16; bn -= 16) {
            if (bn < 128 && (int64_t)NT * bn < n) break;  // narrow tiles only for small n
            const int64_t tok = (int64_t)NT * bn, ttiles = (n + tok - 1) / tok, tiles = ttiles * (M / (kBM * MT));
            const int64_t less = tok - 16 * NT;  // the next narrower tile, better if as many of them cover the tokens
            if (bn > 16 && (bn > 128 || less >= n) && (n + less - 1) / less == ttiles) continue;
            for (int ks = 1; ks <= 4; ++ks) {
                // the exchange takes the stages' shared memory
                const int64_t room = MT * NT == 2 ? Cfg<2, 1, true>::kOffBar : Cfg<1, 1, true>::kOffBar;
                if (ks > 1 && (ks * 4 > KT || (int64_t)ks * split_cols((int)tok, ks) * kBM * MT * 4 > room)) continue;
                const int lost[5] = {0, 0, 4, 10, 20};
                const int64_t places = num_sms > lost[ks] + ks ? num_sms - lost[ks] : ks;
                const int64_t rounds = (tiles * ks + places - 1) / places;
                const double mma = 2.0 * kBM * MT * (double)tok * kBK / 5700.0;
                const double chain = (MT == 2 ? 1270.0 : NT == 2 ? 970.0 : 750.0) + 0.18 * mma;
                const double step = (chain > 1.05 * mma ? chain : 1.05 * mma) * (ks == 4 ? 1.2 : 1.0);
                const double cost = rounds * (((KT + ks - 1) / ks + 1) * step + 3350.0 + 43.0 * MT * (double)tok + (ks > 1 ? 5400.0 : 0.0)) *
                                    (1.0 + 1e-4 * (double)(ttiles * tok - n) / (double)n);
                if (cost < best_cost * 0.999) {
                    best_cost = cost;
                    best = MultiShape{{MT, NT, bn}, ks};
                }
            }
        }
    }
    return best;
}

template <bool TRANS, int MT, int NT, bool MULTI>
static cudaError_t launch_t(const CUtensorMap &m_codes, const CUtensorMap &m_act, const CUtensorMap &m_lw,
                            const CUtensorMap &m_lact, const Params &p, const MultiParams &mp, dim3 grid, cudaStream_t st) {
    using C = Cfg<MT, NT, MULTI>;
    constexpr uint32_t smem = MULTI ? C::kSmemBytesMulti : C::kSmemBytes;
    cudaError_t e = cudaFuncSetAttribute(nf4_tc_gemm_kernel<TRANS, MT, NT, MULTI>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (MULTI && grid.z > 1) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = grid.z;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = grid;
        cfg.blockDim = dim3(C::kThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        qln::note_launch();
        return cudaLaunchKernelEx(&cfg, nf4_tc_gemm_kernel<TRANS, MT, NT, MULTI>, m_codes, m_act, m_lw, m_lact, p, mp);
    }
    return qln::launch_pdl(nf4_tc_gemm_kernel<TRANS, MT, NT, MULTI>, grid, dim3(C::kThreads), (size_t)smem, st,
                           m_codes, m_act, m_lw, m_lact, p, mp);
}

template <bool MULTI>
static cudaError_t launch_shape(bool trans, const TileShape &sh, const CUtensorMap &m_codes, const CUtensorMap &m_act,
                                const CUtensorMap &m_lw, const CUtensorMap &m_lact, const Params &p,
                                const MultiParams &mp, dim3 grid, cudaStream_t st) {
    if (trans) {
        if (sh.MT == 2) return launch_t<true, 2, 1, MULTI>(m_codes, m_act, m_lw, m_lact, p, mp, grid, st);
        if (sh.NT == 2) return launch_t<true, 1, 2, MULTI>(m_codes, m_act, m_lw, m_lact, p, mp, grid, st);
        return launch_t<true, 1, 1, MULTI>(m_codes, m_act, m_lw, m_lact, p, mp, grid, st);
    }
    if (sh.MT == 2) return launch_t<false, 2, 1, MULTI>(m_codes, m_act, m_lw, m_lact, p, mp, grid, st);
    if (sh.NT == 2) return launch_t<false, 1, 2, MULTI>(m_codes, m_act, m_lw, m_lact, p, mp, grid, st);
    return launch_t<false, 1, 1, MULTI>(m_codes, m_act, m_lw, m_lact, p, mp, grid, st);
}

}  // namespace tc

bool nf4_tc_gemm_supported(const qln_nf4_weight *w, bool trans, int64_t n, int r) {
    const int64_t M = trans ? w->cols : w->rows;
    const int64_t K = trans ? w->rows : w->cols;
    return n >= 64 && (M % tc::kBM) == 0 && (K % tc::kBK) == 0 && r >= 8 && r <= 128 && (r % 8) == 0 &&
           tc::encode_fn() != nullptr;
}

bool nf4_tc_gemm_multi_supported(const qln_nf4_weight *w, bool trans, int r) {
    return nf4_tc_gemm_supported(w, trans, 64, r);
}

int64_t nf4_tc_gemm_ctas(const qln_nf4_weight *w, bool trans, int64_t n, int r, int num_sms) {
    if (!nf4_tc_gemm_supported(w, trans, n, r)) return 0;
    const int64_t M = trans ? w->cols : w->rows;
    const int64_t K = trans ? w->rows : w->cols;
    const tc::TileShape shape = tc::choose_shape(M, K, n, num_sms > 0 ? num_sms : 148);
    return ((n + (int64_t)shape.NT * shape.BN - 1) / ((int64_t)shape.NT * shape.BN)) * (M / (tc::kBM * shape.MT));
}

// view: null for one adapter [lw as in launch_nf4_mma_gemm], else the pool's (lw its factors' base).
static cudaError_t launch_tc(const qln_nf4_weight *w, bool trans, const uint16_t *act, int64_t n, const uint16_t *lact,
                             const uint16_t *lw, int r, const AdapterView *view, uint16_t *out, int *status,
                             cudaStream_t st, int num_sms) {
    using namespace tc;
    const int64_t rows = w->rows, cols = w->cols;
    const int64_t M = trans ? cols : rows;
    const int64_t K = trans ? rows : cols;
    const MultiShape ms = view ? choose_multi(M, K, n, num_sms > 0 ? num_sms : 148)
                               : MultiShape{choose_shape(M, K, n, num_sms > 0 ? num_sms : 148), 1};
    const TileShape shape = ms.t;
    const int NT = shape.NT, BN = shape.BN;
    const int TM = kBM * shape.MT;
    CUtensorMap m_codes, m_act, m_lw, m_lact;
    bool ok = true;
    // codes as bytes [rows][cols/2]
    if (!trans) ok &= make_map(&m_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w->codes, cols / 2, rows, 32, TM,
                               CU_TENSOR_MAP_SWIZZLE_NONE);
    else ok &= make_map(&m_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w->codes, cols / 2, rows, 32, kBK,
                        CU_TENSOR_MAP_SWIZZLE_NONE);
    ok &= make_map(&m_act, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, act, K, n, kBK, BN, CU_TENSOR_MAP_SWIZZLE_128B);
    if (view) {
        ok &= trans ? make_map_3d(&m_lw, lw, cols, r, view->count, 64, 16, CU_TENSOR_MAP_SWIZZLE_128B)   // A [count][r][cols]
                    : make_map_3d(&m_lw, lw, r, rows, view->count, 16, TM, CU_TENSOR_MAP_SWIZZLE_32B);   // B [count][rows][r]
        m_lact = m_act;  // not used
    } else {
        if (!trans) ok &= make_map(&m_lw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, lw, r, rows, kBK, TM,
                                   CU_TENSOR_MAP_SWIZZLE_128B);                       // B [rows][r]
        else ok &= make_map(&m_lw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, lw, cols, r, 64, kBK,
                            CU_TENSOR_MAP_SWIZZLE_128B);                               // A [r][cols]
        ok &= make_map(&m_lact, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, lact, r, n, kBK, BN, CU_TENSOR_MAP_SWIZZLE_128B);
    }
    if (!ok) return cudaErrorInvalidValue;

    Params p;
    p.qabs = w->qabs;
    p.e4m3 = w->dq_format == QLN_DQ_E4M3;
    p.absmax = w->absmax;
    p.dq_scale = w->dq_scale;
    p.dq_mean = w->dq_mean;
    p.cols = cols;
    p.n = n;
    p.out = out;
    p.out_ld = M;
    p.status = status;
    p.KT = (int)(K / kBK);
    p.RT = (r + kBK - 1) / kBK;
    p.BN = BN;
    dim3 grid((unsigned)((n + (int64_t)NT * BN - 1) / ((int64_t)NT * BN)), (unsigned)(M / TM), (unsigned)ms.ks);
    if (!view) return launch_shape<false>(trans, shape, m_codes, m_act, m_lw, m_lact, p, MultiParams{}, grid, st);
    const MultiParams mp{view->ids, view->rank, lact, lw, view->count, r};
    return launch_shape<true>(trans, shape, m_codes, m_act, m_lw, m_lact, p, mp, grid, st);
}

cudaError_t launch_nf4_tc_gemm(const qln_nf4_weight *w, bool trans, const uint16_t *act, int64_t n,
                               const uint16_t *lact, const uint16_t *lw, int r, uint16_t *out, int *status,
                               cudaStream_t st, int num_sms) {
    return launch_tc(w, trans, act, n, lact, lw, r, nullptr, out, status, st, num_sms);
}

cudaError_t launch_nf4_tc_gemm_multi(const qln_nf4_weight *w, bool trans, const uint16_t *act, int64_t n,
                                     const uint16_t *lact, const uint16_t *lw, int r, const AdapterView &v,
                                     uint16_t *out, int *status, cudaStream_t st, int num_sms) {
    return launch_tc(w, trans, act, n, lact, lw, r, &v, out, status, st, num_sms);
}

}  // namespace qln

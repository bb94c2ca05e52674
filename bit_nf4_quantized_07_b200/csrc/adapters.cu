// Products around a pool of adapters, where every token has an adapter of its
// own (or none): the plan that groups tokens by adapter and the products down
// to the rank.  (The gradients of the factors: adapter_grads.cu.)
//
// Method: "LoRA 与 QLoRA" section LoRA (y = W0 x + s B(A x), A x formed first;
// only A and B are trained); deck "3 QLoRA Finetuning" card 1 (gradients flow
// through the dequantized weight, only the adapters receive updates).  For
// token t with adapter a = ids[t]:
//   U_t = X_t A_a^T (forward),  G_t = dY_t B_a (backward)
// Tokens are never multiplied with another adapter's factors, not even by a
// zero: an infinity or NaN in one adapter or token stays with it.
#include "qln_common.cuh"
#include "qln_internal.h"

namespace qln {

// ===========================================================================
// Plan: a stable counting sort of the tokens by adapter, in one CTA.
//   order [n]         tokens of adapter 0, then 1, ... (ascending within one),
//                     and at the end those without an adapter (group `count`)
//   start [count + 2] first place of each group in order
//   tiles [count + 2] first 64-token tile of each group (tiles never mix)
// Warp w owns the w-th of nw contiguous token ranges and a histogram of its
// own, so places follow from two passes over the ids and one scan, and do not
// depend on timing.  Latency-bound: a few dependent reads of the ids, and loops
// over the histograms, so there are no more of them than ranges of 32 tokens.
// Alone and with cold caches 4.6 us for 203 tokens of 24 adapters, 6.2 us for
// 2048 tokens.
// ===========================================================================
constexpr int kPlanWarps = 32;

static int plan_ranges(int64_t n) { return n >= 32 * kPlanWarps ? kPlanWarps : (int)((n + 31) / 32); }

__global__ void __launch_bounds__(kPlanWarps * 32) adapter_plan_kernel(const int32_t *__restrict__ ids, int n, int count, int nw,
                                                                       int32_t *__restrict__ order,
                                                                       int32_t *__restrict__ start,
                                                                       int32_t *__restrict__ tiles, int *status) {
    extern __shared__ int hist[];  // [nw][count]
    __shared__ int wsum[2][kPlanWarps], s_none[kPlanWarps];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) *status = QLN_OK;  // the first kernel of the call clears the status word
    for (int i = tid; i < nw * count; i += kPlanWarps * 32) hist[i] = 0;
    __syncthreads();
    const int t0 = warp < nw ? (int)((int64_t)n * warp / nw) : n, t1 = warp < nw ? (int)((int64_t)n * (warp + 1) / nw) : n;
    int none = 0;  // tokens of this warp's range without an adapter
    for (int tb = t0; tb < t1; tb += 32) {
        const int t = tb + lane;
        const int a = t < t1 ? __ldg(ids + t) : 0;
        const bool in = (unsigned)a < (unsigned)count;
        if (in && t < t1) atomicAdd(&hist[warp * count + a], 1);  // a count: order plays no part
        none += __popc(__ballot_sync(0xffffffffu, !in));
    }
    if (lane == 0) s_none[warp] = none;
    __syncthreads();
    // thread a: this adapter's places within the warps' ranges, and its total
    int total = 0;
    if (tid < count)
        for (int w0 = 0; w0 < nw; w0 += 8) {
            int c[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) c[u] = w0 + u < nw ? hist[(w0 + u) * count + tid] : 0;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (w0 + u < nw) hist[(w0 + u) * count + tid] = total;
                total += c[u];
            }
        }
    // block-wide exclusive scans of the totals and of their 64-token tiles
    int v[2] = {total, (total + 63) >> 6}, inc[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        inc[q] = v[q];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, inc[q], d);
            if (lane >= d) inc[q] += x;
        }
        if (lane == 31) wsum[q][warp] = inc[q];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q)  // exclusive
        inc[q] += __reduce_add_sync(0xffffffffu, lane < warp ? wsum[q][lane] : 0) - v[q];
    // tokens without an adapter: all, and of the warps before this one
    const int nall = __reduce_add_sync(0xffffffffu, s_none[lane]);
    const int nbase = __reduce_add_sync(0xffffffffu, lane < warp ? s_none[lane] : 0);
    if (tid < count) {
        start[tid] = inc[0];
        tiles[tid] = inc[1];
        if (tid == count - 1) {
            start[count] = inc[0] + v[0];
            start[count + 1] = n;
            tiles[count] = inc[1] + v[1];
            tiles[count + 1] = inc[1] + v[1] + ((nall + 63) >> 6);
        }
        for (int w0 = 0; w0 < nw; w0 += 8) {
            int c[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) c[u] = w0 + u < nw ? hist[(w0 + u) * count + tid] : 0;
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (w0 + u < nw) hist[(w0 + u) * count + tid] = c[u] + inc[0];
        }
    }
    __syncthreads();
    int at_none = n - nall + nbase;
    for (int tb = t0; tb < t1; tb += 32) {
        const int t = tb + lane;
        const int a = t < t1 ? __ldg(ids + t) : 0;
        const bool in = t < t1 && (unsigned)a < (unsigned)count, out = t < t1 && !in;
        const uint32_t same = __match_any_sync(0xffffffffu, in ? a : -1);
        const uint32_t below = (1u << lane) - 1u, outs = __ballot_sync(0xffffffffu, out);
        if (in) order[hist[warp * count + a] + __popc(same & below)] = t;
        if (out) order[at_none + __popc(outs & below)] = t;
        at_none += __popc(outs);
        __syncwarp();
        if (in && (same & below) == 0) hist[warp * count + a] += __popc(same);
        __syncwarp();
    }
}

// Tile i of the plan: its group, its first place in order, its tokens (0: there
// is no such tile).  For a whole warp, which reads 32 entries of the tables at a
// time: one dependent read for up to 30 adapters, three at most (a bisection
// takes up to ten).
struct PlanTile {
    int a, p0, rows;
};
__device__ __forceinline__ PlanTile plan_tile(const int32_t *start, const int32_t *tiles, int count, int i) {
    const int lane = threadIdx.x & 31;
    int a, s0, s1, v0, all;
    if (count + 2 <= 32) {
        const int k = min(lane, count + 1), v = __ldg(tiles + k), s = __ldg(start + k);
        a = 31 - __clz(__ballot_sync(0xffffffffu, lane <= count && v <= i));  // the last with tiles[a] <= i
        all = __shfl_sync(0xffffffffu, v, count + 1);
        v0 = __shfl_sync(0xffffffffu, v, a);
        s0 = __shfl_sync(0xffffffffu, s, a);
        s1 = __shfl_sync(0xffffffffu, s, a + 1);
    } else {
        static_assert(QLN_MAX_ADAPTERS <= 32 * 33 - 1, "two levels");
        all = __ldg(tiles + count + 1);
        const int b = 33 * (31 - __clz(__ballot_sync(0xffffffffu, 33 * lane <= count && __ldg(tiles + min(33 * lane, count)) <= i)));
        const int k = b + 1 + lane;
        a = b + __popc(__ballot_sync(0xffffffffu, k <= count && __ldg(tiles + min(k, count)) <= i));
        v0 = __ldg(tiles + a);
        s0 = __ldg(start + a);
        s1 = __ldg(start + a + 1);
    }
    if (i >= all) return PlanTile{0, 0, 0};
    const int p0 = s0 + 64 * (i - v0);
    return PlanTile{a, p0, min(64, s1 - p0)};
}

__device__ __forceinline__ int adapter_rank(const int32_t *rank, int a, int r) {
    if (!rank) return r;
    const int k = __ldg(rank + a);
    return k < 0 ? 0 : (k > r ? r : k);
}

// ---- clusters ------------------------------------------------------------------
__device__ __forceinline__ void ad_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ad_peer_f32(uint32_t saddr, uint32_t rank) {
    uint32_t d;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(saddr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(d) : "memory");
    return v;
}

// v as a sum of three bf16 values (24 bits of mantissa, what v holds): the
// operand of the fp32 gradients.  All three have v's sign and none is zero
// unless v is (or below 2^-100, where the last ones underflow): an infinite
// element of dY or X times v is then the infinity of their product, where a zero
// part would make it NaN and parts of both signs would cancel.  So each part is
// cut off towards zero and, if that leaves nothing, lowered by one unit.  An
// infinity or NaN is all three.
__device__ __forceinline__ void split3(float v, uint16_t (&q)[3]) {
    if (!isfinite(v)) {
        q[0] = q[1] = q[2] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
        return;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        uint32_t h = __float_as_uint(v) & 0xffff0000u;
        if (k < 2 && h == __float_as_uint(v) && (h << 1) != 0u) h -= 0x10000u;
        q[k] = (uint16_t)(h >> 16);
        v = __fsub_rn(v, __uint_as_float(h));
    }
}

// ===========================================================================
// Down product: v[t][j] = sum_k in[t][k] f_a(j, k), f_a = A_a [r][K] (WKM =
// false) or B_a [K][r] (WKM = true).  A cluster of 8 or 4 CTAs owns a tile of up
// to 64 tokens of one adapter (gathered rows) x all r columns; each CTA takes
// its share of K, streamed through a 4-stage cp.async ring, 4 warps x 16 tokens;
// the partial tiles meet in shared memory and are added in the order of the
// CTAs, each CTA finishing its share of the tokens.  The activations are read
// once, each adapter once per tile, and nothing is written but the result.
// 2048 tokens x 11008 columns, rank 16, cold: 18 us, 2.6 TB/s, bound by the reads
// of gathered 128-byte pieces (neither more stages nor steps of 128 columns
// change it); 4096 tokens x 28672, rank 64: 99 us, where a tile reads as much of
// the factor, from L2, as of the tokens (5 TB/s together).
// The tensor cores' running sums move into fp32 registers every 8 chunks of 64
// (their additions truncate, and the error would grow with K).
// Results: fp32 (full), bf16(s v) for the GEMM (scaled: its product is rounded
// to bf16 anyway), and three bf16 parts for the gradients (split, planes of
// n * r); each may be null.  Zero past an adapter's rank.  Tokens without an
// adapter get zeros in full only (nothing else of them is read).  With `aux`,
// its rows (an fp32 [n][r]) are split into aux_split along the way.
// ===========================================================================
constexpr int kAdStages = 4, kAdFlush = 8, kAdCluster = 8;  // kAdCluster: at most
constexpr int kAdLd = 72;  // padded row (bf16) of the staged tiles

struct DownArgs {
    const uint16_t *in, *pool;
    int64_t n, K;
    int r, count;
    const int32_t *order, *start, *tiles, *rank;
    const float *scale;
    float *full;
    uint16_t *scaled, *split;
    const float *aux;
    uint16_t *aux_split;
};

template <int NT, bool WKM>
__global__ void __launch_bounds__(128) adapter_down_kernel(const DownArgs p) {
    extern __shared__ __align__(16) uint16_t dsm[];
    constexpr int WR = NT * 8;
    constexpr int WKLD = WR + 8;
    constexpr int STAGE = 64 * kAdLd + (WKM ? 64 * WKLD : WR * kAdLd);
    pdl_wait();
    pdl_trigger();
    const int count = p.count, r = p.r;
    const int64_t n = p.n, K = p.K;
    const PlanTile pt = plan_tile(p.start, p.tiles, count, blockIdx.x);
    const int a = pt.a, p0 = pt.p0, rows = pt.rows;
    if (rows == 0) return;  // the whole cluster
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, part = blockIdx.y;
    const int cl = gridDim.y, own = 64 / cl;  // CTAs of the cluster, rows that each finishes
    if (a == count) {  // tokens without an adapter
        if (p.full)
            for (int i = tid; i < own * r; i += 128)
                if (own * part + i / r < rows) p.full[(int64_t)__ldg(p.order + p0 + own * part + i / r) * r + i % r] = 0.f;
        return;
    }
    const uint16_t *wt = p.pool + (int64_t)a * r * K;
    const int rk = adapter_rank(p.rank, a, r);
    const float s = __ldg(p.scale + a);
    const int g = lane >> 2, c = lane & 3;
    const int nch = (int)(K / 64);
    const int ch0 = nch * part / cl, ch1 = nch * (part + 1) / cl;

    const uint16_t *src[4];  // this thread's four token rows of a stage (null: a row past the tile)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = (tid + 128 * i) >> 3;
        src[i] = row < rows ? p.in + (int64_t)__ldg(p.order + p0 + row) * K + 8 * (tid & 7) : nullptr;
    }
    float acc[NT][4], sum[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][e] = sum[nt][e] = 0.f;

    auto load = [&](int stage, int ch) {
        uint16_t *Xs = dsm + stage * STAGE;
        uint16_t *Ws = Xs + 64 * kAdLd;
        const int64_t k0 = (int64_t)ch * 64;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            cp_async16_zfill(Xs + ((tid + 128 * i) >> 3) * kAdLd + 8 * (tid & 7), src[i] ? src[i] + k0 : p.in, src[i] ? 16 : 0);
        if (WKM) {
            for (int idx = tid; idx < 64 * (WR / 8); idx += 128) {
                const int row = idx / (WR / 8), ck = idx % (WR / 8);
                const bool ok = 8 * ck < r;
                cp_async16_zfill(Ws + row * WKLD + 8 * ck, ok ? wt + (k0 + row) * (int64_t)r + 8 * ck : wt, ok ? 16 : 0);
            }
        } else {
            for (int idx = tid; idx < WR * 8; idx += 128) {
                const int row = idx >> 3, ck = idx & 7;
                const bool ok = row < r;
                cp_async16_zfill(Ws + row * kAdLd + 8 * ck, ok ? wt + (int64_t)row * K + k0 + 8 * ck : wt, ok ? 16 : 0);
            }
        }
    };
    auto flush = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sum[nt][e] = __fadd_rn(sum[nt][e], acc[nt][e]);
                acc[nt][e] = 0.f;
            }
    };
#pragma unroll
    for (int i = 0; i < kAdStages - 1; ++i) {
        if (ch0 + i < ch1) load(i, ch0 + i);
        cp_async_commit();
    }
    for (int ch = ch0; ch < ch1; ++ch) {
        const int it = ch - ch0;
        {
            const int nx = ch + kAdStages - 1;
            if (nx < ch1) load((it + kAdStages - 1) % kAdStages, nx);
            cp_async_commit();
        }
        cp_async_wait<kAdStages - 1>();
        __syncthreads();
        const uint16_t *Xs = dsm + (it % kAdStages) * STAGE;
        const uint16_t *Ws = Xs + 64 * kAdLd;
#pragma unroll
        for (int kk = 0; kk < 64; kk += 16) {
            uint32_t af[4];
            ldmatrix_x4(af[0], af[1], af[2], af[3], Xs + (16 * warp + (lane & 15)) * kAdLd + kk + (lane >> 4) * 8);
#pragma unroll
            for (int np = 0; np < NT / 2; ++np) {
                uint32_t r0, r1, r2, r3;
                if (WKM)
                    ldmatrix_x4_trans(r0, r1, r2, r3, Ws + (kk + (lane & 15)) * WKLD + np * 16 + (lane >> 4) * 8);
                else
                    ldmatrix_x4(r0, r1, r2, r3, Ws + (np * 16 + (lane & 7) + (lane >> 4) * 8) * kAdLd + kk + ((lane >> 3) & 1) * 8);
                const uint32_t b0[2] = {r0, r1}, b1[2] = {r2, r3};
                mma_bf16_16816(acc[2 * np], af, b0);
                mma_bf16_16816(acc[2 * np + 1], af, b1);
            }
            if (NT & 1) {
                uint32_t r0, r1;
                if (WKM)
                    ldmatrix_x2_trans(r0, r1, Ws + (kk + (lane & 15)) * WKLD + (NT - 1) * 8);
                else
                    ldmatrix_x2(r0, r1, Ws + ((NT - 1) * 8 + (lane & 7)) * kAdLd + kk + ((lane >> 3) & 1) * 8);
                const uint32_t b0[2] = {r0, r1};
                mma_bf16_16816(acc[NT - 1], af, b0);
            }
        }
        if (it % kAdFlush == kAdFlush - 1) flush();
        __syncthreads();
    }
    cp_async_wait<0>();
    flush();
    // this CTA's partial tile [64][WR + 4], for the cluster
    constexpr int PLD = WR + 4;
    float *part_s = reinterpret_cast<float *>(dsm);
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            *reinterpret_cast<float2 *>(part_s + (16 * warp + g + 8 * h) * PLD + 8 * nt + 2 * c) =
                make_float2(sum[nt][2 * h], sum[nt][2 * h + 1]);
    ad_cluster_sync();
    const uint32_t base = smem_u32(part_s);
    const int64_t plane = n * r;
    for (int i = tid; i < own * r; i += 128) {
        const int row = own * part + i / r, j = i % r;
        if (row >= rows) break;
        float x[kAdCluster], v = 0.f;
#pragma unroll
        for (int q = 0; q < kAdCluster; ++q) x[q] = q < cl ? ad_peer_f32(base + (uint32_t)(row * PLD + j) * 4u, q) : 0.f;
#pragma unroll
        for (int q = 0; q < kAdCluster; ++q)
            if (q < cl) v = __fadd_rn(v, x[q]);
        if (j >= rk) v = 0.f;
        const int64_t at = (int64_t)__ldg(p.order + p0 + row) * r + j;
        if (p.full) p.full[at] = v;
        if (p.scaled)  // (past the rank a zero, whatever the scale)
            p.scaled[at] = __bfloat16_as_ushort(__float2bfloat16_rn(j < rk ? __fmul_rn(s, v) : 0.f));
        uint16_t q3[3];
        if (p.split) {
            split3(v, q3);
#pragma unroll
            for (int k = 0; k < 3; ++k) p.split[k * plane + at] = q3[k];
        }
        if (p.aux_split) {
            split3(j < rk ? p.aux[at] : 0.f, q3);
#pragma unroll
            for (int k = 0; k < 3; ++k) p.aux_split[k * plane + at] = q3[k];
        }
    }
    __syncwarp();
    ad_cluster_sync();  // no CTA ends while another reads its tile
}

// ===========================================================================
// Down product of a decode-sized batch (n <= 32), without a plan: every cluster
// groups the ids by itself (one warp holds them all) and takes the x-th adapter
// present and 16 of its columns; its CTAs x 4 warps take the 64-blocks of K in
// turn, factor rows and tokens straight from global memory into MMA fragments
// (A operand: 16 factor rows; B operand: 8 tokens; both with the same
// permutation of k within a block, so each load is 16 bytes).  Latency-bound: a
// warp has all loads of two blocks in flight, and partial sums meet in shared
// memory, first of the warps, then of the CTAs, in a fixed order.  The warps add
// theirs one after the other into one tile: with under 4.5 KB a CTA fits beside
// a CTA of the GEMM, which then need not wait for this kernel to start its
// weight steps (clusters of 4 keep it to one CTA per SM).
// Cold: 6.7 us for one token x 4096 columns, 8.7 us for 32 tokens of 32 adapters.
// ===========================================================================
struct SmallArgs {
    const uint16_t *in, *A;
    int n, r, count;
    int64_t K;
    const int32_t *ids, *rank;
    const float *scale;
    float *full;       // [n][r] or null
    uint16_t *scaled;  // [n][r]
    int *status;       // cleared: this is the first kernel of its call
};

template <int NT, int CL>  // n <= 8 NT; CTAs of a cluster
__global__ void __launch_bounds__(128) adapter_down_small_kernel(const SmallArgs p) {
    constexpr int LD = 8 * NT + 2, kCols = 16 / CL;  // columns that a CTA finishes
    __shared__ float s_sum[16][LD];
    __shared__ int8_t s_tok[4][32];  // per warp: the adapter's tokens
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, part = blockIdx.z;
    if (tid == 0 && blockIdx.x == 0 && blockIdx.y == 0 && part == 0) *p.status = QLN_OK;
    const int g = lane >> 2, c = lane & 3, n = p.n, r = p.r;
    const int id = lane < n ? __ldg(p.ids + lane) : -1;
    const bool in = (unsigned)id < (unsigned)p.count;
    const uint32_t with = __ballot_sync(0xffffffffu, in), below = (1u << lane) - 1u;
    const uint32_t same = __match_any_sync(0xffffffffu, in ? id : -1) & with;
    const bool first = in && (same & below) == 0;
    const uint32_t leads = __ballot_sync(0xffffffffu, first);
    const int j0 = 16 * blockIdx.y;
    if (p.full && blockIdx.x == 0 && warp == 0 && lane < n && !in)  // tokens without an adapter
        for (int j = j0 + kCols * part; j < min(r, j0 + kCols * (part + 1)); ++j) p.full[lane * r + j] = 0.f;
    const uint32_t mine = __ballot_sync(0xffffffffu, first && __popc(leads & below) == (int)blockIdx.x);
    if (!mine) return;  // the whole cluster
    const int lead = __ffs(mine) - 1;
    const int a = __shfl_sync(0xffffffffu, id, lead);
    const uint32_t mask = __shfl_sync(0xffffffffu, same, lead);  // its tokens
    if ((mask >> lane) & 1u) s_tok[warp][__popc(mask & below)] = (int8_t)lane;
    __syncwarp();
    const int8_t *tok = s_tok[warp];
    const int rk = adapter_rank(p.rank, a, r), cnt = __popc(mask);
    if (j0 >= rk) {  // zero past the rank
        if (part == 0)
            for (int i = tid; i < 16 * cnt; i += 128) {
                const int at = tok[i / 16] * r + j0 + i % 16;
                if (j0 + i % 16 >= r) continue;
                p.scaled[at] = 0;
                if (p.full) p.full[at] = 0.f;
            }
        return;
    }
    const uint16_t *xr[NT];  // this lane's token of each tile, at its 16 columns of a block
    bool xok[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        xok[nt] = 8 * nt + g < cnt;
        xr[nt] = p.in + (xok[nt] ? (int64_t)tok[8 * nt + g] * p.K : 0) + 16 * c;
    }
    const bool ok0 = j0 + g < r, ok1 = j0 + g + 8 < r;
    const uint16_t *f0 = p.A + ((int64_t)a * r + (ok0 ? j0 + g : 0)) * p.K + 16 * c;
    const uint16_t *f1 = p.A + ((int64_t)a * r + (ok1 ? j0 + g + 8 : 0)) * p.K + 16 * c;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
    const int KB = (int)(p.K / 64);
#pragma unroll 2
    for (int b = part * 4 + warp; b < KB; b += 4 * CL) {
        const int64_t o = (int64_t)b * 64;
        uint4 fa[4], xa[NT][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            fa[h] = ok0 ? __ldg(reinterpret_cast<const uint4 *>(f0 + o) + h) : z;
            fa[2 + h] = ok1 ? __ldg(reinterpret_cast<const uint4 *>(f1 + o) + h) : z;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) xa[nt][h] = xok[nt] ? __ldg(reinterpret_cast<const uint4 *>(xr[nt] + o) + h) : z;
        }
#pragma unroll
        for (int st = 0; st < 4; ++st) {  // k pairs 16c + 4 st + {0, 1} and {2, 3}
            const uint4 u0 = fa[st >> 1], u1 = fa[2 + (st >> 1)];
            const uint32_t av[4] = {st & 1 ? u0.z : u0.x, st & 1 ? u1.z : u1.x, st & 1 ? u0.w : u0.y, st & 1 ? u1.w : u1.y};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint4 x = xa[nt][st >> 1];
                const uint32_t bv[2] = {st & 1 ? x.z : x.x, st & 1 ? x.w : x.y};
                mma_bf16_16816(acc[nt], av, bv);
            }
        }
    }
#pragma unroll 1
    for (int w = 0; w < 4; ++w) {  // the warps' sums, in their order
        if (warp == w) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float2 *at = reinterpret_cast<float2 *>(&s_sum[g + 8 * h][8 * nt + 2 * c]);
                    float2 v = w ? *at : make_float2(0.f, 0.f);
                    v.x = __fadd_rn(v.x, acc[nt][2 * h]);
                    v.y = __fadd_rn(v.y, acc[nt][2 * h + 1]);
                    *at = v;
                }
        }
        __syncthreads();
    }
    ad_cluster_sync();
    const float s = __ldg(p.scale + a);
    const uint32_t base = smem_u32(&s_sum[0][0]);
    for (int i = tid; i < kCols * cnt; i += 128) {
        const int j = kCols * part + i % kCols, k = i / kCols;
        float x[CL], v = 0.f;
#pragma unroll
        for (int q = 0; q < CL; ++q) x[q] = ad_peer_f32(base + (uint32_t)(j * LD + k) * 4u, q);
#pragma unroll
        for (int q = 0; q < CL; ++q) v = __fadd_rn(v, x[q]);
        if (j0 + j >= r) continue;
        const bool in_rank = j0 + j < rk;  // past it zeros, whatever the scale
        const int at = tok[k] * r + j0 + j;
        if (p.full) p.full[at] = in_rank ? v : 0.f;
        p.scaled[at] = __bfloat16_as_ushort(__float2bfloat16_rn(in_rank ? __fmul_rn(s, v) : 0.f));
    }
    __syncwarp();
    ad_cluster_sync();  // no CTA ends while another reads its sums
}

// ---- host --------------------------------------------------------------------
static size_t r256(size_t x) { return (x + 255) & ~size_t(255); }

static size_t plan_table() { return r256((QLN_MAX_ADAPTERS + 2) * 4); }

size_t adapter_plan_bytes(int64_t n) { return r256((size_t)n * 4) + 2 * plan_table(); }

AdapterPlan adapter_plan_at(void *base, int64_t n) {
    char *b = static_cast<char *>(base);
    AdapterPlan p;
    p.order = reinterpret_cast<int32_t *>(b);
    p.start = reinterpret_cast<int32_t *>(b + r256((size_t)n * 4));
    p.tiles = reinterpret_cast<int32_t *>(b + r256((size_t)n * 4) + plan_table());
    return p;
}

cudaError_t launch_adapter_plan(const int32_t *ids, int64_t n, int count, const AdapterPlan &p, int *status, cudaStream_t st) {
    const int nw = plan_ranges(n);
    const size_t smem = (size_t)nw * count * sizeof(int);
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(adapter_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(adapter_plan_kernel, dim3(1), dim3(kPlanWarps * 32), smem, st, ids, (int)n, count, nw, p.order, p.start,
                      p.tiles, status);
}

// launch_pdl with a thread-block cluster.
template <typename Args>
static cudaError_t launch_cluster(void (*kernel)(const Args), dim3 grid, dim3 cluster, size_t smem, cudaStream_t st,
                                  const Args &args) {
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster.x;
    attr[0].val.clusterDim.y = cluster.y;
    attr[0].val.clusterDim.z = cluster.z;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    note_launch();
    return cudaLaunchKernelEx(&cfg, kernel, args);
}

template <int NT, bool WKM>
static cudaError_t launch_ad_down(const DownArgs &a, cudaStream_t st, int num_sms) {
    constexpr size_t smem = (size_t)kAdStages * (64 * kAdLd + (WKM ? 64 * (NT * 8 + 8) : NT * 8 * kAdLd)) * sizeof(uint16_t);
    static_assert(smem >= 64 * (NT * 8 + 4) * 4, "the partial tile fits into the ring");
    // every group's last tile may be partial: at most n / 64 whole tiles and one more per group present
    const int64_t tiles = a.n / 64 + (a.count + 1 < a.n ? a.count + 1 : a.n);
    // Eight CTAs per tile while all fit at once, for the shortest chain (4096 columns, 100 tokens of 8 adapters: 27.3 us
    // for the whole call, 29.4 us with four), else four (28672 columns, rank 64, 4096 tokens: 99 us against 115).
    const int64_t slots = num_sms * ((int64_t)(228 * 1024) / (int64_t)(smem + 1024));
    const unsigned cl = tiles * kAdCluster <= slots ? kAdCluster : kAdCluster / 2;
    return launch_cluster(adapter_down_kernel<NT, WKM>, dim3((unsigned)tiles, cl), dim3(1, cl), smem, st, a);
}

cudaError_t launch_adapter_down(const uint16_t *in, int64_t n, int64_t K, const qln_adapter_pool *pool, bool kmajor,
                                const AdapterPlan &p, float *full, uint16_t *scaled, uint16_t *split, const float *aux,
                                uint16_t *aux_split, cudaStream_t st, int num_sms) {
    const DownArgs a{in, kmajor ? pool->B : pool->A, n, K, pool->r, pool->count, p.order, p.start, p.tiles, pool->rank,
                     pool->scale, full, scaled, split, aux, aux_split};
#define QLN_AD_DOWN(NT) (kmajor ? launch_ad_down<NT, true>(a, st, num_sms) : launch_ad_down<NT, false>(a, st, num_sms))
    if (a.r <= 8) return QLN_AD_DOWN(1);
    if (a.r <= 16) return QLN_AD_DOWN(2);
    if (a.r <= 32) return QLN_AD_DOWN(4);
    if (a.r <= 64) return QLN_AD_DOWN(8);
    return QLN_AD_DOWN(16);
#undef QLN_AD_DOWN
}

cudaError_t launch_adapter_down_small(const uint16_t *in, int64_t n, int64_t K, const qln_adapter_pool *pool,
                                      const int32_t *ids, float *full, uint16_t *scaled, int *status, cudaStream_t st,
                                      int num_sms) {
    const SmallArgs a{in, pool->A, (int)n, pool->r, pool->count, K, ids, pool->rank, pool->scale, full, scaled, status};
    const unsigned groups = (unsigned)(n < pool->count ? n : pool->count), jt = (unsigned)((pool->r + 15) / 16);
    // Clusters of 8 for the shortest chain; of 4 where those would put two CTAs on an SM (whole calls of 4096 x 4096, 8 / 4:
    // one token 12.6 / 13.2 us; 32 tokens of 32 adapters, rank 16: 25.9 / 22.7 us, rank 64: 41 / 38 us).
    const bool eight = groups * jt * 8 <= (unsigned)num_sms;
#define QLN_AD_SMALL(NT) \
    (eight ? launch_cluster(adapter_down_small_kernel<NT, 8>, dim3(groups, jt, 8), dim3(1, 1, 8), 0, st, a) \
           : launch_cluster(adapter_down_small_kernel<NT, 4>, dim3(groups, jt, 4), dim3(1, 1, 4), 0, st, a))
    switch ((n + 7) / 8) {
        case 1: return QLN_AD_SMALL(1);
        case 2: return QLN_AD_SMALL(2);
        case 3: return QLN_AD_SMALL(3);
        default: return QLN_AD_SMALL(4);
    }
#undef QLN_AD_SMALL
}

}  // namespace qln

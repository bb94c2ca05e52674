// Products around a pool of adapters, where every token has an adapter of its
// own (or none): the plan that groups tokens by adapter, the products down to
// the rank, and the gradients of the factors.
//
// Method: "LoRA 与 QLoRA" section LoRA (y = W0 x + s B(A x), A x formed first;
// only A and B are trained); deck "3 QLoRA Finetuning" card 1 (gradients flow
// through the dequantized weight, only the adapters receive updates).  For
// token t with adapter a = ids[t]:
//   U_t = X_t A_a^T                    (forward)
//   G_t = dY_t B_a                     (backward)
//   dA_a = s_a sum_{t: ids[t] = a} G_t^T X_t,  dB_a = s_a sum dY_t^T U_t
// Tokens are never multiplied with another adapter's factors, not even by a
// zero: an infinity or NaN in one adapter or token stays with it.
#include "qln_common.cuh"
#include "qln_internal.h"

namespace qln {

// ===========================================================================
// Plan: a stable counting sort of the tokens by adapter, in one CTA.
//   order [n]         tokens of adapter 0, then 1, ... (ascending within one)
//   start [count + 1] first place of each adapter in order
//   tiles [count + 1] first 64-token tile of each adapter (tiles never mix)
// Warp w owns the w-th of 32 contiguous token ranges and a histogram of its
// own, so places follow from two passes over the ids and one scan, and do not
// depend on timing.  Latency-bound: a few dependent reads of the ids.
// ===========================================================================
constexpr int kPlanWarps = 32;

__global__ void __launch_bounds__(kPlanWarps * 32) adapter_plan_kernel(const int32_t *__restrict__ ids, int n, int count,
                                                                       int32_t *__restrict__ order,
                                                                       int32_t *__restrict__ start,
                                                                       int32_t *__restrict__ tiles, int *status) {
    extern __shared__ int hist[];  // [warp][count]
    __shared__ int wsum[2][kPlanWarps];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) *status = QLN_OK;  // the first kernel of the call clears the status word
    for (int i = tid; i < kPlanWarps * count; i += kPlanWarps * 32) hist[i] = 0;
    __syncthreads();
    const int t0 = (int)((int64_t)n * warp / kPlanWarps), t1 = (int)((int64_t)n * (warp + 1) / kPlanWarps);
    for (int t = t0 + lane; t < t1; t += 32) {
        const int a = __ldg(ids + t);
        if ((unsigned)a < (unsigned)count) atomicAdd(&hist[warp * count + a], 1);  // a count: order plays no part
    }
    __syncthreads();
    // thread a: this adapter's places within the warps' ranges, and its total
    int total = 0;
    if (tid < count)
        for (int w = 0; w < kPlanWarps; ++w) {
            const int c = hist[w * count + tid];
            hist[w * count + tid] = total;
            total += c;
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
    for (int q = 0; q < 2; ++q) {
        int base = 0;
        for (int w = 0; w < warp; ++w) base += wsum[q][w];
        inc[q] += base - v[q];  // exclusive
    }
    if (tid < count) {
        start[tid] = inc[0];
        tiles[tid] = inc[1];
        if (tid == count - 1) {
            start[count] = inc[0] + v[0];
            tiles[count] = inc[1] + v[1];
        }
        for (int w = 0; w < kPlanWarps; ++w) hist[w * count + tid] += inc[0];
    }
    __syncthreads();
    for (int tb = t0; tb < t1; tb += 32) {
        const int t = tb + lane;
        const int a = t < t1 ? __ldg(ids + t) : -1;
        const bool in = (unsigned)a < (unsigned)count;
        const uint32_t same = __match_any_sync(0xffffffffu, in ? a : -1);
        const int before = __popc(same & ((1u << lane) - 1u));
        if (in) order[hist[warp * count + a] + before] = t;
        __syncwarp();
        if (in && before == 0) hist[warp * count + a] += __popc(same);
        __syncwarp();
    }
}

// The adapter whose tiles hold tile i: tiles[a] <= i < tiles[a + 1].
__device__ __forceinline__ int tile_adapter(const int32_t *tiles, int count, int i) {
    int lo = 0, hi = count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(tiles + mid) <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int adapter_rank(const int32_t *rank, int a, int r) {
    if (!rank) return r;
    const int k = __ldg(rank + a);
    return k < 0 ? 0 : (k > r ? r : k);
}

// ===========================================================================
// Down product: partial[split][t][j] = sum over a K range of in[t][k] f_a(j, k),
// f_a = A_a [r][K] (WKM = false) or B_a [K][r] (WKM = true).  A CTA owns a tile
// of up to 64 tokens of one adapter (gathered rows) x all r columns x one of
// the K ranges, streamed through a 4-stage cp.async ring; 4 warps x 16 tokens.
// HBM-bound: the activations are read once, each adapter once per tile.
// ===========================================================================
constexpr int kAdStages = 4;
constexpr int kAdLd = 72;  // padded row (bf16) of the staged tiles

template <int NT, bool WKM>
__global__ void __launch_bounds__(128) adapter_down_kernel(const uint16_t *__restrict__ in, int64_t n, int64_t K,
                                                           const uint16_t *__restrict__ pool, int r, int count, int cps,
                                                           const int32_t *__restrict__ order,
                                                           const int32_t *__restrict__ start,
                                                           const int32_t *__restrict__ tiles,
                                                           float *__restrict__ partial) {
    extern __shared__ __align__(16) uint16_t dsm[];
    constexpr int WR = NT * 8;
    constexpr int WKLD = WR + 8;
    constexpr int STAGE = 64 * kAdLd + (WKM ? 64 * WKLD : WR * kAdLd);
    pdl_wait();
    pdl_trigger();
    const int tile = blockIdx.x;
    if (tile >= __ldg(tiles + count)) return;
    const int a = tile_adapter(tiles, count, tile);
    const int p0 = __ldg(start + a) + 64 * (tile - __ldg(tiles + a));
    const int rows = min(64, __ldg(start + a + 1) - p0);
    const uint16_t *wt = pool + (int64_t)a * r * K;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int split = blockIdx.y;
    const int64_t nch = K / 64;
    const int64_t ch0 = (int64_t)split * cps;
    const int64_t ch1 = ch0 + cps < nch ? ch0 + cps : nch;

    const uint16_t *src[4];  // this thread's four token rows of a stage (null: a row past the tile)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = (tid + 128 * i) >> 3;
        src[i] = row < rows ? in + (int64_t)__ldg(order + p0 + row) * K + 8 * (tid & 7) : nullptr;
    }
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;

    auto load = [&](int stage, int64_t ch) {
        uint16_t *Xs = dsm + stage * STAGE;
        uint16_t *Ws = Xs + 64 * kAdLd;
        const int64_t k0 = ch * 64;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            cp_async16_zfill(Xs + ((tid + 128 * i) >> 3) * kAdLd + 8 * (tid & 7), src[i] ? src[i] + k0 : in, src[i] ? 16 : 0);
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
#pragma unroll
    for (int i = 0; i < kAdStages - 1; ++i) {
        if (ch0 + i < ch1) load(i, ch0 + i);
        cp_async_commit();
    }
    for (int64_t ch = ch0; ch < ch1; ++ch) {
        const int it = (int)(ch - ch0);
        {
            const int64_t nx = ch + kAdStages - 1;
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
        __syncthreads();
    }
    cp_async_wait<0>();
    float *dst = partial + (int64_t)split * n * r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = 16 * warp + g + 8 * h;
        if (row >= rows) continue;
        const int64_t t = __ldg(order + p0 + row);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int j = 8 * nt + 2 * c;
            if (j < r) *reinterpret_cast<float2 *>(dst + t * r + j) = make_float2(acc[nt][2 * h], acc[nt][2 * h + 1]);
        }
    }
}

// Sum of the K splits in their order, for token t and column j; zero for a
// token without an adapter and a column past its adapter's rank.  Written as
// fp32 (full), as bf16(s v) for the tensor cores (scaled: the operand of a
// product whose result is rounded to bf16 anyway), and as the pair hi + lo of
// bf16 values that holds v to 2^-17 (the operand of the fp32 gradients); any
// of them may be null.
__global__ void adapter_fold_kernel(const float *__restrict__ partial, int splits, int64_t n, int r,
                                    const int32_t *__restrict__ ids, int count, const int32_t *__restrict__ rank,
                                    const float *__restrict__ scale, float *__restrict__ full,
                                    uint16_t *__restrict__ scaled, uint16_t *__restrict__ hi, uint16_t *__restrict__ lo) {
    pdl_wait();
    pdl_trigger();
    const int64_t total = n * r, stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += stride) {
        const int64_t t = i / r;
        const int j = (int)(i - t * r), a = __ldg(ids + t);
        float v = 0.f, s = 0.f;
        if ((unsigned)a < (unsigned)count && j < adapter_rank(rank, a, r)) {
            for (int z0 = 0; z0 < splits; z0 += 8) {  // eight loads ahead of their adds
                float x[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) x[u] = z0 + u < splits ? __ldcg(partial + (int64_t)(z0 + u) * total + i) : 0.f;
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (z0 + u < splits) v = __fadd_rn(v, x[u]);
            }
            s = __ldg(scale + a);
        }
        if (full) full[i] = v;
        if (scaled) scaled[i] = __bfloat16_as_ushort(__float2bfloat16_rn(__fmul_rn(s, v)));
        if (hi) {
            const __nv_bfloat16 h = __float2bfloat16_rn(v);
            const float rest = __fsub_rn(v, __bfloat162float(h));
            hi[i] = __bfloat16_as_ushort(h);
            lo[i] = __bfloat16_as_ushort(__float2bfloat16_rn(isfinite(rest) ? rest : 0.f));  // inf - inf
        }
    }
}

// ===========================================================================
// Gradients of the factors: C[m][j] = s_a sum_{t of a} P[t][m] Q[t][j], P = dY
// and Q = U (dB_a [dout][r]), or P = X and Q = G (dA_a, stored transposed,
// [r][din]).  A CTA owns 128 m x up to 64 j of one adapter over all of its
// tokens (gathered rows, steps of 32, 4-stage ring): no splits and no partial
// sums in memory, one order of every sum.  Q enters as hi + lo, two MMAs each,
// so that the fp32 result is good to fp32-like accuracy (2^-17 per factor); the
// tensor cores' running sums are moved into fp32 registers every 512 tokens,
// so that their truncation does not grow with the sequence.  Adapters without
// tokens get zeros, and so do columns past an adapter's rank.
// ===========================================================================
constexpr int kAgBM = 128, kAgBK = 32, kAgPad = 136, kAgStages = 4, kAgFlush = 16;

struct GradArgs {
    const uint16_t *P[2], *Qhi[2], *Qlo[2];  // 0: dB, 1: dA
    int64_t M[2];
    float *C[2];
    const int32_t *order, *start, *rank;
    const float *scale;
    int r, tilesB;
};

template <int NTJ>  // 8 NTJ columns
__global__ void __launch_bounds__(128) adapter_grad_kernel(const GradArgs p) {
    extern __shared__ __align__(16) uint16_t sk[];
    constexpr int QW = NTJ * 8, QLD = QW + 8;
    constexpr int STAGE = kAgBK * (kAgPad + 2 * QLD);
    pdl_wait();
    pdl_trigger();
    const int which = (int)blockIdx.x < p.tilesB ? 0 : 1;
    const int a = blockIdx.y, j0 = blockIdx.z * QW, r = p.r;
    const int64_t M = p.M[which], m0 = (int64_t)((int)blockIdx.x - (which ? p.tilesB : 0)) * kAgBM;
    const uint16_t *P = p.P[which], *Qh = p.Qhi[which], *Ql = p.Qlo[which];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3, mat = lane >> 3;
    const int p0 = __ldg(p.start + a), cnt = __ldg(p.start + a + 1) - p0;
    const int steps = (cnt + kAgBK - 1) / kAgBK;

    float acc[2][NTJ][4], sum[2][NTJ][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NTJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = sum[i][j][e] = 0.f;

    auto load = [&](int buf, int step) {
        uint16_t *Ps = sk + buf * STAGE, *Hs = Ps + kAgBK * kAgPad, *Ls = Hs + kAgBK * QLD;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // P: 32 rows x 16 chunks
            const int idx = tid + 128 * i, row = idx >> 4, ck = idx & 15, q = step * kAgBK + row;
            const int64_t col = m0 + 8 * ck;
            const bool ok = q < cnt && col < M;
            cp_async16_zfill(Ps + row * kAgPad + 8 * ck, ok ? P + (int64_t)__ldg(p.order + p0 + q) * M + col : P, ok ? 16 : 0);
        }
        for (int idx = tid; idx < 2 * kAgBK * NTJ; idx += 128) {  // Q: 32 rows x NTJ chunks, hi then lo
            const int h = idx >= kAgBK * NTJ, k = idx - h * kAgBK * NTJ, row = k / NTJ, ck = k % NTJ, q = step * kAgBK + row;
            const bool ok = q < cnt && j0 + 8 * ck < r;
            const uint16_t *Q = h ? Ql : Qh;
            cp_async16_zfill((h ? Ls : Hs) + row * QLD + 8 * ck,
                             ok ? Q + (int64_t)__ldg(p.order + p0 + q) * r + j0 + 8 * ck : Q, ok ? 16 : 0);
        }
    };
#pragma unroll
    for (int i = 0; i < kAgStages - 1; ++i) {
        if (i < steps) load(i, i);
        cp_async_commit();
    }
    for (int it = 0; it < steps; ++it) {
        if (it + kAgStages - 1 < steps) load((it + kAgStages - 1) % kAgStages, it + kAgStages - 1);
        cp_async_commit();
        cp_async_wait<kAgStages - 1>();
        __syncthreads();
        const uint16_t *Ps = sk + (it % kAgStages) * STAGE, *Hs = Ps + kAgBK * kAgPad;
#pragma unroll
        for (int kk = 0; kk < kAgBK; kk += 16) {
            uint32_t af[2][4];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
                ldmatrix_x4_trans(af[mt][0], af[mt][1], af[mt][2], af[mt][3],
                                  Ps + (kk + (mat >> 1) * 8 + (lane & 7)) * kAgPad + warp * 32 + mt * 16 + (mat & 1) * 8);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint16_t *Qs = Hs + h * kAgBK * QLD + (kk + (mat & 1) * 8 + (lane & 7)) * QLD;
#pragma unroll
                for (int np = 0; np < NTJ / 2; ++np) {
                    uint32_t r0, r1, r2, r3;
                    ldmatrix_x4_trans(r0, r1, r2, r3, Qs + np * 16 + (mat >> 1) * 8);
                    const uint32_t b0[2] = {r0, r1}, b1[2] = {r2, r3};
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        mma_bf16_16816(acc[mt][2 * np], af[mt], b0);
                        mma_bf16_16816(acc[mt][2 * np + 1], af[mt], b1);
                    }
                }
                if (NTJ & 1) {
                    uint32_t r0, r1;
                    ldmatrix_x2_trans(r0, r1, Qs + (NTJ - 1) * 8);
                    const uint32_t b0[2] = {r0, r1};
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) mma_bf16_16816(acc[mt][NTJ - 1], af[mt], b0);
                }
            }
        }
        if (it % kAgFlush == kAgFlush - 1) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < NTJ; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sum[i][j][e] = __fadd_rn(sum[i][j][e], acc[i][j][e]);
                        acc[i][j][e] = 0.f;
                    }
        }
        __syncthreads();
    }
    cp_async_wait<0>();
    const int rk = adapter_rank(p.rank, a, r);
    const float s = __ldg(p.scale + a);
    float *C = p.C[which] + (int64_t)a * M * r;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < NTJ; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t m = m0 + warp * 32 + mt * 16 + g + 8 * (e >> 1);
                const int j = j0 + nt * 8 + 2 * c + (e & 1);
                if (m < M && j < r) {
                    const float v = cnt > 0 && j < rk ? __fmul_rn(s, __fadd_rn(sum[mt][nt][e], acc[mt][nt][e])) : 0.f;
                    C[which ? (int64_t)j * M + m : m * r + j] = v;
                }
            }
}

// ---- host --------------------------------------------------------------------
static size_t r256(size_t x) { return (x + 255) & ~size_t(255); }

size_t adapter_plan_bytes(int64_t n) { return r256((size_t)n * 4) + 2 * r256((QLN_MAX_ADAPTERS + 1) * 4); }

AdapterPlan adapter_plan_at(void *base, int64_t n) {
    char *b = static_cast<char *>(base);
    AdapterPlan p;
    p.order = reinterpret_cast<int32_t *>(b);
    p.start = reinterpret_cast<int32_t *>(b + r256((size_t)n * 4));
    p.tiles = reinterpret_cast<int32_t *>(b + r256((size_t)n * 4) + r256((QLN_MAX_ADAPTERS + 1) * 4));
    return p;
}

cudaError_t launch_adapter_plan(const int32_t *ids, int64_t n, int count, const AdapterPlan &p, int *status, cudaStream_t st) {
    const size_t smem = (size_t)kPlanWarps * count * sizeof(int);
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(adapter_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(adapter_plan_kernel, dim3(1), dim3(kPlanWarps * 32), smem, st, ids, (int)n, count, p.order, p.start,
                      p.tiles, status);
}

template <int NT, bool WKM>
static cudaError_t launch_ad_down(const uint16_t *in, int64_t n, int64_t K, const uint16_t *pool, int r, int count,
                                  const AdapterPlan &p, int splits, int cps, float *partial, cudaStream_t st) {
    constexpr size_t smem = (size_t)kAdStages * (64 * kAdLd + (WKM ? 64 * (NT * 8 + 8) : NT * 8 * kAdLd)) * sizeof(uint16_t);
    auto kern = adapter_down_kernel<NT, WKM>;
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    // every adapter's last tile may be partial: at most n / 64 whole tiles and one more per adapter present
    const int64_t tiles = n / 64 + (count < n ? count : n);
    return launch_pdl(kern, dim3((unsigned)tiles, (unsigned)splits), dim3(128), smem, st, in, n, K, pool, r, count, cps,
                      (const int32_t *)p.order, (const int32_t *)p.start, (const int32_t *)p.tiles, partial);
}

cudaError_t launch_adapter_down(const uint16_t *in, int64_t n, int64_t K, const uint16_t *pool, bool kmajor, int r,
                                int count, const AdapterPlan &p, float *partial, int splits, int cps, cudaStream_t st) {
#define QLN_AD_DOWN(NT) \
    (kmajor ? launch_ad_down<NT, true>(in, n, K, pool, r, count, p, splits, cps, partial, st) \
            : launch_ad_down<NT, false>(in, n, K, pool, r, count, p, splits, cps, partial, st))
    if (r <= 8) return QLN_AD_DOWN(1);
    if (r <= 16) return QLN_AD_DOWN(2);
    if (r <= 32) return QLN_AD_DOWN(4);
    if (r <= 64) return QLN_AD_DOWN(8);
    return QLN_AD_DOWN(16);
#undef QLN_AD_DOWN
}

cudaError_t launch_adapter_fold(const float *partial, int splits, int64_t n, const qln_adapter_pool *pool,
                                const int32_t *ids, float *full, uint16_t *scaled, uint16_t *hi, uint16_t *lo, cudaStream_t st) {
    int64_t blocks = (n * pool->r + 255) / 256;
    if (blocks > 2048) blocks = 2048;
    return launch_pdl(adapter_fold_kernel, dim3((unsigned)blocks), dim3(256), 0, st, partial, splits, n, (int)pool->r, ids,
                      (int)pool->count, pool->rank, pool->scale, full, scaled, hi, lo);
}

template <int NTJ>
static cudaError_t launch_ad_grad(const GradArgs &a, int count, cudaStream_t st) {
    constexpr size_t smem = (size_t)kAgStages * kAgBK * (kAgPad + 2 * (NTJ * 8 + 8)) * sizeof(uint16_t);
    auto kern = adapter_grad_kernel<NTJ>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const unsigned tilesA = (unsigned)((a.M[1] + kAgBM - 1) / kAgBM);
    return launch_pdl(kern, dim3((unsigned)a.tilesB + tilesA, (unsigned)count, (unsigned)((a.r + 8 * NTJ - 1) / (8 * NTJ))),
                      dim3(128), smem, st, a);
}

cudaError_t launch_adapter_grads(const uint16_t *dY, const uint16_t *Uhi, const uint16_t *Ulo, int64_t dout,
                                 const uint16_t *X, const uint16_t *Ghi, const uint16_t *Glo, int64_t din,
                                 const qln_adapter_pool *pool, const AdapterPlan &p, float *dA, float *dB, cudaStream_t st) {
    GradArgs a;
    a.P[0] = dY, a.P[1] = X;
    a.Qhi[0] = Uhi, a.Qhi[1] = Ghi;
    a.Qlo[0] = Ulo, a.Qlo[1] = Glo;
    a.M[0] = dout, a.M[1] = din;
    a.C[0] = dB, a.C[1] = dA;
    a.order = p.order, a.start = p.start, a.rank = pool->rank;
    a.scale = pool->scale;
    a.r = pool->r;
    a.tilesB = (int)((dout + kAgBM - 1) / kAgBM);
    if (a.r <= 8) return launch_ad_grad<1>(a, pool->count, st);
    if (a.r <= 16) return launch_ad_grad<2>(a, pool->count, st);
    if (a.r <= 32) return launch_ad_grad<4>(a, pool->count, st);
    return launch_ad_grad<8>(a, pool->count, st);
}

}  // namespace qln
